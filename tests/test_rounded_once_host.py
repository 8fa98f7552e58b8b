"""rounded_once tells results whose rank values (adapters) or gated values
(experts) kept 16 significant bits from those that kept 8: the mistake is
planted in the 64-bit references."""
import pytest
import torch

import token_weights as tw
from rounded_once import LIMIT, error_ratio, rounded_once


def one_part(v):
    return v.float().bfloat16().double()


def two_parts(v):
    hi = one_part(v)
    return hi + one_part(v - hi)


def adapters(n, k, t, count, rank, keep, size=1.0):
    planes, w64 = tw.weight(0, n, k, 6000)
    x = tw.bf16((t, k), 6001).double()
    a = tw.bf16((count, rank, k), 6002, k ** -0.5).double()
    b = tw.bf16((count, n, rank), 6003, size * float(w64.std()) * (k / rank) ** 0.5).double()
    base = x @ w64.t()
    want, got = base.clone(), base.clone()
    for i in range(t):
        u = a[i % count] @ x[i]
        want[i] += b[i % count] @ u
        got[i] += b[i % count] @ keep(u)
    return got.float().bfloat16(), want


def experts(inner, k, t, count, keep):
    _, (gate, up, down) = tw.expert_weights(count, inner, k, 6100)
    x = tw.bf16((t, k), 6101).double()
    want = torch.zeros(t, k, dtype=torch.float64)
    got = want.clone()
    for i in range(t):
        for e, w in ((i % count, 0.6), ((i + 1) % count, 0.4)):
            g, u = gate[e] @ x[i], up[e] @ x[i]
            h = g * torch.sigmoid(g) * u
            want[i] += w * (down[e] @ h)
            got[i] += w * (down[e] @ keep(h))
    return got.float().bfloat16(), want


SHAPES = [(500, 512, 5, 3, 16), (200, 256, 40, 4, 64), (300, 1024, 12, 2, 136)]


@pytest.mark.parametrize("n,k,t,count,rank", SHAPES)
def test_rank_values(n, k, t, count, rank):
    rounded_once(*adapters(n, k, t, count, rank, two_parts), "two parts")
    assert error_ratio(*adapters(n, k, t, count, rank, one_part)) > LIMIT  # half of the variance
    assert error_ratio(*adapters(n, k, t, count, rank, one_part, 4.0)) > 1.2 * LIMIT


@pytest.mark.parametrize("inner,k,t,count", [(512, 1024, 1, 2), (256, 320, 12, 4), (64, 192, 30, 3)])
def test_gated_values(inner, k, t, count):
    rounded_once(*experts(inner, k, t, count, two_parts), "two parts")
    assert error_ratio(*experts(inner, k, t, count, one_part)) > 1.2 * LIMIT
