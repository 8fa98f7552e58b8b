"""Host rules of the mixture of experts, read from the workspace they ask for:
h of every pair, then the down products' sums in parts of their K split (none
where one launch makes the sums)."""
import random

import pytest

import weight_only_bit_q4_amd as q


def al256(v):
    return (v + 255) // 256 * 256


def parts(inner, k, experts, top_k, t):
    """(parts of the down products' sums, bytes that are neither h nor those)."""
    pairs = t * top_k
    sums = q.q4lin_moe_workspace_bytes(inner, k, experts, top_k, t) - al256(pairs * inner * 4)
    return sums // (pairs * k * 4), sums - al256(sums // (pairs * k * 4) * pairs * k * 4)


def check(inner, k, experts, top_k, t):
    n, rest = parts(inner, k, experts, top_k, t)
    # a share of K is one or more quads of 128-k stages
    assert rest == 0 and 1 <= n <= max(1, -(-inner // 512)), (inner, k, experts, top_k, t, n, rest)


@pytest.mark.parametrize("inner,k,experts,top_k,t", [(960, 2048, 7, 7, 12), (448, 1920, 8, 4, 30), (64, 5120, 4, 4, 9),
                                                     (512, 512, 2, 2, 20), (513 * 64, 1024, 3, 1, 50)])
def test_down_products_have_no_empty_share(inner, k, experts, top_k, t):
    check(inner, k, experts, top_k, t)


def test_down_products_have_no_empty_share_drawn():
    rng = random.Random(5)
    for _ in range(3000):
        experts = rng.randint(1, 128)
        check(64 * rng.randint(1, 60), 64 * rng.randint(8, 90), experts, rng.randint(1, min(experts, 8)),
              rng.randint(9, 200))  # more tokens than one launch takes


# sizes at which each form was measured the faster one
@pytest.mark.parametrize("inner,k,experts,top_k,t,one", [
    (3904, 1088, 24, 9, 1, True), (2816, 2048, 64, 16, 1, True), (5120, 640, 40, 20, 1, False),
    (4096, 2048, 32, 16, 1, False), (1792, 2048, 64, 8, 2, True), (704, 1984, 60, 4, 7, True),
    (3904, 1088, 24, 3, 3, False), (2048, 1024, 32, 2, 8, False), (1088, 2048, 64, 4, 8, False)])
def test_down_products_in_one_launch_where_that_is_faster(inner, k, experts, top_k, t, one):
    after_h = q.q4lin_moe_workspace_bytes(inner, k, experts, top_k, t) - al256(t * top_k * inner * 4)
    # (where one launch makes the sums, only a few tokens' logits lie behind h)
    assert (after_h == al256(t * experts * 8)) if one else (after_h >= t * top_k * k * 4)
