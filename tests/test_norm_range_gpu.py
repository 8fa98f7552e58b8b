"""The norm into 8 bits of rows of any magnitude that bf16 holds, against the formula in 64 bits, within a bound that
counts every rounding of binary32."""
import pytest
import torch

import mx8
import weight_only_bit_q4_amd as q4
from gpu_util import announce

pytestmark = pytest.mark.gpu

# Relative error of y = v rstd weight before its rounding to 8 bits, each 2^-24: v is rounded (without a residual it is
# not), which its squares carry into the mean at most once more (half of twice); the mean and its root are binary64; the
# root's reciprocal is rounded, and so are two products (one without a weight).  Powers of two change nothing.  Second
# order and binary64: less than a hundredth of one.
ROUNDING = 1.01 * 2.0 ** -24


def bound(residual, weight):
    return (2 + (2 if residual else 0) + (1 if weight else 0)) * ROUNDING


def rows(t, k, seed):
    return torch.randn(t, k, generator=torch.Generator().manual_seed(seed))


# (bf16 from its subnormals, 9.2e-41 the least of them, to its end; every way the kernel holds a row)
SIZES = [1.0, 1e-30, 1e-36, 1e-37, 3e-38, 6e-39, 3e-39, 1.1e-39, 3e-40, 1e-40, 1e20, 1e30, 1e37, 3e37]


@pytest.mark.parametrize("k", [64, 256, 5120, 16384, 40000])
@pytest.mark.parametrize("form", ["plain", "residual", "weight", "both"])
def test_rows_of_any_magnitude(k, form):
    residual, weight = form in ("residual", "both"), form in ("weight", "both")
    scale = torch.tensor(SIZES, dtype=torch.float64)[:, None]
    x = (rows(len(SIZES), k, k).double() * scale).to(torch.bfloat16)
    r = (rows(len(SIZES), k, k + 1).double() * scale).to(torch.bfloat16) if residual else None
    w = (rows(1, k, k + 2)[0] * 0.3 + 1).to(torch.bfloat16) if weight else None
    announce("rmsnorm_mx8 of rows of any magnitude, k=%d %s" % (k, form))
    out = [v.cpu() for v in q4.rmsnorm_mx8(x.cuda(), w.cuda() if weight else None, 0.0,
                                           residual=r.cuda() if residual else None)]
    v = x.double() + (r.double() if residual else 0)
    y = v / torch.sqrt(v.square().mean(-1, keepdim=True)) * (w.double() if weight else 1)
    mx8.check_mx8(out[0], out[1], y, bound(residual, weight), "norm of rows of any magnitude")
    if residual:
        assert torch.equal(out[2], v.float().to(torch.bfloat16))


@pytest.mark.parametrize("k", [64, 8192, 1 << 17])
def test_one_least_value_in_a_row(k):
    """A row of zeros but for the least bf16 there is, and one with the largest: sqrt(K) in one place."""
    x = torch.zeros(2, k, dtype=torch.bfloat16)
    x.view(torch.int16)[0, 37] = 1
    x[1, 11] = torch.finfo(torch.bfloat16).max
    values, scales = (v.cpu() for v in q4.rmsnorm_mx8(x.cuda(), eps=0.0))
    v = x.double()
    y = v / torch.sqrt(v.square().mean(-1, keepdim=True))
    mx8.check_mx8(values, scales, y, bound(False, False), "one value in a row")
    assert abs(float(y[0, 37]) - k ** 0.5) < 1e-9 * k and abs(float(y[1, 11]) - k ** 0.5) < 1e-9 * k


def test_a_small_eps_beside_small_rows():
    x = (rows(6, 512, 9).double() * 3e-39).to(torch.bfloat16)
    for eps in (2.0 ** -149, 2.0 ** -140, 2.0 ** -126):
        values, scales = (v.cpu() for v in q4.rmsnorm_mx8(x.cuda(), eps=eps))
        v = x.double()
        y = v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps)
        mx8.check_mx8(values, scales, y, bound(False, False), "eps %g" % eps)


def test_rows_of_zeros():
    """eps decides: zeros with one, 0 / 0 without."""
    x = torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
    values, scales = q4.rmsnorm_mx8(x, eps=2.0 ** -149)
    assert not bool(values.view(torch.uint8).any()) and not bool(scales.view(torch.uint8).any())
    _, scales = q4.rmsnorm_mx8(x, eps=0.0)
    assert bool((scales.view(torch.uint8) == 255).all())


@pytest.mark.parametrize("t,k", [(1, 64), (1, 5120), (3, 192), (2, 8256), (5, 17408), (600, 256), (513, 5120)])
@pytest.mark.parametrize("form", ["plain", "both"])
def test_ordinary_rows_to_the_last_bits(t, k, form):
    """The bound of every rounding for rows as a model has them (a residual stream four times as large)."""
    both, eps = form == "both", 2.0 ** -17
    x, w = rows(t, k, 1).to(torch.bfloat16), rows(1, k, 2)[0].to(torch.bfloat16)
    r = (rows(t, k, 3) * 4).to(torch.bfloat16)
    out = q4.rmsnorm_mx8(x.cuda(), w.cuda() if both else None, eps, residual=r.cuda() if both else None)
    v = x.double() + (r.double() if both else 0)
    y = v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps) * (w.double() if both else 1)
    mx8.check_mx8(out[0].cpu(), out[1].cpu(), y, bound(both, both), "ordinary rows")
