"""MXFP8 activations and the operators around them in 64 bits, from the
formats' definitions, and the bounds that go with them."""
import torch


def e4m3(bits):
    """E4M3 bytes as their values: four exponent bits (bias 7), three of mantissa."""
    b = bits.view(torch.uint8).to(torch.int64)
    exp, man = (b // 8) % 16, (b % 8).double()
    v = torch.where(exp > 0, (1 + man / 8) * torch.exp2(exp.double() - 7), man / 8 * 2.0 ** -6)
    v = torch.where(b % 128 == 127, torch.nan, v)
    return torch.where(b >= 128, -v, v)


def block_scales(bits):
    b = bits.view(torch.uint8).double()
    return torch.where(b == 255, torch.nan, torch.exp2(b - 127))


def decode(values, scales):
    return e4m3(values) * block_scales(scales).repeat_interleave(32, -1)


def random_mx8(t, k, seed, spread=0, device="cpu"):
    """Activations as a norm leaves them: every E4M3 magnitude but NaN; block exponents within +-spread."""
    g = torch.Generator().manual_seed(seed)
    v = (torch.randn(t, k, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = torch.randint(119 - spread, 120 + spread, (t, k // 32), generator=g).to(torch.uint8)
    return v.to(device), s.view(torch.float8_e8m0fnu).to(device)


def random_weight(n, k, seed, device="cpu"):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    scales = ((torch.rand(n, k // 64, generator=g) + 0.5) * (k ** -0.5 / 4.6)).to(torch.float16)
    return codes.to(device), scales.to(device)


def weight64(codes, scales):
    """The codes' numbers minus eight [N][G][64] and the scales [N][G]."""
    c = codes.to(torch.int64)
    q = torch.stack((c % 16, c // 16), -1).flatten(-2).double() - 8
    return q.unflatten(-1, (-1, 64)), scales.double()


def linear(values, x_scales, codes, scales, residual=None):
    """(outputs in 64 bits, how far a stored output may be from them).

    The bound counts: one rounding to bf16, 2^-8 of the output; in each group
    64 products q x and as many 8 x, none larger than 15 max|x|, each cut by at
    most 2^-17 of the largest (the scaled matrix instruction's alignment); the
    group sums, their scaling and their sum in binary32: each of G + 8
    operations 2^-24 of the sum of their magnitudes."""
    q, s = weight64(codes, scales)
    x = decode(values, x_scales)
    n, g, _ = q.shape
    y = x @ (q * s[..., None]).flatten(1).t()
    xg = x.unflatten(-1, (-1, 64)).abs()
    big = (xg.amax(-1) @ s.abs().t()) * 15
    total = (xg.sum(-1) @ s.abs().t()) * 15
    if residual is not None:
        y = y + residual.double()
    bound = y.abs() * 2.0 ** -8 + 128 * 2.0 ** -17 * big + (g + 8) * 2.0 ** -24 * (total + y.abs())
    return y, bound


def close(got, want, bound, what):
    got = got.double()
    off = (got - want).abs() - bound
    worst = int(off.argmax())
    assert bool((off <= 0).all()), "%s: element %d is %r, should be %r, may be off by %r" % (
        what, worst, float(got.flatten()[worst]), float(want.flatten()[worst]), float(bound.flatten()[worst]))


# Relative error of y before its rounding to 8 bits: v's rounding; the mean of
# squares, a chain of at most 8 x 16 binary32 additions a thread with errors
# 2^-24 each (half of that in the root), the root's and two products'
# roundings: below 70 x 2^-24.  The gated form: an exponential of 2^-20 at
# |gate| up to 16 (the product with log2 e is rounded), a quotient, a product.
FORM_ERROR = {"norm": 70 * 2.0 ** -24, "quant": 0.0, "gated": 2.0 ** -19}


def check_mx8(values, scales, y, error, what):
    """That the blocks hold ``y`` (64 bits, known to ``error`` of itself) rounded once to E4M3 in the stated scale."""
    b = y.unflatten(-1, (-1, 32))
    most = b.abs().amax(-1)
    byte = scales.view(torch.uint8).to(torch.int64)

    def scale_byte(m):
        man, exp = torch.frexp(m)
        e = torch.where(m > 0, exp - 9 + (man > 0.875), -127).clamp(min=-127)
        return e + 127
    low, high = scale_byte(most * (1 - error)), scale_byte(most * (1 + error))
    wrong = (byte < low) | (byte > high)
    assert not bool(wrong.any()), "%s: scale bytes %s, should be %s to %s" % (what, byte[wrong][:4].tolist(),
                                                                           low[wrong][:4].tolist(),
                                                                           high[wrong][:4].tolist())
    unit = torch.exp2(byte.double() - 127)[..., None]
    scaled = b / unit
    got = e4m3(values).unflatten(-1, (-1, 32))
    # half a step of E4M3 around the value: 2^-4 of its binade, 2^-10 below 2^-6
    step = torch.exp2(torch.floor(torch.log2(scaled.abs().clamp(min=2.0 ** -6))) - 4)
    off = (got - scaled).abs() - step - error * scaled.abs()
    worst = int(off.argmax())
    assert bool((off <= 0).all()), "%s: value %d is %r for %r" % (what, worst, float(got.flatten()[worst]),
                                                                float(scaled.flatten()[worst]))
