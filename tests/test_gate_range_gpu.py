"""The gated quantization with gates so low that e^-gate leaves binary32 (below -88): silu(gate) x is what it is for every x
that bf16 holds."""
import math

import pytest
import torch

import mx8
import weight_only_bit_q4_amd as q4
from gpu_util import announce

pytestmark = pytest.mark.gpu

# Relative error of y before its rounding to 8 bits, |gate| up to 190: four exponentials of a quarter of it (the product with
# log2 e and that constant's own rounding, 1.5 x 47.5 x 2^-24 each; the exponential 2 x 2^-24) and six products: below
# 310 x 2^-24.  One exponential of the whole above -88: 1.5 x 88 x 2^-24 and a few more.  Products under 2^-126 are rounded
# to 2^-150: six of them.
RELATIVE, ABSOLUTE = 310 * 2.0 ** -24, 6 * 2.0 ** -150


def check(got, gate, x):
    g = gate.double()
    # (in binary64 e^-gate is finite up to gates of -709)
    y = x.double() * g / (1 + torch.exp(-g))
    values, scales = mx8.e4m3(got[0].cpu()), got[1].view(torch.uint8).cpu().to(torch.int64)
    most = y.unflatten(-1, (-1, 32)).abs().amax(-1)

    def byte(m):
        man, exp = torch.frexp(m)
        return torch.where(m > 0, exp - 9 + (man > 0.875), -127).clamp(min=-127) + 127
    assert bool((scales >= byte(most * (1 - RELATIVE) - ABSOLUTE)).all()), "scales"
    assert bool((scales <= byte(most * (1 + RELATIVE) + ABSOLUTE)).all()), "scales"
    unit = torch.exp2(scales.double() - 127).repeat_interleave(32, -1)
    scaled = y / unit
    step = torch.exp2(torch.floor(torch.log2(scaled.abs().clamp(min=2.0 ** -6))) - 4)
    off = (values - scaled).abs() - step - RELATIVE * scaled.abs() - ABSOLUTE / unit
    worst = int(off.argmax())
    assert bool((off <= 0).all()), "gate %r, x %r: %r for %r" % tuple(
        float(v.flatten()[worst]) for v in (gate, x, values, scaled))


@pytest.mark.parametrize("size", [1.0, 1e5, 1e20, 1e30, 7e37])
def test_low_gates(size):
    """Rows whose gates lie around one number, from where nothing special happens to where nothing is left."""
    gen = torch.Generator().manual_seed(3)
    at = torch.tensor([-60, -80, -86, -87.5, -88, -88.5, -89, -92, -100, -120, -150, -170, -186])[:, None]
    gate = (at + 3 * torch.rand(len(at), 512, generator=gen) - 1.5).to(torch.bfloat16)
    x = (torch.randn(len(at), 512, generator=gen) * size).to(torch.bfloat16)
    announce("quantize_mx8 with low gates, x of %g" % size)
    check(q4.quantize_mx8(x.cuda(), gate=gate.cuda()), gate, x)


def test_every_gate():
    """All of bf16's gates from -186 up to 88, beside x that bring the products to about one."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    every = bits.view(torch.bfloat16)
    gate = every[(every >= -186) & (every <= 88)]
    gate = torch.nn.functional.pad(gate, (0, -len(gate) % 64)).view(1, -1)
    g = gate.double()
    silu = g / (1 + torch.exp(-g))
    x = (1 / silu.abs().clamp(min=1e-38)).clamp(max=3e38).to(torch.bfloat16)
    check(q4.quantize_mx8(x.cuda(), gate=gate.cuda()), gate, x)


def test_one_low_gate_beside_ordinary_ones():
    gen = torch.Generator().manual_seed(4)
    gate, x = torch.randn(3, 256, generator=gen), torch.randn(3, 256, generator=gen)
    for i in range(0, 256, 8):
        gate[:, i + i // 8 % 8], x[:, i + i // 8 % 8] = -91.0, 3e37
    gate, x = gate.to(torch.bfloat16), x.to(torch.bfloat16)
    check(q4.quantize_mx8(x.cuda(), gate=gate.cuda()), gate, x)


def test_gates_past_every_number():
    """The lowest finite gate leaves zeros; infinities and NaN their blocks NaN."""
    gate = torch.zeros(1, 192, dtype=torch.bfloat16)
    x = torch.ones(1, 192, dtype=torch.bfloat16)
    gate[0, :32] = torch.finfo(torch.bfloat16).min
    gate[0, 33], gate[0, 70], gate[0, 100] = -math.inf, math.nan, -95.0
    x[0, 100] = math.inf
    gate[0, 128:160] = -1000.0
    values, scales = (v.view(torch.uint8).cpu() for v in q4.quantize_mx8(x.cuda(), gate=gate.cuda()))
    assert scales[0].tolist() == [0, 255, 255, 255, 0, 0]
    assert not bool((values[0, :32] & 127).any()) and not bool((values[0, 128:] & 127).any())
