"""The operators of 8-bit activations and log probabilities at sizes past 2^32 elements; linear_logprobs of more
activations than one dimension of a grid has threads for (2^32 of eight values each)."""
import pytest
import torch

import mx8
import weight_only_bit_q4_amd as q4
from gpu_util import announce

pytestmark = pytest.mark.gpu


def test_activations_past_a_grid():
    """2^35 values and some: tokens repeat with a period, and so must their numbers."""
    n, k, t, rows, period = 3, 1 << 17, (1 << 18) + 9, 4096, 4096 * 5
    codes, scales = mx8.random_weight(n, k, 1)
    need = t * k + t * (k // 32) + q4.q4lin_linear_logprobs_workspace_bytes(n, k, t, 2)
    if torch.cuda.mem_get_info()[0] < need + (8 << 30):
        pytest.skip("needs %d GiB of the GPU" % (need >> 30))
    base, _ = mx8.random_mx8(rows, 1024, 2)
    base = base.view(torch.uint8).cuda().repeat(1, k // 1024)
    values = torch.empty(t, k, dtype=torch.uint8, device="cuda")
    for t0 in range(0, t, rows):
        part = values[t0:t0 + rows]
        part.copy_(base[:len(part)])
    bytes_ = (torch.arange(t, device="cuda") % 5 + 112).to(torch.uint8)[:, None].expand(t, k // 32).contiguous()
    tokens = (torch.arange(t, device="cuda") % period % n).to(torch.int32)
    announce("linear_logprobs of %d tokens of %d" % (t, k))
    values = values.view(torch.float8_e4m3fn)
    x_scales = bytes_.view(torch.float8_e8m0fnu)
    out = q4.linear_logprobs(values, x_scales, codes.cuda(), scales.cuda(), tokens, 2)
    torch.cuda.synchronize()
    q, s = mx8.weight64(codes, scales)
    w = (q * s[..., None]).flatten(1)
    for i in (0, 1, 4095, 77 * 64 + 3, t - 10, t - 9, t - 1):
        x = mx8.decode(values[i:i + 1].cpu(), x_scales[i:i + 1].cpu())
        logp = torch.log_softmax(x @ w.t(), -1)[0]
        # k / 64 + 80 operations of 2^-24 of the magnitudes (q + 8 and the offsets: up to 136 / 8 of them)
        own = 20 * (k // 64 + 80) * 2.0 ** -24 * float((x.abs() @ w.abs().t()).max())
        want = float(logp[int(tokens[i])])
        assert abs(float(out[0][i]) - want) <= 2.0 ** -19 + own + 2.0 ** -23 * abs(want), i
    first = [v[:period].view(torch.int32) for v in out]
    for t0 in range(0, t, period):
        for v, f in zip(out, first):
            part = v[t0:t0 + period].view(torch.int32)
            assert torch.equal(part, f[:len(part)]), "tokens from %d" % t0


def repeats(out, first, period, what):
    """That ``out``'s rows are ``first``'s again and again, to the bit."""
    for t0 in range(0, len(out), period):
        part = out[t0:t0 + period]
        assert torch.equal(part.view(torch.uint8), first[:len(part)].view(torch.uint8)), "%s from row %d" % (what, t0)


def repeated(base, t):
    x = torch.empty((t,) + base.shape[1:], dtype=base.dtype, device="cuda")
    for t0 in range(0, t, len(base)):
        part = x[t0:t0 + len(base)]
        part.copy_(base[:len(part)])
    return x


def room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip("needs %d GiB of the GPU" % gib)


def test_norm_past_32_bits():
    """Offsets past 2^32 elements, the residual stream updated in place."""
    room(48)
    t, k, period = (1 << 18) + 5, 16448, 1000
    g = torch.Generator().manual_seed(1)
    x, r = (torch.randn(period, k, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    first = q4.rmsnorm_mx8(x, residual=r)
    announce("rmsnorm_mx8 of %d rows of %d" % (t, k))
    big = repeated(x, t)
    out = q4.rmsnorm_mx8(big, residual=repeated(r, t), h=big)
    for v, f, what in zip(out, first, ("values", "scales", "h")):
        repeats(v, f, period, what)


def test_gated_halves_past_32_bits():
    room(48)
    t, k, period = (1 << 19) + 5, 8256, 1000
    both = torch.randn(period, 2 * k, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    first = q4.quantize_mx8(both[:, k:], gate=both[:, :k])
    announce("quantize_mx8 of %d rows of %d" % (t, k))
    big = repeated(both, t)
    for v, f, what in zip(q4.quantize_mx8(big[:, k:], gate=big[:, :k]), first, ("values", "scales")):
        repeats(v, f, period, what)


def test_product_past_32_bits():
    room(24)
    n, k, t, period = 8200, 64, (1 << 19) + 7, 6144  # (a multiple of every tile's tokens)
    act = [v.cuda() for v in mx8.random_mx8(period, k, 3)]
    w = [v.cuda() for v in mx8.random_weight(n, k, 4)]
    big = [repeated(v.view(torch.uint8), t) for v in act]
    announce("linear_mx8 of %d tokens and %d rows" % (t, n))
    y = q4.linear_mx8(*big, *w)
    want, bound = mx8.linear(act[0][:500], act[1][:500], *w)
    mx8.close(y[:500], want, bound, "linear_mx8")
    repeats(y, y[:period].clone(), period, "outputs")


def test_logits_past_32_bits():
    room(32)
    n, t, period = 70001, (1 << 16) + 3, 500
    logits = torch.randn(period, n, generator=torch.Generator().manual_seed(5)).cuda()
    tokens = (torch.arange(t) % period * 137 % n).to(torch.int32).cuda()
    announce("logprobs of %d rows of %d" % (t, n))
    out = q4.logprobs(repeated(logits, t), tokens, 3)
    logp = torch.log_softmax(logits.double(), -1)
    want = logp.gather(1, tokens[:period].long()[:, None])[:, 0]
    # binary32 sums of up to 32 x 9 exponentials a thread, each good to 2^-20 (|l - m| < 16), and one rounding
    assert bool(((out[0][:period] - want).abs() <= 300 * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * want.abs()).all())
    assert torch.equal(out[3][:period].long(), torch.topk(logits, 3, -1).indices)
    for v, what in zip(out, ("log probabilities", "entropy", "best", "their numbers")):
        repeats(v, v[:period].clone(), period, what)
