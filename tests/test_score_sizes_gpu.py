"""linear_logprobs of more activations than one dimension of a grid has threads for (2^32 of eight values each)."""
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
