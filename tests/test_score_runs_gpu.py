"""linear_logprobs of more tokens than a run holds, with a last run shorter than the others: in a workspace of the asked
size and not a byte more, against the same tokens a part at a time and against 64 bits."""
import pytest
import torch

import mx8
import weight_only_bit_q4_amd as q4
from gpu_util import announce

pytestmark = pytest.mark.gpu

GUARD = 1 << 18


# (runs of 147 and 146 tokens with 6 and 8 shares a row, 205 and 204 with 4 and 6, 512 and 511 with 2 and 3,
# 69 and 68 with 11 and 16, 342 and 341)
@pytest.mark.parametrize("n,t,top", [(131072, 293, 20), (131072, 293, 0), (128256, 409, 5), (65000, 1023, 20),
                                     (256000, 137, 32), (65000, 683, 3)])
@pytest.mark.parametrize("form", ["mx8", "bf16"])
def test_a_shorter_last_run(n, t, top, form):
    k = 64
    codes, scales = (v.cuda() for v in mx8.random_weight(n, k, n))
    if form == "mx8":
        given = tuple(v.cuda() for v in mx8.random_mx8(t, k, t))
        x = mx8.decode(*given)
    else:
        given = (torch.randn(t, k, generator=torch.Generator().manual_seed(t)).to(torch.bfloat16).cuda(), None)
        x = given[0].double()
    tokens = (torch.arange(t, dtype=torch.int64) * 7919 % n).to(torch.int32).cuda()
    need = q4.q4lin_linear_logprobs_workspace_bytes(n, k, t, top)
    room = torch.full((need + 2 * GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
    announce("linear_logprobs n=%d t=%d top=%d %s in %d bytes" % (n, t, top, form, need))
    logprob, entropy, best, ids = q4.linear_logprobs(*given, codes, scales, tokens, top, workspace=room[GUARD:GUARD + need])
    torch.cuda.synchronize()
    assert bool((room[:GUARD] == 0x5A).all()) and bool((room[GUARD + need:] == 0x5A).all())

    q, s = mx8.weight64(codes, scales)
    w = (q * s[..., None]).flatten(1)
    # k / 64 + 80 operations of 2^-24 of the magnitudes (q + 8 and the offsets: up to 136 / 8 of them)
    own = 20 * (k // 64 + 80) * 2.0 ** -24 * float((x.abs() @ w.abs().t()).max())
    off = 2.0 ** -19 + own
    for t0 in range(0, t, 128):
        part = slice(t0, min(t0 + 128, t))
        logp = torch.log_softmax(x[part] @ w.t(), -1)
        want = logp.gather(1, tokens[part].long()[:, None])[:, 0]
        assert bool(((logprob[part] - want).abs() <= off + 2.0 ** -23 * want.abs()).all())
        ent = -(logp.exp() * logp).sum(-1)
        assert bool(((entropy[part] - ent).abs() <= 2.0 ** -15 + 40 * own).all())
        if top:
            picked = logp.gather(1, ids[part].long())
            assert bool(((best[part] - picked).abs() <= off + 2.0 ** -23 * picked.abs()).all())
            assert bool(((picked - logp.topk(top, -1).values).abs() <= 2 * own).all())
