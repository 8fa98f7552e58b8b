"""Log probabilities, entropy and alternatives on the GPU against 64 bits."""
import math

import pytest
import torch

import mx8
import weight_only_bit_q4_amd as q4
from gpu_util import announce

pytestmark = pytest.mark.gpu


def reference(logits, tokens, top):
    """In 64 bits; equal ones by the lowest number, a NaN last."""
    l = logits.double()
    m = l.amax(-1, keepdim=True)
    nothing = m[:, 0] == -math.inf
    d = l - torch.where(nothing[:, None], 0.0, m)
    e = torch.exp(d)
    z = e.sum(-1)
    entropy = torch.log(z) - torch.where(e > 0, e * d, 0.0).sum(-1) / z
    entropy = torch.where(nothing, 0.0, entropy)
    lp = torch.where(nothing[:, None], -math.inf, d - torch.log(z)[:, None])
    inside = (tokens >= 0) & (tokens < l.shape[1])
    logprob = torch.where(inside, lp.gather(1, torch.where(inside, tokens, 0).long()[:, None])[:, 0], 0.0)
    order = torch.sort(torch.where(torch.isnan(l), -math.inf, l), dim=-1, descending=True, stable=True).indices
    # (a NaN after every -inf)
    nan = torch.isnan(l).gather(1, order)
    order = order.gather(1, torch.sort(nan.to(torch.uint8), dim=-1, stable=True).indices)
    ids = order[:, :top]
    return logprob, entropy, lp.gather(1, ids), ids.to(torch.int32)


def check(out, want, logits, what):
    """A log probability of size L: 2^-24 of it for its store, and of the logarithm of z: 2^-21 for the exponentials
    (argument times log2 e rounded in binary32, arguments down to -16 carry nearly all of z) and for binary32 sums of
    256 terms a thread at most (2^-24 each, a random walk's 16 at worst on average: 2^-20).  The entropy takes both z's
    and w / z's error: w's terms are z's times |l - m| <= 24, so 2^-15 at most; both checked with room for no more than
    that."""
    logprob, entropy, top, ids = out
    for got, ref, off in ((logprob, want[0], 2.0 ** -19), (top, want[2], 2.0 ** -19), (entropy, want[1], 2.0 ** -15)):
        if got is None:
            continue
        got, ref = got.double().cpu(), ref.cpu()
        fine = torch.isfinite(ref)
        assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
        assert torch.equal(got[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)]), what
        err = (got - ref)[fine].abs()
        assert bool((err <= off + 2.0 ** -23 * ref[fine].abs()).all()), "%s: off by %r" % (what, float(err.max()))
    assert torch.equal(ids.cpu(), want[3].cpu()), what


SHAPES = [(1, 1, 1), (2, 3, 3), (1, 7, 1), (1, 1000, 5), (3, 2048, 32), (1, 131072, 20), (5, 50001, 4), (70, 8191, 8),
          (300, 30011, 3), (33, 8193, 32), (1500, 1000, 2), (2, 200003, 32), (1, 1 << 20, 7), (4, 32768, 0)]


@pytest.mark.parametrize("t,n,top", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logprobs(t, n, top, dtype):
    g = torch.Generator().manual_seed(t + n)
    logits = (torch.randn(t, n, generator=g) * 2.5).to(dtype)
    tokens = torch.randint(0, n, (t,), generator=g, dtype=torch.int32)
    announce("logprobs t=%d n=%d top=%d %s" % (t, n, top, dtype))
    out = q4.logprobs(logits.cuda(), tokens.cuda(), top)
    torch.cuda.synchronize()
    check(out, reference(logits, tokens, top), logits, "logprobs")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masks_ties_and_specials(dtype):
    n, inf = 20000, math.inf
    g = torch.Generator().manual_seed(3)
    l = torch.randn(14, n, generator=g)
    l[0] = -inf                                             # nothing is left
    l[1] = -inf
    l[1, 777] = 3.0                                         # one is
    l[2] = torch.finfo(dtype).min                           # every one at the type's lowest
    l[3, ::2] = torch.finfo(dtype).min                      # half of them
    l[4, ::3] = -inf
    l[5] = 0.0                                              # all equal
    l[6] = l[6].round()                                     # many equal
    l[7, 5] = math.nan
    l[8, 19999] = inf
    l[9, :100] = torch.linspace(50, 60, 100)                # the best behind one another
    l[10] = torch.linspace(-5, 5, n)                        # ascending
    l[11] = torch.linspace(5, -5, n)                        # descending
    l[12] = 0.0
    l[12, ::2] = -0.0                                       # both zeros are equal
    l[13] = -inf
    l[13, 3] = math.nan
    l = l.to(dtype)
    tokens = torch.tensor([5, 777, 9, 2, 3, 0, 1, 1, 19999, 99, 19999, 0, 7, 3], dtype=torch.int32)
    for top in (1, 20, 32):
        announce("logprobs of masked and special rows, top=%d" % top)
        out = q4.logprobs(l.cuda(), tokens.cuda(), top)
        want = reference(l, tokens, top)
        # (rows with a NaN or +inf: the numbers are NaN, the order is checked)
        for i in (7, 8, 13):
            for j in (0, 1, 2):
                want[j][i] = math.nan
        check(out, want, l, "special rows")


def test_tokens_outside_and_optional_outputs():
    l = torch.randn(6, 500, generator=torch.Generator().manual_seed(1))
    tokens = torch.tensor([-1, 500, 2 ** 31 - 1, -2 ** 31, 0, 499], dtype=torch.int32)
    out = q4.logprobs(l.cuda(), tokens.cuda())
    assert out[0][:4].tolist() == [0.0] * 4
    check(out, reference(l, tokens, 0), l, "padding")
    assert out[2].shape == (6, 0)
    none = q4.logprobs(l.cuda(), None, 3)
    assert none[0] is None
    check(none, reference(l, tokens, 3), l, "no tokens")
    empty = q4.logprobs(torch.empty(0, 500, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), 3)
    assert [tuple(v.shape) for v in empty] == [(0,), (0,), (0, 3), (0, 3)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_and_unaligned_rows(dtype):
    g = torch.Generator().manual_seed(8)
    wide = torch.randn(9, 9001, generator=g).to(dtype)
    tokens = torch.arange(9, dtype=torch.int32) * 100
    for first, n in ((1, 8999), (3, 4096), (8, 8192)):
        l = wide.cuda()[:, first:first + n]
        check(q4.logprobs(l, tokens.cuda(), 6), reference(l.cpu(), tokens, 6), l, "strided")
    l = wide[:1].cuda().expand(9, 9001)  # one row, seen nine times
    check(q4.logprobs(l, tokens.cuda(), 6), reference(l.cpu(), tokens, 6), l, "repeated")


def test_offsets_past_32_bits():
    """A row that begins more than 2^32 elements behind the first."""
    n, far = 5000, (1 << 32) + 8
    store = torch.zeros(far + n, dtype=torch.bfloat16, device="cuda")
    l = store.as_strided((2, n), (far, 1))
    l[0] = torch.randn(n, device="cuda")
    l[1] = torch.randn(n, device="cuda")
    tokens = torch.tensor([4, 4999], dtype=torch.int32)
    announce("logprobs of rows 2^32 elements apart")
    check(q4.logprobs(l, tokens.cuda(), 4), reference(l.cpu(), tokens, 4), l, "far rows")


SCORES = [(1000, 512, 1, 5), (1000, 256, 9, 3), (511, 640, 65, 2), (8200, 320, 8, 2), (50, 192, 3, 4), (3001, 1024, 3, 20), (40000, 256, 7, 8), (2000, 2048, 40, 4), (5003, 320, 128, 2),
          (1500, 512, 129, 3), (900, 192, 300, 2), (130, 64, 2, 32), (777, 20480, 6, 3)]


@pytest.mark.parametrize("n,k,t,top", SCORES)
@pytest.mark.parametrize("form", ["mx8", "bf16"])
def test_linear_logprobs(n, k, t, top, form):
    values, x_scales = mx8.random_mx8(t, k, n + t)
    codes, scales = mx8.random_weight(n, k, n)
    x = mx8.decode(values, x_scales)
    q, s = mx8.weight64(codes, scales)
    logits = x @ (q * s[..., None]).flatten(1).t()
    tokens = torch.randint(-1, n, (t,), generator=torch.Generator().manual_seed(t), dtype=torch.int32)
    announce("linear_logprobs n=%d k=%d t=%d %s" % (n, k, t, form))
    given = (values.cuda(), x_scales.cuda()) if form == "mx8" else (x.to(torch.bfloat16).cuda(), None)
    out = q4.linear_logprobs(*given, codes.cuda(), scales.cuda(), tokens.cuda(), top)
    torch.cuda.synchronize()
    want = reference(logits, tokens, top)
    # a logit's own error: its group sums and their sum in binary32, G + 80 operations of 2^-24 of the magnitudes
    own = (k // 64 + 80) * 2.0 ** -24 * float((x.abs() @ (q.abs() * s[..., None]).flatten(1).t()).max())
    for got, ref, off in ((out[0], want[0], 2.0 ** -19), (out[2], want[2], 2.0 ** -19), (out[1], want[1], 2.0 ** -15)):
        assert bool(((got.double().cpu() - ref).abs() <= off + 20 * own + 2.0 ** -23 * ref.abs()).all())
    # the alternatives are the largest logits, to that error
    chosen = logits.gather(1, out[3].cpu().long())
    assert bool(((chosen - logits.sort(-1, descending=True).values[:, :top]).abs() <= 2 * own).all())
    assert all(len(set(r)) == top for r in out[3].cpu().tolist())


def test_linear_logprobs_in_a_graph():
    n, k, t = 3000, 512, 4
    codes, scales = (v.cuda() for v in mx8.random_weight(n, k, 1))
    values, x_scales = (v.cuda() for v in mx8.random_mx8(t, k, 2))
    tokens = torch.tensor([0, 5, -1, 2999], dtype=torch.int32, device="cuda")

    def call():
        return q4.linear_logprobs(values, x_scales, codes, scales, tokens, 6)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for i in range(4):
        v, s = mx8.random_mx8(t, k, 10 + i)
        values.copy_(v)
        x_scales.copy_(s)
        want = call()
        graph.replay()
        torch.cuda.synchronize()
        for u, w in zip(got, want):
            assert torch.equal(u, w)
