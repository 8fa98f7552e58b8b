"""The operators with 8-bit activations and log probabilities as a user's
program runs them: together, on other streams, side by side, in captured
graphs that share a workspace; and the borders between their kernels."""
import math

import pytest
import torch

import mx8
import weight_only_bit_q4_amd as q4
from gpu_util import announce

pytestmark = pytest.mark.gpu


def bf16(shape, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(torch.bfloat16).cuda()


def weight(n, k, seed):
    return tuple(v.cuda() for v in mx8.random_weight(n, k, seed))


def activations(t, k, seed):
    return tuple(v.cuda() for v in mx8.random_mx8(t, k, seed))


def same(got, want, what):
    for u, v in zip(got, want):
        if v is None:
            assert u is None
        else:
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8)), what


class Model:
    """Two layers and the head: norm, product, gated quantization, product with the residual, log probabilities."""

    def __init__(self, k, inner, vocab, seed):
        self.inner = inner
        self.layers = [(bf16((k,), seed + 7 * i, 0.2) + 1, weight(2 * inner, k, seed + 7 * i + 1),
                        weight(k, inner, seed + 7 * i + 2)) for i in range(2)]
        self.norm = bf16((k,), seed + 50, 0.2) + 1
        self.head = weight(vocab, k, seed + 51)

    def __call__(self, x, tokens, top, exact=False):
        r = torch.zeros_like(x)
        for norm, up, down in self.layers:
            v, s, h = q4.rmsnorm_mx8(x, norm, residual=r)
            both = q4.linear_mx8(v, s, *up)
            v, s = q4.quantize_mx8(both[:, self.inner:], gate=both[:, :self.inner])
            x, r = q4.linear_mx8(v, s, *down), h
        v, s, h = q4.rmsnorm_mx8(x, self.norm, residual=r)
        if exact:
            return (h,) + q4.linear_logprobs(h, None, *self.head, tokens, top)
        return (h,) + q4.linear_logprobs(v, s, *self.head, tokens, top)


@pytest.mark.parametrize("t", [1, 6, 24, 150])
def test_a_model_eager_and_replayed(t):
    k, inner, vocab, top = 512, 640, 3001, 5
    model = Model(k, inner, vocab, 100)
    x, tokens = bf16((t, k), 1), torch.arange(t, dtype=torch.int32, device="cuda") * 19 - 1
    announce("a model of two layers, t=%d" % t)
    outs = model(x, tokens, top)
    torch.cuda.synchronize()
    # its last step against 64 bits: from the h that it gives
    h = outs[0].double().cpu()
    norm = h / torch.sqrt(h.square().mean(-1, keepdim=True) + 1e-6) * model.norm.double().cpu()
    q, s = mx8.weight64(*(v.cpu() for v in model.head))
    logits = norm @ (q * s[..., None]).flatten(1).t()
    logp = torch.log_softmax(logits, -1)
    inside = tokens.cpu() >= 0
    got = outs[1].double().cpu()
    # a logit is a sum of 512 products, each value rounded to E4M3: 2^-4 of it at most, so a random walk of
    # 2^-5 sqrt(sum (w x)^2) on average; eight times that for the largest of all
    walk = 8 * 2.0 ** -5 * float((norm.square() @ (q * s[..., None]).flatten(1).square().t()).sqrt().max())
    want = logp.gather(1, tokens.cpu().clamp(min=0).long()[:, None])[:, 0]
    assert bool(((got - want).abs()[inside] <= 2 * walk).all()) and not bool(got[~inside].any())
    assert torch.equal(outs[3], outs[3].sort(-1, descending=True).values)
    exact = model(x, tokens, top, exact=True)
    logp = torch.log_softmax(h @ (q * s[..., None]).flatten(1).t(), -1)
    want = logp.gather(1, tokens.cpu().clamp(min=0).long()[:, None])[:, 0]
    # bf16 activations are exact: binary32 sums of 512 products (2^-24 each of the magnitudes)
    own = 90 * 2.0 ** -24 * float((h.abs() @ (q.abs() * s[..., None]).flatten(1).t()).max())
    assert bool(((exact[1].double().cpu() - want).abs()[inside] <= 2.0 ** -19 + 20 * own + 2.0 ** -23 * want.abs()[inside]).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = model(x, tokens, top)
        held_exact = model(x, tokens, top, exact=True)
    for i in range(4):
        x.copy_(bf16((t, k), 20 + i))
        tokens.copy_(torch.randint(-1, vocab, (t,), generator=torch.Generator().manual_seed(i), dtype=torch.int32))
        want, want_exact = model(x, tokens, top), model(x, tokens, top, exact=True)
        graph.replay()
        torch.cuda.synchronize()
        same(held, want, "replay %d" % i)
        same(held_exact, want_exact, "replay %d" % i)


def calls(t=24, k=512, n=3001):
    x, r = bf16((t, k), 1), bf16((t, k), 2)
    act, w, add = activations(t, k, 3), weight(n, k, 4), bf16((t, n), 5)
    shared = weight(64, 20480, 6), activations(t, 20480, 7)  # (K shares)
    tokens = torch.arange(t, dtype=torch.int32, device="cuda")
    wide = torch.randn(t, 30011, generator=torch.Generator().manual_seed(8)).cuda()
    return {
        "rmsnorm_mx8": lambda **kw: q4.rmsnorm_mx8(x, residual=r, **kw),
        "quantize_mx8": lambda **kw: q4.quantize_mx8(x, r, **kw),
        "linear_mx8": lambda **kw: (q4.linear_mx8(*act, *w, residual=add, **kw),),
        "linear_mx8_shares": lambda **kw: (q4.linear_mx8(*shared[1], *shared[0], **kw),),
        "logprobs": lambda **kw: q4.logprobs(wide, tokens, 5, **kw),
        "logprobs_no_tokens": lambda **kw: q4.logprobs(wide, None, 5, **kw),
        "linear_logprobs": lambda **kw: q4.linear_logprobs(*act, *w, tokens, 5, **kw),
        "linear_logprobs_bf16": lambda **kw: q4.linear_logprobs(x, None, *w, tokens, 5, **kw),
    }


NAMES = ["rmsnorm_mx8", "quantize_mx8", "linear_mx8", "linear_mx8_shares", "logprobs", "logprobs_no_tokens",
         "linear_logprobs", "linear_logprobs_bf16"]


@pytest.mark.parametrize("name", NAMES)
def test_own_memory_on_another_stream(name):
    call = calls()[name]
    want = [v.clone() if v is not None else None for v in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    announce("%s on another stream" % name)
    busy = torch.randn(2048, 2048, device="cuda")
    for _ in range(3):
        # memory of the current stream, free again for it, with writes to it still waiting behind long work
        scratch = [torch.empty_like(v) for v in want if v is not None for _ in range(8)]
        scratch += [torch.empty(1 << 16, dtype=torch.uint8, device="cuda") for _ in range(8)]
        taken = {v.data_ptr() for v in scratch}
        for _ in range(20):
            busy = (busy @ busy).mul_(1e-3)
        for v in scratch:
            v.view(torch.uint8).fill_(7)
        del scratch, v
        got = call(stream=side.cuda_stream)
        assert not taken & {v.data_ptr() for v in got if v is not None}
        torch.cuda.synchronize()
        same(got, want, name)


def test_two_calls_at_once():
    """Every operator on two streams side by side, each with memory of its own."""
    every = calls()
    want = {name: [v.clone() if v is not None else None for v in every[name]()] for name in NAMES}
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    announce("two streams at once")
    for _ in range(5):
        got = []
        for i in range(len(NAMES)):
            for side, name in zip(sides, (NAMES[i], NAMES[-1 - i])):
                got.append((name, every[name](stream=side.cuda_stream)))
        torch.cuda.synchronize()
        for name, g in got:
            same(g, want[name], name)


def test_two_graphs_share_a_workspace():
    """Captured calls of different sizes with one workspace, replayed in turn on one stream."""
    act, w = activations(20, 20480, 1), weight(64, 20480, 2)
    x, head = bf16((9, 512), 3), weight(5000, 512, 4)
    logits = torch.randn(40, 60000, generator=torch.Generator().manual_seed(5)).cuda()
    need = max(q4.q4lin_linear_mx8_workspace_bytes(64, 20480, 20), q4.q4lin_linear_logprobs_workspace_bytes(5000, 512, 9, 4),
               q4.q4lin_logprobs_workspace_bytes(60000, 40, 4))
    workspace = torch.empty(need, dtype=torch.uint8, device="cuda")

    def one():
        return (q4.linear_mx8(*act, *w, workspace=workspace),) + q4.linear_logprobs(x, None, *head, None, 4, workspace=workspace)

    def two():
        return q4.logprobs(logits, None, 4, workspace=workspace)
    want = [[v.clone() if v is not None else None for v in f()] for f in (one, two)]
    torch.cuda.synchronize()
    announce("two graphs with one workspace")
    graphs = []
    for f in (one, two):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f()
        graphs.append((g, out))
    for i in range(6):
        workspace.fill_(0xFF if i % 2 else 0x7F)  # (nothing is expected of it)
        for g, _ in (graphs if i % 3 else graphs[::-1]):
            g.replay()
        torch.cuda.synchronize()
        for (_, out), v in zip(graphs, want):
            same(out, v, "round %d" % i)


# -- the borders between the product's kernels -------------------------------------
BORDERS = [(1001, 576, t) for t in (1, 2, 8, 9, 16, 17, 32, 33, 64, 65, 96, 97, 128, 129, 191, 256, 257)]
BORDERS += [(16500, 192, 16), (8193, 128, 33), (12288, 1024, 20), (12288, 1024, 64), (9000, 4096, 23), (9001, 4160, 40),
            (131, 20480, 23), (70, 8256, 48), (200, 4160, 100), (385, 2112, 129), (1, 320, 31), (3, 64, 300), (5120, 4416, 32)]
# one token: rows of every number of pieces a lane and of waves
BORDERS += [(n, k, 1) for n, k in ((300, 64), (6144, 16384), (513, 16448), (2000, 20480), (300, 24576),
                                     (300, 24640), (70, 32832), (9, 1 << 17), (34816, 192), (65000, 576))]


@pytest.mark.parametrize("n,k,t", BORDERS)
def test_linear_at_the_kernels_borders(n, k, t):
    act, w, r = activations(t, k, n + t), weight(n, k, t), bf16((t, n), 9)
    room = torch.full((t + 2, n), 7.0, dtype=torch.bfloat16, device="cuda")
    announce("linear_mx8 n=%d k=%d t=%d between neighbours" % (n, k, t))
    y = q4.linear_mx8(*act, *w, residual=r, y=room[1:t + 1])
    torch.cuda.synchronize()
    want, bound = mx8.linear(*act, *w, residual=r)
    mx8.close(y, want, bound, "linear_mx8")
    assert bool((room[0] == 7).all()) and bool((room[t + 1] == 7).all())


@pytest.mark.parametrize("t,k", [(1, 512), (4, 192), (12, 512), (20, 512), (60, 128), (300, 512)])
def test_linear_nan_and_infinite_scales(t, k):
    """A NaN in a token, in a weight's scale, an infinite scale: each stays in its column or row."""
    act, (codes, scales) = activations(t, k, 5), weight(150, k, 6)
    clean = q4.linear_mx8(*act, codes, scales)
    scales[77, 1] = math.nan
    scales[80, 0] = math.inf
    act[0].view(torch.uint8)[t - 1, 5] = 0xFF  # (the other NaN)
    y = q4.linear_mx8(*act, codes, scales)
    assert bool(torch.isnan(y[t - 1]).all()) and bool(torch.isnan(y[:, 77]).all())
    assert not bool(torch.isfinite(y[:, 80]).any())
    keep = [i for i in range(150) if i not in (77, 80)]
    assert torch.equal(y[:t - 1][:, keep], clean[:t - 1][:, keep])


@pytest.mark.parametrize("n,k,t", [(300, 32768, 3), (300, 32832, 3), (70, 1 << 17, 2), (70, 1 << 17, 9), (500, 256, 8),
                                   (500, 192, 4), (1, 64, 1), (1, 320, 200), (255, 128, 64), (257, 1088, 65),
                                   (131085, 64, 300)])  # (the last: runs of tokens)
@pytest.mark.parametrize("form", ["mx8", "bf16"])
def test_linear_logprobs_at_the_kernels_borders(n, k, t, form):
    top = min(n, 3)
    x, (codes, scales) = bf16((t, k), n + t), weight(n, k, 3)
    given = (x, None)
    if form == "mx8":
        given = activations(t, k, n)
        x = mx8.decode(*given)
    announce("linear_logprobs n=%d k=%d t=%d %s" % (n, k, t, form))
    tokens = torch.full((t,), n - 1, dtype=torch.int32, device="cuda")
    logprob, entropy, best, ids = q4.linear_logprobs(*given, codes, scales, tokens, top)
    torch.cuda.synchronize()
    q, s = mx8.weight64(codes, scales)
    w = (q * s[..., None]).flatten(1)
    logits = x.double() @ w.t()
    logp = torch.log_softmax(logits, -1)
    # a logit's error: k / 64 + 80 operations of 2^-24 of the magnitudes (q + 8 and the offsets: up to 136 / 8 of them)
    own = 20 * (k // 64 + 80) * 2.0 ** -24 * float((x.double().abs() @ w.abs().t()).max())
    off = 2.0 ** -19 + own
    assert bool(((logprob - logp[:, n - 1]).abs() <= off + 2.0 ** -23 * logp[:, n - 1].abs()).all())
    picked = logp.gather(1, ids.long())
    assert bool(((best - picked).abs() <= off + 2.0 ** -23 * picked.abs()).all())
    assert bool(((picked - logp.sort(-1, descending=True).values[:, :top]).abs() <= 2 * own).all())
    ent = -(logp.exp() * logp).sum(-1)
    assert bool(((entropy - ent).abs() <= 2.0 ** -15 + 40 * own).all())


@pytest.mark.parametrize("t", [4, 8, 40, 200])
@pytest.mark.parametrize("form", ["mx8", "bf16"])
def test_linear_logprobs_nan_stays_in_its_token(t, form):
    codes, scales = weight(700, 512, 2)
    given = list(activations(t, 512, 3)) if form == "mx8" else [bf16((t, 512), 3), None]
    clean = q4.linear_logprobs(*given, codes, scales, None, 3)
    if form == "mx8":
        given[0].view(torch.uint8)[1, 70] = 0x7F
        given[1].view(torch.uint8)[t - 1, 15] = 255
    else:
        given[0][1, 70] = math.nan
        given[0][t - 1, 500] = math.inf
    _, entropy, best, ids = q4.linear_logprobs(*given, codes, scales, None, 3)
    bad = torch.isnan(entropy)
    assert bad.nonzero().flatten().tolist() == [1, t - 1]
    assert bool(torch.isnan(best[bad]).all())
    same([v[~bad] for v in (entropy, best, ids)], [v[~bad] for v in clean[1:]], "other tokens")


@pytest.mark.parametrize("n", [4000, 70000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logprobs_more_equal_alternatives_than_a_list_holds(n, dtype):
    """Every number equal, or all but a few: the lowest numbers are taken."""
    l = torch.zeros(4, n)
    l[1, n // 2:] = 1.0
    l[2, 5::7] = 2.0
    l[3] = torch.arange(n) % 64
    l = l.to(dtype).cuda()
    _, _, best, ids = q4.logprobs(l, None, 32)
    for i in range(4):
        want = torch.sort(l[i].cpu(), descending=True, stable=True).indices[:32]
        assert ids[i].tolist() == want.tolist(), i


def test_nothing_to_do():
    codes, scales = weight(100, 512, 1)
    none = torch.empty(0, 512, dtype=torch.bfloat16, device="cuda")
    v, s, h = q4.rmsnorm_mx8(none, residual=none)
    assert v.shape == (0, 512) and s.shape == (0, 16) and h.shape == (0, 512)
    v, s = q4.quantize_mx8(none, none)
    assert q4.linear_mx8(v, s, codes, scales).shape == (0, 100)
    assert q4.linear_mx8(*activations(3, 512, 1), codes[:0], scales[:0]).shape == (3, 0)
    for given in ((v, s), (none, None)):
        out = q4.linear_logprobs(*given, codes, scales, torch.empty(0, dtype=torch.int32, device="cuda"), 4)
        assert [tuple(u.shape) for u in out] == [(0,), (0,), (0, 4), (0, 4)]
