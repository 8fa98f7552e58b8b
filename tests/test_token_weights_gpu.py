"""The operators in which each token picks its own weights (low-rank
adapters beside a projection, mixture of experts) on the GPU against 64-bit
references; the bounds are derived in token_weights.py."""
import pytest
import torch

import token_weights as tw
import weight_only_bit_q4_amd as q4
from gpu_util import announce


pytestmark = pytest.mark.gpu


def dev(v):
    return None if v is None else v.cuda()


# -- low-rank adapters ---------------------------------------------------------
def lora_case(fmt, n, k, t, adapters, rank, order, seed, none=0.25):
    planes, w64 = tw.weight(fmt, n, k, seed)
    x = tw.bf16((t, k), seed + 1)
    # an adapter's term about as large as the weight's
    std = float(w64.std())
    a, b = tw.bf16((adapters, rank, k), seed + 2, k ** -0.5), tw.bf16((adapters, n, rank), seed + 3,
                                                                      std * (k / rank) ** 0.5)
    g = torch.Generator().manual_seed(seed + 4)
    ids = torch.randint(0, adapters, (t,), generator=g, dtype=torch.int32)
    ids[torch.rand(t, generator=g) < none] = -1
    if order == "runs":
        ids = ids.sort().values
    scale = torch.rand(adapters, generator=g) + 0.5
    return planes, w64, x, a, b, ids, scale


def run_lora(fmt, planes, x, a, b, ids, scale, what, **kw):
    n, k = planes[0].shape[0], x.shape[1]
    announce("linear_lora %s fmt=%d n=%d k=%d t=%d adapters=%d rank=%d" % (what, fmt, n, k, x.shape[0], a.shape[0],
                                                                           a.shape[1]))
    y = q4.linear_lora(dev(x), dev(planes[0]), dev(planes[2]), dev(a), dev(b), dev(ids), dev(scale), fmt=fmt,
                       codes_hi=dev(planes[1]), **kw)
    torch.cuda.synchronize()
    return y


def tiled(fmt, n, k, t):
    return fmt == 0 and q4.q4lin_route(n, k, t) == q4.Q4LIN_ROUTE_TILED


LORA = [
    # every route of the Q4 base product; odd rows, odd groups, every rank step
    (0, 512, 1024, 1, 3, 16, "mixed"), (0, 333, 64, 1, 1, 8, "mixed"), (0, 1000, 2048, 2, 5, 24, "mixed"),
    (0, 517, 1216, 5, 40, 64, "mixed"), (0, 256, 512, 16, 16, 256, "mixed"), (0, 700, 320, 17, 4, 40, "runs"),
    (0, 96, 1024, 33, 2, 136, "mixed"), (0, 1001, 192, 100, 7, 16, "mixed"), (0, 640, 256, 129, 3, 128, "runs"),
    (0, 384, 640, 300, 6, 32, "mixed"), (0, 1030, 320, 300, 2, 64, "runs"), (0, 64, 20480, 3, 2, 16, "mixed"),
    (0, 2, 128, 1, 1, 8, "mixed"), (0, 2048, 512, 600, 8, 96, "runs"),
    # the other formats
    (1, 300, 512, 1, 3, 16, "mixed"), (2, 301, 448, 7, 3, 32, "mixed"), (3, 256, 1024, 20, 4, 16, "runs"),
    (4, 130, 704, 3, 2, 8, "mixed"), (5, 200, 1088, 40, 5, 48, "mixed"), (5, 128, 512, 1, 1, 200, "mixed"),
    (3, 100, 256, 150, 3, 16, "mixed"), (1, 77, 128, 200, 9, 64, "runs"),
]


@pytest.mark.parametrize("fmt,n,k,t,adapters,rank,order", LORA)
def test_lora_matches_reference(fmt, n, k, t, adapters, rank, order):
    planes, w64, x, a, b, ids, scale = lora_case(fmt, n, k, t, adapters, rank, order, 11 + n + t)
    if t == 1:
        ids[:] = adapters - 1
    y = run_lora(fmt, planes, x, a, b, ids, scale, "seeded")
    want, bound = tw.lora_reference(x, w64, a, b, ids, scale, tiled(fmt, n, k, t))
    tw.close(y, want, bound, "linear_lora")


@pytest.mark.parametrize("t", [1, 3, 20, 70, 200])
def test_lora_without_adapters_and_scale(t):
    planes, w64, x, a, b, ids, _ = lora_case(0, 260, 512, t, 3, 16, "mixed", 50 + t)
    for value in (-1, 3, 2 ** 31 - 1, -2 ** 31):  # none of them names an adapter
        ids[:] = value
        y = run_lora(0, planes, x, a, b, ids, None, "no adapter")
        want, bound = tw.lora_reference(x, w64, a, b, ids, None, tiled(0, 260, 512, t))
        tw.close(y, want, bound, "no adapter")
    ids[:] = 2
    y = run_lora(0, planes, x, a, b, ids, None, "scale None")
    want, bound = tw.lora_reference(x, w64, a, b, ids, None, tiled(0, 260, 512, t))
    tw.close(y, want, bound, "scale None")


@pytest.mark.parametrize("t", [2, 16, 40, 200])
def test_lora_keeps_infinities_in_their_rows(t):
    planes, w64, x, a, b, ids, scale = lora_case(0, 200, 256, t, 3, 16, "mixed", 70 + t, none=0.0)
    ids[0], ids[1] = 0, 1
    clean = run_lora(0, planes, x, a, b, ids, scale, "finite")
    a[1, 3, 7] = float("nan")
    b[1, 5, 2] = float("inf")
    y = run_lora(0, planes, x, a, b, ids, scale, "NaN and infinity in adapter 1")
    others = ids.cuda() != 1
    assert torch.equal(y[others].view(torch.int16), clean[others].view(torch.int16))
    assert torch.isnan(y[~others]).all()


@pytest.mark.parametrize("t,n", [(1, 320), (20, 320), (300, 320), (20, 323)])
def test_lora_unaligned_output_and_guards(t, n):
    planes, w64, x, a, b, ids, scale = lora_case(0, n, 512, t, 4, 24, "mixed", 90 + t)
    whole = torch.full((t * n + 66,), 7.0, dtype=torch.bfloat16, device="cuda")
    need = q4.q4lin_lora_workspace_bytes(0, n, 512, t, 4, 24)
    ws = torch.full((need + 512,), 0xAB, dtype=torch.uint8, device="cuda")
    y = whole[33:33 + t * n].view(t, n)
    run_lora(0, planes, x, a, b, ids, scale, "odd address", y=y, workspace=ws[:need])
    want, bound = tw.lora_reference(x, w64, a, b, ids, scale, tiled(0, n, 512, t))
    tw.close(y, want, bound, "odd address")
    assert (whole[:33] == 7).all() and (whole[33 + t * n:] == 7).all() and (ws[need:] == 0xAB).all()


@pytest.mark.parametrize("fmt,t", [(0, 1), (0, 12), (0, 90), (0, 260), (3, 5)])
def test_lora_graph_replay(fmt, t):
    n, k, adapters, rank = 260, 512, 4, 32
    cases = [lora_case(fmt, n, k, t, adapters, rank, "mixed", 200 + 7 * i + t) for i in range(3)]
    hold = [dev(v) for v in (*cases[0][0], *cases[0][2:])]
    need = q4.q4lin_lora_workspace_bytes(fmt, n, k, t, adapters, rank)
    ws, y = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty(t, n, dtype=torch.bfloat16, device="cuda")

    def call():
        q4.linear_lora(hold[3], hold[0], hold[2], hold[4], hold[5], hold[6], hold[7], fmt=fmt, codes_hi=hold[1], y=y,
                       workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    announce("linear_lora graph fmt=%d t=%d" % (fmt, t))
    with torch.cuda.graph(graph):
        call()
    for planes, w64, x, a, b, ids, scale in cases[::-1]:
        for h, v in zip(hold, (*planes, x, a, b, ids, scale)):
            if h is not None:
                h.copy_(v)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        want, bound = tw.lora_reference(x, w64, a, b, ids, scale, tiled(fmt, n, k, t))
        tw.close(y, want, bound, "replay")
        torch.randn(1 << 20, device="cuda").sum().item()


def test_lora_on_another_stream():
    planes, w64, x, a, b, ids, scale = lora_case(0, 512, 512, 9, 4, 16, "mixed", 321)
    args = [dev(v) for v in (x, planes[0], planes[2], a, b, ids, scale)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = q4.linear_lora(*args, stream=side.cuda_stream)
    side.synchronize()
    want, bound = tw.lora_reference(x, w64, a, b, ids, scale, False)
    tw.close(y, want, bound, "side stream")


# -- mixture of experts ----------------------------------------------------------
def run_experts(x, ids, weights, planes, what, **kw):
    announce("moe_experts %s t=%d top_k=%d experts=%d inner=%d k=%d" % (what, *ids.shape, *planes[0].shape[:2],
                                                                      x.shape[1]))
    y = q4.moe_experts(dev(x), dev(ids), dev(weights), *[dev(p) for p in planes], **kw)
    torch.cuda.synchronize()
    return y


def routing(t, top_k, experts, seed, outside=0.0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(t, max(experts, top_k), generator=g).argsort(1)[:, :top_k].to(torch.int32)
    ids[torch.rand(t, top_k, generator=g) < outside] = -1
    return ids, torch.rand(t, top_k, generator=g)


EXPERTS = [  # t, top_k, experts, inner, k, outside
    (1, 1, 1, 64, 64, 0.0), (1, 2, 4, 128, 192, 0.0), (1, 8, 16, 192, 256, 0.0), (2, 3, 5, 320, 704, 0.2),
    (7, 4, 60, 64, 128, 0.0), (16, 4, 8, 192, 448, 0.0), (17, 1, 1, 128, 320, 0.0), (40, 2, 3, 128, 256, 0.3),
    (70, 6, 6, 64, 192, 0.0), (130, 2, 4, 192, 128, 0.0), (65, 1, 200, 64, 64, 0.0), (33, 8, 64, 64, 64, 0.75),
    (21, 3, 7, 1088, 64, 0.0), (3, 2, 4, 64, 2176, 0.0), (300, 2, 2, 64, 64, 0.1), (11, 6, 1024, 64, 64, 0.0),
]


@pytest.mark.parametrize("t,top_k,experts,inner,k,outside", EXPERTS)
def test_experts_match_reference(t, top_k, experts, inner, k, outside):
    planes, values = tw.expert_weights(experts, inner, k, 400 + t)
    x = tw.bf16((t, k), 401 + t)
    ids, weights = routing(t, top_k, experts, 402 + t, outside)
    y = run_experts(x, ids, weights, planes, "seeded")
    want, bound = tw.experts_reference(x, ids, weights, values)
    tw.close(y, want, bound, "moe_experts")


@pytest.mark.parametrize("t", [3, 90])
def test_experts_odd_routing(t):
    """Ids outside the experts, tokens without any, an expert named twice, every token on one expert."""
    inner, k, experts, top_k = 128, 192, 5, 3
    planes, values = tw.expert_weights(experts, inner, k, 500 + t)
    x = tw.bf16((t, k), 501)
    ids, weights = routing(t, top_k, experts, 502)
    ids[0] = torch.tensor([-1, experts, 2 ** 31 - 1], dtype=torch.int32)
    ids[1] = torch.tensor([2, 2, -2 ** 31], dtype=torch.int32)
    weights[0] = float("nan")  # of choices that count for nothing
    weights[2, 1] = 0.0
    y = run_experts(x, ids, weights, planes, "odd routing")
    assert (y[0] == 0).all()
    want, bound = tw.experts_reference(x, ids, weights, values)
    tw.close(y, want, bound, "odd routing")
    ids[:] = 4
    weights[0] = 0.5
    y = run_experts(x, ids, weights, planes, "one expert")
    want, bound = tw.experts_reference(x, ids, weights, values)
    tw.close(y, want, bound, "one expert")
    ids[:] = -1
    assert (run_experts(x, ids, weights, planes, "no expert") == 0).all()


@pytest.mark.parametrize("t", [2, 40])
def test_experts_keep_nan_in_its_row(t):
    planes, values = tw.expert_weights(4, 64, 128, 600)
    x = tw.bf16((t, 128), 601)
    ids, weights = routing(t, 2, 4, 602)
    clean = run_experts(x, ids, weights, planes, "finite")
    x[1, 5] = float("nan")
    y = run_experts(x, ids, weights, planes, "NaN in token 1")
    assert torch.isnan(y[1]).all()
    rest = torch.arange(t) != 1
    assert torch.equal(y[rest.cuda()].view(torch.int16), clean[rest.cuda()].view(torch.int16))


@pytest.mark.parametrize("t", [1, 50])
def test_experts_unaligned_output_and_guards(t):
    planes, values = tw.expert_weights(6, 192, 320, 700)
    x = tw.bf16((t, 320), 701)
    ids, weights = routing(t, 3, 6, 702)
    whole = torch.full((t * 320 + 66,), 7.0, dtype=torch.bfloat16, device="cuda")
    need = q4.q4lin_moe_workspace_bytes(192, 320, 6, 3, t)
    ws = torch.full((need + 512,), 0xAB, dtype=torch.uint8, device="cuda")
    y = whole[33:33 + t * 320].view(t, 320)
    run_experts(x, ids, weights, planes, "odd address", y=y, workspace=ws[:need])
    want, bound = tw.experts_reference(x, ids, weights, values)
    tw.close(y, want, bound, "odd address")
    assert (whole[:33] == 7).all() and (whole[33 + t * 320:] == 7).all() and (ws[need:] == 0xAB).all()


@pytest.mark.parametrize("t,k,experts,top_k", [(1, 64, 1, 1), (1, 2048, 128, 8), (5, 192, 60, 4), (70, 1984, 8, 2),
                                               (3, 576, 1024, 64), (2, 320, 257, 10), (9, 64, 64, 64)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_matches_reference(t, k, experts, top_k, renorm):
    x, router = tw.bf16((t, k), 800 + t), tw.bf16((experts, k), 801, 1.5 * k ** -0.5)
    announce("moe_route t=%d k=%d experts=%d top_k=%d" % (t, k, experts, top_k))
    ids, weights = q4.moe_route(dev(x), dev(router), top_k, renorm)
    torch.cuda.synchronize()
    want_ids, want, bound = tw.route_reference(x, router, top_k, renorm)
    assert torch.equal(ids.cpu().long(), want_ids)
    assert ((weights.cpu().double() - want).abs() <= bound).all()


def test_route_ties_and_nan():
    t, k, experts, top_k = 4, 128, 70, 5
    router = tw.bf16((experts, k), 850, 0.1)
    router[:] = router[:1]  # all equal: the lowest indexes
    x = tw.bf16((t, k), 851)
    ids, weights = q4.moe_route(dev(x), dev(router), top_k)
    assert (ids.cpu() == torch.arange(top_k, dtype=torch.int32)).all()
    assert ((weights.cpu() - 0.2).abs() < 1e-6).all()
    router[3:] = -router[3:]
    router[0, 0] = float("nan")  # the lowest of all, whatever its row
    ids, weights = q4.moe_route(dev(x), dev(router), experts)
    assert (ids.cpu()[:, -1] == 0).all()
    assert (ids.cpu().sort(1).values == torch.arange(experts, dtype=torch.int32)).all()


@pytest.mark.parametrize("t,experts,top_k,inner,k", [(1, 16, 4, 128, 512), (9, 12, 3, 192, 320), (80, 8, 2, 64, 256)])
@pytest.mark.parametrize("renorm", [True, False])
def test_layer_matches_reference(t, experts, top_k, inner, k, renorm):
    planes, values = tw.expert_weights(experts, inner, k, 900 + t)
    x, router = tw.bf16((t, k), 901), tw.bf16((experts, k), 902, 1.5 * k ** -0.5)
    announce("moe t=%d experts=%d top_k=%d inner=%d k=%d" % (t, experts, top_k, inner, k))
    y, ids, weights = q4.moe(dev(x), dev(router), *[dev(p) for p in planes], top_k, renormalize=renorm)
    torch.cuda.synchronize()
    want_ids, want_w, w_bound = tw.route_reference(x, router, top_k, renorm)
    assert torch.equal(ids.cpu().long(), want_ids)
    assert ((weights.cpu().double() - want_w).abs() <= w_bound).all()
    want, bound = tw.experts_reference(x, ids.cpu(), weights.cpu(), values)
    tw.close(y, want, bound, "moe")


@pytest.mark.parametrize("t", [1, 6, 70])
def test_layer_graph_replay(t):
    experts, top_k, inner, k = 12, 3, 128, 320
    cases = []
    for i in range(3):
        planes, values = tw.expert_weights(experts, inner, k, 1000 + 10 * i)
        cases.append((planes, values, tw.bf16((t, k), 1001 + i), tw.bf16((experts, k), 1050 + i, 1.5 * k ** -0.5)))
    hold = [dev(p) for p in (cases[0][2], cases[0][3], *cases[0][0])]
    ws = torch.empty(q4.q4lin_moe_workspace_bytes(inner, k, experts, top_k, t), dtype=torch.uint8, device="cuda")
    q4.moe(*hold, top_k, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    announce("moe graph t=%d" % t)
    with torch.cuda.graph(graph):
        y, ids, weights = q4.moe(*hold, top_k, workspace=ws)
    for planes, values, x, router in cases[::-1]:
        for h, v in zip(hold, (x, router, *planes)):
            h.copy_(v)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids.cpu().long(), tw.route_reference(x, router, top_k, True)[0])
        want, bound = tw.experts_reference(x, ids.cpu(), weights.cpu(), values)
        tw.close(y, want, bound, "replay")
        torch.randn(1 << 20, device="cuda").sum().item()
