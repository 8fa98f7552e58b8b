"""Further shapes, routings and layouts of the operators in which each token
picks its own weights, where their kernels change path: few tokens that choose
in the kernel, row counts around the tiles' sizes, planes that start in the
middle of a dword, adapters' term in the base product's kernel."""
import pytest
import torch

import token_weights as tw
import weight_only_bit_q4_amd as q4
from gpu_util import announce


pytestmark = pytest.mark.gpu


def dev(v):
    return None if v is None else v.cuda()


def shifted(v):
    """The same values on the GPU, two bytes behind a 16-byte boundary."""
    whole = torch.empty(v.numel() + 1, dtype=v.dtype, device="cuda")
    assert whole.element_size() == 2 and whole.data_ptr() % 16 == 0
    out = whole[1:].view(v.shape)
    out.copy_(v)
    return out


def experts(x, ids, weights, planes, what):
    announce("moe_experts %s t=%d top_k=%d experts=%d inner=%d k=%d" % (what, *ids.shape, *planes[0].shape[:2],
                                                                      x.shape[1]))
    y = q4.moe_experts(dev(x), dev(ids), dev(weights), *[p if p.is_cuda else p.cuda() for p in planes])
    torch.cuda.synchronize()
    return y


# -- few tokens: the layer's choice in the kernel ---------------------------------
FEW = [  # t, experts, top_k, inner, k
    (2, 16, 4, 128, 192), (3, 5, 2, 192, 704), (5, 200, 6, 64, 320), (8, 8, 8, 64, 128), (8, 256, 8, 64, 64),
    (7, 60, 4, 704, 320), (1, 64, 64, 64, 64), (4, 1, 1, 64, 64), (2, 256, 32, 64, 128), (8, 257, 8, 64, 64),
    (1, 300, 70, 64, 64), (9, 30, 7, 64, 192), (1, 16, 2, 2112, 4160),
]


@pytest.mark.parametrize("t,n,top_k,inner,k", FEW)
@pytest.mark.parametrize("renorm", [True, False])
def test_layer_of_few_tokens(t, n, top_k, inner, k, renorm):
    planes, values = tw.expert_weights(n, inner, k, 1200 + t)
    x, router = tw.bf16((t, k), 1201 + n), tw.bf16((n, k), 1202, 1.5 * k ** -0.5)
    announce("moe t=%d experts=%d top_k=%d inner=%d k=%d" % (t, n, top_k, inner, k))
    y, ids, weights = q4.moe(dev(x), dev(router), *[dev(p) for p in planes], top_k, renormalize=renorm)
    torch.cuda.synchronize()
    want_ids, want_w, w_bound = tw.route_reference(x, router, top_k, renorm)
    assert torch.equal(ids.cpu().long(), want_ids)
    assert ((weights.cpu().double() - want_w).abs() <= w_bound).all()
    want, bound = tw.experts_reference(x, ids.cpu(), weights.cpu(), values)
    tw.close(y, want, bound, "moe")


@pytest.mark.parametrize("t", [1, 2, 6, 8])
def test_layer_ties_and_nan(t):
    n, top_k, inner, k = 70, 5, 64, 128
    planes, values = tw.expert_weights(n, inner, k, 1300)
    router = tw.bf16((n, k), 1301, 0.1)
    router[:] = router[:1]  # all equal: the lowest indexes
    x = tw.bf16((t, k), 1302)
    call = [dev(p) for p in planes]
    y, ids, weights = q4.moe(dev(x), dev(router), *call, top_k)
    assert (ids.cpu() == torch.arange(top_k, dtype=torch.int32)).all()
    want, bound = tw.experts_reference(x, ids.cpu(), weights.cpu(), values)
    tw.close(y, want, bound, "ties")
    router[0, 0] = float("nan")  # the lowest of all, whatever its row
    router[2, 1] = float("-inf") if x[0, 1] > 0 else float("inf")
    y, ids, weights = q4.moe(dev(x[:1]), dev(router), *call, top_k)
    assert ids.cpu().tolist() == [[1, 3, 4, 5, 6]]


# -- row counts around the tiles' sizes --------------------------------------------
@pytest.mark.parametrize("t", [1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 64, 65, 100])
def test_experts_with_every_row_count(t):
    inner, k = 192, 320
    planes, values = tw.expert_weights(3, inner, k, 1400)
    x = tw.bf16((t, k), 1401 + t)
    ids = torch.full((t, 1), 1, dtype=torch.int32)
    weights = torch.rand(t, 1, generator=torch.Generator().manual_seed(t))
    y = experts(x, ids, weights, planes, "one expert")
    want, bound = tw.experts_reference(x, ids, weights, values)
    tw.close(y, want, bound, "one expert")


# few pairs per expert on the whole, many on some; many on the whole, few on some
COUNTS = [[8, 1, 9, 16, 0, 17, 3], [2, 33, 1, 40, 1, 1, 1, 2, 1], [32, 0, 1, 8, 9, 33, 65, 16, 17], [31, 48, 49]]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("inner,k", [(192, 320), (1088, 64)])
def test_experts_with_unequal_counts(counts, inner, k):
    n, t = len(counts), sum(counts)
    planes, values = tw.expert_weights(n, inner, k, 1450)
    x = tw.bf16((t, k), 1451 + t)
    g = torch.Generator().manual_seed(1452)
    chosen = torch.tensor([e for e, c in enumerate(counts) for _ in range(c)], dtype=torch.int32)
    ids = chosen[torch.randperm(t, generator=g)][:, None].contiguous()
    weights = torch.rand(t, 1, generator=g)
    y = experts(x, ids, weights, planes, "counts " + "-".join(map(str, counts)))
    want, bound = tw.experts_reference(x, ids, weights, values)
    tw.close(y, want, bound, "unequal counts")


@pytest.mark.parametrize("t,top_k,n,inner,k", [(2, 1, 2, 64, 8256), (40, 1, 1, 64, 8256), (2, 1, 2, 8256, 64),
                                               (40, 1, 1, 8256, 64), (70, 3, 3, 1088, 1984), (3, 2, 1024, 64, 64),
                                               (50, 2, 300, 64, 64), (600, 1, 2, 64, 64)])
def test_experts_of_long_and_odd_rows(t, top_k, n, inner, k):
    planes, values = tw.expert_weights(n, inner, k, 1500)
    x = tw.bf16((t, k), 1501)
    g = torch.Generator().manual_seed(1502)
    ids = torch.rand(t, max(n, top_k), generator=g).argsort(1)[:, :top_k].to(torch.int32)
    weights = torch.rand(t, top_k, generator=g)
    y = experts(x, ids, weights, planes, "long rows")
    want, bound = tw.experts_reference(x, ids, weights, values)
    tw.close(y, want, bound, "long rows")


@pytest.mark.parametrize("t", [1, 6, 30, 100])
@pytest.mark.parametrize("inner,k", [(192, 320), (128, 256)])
def test_experts_with_shifted_scales(t, inner, k):
    """Scale planes that start in the middle of a dword."""
    planes, values = tw.expert_weights(4, inner, k, 1600)
    moved = [shifted(p) if i & 1 else p for i, p in enumerate(planes)]
    x = tw.bf16((t, k), 1601)
    g = torch.Generator().manual_seed(1602)
    ids = torch.rand(t, 4, generator=g).argsort(1)[:, :2].to(torch.int32)
    weights = torch.rand(t, 2, generator=g)
    y = experts(x, ids, weights, moved, "shifted scales")
    want, bound = tw.experts_reference(x, ids, weights, values)
    tw.close(y, want, bound, "shifted scales")


@pytest.mark.parametrize("t", [2, 12, 40, 100])
@pytest.mark.parametrize("k", [128, 192, 320])
def test_experts_keep_infinities_in_their_rows(t, k):
    """A row's last group ends inside a stage: the next token's values must not come in."""
    planes, _ = tw.expert_weights(4, 192, k, 1700)
    x = tw.bf16((t, k), 1701)
    g = torch.Generator().manual_seed(1702)
    ids = torch.rand(t, 4, generator=g).argsort(1)[:, :2].to(torch.int32)
    weights = torch.rand(t, 2, generator=g)
    clean = experts(x, ids, weights, planes, "finite")
    x[1, 0], x[1, k - 1] = float("nan"), float("inf")
    y = experts(x, ids, weights, planes, "NaN and infinity in token 1")
    assert torch.isnan(y[1]).all()
    rest = (torch.arange(t) != 1).cuda()
    assert torch.equal(y[rest].view(torch.int16), clean[rest].view(torch.int16))


@pytest.mark.parametrize("t", [1, 5, 12, 60, 90])
def test_experts_of_zero_weights(t):
    """Codes of eight are zeros: exact zeros come out, whatever the scales."""
    planes, _ = tw.expert_weights(3, 192, 320, 1800)
    ids = torch.arange(t, dtype=torch.int32).remainder(3)[:, None]
    weights = torch.ones(t, 1)
    x = tw.bf16((t, 320), 1801, 100.0)
    for i in (0, 2, 4):
        zero = list(planes)
        zero[i] = torch.full_like(planes[i], 0x88)
        assert (experts(x, ids, weights, zero, "zero weights") == 0).all()


# -- adapters ------------------------------------------------------------------------
def lora(fmt, n, k, t, adapters, rank, seed, ids=None):
    planes, w64 = tw.weight(fmt, n, k, seed)
    x = tw.bf16((t, k), seed + 1)
    std = float(w64.std())
    a = tw.bf16((adapters, rank, k), seed + 2, k ** -0.5)
    b = tw.bf16((adapters, n, rank), seed + 3, std * (k / rank) ** 0.5)
    g = torch.Generator().manual_seed(seed + 4)
    own = torch.randint(-1, adapters, (t,), generator=g, dtype=torch.int32)
    ids = own if ids is None else ids
    scale = torch.rand(adapters, generator=g) + 0.5
    announce("linear_lora fmt=%d n=%d k=%d t=%d adapters=%d rank=%d" % (fmt, n, k, t, adapters, rank))
    y = q4.linear_lora(dev(x), dev(planes[0]), dev(planes[2]), dev(a), dev(b), dev(ids), dev(scale), fmt=fmt,
                       codes_hi=dev(planes[1]))
    torch.cuda.synchronize()
    tiled = fmt == 0 and q4.q4lin_route(n, k, t) == q4.Q4LIN_ROUTE_TILED
    want, bound = tw.lora_reference(x, w64, a, b, ids, scale, tiled)
    tw.close(y, want, bound, "linear_lora")


# up to 32 tokens (and 4096 rank values) the base product's kernel adds the
# term; beyond, the rank products run in tiles, with K split or not
@pytest.mark.parametrize("fmt", range(6))
@pytest.mark.parametrize("t,rank", [(1, 8), (1, 256), (2, 40), (4, 128), (16, 256), (17, 24), (32, 128), (32, 136),
                                    (33, 16)])
def test_lora_paths(fmt, t, rank):
    lora(fmt, 210, 640, t, 5, rank, 1900 + 10 * t)


@pytest.mark.parametrize("n,k,t,adapters,rank", [(1030, 5120, 64, 3, 128), (260, 4160, 700, 40, 48),
                                                 (2050, 1024, 130, 1, 256), (64, 64, 200, 300, 72),
                                                 (600, 2048, 257, 2, 200), (96, 16448, 2, 3, 16), (96, 20544, 40, 3, 120)])
def test_lora_larger(n, k, t, adapters, rank):
    lora(0, n, k, t, adapters, rank, 2000 + t)


@pytest.mark.parametrize("t,adapters,rank,order", [(33, 40, 128, "mixed"), (130, 3, 40, "falling"), (257, 300, 16, "mixed"),
                                                   (1000, 7, 8, "mixed"), (300, 1, 16, "mixed"), (600, 5, 72, "runs"),
                                                   (4096, 9, 8, "mixed"), (4100, 9, 8, "mixed")])
def test_lora_orders_of_tokens(t, adapters, rank, order):
    """Many tokens whose adapters come in any order, many without one."""
    g = torch.Generator().manual_seed(1901 + t)
    ids = torch.randint(-2, adapters + 1, (t,), generator=g, dtype=torch.int32)
    if order != "mixed":
        ids = ids.sort(descending=order == "falling").values.contiguous()
    lora(0, 100, 128, t, adapters, rank, 2100 + t, ids)
    lora(3, 300, 192, t, adapters, rank, 2200 + t, ids)
