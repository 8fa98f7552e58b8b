"""Values at the ends of the range in the operators in which each token picks
its own weights: activations whose products with the codes leave binary32
although the exact sums may not.  The base product beside adapters gives what
it gives alone, on every path; the bounds are those of token_weights.py."""
import pytest
import torch

import token_weights as tw
import weight_only_bit_q4_amd as q4
from gpu_util import announce


pytestmark = pytest.mark.gpu

LARGEST = torch.finfo(torch.bfloat16).max
OVER = LARGEST * (1 + 2.0 ** -9)  # half a step past the largest bf16: rounds to infinity


def dev(v):
    return None if v is None else v.cuda()


def check(got, want, bound, what):
    """As tw.close's element bounds, where a value past the bf16 range is an
    infinity (either side within the bound of the border)."""
    got, sign = got.double().cpu(), torch.sign(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "%s: NaN elsewhere than in the reference" % what
    inf_ok = (want.abs() + bound >= OVER) & (got == sign * float("inf"))
    finite_ok = torch.isfinite(got) & ((got - want).abs() <= bound)
    bad = ~(inf_ok | finite_ok | torch.isnan(want))
    assert not bad.any(), "%s: %d of %d outside their bounds" % (what, int(bad.sum()), bad.numel())


def case(fmt, n, k, t, rank, seed):
    planes, w64 = tw.weight(fmt, n, k, seed)
    x = tw.bf16((t, k), seed + 1)
    std = float(w64.std())
    a = tw.bf16((3, rank, k), seed + 2, k ** -0.5)
    b = tw.bf16((3, n, rank), seed + 3, std * (k / rank) ** 0.5)
    g = torch.Generator().manual_seed(seed + 4)
    ids = torch.randint(-1, 3, (t,), generator=g, dtype=torch.int32)
    ids[0] = -1  # the base weight alone
    return planes, w64, x, a, b, ids, torch.rand(3, generator=g) + 0.5


def run(fmt, planes, x, a, b, ids, scale, what):
    announce("linear_lora %s fmt=%d n=%d k=%d t=%d rank=%d" % (what, fmt, planes[0].shape[0], x.shape[1], x.shape[0],
                                                               a.shape[1]))
    y = q4.linear_lora(dev(x), dev(planes[0]), dev(planes[2]), dev(a), dev(b), dev(ids), dev(scale), fmt=fmt,
                       codes_hi=dev(planes[1]))
    torch.cuda.synchronize()
    return y


def is_tiled(fmt, n, k, t):
    return fmt == 0 and q4.q4lin_route(n, k, t) == q4.Q4LIN_ROUTE_TILED


# every way in which the base product's sums come to the adapters' term
PATHS = [(1, 16), (1, 256), (5, 16), (5, 200), (20, 24), (40, 16), (40, 136), (200, 24), (300, 8)]


@pytest.mark.parametrize("fmt", range(6))
@pytest.mark.parametrize("t,rank", PATHS)
def test_lora_of_large_activations(fmt, t, rank):
    """Eight values from 2^119 in one scale group: (128 + q) x overflows, (q - 8) s x does not."""
    n, k = 210, 640
    planes, w64, x, a, b, ids, scale = case(fmt, n, k, t, rank, 4000 + t + rank)
    g = torch.Generator().manual_seed(4001)
    x[::2, 67:75] = 2.0 ** 119 * torch.randint(1, 3, ((t + 1) // 2, 8), generator=g).to(torch.bfloat16)
    y = run(fmt, planes, x, a, b, ids, scale, "large activations")
    want, bound = tw.lora_reference(x, w64, a, b, ids, scale, is_tiled(fmt, n, k, t))
    check(y, want, bound, "large activations")


@pytest.mark.parametrize("fmt", range(6))
@pytest.mark.parametrize("t,rank", PATHS)
def test_lora_of_sums_that_cancel(fmt, t, rank):
    """Terms past the binary32 range whose exact sum is zero or small."""
    n, k = 130, 512
    planes, w64, x, a, b, ids, scale = case(fmt, n, k, t, rank, 4100 + t + rank)
    if fmt in (0, 5):  # a row whose terms are about 2^132 and cancel
        if fmt == 0:
            planes[0][7, 32:36], planes[2].view(torch.float16)[7, 1] = 0xFF, 1024.0
            w64[7, 64:128] = (torch.stack((planes[0][7, 32:64] & 15, planes[0][7, 32:64] >> 4), -1).flatten().double() -
                              8) * 1024.0
        else:
            planes[0].view(torch.bfloat16)[7, 64:72] = 64.0
            w64[7, 64:72] = 64.0
        a[:, :, 64:72] = 0.0
        x[0, 64:72] = 1.5 * 2.0 ** 126 * torch.tensor([1, 1, 1, 1, -1, -1, -1, -1]).to(torch.bfloat16)
    x[::2, 256:262] = 1.5 * 2.0 ** 126 * torch.tensor([1, 1, 1, -1, -1, -1]).to(torch.bfloat16)
    a[:, :, 256:262] *= 2.0 ** -20  # (the rank values stay within binary32)
    y = run(fmt, planes, x, a, b, ids, scale, "sums that cancel")
    want, bound = tw.lora_reference(x, w64, a, b, ids, scale, is_tiled(fmt, n, k, t))
    check(y, want, bound, "sums that cancel")


@pytest.mark.parametrize("fmt", range(1, 6))
@pytest.mark.parametrize("t,rank", PATHS)
def test_lora_infinite_activations(fmt, t, rank):
    """An infinite activation beside the base weight alone: what linear_fmt gives for it."""
    n, k = 130, 512
    planes, w64, x, a, b, ids, scale = case(fmt, n, k, t, rank, 4200 + t + rank)
    x[0, 100] = float("inf")
    y = run(fmt, planes, x, a, b, ids, scale, "infinite activation")
    alone = q4.linear_fmt(fmt, dev(x[:1]), dev(planes[0]), dev(planes[1]), dev(planes[2]))
    want, bound = tw.lora_reference(x, w64, a, b, ids, scale, False)
    check(y, want, bound, "infinite activation")
    assert torch.equal(y[0].isinf(), alone[0].isinf()) and torch.equal(y[0].isnan(), alone[0].isnan())


@pytest.mark.parametrize("n,k,t,rank", [(96, 5120, 300, 16), (1030, 1024, 1100, 32)])
def test_lora_of_large_activations_on_many_tokens(n, k, t, rank):
    """The many-token route with and without a K split, four rows a thread, tokens by adapter."""
    planes, w64, x, a, b, ids, scale = case(0, n, k, t, rank, 4300 + t)
    x[5::7, 67:75] = 2.0 ** 120
    x[::64, k - 3:] = 1.5 * 2.0 ** 126
    a[:, :, k - 3:] *= 2.0 ** -20
    y = run(0, planes, x, a, b, ids, scale, "many tokens")
    want, bound = tw.lora_reference(x, w64, a, b, ids, scale, is_tiled(0, n, k, t))
    check(y, want, bound, "many tokens")


# both sides of where the adapters' term changes its path, one and four rows a thread
@pytest.mark.parametrize("fmt,n,t,rank", [(0, 200, 2, 16), (0, 200, 16, 64), (0, 200, 32, 128), (0, 200, 32, 136),
                                          (0, 200, 33, 16), (0, 200, 40, 40), (0, 200, 200, 24), (0, 1040, 1100, 48),
                                          (3, 200, 1, 16), (5, 200, 1, 200), (4, 200, 20, 24), (1, 200, 40, 256)])
def test_lora_infinities_in_b_and_a(fmt, n, t, rank):
    """An infinity in B is one of its row's outputs, with its sign; one in A is one of every output."""
    planes, w64, x, a, b, ids, scale = case(fmt, n, 256, t, rank, 4400 + t + rank)
    ids[t // 2:] = 1
    clean = run(fmt, planes, x, a, b, ids, scale, "finite")
    b[1, 5, 2] = float("inf")
    b[1, 9, 3] = -float("inf")
    b[1, 11, 0], b[1, 11, 1] = float("inf"), -float("inf")  # (an infinity or NaN, by the rank values' signs)
    y = run(fmt, planes, x, a, b, ids, scale, "infinities in B").cpu()
    want, _ = tw.lora_reference(x, w64, a, b, ids, scale, False)
    edge = ~torch.isfinite(want)
    assert edge.any() and edge.sum(1).max() == 3
    assert torch.equal(y[edge].double().nan_to_num(nan=7.0), want[edge].nan_to_num(nan=7.0))
    assert torch.equal(y[~edge].view(torch.int16), clean.cpu()[~edge].view(torch.int16))
    a[1, 7, 100] = -float("inf")
    y = run(fmt, planes, x, a, b, ids, scale, "infinities in A and B").cpu()
    want, _ = tw.lora_reference(x, w64, a, b, ids, scale, False)
    assert torch.equal(y[ids == 1].double().nan_to_num(nan=7.0), want[ids == 1].nan_to_num(nan=7.0))


# -- experts: within the range that the header states, and past it -------------------
def layer_case(t, experts=6, top_k=2, inner=192, k=320, seed=4500):
    planes, values = tw.expert_weights(experts, inner, k, seed)
    x = tw.bf16((t, k), seed + t)
    g = torch.Generator().manual_seed(seed + 1)
    ids = torch.rand(t, experts, generator=g).argsort(1)[:, :top_k].to(torch.int32)
    return planes, values, x, ids, torch.rand(t, top_k, generator=g)


def run_experts(planes, x, ids, weights, what):
    announce("moe_experts %s t=%d" % (what, x.shape[0]))
    y = q4.moe_experts(x.cuda(), ids.cuda(), weights.cuda(), *[p.cuda() for p in planes])
    torch.cuda.synchronize()
    return y


@pytest.mark.parametrize("t", [1, 4, 12, 40, 90])
@pytest.mark.parametrize("power", [-60, -20, 20, 50])
def test_experts_of_large_and_small_activations(t, power):
    """Gated values of up to about 2^105, and down to the subnormals."""
    planes, values, x, ids, weights = layer_case(t)
    x = (x.double() * 2.0 ** power).to(torch.bfloat16)
    y = run_experts(planes, x, ids, weights, "2^%d" % power)
    want, bound = tw.experts_reference(x, ids, weights, values)
    # (a gated value below the smallest normal bf16 keeps that one's last place)
    check(y, want, bound + 192 * 2.0 ** -133, "large and small activations")


@pytest.mark.parametrize("t", [2, 4, 12, 40, 90])
@pytest.mark.parametrize("value", [2.0 ** 120, float("inf"), float("nan")])
def test_experts_past_the_range(t, value):
    """The row of a token with such values is not finite, all others as without them."""
    planes, values, x, ids, weights = layer_case(t)
    clean = run_experts(planes, x, ids, weights, "finite").cpu()
    x[1, 64:128] = value
    y = run_experts(planes, x, ids, weights, "past the range").cpu()
    assert not torch.isfinite(y[1].float()).any()
    rest = torch.arange(t) != 1
    assert torch.equal(y[rest].view(torch.int16), clean[rest].view(torch.int16))
