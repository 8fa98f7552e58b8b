"""Activations in 8 bits on the GPU: the norm and the gated quantization that
write them and the product that reads them, against 64-bit references (the
bounds are derived in mx8.py)."""
import pytest
import torch

import mx8
import rounded_once
import weight_only_bit_q4_amd as q4
from gpu_util import announce

pytestmark = pytest.mark.gpu


def bf16(shape, seed, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(torch.bfloat16)


# -- norm and quantization -----------------------------------------------------
NORM = [(1, 64), (1, 5120), (3, 192), (2, 8192), (1, 8256), (5, 17408), (1, 40000 // 64 * 64), (600, 256), (513, 5120),
        (1024, 8256), (2, 1 << 17)]


@pytest.mark.parametrize("t,k", NORM)
@pytest.mark.parametrize("form", ["plain", "residual", "weight", "both"])
def test_norm(t, k, form):
    if t * k > 1 << 20 and form in ("plain", "weight"):
        pytest.skip("the largest sizes once")
    x, w = bf16((t, k), 1 + t), bf16((k,), 2 + t)
    r = bf16((t, k), 3 + t, 4.0) if form in ("residual", "both") else None
    w = w if form in ("weight", "both") else None
    announce("rmsnorm_mx8 t=%d k=%d %s" % (t, k, form))
    out = q4.rmsnorm_mx8(x.cuda(), w.cuda() if w is not None else None, 1e-5,
                         residual=r.cuda() if r is not None else None)
    torch.cuda.synchronize()
    v = x.double() + (r.double() if r is not None else 0)
    y = v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-5) * (w.double() if w is not None else 1)
    mx8.check_mx8(out[0].cpu(), out[1].cpu(), y, mx8.FORM_ERROR["norm"], "norm")
    if r is not None:
        assert torch.equal(out[2].cpu(), v.float().to(torch.bfloat16))
    else:
        assert len(out) == 2


@pytest.mark.parametrize("k", [256, 5120, 40000 // 64 * 64])
def test_norm_of_very_large_and_small_rows(k):
    """Squares that leave binary32 on either side: the formula holds where the values are finite."""
    x = bf16((5, k), k).double()
    x = (x * torch.tensor([1e30, 3e37, 1e-25, 1e-36, 1.0], dtype=torch.float64)[:, None]).to(torch.bfloat16)
    values, scales = (v.cpu() for v in q4.rmsnorm_mx8(x.cuda(), eps=0.0))
    v = x.double()
    y = v / torch.sqrt(v.square().mean(-1, keepdim=True))
    # (1 / sqrt near 2^-127 is subnormal: 2^-21 of it at worst)
    mx8.check_mx8(values, scales, y, mx8.FORM_ERROR["norm"] + 2.0 ** -20, "norm of rows of any size")


def test_norm_in_place():
    x, r = bf16((9, 1024), 1).cuda(), bf16((9, 1024), 2).cuda()
    want = q4.rmsnorm_mx8(x, None, residual=r)
    for k, which in ((1024, "residual"), (1024, "x"), (1 << 16, "residual"), (1 << 16, "x")):
        if k != 1024:
            x, r = bf16((2, k), 3).cuda(), bf16((2, k), 4).cuda()
            want = q4.rmsnorm_mx8(x, None, residual=r)
        a, b = x.clone(), r.clone()
        h = a if which == "x" else b
        got = q4.rmsnorm_mx8(a, None, residual=b, h=h)
        assert got[2] is h
        for u, v in zip(got, want):
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


@pytest.mark.parametrize("t,k", [(1, 64), (1, 6144), (9, 17408), (77, 320), (700, 2048), (40000, 64)])
@pytest.mark.parametrize("form", ["plain", "gated", "halves"])
def test_quantize(t, k, form):
    announce("quantize_mx8 t=%d k=%d %s" % (t, k, form))
    both = bf16((t, 2 * k), t + k, 2.0)
    gate, x = both[:, :k], both[:, k:]
    if form == "halves":
        d = both.cuda()
        got = q4.quantize_mx8(d[:, k:], gate=d[:, :k])
    else:
        got = q4.quantize_mx8(x.contiguous().cuda(), gate=gate.contiguous().cuda() if form == "gated" else None)
    torch.cuda.synchronize()
    y = x.double()
    if form != "plain":
        y = y * gate.double() / (1 + torch.exp(-gate.double()))
    mx8.check_mx8(got[0].cpu(), got[1].cpu(), y, mx8.FORM_ERROR["quant" if form == "plain" else "gated"], form)


def test_block_edges():
    """Zeros, the border 448, magnitudes of bf16's ends, infinities and NaN: each block by itself."""
    blocks = torch.zeros(10, 32)
    blocks[1, 3] = 448.0
    blocks[2, 0], blocks[2, 31] = 450.0, -1.0
    blocks[3] = 3.3e38
    blocks[4] = 1e-38
    blocks[5, 7] = 9.2e-41  # (subnormal)
    blocks[6, 1], blocks[6, 2] = float("inf"), 1.0
    blocks[7, 1], blocks[7, 2] = float("nan"), 1.0
    blocks[8, 5] = -448.0 * 2.0 ** -20
    blocks[9, 9], blocks[9, 8] = 1.0, 2.0 ** -12
    x = blocks.to(torch.bfloat16).view(2, 160)
    x = torch.nn.functional.pad(x, (0, 32)).contiguous()  # K = 192
    v, s = (u.cpu() for u in q4.quantize_mx8(x.cuda()))
    byte = s.view(torch.uint8)
    for i in range(10):
        row, col = i // 5, i % 5
        want, got = x[row, 32 * col:32 * col + 32].double(), v[row, 32 * col:32 * col + 32]
        if i in (6, 7):
            assert byte[row, col] == 255 and bool(torch.isnan(mx8.e4m3(got)).all())
            continue
        mx8.check_mx8(got[None], s[row:row + 1, col:col + 1], want[None], 0.0, "block %d" % i)
    assert byte[0, 0] == 0 and byte[0, 1] == 127 and byte[0, 2] == 128
    n, e = (u.cpu() for u in q4.rmsnorm_mx8(x[:1].contiguous().cuda()))  # an infinity nowhere in this row's first half
    assert bool((e.view(torch.uint8) < 255).all())
    n, e = (u.cpu() for u in q4.rmsnorm_mx8(torch.stack((x[1], x[1] * 0 + 1)).nan_to_num(1.0, 1e30, 0).cuda()))
    assert bool((e.view(torch.uint8) < 255).all()), "finite rows"
    bad = bf16((3, 256), 5)
    bad[1, 17] = float("nan")
    e = q4.rmsnorm_mx8(bad.cuda())[1].view(torch.uint8).cpu()
    assert bool((e[1] == 255).all()) and bool((e[0] < 255).all()) and bool((e[2] < 255).all())


# -- the product ------------------------------------------------------------------
LINEAR = [  # (n, k, t): every kernel and tile; odd rows, groups and tokens
    (1, 64, 1), (33, 64, 1), (512, 1024, 1), (517, 1216, 2), (1000, 2048, 5), (31, 4096, 8), (6144, 512, 16),
    (300, 5120, 17), (64, 20480, 32), (8192, 256, 31), (9001, 320, 3), (16400, 128, 20), (17000, 192, 40),
    (700, 1984, 33), (333, 640, 64), (8300, 256, 64), (500, 2048, 65), (1001, 192, 100), (16385, 64, 128),
    (640, 256, 129), (192, 64, 129), (385, 1152, 200), (1030, 320, 300), (100, 8192, 256), (2048, 512, 600),
    (7703, 576, 257), (5, 128, 2000), (129, 448, 4097),
]


def run_linear(n, k, t, seed, spread=0, residual=False):
    values, x_scales = mx8.random_mx8(t, k, seed, spread)
    codes, scales = mx8.random_weight(n, k, seed + 1)
    r = bf16((t, n), seed + 2) if residual else None
    announce("linear_mx8 n=%d k=%d t=%d" % (n, k, t))
    d = [v.cuda() for v in (values, x_scales, codes, scales)]
    y = q4.linear_mx8(*d, residual=r.cuda() if residual else None)
    torch.cuda.synchronize()
    want, bound = mx8.linear(*d, residual=r.cuda() if residual else None)
    return y, want, bound


@pytest.mark.parametrize("n,k,t", LINEAR)
def test_linear(n, k, t):
    y, want, bound = run_linear(n, k, t, n + t)
    mx8.close(y, want, bound, "linear_mx8")
    if n * t >= 1000:
        rounded_once.rounded_once(y, want.cpu(), "linear_mx8")


@pytest.mark.parametrize("n,k,t", [(300, 512, 1), (300, 512, 30), (1000, 448, 70), (400, 320, 300), (100, 4096, 200)])
def test_linear_add_and_wide_exponents(n, k, t):
    y, want, bound = run_linear(n, k, t, 5 * n + t, spread=20, residual=True)
    mx8.close(y, want, bound, "linear_mx8 with a residual")


@pytest.mark.parametrize("t", [1, 20, 60, 100, 200])
def test_linear_add_in_place(t):
    values, x_scales = (v.cuda() for v in mx8.random_mx8(t, 512, t))
    codes, scales = (v.cuda() for v in mx8.random_weight(200, 512, t + 1))
    r = bf16((t, 200), t + 2).cuda()
    want = q4.linear_mx8(values, x_scales, codes, scales, residual=r)
    y = r.clone()
    assert q4.linear_mx8(values, x_scales, codes, scales, residual=y, y=y) is y
    assert torch.equal(y, want)


@pytest.mark.parametrize("t", [1, 33, 130])
def test_linear_all_eight_codes_are_zero_weights(t):
    """The codes' offset and the codes go through the same instruction; one exponent for all keeps every sum exact."""
    values, x_scales = (v.cuda() for v in mx8.random_mx8(t, 576, 3))
    codes = torch.full((70, 288), 0x88, dtype=torch.uint8, device="cuda")
    scales = torch.ones(70, 9, dtype=torch.float16, device="cuda")
    x_scales.view(torch.uint8).fill_(127)
    assert not bool(q4.linear_mx8(values, x_scales, codes, scales).any())


@pytest.mark.parametrize("t", [3, 40, 140])
def test_linear_exact_integers(t):
    """Small whole numbers: every product and sum is exact, so the outputs are."""
    g = torch.Generator().manual_seed(t)
    x = torch.randint(-7, 8, (t, 320), generator=g).float()
    values = x.to(torch.float8_e4m3fn)
    x_scales = torch.full((t, 10), 127, dtype=torch.uint8)
    codes, _ = mx8.random_weight(90, 320, t)
    scales = torch.randint(1, 4, (90, 5), generator=g).to(torch.float16)
    y = q4.linear_mx8(*(v.cuda() for v in (values, x_scales, codes, scales)))
    q, s = mx8.weight64(codes, scales)
    want = x.double() @ (q * s[..., None]).flatten(1).t()
    assert torch.equal(y.cpu(), want.to(torch.bfloat16))


@pytest.mark.parametrize("t", [5, 50, 120, 200])
def test_linear_nan_stays_in_its_token(t):
    values, x_scales = mx8.random_mx8(t, 512, 9)
    codes, scales = (v.cuda() for v in mx8.random_weight(100, 512, 10))
    want = q4.linear_mx8(values.cuda(), x_scales.cuda(), codes, scales)
    values.view(torch.uint8)[t // 2, 100] = 0x7F
    x_scales.view(torch.uint8)[t - 1, 3] = 255
    y = q4.linear_mx8(values.cuda(), x_scales.cuda(), codes, scales)
    bad = torch.isnan(y).all(1).cpu()
    assert bad.nonzero().flatten().tolist() == [t // 2, t - 1]
    assert torch.equal(y[~bad.cuda()], want[~bad.cuda()])


@pytest.mark.parametrize("t", [2, 48, 128, 160])
def test_linear_unaligned_scales_and_untouched_surroundings(t):
    n, k = 130, 448  # (an odd number of groups: rows of scales begin on two bytes)
    values, x_scales = mx8.random_mx8(t, k, 21)
    codes, scales = mx8.random_weight(n, k, 22)
    want = q4.linear_mx8(*(v.cuda() for v in (values, x_scales, codes, scales)))
    xs = torch.zeros(2 + x_scales.numel(), dtype=torch.uint8, device="cuda")
    xs[2:] = x_scales.view(torch.uint8).flatten().cuda()
    ws = torch.zeros(1 + scales.numel(), dtype=torch.float16, device="cuda")
    ws[1:] = scales.flatten().cuda()
    room = torch.full((t + 2, n), 7.0, dtype=torch.bfloat16, device="cuda")
    y = q4.linear_mx8(values.cuda(), xs[2:].view(t, -1), codes.cuda(), ws[1:].view(n, -1), y=room[1:t + 1])
    assert torch.equal(y, want)
    assert bool((room[0] == 7).all()) and bool((room[t + 1] == 7).all())


@pytest.mark.parametrize("t", [1, 30, 64, 100, 300])
def test_linear_repeats_to_the_bit(t):
    d = [v.cuda() for v in (*mx8.random_mx8(t, 1024, 31), *mx8.random_weight(600, 1024, 32))]
    want = q4.linear_mx8(*d)
    for _ in range(5):
        assert torch.equal(q4.linear_mx8(*d), want)


def test_a_layer_in_a_graph():
    """Norm, gate and up product, gated quantization and down product as a layer runs them, captured and replayed with
    other inputs, each replay against the eager calls."""
    t, k, inner = 5, 512, 768
    up_c, up_s = (v.cuda() for v in mx8.random_weight(2 * inner, k, 41))
    down_c, down_s = (v.cuda() for v in mx8.random_weight(k, inner, 42))
    w = bf16((k,), 43).cuda()
    x, r = torch.zeros(t, k, dtype=torch.bfloat16, device="cuda"), torch.zeros(t, k, dtype=torch.bfloat16, device="cuda")

    def layer():
        v, s, h = q4.rmsnorm_mx8(x, w, residual=r)
        both = q4.linear_mx8(v, s, up_c, up_s)
        v, s = q4.quantize_mx8(both[:, inner:], gate=both[:, :inner])
        return q4.linear_mx8(v, s, down_c, down_s, residual=h)
    x.copy_(bf16((t, k), 44))
    r.copy_(bf16((t, k), 45))
    announce("a layer of 8-bit activations in a graph")
    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer()
    for i in range(4):
        x.copy_(bf16((t, k), 50 + i))
        r.copy_(bf16((t, k), 60 + i))
        want = layer()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
    # the whole layer against 64 bits: three roundings to E4M3 and bf16 on the way
    v = x.double() + r.double()
    n = v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w.double()
    q, s = mx8.weight64(up_c, up_s)
    both = n @ (q * s[..., None]).flatten(1).t()
    g = both[:, :inner] * torch.sigmoid(both[:, :inner]) * both[:, inner:]
    q, s = mx8.weight64(down_c, down_s)
    z = g @ (q * s[..., None]).flatten(1).t() + v
    # E4M3's error is 2^-4 of a value at most, 2^-5 or less on average: twice, and as much again through the gate
    assert float((y.double() - z).norm() / z.norm()) < 4 * 2.0 ** -5
