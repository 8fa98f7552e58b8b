"""Refusals of the operators around 8-bit activations and log probabilities:
every call here returns from host-side checks (no GPU needed)."""
import pytest
import torch

import weight_only_bit_q4_amd as q

P = 0x1000  # an aligned address that nothing reads


def norm(x=P, r=P, w=P, h=P, v=P, s=P, k=128, t=2):
    return q.q4lin_rmsnorm_mx8(x, r, w, 1e-6, h, v, s, k, t, 0)


def quant(x=P, xs=128, g=P, gs=128, v=P, s=P, k=128, t=2):
    return q.q4lin_quantize_mx8(x, xs, g, gs, v, s, k, t, 0)


def linear(v=P, e=P, c=P, s=P, r=P, y=P, n=96, k=128, t=2, ws=P, wb=1 << 40):
    return q.q4lin_linear_mx8(v, e, c, s, r, y, n, k, t, ws, wb, 0)


def logprobs(l=P, f32=1, stride=500, tok=P, lp=P, en=P, tp=P, ti=P, n=500, t=2, top=3, ws=P, wb=1 << 40):
    return q.q4lin_logprobs(l, f32, stride, tok, lp, en, tp, ti, n, t, top, ws, wb, 0)


def scores(x=P, e=P, c=P, s=P, tok=P, lp=P, en=P, tp=P, ti=P, n=96, k=128, t=2, top=3, ws=P, wb=1 << 40):
    return q.q4lin_linear_logprobs(x, e, c, s, tok, lp, en, tp, ti, n, k, t, top, ws, wb, 0)


@pytest.mark.parametrize("call,name", [(norm, "x"), (norm, "v"), (norm, "s"), (norm, "h"), (quant, "x"), (quant, "v"),
                                       (quant, "s"), (linear, "v"), (linear, "e"), (linear, "c"), (linear, "s"),
                                       (linear, "y"), (logprobs, "l"), (logprobs, "tok"), (logprobs, "lp"),
                                       (logprobs, "tp"), (logprobs, "ti"), (logprobs, "ws"), (scores, "x"),
                                       (scores, "c"), (scores, "s"), (scores, "tok"), (scores, "lp"), (scores, "tp"),
                                       (scores, "ti"), (scores, "ws")])
def test_null(call, name):
    assert call(**{name: None}) == q.Q4LIN_E_NULL


@pytest.mark.parametrize("call,name,off", [
    (norm, "x", 8), (norm, "r", 8), (norm, "w", 8), (norm, "h", 8), (norm, "v", 8), (quant, "x", 8), (quant, "g", 8),
    (quant, "v", 8), (linear, "v", 8), (linear, "e", 1), (linear, "c", 8), (linear, "s", 1), (linear, "r", 1),
    (linear, "y", 1), (logprobs, "l", 2), (logprobs, "tok", 2), (logprobs, "lp", 2), (logprobs, "en", 2),
    (logprobs, "tp", 2), (logprobs, "ti", 2), (logprobs, "ws", 128), (scores, "x", 8), (scores, "c", 8),
    (scores, "s", 1), (scores, "en", 2), (scores, "ws", 128)])
def test_misaligned(call, name, off):
    assert call(**{name: P + off}) == q.Q4LIN_E_ALIGN


@pytest.mark.parametrize("call,args", [
    (norm, {"k": 96}), (norm, {"k": 0}), (norm, {"t": -1}), (norm, {"k": (1 << 20) + 64}), (norm, {"t": (1 << 21) + 1}),
    (quant, {"k": 32}), (quant, {"xs": 132}), (quant, {"gs": -128}), (quant, {"xs": 1 << 40}), (quant, {"xs": 1 << 62}),
    (quant, {"gs": 1 << 62}), (linear, {"k": 100}),
    (linear, {"n": -1}), (linear, {"n": (1 << 24) + 1}), (logprobs, {"n": 0}), (logprobs, {"top": 33}),
    (logprobs, {"top": -1}), (logprobs, {"n": 2, "top": 3}), (logprobs, {"t": -1}), (logprobs, {"stride": -1}),
    (logprobs, {"stride": 1 << 61}),
    (logprobs, {"n": (1 << 24) + 1}), (scores, {"n": 0}), (scores, {"n": 2}), (scores, {"k": 100}), (scores, {"top": 40})])
def test_shape(call, args):
    assert call(**args) == q.Q4LIN_E_SHAPE


def test_bf16_logits_need_two_bytes_only():
    assert logprobs(f32=0, l=P + 1) == q.Q4LIN_E_ALIGN
    assert logprobs(f32=0, l=P + 2, ws=None) == q.Q4LIN_E_NULL  # (past the alignment)


def test_empty_calls_touch_nothing():
    assert norm(x=None, t=0) == quant(x=None, t=0) == linear(v=None, t=0) == linear(v=None, n=0) == q.Q4LIN_OK
    assert logprobs(l=None, t=0) == scores(x=None, t=0) == q.Q4LIN_OK


def test_workspaces():
    assert q.q4lin_linear_mx8_workspace_bytes(96, 128, 100) == 0
    assert linear(t=100, ws=None, wb=0, y=None) == q.Q4LIN_E_NULL
    need = q.q4lin_linear_mx8_workspace_bytes(512, 8192, 200)
    assert need > 0
    assert linear(n=512, k=8192, t=200, wb=need - 1) == q.Q4LIN_E_WORKSPACE
    assert linear(n=512, k=8192, t=200, ws=None) == q.Q4LIN_E_NULL
    assert linear(n=512, k=8192, t=200, ws=P + 128) == q.Q4LIN_E_ALIGN
    assert logprobs(wb=q.q4lin_logprobs_workspace_bytes(500, 2, 3) - 1) == q.Q4LIN_E_WORKSPACE
    assert scores(wb=q.q4lin_linear_logprobs_workspace_bytes(96, 128, 2, 3) - 1) == q.Q4LIN_E_WORKSPACE
    assert q.q4lin_linear_logprobs_workspace_bytes(96, 128, 2, 97) == -q.Q4LIN_E_SHAPE
    assert q.q4lin_logprobs_workspace_bytes(96, 2, 33) == -q.Q4LIN_E_SHAPE
    assert q.q4lin_linear_mx8_workspace_bytes(96, 100, 2) == -q.Q4LIN_E_SHAPE


def test_scoring_holds_a_run_of_tokens_only():
    """The logits' room does not grow with the prompt, only the activations' does."""
    one = q.q4lin_linear_logprobs_workspace_bytes(131072, 512, 256, 5)
    assert q.q4lin_linear_logprobs_workspace_bytes(131072, 512, 256 * 64, 5) == one + (2 * 512 + 4 * 8) * 256 * 63


@pytest.mark.parametrize("k", [64, 4096, 20480, 65536, 1 << 17])
@pytest.mark.parametrize("t", [1, 2, 5, 31, 33, 127, 129, 1000, 1025])
def test_scoring_takes_every_size(k, t):
    assert q.q4lin_linear_logprobs_workspace_bytes(1000, k, t, 5) > 0
    assert q.q4lin_linear_logprobs_workspace_bytes(1000, (1 << 17) + 64, t, 5) == -q.Q4LIN_E_SHAPE


# -- the torch calls ---------------------------------------------------------------
def arguments():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    v, e = torch.zeros(3, 128, dtype=torch.uint8), torch.zeros(3, 4, dtype=torch.uint8)
    c, s = torch.zeros(10, 64, dtype=torch.uint8), torch.zeros(10, 2, dtype=torch.float16)
    tok = torch.zeros(3, dtype=torch.int32)
    return {
        "rmsnorm_mx8": (q.rmsnorm_mx8, dict(x=bf(3, 128), weight=bf(128), residual=bf(3, 128), h=bf(3, 128))),
        "quantize_mx8": (q.quantize_mx8, dict(x=bf(3, 128), gate=bf(3, 128))),
        "linear_mx8": (q.linear_mx8, dict(values=v, x_scales=e, codes=c, scales=s, residual=bf(3, 10), y=bf(3, 10))),
        "logprobs": (q.logprobs, dict(logits=bf(3, 50), tokens=tok)),
        "linear_logprobs": (q.linear_logprobs, dict(x=v, x_scales=e, codes=c, scales=s, tokens=tok)),
    }


CALLS = list(arguments())


@pytest.mark.parametrize("name", CALLS)
def test_host_memory_is_refused(name):
    call, kw = arguments()[name]
    with pytest.raises(ValueError, match="GPU"):
        call(**kw)


@pytest.mark.parametrize("name", CALLS)
def test_other_types_and_shapes_are_refused(name):
    call, kw = arguments()[name]
    for arg, ten in kw.items():
        other = torch.float64 if ten.dtype != torch.float64 else torch.float32
        with pytest.raises(ValueError, match="GPU" if arg in ("y", "h") else arg + " must be a"):
            call(**dict(kw, **{arg: ten.to(other)}))
        if arg in ("x", "values", "logits", "codes"):
            continue  # (these give the sizes)
        with pytest.raises(ValueError):
            call(**dict(kw, **{arg: ten[:-1]}))


def test_other_device_is_refused():
    for name in CALLS:
        call, kw = arguments()[name]
        for arg, ten in kw.items():
            with pytest.raises(ValueError):
                call(**dict(kw, **{arg: ten.to("meta")}))


def test_h_without_a_residual():
    call, kw = arguments()["rmsnorm_mx8"]
    with pytest.raises(ValueError, match="residual"):
        call(**dict(kw, residual=None))


def test_rows_must_be_contiguous():
    x = torch.zeros(128, 3, dtype=torch.bfloat16).t()
    with pytest.raises(ValueError, match="contiguous"):
        q.quantize_mx8(x)
    with pytest.raises(ValueError, match="contiguous"):
        q.logprobs(x)
    with pytest.raises(ValueError, match="contiguous"):
        q.rmsnorm_mx8(x)
