"""weight_only_bit_q4_amd -- the Q4_G64_FP16 weight-only Linear on MI355X.

Python binding of the C ABI declared in ``include/q4lin.h``.  The functions
carry the C names and only marshal arguments; every step of the op runs in the
HIP kernels of ``libq4lin.so``.  The library is loaded on the first call
(``load()``) and a missing library raises at once (build it with
``python -m weight_only_bit_q4_amd.build``); there is no fallback path.  The
seeded input generators in ``weight_only_bit_q4_amd.inputs`` import without
it.

``linear`` is a convenience over torch tensors (device memory and streams
only): it checks dtypes/shapes, allocates the output and workspace when the
caller does not pass them, and calls ``q4lin_linear`` on the current stream.
The other operators have the like: ``rmsnorm_mx8``, ``quantize_mx8`` and
``linear_mx8`` for activations in 8 bits, ``logprobs`` and ``linear_logprobs``
for what follows the last product.
"""
from __future__ import annotations

import ctypes
import functools
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libq4lin.so")

Q4LIN_OK = 0
Q4LIN_E_NULL = 1
Q4LIN_E_SHAPE = 2
Q4LIN_E_ALIGN = 3
Q4LIN_E_WORKSPACE = 4
Q4LIN_E_LAUNCH = 5
Q4LIN_E_FORMAT = 6

Q4LIN_FMT_Q4G64_F16S = 0
Q4LIN_FMT_Q5G64_F16S = 1
Q4LIN_FMT_Q6G64_F16S = 2
Q4LIN_FMT_W8G32_F16S = 3
Q4LIN_FMT_NVFP4 = 4
Q4LIN_FMT_BF16 = 5

Q4LIN_ROUTE_NONE = 0
Q4LIN_ROUTE_GEMV = 1
Q4LIN_ROUTE_SKINNY = 2
Q4LIN_ROUTE_TILED = 3
Q4LIN_ROUTE_DECODE = 4
Q4LIN_ROUTE_MID = 5

EXPORTED = ("q4lin_workspace_bytes", "q4lin_linear", "q4lin_linear_add", "q4lin_linear_pair",
            "q4lin_pair_workspace_bytes", "q4lin_linear_swiglu", "q4lin_swiglu_workspace_bytes",
            "q4lin_status_string", "q4lin_route", "q4lin_version", "q4lin_linear_noalloc",
            "q4lin_noalloc_scratch_bytes", "q4lin_linear_fmt", "q4lin_fmt_weight_bytes",
            "q4lin_fmt_workspace_bytes", "q4lin_linear_lora", "q4lin_lora_workspace_bytes", "q4lin_moe",
            "q4lin_moe_route", "q4lin_moe_experts", "q4lin_moe_workspace_bytes", "q4lin_rmsnorm_mx8",
            "q4lin_quantize_mx8", "q4lin_linear_mx8", "q4lin_linear_mx8_workspace_bytes", "q4lin_logprobs",
            "q4lin_logprobs_workspace_bytes", "q4lin_linear_logprobs", "q4lin_linear_logprobs_workspace_bytes")


class Q4LinError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        super().__init__("q4lin: %s (status %d)" % (q4lin_status_string(status), status))


def _load() -> ctypes.CDLL:
    # Device memory and streams come from torch, which carries its own HIP
    # runtime; import it first so libq4lin.so binds to that runtime instead of
    # mapping a second one (pointers and streams are only valid in the runtime
    # that made them).
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    if not os.path.exists(LIB_PATH):
        raise ImportError("libq4lin.so is not built: run `python -m weight_only_bit_q4_amd.build` "
                          "(expected at %s)" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    i64 = ctypes.c_int64
    vp = ctypes.c_void_p
    lib.q4lin_workspace_bytes.argtypes = [i64, i64, i64]
    lib.q4lin_workspace_bytes.restype = i64
    lib.q4lin_linear.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, ctypes.c_size_t, vp]
    lib.q4lin_linear.restype = ctypes.c_int
    lib.q4lin_linear_add.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp, ctypes.c_size_t, vp]
    lib.q4lin_linear_add.restype = ctypes.c_int
    lib.q4lin_linear_pair.argtypes = [vp, vp, vp, vp, i64, vp, vp, vp, i64, i64, i64, vp, ctypes.c_size_t, vp]
    lib.q4lin_linear_pair.restype = ctypes.c_int
    lib.q4lin_pair_workspace_bytes.argtypes = [i64, i64, i64, i64]
    lib.q4lin_pair_workspace_bytes.restype = i64
    lib.q4lin_linear_swiglu.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp, ctypes.c_size_t, vp]
    lib.q4lin_linear_swiglu.restype = ctypes.c_int
    lib.q4lin_swiglu_workspace_bytes.argtypes = [i64, i64, i64]
    lib.q4lin_swiglu_workspace_bytes.restype = i64
    lib.q4lin_status_string.argtypes = [ctypes.c_int]
    lib.q4lin_status_string.restype = ctypes.c_char_p
    lib.q4lin_route.argtypes = [i64, i64, i64]
    lib.q4lin_route.restype = ctypes.c_int
    lib.q4lin_version.argtypes = []
    lib.q4lin_version.restype = ctypes.c_int
    lib.q4lin_linear_noalloc.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
    lib.q4lin_linear_noalloc.restype = ctypes.c_int
    lib.q4lin_noalloc_scratch_bytes.argtypes = []
    lib.q4lin_noalloc_scratch_bytes.restype = i64
    ci = ctypes.c_int
    lib.q4lin_linear_fmt.argtypes = [ci, vp, vp, vp, vp, vp, i64, i64, i64, vp, ctypes.c_size_t, vp]
    lib.q4lin_linear_fmt.restype = ci
    lib.q4lin_fmt_weight_bytes.argtypes = [ci, i64, i64]
    lib.q4lin_fmt_weight_bytes.restype = i64
    lib.q4lin_fmt_workspace_bytes.argtypes = [ci, i64, i64, i64]
    lib.q4lin_fmt_workspace_bytes.restype = i64
    cz = ctypes.c_size_t
    lib.q4lin_linear_lora.argtypes = [ci] + [vp] * 9 + [i64] * 5 + [vp, cz, vp]
    lib.q4lin_linear_lora.restype = ci
    lib.q4lin_lora_workspace_bytes.argtypes = [ci] + [i64] * 5
    lib.q4lin_lora_workspace_bytes.restype = i64
    lib.q4lin_moe.argtypes = [vp] * 11 + [i64] * 5 + [ci, vp, cz, vp]
    lib.q4lin_moe.restype = ci
    lib.q4lin_moe_route.argtypes = [vp] * 4 + [i64] * 4 + [ci, vp]
    lib.q4lin_moe_route.restype = ci
    lib.q4lin_moe_experts.argtypes = [vp] * 10 + [i64] * 5 + [vp, cz, vp]
    lib.q4lin_moe_experts.restype = ci
    lib.q4lin_moe_workspace_bytes.argtypes = [i64] * 5
    lib.q4lin_moe_workspace_bytes.restype = i64
    lib.q4lin_rmsnorm_mx8.argtypes = [vp] * 3 + [ctypes.c_float] + [vp] * 3 + [i64] * 2 + [vp]
    lib.q4lin_rmsnorm_mx8.restype = ci
    lib.q4lin_quantize_mx8.argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, vp]
    lib.q4lin_quantize_mx8.restype = ci
    lib.q4lin_linear_mx8.argtypes = [vp] * 6 + [i64] * 3 + [vp, cz, vp]
    lib.q4lin_linear_mx8.restype = ci
    lib.q4lin_linear_mx8_workspace_bytes.argtypes = [i64] * 3
    lib.q4lin_linear_mx8_workspace_bytes.restype = i64
    lib.q4lin_logprobs.argtypes = [vp, ci, i64] + [vp] * 5 + [i64] * 3 + [vp, cz, vp]
    lib.q4lin_logprobs.restype = ci
    lib.q4lin_logprobs_workspace_bytes.argtypes = [i64] * 3
    lib.q4lin_logprobs_workspace_bytes.restype = i64
    lib.q4lin_linear_logprobs.argtypes = [vp] * 9 + [i64] * 4 + [vp, cz, vp]
    lib.q4lin_linear_logprobs.restype = ci
    lib.q4lin_linear_logprobs_workspace_bytes.argtypes = [i64] * 4
    lib.q4lin_linear_logprobs_workspace_bytes.restype = i64
    return lib


_lib = None


def load() -> ctypes.CDLL:
    """Load libq4lin.so (once); raises ImportError when it is not built."""
    global _lib
    if _lib is None:
        _lib = _load()
    return _lib


# -- the C ABI, same names ---------------------------------------------------
def q4lin_workspace_bytes(n: int, k: int, t: int) -> int:
    return int(load().q4lin_workspace_bytes(int(n), int(k), int(t)))


def q4lin_linear(x: int, codes: int, scales: int, y: int, n: int, k: int, t: int,
                 workspace: int, workspace_bytes: int, stream: int) -> int:
    """Raw call: device addresses as integers (0 for NULL); returns the status."""
    return int(load().q4lin_linear(x or None, codes or None, scales or None, y or None,
                                 int(n), int(k), int(t), workspace or None,
                                 int(workspace_bytes), stream or None))


def q4lin_linear_add(x: int, codes: int, scales: int, residual: int, y: int, n: int, k: int, t: int,
                     workspace: int, workspace_bytes: int, stream: int) -> int:
    """Raw call of the LinearAdd entry point (Y = W x X + R); returns the status."""
    return int(load().q4lin_linear_add(x or None, codes or None, scales or None, residual or None, y or None,
                                       int(n), int(k), int(t), workspace or None,
                                       int(workspace_bytes), stream or None))


def q4lin_linear_pair(x: int, codes1: int, scales1: int, y1: int, n1: int, codes2: int, scales2: int, y2: int,
                      n2: int, k: int, t: int, workspace: int, workspace_bytes: int, stream: int) -> int:
    """Raw call of the LinearPair entry point (Y1 = W1 x X, Y2 = W2 x X); returns the status."""
    return int(load().q4lin_linear_pair(x or None, codes1 or None, scales1 or None, y1 or None, int(n1),
                                        codes2 or None, scales2 or None, y2 or None, int(n2), int(k), int(t),
                                        workspace or None, int(workspace_bytes), stream or None))


def q4lin_pair_workspace_bytes(n1: int, n2: int, k: int, t: int) -> int:
    return int(load().q4lin_pair_workspace_bytes(int(n1), int(n2), int(k), int(t)))


def q4lin_linear_swiglu(x: int, codes_gate: int, scales_gate: int, codes_up: int, scales_up: int, y: int,
                        n: int, k: int, t: int, workspace: int, workspace_bytes: int, stream: int) -> int:
    """Raw call of the LinearSwiGLU entry point (Y = silu(Wg x X) * (Wu x X)); returns the status."""
    return int(load().q4lin_linear_swiglu(x or None, codes_gate or None, scales_gate or None, codes_up or None,
                                          scales_up or None, y or None, int(n), int(k), int(t),
                                          workspace or None, int(workspace_bytes), stream or None))


def q4lin_swiglu_workspace_bytes(n: int, k: int, t: int) -> int:
    return int(load().q4lin_swiglu_workspace_bytes(int(n), int(k), int(t)))


def q4lin_linear_noalloc(x: int, codes: int, scales: int, y: int, n: int, k: int, t: int, stream: int) -> int:
    """Raw call of the no-allocation entry point (scratch inside the library); returns the status."""
    return int(load().q4lin_linear_noalloc(x or None, codes or None, scales or None, y or None,
                                           int(n), int(k), int(t), stream or None))


def q4lin_noalloc_scratch_bytes() -> int:
    return int(load().q4lin_noalloc_scratch_bytes())


def q4lin_linear_fmt(fmt: int, x: int, w: int, w_hi: int, scales: int, y: int, n: int, k: int, t: int,
                     workspace: int, workspace_bytes: int, stream: int) -> int:
    """Raw call of the weight-format entry point (Q4LIN_FMT_*); returns the status."""
    return int(load().q4lin_linear_fmt(int(fmt), x or None, w or None, w_hi or None, scales or None, y or None,
                                       int(n), int(k), int(t), workspace or None, int(workspace_bytes),
                                       stream or None))


def q4lin_fmt_weight_bytes(fmt: int, n: int, k: int) -> int:
    return int(load().q4lin_fmt_weight_bytes(int(fmt), int(n), int(k)))


def q4lin_fmt_workspace_bytes(fmt: int, n: int, k: int, t: int) -> int:
    return int(load().q4lin_fmt_workspace_bytes(int(fmt), int(n), int(k), int(t)))


def q4lin_linear_lora(fmt: int, x: int, w: int, w_hi: int, scales: int, lora_a: int, lora_b: int, lora_scale: int,
                      adapter_ids: int, y: int, n: int, k: int, t: int, adapters: int, rank: int, workspace: int,
                      workspace_bytes: int, stream: int) -> int:
    """Raw call of the low-rank-adapter entry point; returns the status."""
    return int(load().q4lin_linear_lora(fmt, x, w, w_hi, scales, lora_a, lora_b, lora_scale, adapter_ids, y,
                                        n, k, t, adapters, rank, workspace, workspace_bytes, stream))


@functools.lru_cache(maxsize=4096)
def q4lin_lora_workspace_bytes(fmt: int, n: int, k: int, t: int, adapters: int, rank: int) -> int:
    return int(load().q4lin_lora_workspace_bytes(fmt, n, k, t, adapters, rank))


def q4lin_moe(x: int, router: int, codes_gate: int, scales_gate: int, codes_up: int, scales_up: int, codes_down: int,
              scales_down: int, y: int, ids: int, weights: int, inner: int, k: int, experts: int, top_k: int, t: int,
              renormalize: int, workspace: int, workspace_bytes: int, stream: int) -> int:
    """Raw call of the mixture-of-experts layer; returns the status."""
    return int(load().q4lin_moe(x, router, codes_gate, scales_gate, codes_up, scales_up, codes_down, scales_down, y,
                                ids, weights, inner, k, experts, top_k, t, renormalize, workspace, workspace_bytes,
                                stream))


def q4lin_moe_route(x: int, router: int, ids: int, weights: int, k: int, experts: int, top_k: int, t: int,
                    renormalize: int, stream: int) -> int:
    """Raw call of the experts' router; returns the status."""
    return int(load().q4lin_moe_route(x, router, ids, weights, k, experts, top_k, t, renormalize, stream))


def q4lin_moe_experts(x: int, ids: int, weights: int, codes_gate: int, scales_gate: int, codes_up: int,
                      scales_up: int, codes_down: int, scales_down: int, y: int, inner: int, k: int, experts: int,
                      top_k: int, t: int, workspace: int, workspace_bytes: int, stream: int) -> int:
    """Raw call of the experts on given routing; returns the status."""
    return int(load().q4lin_moe_experts(x, ids, weights, codes_gate, scales_gate, codes_up, scales_up, codes_down,
                                        scales_down, y, inner, k, experts, top_k, t, workspace, workspace_bytes,
                                        stream))


@functools.lru_cache(maxsize=4096)
def q4lin_moe_workspace_bytes(inner: int, k: int, experts: int, top_k: int, t: int) -> int:
    return int(load().q4lin_moe_workspace_bytes(inner, k, experts, top_k, t))


def q4lin_rmsnorm_mx8(x: int, residual: int, weight: int, eps: float, h: int, values: int, scales: int, k: int, t: int,
                      stream: int) -> int:
    """Raw call of the root-mean-square norm into MXFP8; returns the status."""
    return int(load().q4lin_rmsnorm_mx8(x, residual, weight, eps, h, values, scales, k, t, stream))


def q4lin_quantize_mx8(x: int, x_stride: int, gate: int, gate_stride: int, values: int, scales: int, k: int, t: int,
                       stream: int) -> int:
    """Raw call of the (gated) quantization into MXFP8; returns the status."""
    return int(load().q4lin_quantize_mx8(x, x_stride, gate, gate_stride, values, scales, k, t, stream))


def q4lin_linear_mx8(values: int, x_scales: int, codes: int, scales: int, residual: int, y: int, n: int, k: int,
                     t: int, workspace: int, workspace_bytes: int, stream: int) -> int:
    """Raw call of the product of MXFP8 activations; returns the status."""
    return int(load().q4lin_linear_mx8(values, x_scales, codes, scales, residual, y, n, k, t, workspace,
                                       workspace_bytes, stream))


@functools.lru_cache(maxsize=4096)
def q4lin_linear_mx8_workspace_bytes(n: int, k: int, t: int) -> int:
    return int(load().q4lin_linear_mx8_workspace_bytes(n, k, t))


def q4lin_logprobs(logits: int, f32: int, stride: int, tokens: int, logprob: int, entropy: int, top_logprobs: int,
                   top_ids: int, n: int, t: int, top: int, workspace: int, workspace_bytes: int, stream: int) -> int:
    """Raw call of the log probabilities of logits; returns the status."""
    return int(load().q4lin_logprobs(logits, f32, stride, tokens, logprob, entropy, top_logprobs, top_ids, n, t, top,
                                     workspace, workspace_bytes, stream))


@functools.lru_cache(maxsize=4096)
def q4lin_logprobs_workspace_bytes(n: int, t: int, top: int) -> int:
    return int(load().q4lin_logprobs_workspace_bytes(n, t, top))


def q4lin_linear_logprobs(x: int, x_scales: int, codes: int, scales: int, tokens: int, logprob: int, entropy: int,
                          top_logprobs: int, top_ids: int, n: int, k: int, t: int, top: int, workspace: int,
                          workspace_bytes: int, stream: int) -> int:
    """Raw call of the log probabilities of a product; returns the status."""
    return int(load().q4lin_linear_logprobs(x, x_scales, codes, scales, tokens, logprob, entropy, top_logprobs,
                                            top_ids, n, k, t, top, workspace, workspace_bytes, stream))


@functools.lru_cache(maxsize=4096)
def q4lin_linear_logprobs_workspace_bytes(n: int, k: int, t: int, top: int) -> int:
    return int(load().q4lin_linear_logprobs_workspace_bytes(n, k, t, top))


def q4lin_status_string(status: int) -> str:
    return load().q4lin_status_string(int(status)).decode()


def q4lin_route(n: int, k: int, t: int) -> int:
    return int(load().q4lin_route(int(n), int(k), int(t)))


def q4lin_version() -> int:
    return int(load().q4lin_version())


# -- torch convenience (marshalling only) -------------------------------------
def linear(x, codes, scales, y=None, workspace=None, stream=None, residual=None):
    """Y = W x X (or, with ``residual``, the LinearAdd Y = W x X + R) on torch
    device tensors.

    ``x``: uint16/int16/bfloat16 ``[T, K]`` (bf16 bits, token-major);
    ``codes``: uint8 ``[N, K/2]``; ``scales``: float16/int16/uint16 ``[N, K/64]``;
    ``y``: optional bfloat16/int16/uint16 ``[T, N]`` output; ``residual``:
    optional ``[T, N]`` bf16 bits (may be ``y`` itself).  Returns ``y``.
    """
    import torch

    t, k = x.shape
    n = codes.shape[0]
    if codes.shape[1] * 2 != k or tuple(scales.shape) != (n, k // 64):
        raise ValueError("shape mismatch: x %s codes %s scales %s" % (tuple(x.shape), tuple(codes.shape),
                                                                      tuple(scales.shape)))
    for name, ten, size in (("x", x, 2), ("codes", codes, 1), ("scales", scales, 2)):
        if not ten.is_contiguous() or ten.element_size() != size:
            raise ValueError("%s must be contiguous with %d-byte elements" % (name, size))
    if y is None:
        y = torch.empty((t, n), dtype=torch.bfloat16, device=x.device)
    if tuple(y.shape) != (t, n) or y.element_size() != 2 or not y.is_contiguous():
        raise ValueError("y must be a contiguous [T, N] tensor of 2-byte elements")
    need = q4lin_workspace_bytes(n, k, t)
    if need < 0:
        raise Q4LinError(-need)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else 0
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if stream is None:
        stream = torch.cuda.current_stream(x.device).cuda_stream
    if residual is None:
        st = q4lin_linear(x.data_ptr(), codes.data_ptr(), scales.data_ptr(), y.data_ptr(), n, k, t,
                          ws_ptr, ws_bytes, stream)
    else:
        if tuple(residual.shape) != (t, n) or residual.element_size() != 2 or not residual.is_contiguous():
            raise ValueError("residual must be a contiguous [T, N] tensor of 2-byte elements")
        st = q4lin_linear_add(x.data_ptr(), codes.data_ptr(), scales.data_ptr(), residual.data_ptr(),
                              y.data_ptr(), n, k, t, ws_ptr, ws_bytes, stream)
    if st != Q4LIN_OK:
        raise Q4LinError(st)
    return y


def linear_pair(x, codes1, scales1, codes2, scales2, y1=None, y2=None, workspace=None, stream=None):
    """LinearPair on torch device tensors: ``(W1 x X, W2 x X)`` for two weights
    of the same K over one ``x`` (layouts as in ``linear``).  Returns
    ``(y1, y2)``."""
    import torch

    t, k = x.shape
    n1, n2 = codes1.shape[0], codes2.shape[0]
    for i, (c, sc) in enumerate(((codes1, scales1), (codes2, scales2)), 1):
        n = c.shape[0]
        if c.shape[1] * 2 != k or tuple(sc.shape) != (n, k // 64):
            raise ValueError("shape mismatch: x %s codes%d %s scales%d %s" % (tuple(x.shape), i, tuple(c.shape),
                                                                           i, tuple(sc.shape)))
    for name, ten, size in (("x", x, 2), ("codes1", codes1, 1), ("scales1", scales1, 2), ("codes2", codes2, 1),
                            ("scales2", scales2, 2)):
        if not ten.is_contiguous() or ten.element_size() != size:
            raise ValueError("%s must be contiguous with %d-byte elements" % (name, size))
    outs = []
    for y, n in ((y1, n1), (y2, n2)):
        if y is None:
            y = torch.empty((t, n), dtype=torch.bfloat16, device=x.device)
        if tuple(y.shape) != (t, n) or y.element_size() != 2 or not y.is_contiguous():
            raise ValueError("outputs must be contiguous [T, N] tensors of 2-byte elements")
        outs.append(y)
    need = q4lin_pair_workspace_bytes(n1, n2, k, t)
    if need < 0:
        raise Q4LinError(-need)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else 0
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if stream is None:
        stream = torch.cuda.current_stream(x.device).cuda_stream
    st = q4lin_linear_pair(x.data_ptr(), codes1.data_ptr(), scales1.data_ptr(), outs[0].data_ptr(), n1,
                           codes2.data_ptr(), scales2.data_ptr(), outs[1].data_ptr(), n2, k, t,
                           ws_ptr, ws_bytes, stream)
    if st != Q4LIN_OK:
        raise Q4LinError(st)
    return outs[0], outs[1]


def linear_swiglu(x, codes_gate, scales_gate, codes_up, scales_up, y=None, workspace=None, stream=None):
    """LinearSwiGLU on torch device tensors: ``silu(Wg x X) * (Wu x X)``, both
    weights with ``linear``'s layouts and the same shape.  Returns ``y``."""
    import torch

    t, k = x.shape
    n = codes_gate.shape[0]
    for name, c, sc in (("gate", codes_gate, scales_gate), ("up", codes_up, scales_up)):
        if tuple(c.shape) != (n, k // 2) or tuple(sc.shape) != (n, k // 64):
            raise ValueError("shape mismatch: x %s %s codes %s scales %s" % (tuple(x.shape), name, tuple(c.shape),
                                                                          tuple(sc.shape)))
    for name, ten, size in (("x", x, 2), ("codes_gate", codes_gate, 1), ("scales_gate", scales_gate, 2),
                            ("codes_up", codes_up, 1), ("scales_up", scales_up, 2)):
        if not ten.is_contiguous() or ten.element_size() != size:
            raise ValueError("%s must be contiguous with %d-byte elements" % (name, size))
    if y is None:
        y = torch.empty((t, n), dtype=torch.bfloat16, device=x.device)
    if tuple(y.shape) != (t, n) or y.element_size() != 2 or not y.is_contiguous():
        raise ValueError("y must be a contiguous [T, N] tensor of 2-byte elements")
    need = q4lin_swiglu_workspace_bytes(n, k, t)
    if need < 0:
        raise Q4LinError(-need)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else 0
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if stream is None:
        stream = torch.cuda.current_stream(x.device).cuda_stream
    st = q4lin_linear_swiglu(x.data_ptr(), codes_gate.data_ptr(), scales_gate.data_ptr(), codes_up.data_ptr(),
                             scales_up.data_ptr(), y.data_ptr(), n, k, t, ws_ptr, ws_bytes, stream)
    if st != Q4LIN_OK:
        raise Q4LinError(st)
    return y


def linear_fmt(fmt, x, w, w_hi=None, scales=None, y=None, stream=None):
    """Y = W x X for a weight in format ``fmt`` (Q4LIN_FMT_*) on torch device
    tensors: ``x`` ``[T, K]`` bf16 bits; ``w``, ``w_hi``, ``scales`` the
    format's planes as laid out in ``include/q4lin.h`` (any dtype, read as
    bytes; ``w`` gives N as its first dimension).  Returns ``y`` ``[T, N]``."""
    import torch

    t, k = x.shape
    n = w.shape[0]
    if not x.is_contiguous() or x.element_size() != 2:
        raise ValueError("x must be contiguous with 2-byte elements")
    for name, ten in (("w", w), ("w_hi", w_hi), ("scales", scales)):
        if ten is not None and not ten.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
    if y is None:
        y = torch.empty((t, n), dtype=torch.bfloat16, device=x.device)
    if tuple(y.shape) != (t, n) or y.element_size() != 2 or not y.is_contiguous():
        raise ValueError("y must be a contiguous [T, N] tensor of 2-byte elements")
    need = q4lin_fmt_workspace_bytes(fmt, n, k, t)
    if need < 0:
        raise Q4LinError(-need)
    ws = torch.empty(need, dtype=torch.uint8, device=x.device) if need > 0 else None
    if stream is None:
        stream = torch.cuda.current_stream(x.device).cuda_stream
    st = q4lin_linear_fmt(fmt, x.data_ptr(), w.data_ptr(), w_hi.data_ptr() if w_hi is not None else 0,
                          scales.data_ptr() if scales is not None else 0, y.data_ptr(), n, k, t,
                          ws.data_ptr() if ws is not None else 0, need, stream)
    if st != Q4LIN_OK:
        raise Q4LinError(st)
    return y


_DTYPES = {}  # the element types that are read as each kind of value (bf16 and fp16 also as their bits)
_torch = None  # the module, from the first call on (an import statement a function costs each call 0.3 us)


def _place(x):
    """The index of the GPU that ``x`` is on (-1: none), for the checks of the other tensors."""
    global _torch
    if _torch is None:
        import torch

        _torch, bits = torch, (torch.int16, torch.uint16)
        _DTYPES.update(bf16=(torch.bfloat16, *bits), fp16=(torch.float16, *bits), codes=(torch.uint8, torch.int8),
                       int32=(torch.int32,), float32=(torch.float32,), e4m3=(torch.float8_e4m3fn, torch.uint8),
                       e8m0=(torch.float8_e8m0fnu, torch.uint8))
    return x.get_device()


def _checked(name, ten, shape, kind, place):
    """The tensor's address; it must be contiguous, of this shape and kind of elements, on x's GPU."""
    if ten.shape != shape or ten.dtype not in _DTYPES[kind] or not ten.is_contiguous():
        raise ValueError("%s must be a contiguous tensor of shape %s with %s elements, got %s of %s" % (
            name, tuple(shape), kind, tuple(ten.shape), ten.dtype))
    # (an index costs the host half of what comparing devices does)
    if ten.get_device() != place:
        raise ValueError("%s must be on x's GPU, not on %s" % (name, ten.device))
    return ten.data_ptr()


def _on_gpu(place):
    if place < 0:
        raise ValueError("the tensors must be on a GPU")


def _new(shape, dtype, device):
    """An uninitialised contiguous matrix (``empty_strided`` costs the host less than ``empty``)."""
    return _torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=device)


def _workspace(need, workspace, device):
    """(address, bytes, tensor to keep) of the caller's workspace or a new one of ``need`` bytes."""
    if need < 0:
        raise Q4LinError(-need)
    if need == 0 and workspace is None:
        return None, 0, None
    if workspace is None:
        workspace = _torch.empty_strided((need,), (1,), dtype=_torch.uint8, device=device)
        return workspace.data_ptr(), need, workspace
    if workspace.get_device() != device.index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on x's GPU")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _current(place):
    """The current stream's handle (the handle alone: the Stream object costs
    the host 2 us, as much as an allocation)."""
    return _torch._C._cuda_getCurrentRawStream(place)


def _on_stream(stream, x, y, workspace, call):
    """What ``call()`` gives with ``stream`` (a handle) as the current stream.
    The tensors that the call makes are that stream's own: memory of the
    current stream could still be in use by work of it that has not run.  What
    it returns is kept from reuse until the current stream's work before its
    release is done, and the caller's ``y`` and ``workspace`` until ``stream``'s
    is."""
    place = _place(x)
    _on_gpu(place)
    current = _torch.cuda.current_stream(place)
    if stream == current.cuda_stream:
        return call()
    other = _torch.cuda.ExternalStream(stream, device=place)
    with _torch.cuda.stream(other):
        out = call()
    for ten in out if isinstance(out, tuple) else (out,):
        if ten is not None:
            ten.record_stream(current)
    for ten in (y, workspace):
        if ten is not None:
            ten.record_stream(other)
    return out


_FMT_PLANES = {  # bytes per row of K weights: codes, high plane, scales
    Q4LIN_FMT_Q4G64_F16S: lambda k: (k // 2, 0, k // 32),
    Q4LIN_FMT_Q5G64_F16S: lambda k: (k // 2, k // 8, k // 32),
    Q4LIN_FMT_Q6G64_F16S: lambda k: (k // 2, k // 4, k // 32),
    Q4LIN_FMT_W8G32_F16S: lambda k: (k, 0, k // 16),
    Q4LIN_FMT_NVFP4: lambda k: (k // 2, 0, k // 16),
    Q4LIN_FMT_BF16: lambda k: (2 * k, 0, 0),
}


def _plane(name, ten, rows, per_row, place):
    """The address of a weight's plane (None: the format has none)."""
    if per_row == 0:
        return None
    if ten is None or not ten.is_contiguous() or ten.numel() * ten.element_size() != rows * per_row:
        raise ValueError("%s must be a contiguous plane of %d bytes for each of the %d rows" % (name, per_row, rows))
    if ten.get_device() != place:
        raise ValueError("%s must be on x's GPU, not on %s" % (name, ten.device))
    return ten.data_ptr()


def linear_lora(x, codes, scales, lora_a, lora_b, adapter_ids, lora_scale=None, fmt=Q4LIN_FMT_Q4G64_F16S,
                codes_hi=None, y=None, workspace=None, stream=None):
    """Y = W x X plus each token's own low-rank adapter, on torch device
    tensors: ``y[t] = W x[t] + s_a B_a (A_a x[t])`` with ``a = adapter_ids[t]``
    (outside ``0..L-1``: the base weight alone).

    ``x`` ``[T, K]`` bf16; ``codes``, ``codes_hi``, ``scales`` the weight's
    planes in format ``fmt`` (Q4LIN_FMT_*; read as bytes, ``codes`` gives N);
    ``lora_a`` bf16 ``[L, R, K]``, ``lora_b`` bf16 ``[L, N, R]`` (R a multiple
    of 8 up to 256), ``adapter_ids`` int32 ``[T]``, ``lora_scale`` float32
    ``[L]`` or None for ones.  Returns ``y`` ``[T, N]``.
    """
    if stream is not None:
        return _on_stream(stream, x, y, workspace, lambda: linear_lora(
            x, codes, scales, lora_a, lora_b, adapter_ids, lora_scale, fmt, codes_hi, y, workspace))
    t, k = x.shape
    n = codes.shape[0]
    adapters, rank = lora_a.shape[0], lora_a.shape[1]
    if fmt not in _FMT_PLANES:
        raise Q4LinError(Q4LIN_E_FORMAT)
    per_row = _FMT_PLANES[fmt](k)
    device, place = x.device, _place(x)
    wp = _plane("codes", codes, n, per_row[0], place)
    hp = _plane("codes_hi", codes_hi, n, per_row[1], place)
    cp = _plane("scales", scales, n, per_row[2], place)
    xp = _checked("x", x, (t, k), "bf16", place)
    ap = _checked("lora_a", lora_a, (adapters, rank, k), "bf16", place)
    bp = _checked("lora_b", lora_b, (adapters, n, rank), "bf16", place)
    ip = _checked("adapter_ids", adapter_ids, (t,), "int32", place)
    sp = _checked("lora_scale", lora_scale, (adapters,), "float32", place) if lora_scale is not None else None
    _on_gpu(place)
    if y is None:
        y = _new((t, n), _torch.bfloat16, device)
        yp = y.data_ptr()
    else:
        yp = _checked("y", y, (t, n), "bf16", place)
    work, work_bytes, workspace = _workspace(q4lin_lora_workspace_bytes(fmt, n, k, t, adapters, rank), workspace, device)
    st = load().q4lin_linear_lora(fmt, xp, wp, hp, cp, ap, bp, sp, ip, yp, n, k, t, adapters, rank, work, work_bytes,
                                  _current(place))
    if st != Q4LIN_OK:
        raise Q4LinError(st)
    return y


def _expert_planes(k, codes_gate, scales_gate, codes_up, scales_up, codes_down, scales_down, place):
    """(experts, inner, the six addresses) of a layer's expert weights."""
    experts, inner = codes_gate.shape[0], codes_gate.shape[1]
    return experts, inner, (
        _checked("codes_gate", codes_gate, (experts, inner, k // 2), "codes", place),
        _checked("scales_gate", scales_gate, (experts, inner, k // 64), "fp16", place),
        _checked("codes_up", codes_up, (experts, inner, k // 2), "codes", place),
        _checked("scales_up", scales_up, (experts, inner, k // 64), "fp16", place),
        _checked("codes_down", codes_down, (experts, k, inner // 2), "codes", place),
        _checked("scales_down", scales_down, (experts, k, inner // 64), "fp16", place))


def moe_route(x, router, top_k, renormalize=True, stream=None):
    """The experts of each token, on torch device tensors: softmax over
    ``x router^T``, the ``top_k`` largest (ties: the lowest index), weights
    divided by their sum where ``renormalize``.  ``x`` bf16 ``[T, K]``,
    ``router`` bf16 ``[E, K]``.  Returns ``(ids int32 [T, top_k], weights
    float32 [T, top_k])``."""
    if stream is not None:
        return _on_stream(stream, x, None, None, lambda: moe_route(x, router, top_k, renormalize))
    t, k = x.shape
    experts = router.shape[0]
    device, place = x.device, _place(x)
    xp = _checked("x", x, (t, k), "bf16", place)
    rp = _checked("router", router, (experts, k), "bf16", place)
    _on_gpu(place)
    ids = _new((t, top_k), _torch.int32, device)
    weights = _new((t, top_k), _torch.float32, device)
    st = load().q4lin_moe_route(xp, rp, ids.data_ptr(), weights.data_ptr(), k, experts, top_k, t,
                                1 if renormalize else 0, _current(place))
    if st != Q4LIN_OK:
        raise Q4LinError(st)
    return ids, weights


def _by_expert(ids, weights, experts):
    """Routing of more choices than there are experts, as one place for each
    expert: its number where the token chose it (else -1) and the sum of the
    weights with which it did."""
    each = _torch.arange(experts, dtype=_torch.int32, device=ids.device)
    chosen = ids[:, None, :] == each[:, None]
    total = _torch.where(chosen, weights[:, None, :], 0.0).sum(2)
    return _torch.where(chosen.any(2), each, -1), total


def moe_experts(x, ids, weights, codes_gate, scales_gate, codes_up, scales_up, codes_down, scales_down, y=None,
                workspace=None, stream=None):
    """``y[t] = sum_j weights[t, j] Wd_e (silu(Wg_e x[t]) * (Wu_e x[t]))`` with
    ``e = ids[t, j]`` (outside ``0..E-1``: nothing), on torch device tensors.
    ``x`` bf16 ``[T, K]``; ``ids`` int32, ``weights`` float32 ``[T, top_k]``;
    gate and up codes uint8 ``[E, I, K/2]``, scales fp16 ``[E, I, K/64]``;
    down codes ``[E, K, I/2]``, scales ``[E, K, I/64]``.  ``top_k`` may exceed
    E (a share of the experts smaller than ``top_k``).  Returns ``y`` bf16
    ``[T, K]``."""
    if stream is not None:
        return _on_stream(stream, x, y, workspace, lambda: moe_experts(
            x, ids, weights, codes_gate, scales_gate, codes_up, scales_up, codes_down, scales_down, y, workspace))
    t, k = x.shape
    top_k = ids.shape[1]
    device, place = x.device, _place(x)
    xp = _checked("x", x, (t, k), "bf16", place)
    ip = _checked("ids", ids, (t, top_k), "int32", place)
    vp = _checked("weights", weights, (t, top_k), "float32", place)
    experts, inner, planes = _expert_planes(k, codes_gate, scales_gate, codes_up, scales_up, codes_down, scales_down,
                                            place)
    _on_gpu(place)
    if top_k > experts:  # the library takes at most one place for each expert
        ids, weights = _by_expert(ids, weights, experts)
        top_k, ip, vp = experts, ids.data_ptr(), weights.data_ptr()
    if y is None:
        y = _new((t, k), _torch.bfloat16, device)
    yp = _checked("y", y, (t, k), "bf16", place)
    wp, wb, workspace = _workspace(q4lin_moe_workspace_bytes(inner, k, experts, top_k, t), workspace, device)
    st = load().q4lin_moe_experts(xp, ip, vp, *planes, yp, inner, k, experts, top_k, t, wp, wb, _current(place))
    if st != Q4LIN_OK:
        raise Q4LinError(st)
    return y


def moe(x, router, codes_gate, scales_gate, codes_up, scales_up, codes_down, scales_down, top_k, renormalize=True,
        y=None, workspace=None, stream=None):
    """A whole mixture-of-experts layer on torch device tensors: ``moe_route``
    and ``moe_experts`` in one call (their arguments).  Returns ``(y, ids,
    weights)``."""
    if stream is not None:
        return _on_stream(stream, x, y, workspace, lambda: moe(
            x, router, codes_gate, scales_gate, codes_up, scales_up, codes_down, scales_down, top_k, renormalize, y,
            workspace))
    t, k = x.shape
    device, place = x.device, _place(x)
    xp = _checked("x", x, (t, k), "bf16", place)
    experts, inner, planes = _expert_planes(k, codes_gate, scales_gate, codes_up, scales_up, codes_down, scales_down,
                                            place)
    rp = _checked("router", router, (experts, k), "bf16", place)
    _on_gpu(place)
    ids = _new((t, top_k), _torch.int32, device)
    weights = _new((t, top_k), _torch.float32, device)
    if y is None:
        y = _new((t, k), _torch.bfloat16, device)
    yp = _checked("y", y, (t, k), "bf16", place)
    wp, wb, workspace = _workspace(q4lin_moe_workspace_bytes(inner, k, experts, top_k, t), workspace, device)
    st = load().q4lin_moe(xp, rp, *planes, yp, ids.data_ptr(), weights.data_ptr(), inner, k, experts, top_k, t,
                          1 if renormalize else 0, wp, wb, _current(place))
    if st != Q4LIN_OK:
        raise Q4LinError(st)
    return y, ids, weights


def rmsnorm_mx8(x, weight=None, eps=1e-6, residual=None, h=None, stream=None):
    """The root-mean-square norm of ``x`` (plus ``residual``) in 8 bits, on
    torch device tensors: ``v = x + residual``, ``y = v / sqrt(mean(v^2) + eps) *
    weight``, in blocks of 32 that share a power of two (MXFP8, as laid out in
    ``include/q4lin.h``).  ``x``, ``residual`` bf16 ``[T, K]``, ``weight`` bf16
    ``[K]`` or None for ones.  Returns ``(values float8_e4m3fn [T, K], scales
    float8_e8m0fnu [T, K/32])``, and with ``residual`` also ``h``, bf16 of ``v``
    (``h`` may be given, also as ``x`` or ``residual`` itself)."""
    if stream is not None:
        return _on_stream(stream, x, h, None, lambda: rmsnorm_mx8(x, weight, eps, residual, h))
    t, k = x.shape
    device, place = x.device, _place(x)
    xp = _checked("x", x, (t, k), "bf16", place)
    wp = _checked("weight", weight, (k,), "bf16", place) if weight is not None else None
    rp = hp = None
    if residual is not None:
        rp = _checked("residual", residual, (t, k), "bf16", place)
        _on_gpu(place)
        if h is None:
            h = _new((t, k), _torch.bfloat16, device)
            hp = h.data_ptr()
        else:
            hp = _checked("h", h, (t, k), "bf16", place)
    elif h is not None:
        raise ValueError("h is written only with a residual")
    _on_gpu(place)
    values = _new((t, k), _torch.float8_e4m3fn, device)
    scales = _new((t, k // 32), _torch.float8_e8m0fnu, device)
    st = load().q4lin_rmsnorm_mx8(xp, rp, wp, eps, hp, values.data_ptr(), scales.data_ptr(), k, t, _current(place))
    if st != Q4LIN_OK:
        raise Q4LinError(st)
    return (values, scales) if residual is None else (values, scales, h)


def _rows(name, ten, shape, dtypes, place):
    """(address, elements between rows) of a matrix whose rows are contiguous."""
    if ten.shape != shape or ten.dtype not in dtypes or (shape[1] > 1 and ten.stride(1) != 1):
        raise ValueError("%s must be a tensor of shape %s with contiguous rows of %s, got %s of %s" % (
            name, tuple(shape), dtypes[0], tuple(ten.shape), ten.dtype))
    if ten.get_device() != place:
        raise ValueError("%s must be on x's GPU, not on %s" % (name, ten.device))
    return ten.data_ptr(), ten.stride(0)


def quantize_mx8(x, gate=None, stream=None):
    """``x``, or ``silu(gate) * x``, in 8 bits (``rmsnorm_mx8``'s form) on torch
    device tensors: bf16 ``[T, K]``, rows contiguous and any multiple of eight
    elements apart (the halves of one product's rows).  Returns ``(values,
    scales)``."""
    if stream is not None:
        return _on_stream(stream, x, None, None, lambda: quantize_mx8(x, gate))
    t, k = x.shape
    device, place = x.device, _place(x)
    xp, xs = _rows("x", x, (t, k), _DTYPES["bf16"], place)
    gp, gs = _rows("gate", gate, (t, k), _DTYPES["bf16"], place) if gate is not None else (None, 0)
    _on_gpu(place)
    values = _new((t, k), _torch.float8_e4m3fn, device)
    scales = _new((t, k // 32), _torch.float8_e8m0fnu, device)
    st = load().q4lin_quantize_mx8(xp, xs, gp, gs, values.data_ptr(), scales.data_ptr(), k, t, _current(place))
    if st != Q4LIN_OK:
        raise Q4LinError(st)
    return values, scales


def linear_mx8(values, x_scales, codes, scales, residual=None, y=None, workspace=None, stream=None):
    """Y = W x X (+ R) with activations in 8 bits, on torch device tensors:
    ``values`` float8_e4m3fn ``[T, K]`` and ``x_scales`` float8_e8m0fnu ``[T,
    K/32]`` as ``rmsnorm_mx8`` and ``quantize_mx8`` give them (or their bytes);
    ``codes`` uint8 ``[N, K/2]``, ``scales`` fp16 ``[N, K/64]``; ``residual`` bf16
    ``[T, N]`` (may be ``y``).  Returns ``y`` bf16 ``[T, N]``."""
    if stream is not None:
        return _on_stream(stream, values, y, workspace, lambda: linear_mx8(
            values, x_scales, codes, scales, residual, y, workspace))
    t, k = values.shape
    n = codes.shape[0]
    device, place = values.device, _place(values)
    vp = _checked("values", values, (t, k), "e4m3", place)
    ep = _checked("x_scales", x_scales, (t, k // 32), "e8m0", place)
    cp = _checked("codes", codes, (n, k // 2), "codes", place)
    sp = _checked("scales", scales, (n, k // 64), "fp16", place)
    rp = _checked("residual", residual, (t, n), "bf16", place) if residual is not None else None
    _on_gpu(place)
    if y is None:
        y = _new((t, n), _torch.bfloat16, device)
        yp = y.data_ptr()
    else:
        yp = _checked("y", y, (t, n), "bf16", place)
    wp, wb, workspace = _workspace(q4lin_linear_mx8_workspace_bytes(n, k, t), workspace, device)
    st = load().q4lin_linear_mx8(vp, ep, cp, sp, rp, yp, n, k, t, wp, wb, _current(place))
    if st != Q4LIN_OK:
        raise Q4LinError(st)
    return y


def _logprob_outputs(tokens, t, top, place, device):
    """(tokens' address, the four outputs, their addresses) of a log probability call."""
    tp = _checked("tokens", tokens, (t,), "int32", place) if tokens is not None else None
    _on_gpu(place)
    if top < 0:
        raise Q4LinError(Q4LIN_E_SHAPE)
    logprob = _torch.empty_strided((t,), (1,), dtype=_torch.float32, device=device) if tokens is not None else None
    entropy = _torch.empty_strided((t,), (1,), dtype=_torch.float32, device=device)
    best = _new((t, top), _torch.float32, device)
    ids = _new((t, top), _torch.int32, device)
    return tp, (logprob, entropy, best, ids), (logprob.data_ptr() if tokens is not None else None, entropy.data_ptr(),
                                               best.data_ptr(), ids.data_ptr())


def logprobs(logits, tokens=None, top=0, workspace=None, stream=None):
    """Log probabilities of rows of logits on torch device tensors: ``logits``
    bf16 or float32 ``[T, N]`` (rows contiguous, any distance apart),
    ``tokens`` int32 ``[T]`` (a number outside the row gives 0) or None.
    Returns ``(logprob, entropy, top_logprobs, top_ids)``: float32 ``[T]`` (None
    without ``tokens``), float32 ``[T]``, float32 and int32 ``[T, top]``, largest
    first and equal ones by the lowest number (``top`` up to 32)."""
    if stream is not None:
        return _on_stream(stream, logits, None, workspace, lambda: logprobs(logits, tokens, top, workspace))
    t, n = logits.shape
    device, place = logits.device, _place(logits)
    f32 = logits.dtype == _torch.float32
    lp, stride = _rows("logits", logits, (t, n), _DTYPES["float32" if f32 else "bf16"], place)
    tp, outs, at = _logprob_outputs(tokens, t, top, place, device)
    wp, wb, workspace = _workspace(q4lin_logprobs_workspace_bytes(n, t, top), workspace, device)
    st = load().q4lin_logprobs(lp, 1 if f32 else 0, stride, tp, *at, n, t, top, wp, wb, _current(place))
    if st != Q4LIN_OK:
        raise Q4LinError(st)
    return outs


def linear_logprobs(x, x_scales, codes, scales, tokens=None, top=0, workspace=None, stream=None):
    """``logprobs`` of the logits ``W x X`` (the vocabulary's projection), which
    are neither rounded nor kept, on torch device tensors: ``x`` float8_e4m3fn
    ``[T, K]`` with ``x_scales`` (as for ``linear_mx8``), or bf16 ``[T, K]`` with
    ``x_scales`` None; ``codes`` uint8 ``[N, K/2]``, ``scales`` fp16 ``[N, K/64]``.
    Returns what ``logprobs`` does."""
    if stream is not None:
        return _on_stream(stream, x, None, workspace, lambda: linear_logprobs(
            x, x_scales, codes, scales, tokens, top, workspace))
    t, k = x.shape
    n = codes.shape[0]
    device, place = x.device, _place(x)
    mx8 = x_scales is not None
    xp = _checked("x", x, (t, k), "e4m3" if mx8 else "bf16", place)
    ep = _checked("x_scales", x_scales, (t, k // 32), "e8m0", place) if mx8 else None
    cp = _checked("codes", codes, (n, k // 2), "codes", place)
    sp = _checked("scales", scales, (n, k // 64), "fp16", place)
    tp, outs, at = _logprob_outputs(tokens, t, top, place, device)
    wp, wb, workspace = _workspace(q4lin_linear_logprobs_workspace_bytes(n, k, t, top), workspace, device)
    st = load().q4lin_linear_logprobs(xp, ep, cp, sp, tp, *at, n, k, t, top, wp, wb, _current(place))
    if st != Q4LIN_OK:
        raise Q4LinError(st)
    return outs
