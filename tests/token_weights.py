"""Inputs and 64-bit references of the operators in which each token picks
its own weights (low-rank adapters, experts), on the CPU, with bounds of what
the kernels' roundings may cost.

The bounds count roundings.  A sum of products in binary32 on the matrix
cores: at most 64 terms of (128 + q) x per scale group (thirty times the
terms (q - 8) x on average), each rounding 2^-24 of the group's sum, so
2^-13 of A = sum |w x| covers the group sums, and the sums over groups and
waves after them.  The many-token route rounds each weight to fp16 (half a
step: 2^-11 of it): 2^-11 A.  The store rounds to bf16: 2^-8 of |y|.
"""
import numpy as np
import torch

from weight_only_bit_q4_amd import inputs

STORE = 2.0 ** -8       # bf16, half a step
SUMS = 2.0 ** -13       # binary32 sums of exact products, of A
F16_WEIGHT = 2.0 ** -11  # a weight rounded to fp16, of its own
SPLIT = 2.0 ** -16      # a value in two bf16 parts

_E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def bf16(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def _tensor(a):
    return None if a is None else torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a)


def weight(fmt, n, k, seed):
    """((codes, codes_hi, scales) tensors, their values in 64 bits)."""
    lo, hi, sc = inputs.gen_fmt_weight(fmt, n, k, seed)
    if fmt == inputs.FMT_BF16:
        v = torch.from_numpy(lo.view(np.int16)).view(torch.bfloat16).double().numpy()
    elif fmt == inputs.FMT_W8:
        v = lo.view(np.int8).astype(np.float64) * np.repeat(sc.view(np.float16).astype(np.float64), 32, 1)
    else:
        q = np.empty((n, k), dtype=np.int64)
        q[:, 0::2], q[:, 1::2] = lo & 15, lo >> 4
        if fmt == inputs.FMT_NVFP4:
            s = torch.from_numpy(sc).view(torch.float8_e4m3fn).double().numpy()
            v = _E2M1[q] * np.repeat(s, 16, 1)
        else:
            width = {inputs.FMT_Q4: 0, inputs.FMT_Q5: 1, inputs.FMT_Q6: 2}[fmt]
            if width:
                per = 8 // width
                for j in range(per):
                    q[:, j::per] += (((hi >> (width * j)) & ((1 << width) - 1)).astype(np.int64)) << 4
            v = (q - (8 << width)) * np.repeat(sc.view(np.float16).astype(np.float64), 64, 1)
    return tuple(_tensor(p) for p in (lo, hi, sc)), torch.from_numpy(v)


def close(got, want, bound, what):
    """Every value within its bound; NaN where the reference has NaN."""
    got = got.double().cpu()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), "%s: NaN elsewhere than in the reference" % what
    same = (got == want) | nan
    err = torch.where(same, 0.0, (got - want).abs())
    bad = ~(err <= bound) & ~same
    assert not bad.any(), "%s: %d of %d outside their bounds (worst %.3g times)" % (
        what, int(bad.sum()), bad.numel(), float((err / bound.clamp_min(1e-300))[~same].max()))
    fine = torch.isfinite(want)
    if fine.any() and float(want[fine].norm()) > 0:
        # all errors together: the stores' roundings and a quarter of that for the sums
        rel = float((err[fine].norm()) / want[fine].norm())
        assert rel <= STORE * 1.25, "%s: relative error %.3g" % (what, rel)


def lora_reference(x, w64, a, b, ids, scale, tiled):
    """(y, bound) of a linear_lora call from CPU tensors."""
    xd = x.double()
    y = xd @ w64.t()
    mag = xd.abs() @ w64.abs().t()
    bound = (SUMS + (F16_WEIGHT if tiled else 0.0)) * mag
    for t, ad in enumerate(ids.tolist()):
        if 0 <= ad < a.shape[0]:
            s = 1.0 if scale is None else float(scale[ad])
            ad64, bd64 = a[ad].double(), b[ad].double()
            y[t] += s * (bd64 @ (ad64 @ xd[t]))
            bound[t] += (SUMS + SPLIT) * abs(s) * (bd64.abs() @ (ad64.abs() @ xd[t].abs()))
    return y, bound + STORE * y.abs()


def expert_weights(experts, inner, k, seed):
    """(the six planes of moe's experts, [gate, up, down] in 64 bits [E, rows, cols])."""
    planes, values = [], []
    for i, (n, kk) in enumerate(((inner, k), (inner, k), (k, inner))):
        (c, _, s), v = weight(inputs.FMT_Q4, experts * n, kk, seed + i)
        # scales that keep the sums near one
        s = (s.view(torch.float16) * (kk ** -0.5 * 16)).view(torch.int16)
        q = torch.empty(experts * n, kk, dtype=torch.float64)
        q[:, 0::2], q[:, 1::2] = (c & 15).double(), (c >> 4).double()
        v = (q - 8) * s.view(torch.float16).double().repeat_interleave(64, 1)
        planes += [c.view(experts, n, kk // 2), s.view(experts, n, kk // 64)]
        values.append(v.view(experts, n, kk))
    return planes, values


def route_reference(x, router, top_k, renorm):
    """(ids, weights, bound of the weights)."""
    xd, rd = x.double(), router.double()
    logits = xd @ rd.t()
    key = torch.where(torch.isnan(logits), -np.inf, logits)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :top_k]
    p = torch.softmax(logits, 1)
    w = p.gather(1, ids)
    if renorm:
        w = torch.softmax(logits.gather(1, ids), 1)
    # eight exact products summed in binary32 at a time, twice in a quotient
    rel = 2 * 8 * 2.0 ** -24 * (xd.abs() @ rd.abs().t()).max(1, keepdim=True).values + 2.0 ** -22
    return ids, w, w * rel


def experts_reference(x, ids, weights, values):
    """(y, bound) of a moe_experts call from CPU tensors."""
    xd = x.double()
    gate, up, down = values
    t, k = x.shape
    y = torch.zeros(t, k, dtype=torch.float64)
    bound = torch.zeros_like(y)
    for i in range(t):
        for e, w in zip(ids[i].tolist(), weights[i].double().tolist()):
            if not 0 <= e < gate.shape[0]:
                continue
            g, u = gate[e] @ xd[i], up[e] @ xd[i]
            eg, eu = (SUMS * (m[e].abs() @ xd[i].abs()) for m in (gate, up))
            sig = torch.sigmoid(g)
            h = g * sig * u
            eh = 1.1 * u.abs() * eg + (g * sig).abs() * eu + SPLIT * h.abs()  # |silu'| < 1.1
            y[i] += w * (down[e] @ h)
            bound[i] += abs(w) * (down[e].abs() @ (eh + SUMS * h.abs()))
    return y, bound + STORE * y.abs()
