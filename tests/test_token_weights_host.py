"""Refusals of the operators in which each token picks its own weights
(low-rank adapters, experts): bad arguments are reported before any HIP
call."""
import pytest
import torch

import weight_only_bit_q4_amd as q

P = 0x10000
BIG = 1 << 40


def lora(fmt=0, ptrs=None, n=64, k=128, t=4, adapters=3, rank=16, ws=P, wb=BIG):
    ptrs = [P] * 9 if ptrs is None else ptrs  # x w w_hi scales a b scale ids y
    return q.q4lin_linear_lora(fmt, *ptrs, n, k, t, adapters, rank, ws, wb, 0)


@pytest.mark.parametrize("bad", [dict(k=96), dict(n=-1), dict(t=-1), dict(adapters=0), dict(rank=0), dict(rank=12),
                                 dict(rank=264), dict(t=(1 << 19) + 1), dict(adapters=(1 << 20) + 1)])
def test_lora_shapes(bad):
    args = dict(n=64, k=128, t=4, adapters=3, rank=16)
    args.update(bad)
    for fmt in range(6):
        assert lora(fmt=fmt, **args) == q.Q4LIN_E_SHAPE
        assert q.q4lin_lora_workspace_bytes(fmt, *(args[v] for v in ("n", "k", "t", "adapters", "rank"))) == \
            -q.Q4LIN_E_SHAPE


def test_lora_format_empty_and_workspace():
    assert lora(fmt=6) == q.Q4LIN_E_FORMAT and lora(fmt=-1) == q.Q4LIN_E_FORMAT
    assert q.q4lin_lora_workspace_bytes(9, 64, 128, 4, 3, 16) == -q.Q4LIN_E_FORMAT
    for n, t in ((0, 4), (64, 0)):
        assert lora(ptrs=[0] * 9, n=n, t=t, ws=0, wb=0) == q.Q4LIN_OK
        assert q.q4lin_lora_workspace_bytes(0, n, 128, t, 3, 16) == 0
    for t in (1, 4, 20, 100, 300):
        need = q.q4lin_lora_workspace_bytes(0, 64, 128, t, 3, 16)
        assert need >= 64 * t * 4 + t * 16 * 4
        assert lora(t=t, wb=need - 1) == q.Q4LIN_E_WORKSPACE
        assert lora(t=t, ws=0) == q.Q4LIN_E_NULL
        assert lora(t=t, ws=P + 16) == q.Q4LIN_E_ALIGN


@pytest.mark.parametrize("which", [0, 1, 3, 4, 5, 7, 8])
def test_lora_null(which):
    ptrs = [P] * 9
    ptrs[which] = 0
    assert lora(ptrs=ptrs) == q.Q4LIN_E_NULL


@pytest.mark.parametrize("which,off", [(0, 8), (1, 8), (3, 1), (4, 8), (5, 8), (6, 2), (7, 2), (8, 1)])
def test_lora_alignment(which, off):
    ptrs = [P] * 9
    ptrs[which] += off
    assert lora(ptrs=ptrs) == q.Q4LIN_E_ALIGN


def test_lora_high_plane():
    ptrs = [P] * 9
    ptrs[2] = 0
    assert lora(fmt=q.Q4LIN_FMT_Q5G64_F16S, ptrs=ptrs) == q.Q4LIN_E_NULL
    ptrs[2] = P + 4
    assert lora(fmt=q.Q4LIN_FMT_Q6G64_F16S, ptrs=ptrs) == q.Q4LIN_E_ALIGN


def experts(ptrs=None, inner=64, k=128, e=4, top_k=2, t=3, ws=P, wb=BIG):
    ptrs = [P] * 10 if ptrs is None else ptrs  # x ids weights six planes y
    return q.q4lin_moe_experts(*ptrs, inner, k, e, top_k, t, ws, wb, 0)


def layer(ptrs=None, inner=64, k=128, e=4, top_k=2, t=3, ws=P, wb=BIG):
    ptrs = [P] * 11 if ptrs is None else ptrs  # x router six planes y ids weights
    return q.q4lin_moe(*ptrs, inner, k, e, top_k, t, 1, ws, wb, 0)


@pytest.mark.parametrize("bad", [dict(inner=0), dict(inner=96), dict(k=96), dict(k=0), dict(e=0), dict(e=1025),
                                 dict(top_k=0), dict(top_k=5), dict(t=-1),
                                 dict(k=1 << 20, t=1 << 10), dict(inner=1 << 20, t=1 << 9)])
def test_moe_shapes(bad):
    args = dict(inner=64, k=128, e=4, top_k=2, t=3)
    args.update(bad)
    assert experts(**args) == q.Q4LIN_E_SHAPE
    assert layer(**args) == q.Q4LIN_E_SHAPE
    assert q.q4lin_moe_workspace_bytes(args["inner"], args["k"], args["e"], args["top_k"], args["t"]) == \
        -q.Q4LIN_E_SHAPE


@pytest.mark.parametrize("bad", [dict(k=96), dict(e=0), dict(e=1025), dict(top_k=0), dict(top_k=5), dict(t=-1)])
def test_moe_route_shapes(bad):
    a = dict(k=128, e=4, top_k=2, t=3)
    a.update(bad)
    assert q.q4lin_moe_route(P, P, P, P, a["k"], a["e"], a["top_k"], a["t"], 1, 0) == q.Q4LIN_E_SHAPE


def test_moe_empty_and_workspace():
    assert experts(ptrs=[0] * 10, t=0, ws=0, wb=0) == q.Q4LIN_OK
    assert layer(ptrs=[0] * 11, t=0, ws=0, wb=0) == q.Q4LIN_OK
    assert q.q4lin_moe_route(0, 0, 0, 0, 128, 4, 2, 0, 1, 0) == q.Q4LIN_OK
    assert q.q4lin_moe_workspace_bytes(64, 128, 4, 2, 0) == 0
    need = q.q4lin_moe_workspace_bytes(64, 128, 4, 2, 3)
    assert need > 0
    for call in (experts, layer):
        assert call(wb=need - 1) == q.Q4LIN_E_WORKSPACE
        assert call(ws=0) == q.Q4LIN_E_NULL
        assert call(ws=P + 16) == q.Q4LIN_E_ALIGN


@pytest.mark.parametrize("which", range(11))
def test_moe_null_and_alignment(which):
    off = {0: 8, 1: 8, 2: 8, 3: 1, 4: 8, 5: 1, 6: 8, 7: 1, 8: 1, 9: 2, 10: 2}[which]
    for value, status in ((0, q.Q4LIN_E_NULL), (P + off, q.Q4LIN_E_ALIGN)):
        ptrs = [P] * 11
        ptrs[which] = value
        assert layer(ptrs=ptrs) == status
    if which < 10:
        off = {0: 8, 1: 2, 2: 2, 3: 8, 4: 1, 5: 8, 6: 1, 7: 8, 8: 1, 9: 1}[which]
        for value, status in ((0, q.Q4LIN_E_NULL), (P + off, q.Q4LIN_E_ALIGN)):
            ptrs = [P] * 10
            ptrs[which] = value
            assert experts(ptrs=ptrs) == status
    if which < 4:
        ptrs = [P] * 4
        ptrs[which] = 0
        assert q.q4lin_moe_route(*ptrs, 128, 4, 2, 3, 1, 0) == q.Q4LIN_E_NULL
        ptrs[which] = P + (8 if which < 2 else 2)
        assert q.q4lin_moe_route(*ptrs, 128, 4, 2, 3, 1, 0) == q.Q4LIN_E_ALIGN


# -- the torch calls name what does not fit (CPU tensors: refused before any launch)
def test_torch_calls_refuse_shapes():
    x = torch.zeros(3, 128, dtype=torch.bfloat16)
    c, s = torch.zeros(64, 64, dtype=torch.uint8), torch.zeros(64, 2, dtype=torch.float16)
    a, b = torch.zeros(2, 8, 128, dtype=torch.bfloat16), torch.zeros(2, 64, 8, dtype=torch.bfloat16)
    ids = torch.zeros(3, dtype=torch.int32)
    for bad in (dict(x=x[:, ::2]), dict(lora_a=a[:, :, :64]), dict(lora_b=b[:1]), dict(adapter_ids=ids.long()),
                dict(adapter_ids=ids[:2]), dict(codes=c[:, :32]), dict(scales=s[:, :1]),
                dict(lora_scale=torch.zeros(3)), dict(fmt=q.Q4LIN_FMT_Q5G64_F16S)):
        args = dict(x=x, codes=c, scales=s, lora_a=a, lora_b=b, adapter_ids=ids)
        args.update(bad)
        with pytest.raises(ValueError):
            q.linear_lora(**args)
    with pytest.raises(q.Q4LinError):
        q.linear_lora(x, c, s, a, b, ids, fmt=17)
    planes = [torch.zeros(4, 64, 64, dtype=torch.uint8), torch.zeros(4, 64, 2, dtype=torch.float16)] * 2 + \
        [torch.zeros(4, 128, 32, dtype=torch.uint8), torch.zeros(4, 128, 1, dtype=torch.float16)]
    w = torch.zeros(3, 2)
    for i in range(6):
        bad = list(planes)
        bad[i] = bad[i][:, 1:]
        with pytest.raises(ValueError):
            q.moe_experts(x, torch.zeros(3, 2, dtype=torch.int32), w, *bad)
    with pytest.raises(ValueError):
        q.moe_experts(x, torch.zeros(3, 2, dtype=torch.int64), w, *planes)
    with pytest.raises(ValueError):
        q.moe(x, torch.zeros(5, 128, dtype=torch.bfloat16), *planes, 2)
