"""The torch calls of the operators in which each token picks its own weights
on a stream other than the current one: what they allocate is that stream's, so
that work of the current stream that has not run yet cannot write into it."""
import pytest
import torch

import token_weights as tw
import weight_only_bit_q4_amd as q4
from gpu_util import announce


pytestmark = pytest.mark.gpu

T, K = 24, 256


def calls():
    planes, values = tw.expert_weights(6, 192, K, 7300)
    x, router = tw.bf16((T, K), 7301), tw.bf16((6, K), 7302, 0.1)
    w, _ = tw.weight(0, K, K, 7303)
    a, b = tw.bf16((3, 16, K), 7304, 0.06), tw.bf16((3, K, 16), 7305)
    adapters = torch.arange(T, dtype=torch.int32) % 4 - 1
    d = lambda *v: [u.cuda() for u in v]  # noqa: E731
    x, router, codes, scales, a, b, adapters = d(x, router, w[0], w[2], a, b, adapters)
    planes = d(*planes)
    ids, weights = q4.moe_route(x, router, 2)
    many = torch.arange(8, dtype=torch.int32, device="cuda").repeat(T, 1)  # (more choices than experts)
    some = torch.rand(T, 8, device="cuda")
    return {
        "linear_lora": lambda **kw: (q4.linear_lora(x, codes, scales, a, b, adapters, **kw),),
        "moe_route": lambda **kw: q4.moe_route(x, router, 2, **kw),
        "moe_experts": lambda **kw: (q4.moe_experts(x, ids, weights, *planes, **kw),),
        "moe_experts_share": lambda **kw: (q4.moe_experts(x, many, some, *planes, **kw),),
        "moe": lambda **kw: q4.moe(x, router, *planes, 2, **kw),
    }


@pytest.mark.parametrize("name", ["linear_lora", "moe_route", "moe_experts", "moe_experts_share", "moe"])
def test_own_memory_on_another_stream(name):
    call = calls()[name]
    want = [v.clone() for v in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    announce("%s on another stream" % name)
    busy = torch.randn(2048, 2048, device="cuda")
    for _ in range(3):
        # memory of the current stream, free again for it, with writes to it still waiting behind long work
        scratch = [torch.empty_like(v) for v in want for _ in range(8)]
        scratch += [torch.empty(1 << 16, dtype=torch.uint8, device="cuda") for _ in range(8)]
        taken = {v.data_ptr() for v in scratch}
        for _ in range(20):
            busy = (busy @ busy).mul_(1e-3)
        for v in scratch:
            v.fill_(7)
        del scratch, v
        got = call(stream=side.cuda_stream)
        assert not taken & {v.data_ptr() for v in got}
        torch.cuda.synchronize()
        for u, v in zip(got, want):
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


def test_current_and_given_streams():
    call = calls()["moe"]
    want = [v.clone() for v in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (torch.cuda.current_stream().cuda_stream, 0, side.cuda_stream):
        got = call(stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want))
    with torch.cuda.stream(side):
        for stream in (None, side.cuda_stream, torch.cuda.default_stream().cuda_stream):
            got = call(stream=stream)
            torch.cuda.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(got, want))
            assert torch.cuda.current_stream() == side


def test_own_output_and_workspace():
    """The caller's y and workspace on another stream."""
    x, w = tw.bf16((T, K), 7310), tw.weight(0, K, K, 7303)[0]
    a, b = tw.bf16((3, 16, K), 7304, 0.06), tw.bf16((3, K, 16), 7305)
    args = [v.cuda() for v in (x, w[0], w[2], a, b, torch.arange(T, dtype=torch.int32) % 3)]
    want = q4.linear_lora(*args)
    y = torch.empty_like(want)
    ws = torch.empty(q4.q4lin_lora_workspace_bytes(0, K, K, T, 3, 16), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = q4.linear_lora(*args, y=y, workspace=ws, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert out is y and torch.equal(y, want)
