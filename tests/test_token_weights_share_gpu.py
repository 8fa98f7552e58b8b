"""One process's share of a layer's experts, smaller than the number of
choices of a token."""
import pytest
import torch

import token_weights as tw
import weight_only_bit_q4_amd as q4
from gpu_util import announce


pytestmark = pytest.mark.gpu


def share(t, top_k, every, experts, inner, k, seed):
    planes, values = tw.expert_weights(experts, inner, k, seed)
    x = tw.bf16((t, k), seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    ids = torch.rand(t, every, generator=g).argsort(1)[:, :top_k].to(torch.int32)
    return [p.cuda() for p in planes], values, x, ids, torch.rand(t, top_k, generator=g)


@pytest.mark.parametrize("t,top_k,every,experts,inner,k", [
    (1, 8, 128, 4, 128, 192), (5, 8, 16, 4, 64, 320), (40, 8, 12, 7, 192, 256), (200, 6, 8, 1, 64, 128),
    (3, 3, 3, 2, 64, 64), (70, 10, 128, 3, 64, 128)])
def test_share_smaller_than_top_k(t, top_k, every, experts, inner, k):
    planes, values, x, ids, weights = share(t, top_k, every, experts, inner, k, 5000 + t)
    weights[ids >= experts] = float("nan")  # of choices that count for nothing here
    if t > 2:
        ids[1] = -1
        ids[2], weights[2] = 0, 0.25  # an expert named by every choice counts as often
    announce("moe_experts share t=%d top_k=%d experts=%d" % (t, top_k, experts))
    y = q4.moe_experts(x.cuda(), ids.cuda(), weights.cuda(), *planes)
    torch.cuda.synchronize()
    want, bound = tw.experts_reference(x, ids, weights, values)
    tw.close(y, want, bound, "share")
    if t > 2:
        assert (y[1] == 0).all()


def test_share_on_another_stream():
    planes, values, x, ids, weights = share(9, 8, 12, 4, 64, 128, 5100)
    args = [v.cuda() for v in (x, ids, weights)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    announce("moe_experts share on another stream")
    y = q4.moe_experts(*args, *planes, stream=side.cuda_stream)
    side.synchronize()
    want, bound = tw.experts_reference(x, ids, weights, values)
    tw.close(y, want, bound, "side stream")


def test_share_graph_replay():
    t, top_k, experts, inner, k = 20, 8, 4, 64, 128
    cases = [share(t, top_k, 12, experts, inner, k, 5200 + 10 * i) for i in range(3)]
    hold = [v.cuda() for v in cases[0][2:]]
    planes = cases[0][0]
    ws = torch.empty(q4.q4lin_moe_workspace_bytes(inner, k, experts, experts, t), dtype=torch.uint8, device="cuda")
    q4.moe_experts(*hold, *planes, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    announce("moe_experts share graph")
    with torch.cuda.graph(graph):
        y = q4.moe_experts(*hold, *planes, workspace=ws)
    for _, _, x, ids, weights in cases[::-1]:
        for h, v in zip(hold, (x, ids, weights)):
            h.copy_(v)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        want, bound = tw.experts_reference(x, ids, weights, cases[0][1])
        tw.close(y, want, bound, "replay")
        torch.randn(1 << 20, device="cuda").sum().item()
