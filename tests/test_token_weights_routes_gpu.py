"""The layer's routing where the logits are made over the whole chip (more
than 65536 router values, or more than a few tokens, experts or pairs), and
the few-token choice of 65 to 256 experts beside rows of whole lines."""
import pytest
import torch

import token_weights as tw
import weight_only_bit_q4_amd as q4
from gpu_util import announce


pytestmark = pytest.mark.gpu

ROUTES = [  # t, experts, top_k, inner, k
    # a logit a workgroup, then the choice of up to 256 experts
    (12, 64, 6, 64, 1088), (9, 70, 8, 64, 960),
    # four logits a wave, then the choice of up to 256 experts, of up to 1024
    (33, 67, 8, 64, 1024), (64, 128, 8, 64, 576), (17, 256, 3, 64, 320), (21, 300, 8, 64, 256), (13, 1024, 70, 64, 128),
    # few tokens, but more than 256 experts or more than 64 pairs
    (3, 300, 4, 64, 256), (8, 128, 10, 64, 576), (1, 1024, 65, 64, 128),
    # few tokens, 65 to 256 experts, rows of whole 128-byte lines
    (2, 100, 4, 64, 256), (5, 128, 8, 64, 512), (8, 65, 8, 128, 256), (7, 200, 6, 64, 512), (8, 256, 8, 64, 256),
    (1, 129, 5, 64, 768), (4, 16, 3, 64, 512),
]


def layer(t, experts, top_k, k, x, router, planes, renorm=True):
    announce("moe t=%d experts=%d top_k=%d k=%d" % (t, experts, top_k, k))
    out = q4.moe(x.cuda(), router.cuda(), *[p.cuda() for p in planes], top_k, renormalize=renorm)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("t,experts,top_k,inner,k", ROUTES)
@pytest.mark.parametrize("renorm", [True, False])
def test_layer(t, experts, top_k, inner, k, renorm):
    planes, values = tw.expert_weights(experts, inner, k, 7000 + experts)
    x, router = tw.bf16((t, k), 7001 + t), tw.bf16((experts, k), 7002, 1.5 * k ** -0.5)
    y, ids, weights = layer(t, experts, top_k, k, x, router, planes, renorm)
    want_ids, want_w, w_bound = tw.route_reference(x, router, top_k, renorm)
    assert torch.equal(ids.cpu().long(), want_ids)
    assert ((weights.cpu().double() - want_w).abs() <= w_bound).all()
    want, bound = tw.experts_reference(x, ids.cpu(), weights.cpu(), values)
    tw.close(y, want, bound, "moe")
    # the routing alone
    ids2, weights2 = q4.moe_route(x.cuda(), router.cuda(), top_k, renorm)
    assert torch.equal(ids2.cpu().long(), want_ids)
    assert ((weights2.cpu().double() - want_w).abs() <= w_bound).all()


@pytest.mark.parametrize("t,experts,k", [(12, 64, 1088), (33, 128, 576), (11, 300, 256), (3, 300, 256), (6, 100, 256),
                                         (8, 200, 512)])
def test_ties_and_nan(t, experts, k):
    top_k = 6
    planes, values = tw.expert_weights(experts, 64, k, 7100)
    router = tw.bf16((experts, k), 7101, 0.1)
    router[:] = router[:1]  # all equal: the lowest indexes
    x = tw.bf16((t, k), 7102)
    y, ids, weights = layer(t, experts, top_k, k, x, router, planes)
    assert (ids.cpu() == torch.arange(top_k, dtype=torch.int32)).all()
    assert ((weights.cpu() - 1 / top_k).abs() < 1e-6).all()
    want, bound = tw.experts_reference(x, ids.cpu(), weights.cpu(), values)
    tw.close(y, want, bound, "ties")
    router[0, 0] = float("nan")  # the lowest of all, whatever its row
    router[3, 1:] = router[3, 1:] + 0.5 * torch.sign(x[0, 1:])  # the largest for token 0
    _, ids, _ = layer(t, experts, top_k, k, x, router, planes)
    assert ids[0].cpu().tolist() == [3, 1, 2, 4, 5, 6]
    assert (ids.cpu() != 0).all()


@pytest.mark.parametrize("t,experts,top_k,k", [(12, 64, 4, 1088), (40, 300, 3, 256), (5, 100, 4, 512)])
def test_graph_replay(t, experts, top_k, k):
    inner = 64
    planes, values = tw.expert_weights(experts, inner, k, 7200)
    cases = [(tw.bf16((t, k), 7201 + i), tw.bf16((experts, k), 7250 + i, 1.5 * k ** -0.5)) for i in range(3)]
    call = [p.cuda() for p in planes]
    hold = [v.cuda() for v in cases[0]]
    ws = torch.empty(q4.q4lin_moe_workspace_bytes(inner, k, experts, top_k, t), dtype=torch.uint8, device="cuda")
    q4.moe(*hold, *call, top_k, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    announce("moe graph t=%d experts=%d" % (t, experts))
    with torch.cuda.graph(graph):
        y, ids, weights = q4.moe(*hold, *call, top_k, workspace=ws)
    for x, router in cases[::-1]:
        hold[0].copy_(x)
        hold[1].copy_(router)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids.cpu().long(), tw.route_reference(x, router, top_k, True)[0])
        want, bound = tw.experts_reference(x, ids.cpu(), weights.cpu(), values)
        tw.close(y, want, bound, "replay")
        torch.randn(1 << 20, device="cuda").sum().item()
