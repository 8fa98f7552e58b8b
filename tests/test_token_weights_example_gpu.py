"""The example that runs the adapters and the experts together."""
import importlib.util
import os

import pytest
import torch

import token_weights as tw
import weight_only_bit_q4_amd as q4
from gpu_util import announce

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "token_weights_block.py")


def block(tokens):
    spec = importlib.util.spec_from_file_location("token_weights_block", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module.TokenWeightsBlock(tokens, width=256, inner=128, experts=12, top_k=3, adapters=4, rank=16)


def values(codes, scales):
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double() - 8
    return q * scales.double().repeat_interleave(64, -1)


@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_block(tokens):
    b = block(tokens)
    announce("token_weights_block tokens=%d" % tokens)
    graph, x, adapter_ids, y, ids = b.capture(tokens)
    for seed in range(3):
        x.copy_(tw.bf16((tokens, 256), 3000 + seed))
        adapter_ids.copy_(torch.randint(-1, 4, (tokens,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        # step by step in 64 bits, from what the step before gave
        p = q4.linear_lora(x, *b.w, b.lora_a, b.lora_b, adapter_ids, b.lora_scale)
        want, bound = tw.lora_reference(x.cpu(), values(*(v.cpu() for v in b.w)), b.lora_a.cpu(), b.lora_b.cpu(),
                                        adapter_ids.cpu(), b.lora_scale.cpu(), False)
        tw.close(p, want, bound, "projection")
        h = x + p
        m, chosen, weights = q4.moe(h, b.router, *b.experts, b.top_k)
        e = [v.cpu() for v in b.experts]
        want, bound = tw.experts_reference(h.cpu(), chosen.cpu(), weights.cpu(),
                                           [values(e[0], e[1]), values(e[2], e[3]), values(e[4], e[5])])
        tw.close(m, want, bound, "experts")
        assert torch.equal(ids, chosen) and torch.equal(y, h + m)
        torch.randn(1 << 20, device="cuda").sum().item()
