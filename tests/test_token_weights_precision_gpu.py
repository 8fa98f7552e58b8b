"""Rank values and gated values keep 16 significant bits on their way through
the matrix cores: on every kernel that takes them the result is the exact
value rounded once (rounded_once.py)."""
import pytest
import torch

import token_weights as tw
import weight_only_bit_q4_amd as q4
from gpu_util import announce
from rounded_once import rounded_once


pytestmark = pytest.mark.gpu


def dev(v):
    return None if v is None else v.cuda()


# the term in the base product's kernel; the finish by ranks (up to 32, 64, 128, 256) and rows a thread (one, four)
LORA = [(0, 512, 512, 2, 3, 64), (0, 300, 512, 12, 3, 40), (3, 260, 512, 20, 3, 64), (5, 1024, 256, 1, 1, 200),
        (0, 200, 256, 200, 3, 24), (0, 200, 256, 40, 4, 64), (2, 200, 256, 40, 4, 104), (0, 200, 256, 40, 4, 200),
        (0, 2048, 256, 600, 5, 32), (0, 2048, 256, 600, 5, 48), (0, 2050, 256, 600, 5, 128),
        (0, 2048, 256, 600, 5, 256), (1, 2048, 256, 600, 5, 136), (0, 200, 4096, 60, 3, 72)]


@pytest.mark.parametrize("fmt,n,k,t,adapters,rank", LORA)
def test_rank_values(fmt, n, k, t, adapters, rank):
    planes, w64 = tw.weight(fmt, n, k, 6200 + rank)
    x, a = tw.bf16((t, k), 6201 + t), tw.bf16((adapters, rank, k), 6202, k ** -0.5)
    # (a term of four times the base product's size: nearly all of y goes through the rank values)
    b = tw.bf16((adapters, n, rank), 6203, 4.0 * float(w64.std()) * (k / rank) ** 0.5)
    ids = torch.arange(t, dtype=torch.int32) * 7 % adapters
    announce("linear_lora precision fmt=%d n=%d k=%d t=%d rank=%d" % (fmt, n, k, t, rank))
    y = q4.linear_lora(dev(x), dev(planes[0]), dev(planes[2]), dev(a), dev(b), dev(ids), fmt=fmt, codes_hi=dev(planes[1]))
    torch.cuda.synchronize()
    want, bound = tw.lora_reference(x, w64, a, b, ids, None, False)
    rounded_once(y, want, "linear_lora")


# tokens of each expert: down products of few pairs (16 and 32 rows a workgroup); shared activations with up to 8 and
# 16 pairs a pass; 32 a pass with few and many of them
EXPERTS = [([1], 512, 1024), ([1], 256, 4160), ([2, 1, 0, 0, 0, 0, 0, 0, 2, 0, 0, 0, 0, 0, 0, 0], 256, 1024),
           ([6, 3, 8], 512, 1024), ([12, 16, 9, 13], 512, 640), ([40, 10, 30, 9], 192, 320), ([20, 33, 64], 512, 320),
           ([17, 31], 1088, 256)]


@pytest.mark.parametrize("counts,inner,k", EXPERTS)
def test_gated_values(counts, inner, k):
    t = sum(counts)
    planes, values = tw.expert_weights(len(counts), inner, k, 6300)
    x = tw.bf16((t, k), 6301)
    ids = torch.tensor([e for e, c in enumerate(counts) for _ in range(c)], dtype=torch.int32)[:, None]
    ids = ids[torch.randperm(t, generator=torch.Generator().manual_seed(6302))].contiguous()
    weights = torch.rand(t, 1, generator=torch.Generator().manual_seed(6303)) + 0.5
    announce("moe_experts precision counts=%s inner=%d k=%d" % (counts, inner, k))
    y = q4.moe_experts(dev(x), dev(ids), dev(weights), *[dev(p) for p in planes])
    torch.cuda.synchronize()
    want, bound = tw.experts_reference(x, ids, weights, values)
    rounded_once(y, want, "moe_experts")


@pytest.mark.parametrize("t,experts,top_k,inner,k", [(1, 16, 4, 256, 1024), (6, 40, 3, 192, 512), (8, 4, 4, 128, 512)])
def test_gated_values_of_the_layer(t, experts, top_k, inner, k):
    planes, values = tw.expert_weights(experts, inner, k, 6400)
    x, router = tw.bf16((t, k), 6401), tw.bf16((experts, k), 6402, 1.5 * k ** -0.5)
    announce("moe precision t=%d experts=%d" % (t, experts))
    y, ids, weights = q4.moe(dev(x), dev(router), *[dev(p) for p in planes], top_k)
    torch.cuda.synchronize()
    want, bound = tw.experts_reference(x, ids.cpu(), weights.cpu(), values)
    rounded_once(y, want, "moe")


@pytest.mark.parametrize("t", [1, 7, 30, 100])
def test_calls_repeat_to_the_bit(t):
    """No sum depends on the order in which workgroups run."""
    planes, _ = tw.expert_weights(5, 192, 512, 6500)
    x, router = dev(tw.bf16((t, 512), 6501)), dev(tw.bf16((5, 512), 6502, 0.1))
    call = [dev(p) for p in planes]
    w, _ = tw.weight(0, 300, 512, 6503)
    a, b = dev(tw.bf16((4, 48, 512), 6504, 0.05)), dev(tw.bf16((4, 300, 48), 6505))
    adapter_ids = dev(torch.arange(t, dtype=torch.int32) % 5 - 1)
    announce("repeats t=%d" % t)
    first = (*q4.moe(x, router, *call, 2), q4.linear_lora(x, dev(w[0]), dev(w[2]), a, b, adapter_ids))
    for _ in range(5):
        again = (*q4.moe(x, router, *call, 2), q4.linear_lora(x, dev(w[0]), dev(w[2]), a, b, adapter_ids))
        for u, v in zip(first, again):
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))
