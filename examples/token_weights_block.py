#!/usr/bin/env python3
"""A decoding step in which each token picks its own weights: a projection
with the request's low-rank adapter, then a mixture-of-experts layer, captured
in one HIP graph and replayed step by step.

    python examples/token_weights_block.py [--tokens 16] [--steps 50]

Random weights; prints the time of a step.  The requests' adapters are an
input (``adapter_ids``), so one graph serves any mix of requests.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import weight_only_bit_q4_amd as q4  # noqa: E402


class TokenWeightsBlock:
    """x -> h = x + W x + s_a B_a A_a x -> h + experts(h), for up to ``tokens`` requests."""

    def __init__(self, tokens, width, inner, experts, top_k, adapters, rank, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.top_k = top_k

        def q4_weight(*shape):  # [..., rows, K]: codes and scales of values of about one after a sum over K
            *rows, k = shape
            codes = torch.randint(0, 256, (*rows, k // 2), generator=g, device=device, dtype=torch.uint8)
            scales = (torch.rand(*rows, k // 64, generator=g, device=device) + 0.5) * (k ** -0.5 / 4.6)
            return codes, scales.to(torch.float16)

        def bf16(*shape, std):
            return (torch.randn(*shape, generator=g, device=device) * std).to(torch.bfloat16)

        self.w = q4_weight(width, width)
        self.lora_a, self.lora_b = bf16(adapters, rank, width, std=width ** -0.5), bf16(adapters, width, rank,
                                                                                       std=rank ** -0.5)
        self.lora_scale = torch.full((adapters,), 0.5, device=device)
        self.router = bf16(experts, width, std=1.5 * width ** -0.5)
        self.experts = (*q4_weight(experts, inner, width), *q4_weight(experts, inner, width),
                        *q4_weight(experts, width, inner))
        # one workspace for both calls of a step, which follow one another on a stream
        need = max(q4.q4lin_lora_workspace_bytes(q4.Q4LIN_FMT_Q4G64_F16S, width, width, tokens, adapters, rank),
                   q4.q4lin_moe_workspace_bytes(inner, width, experts, top_k, tokens))
        self.workspace = torch.empty(need, dtype=torch.uint8, device=device)

    def step(self, x, adapter_ids):
        """(y [T, width] bf16, the experts of each token) of x [T, width] bf16 and adapter_ids int32 [T]."""
        p = q4.linear_lora(x, *self.w, self.lora_a, self.lora_b, adapter_ids, self.lora_scale,
                           workspace=self.workspace)
        h = x + p
        m, ids, _ = q4.moe(h, self.router, *self.experts, self.top_k, workspace=self.workspace)
        return h + m, ids

    def capture(self, tokens):
        """(graph, x, adapter_ids, y, ids): fill x and adapter_ids, replay, read y and ids."""
        x = torch.zeros(tokens, self.router.shape[1], dtype=torch.bfloat16, device=self.router.device)
        adapter_ids = torch.full((tokens,), -1, dtype=torch.int32, device=x.device)
        self.step(x, adapter_ids)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, ids = self.step(x, adapter_ids)
        return graph, x, adapter_ids, y, ids


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=768)
    ap.add_argument("--experts", type=int, default=128)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--adapters", type=int, default=32)
    ap.add_argument("--rank", type=int, default=16)
    a = ap.parse_args()
    block = TokenWeightsBlock(a.tokens, a.width, a.inner, a.experts, a.top_k, a.adapters, a.rank)
    graph, x, adapter_ids, y, ids = block.capture(a.tokens)
    x.normal_()
    adapter_ids.copy_(torch.randint(-1, a.adapters, (a.tokens,), dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    us = (time.perf_counter() - t0) / a.steps * 1e6
    print("%d tokens, %d of %d experts in use: %.1f us a step" % (a.tokens, ids.unique().numel(), a.experts, us))


if __name__ == "__main__":
    main()
