"""The torch calls of the operators in which each token picks its own weights
refuse tensors of another type or place before any launch: a float16 is not
read as a bf16 of the same size, an address of the host's memory or of another
device never reaches a kernel."""
import pytest
import torch

import weight_only_bit_q4_amd as q


def lora_arguments(device="cpu"):
    z = lambda *shape, dtype: torch.zeros(*shape, dtype=dtype, device=device)  # noqa: E731
    return dict(x=z(3, 128, dtype=torch.bfloat16), codes=z(64, 64, dtype=torch.uint8),
                scales=z(64, 2, dtype=torch.float16), lora_a=z(2, 8, 128, dtype=torch.bfloat16),
                lora_b=z(2, 64, 8, dtype=torch.bfloat16), adapter_ids=z(3, dtype=torch.int32),
                lora_scale=z(2, dtype=torch.float32))


def layer_arguments(device="cpu"):
    z = lambda *shape, dtype: torch.zeros(*shape, dtype=dtype, device=device)  # noqa: E731
    return dict(x=z(3, 128, dtype=torch.bfloat16), router=z(4, 128, dtype=torch.bfloat16),
                ids=z(3, 2, dtype=torch.int32), weights=z(3, 2, dtype=torch.float32),
                codes_gate=z(4, 64, 64, dtype=torch.uint8), scales_gate=z(4, 64, 2, dtype=torch.float16),
                codes_up=z(4, 64, 64, dtype=torch.uint8), scales_up=z(4, 64, 2, dtype=torch.float16),
                codes_down=z(4, 128, 32, dtype=torch.uint8), scales_down=z(4, 128, 1, dtype=torch.float16))


PLANES = ("codes_gate", "scales_gate", "codes_up", "scales_up", "codes_down", "scales_down")
CALLS = {
    "linear_lora": (lora_arguments, tuple(lora_arguments()), {}),
    "moe": (layer_arguments, ("x", "router", *PLANES), {"top_k": 2}),
    "moe_route": (layer_arguments, ("x", "router"), {"top_k": 2}),
    "moe_experts": (layer_arguments, ("x", "ids", "weights", *PLANES), {}),
}
EACH = [(call, name) for call, (_, names, _) in CALLS.items() for name in names]


def refused(call, change, match):
    make, names, more = CALLS[call]
    args = {name: v for name, v in make().items() if name in names}
    args.update(more)
    args.update(change)
    with pytest.raises(ValueError, match=match):
        getattr(q, call)(**args)


# (the planes of a linear_lora weight are read as bytes)
@pytest.mark.parametrize("call,name", [v for v in EACH if v not in (("linear_lora", "codes"), ("linear_lora", "scales"))])
def test_other_types_of_the_same_size(call, name):
    v = CALLS[call][0]()[name]
    other = {torch.bfloat16: torch.float16, torch.float16: torch.bfloat16, torch.uint8: torch.bool,
             torch.int32: torch.float32, torch.float32: torch.int32}[v.dtype]
    refused(call, {name: v.to(other)}, name + " must be a contiguous tensor")


@pytest.mark.parametrize("call,name", EACH)
def test_other_devices(call, name):
    refused(call, {name: CALLS[call][0]("meta")[name]}, "must be on ")


@pytest.mark.parametrize("call", CALLS)
def test_host_memory(call):
    refused(call, {}, "must be on a GPU")
