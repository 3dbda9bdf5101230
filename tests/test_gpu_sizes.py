"""Sizes past 32 bits are refused by the calls without a layer: their low bits alone would be a small call.
(Nothing is written to these tensors, which torch.empty only reserves.)"""
import pytest
import torch

import block_quantized_expert_gb300 as bqe

pytestmark = pytest.mark.gpu
FAR = (1 << 32) + 4


def empty(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda")


def f32(*shape):
    return empty(*shape, dtype=torch.float32)


def u8(*shape):
    return empty(*shape, dtype=torch.uint8)


def i32(*shape):
    return empty(*shape, dtype=torch.int32)


CALLS = {
    "norm, rows": lambda: bqe.moe_norm_rows(empty(FAR, 1), f32(1), empty(FAR, 1)),
    "norm, hidden": lambda: bqe.moe_norm_rows(empty(1, FAR), f32(FAR), empty(1, FAR)),
    "norm's gradient": lambda: bqe.moe_norm_rows_backward(empty(FAR, 1), empty(FAR, 1), f32(1), f32(FAR), empty(FAR, 1)),
    "norm, a stream": lambda: bqe.moe_norm_rows(empty(FAR, 1), f32(1), empty(FAR, 1), stream=torch.cuda.current_stream()),
    "block product, positions": lambda: bqe.moe_block_product(u8(4, 16), u8(4, 2), u8(1, 1, 16), u8(1, 1, 2), empty(FAR, 1)),
    "block product, channels": lambda: bqe.moe_block_product(u8(1, 16), u8(1, 2), u8(1, FAR, 16), u8(1, FAR, 2), empty(1, FAR)),
    "block product, rows": lambda: bqe.moe_block_product(u8(FAR, 16), u8(FAR, 2), u8(1, 1, 16), u8(1, 1, 2), empty(4, 1)),
    "block product, top_k": lambda: bqe.moe_block_product(u8(4, 16), u8(4, 2), u8(1, 1, 16), u8(1, 1, 2), empty(4, 1), None, i32(4), FAR),
    "integer product, positions": lambda: bqe.moe_expert_product(empty(4, 16, dtype=torch.int8), f32(4),
                                                                  empty(1, 1, 16, dtype=torch.int8), f32(1, 1), empty(FAR, 1)),
    "8-bit codes": lambda: bqe.moe_quantize_rows(empty(FAR, 1), empty(FAR, 1, dtype=torch.int8), f32(FAR)),
    "dispatch": lambda: bqe.moe_dispatch(empty(FAR, 1), i32(2), i32(FAR), empty(FAR, 1)),
    "combine": lambda: bqe.moe_combine(empty(FAR, 1), f32(FAR, 1), i32(FAR), empty(FAR, 1)),
    "router's gradient": lambda: bqe.moe_route_backward(f32(FAR, 1), i32(FAR, 1), f32(FAR, 1), f32(FAR, 1)),
    "sort": lambda: bqe.moe_permute_noalloc(i32(FAR, 1), 1, i32(2), i32(FAR), i32(FAR)),
}


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("call", CALLS)
def test_sizes_past_32_bits(call):
    with pytest.raises(ValueError, match="below 2\\^31"):
        CALLS[call]()


def test_scratch_of_such_sizes():
    assert bqe.moe_norm_scratch_bytes(FAR, 64) == bqe.moe_norm_scratch_bytes(4, FAR) == 0
    assert bqe.moe_permute_scratch_bytes(FAR, 1, 8) == bqe.moe_permute_scratch_bytes(4, 1, FAR) == 0
