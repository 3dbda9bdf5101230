"""Host-side checks of the sorted-row and integer-product entry points: every
refusal happens before anything is enqueued, so no GPU is needed (the pointers
are never followed)."""
import pytest

import block_quantized_expert_gb300 as bqe

P = 4096  # any aligned, non-NULL address
BAD = bqe.MOE_ERR_INVALID_ARG


def refused(call, name, args, word):
    lib = bqe.load_library()
    assert getattr(lib, name)(*args) == BAD, (name, call)
    msg = bqe.moe_last_error()
    assert name in msg and word in msg, msg


GOOD = {
    "moe_dispatch": [P, 1, 64, 4, 2, 64, P, 8, P, P, 64, None],
    "moe_dispatch_backward": [P, 1, 64, 4, 2, 64, P, P, 0, 64, None],
    "moe_combine": [P, 1, 64, P, 4, 2, 64, P, P, 0, 64, None],
    "moe_combine_backward": [P, 1, 64, P, 1, 64, P, 4, 2, 64, P, 8, P, P, 64, P, None],
    "moe_route_backward": [P, P, P, 4, 8, 2, 1.5, P, None],
    "moe_quantize_rows": [P, 1, 64, 0, 4, 64, P, 64, P, None],
    "moe_expert_product": [P, 64, 4, P, 64, P, P, 8, 32, P, P, 2, 8, P, 1, 32, None],
}
REFUSALS = [
    # name, argument, value, word of the message
    ("moe_dispatch", 0, None, "NULL"), ("moe_dispatch", 1, 3, "dtype"), ("moe_dispatch", 2, 63, "stride"),
    ("moe_dispatch", 3, -1, "T"), ("moe_dispatch", 3, 1 << 30, "T"), ("moe_dispatch", 4, 0, "top_k"),
    ("moe_dispatch", 4, 9, "top_k"), ("moe_dispatch", 5, 0, "hidden"), ("moe_dispatch", 6, None, "NULL"),
    ("moe_dispatch", 7, 0, "n_experts"), ("moe_dispatch", 7, 1025, "n_experts"), ("moe_dispatch", 8, None, "NULL"),
    ("moe_dispatch", 9, P + 1, "aligned"), ("moe_dispatch", 10, 1 << 41, "stride"),
    ("moe_dispatch_backward", 0, P + 1, "aligned"), ("moe_dispatch_backward", 6, None, "NULL"),
    ("moe_dispatch_backward", 8, 2, "dtype"), ("moe_dispatch_backward", 9, 1, "stride"),
    ("moe_combine", 1, -1, "dtype"), ("moe_combine", 3, None, "NULL"), ("moe_combine", 8, None, "NULL"),
    ("moe_combine", 9, 2, "dtype"), ("moe_combine", 5, 0, "top_k"),
    ("moe_combine_backward", 0, None, "NULL"), ("moe_combine_backward", 1, 2, "dtype"),
    ("moe_combine_backward", 6, None, "NULL"), ("moe_combine_backward", 10, None, "NULL"),
    ("moe_combine_backward", 13, None, "NULL"), ("moe_combine_backward", 15, None, "NULL"),
    ("moe_combine_backward", 14, 63, "stride"),
    ("moe_route_backward", 0, None, "NULL"), ("moe_route_backward", 4, 1, "n_experts"),
    ("moe_route_backward", 6, float("nan"), "w_scale"), ("moe_route_backward", 5, 9, "top_k"),
    ("moe_quantize_rows", 0, None, "NULL"), ("moe_quantize_rows", 1, 7, "dtype"), ("moe_quantize_rows", 2, 63, "stride"),
    ("moe_quantize_rows", 3, 1, "stride"), ("moe_quantize_rows", 4, -1, "rows"), ("moe_quantize_rows", 5, 0, "K"),
    ("moe_quantize_rows", 5, 131073, "K"), ("moe_quantize_rows", 7, 8, "stride"), ("moe_quantize_rows", 8, None, "NULL"),
    ("moe_expert_product", 0, None, "NULL"), ("moe_expert_product", 1, 63, "stride"), ("moe_expert_product", 4, 0, "K"),
    ("moe_expert_product", 4, 131073, "K"), ("moe_expert_product", 7, 0, "n_experts"),
    ("moe_expert_product", 7, 1025, "n_experts"), ("moe_expert_product", 8, 0, "N"),
    ("moe_expert_product", 9, None, "offsets"), ("moe_expert_product", 11, 0, "top_k"),
    ("moe_expert_product", 12, -1, "R"), ("moe_expert_product", 12, (1 << 20) + 1, "R"),
    ("moe_expert_product", 10, None, "rows"), ("moe_expert_product", 13, P + 1, "aligned"),
    ("moe_expert_product", 14, 5, "dtype"), ("moe_expert_product", 15, 31, "stride"),
]


@pytest.mark.parametrize("name,arg,value,word", REFUSALS)
def test_refusals(name, arg, value, word):
    args = list(GOOD[name])
    args[arg] = value
    refused((arg, value), name, args, word)


@pytest.mark.parametrize("name,size", [("moe_dispatch", 3), ("moe_dispatch_backward", 3), ("moe_combine", 4),
                                       ("moe_combine_backward", 7), ("moe_route_backward", 3),
                                       ("moe_quantize_rows", 4), ("moe_expert_product", 12)])
def test_nothing_to_do_is_not_an_error(name, size):
    args = [None if a == P else a for a in GOOD[name]]
    args[size] = 0
    if name == "moe_expert_product":
        args[7], args[9] = 1, None
    assert getattr(bqe.load_library(), name)(*args) == bqe.MOE_OK


def test_binding_checks_tensors():
    import torch

    cpu = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        bqe.moe_quantize_rows(cpu, torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(ValueError, match="top_k"):
        bqe.moe_dispatch_backward(cpu, torch.zeros(9, dtype=torch.int32), cpu)
    with pytest.raises(ValueError, match="CUDA"):
        bqe.moe_dispatch(cpu, torch.zeros(3, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), cpu)
