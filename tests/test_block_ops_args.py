"""Host-side checks of the norm's and the 4-bit blocks' entry points: every refusal
happens before anything is enqueued, so no GPU is needed (the pointers are never
followed)."""
import pytest

import block_quantized_expert_gb300 as bqe
from tests import _blocks as B
from tests.test_sorted_ops_args import P, refused

NAN, INF = float("nan"), float("inf")
GOOD = {
    # x dtype stride residual stride gamma dtype T hidden eps h stride y stride rstd q stride scale
    "moe_norm_rows": [P, 1, 64, P, 64, P, 0, 4, 64, 1e-6, P, 64, P, 64, P, P, 64, P, None],
    # dy dtype stride dh stride h stride gamma dtype rstd T hidden dx stride dgamma scratch bytes
    "moe_norm_rows_backward": [P, 1, 64, P, 64, P, 64, P, 0, P, 4, 64, P, 64, P, P, 1 << 20, None],
    # x dtype stride gated rows K format q stride s scale given
    "moe_quantize_blocks": [P, 1, 64, 0, 4, 64, 1, P, 32, P, P, 0, None],
    # q stride s scale rows K format x dtype stride
    "moe_dequantize_blocks": [P, 32, P, P, 4, 64, 1, P, 1, 64, None],
    # q stride rows s scale K format wq ws w_scale E N offsets row_src top_k R out dtype stride
    "moe_block_product": [P, 32, 4, P, P, 64, 1, P, P, P, 8, 32, P, P, 2, 8, P, 1, 32, None],
}
REFUSALS = [
    ("moe_norm_rows", 0, None, "x is NULL"), ("moe_norm_rows", 0, P + 1, "aligned"), ("moe_norm_rows", 1, 3, "dtype"),
    ("moe_norm_rows", 2, 63, "stride"), ("moe_norm_rows", 3, P + 1, "aligned"), ("moe_norm_rows", 4, 1 << 41, "stride"),
    ("moe_norm_rows", 5, None, "gamma"), ("moe_norm_rows", 6, 2, "gamma"), ("moe_norm_rows", 7, -1, "T"),
    ("moe_norm_rows", 7, (1 << 24) + 1, "T"), ("moe_norm_rows", 8, 0, "hidden"), ("moe_norm_rows", 8, 131073, "hidden"),
    ("moe_norm_rows", 9, -1e-6, "eps"), ("moe_norm_rows", 9, NAN, "eps"), ("moe_norm_rows", 9, INF, "eps"),
    ("moe_norm_rows", 10, P + 1, "aligned"), ("moe_norm_rows", 11, 8, "stride"), ("moe_norm_rows", 13, 8, "stride"),
    ("moe_norm_rows", 15, None, "scale"), ("moe_norm_rows", 16, 8, "stride"), ("moe_norm_rows", 17, None, "scale"),
    ("moe_norm_rows_backward", 0, None, "dy"), ("moe_norm_rows_backward", 1, -1, "dtype"), ("moe_norm_rows_backward", 2, 1, "stride"),
    ("moe_norm_rows_backward", 3, P + 1, "aligned"), ("moe_norm_rows_backward", 5, None, "NULL"),
    ("moe_norm_rows_backward", 7, None, "gamma"), ("moe_norm_rows_backward", 8, 2, "gamma"),
    ("moe_norm_rows_backward", 9, None, "rstd"), ("moe_norm_rows_backward", 10, -1, "T"),
    ("moe_norm_rows_backward", 11, 0, "hidden"), ("moe_norm_rows_backward", 12, None, "dx"),
    ("moe_norm_rows_backward", 13, 63, "stride"), ("moe_norm_rows_backward", 15, None, "scratch"),
    ("moe_norm_rows_backward", 15, P + 8, "scratch"), ("moe_norm_rows_backward", 16, 4 * 64 * 4 - 1, "scratch"),
    ("moe_quantize_blocks", 0, None, "NULL"), ("moe_quantize_blocks", 0, P + 1, "aligned"), ("moe_quantize_blocks", 1, 5, "dtype"),
    ("moe_quantize_blocks", 2, 63, "stride"), ("moe_quantize_blocks", 3, 1, "stride"), ("moe_quantize_blocks", 4, -1, "rows"),
    ("moe_quantize_blocks", 5, 48, "K"), ("moe_quantize_blocks", 5, 0, "K"), ("moe_quantize_blocks", 5, 131104, "K"),
    ("moe_quantize_blocks", 6, 2, "format"), ("moe_quantize_blocks", 6, 0, "scale"), ("moe_quantize_blocks", 7, None, "NULL"),
    ("moe_quantize_blocks", 8, 31, "stride"), ("moe_quantize_blocks", 9, None, "NULL"), ("moe_quantize_blocks", 10, None, "NULL"),
    ("moe_dequantize_blocks", 0, None, "NULL"), ("moe_dequantize_blocks", 1, 31, "stride"), ("moe_dequantize_blocks", 2, None, "NULL"),
    ("moe_dequantize_blocks", 4, -1, "rows"), ("moe_dequantize_blocks", 5, 40, "K"), ("moe_dequantize_blocks", 6, -1, "format"),
    ("moe_dequantize_blocks", 7, P + 1, "aligned"), ("moe_dequantize_blocks", 8, 3, "dtype"), ("moe_dequantize_blocks", 9, 63, "stride"),
    ("moe_block_product", 0, None, "NULL"), ("moe_block_product", 0, P + 8, "aligned"), ("moe_block_product", 1, 31, "stride"),
    ("moe_block_product", 1, 40, "stride"), ("moe_block_product", 1, 1 << 40, "stride"), ("moe_block_product", 2, -1, "R"), ("moe_block_product", 3, None, "NULL"),
    ("moe_block_product", 5, 0, "K"), ("moe_block_product", 5, 48, "K"), ("moe_block_product", 6, 3, "format"),
    ("moe_block_product", 7, None, "NULL"), ("moe_block_product", 7, P + 4, "aligned"), ("moe_block_product", 8, None, "NULL"),
    ("moe_block_product", 10, 0, "n_experts"), ("moe_block_product", 10, 1025, "n_experts"), ("moe_block_product", 11, 0, "N"),
    ("moe_block_product", 12, None, "offsets"), ("moe_block_product", 13, None, "rows"), ("moe_block_product", 14, 9, "top_k"),
    ("moe_block_product", 15, -1, "R"), ("moe_block_product", 15, (1 << 20) + 1, "R"), ("moe_block_product", 16, None, "NULL"),
    ("moe_block_product", 16, P + 1, "aligned"), ("moe_block_product", 17, 5, "dtype"), ("moe_block_product", 18, 31, "stride"),
]


@pytest.mark.parametrize("name,arg,value,word", REFUSALS)
def test_refusals(name, arg, value, word):
    args = list(GOOD[name])
    args[arg] = value
    refused((arg, value), name, args, word)


def test_codes_need_rows_or_an_output():
    args = list(GOOD["moe_norm_rows"])
    args[12] = args[15] = args[17] = None  # neither y nor codes
    refused("no output", "moe_norm_rows", args, "y is NULL")


@pytest.mark.parametrize("name,size", [("moe_norm_rows", 7), ("moe_quantize_blocks", 4), ("moe_dequantize_blocks", 4),
                                       ("moe_block_product", 15)])
def test_nothing_to_do_is_not_an_error(name, size):
    args = [None if a == P else a for a in GOOD[name]]
    args[size] = 0
    if name == "moe_block_product":
        args[10], args[12] = 1, None
    assert getattr(bqe.load_library(), name)(*args) == bqe.MOE_OK


def test_scratch_sizes():
    f = bqe.moe_norm_scratch_bytes
    assert f(1, 64) == 256 and f(0, 64) == 256 and f(10 ** 6, 64) == f(10 ** 5, 64) > f(100, 64) == 25600
    assert f(-1, 64) == f(4, 0) == f(4, 131073) == f((1 << 24) + 1, 64) == 0


def test_binding_checks_tensors():
    import torch

    f, u = torch.zeros(4, 64), torch.zeros(4, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        bqe.moe_norm_rows(f, torch.ones(64), f)
    with pytest.raises(ValueError, match="CUDA"):
        bqe.moe_norm_rows_backward(f, f, torch.ones(64), torch.ones(4), f)
    with pytest.raises(ValueError, match="fmt"):
        bqe.moe_quantize_blocks(f, u, u, None, 2)
    with pytest.raises(ValueError, match="CUDA"):
        bqe.moe_quantize_blocks(f, u, u)
    with pytest.raises(ValueError, match="CUDA"):
        bqe.moe_dequantize_blocks(u, u, f)
    with pytest.raises(ValueError, match="E, N, K"):
        bqe.moe_block_product(u, u, u, u, f)


def test_the_definitions_round_as_the_encoder_does():
    """tests/_blocks.py against the workloads' encoders, on rows away from fp32's own roundings."""
    import numpy as np
    from workloads.generate import encode_mxfp4_rows, encode_nvfp4_rows

    w = np.random.default_rng(0).standard_normal((20, 256)).astype(np.float32)
    q, s = encode_mxfp4_rows(w)
    mine = B.scale_bytes(w.astype(np.float64), B.MXFP4)
    assert np.array_equal(mine, s)
    assert np.array_equal(B.pack(B.codes(w.astype(np.float64), B.scale_values(s, B.MXFP4))), q)
    q, s, g = encode_nvfp4_rows(w)
    wide = np.full(20, float(g))
    assert np.array_equal(B.scale_bytes(w.astype(np.float64), B.NVFP4, wide), s)
    assert np.array_equal(B.pack(B.codes(w.astype(np.float64), B.scale_values(s, B.NVFP4), wide)), q)
