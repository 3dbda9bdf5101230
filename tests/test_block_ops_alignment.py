"""Pointers to 4-byte elements off their alignment are refused by the norm's and the 4-bit blocks' C
entries before anything is enqueued (no GPU: the pointers are never followed)."""
import pytest

from tests.test_block_ops_args import GOOD, refused
from tests.test_sorted_ops_args import P

PLACES = [("moe_norm_rows", 14), ("moe_norm_rows", 17), ("moe_norm_rows_backward", 9), ("moe_norm_rows_backward", 14),
          ("moe_quantize_blocks", 10), ("moe_dequantize_blocks", 3), ("moe_block_product", 4), ("moe_block_product", 9),
          ("moe_block_product", 12), ("moe_block_product", 13)]


@pytest.mark.parametrize("name,arg", PLACES)
@pytest.mark.parametrize("off", [1, 2, 3])
def test_misaligned_elements(name, arg, off):
    args = list(GOOD[name])
    assert args[arg] == P
    args[arg] = P + off
    refused((arg, off), name, args, "not aligned to its elements")
