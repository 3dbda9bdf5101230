"""A position whose row is outside q reads zeros, whatever kernel takes the call: 0 times a channel's NaN
byte is NaN, and so is 0 times its NaN or infinite scale; every other channel's product is 0."""
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from tests import _blocks as B
from tests.test_gpu_block_product import FMTS, blocks

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,N", [(1, 40), (2, 203), (3, 40), (40, 203), (300, 300), (4000, 1000)])
@pytest.mark.parametrize("fmt", FMTS)
def test_no_row_times_nan(R, N, fmt):
    K = 4096 if R == 4000 else 256
    q, s = blocks((3,), K, fmt, 1)
    wq, ws = blocks((1, N), K, fmt, 2)
    w_scale = torch.ones(1, N, device="cuda")
    ws[0, 5, 2] = 255 if fmt == B.MXFP4 else 127
    w_scale[0, 9], w_scale[0, 11] = float("nan"), float("inf")
    src = torch.full((R,), 7, dtype=torch.int32, device="cuda")  # past q's three rows
    src[::2] = -1
    out = torch.full((R, N), 3.0, device="cuda")
    bqe.moe_block_product(q, s, wq, ws, out, None, src, 1, None, w_scale, fmt)
    bqe.moe_check_product()
    nan = torch.zeros(N, dtype=torch.bool, device="cuda")
    nan[[5, 9, 11]] = True
    assert torch.equal(torch.isnan(out), nan.expand(R, N)) and not out[:, ~nan].any()
