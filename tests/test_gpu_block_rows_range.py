"""moe_dequantize_blocks at the ends of fp32's range: code * block scale * row scale is rounded
once, also where block scale * row scale alone overflows or falls below the normal numbers."""
import numpy as np
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from tests import _blocks as B
from tests.test_gpu_sorted_rows import BF16, F32

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
# row scales that take 2^-127 .. 2^127 over both ends, and ordinary ones between them
SCALES = [2.0 ** 30, 3e38, 1.7 * 2.0 ** 100, 2.0, 0.3, 1.0, -1.3, 1e-3, 1.1 * 2.0 ** -60, 2.0 ** -126, 1e-45, 0.0, -2.0 ** 120, INF, NAN]


@pytest.mark.parametrize("K", [32, 4096, 2080])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_mxfp4_bytes_times_a_row_scale(K, dtype):
    rows = len(SCALES) * 16
    g = torch.tensor(SCALES * 16, device="cuda")
    s = (torch.arange(rows * K // 32, device="cuda") * 37 % 256).to(torch.uint8).view(rows, -1)
    s[:, 0] = torch.arange(rows, device="cuda") // len(SCALES) * 17  # 0, 17, .. 255 beside every scale
    q = (torch.arange(rows * K // 2, device="cuda") * 41 % 256).to(torch.uint8).view(rows, -1)
    q[:, ::5] = 0  # codes 0 in every block
    x = torch.empty(rows, K, dtype=dtype, device="cuda")
    bqe.moe_dequantize_blocks(q, s, x, g, B.MXFP4)
    v = torch.from_numpy(B.values(q.cpu().numpy(), s.cpu().numpy(), B.MXFP4)).cuda()
    want = (v * g.double()[:, None]).float().to(dtype)  # v g is exact in 64 bits: 2 bits and 24
    assert torch.equal(torch.isnan(x), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(x, 0.0, INF, -INF), torch.nan_to_num(want, 0.0, INF, -INF))


@pytest.mark.parametrize("byte,g", [(227, 2.0 ** 30), (254, 2.0), (0, 2.0 ** -20), (3, 0.7)])
def test_one_block(byte, g):
    """2^100 by 2^30 leaves fp32, 0 times it does not, nor does 2^127 by half of 2."""
    q = torch.from_numpy(B.pack(np.arange(32, dtype=np.uint8)[None] % 16)).cuda()
    s, x = torch.full((1, 1), byte, dtype=torch.uint8, device="cuda"), torch.empty(1, 32, device="cuda")
    bqe.moe_dequantize_blocks(q, s, x, torch.full((1,), g, device="cuda"), B.MXFP4)
    c = np.arange(32) % 16
    want = np.where(c > 7, -1, 1) * B.GRID[c & 7] * 2.0 ** (byte - 127) * float(np.float32(g))
    with np.errstate(over="ignore"):
        assert np.array_equal(x[0].cpu().numpy(), want.astype(np.float32))
