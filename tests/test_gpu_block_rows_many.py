"""Rows to blocks where there are 1024 of them and more, of 129 to 256 units: NVFP4 rows with scales of their
own take two units a thread there.  Bytes as in test_gpu_block_rows.py."""
import numpy as np
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from tests import _blocks as B
from tests import test_gpu_block_rows as rows_tests
from tests.test_gpu_block_product import blocks, check, product64
from tests.test_gpu_sorted_rows import BF16, F16, F32, rows_of

pytestmark = pytest.mark.gpu
SHAPES = [(1024, 4096, 0), (1500, 2080, 0), (1100, 3104, 8), (1025, 4064, 1), (1023, 4096, 0)]


@pytest.mark.parametrize("rows,K,pad", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_many_rows(rows, K, pad, dtype):
    rows_tests.test_quantize_blocks(rows, K, pad, dtype, B.NVFP4)


@pytest.mark.parametrize("rows,K,pad", SHAPES[1:3])
@pytest.mark.parametrize("fmt", [B.MXFP4, B.NVFP4])
def test_many_gated_rows(rows, K, pad, fmt):
    rows_tests.test_quantize_gated_blocks(rows, K, pad, BF16, fmt)


@pytest.mark.parametrize("rows,K,pad", SHAPES[:3])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_rows_with_given_scales(rows, K, pad, dtype):
    """Each quotient rounded in fp32, here by numpy."""
    x = rows_of(rows, K, dtype, 3, pad)
    g = torch.rand(rows, generator=torch.Generator().manual_seed(K)).add_(0.1).mul_(1e-3).cuda()
    q, s, _ = rows_tests.outputs(rows, K, B.NVFP4)
    bqe.moe_quantize_blocks(x, q, s, g, B.NVFP4, given=True)
    v, g32 = x.float().cpu().numpy(), g.cpu().numpy()
    most = np.abs(v).reshape(rows, -1, 16).max(2)
    want = B.nearest((most / np.float32(6) / g32[:, None]).astype(np.float64), B.FINE)
    assert np.array_equal(s.cpu().numpy(), want)
    d = np.repeat(B.FINE[want].astype(np.float32) * g32[:, None], 16, 1)
    y = np.where(d > 0, v / np.where(d > 0, d, np.float32(1)), np.float32(0))
    c = np.where(d > 0, B.nearest(np.abs(y).astype(np.float64), B.GRID) + 8 * np.signbit(v), 0).astype(np.uint8)
    assert np.array_equal(q.cpu().numpy(), B.pack(c))


@pytest.mark.parametrize("g", [-1.0, -1e-3, float("-inf")])
def test_given_scales_below_zero(g):
    """Block scales are not negative: a row whose given scale is gets scale bytes and codes of 0."""
    x = rows_of(3, 64, F32, 1)
    q, s, _ = rows_tests.outputs(3, 64, B.NVFP4)
    bqe.moe_quantize_blocks(x, q, s, torch.full((3,), g, device="cuda"), B.NVFP4, given=True)
    assert not s.any() and not (q & 0x77).any()


@pytest.mark.parametrize("R,K", [(2, 128), (6, 128), (400, 128)])
def test_offsets_out_of_range(R, K):
    """Offsets are held inside [0, R], whichever form takes the call."""
    E, N, fmt = 4, 72, B.NVFP4
    q, s = blocks((R,), K, fmt, 1)
    wq, ws = blocks((E, N), K, fmt, 2)
    far = torch.tensor([0, -5, R // 2, R // 2, 10 ** 9], dtype=torch.int32, device="cuda")
    out = torch.full((R, N), float("nan"), device="cuda")
    bqe.moe_block_product(q, s, wq, ws, out, far, fmt=fmt)
    want, mag = product64(q, s, None, wq, ws, None, [0, 0, R // 2, R // 2, R], np.arange(R), fmt)
    check(out, want, mag, K, F32)


@pytest.mark.parametrize("K", [96, 4096])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("fmt", [B.MXFP4, B.NVFP4])
def test_zeros_keep_their_sign(K, dtype, fmt):
    """-0 is code 8 beside other values, with scales found and given and behind a gate."""
    x = rows_of(40, 2 * K, dtype, 4)
    x[:, 1::7], x[:, 3::7] = -0.0, 0.0
    for gated in (False, True):
        v = x if gated else x[:, :K]
        q, s, g = rows_tests.outputs(40, K, fmt)
        bqe.moe_quantize_blocks(v, q, s, g, fmt, gated=gated)
        sign = torch.signbit(v[:, :K]) ^ torch.signbit(v[:, K:]) if gated else torch.signbit(v)
        zero = ((v[:, :K] == 0) | (v[:, K:] == 0)) if gated else v == 0
        codes = torch.from_numpy(B.unpack(q.cpu().numpy())).cuda()
        assert torch.equal(codes[zero], sign[zero].to(torch.uint8) * 8)
        if g is not None:
            q2, s2, _ = rows_tests.outputs(40, K, fmt)
            bqe.moe_quantize_blocks(v, q2, s2, g, fmt, gated=gated, given=True)
            assert torch.equal(q2, q) and torch.equal(s2, s)
