"""moe_block_product at the ends of its ranges, in each of its forms: rows and blocks of zeros (MXFP4 byte 0),
the longest K, a first call that is captured."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from tests import _blocks as B
from tests.test_gpu_block_product import FMTS, blocks, check, product64, scales
from tests.test_gpu_sorted_rows import BF16, F32, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,N", [(1, 512, 40), (2, 512, 40), (40, 512, 200), (4000, 4096, 1000)])
@pytest.mark.parametrize("fmt", FMTS)
def test_rows_and_blocks_of_zeros(M, K, N, fmt):
    """Tokens and weights as moe_quantize_blocks makes them, with zeros among them."""
    n = B.size(fmt)
    x, w = rows_of(M, K, BF16, 1), rows_of(N, K, F32, 2)
    x[::3, 32:96], x[:, -32:], x[M // 2] = 0, 0, 0
    w[::5, :64], w[7] = 0, 0

    def made(t):
        q, s = torch.empty(t.shape[0], K // 2, dtype=torch.uint8, device="cuda"), torch.empty(t.shape[0], K // n, dtype=torch.uint8, device="cuda")
        g = torch.empty(t.shape[0], device="cuda") if fmt == B.NVFP4 else None
        bqe.moe_quantize_blocks(t, q, s, g, fmt)
        return q, s, g

    (q, s, g), (wq, ws, wg) = made(x), made(w)
    out = torch.full((M, N), float("nan"), device="cuda")
    wq, ws, wg = wq[None], ws[None], None if wg is None else wg[None]
    bqe.moe_block_product(q, s, wq, ws, out, scale=g, w_scale=wg, fmt=fmt)
    bqe.moe_check_product()
    assert not out[M // 2].any() and not out[:, 7].any()
    want, mag = product64(q, s, g, wq, ws, wg, [0, M], np.arange(M), fmt)
    check(out, want, mag, K, F32)


@pytest.mark.parametrize("M,N", [(1, 9), (2, 40), (20, 130), (2000, 1200)])
@pytest.mark.parametrize("fmt", FMTS)
def test_longest_rows(M, N, fmt):
    K = 131072
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert bqe.moe_test_block_product_form(1, M, K, N, sms) == {1: 0, 2: 0, 20: 1, 2000: 2}[M]
    q, s = blocks((M,), K, fmt, 1)
    wq, ws = blocks((1, N), K, fmt, 2)
    scale, w_scale = scales((M,), 3), scales((1, N), 4)
    out = torch.empty(M, N, device="cuda")
    bqe.moe_block_product(q, s, wq, ws, out, scale=scale, w_scale=w_scale, fmt=fmt)
    bqe.moe_check_product()
    want, mag = product64(q, s, scale, wq, ws, w_scale, [0, M], np.arange(M), fmt)
    check(out, want, mag, K, F32)


FIRST = """
import torch, block_quantized_expert_gb300 as bqe
z = lambda *n, d=torch.uint8: torch.zeros(*n, dtype=d, device="cuda")
f = lambda *n: torch.ones(*n, device="cuda")
M, K, N = {M}, 4096, 1000
x, y, h, dx, r, g = f(M, K), f(M, K), f(M, K), f(M, K), f(M), f(K)
q, s, sc, wq, ws, out = z(M, K // 2), z(M, K // 16), f(M), z(1, N, K // 2) + 0x22, z(1, N, K // 16) + 56, f(M, N)
scratch = z(bqe.moe_norm_scratch_bytes(M, K))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    bqe.moe_norm_rows(x, g, y, 0.0, x, h, r)
    bqe.moe_norm_rows_backward(y, h, g, r, dx, g.clone(), scratch)
    bqe.moe_quantize_blocks(y, q, s, sc)
    bqe.moe_dequantize_blocks(q, s, dx, sc)
    bqe.moe_block_product(q, s, wq, ws, out, scale=sc)
graph.replay()
bqe.moe_check_product()
d = dx[0, 0].item()  # the norm of rows of ones, as 4-bit blocks hold it
assert abs(d - 1) < 0.07 and torch.equal(out, torch.full_like(out, d * K)), (d, out)
print("captured")
"""


@pytest.mark.parametrize("M", [1, 40, 4000])
def test_first_calls_of_a_process_are_captured(M):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(M=M)], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
