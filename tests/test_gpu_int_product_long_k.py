"""moe_expert_product at long K: the sums of codes at and past 2^24.

Tolerances.  On the CUDA cores (few rows; K, strides or bases off 16 bytes) the sum
is an exact integer up to 2^31, which is what K = 131072 codes of -128 on both sides
make: three roundings follow, 3 * 2^-24 of the result.  On the tensor cores a sum
past 2^24 rounds once in every 16 products: 2^-23 (2 + K / 16) of the sum of |q wq|.
"""
import numpy as np
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from tests.test_gpu_int_product import check, codes, product64, scales
from tests.test_gpu_sorted_rows import BF16, EPS, F32, f64

pytestmark = pytest.mark.gpu


def operands(M, N, K, kind):
    if kind == "least":  # every product 2^14, every sum 2^14 K
        return (torch.full((M, K), -128, dtype=torch.int8, device="cuda"),
                torch.full((1, N, K), -128, dtype=torch.int8, device="cuda"))
    if kind == "opposite":  # every product -128 * 127
        return (torch.full((M, K), -128, dtype=torch.int8, device="cuda"),
                torch.full((1, N, K), 127, dtype=torch.int8, device="cuda"))
    q, wq = codes((M, K), 1, full=kind == "full"), codes((1, N, K), 2, full=kind == "full")
    if kind == "one sign":  # as activations after a gate: all sums of one sign
        q, wq = q.abs(), wq.abs()
    return q, wq


KINDS = ["least", "opposite", "one sign", "full"]


def exact_sums(q, wq, M, N, K, dtype):
    scale, w_scale = scales((M,), 3), scales((1, N), 4)
    out = torch.empty(M, N, dtype=dtype, device="cuda")
    bqe.moe_expert_product(q, scale, wq, w_scale, out)
    want, _, _ = product64(q, scale, wq, w_scale, [0, M], np.arange(M))
    if dtype == F32:
        assert np.all(np.abs(f64(out) - want) <= 3 * EPS * np.abs(want))
    else:
        check(out, want, np.abs(want), 0, K, dtype)


@pytest.mark.parametrize("M", [1, 3, 8])
@pytest.mark.parametrize("K", [16384, 131056, 131072])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_few_rows(M, K, kind, dtype):
    q, wq = operands(M, 40, K, kind)
    exact_sums(q, wq, M, 40, K, dtype)


@pytest.mark.parametrize("M,K", [(2, 131072), (70, 131072), (70, 131071), (5, 16383)])
@pytest.mark.parametrize("kind", KINDS)
def test_any_alignment(M, K, kind):
    N = 70
    q, wq = operands(M, N, K, kind)
    odd = torch.empty(M * K + 1, dtype=torch.int8, device="cuda")[1:].view(M, K)
    odd.copy_(q)
    exact_sums(odd, wq, M, N, K, F32)


# the last is taken by pairs of CTAs
@pytest.mark.parametrize("M,N", [(20, 64), (300, 200), (2304, 2048)])
@pytest.mark.parametrize("K", [2048, 16384, 131072])
@pytest.mark.parametrize("kind", KINDS)
def test_tensor_cores(M, N, K, kind):
    q, wq = operands(M, N, K, kind)
    scale, w_scale = scales((M,), 3), scales((1, N), 4)
    out = torch.empty(M, N, device="cuda")
    bqe.moe_expert_product(q, scale, wq, w_scale, out)
    bqe.moe_check_product()
    want, mag, top = product64(q, scale, wq, w_scale, [0, M], np.arange(M))
    check(out, want, mag, top, K, F32)
