"""quantize_layer_weights on matrices of zeros and with infinities or NaN: a matrix that cannot be held shows."""
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from block_quantized_expert_gb300 import sorted_experts as se
from tests import _blocks as B
from tests.test_gpu_block_experts import weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", [B.MXFP4, B.NVFP4])
def test_matrices_that_are_not_finite(fmt, dtype):
    E, N, K = 5, 64, 128
    w = weights(E, K, N)[0].to(dtype)  # gate: [E][N][K]
    want = se.quantize_layer_weights(w, fmt)
    w[0, 3, 40], w[1, 0, 0], w[2] = float("nan"), float("-inf"), 0
    q, s, g = se.quantize_layer_weights(w, fmt)
    back = torch.empty(E * N, K, device="cuda")
    bqe.moe_dequantize_blocks(q.view(E * N, -1), s.view(E * N, -1), back, None if g is None else g.repeat_interleave(N), fmt)
    back = back.view(E, N, K)
    if fmt == B.NVFP4:
        assert torch.isnan(back[:2]).all() and g[2] == 1
    else:
        assert torch.isnan(back[0, 3, 32:64]).all() and torch.isnan(back[1, 0, :32]).all()
    assert not back[2].any()
    for a, b in zip((q, s, g), want):
        assert a is None or torch.equal(a[3:], b[3:])
