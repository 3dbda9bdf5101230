"""Int8Experts with its rows between the products in fp32.

Tolerance against the definition in 64 bits on the same codes of x: fp32 sums and
scales give each value of h within 16 * 2^-24 of itself and of its row's maximum, so
that a code, up to 127, moves by one step where it is within 2^-12 of half way: a
share of 2^-11 of the codes.  With a root mean square of 127 / 4 codes a row at most
a step on such a share is 2^-5.5 / 32 < 1e-3 of h's norm, and so of the output's,
whose own fp32 sums are far below.
"""
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from block_quantized_expert_gb300 import sorted_experts as se
from tests.test_gpu_sorted_experts import routed, weights

pytestmark = pytest.mark.gpu


def definition(layer, x, ids, w):
    """The layer on the codes of x, in 64 bits."""
    T, H, I = x.shape[0], layer.H, layer.I
    q, scale = torch.empty(T, H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    bqe.moe_quantize_rows(x, q, scale)
    x64 = q.double() * scale.double()[:, None]
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(layer.E):
        t, j = (ids == e).nonzero(as_tuple=True)
        gu = x64[t] @ (layer.gate_up[e].double() * layer.gate_up_scale[e].double()[:, None]).T
        h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        m = h.abs().amax(1, keepdim=True)
        y = (torch.round(127 * h / m) * m / 127) @ (layer.down[e].double() * layer.down_scale[e].double()[:, None]).T
        want.index_add_(0, t, y * w[t, j].double()[:, None])
    return want


@pytest.mark.parametrize("T,k,E,H,I", [(1, 6, 64, 1024, 512), (300, 4, 24, 512, 272)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_in_fp32(T, k, E, H, I, dtype):
    gate, up, down = weights(E, H, I)
    logits, ids = routed(T, k, E, 0.1)
    s, w = se.sort_tokens(ids, E), se.router_weights(logits, ids)
    x = torch.randn(T, H, generator=torch.Generator("cuda").manual_seed(3), device="cuda").to(dtype)
    fine, coarse = se.Int8Experts(gate, up, down, rows=torch.float32), se.Int8Experts(gate, up, down)
    want = definition(fine, x, ids, w)
    got = fine(x, s, w)
    bqe.moe_check_product()
    err = float((got.double() - want).norm() / want.norm())
    assert err <= 1e-3, err
    assert float((coarse(x, s, w).double() - want).norm() / want.norm()) > err


def test_rows_must_be_a_floating_type():
    gate, up, down = weights(2, 32, 16)
    with pytest.raises(ValueError, match="rows"):
        se.Int8Experts(gate, up, down, rows=torch.int8)
