"""One check reports the waits of both products that ran out, by name, and takes them both."""
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from tests.test_gpu_int_product import codes, scales

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", [("expert",), ("block",), ("expert", "block"), ("block", "expert")])
def test_names(which):
    M, N, K = 100, 256, 512
    u8 = lambda *n: torch.zeros(*n, dtype=torch.uint8, device="cuda")  # noqa: E731
    calls = {"expert": (bqe.moe_expert_product, (codes((M, K), 1), scales((M,), 3), codes((1, N, K), 2), scales((1, N), 4))),
             "block": (bqe.moe_block_product, (u8(M, K // 2), u8(M, K // 16), u8(1, N, K // 2), u8(1, N, K // 16)))}
    out = torch.empty(M, N, device="cuda")
    bqe.moe_check_product()
    for name in which:
        bqe.moe_test_stall_next_product()
        calls[name][0](*calls[name][1], out)
    with pytest.raises(bqe.MoeError) as e:
        bqe.moe_check_product()
    assert e.value.status == bqe.MOE_ERR_TIMEOUT
    for name in calls:
        assert (f"moe_{name}_product" in str(e.value)) == (name in which), str(e.value)
    bqe.moe_check_product()
    for f, args in calls.values():
        f(*args, out)
    bqe.moe_check_product()
