"""sorted_experts.router_weights: its forward is plain PyTorch and runs on the CPU;
its gradient is moe_route_backward's."""
import numpy as np
import pytest
import torch

from block_quantized_expert_gb300 import sorted_experts as se
from tests import _sorted as S

EPS = 2.0 ** -24


@pytest.mark.parametrize("device", ["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def test_slots_that_are_not_kept_are_not_read(device):
    """Ids outside [0, E) are empty slots, and no logit of an empty slot matters."""
    nan, inf = float("nan"), float("inf")
    logits = torch.tensor([[nan, 1.0, 2.0, 0.5], [inf, 1.0, 2.0, 0.5], [3.0, 1.0, 2.0, 0.5], [0.0, 0.0, 0.0, 0.0]], device=device)
    ids = torch.tensor([[1, 2, -1], [2, 4, 1], [3, 2 ** 31 - 1, -2 ** 31], [-1, 4, -7]], dtype=torch.int32, device=device)
    w = se.router_weights(logits, ids).cpu().numpy()
    kept = np.array([[1, 1, 0], [1, 0, 1], [1, 0, 0], [0, 0, 0]], bool)
    assert np.array_equal(w != 0, kept)
    l = np.nan_to_num(logits.cpu().numpy().astype(np.float64), nan=0.0, posinf=0.0)
    want = S.route_weights64(l, np.where(kept, ids.cpu().numpy(), -1))
    # two transcendentals of 2 units, a root, k sums, a product and a quotient
    assert np.all(np.abs(w - want) <= 16 * EPS * want)


@pytest.mark.parametrize("device", ["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
@pytest.mark.parametrize("base", [3e38, 1000.0, 300.0, 89.0, 88.0, 20.0, 0.0, -17.0, -60.0, -88.0, -95.0, -103.0, -110.0, -170.0])
def test_weights_over_the_range_of_logits(base, device):
    """The same bound wherever s = sqrt(softplus(logit)) is a normal number: a
    logit's half is exact, so exp(l / 2) has no more than its own two units."""
    T, k, E = 6, 4, 5
    logits = (np.float32(base) + np.random.default_rng(1).uniform(-2, 2, (T, E))).astype(np.float32)
    ids = np.tile(np.arange(k, dtype=np.int32), (T, 1))
    w = se.router_weights(torch.from_numpy(logits).to(device), torch.from_numpy(ids).to(device)).cpu().numpy()
    want = S.route_weights64(logits.astype(np.float64), ids)
    assert np.all(np.abs(w - want) <= 16 * EPS * want), (w, want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16, torch.float64])
@pytest.mark.parametrize("id_dtype", [torch.int32, torch.int64])
def test_the_gradient_takes_what_the_forward_takes(dtype, id_dtype):
    """Ids as topk returns them, logits of other types and orders: the gradient is
    that of contiguous fp32 logits, in the type of the logits."""
    T, k, E = 7, 3, 9
    base = torch.randn(E, T, generator=torch.Generator("cuda").manual_seed(2), device="cuda").to(dtype)
    logits = base.t().requires_grad_()
    ids = logits.detach().topk(k, dim=1).indices.to(id_dtype)
    up = torch.randn(k, T, device="cuda").t()
    w = se.router_weights(logits, ids)
    assert w.dtype == torch.float32
    (got,) = torch.autograd.grad(w, logits, up)
    plain = base.t().float().contiguous().requires_grad_()
    (want,) = torch.autograd.grad(se.router_weights(plain, ids.int().contiguous()), plain, up.contiguous())
    assert got.dtype == dtype and torch.equal(got, want.to(dtype))


def test_ids_must_be_whole_numbers():
    with pytest.raises(ValueError, match="ids"):
        se.router_weights(torch.zeros(2, 4), torch.zeros(2, 2))
    with pytest.raises(ValueError, match="logits"):
        se.router_weights(torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="ids"):
        se.router_weights(torch.zeros(2, 4), torch.zeros(3, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="top_k"):
        se.router_weights(torch.zeros(2, 16), torch.zeros(2, 9, dtype=torch.int32))


def test_64_bit_ids_do_not_wrap():
    """2^32 + 1 is no expert."""
    w = se.router_weights(torch.zeros(1, 4), torch.tensor([[2, 2 ** 32 + 1, -2 ** 32]]))
    assert w.tolist() == [[1.5, 0.0, 0.0]]
