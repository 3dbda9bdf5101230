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
