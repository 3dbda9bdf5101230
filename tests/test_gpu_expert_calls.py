"""Int8Experts and BlockExperts refuse rows, codes, routings and weights of different batches: the products
read a row that is not there as zeros."""
import pytest
import torch

from block_quantized_expert_gb300 import sorted_experts as se
from tests import _blocks as B
from tests.test_gpu_sorted_experts import routed, weights
from tests.test_gpu_sorted_rows import BF16

pytestmark = pytest.mark.gpu
T, k, E, H, I = 8, 2, 4, 128, 64


def batch(tokens=T):
    logits, ids = routed(tokens, k, E, 0.0)
    return torch.randn(tokens, H, device="cuda").to(BF16), se.sort_tokens(ids, E), se.router_weights(logits, ids)


@pytest.mark.parametrize("make", [se.Int8Experts, lambda *w: se.BlockExperts(*w, B.MXFP4), lambda *w: se.BlockExperts(*w, B.NVFP4)])
def test_rows_of_another_batch(make):
    layer = make(*weights(E, H, I))
    x, s, w = batch()
    want = layer(x, s, w)
    for bad in (x[:T - 1], torch.cat([x, x[:1]]), x[:, :64], x[0]):
        with pytest.raises(ValueError, match="x must have shape"):
            layer(bad, s, w)
    _, more, wider = batch(T + 1)
    with pytest.raises(ValueError, match="w must have"):
        layer(x, s, wider)
    with pytest.raises(ValueError, match="w must have"):
        layer(x, more, w)
    with pytest.raises(ValueError, match="w must have"):  # as many slots, but of other tokens
        layer(x[:T // 2], s, w.view(T // 2, 2 * k))
    assert torch.equal(layer(x, s, w), want)


def test_codes_of_another_batch():
    layer = se.Int8Experts(*weights(E, H, I))
    x, s, w = batch()
    y, _, codes = se.norm_codes(x, torch.ones(H, device="cuda"))
    want = layer(y, s, w)
    assert torch.equal(layer(y, s, w, codes), want)
    for n in (T - 1, T // 2):
        with pytest.raises(ValueError, match="codes must have shape"):
            layer(y, s, w, (codes[0][:n], codes[1][:n]))
    with pytest.raises(ValueError, match="scale"):
        layer(y, s, w, (codes[0], codes[1][:T - 1]))


def test_no_tokens():
    x, s, w = torch.empty(0, H, device="cuda"), se.sort_tokens(torch.empty(0, k, dtype=torch.int32, device="cuda"), E), torch.empty(0, k, device="cuda")
    for layer in (se.Int8Experts(*weights(E, H, I)), se.BlockExperts(*weights(E, H, I))):
        assert layer(x, s, w).shape == (0, H)
