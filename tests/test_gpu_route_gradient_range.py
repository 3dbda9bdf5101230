"""moe_route_backward where every kept logit is very negative: s = sqrt(softplus(l))
is small, but the weights are ordinary numbers, and so are their gradients.

Tolerance: that of test_gpu_sorted_rows.test_route_backward, (2 k + 40) 2^-24 of the
terms' absolute values.  A logit's half is exact, its exponential within 2 units and,
down to l = -174, a normal number; exp(l / 2) differs from s by exp(l) / 4 of it,
below 2^-26 for l < -17.
"""
import numpy as np
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from tests import _sorted as S
from tests.test_gpu_sorted_rows import EPS, dev, f64

pytestmark = pytest.mark.gpu


def gradient(logits, ids, dw):
    got = torch.full(logits.shape, float("nan"), device="cuda")
    bqe.moe_route_backward(dev(logits), dev(ids), dev(dw), got, S.W_SCALE)
    return f64(got)


def check(logits, ids, dw):
    got = gradient(logits, ids, dw)
    want, mag = S.route_grad64(logits, ids, dw.astype(np.float64))
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want) <= (2 * ids.shape[1] + 40) * EPS * mag), (got, want)


def kept_first(T, k):
    return np.tile(np.arange(k, dtype=np.int32), (T, 1))


@pytest.mark.parametrize("k", [1, 2, 3, 6, 8])
@pytest.mark.parametrize("base", [-16.5, -17.5, -60.0, -87.0, -89.0, -92.0, -95.0, -100.0, -103.0, -110.0, -172.0])
def test_all_kept_logits_far_below_zero(base, k):
    T, E = 9, 12
    g = np.random.default_rng(k)
    logits = g.standard_normal((T, E)).astype(np.float32)
    logits[:, :k] = np.float32(base) + g.uniform(-1.5, 1.5, (T, k)).astype(np.float32)
    dw = g.standard_normal((T, k)).astype(np.float32)
    check(logits, kept_first(T, k), dw)
    if k == 1:
        assert not gradient(logits, kept_first(T, 1), dw).any()


@pytest.mark.parametrize("l", [-89.0, -92.0, -95.0, -100.0, -103.9, -104.5, -150.0, -174.0, -190.0, -300.0, 0.0, 88.0, 300.0])
def test_one_kept_slot_gives_exactly_zero(l):
    """One slot, and one left over by pruning."""
    logits = np.full((1, 8), l, np.float32)
    assert not gradient(logits, np.array([[3]], np.int32), np.array([[2.5]], np.float32)).any()
    ids = np.array([[-1, -1, 5, -1, -1, -1, -1, -1]], np.int32)
    assert not gradient(logits, ids, np.full((1, 8), 2.5, np.float32)).any()


def test_very_negative_beside_ordinary_and_large():
    logits = np.array([[-100.0, 2.0, -30.0, 0.5], [90.0, -95.0, -17.0, 3.0], [-120.0, -90.0, -92.0, -160.0],
                       [300.0, 100.0, -100.0, -17.25]], np.float32)
    dw = np.array([[1.0, -2.0, 0.5, 3.0]] * 4, np.float32)
    check(logits, kept_first(4, 4), dw)


def test_stated_band():
    """Logits (-92, -93, -91.5): the gradient is (0.22, -0.34, 0.12)."""
    logits, dw = np.array([[-92.0, -93.0, -91.5, 0.0]], np.float32), np.array([[1.0, -2.0, 0.5]], np.float32)
    assert np.allclose(gradient(logits, kept_first(1, 3), dw), [[0.221, -0.338, 0.117, 0.0]], atol=1e-3)


def test_below_the_normal_range_counts_as_zero():
    """exp(l / 2) below fp32's normal numbers: such an expert has no weight and no gradient."""
    logits = np.array([[-180.0, -181.0, -200.0], [-180.0, 1.0, 2.0]], np.float32)
    dw = np.array([[1.0, -2.0, 0.5]] * 2, np.float32)
    got = gradient(logits, kept_first(2, 3), dw)
    assert not got[0].any() and got[1, 0] == 0
    alone, mag = S.route_grad64(logits[1:, 1:], kept_first(1, 2), dw[1:, 1:].astype(np.float64))
    assert np.all(np.abs(got[1:, 1:] - alone) <= 46 * EPS * mag)


def test_nan_stays_visible():
    """A kept NaN makes its own token's gradients NaN, one that is not kept nothing."""
    logits = np.array([[np.nan, 1.0, 2.0], [1.0, 2.0, np.nan], [1.0, 2.0, 0.5]], np.float32)
    got = gradient(logits, kept_first(3, 2), np.ones((3, 2), np.float32))
    assert np.isnan(got[0, :2]).all() and got[0, 2] == 0 and not got[1:].any()
