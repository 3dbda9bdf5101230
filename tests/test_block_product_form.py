"""Which form moe_block_product takes (host computation): the rule at sizes whose both sides were measured,
and at the sizes that the tests of the pair of CTAs rely on."""
import pytest

import block_quantized_expert_gb300 as bqe
from tests._blocks import PAIRS

FORM = bqe.moe_test_block_product_form


@pytest.mark.parametrize("E,R,K,N,form", [(1, 1, 4096, 4096, 0), (2, 2, 4096, 4096, 0), (1, 3, 4096, 4096, 1), (1, 256, 4096, 4096, 1),
                                          (1, 1024, 4096, 4096, 2), (1, 8192, 4096, 4096, 2), (32, 1024, 4096, 4096, 1),
                                          (32, 2048, 4096, 4096, 2), (1, 777, 1120, 1001, 1), (256, 49152, 4096, 4096, 2),
                                          (256, 6, 4096, 4096, 1), (256, 3000, 4096, 4096, 1)])
def test_form(E, R, K, N, form):
    assert FORM(E, R, K, N, 152) == form


@pytest.mark.parametrize("E,R,K,N", PAIRS)
def test_sizes_of_the_pairs_tests(E, R, K, N):
    assert all(FORM(E, R, K, N, sms) == 2 for sms in (148, 152, 160))


def test_sizes_below_one():
    for i, bad in enumerate([0, 0, 0, 0, 1]):
        sizes = [1, 1, 32, 1, 2]
        assert FORM(*sizes) == 0
        sizes[i] = bad
        assert FORM(*sizes) == -1
