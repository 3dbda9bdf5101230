"""Host-side checks of moe_permute_scratch (nothing is enqueued, no GPU is needed)."""
import pytest

import block_quantized_expert_gb300 as bqe

P = 4096
GOOD = [P, 4, 2, 8, P, P, P, P, 1 << 20, None]


@pytest.mark.parametrize("arg,value,word", [(0, None, "NULL"), (1, -1, "T"), (1, (1 << 19) + 1, "T"), (2, 0, "top_k"),
                                            (2, 9, "top_k"), (3, 0, "n_experts"), (3, 1025, "n_experts"), (4, None, "NULL"),
                                            (5, None, "NULL"), (6, None, "NULL"), (7, None, "NULL"), (7, P + 2, "aligned"),
                                            (8, 100, "smaller")])
def test_refusals(arg, value, word):
    args = list(GOOD)
    args[arg] = value
    assert bqe.load_library().moe_permute_scratch(*args) == bqe.MOE_ERR_INVALID_ARG
    msg = bqe.moe_last_error()
    assert "moe_permute_scratch" in msg and word in msg, msg


def test_scratch_bytes():
    f = bqe.moe_permute_scratch_bytes
    for T, k, E in ((0, 1, 1), (1, 1, 1), (1365, 6, 256), (1366, 6, 256), (131072, 8, 1024)):
        R = T * k
        chunks = (R + 1023) // 1024 if R > 8192 else 0
        # counts, three scans, rows' places, the padded rows (each segment up to 127 more), the chunks' counts
        assert f(T, k, E) == 4 * (E + 3 * (E + 1) + R + R + 127 * E + chunks * E)
    assert f(-1, 1, 1) == f(1, 0, 1) == f(1, 9, 16) == f(1, 1, 0) == f(1, 1, 1025) == f(131073, 8, 8) == 0
