"""moe_check_product takes the device's flag in one step: a wait that ran out is
reported to one of the checks around it, whatever stream they are on."""
import threading

import pytest
import torch

import block_quantized_expert_gb300 as bqe
from tests.test_gpu_int_product import codes, scales

pytestmark = pytest.mark.gpu


def timed_out(stream=None):
    try:
        bqe.moe_check_product(stream)
    except bqe.MoeError as e:
        assert e.status == bqe.MOE_ERR_TIMEOUT
        return True
    return False


def test_checks_on_another_stream_lose_nothing():
    M, N, K = 100, 256, 512
    q, wq, scale, w_scale = codes((M, K), 1), codes((1, N, K), 2), scales((M,), 3), scales((1, N), 4)
    out, want = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    bqe.moe_expert_product(q, scale, wq, w_scale, want)
    assert not timed_out()
    side = torch.cuda.Stream()
    for _ in range(15):
        bqe.moe_test_stall_next_product()
        bqe.moe_expert_product(q, scale, wq, w_scale, out, stream=side)
        seen = 0
        while not side.query():
            seen += timed_out()
        assert seen + timed_out(side) >= 1
    assert not timed_out() and not timed_out(side)
    bqe.moe_expert_product(q, scale, wq, w_scale, out)
    assert not timed_out() and torch.equal(out, want)


def test_checks_of_several_threads():
    """Each check returns its own answer: one call that ran out, four threads that
    check after it, one report."""
    M, N, K = 100, 256, 512
    q, wq, scale, w_scale = codes((M, K), 1), codes((1, N, K), 2), scales((M,), 3), scales((1, N), 4)
    out = torch.empty(M, N, device="cuda")
    for _ in range(5):
        bqe.moe_test_stall_next_product()
        bqe.moe_expert_product(q, scale, wq, w_scale, out)
        torch.cuda.synchronize()
        reports = []
        streams = [torch.cuda.Stream() for _ in range(4)]

        def run(s):
            reports.extend(timed_out(s) for _ in range(10))

        threads = [threading.Thread(target=run, args=(s,)) for s in streams]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert len(reports) == 40 and sum(reports) == 1
