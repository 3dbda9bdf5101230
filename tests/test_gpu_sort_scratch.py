"""moe_permute_scratch and sort_tokens: the stable sort by expert in scratch of the
call's own."""
import numpy as np
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from block_quantized_expert_gb300 import sorted_experts as se

pytestmark = pytest.mark.gpu


def random_ids(T, k, E, seed, bad=0.1):
    g = torch.Generator("cuda").manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    return torch.where(torch.rand(T, k, generator=g, device="cuda") < bad, -1, ids)


def check(s, ids, E):
    flat = ids.cpu().numpy().reshape(-1).astype(np.int64)
    live = (flat >= 0) & (flat < E)
    order = np.nonzero(live)[0][np.argsort(flat[live], kind="stable")]
    dst = np.full(len(flat), -1)
    dst[order] = np.arange(len(order))
    off = np.concatenate([[0], np.cumsum(np.bincount(flat[live], minlength=E))])
    assert np.array_equal(s.offsets.cpu().numpy(), off)
    assert np.array_equal(s.row_src.cpu().numpy()[:len(order)], order)
    assert np.array_equal(s.row_dst.cpu().numpy(), dst)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 1024), (7, 3, 5), (1365, 6, 256), (1366, 6, 256), (2731, 3, 64),
                                   (8192, 8, 256), (10923, 6, 256), (32771, 7, 1024), (131072, 8, 130)])
def test_sort_of_any_size(T, k, E):
    ids = random_ids(T, k, E, T)
    check(se.sort_tokens(ids, E), ids, E)


def test_empty_batch_and_no_live_row():
    s = se.sort_tokens(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 6)
    assert s.offsets.tolist() == [0] * 7 and s.row_src.numel() == 0
    x = torch.empty(0, 8, device="cuda", requires_grad=True)
    w = se.router_weights(torch.empty(0, 6, device="cuda"), s.ids)
    se.combine(se.dispatch(x, s), w, s).sum().backward()
    assert x.grad.shape == (0, 8)
    for T in (3, 3000):
        ids = torch.full((T, 4), 9, dtype=torch.int32, device="cuda")
        check(se.sort_tokens(ids, 6), ids, 6)


def test_too_many_rows_are_refused():
    assert bqe.moe_permute_scratch_bytes(131073, 8, 16) == 0
    ids = torch.zeros((131073, 8), dtype=torch.int32, device="cuda")
    with pytest.raises(bqe.MoeError, match="2\\^20"):
        se.sort_tokens(ids, 16)


@pytest.mark.parametrize("T,k,E", [(900, 6, 64), (6000, 6, 256)])
def test_two_streams_at_once(T, k, E):
    """Sorts that overlap on two streams do not see each other."""
    n = 40
    ids = [[random_ids(T, k, E, 100 * a + i) for i in range(n)] for a in (0, 1)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for i in range(n):
        for a, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[a].append(se.sort_tokens(ids[a][i], E))
    torch.cuda.synchronize()
    for a in (0, 1):
        for i in range(n):
            check(got[a][i], ids[a][i], E)


def test_scratch_is_left_alone_past_its_end():
    T, k, E = 1500, 6, 33
    ids, n = random_ids(T, k, E, 5), bqe.moe_permute_scratch_bytes(1500, 6, 33)
    scratch = torch.full((n + 4096,), 171, dtype=torch.uint8, device="cuda")
    s = se.Sorted(ids, *(torch.empty(m, dtype=torch.int32, device="cuda") for m in (E + 1, T * k, T * k)))
    bqe.moe_permute_scratch(ids, E, s.offsets, s.row_src, s.row_dst, scratch)
    check(s, ids, E)
    assert torch.all(scratch[n:] == 171)
    with pytest.raises(bqe.MoeError, match="smaller"):
        bqe.moe_permute_scratch(ids, E, s.offsets, s.row_src, s.row_dst, scratch[:n - 4])
