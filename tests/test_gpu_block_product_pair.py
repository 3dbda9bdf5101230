"""moe_block_product in the form with pairs of CTAs (at sizes that its rule sends there), against the
definition in 64 bits: rows adjacent and looked up, every type of output, codes, scales, NaN, bad positions,
graphs, streams, chains of calls and the wait that runs out.  Tolerances as in test_gpu_block_product.py."""
import numpy as np
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from tests import _blocks as B
from tests.test_gpu_block_product import FMTS, blocks, check, product64, scales, values
from tests.test_gpu_sorted_rows import BF16, F16, F32, dev, f64, rows_of

pytestmark = pytest.mark.gpu


def pairs(E, R, K, N):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert bqe.moe_test_block_product_form(E, R, K, N, sms) == 2


# positions of each segment: their number and sum with K and N are of B.PAIRS
SEGMENTS = [(1056, 4096, [700, 0, 1301]), (512, 2048, [1500, 33, 2500, 63]), (288, 8192, [300, 100, 2000, 33, 1, 0, 257]),
            (128, 8192, [2399, 1]), (2048, 1000, [225, 224, 951]),
            (4096, 2048, [250, 1, 600, 0, 255, 256, 257, 90, 512, 513, 31, 700, 333, 64, 0, 600])]


def ends_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


@pytest.mark.parametrize("M,K,N", [(4000, 4096, 1000), (2500, 512, 2560), (4000, 256, 8192), (2100, 992, 4100)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("scaled", [False, True])
def test_dense(M, K, N, dtype, fmt, scaled):
    pairs(1, M, K, N)
    q, s = blocks((M,), K, fmt, 11, 16 * scaled)
    wq, ws = blocks((1, N), K, fmt, 12)
    scale, w_scale = (scales((M,), 13), scales((1, N), 14)) if scaled else (None, None)
    out = rows_of(M, N, dtype, 15, 3 * scaled)
    bqe.moe_block_product(q, s, wq, ws, out, scale=scale, w_scale=w_scale, fmt=fmt)
    want, mag = product64(q, s, scale, wq, ws, w_scale, [0, M], np.arange(M), fmt)
    check(out, want, mag, K, dtype)
    assert not scaled or torch.isnan(out._base[:, N:]).all()
    again = torch.empty(M, N, dtype=dtype, device="cuda")
    bqe.moe_block_product(q, s, wq, ws, again, scale=scale, w_scale=w_scale, fmt=fmt)
    bqe.moe_check_product()
    assert torch.equal(out, again)


@pytest.mark.parametrize("K,N,counts", SEGMENTS)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("gather", [False, True])
def test_segments(K, N, counts, dtype, fmt, gather):
    ends, E, R = ends_of(counts), len(counts), sum(counts)
    pairs(E, R, K, N)
    src = np.random.default_rng(N).permutation(R).astype(np.int32)
    T = (R + 2) // 3 if gather else R
    q, s = blocks((T,), K, fmt, 21)
    wq, ws = blocks((E, N), K, fmt, 22)
    scale, w_scale = (scales((T,), 23), scales((E, N), 24)) if fmt == B.NVFP4 else (None, None)
    out = torch.full((R, N), float("nan"), dtype=dtype, device="cuda")
    bqe.moe_block_product(q, s, wq, ws, out, dev(ends), dev(src) if gather else None, 3, scale, w_scale, fmt)
    bqe.moe_check_product()
    rows = src.astype(np.int64) // 3 if gather else np.arange(R)
    want, mag = product64(q, s, scale, wq, ws, w_scale, ends, rows, fmt)
    check(out, want, mag, K, dtype)


@pytest.mark.parametrize("K,N,counts", SEGMENTS)
@pytest.mark.parametrize("fmt", FMTS)
def test_adjacent_rows_are_those_of_row_src(K, N, counts, fmt):
    """A box of 16 rows takes the next segment's with it: equal bits to rows looked up one by one, and a bad
    row or a bad channel stays alone."""
    ends, E, R = ends_of(counts), len(counts), sum(counts)
    pairs(E, R, K, N)
    q, s = blocks((R,), K, fmt, 31)
    wq, ws = blocks((E, N), K, fmt, 32)
    nan = 255 if fmt == B.MXFP4 else 127
    bad_row, bad_e, bad_n = int(ends[1]), E - 1, N - 2  # the first row after a segment's end
    s[bad_row, 1], ws[bad_e, bad_n, 2] = nan, nan
    outs = [torch.zeros(R, N, device="cuda") for _ in range(2)]
    for out, src in zip(outs, (None, torch.arange(R, dtype=torch.int32, device="cuda"))):
        bqe.moe_block_product(q, s, wq, ws, out, dev(ends), src, 1, None, None, fmt)
    bqe.moe_check_product()
    assert torch.equal(outs[0].view(torch.int32), outs[1].view(torch.int32))
    want = torch.zeros(R, N, dtype=torch.bool, device="cuda")
    want[bad_row], want[ends[bad_e]:, bad_n] = True, True
    assert torch.equal(torch.isnan(outs[0]), want)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("gather", [False, True])
def test_every_code_and_scale(fmt, gather):
    """Each pair of codes alone in its row, at each block scale: exact."""
    M, K, N = 4000, 256, 8192
    pairs(1, M, K, N)
    n = B.size(fmt)
    q = torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda")
    r = torch.arange(M, device="cuda")
    at = (r * 7) % K
    code = (r * 5 + 3) % 16
    q[r, at // 2] = (code << (4 * (at % 2))).to(torch.uint8)
    low, high = (100, 150) if fmt == B.MXFP4 else (0, 127)
    s = (low + (torch.arange(M * K // n, device="cuda") * 11) % (high - low)).to(torch.uint8).view(M, -1)
    wq = ((torch.arange(N, device="cuda") % 16) * 17).to(torch.uint8)[None, :, None].expand(1, N, K // 2).contiguous()
    ws = (low + (torch.arange(N * K // n, device="cuda") * 3) % (high - low)).to(torch.uint8).view(1, N, -1)
    out = torch.empty(M, N, device="cuda")
    src = torch.arange(M, dtype=torch.int32, device="cuda") if gather else None
    bqe.moe_block_product(q, s, wq, ws, out, None, src, fmt=fmt)
    assert torch.equal(out.double(), values(q, s, fmt) @ values(wq[0], ws[0], fmt).T)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("gather", [False, True])
def test_nan_scales_show(fmt, gather):
    """Rows and channels with a NaN byte or scale give NaN, and no others do."""
    M, K, N = 4000, 4096, 1000
    pairs(1, M, K, N)
    q, s = blocks((M,), K, fmt, 1)
    wq, ws = blocks((1, N), K, fmt, 2)
    scale, w_scale = scales((M,), 3), scales((1, N), 4)
    nan = 255 if fmt == B.MXFP4 else 127
    want = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    for row, byte in ((M - 1, 1), (223, 100), (224, 5), (127, 0), (1111, 70)):
        s[row, byte] = nan
        want[row] = True
    for n, byte in ((5, 2), (128, 0), (255, 127), (999, 64)):
        ws[0, n, byte] = nan
        want[:, n] = True
    scale[0], w_scale[0, 9] = float("nan"), float("nan")
    want[0], want[:, 9] = True, True
    out = torch.empty(M, N, device="cuda")
    src = torch.arange(M, dtype=torch.int32, device="cuda") if gather else None
    bqe.moe_block_product(q, s, wq, ws, out, None, src, 1, scale, w_scale, fmt)
    assert torch.equal(torch.isnan(out), want)


@pytest.mark.parametrize("fmt", FMTS)
def test_bad_positions_and_offsets(fmt):
    """Rows outside q read as zeros, offsets out of range are held inside it; zeros past the last segment."""
    K, N, E, R, k = 512, 2048, 4, 4096, 2
    pairs(E, R, K, N)
    T = R // k
    q, s = blocks((T,), K, fmt, 1)
    wq, ws = blocks((E, N), K, fmt, 2)
    src = torch.arange(R, dtype=torch.int32, device="cuda")
    gone = torch.tensor([0, 1, 2, 500, 1023, 1024, 2000, 3000], device="cuda")
    src[gone] = torch.tensor([-1, R + 5, 2 ** 31 - 1, -7, -1, -1, 2 * T, -(2 ** 31)], dtype=torch.int32, device="cuda")
    ends = torch.tensor([0, R // 4, R // 2, R // 2, R - 777], dtype=torch.int32, device="cuda")
    rows = src.cpu().numpy().astype(np.int64)
    rows[gone.cpu().numpy()] = 0
    live = np.ones(R, bool)
    live[gone.cpu().numpy()] = False
    for given, held in ((ends, ends.tolist()), (torch.tensor([0, -5, R // 2, R // 2, 10 ** 9], dtype=torch.int32, device="cuda"),
                                               [0, 0, R // 2, R // 2, R])):
        out = torch.full((R, N), float("nan"), device="cuda")
        bqe.moe_block_product(q, s, wq, ws, out, given, src, k, fmt=fmt)
        bqe.moe_check_product()
        assert not out[gone].any() and not out[held[-1]:].any()
        want, mag = product64(q, s, None, wq, ws, None, held, rows // k, fmt)
        on = live & (np.arange(R) < held[-1])
        check(out[torch.from_numpy(on).cuda()], want[on], mag[on], K, F32)


def test_other_stream_graph_and_two_at_once():
    K, N, E, fmt = 512, 2048, 4, B.NVFP4
    counts = [1500, 33, 2500, 63]
    ends, R = dev(ends_of(counts)), sum(counts)
    pairs(E, R, K, N)
    wq, ws = blocks((E, N), K, fmt, 2)
    xs = [rows_of(R, K, BF16, i) for i in range(2)]
    bufs = [(torch.empty(R, K // 2, dtype=torch.uint8, device="cuda"), torch.empty(R, K // 16, dtype=torch.uint8, device="cuda"),
             torch.empty(R, device="cuda")) for _ in range(2)]
    outs = [torch.empty(R, N, dtype=BF16, device="cuda") for _ in range(4)]

    def step(i, out, stream=None):
        q, s, g = bufs[i]
        bqe.moe_quantize_blocks(xs[i], q, s, g, fmt, stream=stream)
        bqe.moe_block_product(q, s, wq, ws, out, ends, None, 1, g, None, fmt, stream=stream)

    step(0, outs[0])
    step(1, outs[1])
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i in (0, 1):
            step(i, outs[2 + i], sides[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[2], outs[0]) and torch.equal(outs[3], outs[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0, outs[2])
    xs[0].copy_(rows_of(R, K, BF16, 7))
    for _ in range(3):
        graph.replay()
    step(0, outs[0])
    assert torch.equal(outs[2], outs[0])
    bqe.moe_check_product()


@pytest.mark.parametrize("fmt", FMTS)
def test_chain_of_calls(fmt):
    """Blocks, product, gated blocks, product over the same buffers, captured back to back: the bits of the
    same calls made one at a time."""
    from block_quantized_expert_gb300 import sorted_experts as se
    from tests.test_gpu_chained_calls import N, compare, routed as routes_of
    from tests.test_gpu_sorted_experts import weights

    T, k, E, K, I = 700, 4, 4, 1024, 1024
    R, routes = T * k, routes_of(T, k, E, T)
    x = torch.randn(N, T, K, device="cuda").to(BF16)
    layer = se.BlockExperts(*weights(E, K, I), fmt)
    q, s, g = layer.blocks(x[0])
    gu = torch.empty(R, 2 * I, dtype=BF16, device="cuda")
    hq, hs, hg = layer.blocks(gu.zero_(), gated=True)
    (wq, ws, wg), (dq, ds, dg) = layer.gate_up, layer.down
    pairs(E, R, K, 2 * I)
    pairs(E, R, I, K)

    def step(i, out, done):
        _, _, _, off, src, _ = routes[i]
        bqe.moe_quantize_blocks(x[i], q, s, g, fmt)
        done()
        bqe.moe_block_product(q, s, wq, ws, gu, off, src, k, g, wg, fmt)
        done()
        bqe.moe_quantize_blocks(gu, hq, hs, hg, fmt, gated=True)
        done()
        bqe.moe_block_product(hq, hs, dq, ds, out[0], off, None, 1, hg, dg, fmt)
        done()

    compare(step, lambda: [torch.empty(N, R, K, dtype=BF16, device="cuda")])
    bqe.moe_check_product()


def test_sizes_past_32_bits():
    """Rows of q past 2^32 bytes and outputs past 2^31 elements, boxes and rows looked up."""
    M, K, N, fmt = 2500, 512, 2560, B.MXFP4
    pairs(1, M, K, N)
    base = torch.empty(M, 1 << 21, dtype=torch.uint8, device="cuda")  # 5.2e9 bytes
    q, s = base[:, :K // 2], torch.full((M, K // 32), 120, dtype=torch.uint8, device="cuda")
    q.copy_(blocks((M,), K, fmt, 1)[0])
    wq, ws = blocks((1, N), K, fmt, 2)
    wide = torch.empty(M, 1 << 20, dtype=BF16, device="cuda")  # 2.6e9 elements
    want, mag = product64(q.contiguous(), s, None, wq, ws, None, [0, M], np.arange(M), fmt)
    for src in (None, torch.arange(M, dtype=torch.int32, device="cuda")):
        out = wide[:, :N].fill_(float("nan"))
        bqe.moe_block_product(q, s, wq, ws, out, None, src, fmt=fmt)
        check(out, want, mag, K, BF16)


def test_a_wait_that_runs_out_is_reported():
    """No weight arrives: each CTA of a pair gives up by itself, the flag is set, the next call is right."""
    M, K, N = 4000, 4096, 1000
    pairs(1, M, K, N)
    q, s = blocks((M,), K, B.NVFP4, 1)
    wq, ws = blocks((1, N), K, B.NVFP4, 2)
    out, want = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    for src in (None, torch.arange(M, dtype=torch.int32, device="cuda")):
        bqe.moe_block_product(q, s, wq, ws, want, None, src)
        bqe.moe_check_product()
        bqe.moe_test_stall_next_product()
        bqe.moe_block_product(q, s, wq, ws, out, None, src)
        with pytest.raises(bqe.MoeError, match="moe_block_product") as e:
            bqe.moe_check_product()
        assert e.value.status == bqe.MOE_ERR_TIMEOUT
        out.fill_(7)
        bqe.moe_block_product(q, s, wq, ws, out, None, src)
        bqe.moe_check_product()
        assert torch.equal(out, want)
