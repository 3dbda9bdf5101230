"""moe_block_product against its definition in 64 bits.

A product of two codes times their block scales has at most 14 significant bits and is exact in
fp32; the fp32 sum rounds once in at most every 16 products, 2^-23 (2 + K / 16) of the sum of
their absolute values; two scales and a rounding follow (3 * 2^-24), then the output's own.
"""
import numpy as np
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from tests import _blocks as B
from tests import _sorted as S
from tests.test_gpu_sorted_rows import BF16, EPS, F16, F32, between, dev, f64, rows_of

pytestmark = pytest.mark.gpu
FMTS = [B.MXFP4, B.NVFP4]


def blocks(shape, K, fmt, seed, pad=0):
    """(codes, scale bytes, values in 64 bits on the GPU) of random rows of blocks [*shape][K]."""
    g = torch.Generator("cuda").manual_seed(seed)
    q = torch.randint(0, 256, (*shape, K // 2 + pad), generator=g, dtype=torch.uint8, device="cuda")[..., :K // 2]
    low, high = (123, 130) if fmt == B.MXFP4 else (40, 80)
    s = torch.randint(low, high, (*shape, K // B.size(fmt)), generator=g, dtype=torch.uint8, device="cuda")
    return q, s


def values(q, s, fmt):
    grid = torch.tensor(np.concatenate([B.GRID, -B.GRID]), device="cuda")
    c = torch.stack((q & 15, q >> 4), -1).flatten(-2).long()
    table = torch.from_numpy(B.scale_values(np.arange(256), fmt)).cuda()
    return grid[c] * table[s.long()].repeat_interleave(B.size(fmt), -1)


def product64(q, s, scale, wq, ws, w_scale, ends, rows, fmt):
    """(product, its scales times the sum of the products' absolute values)"""
    R, N = len(rows), wq.shape[1]
    out, mag = np.zeros((R, N)), np.zeros((R, N))
    v = values(q, s, fmt)
    for e in range(len(ends) - 1):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        at = torch.from_numpy(rows[a:b]).cuda()
        x, w = v[at], values(wq[e], ws[e], fmt)
        f = torch.ones(1, 1, dtype=torch.float64, device="cuda")
        if scale is not None:
            f = f * scale.double()[at][:, None]
        if w_scale is not None:
            f = f * w_scale[e].double()
        out[a:b], mag[a:b] = f64(x @ w.T * f), f64(x.abs() @ w.abs().T * f.abs())
    return out, mag


def check(out, want, mag, K, dtype):
    between(out, want, 3 * EPS * np.abs(want) + 2.0 ** -23 * (2 + K / 16) * mag, dtype)


def scales(shape, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.rand(shape, generator=g, device="cuda") * 0.01 + 1e-3


# tokens, k, experts, K, N, share of pruned slots
GROUPED = [(1, 6, 256, 512, 256, 0.0), (1, 1, 1, 32, 1, 0.0), (4, 2, 16, 256, 128, 0.0), (32, 6, 64, 1024, 384, 0.1),
           (7, 8, 8, 64, 130, 0.3), (100, 3, 5, 288, 1001, 0.2), (333, 2, 3, 544, 200, 0.0), (600, 4, 4, 128, 64, 0.5),
           (50, 1, 1024, 64, 32, 0.0), (1500, 6, 40, 416, 136, 0.0), (9, 2, 4, 96, 70, 0.0), (20, 2, 3, 32, 5, 0.0),
           (3, 5, 64, 4096, 4096, 0.0), (2, 6, 256, 2048, 1000, 0.2)]


@pytest.mark.parametrize("T,k,E,K,N,drop", GROUPED)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_product(T, k, E, K, N, drop, dtype, fmt, gather):
    _, _, _, offsets, row_src, _ = S.routing(T, k, E, T + K, drop)
    R = T * k
    q, s = blocks((T if gather else R,), K, fmt, 1)
    wq, ws = blocks((E, N), K, fmt, 2)
    scale, w_scale = scales((q.shape[0],), 3), scales((E, N), 4)
    out = rows_of(R, N, dtype, 5, 3)
    bqe.moe_block_product(q, s, wq, ws, out, dev(offsets), dev(row_src) if gather else None, k, scale, w_scale, fmt)
    rows = row_src.astype(np.int64) // k if gather else np.arange(R)
    want, mag = product64(q, s, scale, wq, ws, w_scale, offsets, rows, fmt)
    check(out, want, mag, K, dtype)
    assert not out[offsets[-1]:].any()
    assert torch.isnan(out._base[:, N:]).all()


@pytest.mark.parametrize("M,K,N", [(1, 4096, 4096), (2, 1120, 1001), (5, 64, 8), (8, 2048, 512), (16, 1024, 130), (17, 512, 257),
                                   (40, 4096, 256), (129, 416, 129), (255, 288, 64), (256, 128, 128), (257, 160, 300),
                                   (777, 1120, 1001), (1000, 96, 96), (2049, 64, 16), (64, 992, 100), (31, 32, 3), (300, 8224, 40)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("scaled", [False, True])
def test_dense_product(M, K, N, dtype, fmt, scaled):
    q, s = blocks((M,), K, fmt, 11, 16 * (K % 64 == 0))
    wq, ws = blocks((1, N), K, fmt, 12)
    scale, w_scale = (scales((M,), 13), scales((1, N), 14)) if scaled else (None, None)
    out = rows_of(M, N, dtype, 15, 1)
    if q.stride(0) % 16:
        q = q.contiguous()
    bqe.moe_block_product(q, s, wq, ws, out, scale=scale, w_scale=w_scale, fmt=fmt)
    want, mag = product64(q, s, scale, wq, ws, w_scale, [0, M], np.arange(M), fmt)
    check(out, want, mag, K, dtype)
    again = torch.empty(M, N, dtype=dtype, device="cuda")
    bqe.moe_block_product(q, s, wq, ws, again, scale=scale, w_scale=w_scale, fmt=fmt)
    assert torch.equal(out, again)


# experts, K, N, positions of each segment: long ones, whole and ragged, several rounds of tiles
@pytest.mark.parametrize("E,K,N,counts", [(1, 512, 2560, [2560]), (1, 4096, 1000, [4000]), (3, 1056, 4096, [700, 0, 1301]),
                                          (16, 4096, 2048, [250, 1, 600, 0, 255, 256, 257, 90, 512, 513, 31, 700, 333, 64, 0, 800]),
                                          (7, 288, 8192, [300, 100, 2000, 33, 1, 0, 257]), (2, 32, 16384, [1500, 900]),
                                          (64, 1024, 1030, [150 + 3 * i for i in range(64)])])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fmt", FMTS)
def test_long_segments(E, K, N, counts, dtype, fmt):
    ends = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R, T = int(ends[-1]), int(ends[-1]) // 3 + 1
    src = np.random.default_rng(N).permutation(R).astype(np.int32)
    q, s = blocks((T,), K, fmt, 21)
    wq, ws = blocks((E, N), K, fmt, 22)
    scale, w_scale = scales((T,), 23), scales((E, N), 24)
    want, mag = product64(q, s, scale, wq, ws, w_scale, ends, src.astype(np.int64) // 3, fmt)
    out = torch.empty(R, N, dtype=dtype, device="cuda")
    for _ in range(3):
        out.fill_(float("nan"))
        bqe.moe_block_product(q, s, wq, ws, out, dev(ends), dev(src), 3, scale, w_scale, fmt)
        check(out, want, mag, K, dtype)


@pytest.mark.parametrize("M", [1, 3, 40, 300])
@pytest.mark.parametrize("fmt", FMTS)
def test_every_code_and_scale(M, fmt):
    """Each pair of codes alone in its row, at each block scale: exact."""
    K, n = 256, B.size(fmt)
    q = torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda")
    r = torch.arange(M, device="cuda")
    at = (r * 7) % K
    code = (r * 5 + 3) % 16
    q[r, at // 2] = (code << (4 * (at % 2))).to(torch.uint8)
    low, high = (100, 150) if fmt == B.MXFP4 else (0, 127)
    s = (low + (torch.arange(M * K // n, device="cuda") * 11) % (high - low)).to(torch.uint8).view(M, -1)
    N = 160
    wq = ((torch.arange(N, device="cuda") % 16) * 17).to(torch.uint8)[None, :, None].expand(1, N, K // 2).contiguous()
    ws = (low + (torch.arange(N * K // n, device="cuda") * 3) % (high - low)).to(torch.uint8).view(1, N, -1)
    out = torch.empty(M, N, device="cuda")
    bqe.moe_block_product(q, s, wq, ws, out, fmt=fmt)
    assert torch.equal(out.double(), values(q, s, fmt) @ values(wq[0], ws[0], fmt).T)


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("fmt", FMTS)
def test_nan_scales_show(M, fmt):
    """A row or channel with a NaN byte or a NaN scale gives NaN, and no other does."""
    K, N = 256, 200
    q, s = blocks((M,), K, fmt, 1)
    wq, ws = blocks((1, N), K, fmt, 2)
    scale, w_scale = scales((M,), 3), scales((1, N), 4)
    nan = 255 if fmt == B.MXFP4 else 127
    s[M - 1, 1], ws[0, 5, 2], w_scale[0, 9] = nan, nan, float("nan")
    if M > 1:
        scale[0] = float("nan")
    out = torch.empty(M, N, device="cuda")
    bqe.moe_block_product(q, s, wq, ws, out, scale=scale, w_scale=w_scale, fmt=fmt)
    want = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    want[M - 1], want[:, 5], want[:, 9] = True, True, True
    if M > 1:
        want[0] = True
    assert torch.equal(torch.isnan(out), want)


@pytest.mark.parametrize("T", [3, 200])
def test_bad_positions_and_offsets(T):
    """Rows outside q read as zeros, offsets out of range are held inside it; zeros past the last segment."""
    k, E, K, N, fmt = 2, 4, 128, 72, B.NVFP4
    R = T * k
    q, s = blocks((T,), K, fmt, 1)
    wq, ws = blocks((E, N), K, fmt, 2)
    src = torch.arange(R, dtype=torch.int32, device="cuda")
    src[0], src[1], src[2] = -1, R + 5, 2 ** 31 - 1
    ends = torch.tensor([0, R // 4, R // 2, R // 2, R - 1], dtype=torch.int32, device="cuda")
    out = torch.full((R, N), float("nan"), device="cuda")
    bqe.moe_block_product(q, s, wq, ws, out, ends, src, k, fmt=fmt)
    assert not out[:3].any() and not out[R - 1:].any()
    rows = src.cpu().numpy().astype(np.int64)
    rows[:3] = 0
    want, mag = product64(q, s, None, wq, ws, None, ends.tolist(), rows // k, fmt)
    check(out[3:], want[3:], mag[3:], K, F32)
    far = torch.tensor([0, -5, R // 2, R // 2, 10 ** 9], dtype=torch.int32, device="cuda")
    out.fill_(float("nan"))
    bqe.moe_block_product(q, s, wq, ws, out, far, src.clamp(0, R - 1), k, fmt=fmt)
    assert torch.isfinite(out).all()


def test_no_segments():
    q, s = blocks((4,), 64, B.NVFP4, 1)
    wq, ws = blocks((3, 40), 64, B.NVFP4, 2)
    out = torch.full((8, 40), float("nan"), device="cuda")
    bqe.moe_block_product(q, s, wq, ws, out, torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda"), 2)
    assert not out.any()


@pytest.mark.parametrize("T,k,E", [(1, 6, 64), (300, 6, 16), (2000, 4, 4)])
def test_other_stream_and_graph(T, k, E):
    K, N, fmt = 512, 384, B.NVFP4
    _, _, _, offsets, row_src, _ = S.routing(T, k, E, T)
    offsets, row_src = dev(offsets), dev(row_src)
    x = rows_of(T, K, BF16, 1)
    wq, ws = blocks((E, N), K, fmt, 2)
    q, s, g = torch.empty(T, K // 2, dtype=torch.uint8, device="cuda"), torch.empty(T, K // 16, dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda")
    outs = [torch.empty(T * k, N, dtype=BF16, device="cuda") for _ in range(2)]

    def step(out, stream=None):
        bqe.moe_quantize_blocks(x, q, s, g, fmt, stream=stream)
        bqe.moe_block_product(q, s, wq, ws, out, offsets, row_src, k, g, None, fmt, stream=stream)

    step(outs[0])
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    step(outs[1], side)
    side.synchronize()
    assert torch.equal(*outs)
    with torch.cuda.graph(graph):
        step(outs[1])
    x.copy_(rows_of(T, K, BF16, 7))
    for _ in range(3):
        graph.replay()
    step(outs[0])
    assert torch.equal(*outs)


def test_offsets_past_32_bits():
    """Weights, codes and outputs past 2^31 and 2^32 elements."""
    E, K, N, fmt = 300, 8192, 2048, B.MXFP4  # 2.5e9 bytes of codes
    gen = torch.Generator("cuda").manual_seed(3)
    wq = torch.randint(0, 256, (E, N, K // 2), generator=gen, dtype=torch.uint8, device="cuda")
    ws = torch.full((E, N, K // 32), 120, dtype=torch.uint8, device="cuda")
    counts = np.zeros(E, np.int64)
    counts[[0, 150, 298, 299]] = [3, 40, 5, 60]
    ends = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(ends[-1])
    qs = 1 << 25
    base = torch.empty(R * qs, dtype=torch.uint8, device="cuda")
    q = base.view(R, qs)[:, :K // 2]
    q.copy_(torch.randint(0, 256, (R, K // 2), generator=gen, dtype=torch.uint8, device="cuda"))
    s = torch.full((R, K // 32), 120, dtype=torch.uint8, device="cuda")
    wide = torch.empty(R, 1 << 26, dtype=BF16, device="cuda")
    out = wide[:, :N]
    bqe.moe_block_product(q, s, wq, ws, out, dev(ends), fmt=fmt)
    for e in (0, 150, 298, 299):
        a, b = ends[e], ends[e + 1]
        w, x = values(wq[e], ws[e], fmt), values(q[a:b], s[a:b], fmt)
        check(out[a:b], f64(x @ w.T), f64(x.abs() @ w.abs().T), K, BF16)


@pytest.mark.parametrize("form", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("counts", [(5, 0, 37), (1, 16, 15, 33), (500, 3, 0, 700, 225), (2000, 17)])
def test_adjacent_rows_are_those_of_row_src(form, counts):
    """Without row_src a tile's rows come in boxes, which take the next segment's rows with them: equal bits
    to rows looked up one by one, and one bad row stays alone."""
    K, N, E, R = 352, 264, len(counts), sum(counts)
    n, fmt = (32, 0) if form == "mxfp4" else (16, 1)
    g = torch.Generator(device="cuda").manual_seed(R)
    rand = lambda *shape, top=256: torch.randint(0, top, shape, generator=g, device="cuda", dtype=torch.uint8)
    q, wq = rand(R, K // 2), rand(E, N, K // 2)
    s, ws = (rand(*shape, top=16) + (120 if form == "mxfp4" else 48) for shape in ((R, K // n), (E, N, K // n)))
    bad = R // 2
    s[bad, 1] = 255 if form == "mxfp4" else 127
    scale = torch.rand(R, generator=g, device="cuda") if fmt else None
    offsets = torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device="cuda")
    outs = [torch.zeros(R, N, device="cuda") for _ in range(2)]
    for out, src in zip(outs, (None, torch.arange(R, dtype=torch.int32, device="cuda"))):
        bqe.moe_block_product(q, s, wq, ws, out, offsets, src, 1, scale, None, fmt)
    bqe.moe_check_product()
    assert torch.equal(outs[0].view(torch.int32), outs[1].view(torch.int32))
    nan = torch.isnan(outs[0])
    assert nan[bad].all() and not nan[:bad].any() and not nan[bad + 1:].any()
