"""moe_quantize_rows and moe_expert_product against their definitions in 64 bits.

Tolerances.  scale: the one correctly rounded division.  A code q is the nearest
integer to 127 v / max|v|: |q - 127 v / max| <= 1/2 plus the roundings of the
product and the division (127 * 2 * 2^-24) and, for a gated row, those of v
(exp to 2 units, four more roundings: 8 * 2^-24 relative, of v and of the maximum).
The product's integer sum is exact while the sum of |q wq| is at most 2^24;
three fp32 roundings follow (its conversion, two scales), then the output's own
(the output lies between the rounded ends of that interval).
Above that the fp32 sum rounds once in at most every 16 products: 2^-23 (2 + K / 16)
of the sum of |q wq|.
"""
import numpy as np
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from tests import _sorted as S
from tests.test_gpu_sorted_rows import BF16, EPS, F16, F32, between, dev, f64, rows_of

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------- quantise --
@pytest.mark.parametrize("rows,K,pad", [(1, 1, 0), (1, 4096, 0), (5, 7, 1), (64, 2048, 0), (33, 1104, 8), (300, 1000, 3),
                                        (3, 20000, 0), (9, 131072, 0), (17, 16, 0)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("gated", [False, True])
def test_quantize_rows(rows, K, pad, dtype, gated):
    x = rows_of(rows, 2 * K if gated else K, dtype, 100 * rows + K, pad)
    x[rows // 2] = 0
    q = torch.full((rows, K + 5), 77, dtype=torch.int8, device="cuda")[:, :K]
    scale = torch.full((rows,), -1.0, device="cuda")
    bqe.moe_quantize_rows(x, q, scale, gated=gated)
    x64 = f64(x)
    v = x64[:, :K] / (1 + np.exp(-x64[:, :K])) * x64[:, K:] if gated else x64
    most = np.abs(v).max(1)
    slack = (127 * 2 + (127 * 16 if gated else 0)) * EPS
    assert np.all(np.abs(f64(scale) - most / 127) <= (9 if gated else 1) * EPS * most / 127)
    want = 127 * v / np.where(most > 0, most, 1)[:, None]
    assert np.all(np.abs(f64(q) - want) <= 0.5 + slack)
    assert not q[rows // 2].any() and scale[rows // 2] == 0
    assert torch.all(q._base[:, K:] == 77)


def test_quantize_halves_go_to_even():
    """Half of the maximum is 63.5 codes: 64; and the last codes are +-127."""
    x = torch.tensor([[2.0, 1.0, -1.0, -2.0, 0.0, 3e-8, 2.0, 1.0]] * 3, device="cuda") * torch.tensor([[1.0], [3.7], [1e-30]], device="cuda")
    q, scale = torch.empty(3, 8, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    bqe.moe_quantize_rows(x, q, scale)
    assert q.tolist() == [[127, 64, -64, -127, 0, 0, 127, 64]] * 3


@pytest.mark.parametrize("K", [8, 9, 4096])
def test_quantize_extremes(K):
    """Infinities and NaN: scale NaN and codes 0; the largest and the smallest finite values."""
    x = torch.ones(6, K, device="cuda")
    x[0, K - 1], x[1, 0], x[2, 3] = float("inf"), float("nan"), float("-inf")
    x[3] = 3.4e38
    x[4] = 1e-44
    x[5, 1:] = 0
    q, scale = torch.empty(6, K, dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
    bqe.moe_quantize_rows(x, q, scale)
    assert torch.isnan(scale[:3]).all() and not q[:3].any()
    assert torch.all(q[3:5] == 127) and q[5, 0] == 127 and not q[5, 1:].any()
    assert torch.isfinite(scale[3:]).all()


# ------------------------------------------------------------------ product --
def product64(q, scale, wq, w_scale, ends, rows):
    """(product, its scales times the sum of |q wq|, the largest sum of |q wq|)"""
    R, N = len(rows), wq.shape[1]
    out, mag = np.zeros((R, N)), np.zeros((R, N))
    top = 0.0
    q64 = q.double()
    for e in range(len(ends) - 1):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        x = q64[torch.from_numpy(rows[a:b]).cuda()]
        w = wq[e].double()
        s = scale.double()[torch.from_numpy(rows[a:b]).cuda()][:, None] * w_scale[e].double()
        sums = x.abs() @ w.abs().T
        top = max(top, float(sums.max()))
        out[a:b], mag[a:b] = f64(x @ w.T * s), f64(sums * s.abs())
    return out, mag, top


def check(out, want, mag, top, K, dtype):
    bound = 3 * EPS * np.abs(want) + (0 if top <= 2 ** 24 else 2.0 ** -23 * (2 + K / 16) * mag)
    between(out, want, bound, dtype)


def codes(shape, seed, full=False):
    g = torch.Generator("cuda").manual_seed(seed)
    if full:
        return torch.randint(-128, 128, shape, generator=g, dtype=torch.int8, device="cuda")
    return (torch.randn(shape, generator=g, device="cuda") * 32).round().clamp(-127, 127).to(torch.int8)


def scales(shape, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.rand(shape, generator=g, device="cuda") * 0.01 + 1e-3


# tokens, k, experts, K, N, share of pruned slots
GROUPED = [(1, 6, 256, 512, 256, 0.0), (1, 1, 1, 16, 1, 0.0), (4, 2, 16, 256, 128, 0.0), (32, 6, 64, 1024, 384, 0.1),
           (7, 8, 8, 48, 130, 0.3), (100, 3, 5, 272, 1001, 0.2), (333, 2, 3, 528, 200, 0.0), (600, 4, 4, 128, 64, 0.5),
           (50, 1, 1024, 64, 32, 0.0), (1500, 6, 40, 400, 136, 0.0), (9, 2, 4, 33, 70, 0.0), (20, 2, 3, 1, 5, 0.0)]


@pytest.mark.parametrize("T,k,E,K,N,drop", GROUPED)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_product(T, k, E, K, N, drop, dtype, gather):
    _, _, _, offsets, row_src, _ = S.routing(T, k, E, T + K, drop)
    R = T * k
    q, wq = codes((T if gather else R, K), 1, full=True), codes((E, N, K), 2, full=True)
    scale, w_scale = scales((q.shape[0],), 3), scales((E, N), 4)
    out = rows_of(R, N, dtype, 5, 3)
    bqe.moe_expert_product(q, scale, wq, w_scale, out, dev(offsets), dev(row_src) if gather else None, k)
    rows = row_src.astype(np.int64) // k if gather else np.arange(R)
    want, mag, top = product64(q, scale, wq, w_scale, offsets, rows)
    check(out, want, mag, top, K, dtype)
    assert not out[offsets[-1]:].any()


@pytest.mark.parametrize("M,K,N", [(1, 4096, 4096), (2, 1104, 1001), (5, 64, 8), (8, 2048, 512), (16, 1024, 130), (17, 512, 257),
                                   (40, 4096, 256), (129, 400, 129), (255, 272, 64), (256, 128, 128), (257, 160, 300),
                                   (777, 1104, 1001), (1000, 96, 96), (2049, 64, 16), (64, 1000, 100), (31, 7, 3)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_dense_product(M, K, N, dtype):
    q, wq = codes((M, K + 16), 11)[:, :K], codes((1, N, K), 12)
    scale, w_scale = scales((M,), 13), scales((1, N), 14)
    out = rows_of(M, N, dtype, 15, 1)
    bqe.moe_expert_product(q, scale, wq, w_scale, out)
    want, mag, top = product64(q, scale, wq, w_scale, [0, M], np.arange(M))
    check(out, want, mag, top, K, dtype)
    again = torch.empty(M, N, dtype=dtype, device="cuda")
    bqe.moe_expert_product(q, scale, wq, w_scale, again)
    assert torch.equal(out, again)


# experts, K, N, positions of each segment: wide tiles (a pair of CTAs), whole and ragged, several rounds of them
@pytest.mark.parametrize("E,K,N,counts", [(1, 512, 2560, [2560]), (1, 4096, 1000, [4000]), (3, 1040, 4096, [700, 0, 1301]),
                                          (16, 4096, 2048, [250, 1, 600, 0, 255, 256, 257, 90, 512, 513, 31, 700, 333, 64, 0, 800]),
                                          (7, 272, 8192, [300, 100, 2000, 33, 1, 0, 257]), (2, 16, 16384, [1500, 900]),
                                          (64, 1024, 1030, [150 + 3 * i for i in range(64)])])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_segments(E, K, N, counts, dtype):
    ends = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R, T = int(ends[-1]), int(ends[-1]) // 3 + 1
    src = np.random.default_rng(N).permutation(R).astype(np.int32)
    q, wq = codes((T, K), 21, full=True), codes((E, N, K), 22, full=True)
    scale, w_scale = scales((T,), 23), scales((E, N), 24)
    out = torch.full((R, N), float("nan"), dtype=dtype, device="cuda")
    for _ in range(3):
        bqe.moe_expert_product(q, scale, wq, w_scale, out, dev(ends), dev(src), 3)
        want, mag, top = product64(q, scale, wq, w_scale, ends, src.astype(np.int64) // 3)
        check(out, want, mag, top, K, dtype)


@pytest.mark.parametrize("M", [1, 3, 40, 300, 3000])
def test_largest_sums(M):
    """Every product 127^2 or -128 * 127: the sums pass 2^24 and stay within fp32's rounding."""
    K, N = 4096, 64 if M < 1000 else 2048
    q = torch.full((M, K), 127, dtype=torch.int8, device="cuda")
    wq = torch.full((1, N, K), 127, dtype=torch.int8, device="cuda")
    wq[:, N // 2:] = -128
    wq[:, 1, ::2] = -127
    scale, w_scale = scales((M,), 1), scales((1, N), 2)
    out = torch.empty(M, N, device="cuda")
    bqe.moe_expert_product(q, scale, wq, w_scale, out)
    want, mag, top = product64(q, scale, wq, w_scale, [0, M], np.arange(M))
    assert top > 2 ** 24 and not out[:, 1].any()
    check(out, want, mag, top, K, F32)


def test_one_expert_takes_everything_and_strides():
    """All rows in the middle expert of five; q and out are columns of wider tensors."""
    M, K, N, E = 150, 192, 72, 5
    offsets = np.array([0, 0, 0, M, M, M], np.int32)
    q, wq = codes((M, 3 * K), 1)[:, K:2 * K], codes((E, N, K), 2)
    scale, w_scale = scales((M,), 3), scales((E, N), 4)
    wide = torch.full((M, 2 * N + 1), 9.0, device="cuda")
    bqe.moe_expert_product(q, scale, wq, w_scale, wide[:, N:2 * N], dev(offsets))
    want, mag, top = product64(q, scale, wq, w_scale, offsets, np.arange(M))
    check(wide[:, N:2 * N], want, mag, top, K, F32)
    assert torch.all(wide[:, :N] == 9) and torch.all(wide[:, 2 * N:] == 9)


@pytest.mark.parametrize("K", [64, 65])
def test_unaligned_codes(K):
    """Codes and weights that start off every 16-byte boundary."""
    M, N = 70, 40
    q = codes((M * K + 3,), 1)[3:].view(M, K)
    wq = codes((N * K + 5,), 2)[5:].view(1, N, K)
    scale, w_scale = scales((M,), 3), scales((1, N), 4)
    out = torch.empty(M, N, device="cuda")
    bqe.moe_expert_product(q, scale, wq, w_scale, out)
    want, mag, top = product64(q, scale, wq, w_scale, [0, M], np.arange(M))
    check(out, want, mag, top, K, F32)


def test_odd_offsets_and_sources_are_held_in_bounds():
    """Offsets past the rows and sources past the tokens read as empty."""
    T, K, N = 6, 64, 48
    q, wq, scale, w_scale = codes((T, K), 1), codes((3, N, K), 2), scales((T,), 3), scales((3, N), 4)
    out = torch.full((T, N), 7.0, device="cuda")
    src = torch.tensor([0, 6, 2, -1, 2 ** 31 - 1, 5], dtype=torch.int32, device="cuda")
    bqe.moe_expert_product(q, scale, wq, w_scale, out, torch.tensor([-4, 3, 3, 99], dtype=torch.int32, device="cuda"), src)
    rows = np.array([0, 0, 2, 0, 0, 5])
    want, mag, top = product64(q, scale, wq, w_scale, [0, 3, 3, 6], rows)
    want[[1, 3, 4]] = 0
    check(out, want, mag, top, K, F32)


@pytest.mark.parametrize("M", [1, 4, 90])
def test_nan_scale_reaches_its_own_row(M):
    K, N = 128, 32
    q, wq = codes((M, K), 1), codes((1, N, K), 2)
    scale, w_scale = scales((M,), 3), scales((1, N), 4)
    scale[M // 2] = float("nan")
    out = torch.empty(M, N, device="cuda")
    bqe.moe_expert_product(q, scale, wq, w_scale, out)
    bad = torch.isnan(out)
    assert bad[M // 2].all() and bad.sum() == N


def test_product_on_another_stream_and_in_a_graph():
    T, k, E, K, N = 40, 3, 8, 256, 128
    _, _, _, offsets, row_src, _ = S.routing(T, k, E, 8)
    q, wq, scale, w_scale = codes((T, K), 1), codes((E, N, K), 2), scales((T,), 3), scales((E, N), 4)
    off, src = dev(offsets), dev(row_src)
    want, out = torch.empty(T * k, N, device="cuda"), torch.zeros(T * k, N, device="cuda")
    bqe.moe_expert_product(q, scale, wq, w_scale, want, off, src, k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bqe.moe_expert_product(q, scale, wq, w_scale, out, off, src, k, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    x = torch.randn(T, K, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bqe.moe_quantize_rows(x, q, scale)
        bqe.moe_expert_product(q, scale, wq, w_scale, out, off, src, k)
    x.copy_(torch.randn(T, K, device="cuda"))
    graph.replay()
    bqe.moe_quantize_rows(x, q, scale)
    bqe.moe_expert_product(q, scale, wq, w_scale, want, off, src, k)
    assert torch.equal(out, want)


def test_no_rows():
    q, wq = torch.empty(0, 64, dtype=torch.int8, device="cuda"), codes((2, 8, 64), 1)
    f = torch.empty(0, device="cuda")
    bqe.moe_quantize_rows(torch.empty(0, 64, device="cuda"), q, f)
    bqe.moe_expert_product(q, f, wq, scales((2, 8), 1), torch.empty(0, 8, device="cuda"),
                           torch.zeros(3, dtype=torch.int32, device="cuda"))


def test_weights_past_32_bits():
    """4.3e9 weights: the last experts' rows read their own matrices."""
    E, K, N = 130, 4096, 8192
    wq = torch.zeros((E, N, K), dtype=torch.int8, device="cuda")
    assert wq.numel() > 2 ** 32
    wq[E - 1] = codes((N, K), 1)
    wq[E - 2] = codes((N, K), 2)
    ends = np.zeros(E + 1, np.int32)
    ends[E - 1], ends[E] = 2, 40
    q, scale, w_scale = codes((40, K), 3), scales((40,), 4), scales((E, N), 5)
    out = torch.empty(40, N, device="cuda")
    bqe.moe_expert_product(q, scale, wq, w_scale, out, dev(ends))
    want, mag, top = product64(q, scale, wq, w_scale, ends, np.arange(40))
    check(out, want, mag, top, K, F32)


@pytest.mark.parametrize("E,M,N", [(1, 100, 256), (1, 2560, 2560)])  # one CTA a tile, a pair of CTAs a tile
def test_a_wait_that_runs_out_is_reported(E, M, N):
    K = 512
    q, wq, scale, w_scale = codes((M, K), 1), codes((E, N, K), 2), scales((M,), 3), scales((E, N), 4)
    out, want = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    bqe.moe_expert_product(q, scale, wq, w_scale, want)
    bqe.moe_check_product()
    bqe.moe_test_stall_next_product()
    bqe.moe_expert_product(q, scale, wq, w_scale, out)
    with pytest.raises(bqe.MoeError) as e:
        bqe.moe_check_product()
    assert e.value.status == bqe.MOE_ERR_TIMEOUT
    bqe.moe_expert_product(q, scale, wq, w_scale, out)
    bqe.moe_check_product()
    assert torch.equal(out, want)


@pytest.mark.parametrize("K,M,N", [(128, 20000, 4096), (384, 12000, 4096), (1152, 12000, 4096), (640, 4000, 2048)])
def test_odd_units_over_many_tiles(K, M, N):
    """An odd number of K units a tile, many tiles a CTA: every call gives the exact sums."""
    q, wq = codes((M, K), 31), codes((3, N, K), 32)
    scale, w_scale = scales((M,), 33), scales((3, N), 34)
    ends = np.array([0, M // 2, M // 2 + 300, M], np.int32)
    want, mag, top = product64(q, scale, wq, w_scale, ends, np.arange(M))
    first = torch.empty(M, N, device="cuda")
    bqe.moe_expert_product(q, scale, wq, w_scale, first, dev(ends))
    check(first, want, mag, top, K, F32)
    out = torch.empty(M, N, device="cuda")
    for _ in range(10):
        out.fill_(float("nan"))
        bqe.moe_expert_product(q, scale, wq, w_scale, out, dev(ends))
        assert torch.equal(out, first)


@pytest.mark.parametrize("M", [2, 90, 3000])
def test_calls_in_a_row_read_what_the_last_one_wrote(M):
    """Codes and scales are written again before every product, into the same buffers."""
    K, N, n = 512, 2048, 30
    wq, w_scale = codes((1, N, K), 2), scales((1, N), 3)
    x = torch.randn(n, M, K, device="cuda")
    q, scale = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    want, got = torch.empty(n, M, N, device="cuda"), torch.zeros(n, M, N, device="cuda")
    for i in range(n):
        bqe.moe_quantize_rows(x[i], q, scale)
        torch.cuda.synchronize()
        bqe.moe_expert_product(q, scale, wq, w_scale, want[i])
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(n):
            bqe.moe_quantize_rows(x[i], q, scale)
            bqe.moe_expert_product(q, scale, wq, w_scale, got[i])
    for _ in range(5):
        got.zero_()
        graph.replay()
        assert torch.equal(got, want)
