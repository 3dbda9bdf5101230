"""moe_quantize_blocks and moe_dequantize_blocks against their definitions in 64 bits.

Scales of their own are powers of two, so block scales and codes are those of the
exact quotients: equal bytes.  With given scales each quotient is rounded in fp32, as
the workloads' own encoder does: equal bytes again.  A gated row's values carry the
roundings of exp (2 units), the sum, the division and the product, 8 * 2^-24 in all: its
scales and codes lie between those of the interval's ends.
Back: code times e4m3 has at most 6 bits, times a power of two it is exact, times any
other scale rounded once in fp32, then to the rows' type.
"""
import numpy as np
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from tests import _blocks as B
from tests.test_gpu_sorted_rows import BF16, EPS, F16, F32, f64, rows_of
from workloads.generate import encode_mxfp4_rows, encode_nvfp4_rows

pytestmark = pytest.mark.gpu
FMTS = [B.MXFP4, B.NVFP4]
# rows, K, padding between rows of x
SHAPES = [(1, 32, 0), (1, 4096, 0), (5, 96, 1), (64, 2048, 0), (33, 1120, 8), (300, 992, 3), (3, 20000, 0), (2, 131072, 0),
          (17, 4128, 0), (9, 8192, 4), (7, 16384, 0), (1000, 64, 0)]


def outputs(rows, K, fmt, pad=0):
    q = torch.full((rows, K // 2 + pad), 0x77, dtype=torch.uint8, device="cuda")[:, :K // 2]
    s = torch.full((rows, K // B.size(fmt)), 0x55, dtype=torch.uint8, device="cuda")
    return q, s, torch.full((rows,), -1.0, device="cuda") if fmt == B.NVFP4 else None


@pytest.mark.parametrize("rows,K,pad", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_blocks(rows, K, pad, dtype, fmt):
    x = rows_of(rows, K, dtype, 100 * rows + K, pad)
    x[rows // 2, :K // 2] = 0
    x[rows // 2, 3] = -0.0
    q, s, scale = outputs(rows, K, fmt, pad)
    bqe.moe_quantize_blocks(x, q, s, scale, fmt)
    v = f64(x)
    g = None if scale is None else B.row_scale(v)
    if scale is not None:
        assert np.array_equal(f64(scale), g)
    want = B.scale_bytes(v, fmt, g)
    assert np.array_equal(s.cpu().numpy(), want)
    assert np.array_equal(q.cpu().numpy(), B.pack(B.codes(v, B.scale_values(want, fmt), g)))
    if pad:
        assert torch.all(q._base[:, K // 2:] == 0x77)


@pytest.mark.parametrize("rows,K,pad", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_gated_blocks(rows, K, pad, dtype, fmt):
    x = rows_of(rows, 2 * K, dtype, 7 * rows + K, pad)
    x[rows // 2, :K] = 0
    q, s, scale = outputs(rows, K, fmt)
    bqe.moe_quantize_blocks(x, q, s, scale, fmt, gated=True)
    x64 = f64(x)
    v = x64[:, :K] / (1 + np.exp(-x64[:, :K])) * x64[:, K:]
    lo, hi = 1 - 8 * EPS, 1 + 8 * EPS
    g = None if scale is None else f64(scale)
    if g is not None:
        assert np.all((B.row_scale(v * lo) <= g) & (g <= B.row_scale(v * hi)))
    b = s.cpu().numpy()
    assert np.all((B.scale_bytes(v * lo, fmt, g) <= b) & (b <= B.scale_bytes(v * hi, fmt, g)))
    sv, c = B.scale_values(b, fmt), B.unpack(q.cpu().numpy())
    low, high = B.codes(v * lo, sv, g), B.codes(v * hi, sv, g)
    live = v != 0
    assert np.all((low <= c) & (c <= high) | ~live)
    assert not (c[~live] & 7).any()


@pytest.mark.parametrize("rows,K", [(1, 32), (40, 2048), (5, 8224), (300, 992)])
def test_given_scales_are_the_encoders_bytes(rows, K):
    """One scale of a whole matrix, as a layer's NVFP4 experts have it, and MXFP4 bytes."""
    w = (np.random.default_rng(K).standard_normal((rows, K)) / np.sqrt(K)).astype(np.float32)
    w[rows // 2, 16:48] = 0
    x = torch.from_numpy(w).cuda()
    packed, bytes_, g = encode_nvfp4_rows(w)
    q, s, _ = outputs(rows, K, B.NVFP4)
    bqe.moe_quantize_blocks(x, q, s, torch.full((rows,), float(g), device="cuda"), B.NVFP4, given=True)
    assert np.array_equal(s.cpu().numpy(), bytes_) and np.array_equal(q.cpu().numpy(), packed)
    packed, bytes_ = encode_mxfp4_rows(w)
    q, s, _ = outputs(rows, K, B.MXFP4)
    bqe.moe_quantize_blocks(x, q, s, None, B.MXFP4)
    assert np.array_equal(s.cpu().numpy(), bytes_) and np.array_equal(q.cpu().numpy(), packed)


@pytest.mark.parametrize("g", [0.0, float("nan"), 1e-38, 1e38, 1e-45])
def test_given_scales_out_of_all_proportion(g):
    """Codes 0 where the scales leave fp32, the largest codes where they are far too small; nothing else."""
    x = torch.randn(3, 64, device="cuda")
    x[1] = 0
    q, s, _ = outputs(3, 64, B.NVFP4)
    bqe.moe_quantize_blocks(x, q, s, torch.full((3,), g, device="cuda"), B.NVFP4, given=True)
    c = B.unpack(q.cpu().numpy()) & 7
    if g in (1e-38,):
        assert np.all(s[0].cpu().numpy() == 126) and np.all(c[0][f64(x)[0] != 0] == 7)
    elif g == 1e38:
        assert not s.any() and not c.any()
    elif g == g and g > 0:
        assert np.all(s[0].cpu().numpy() == 126)
    else:
        assert not c.any()
    assert not c[1].any()


@pytest.mark.parametrize("fmt", FMTS)
def test_every_half_goes_to_even(fmt):
    """Values half way between two codes, and one unit to either side, at several powers of two."""
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    rows = []
    for scale in (1.0, 0.5, 2.0 ** -20, 2.0 ** 30):
        for nudge in (0, -1, 1):
            v = ties.astype(np.float32) * np.float32(scale)
            if nudge:
                v = np.nextafter(v, np.float32(np.inf if nudge > 0 else 0))
            row = np.zeros(64, np.float32)
            row[:7], row[20:27], row[40:47] = v, -v, v
            row[[15, 31, 47, 63]] = 6 * scale  # every block's maximum: d is the power of two
            rows.append(row)
    x = np.stack(rows)
    q, s, g = outputs(len(rows), 64, fmt)
    bqe.moe_quantize_blocks(torch.from_numpy(x).cuda(), q, s, g, fmt)
    want_g = None if g is None else B.row_scale(x.astype(np.float64))
    want = B.scale_bytes(x.astype(np.float64), fmt, want_g)
    assert np.array_equal(s.cpu().numpy(), want)
    assert np.array_equal(q.cpu().numpy(), B.pack(B.codes(x.astype(np.float64), B.scale_values(want, fmt), want_g)))
    assert np.array_equal(B.unpack(q.cpu().numpy())[0, :7], [0, 2, 2, 4, 4, 6, 6])


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("fmt", FMTS)
def test_extremes(dtype, fmt):
    """Infinities and NaN, the largest and the smallest finite values, zeros."""
    K = 128
    x = torch.ones(7, K, device="cuda").to(dtype)
    x[0, K - 1], x[1, 0], x[2, 3] = float("inf"), float("nan"), float("-inf")
    x[3] = torch.finfo(dtype).max
    x[4] = torch.finfo(dtype).smallest_normal * 2.0 ** -3
    x[5] = 0
    q, s, g = outputs(7, K, fmt)
    bqe.moe_quantize_blocks(x, q, s, g, fmt)
    back = torch.empty_like(x)
    bqe.moe_dequantize_blocks(q, s, back, g, fmt)
    per = B.size(fmt)
    nan_at = [(0, (K - 1) // per), (1, 0), (2, 0)]
    nan_byte = 255 if fmt == B.MXFP4 else 127
    for r, b in nan_at:
        assert s[r, b] == nan_byte and not q[r, b * per // 2:(b + 1) * per // 2].any()
        assert torch.isnan(back[r, b * per:(b + 1) * per]).all()
    if fmt == B.NVFP4:
        assert torch.isnan(g[:3]).all() and torch.isnan(back[:3]).all()
    else:
        assert torch.equal(back[0, :per], x[0, :per])
    x64 = f64(x)
    # a block's maximum m: with e2m1's largest step 2 and MXFP4 saturating from 8 to 6, at most a quarter off
    # (NVFP4: half a step of e4m3, 2^-4, and of e2m1); below the smallest scale nothing is left
    if fmt == B.NVFP4:
        # with m = 2^128 in fp32 and bf16 and 2^16 in fp16, m (1 - 2^-8) / 6 / (m 2^-11) = 340 and
        # m / 6 / (m 2^-11) = 341.3 both round to e4m3's 352, and 352 * 6 * m 2^-11 = 1.03 m is past the type
        assert torch.all(s[3] == 123) and B.FINE[123] == 352
        assert g[3] == 2.0 ** (5 if dtype is F16 else 117) and torch.all(back[3] == float("inf"))
    else:
        assert np.all(np.abs(f64(back)[3] - x64[3]) <= x64[3] / 4)
    assert np.all(np.abs(f64(back)[4]) <= 2 * np.abs(x64[4]))
    assert not q[5].any() and not back[5].any()
    # ones: 1 / 6 / 2^-11 = 341.3 rounds to 352, and 352 * 6 * 2^-11 = 1.03125
    assert torch.all(back[6] == (1.03125 if fmt == B.NVFP4 else 1.0))


@pytest.mark.parametrize("rows,K,pad", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("scaled", [False, True])
def test_dequantize_blocks(rows, K, pad, dtype, fmt, scaled):
    gen = torch.Generator("cuda").manual_seed(rows + K)
    q = torch.randint(0, 256, (rows, K // 2 + pad), generator=gen, dtype=torch.uint8, device="cuda")[:, :K // 2]
    low, high = (117, 133) if fmt == B.MXFP4 else (0, 127)
    s = torch.randint(low, high, (rows, K // B.size(fmt)), generator=gen, dtype=torch.uint8, device="cuda")
    g = torch.rand(rows, generator=gen, device="cuda") + 0.01 if scaled else None
    x = torch.full((rows, K + pad), 7.0, dtype=dtype, device="cuda")
    bqe.moe_dequantize_blocks(q, s, x[:, :K], g, fmt)
    v = B.values(q.cpu().numpy(), s.cpu().numpy(), fmt)  # exact in fp32
    want = torch.from_numpy(v.astype(np.float32)).cuda()
    if scaled:
        want = want * g[:, None]
    assert torch.equal(x[:, :K], want.to(dtype))
    assert torch.all(x[:, K:] == 7)


def test_there_and_back_is_a_fixed_point():
    """Values that blocks can hold come back as they are: a second pass changes nothing."""
    for fmt in FMTS:
        x = rows_of(50, 512, F32, 3)
        q, s, g = outputs(50, 512, fmt)
        bqe.moe_quantize_blocks(x, q, s, g, fmt)
        once, twice = torch.empty_like(x), torch.empty_like(x)
        bqe.moe_dequantize_blocks(q, s, once, g, fmt)
        bqe.moe_quantize_blocks(once, q, s, g, fmt, given=g is not None)
        bqe.moe_dequantize_blocks(q, s, twice, g, fmt)
        # (a block's maximum is 6 times an e4m3 scale, or 4 to 6 times a power of two: its scale stays)
        assert torch.equal(once, twice)


def test_other_stream_and_graph():
    x = rows_of(64, 1024, BF16, 5)
    q, s, g = outputs(64, 1024, B.NVFP4)
    bqe.moe_quantize_blocks(x, q, s, g, B.NVFP4)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    q2, s2, g2 = outputs(64, 1024, B.NVFP4)
    back, back2 = torch.empty_like(x), torch.empty_like(x)
    bqe.moe_dequantize_blocks(q, s, back, g, B.NVFP4)
    torch.cuda.synchronize()
    bqe.moe_quantize_blocks(x, q2, s2, g2, B.NVFP4, stream=side)
    side.synchronize()
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(g, g2)
    with torch.cuda.graph(graph):
        bqe.moe_quantize_blocks(x, q2, s2, g2, B.NVFP4)
        bqe.moe_dequantize_blocks(q2, s2, back2, g2, B.NVFP4)
    x.copy_(rows_of(64, 1024, BF16, 6))
    graph.replay()
    bqe.moe_quantize_blocks(x, q, s, g, B.NVFP4)
    bqe.moe_dequantize_blocks(q, s, back, g, B.NVFP4)
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(back, back2)
