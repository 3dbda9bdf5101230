"""moe_norm_rows and moe_norm_rows_backward against their definitions in 64 bits.

h is one fp32 sum rounded to the rows' type: equal bits.  A sum of H squares in fp32
is off by at most its longest chain of additions, below 200 for every kernel form (up to
128 in a thread, 5 in a warp, 32 over the warps), times 2^-24, all terms being positive; with the
division, eps, root and reciprocal rstd is within 104 * 2^-24, y within 107 * 2^-24 of its
value, then rounded.  The dot product of the gradient has H terms of three roundings each:
(200 + 4) 2^-24 of the sum of their absolute values, however it is cut; dgamma sums T
terms: at most T + 40.
"""
import numpy as np
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from tests.test_gpu_sorted_rows import BF16, EPS, F16, F32, between, f64, rows_of

pytestmark = pytest.mark.gpu
# T, H, padding between rows
SHAPES = [(1, 1, 0), (1, 4096, 0), (3, 7, 1), (33, 128, 3), (257, 1030, 0), (64, 4096, 8), (130, 2047, 2), (19, 8200, 0),
          (5, 16384, 0), (3, 33001, 0), (2, 131072, 0), (700, 256, 0), (1300, 96, 5), (9, 6144, 4), (4, 12288, 0),
          (1000, 2048, 8), (459, 4096, 0), (460, 8192, 0)]
TYPES = [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)]


def gamma_of(H, dtype, seed=9):
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(H, generator=g) + 0.5).to(dtype).cuda()


def rstd64(h, eps):
    return 1 / np.sqrt((h ** 2).mean(1) + eps)


@pytest.mark.parametrize("T,H,pad", SHAPES)
@pytest.mark.parametrize("dtype,gamma_dtype", TYPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_rows(T, H, pad, dtype, gamma_dtype, residual):
    x, gamma, eps = rows_of(T, H, dtype, T + H, pad), gamma_of(H, gamma_dtype), 1e-5
    res = rows_of(T, H, dtype, T + H + 1, pad) if residual else None
    h, y = rows_of(T, H, dtype, 2, pad), rows_of(T, H, dtype, 3, pad)
    rstd = torch.full((T,), -1.0, device="cuda")
    bqe.moe_norm_rows(x, gamma, y, eps, res, h, rstd)
    want_h = (x.float() + res.float()).to(dtype) if residual else x
    assert torch.equal(h, want_h)
    r = rstd64(f64(h), eps)
    assert np.all(np.abs(f64(rstd) - r) <= 104 * EPS * r)
    want = f64(h) * r[:, None] * f64(gamma)
    between(y, want, 107 * EPS * np.abs(want), dtype)
    if pad:
        assert torch.isnan(h._base[:, H:]).all() and torch.isnan(y._base[:, H:]).all()


@pytest.mark.parametrize("T,H,pad", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("keep", ["y", "h", "both", "codes alone"])
def test_codes_are_those_of_the_rows(T, H, pad, dtype, keep):
    """q and scale are what moe_quantize_rows makes of y, bit for bit, whichever outputs are asked for."""
    x, res, gamma = rows_of(T, H, dtype, 5, pad), rows_of(T, H, dtype, 6, pad), gamma_of(H, F32)
    x[T // 2], res[T // 2] = 0, 0
    y0, h0 = torch.empty(T, H, dtype=dtype, device="cuda"), torch.empty(T, H, dtype=dtype, device="cuda")
    bqe.moe_norm_rows(x, gamma, y0, 1e-6, res, h0)
    q0, s0 = torch.empty(T, H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    bqe.moe_quantize_rows(y0, q0, s0)
    y = torch.empty_like(y0) if keep in ("y", "both") else None
    h = torch.empty_like(h0) if keep in ("h", "both") else None
    q = torch.full((T, H + pad), 77, dtype=torch.int8, device="cuda")[:, :H]
    s = torch.full((T,), -1.0, device="cuda")
    bqe.moe_norm_rows(x, gamma, y, 1e-6, res, h, None, q, s)
    assert torch.equal(q, q0) and torch.equal(s, s0)
    assert y is None or torch.equal(y, y0)
    assert h is None or torch.equal(h, h0)
    assert s[T // 2] == 0 and not q[T // 2].any()


@pytest.mark.parametrize("H", [64, 2047, 4096, 9001, 33000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_residual_stream_in_place(H, dtype):
    x, res, gamma = rows_of(7, H, dtype, 1), rows_of(7, H, dtype, 2), gamma_of(H, F32)
    y0, h0, y = (torch.empty(7, H, dtype=dtype, device="cuda") for _ in range(3))
    bqe.moe_norm_rows(x, gamma, y0, 1e-6, res, h0)
    q, s = torch.empty(7, H, dtype=torch.int8, device="cuda"), torch.empty(7, device="cuda")
    stream = res.clone()
    bqe.moe_norm_rows(x, gamma, y, 1e-6, stream, stream, None, q, s)
    assert torch.equal(stream, h0) and torch.equal(y, y0)
    stream = x.clone()
    bqe.moe_norm_rows(stream, gamma, y, 1e-6, res, stream)
    assert torch.equal(stream, h0) and torch.equal(y, y0)


def test_rows_at_the_ends_of_the_range():
    """Zeros, tiny and large rows, infinities and NaN stay in their own row."""
    H = 512
    x = torch.randn(6, H, device="cuda")
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 1e15
    x[3, 5] = float("inf")
    x[4, 7] = float("nan")
    y, rstd = torch.empty_like(x), torch.empty(6, device="cuda")
    q, s = torch.empty(6, H, dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
    bqe.moe_norm_rows(x, torch.ones(H, device="cuda"), y, 1e-6, None, None, rstd, q, s)
    assert not y[0].any() and abs(rstd[0].item() - 1000) <= 104 * EPS * 1000 and s[0] == 0 and not q[0].any()
    assert torch.equal(y[1], x[1] * rstd[1])
    r = rstd64(f64(x[[2, 5]]), 1e-6)
    assert np.allclose(f64(rstd[[2, 5]]), r, rtol=104 * EPS, atol=0)
    assert torch.isnan(y[3, 5]) and rstd[3] == 0 and torch.isnan(s[3]) and not q[3].any()
    assert torch.isnan(y[4]).all() and torch.isnan(s[4]) and not q[4].any()
    assert torch.isfinite(y[5]).all() and torch.isfinite(s[5])


# ----------------------------------------------------------------- gradient --
def backward64(dy, h, gamma, rstd, dh):
    """(dx, its magnitude for the tolerance, dgamma, sum of absolute values of its terms)"""
    r, g = rstd[:, None], dy * gamma
    dot, mag = (g * h).mean(1, keepdims=True), np.abs(g * h).mean(1, keepdims=True)
    dx = r * g - h * r ** 3 * dot + dh
    size = 6 * np.abs(r * g) + np.abs(h * r ** 3) * (6 * np.abs(dot) + 204 * mag) + 2 * np.abs(dh)
    return dx, size, (dy * h * r).sum(0), np.abs(dy * h * r).sum(0)


@pytest.mark.parametrize("T,H,pad", SHAPES)
@pytest.mark.parametrize("dtype,gamma_dtype", TYPES)
@pytest.mark.parametrize("stream", [False, True])
def test_norm_rows_backward(T, H, pad, dtype, gamma_dtype, stream):
    h, dy, gamma = rows_of(T, H, dtype, 1, pad), rows_of(T, H, dtype, 2, pad), gamma_of(H, gamma_dtype)
    dh = rows_of(T, H, dtype, 3, pad) if stream else None
    rstd = torch.from_numpy(rstd64(f64(h), 1e-6)).float().cuda()
    dx, dgamma = rows_of(T, H, dtype, 4, pad), torch.full((H,), 7.0, device="cuda")
    scratch = torch.empty(bqe.moe_norm_scratch_bytes(T, H), dtype=torch.uint8, device="cuda")
    bqe.moe_norm_rows_backward(dy, h, gamma, rstd, dx, dgamma, scratch, dh)
    want, size, want_g, mag = backward64(f64(dy), f64(h), f64(gamma), f64(rstd), 0 if dh is None else f64(dh))
    between(dx, want, EPS * size, dtype)
    between(dgamma, want_g, (T + 40) * EPS * mag, F32)
    if pad:
        assert torch.isnan(dx._base[:, H:]).all()
    again, g2 = torch.empty(T, H, dtype=dtype, device="cuda"), torch.empty(H, device="cuda")
    bqe.moe_norm_rows_backward(dy, h, gamma, rstd, again, g2, scratch, dh)
    assert torch.equal(again, dx) and torch.equal(g2, dgamma)
    alone = torch.empty_like(again)
    bqe.moe_norm_rows_backward(dy, h, gamma, rstd, alone, dh=dh)
    assert torch.equal(alone, dx)


@pytest.mark.parametrize("T,H", [(8, 96), (8, 2047), (8, 9000), (8, 33001), (500, 4096), (1000, 2048), (470, 8192)])
def test_gradient_in_place(T, H):
    h, dy, dh, gamma = rows_of(T, H, BF16, 1), rows_of(T, H, BF16, 2), rows_of(T, H, BF16, 3), gamma_of(H, F32)
    rstd = torch.rand(T, device="cuda") + 0.5
    dx, g = torch.empty(T, H, dtype=BF16, device="cuda"), [torch.empty(H, device="cuda") for _ in range(2)]
    scratch = torch.empty(bqe.moe_norm_scratch_bytes(T, H), dtype=torch.uint8, device="cuda")
    bqe.moe_norm_rows_backward(dy, h, gamma, rstd, dx, g[0], scratch, dh)
    for over in (dy.clone(), dh.clone()):
        one = torch.equal(over, dy)
        bqe.moe_norm_rows_backward(over if one else dy, h, gamma, rstd, over, g[1], scratch, dh if one else over)
        assert torch.equal(over, dx) and torch.equal(g[0], g[1])


def test_gradient_of_differences():
    """dx and dgamma against central differences of the forward's own definition in 64 bits."""
    T, H, eps = 3, 40, 1e-4
    x, dy, gamma = rows_of(T, H, F32, 1), rows_of(T, H, F32, 2), gamma_of(H, F32)
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    bqe.moe_norm_rows(x, gamma, y, eps, None, None, rstd)
    dx, dgamma = torch.empty_like(x), torch.empty(H, device="cuda")
    scratch = torch.empty(bqe.moe_norm_scratch_bytes(T, H), dtype=torch.uint8, device="cuda")
    bqe.moe_norm_rows_backward(dy, x, gamma, rstd, dx, dgamma, scratch)

    def loss(a, b):
        return (a * rstd64(a, eps)[:, None] * b * f64(dy)).sum()

    a, b, step = f64(x), f64(gamma), 1e-5
    for t, c in [(0, 0), (1, 17), (2, 39)]:
        e = np.zeros_like(a)
        e[t, c] = step
        # central differences err by step^2 times a third derivative of order 10, and 1e-16 / step
        assert abs((loss(a + e, b) - loss(a - e, b)) / (2 * step) - dx[t, c].item()) < 1e-5
        e = np.zeros_like(b)
        e[c] = step
        assert abs((loss(a, b + e) - loss(a, b - e)) / (2 * step) - dgamma[c].item()) < 1e-5


def test_no_rows():
    x, dgamma = torch.empty(0, 64, device="cuda"), torch.full((64,), 7.0, device="cuda")
    bqe.moe_norm_rows(x, torch.ones(64, device="cuda"), x)
    scratch = torch.empty(bqe.moe_norm_scratch_bytes(0, 64), dtype=torch.uint8, device="cuda")
    bqe.moe_norm_rows_backward(x, x, torch.ones(64, device="cuda"), torch.empty(0, device="cuda"), x, dgamma, scratch)
    assert not dgamma.any()


def test_other_stream_and_graph():
    T, H = 200, 1024
    x, res, gamma = rows_of(T, H, BF16, 1), rows_of(T, H, BF16, 2), gamma_of(H, F32)
    out = [torch.empty(T, H, dtype=BF16, device="cuda") for _ in range(6)]
    rstd, g = torch.empty(T, device="cuda"), [torch.empty(H, device="cuda") for _ in range(2)]
    scratch = torch.empty(bqe.moe_norm_scratch_bytes(T, H), dtype=torch.uint8, device="cuda")

    def step(h, y, dx, dgamma, stream=None):
        bqe.moe_norm_rows(x, gamma, y, 1e-6, res, h, rstd, stream=stream)
        bqe.moe_norm_rows_backward(y, h, gamma, rstd, dx, dgamma, scratch, x, stream=stream)

    step(*out[:3], g[0])
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    step(*out[3:], g[1], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out[:3] + g[:1], out[3:] + g[1:]))
    with torch.cuda.graph(graph):
        step(*out[3:], g[1])
    x.copy_(rows_of(T, H, BF16, 4))
    for _ in range(3):
        graph.replay()
    step(*out[:3], g[0])
    assert all(torch.equal(a, b) for a, b in zip(out[:3] + g[:1], out[3:] + g[1:]))


@pytest.mark.parametrize("T", [70000])
def test_offsets_past_32_bits(T):
    """Rows whose last element lies past 2^32 bytes, and past 2^31 elements by their stride."""
    H, stride = 64, 40000
    base = torch.empty(T * stride, dtype=BF16, device="cuda")
    x = base.view(T, stride)[:, :H]
    x.copy_(rows_of(T, H, BF16, 1))
    gamma, y, h = gamma_of(H, F32), base.view(T, stride)[:, H:2 * H], base.view(T, stride)[:, 2 * H:3 * H]
    small, rstd = torch.empty(T, H, dtype=BF16, device="cuda"), torch.empty(T, device="cuda")
    bqe.moe_norm_rows(x, gamma, y, 1e-6, None, h, rstd)
    bqe.moe_norm_rows(x.contiguous(), gamma, small, 1e-6)
    assert torch.equal(y, small) and torch.equal(h, x)
    dx = base.view(T, stride)[:, 3 * H:4 * H]
    bqe.moe_norm_rows_backward(y, h, gamma, rstd, dx)
    bqe.moe_norm_rows_backward(small, x.contiguous(), gamma, rstd, small)
    assert torch.equal(dx, small)


# Rows of up to 128 chunks, a warp each: every number of chunks a lane, more rows than the
# warps of the grid's blocks walk at once, and a last block that is not full.
SHORT = [(3001, 64, 0), (2049, 504, 0), (5000, 512, 8), (2051, 1024, 0), (4099, 128, 0), (4001, 127, 0), (2500, 33, 2),
         (2048, 1000, 8), (9, 250, 6), (3650, 8, 0)]
# two chunks a thread, with a last one that some threads do not have
SHORT += [(1300, 2040, 0), (700, 4088, 0), (1300, 1100, 4), (650, 511, 1)]


@pytest.mark.parametrize("T,H,pad", SHORT)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_short_rows(T, H, pad, dtype):
    test_norm_rows(T, H, pad, dtype, F32, True)
    test_norm_rows(T, H, pad, dtype, dtype, False)
    test_codes_are_those_of_the_rows(T, H, pad, dtype, "both")
    test_codes_are_those_of_the_rows(T, H, pad, dtype, "codes alone")


@pytest.mark.parametrize("T,H,pad", SHORT)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_short_rows_backward(T, H, pad, dtype):
    test_norm_rows_backward(T, H, pad, dtype, F32, True)
    test_norm_rows_backward(T, H, pad, dtype, dtype, False)


@pytest.mark.parametrize("T,H", [(2500, 64), (4000, 256), (2049, 1024), (5000, 127)])
def test_short_rows_in_place(T, H):
    """h over an input, dx over dy: a warp has read its row before it writes it."""
    test_gradient_in_place(T, H)
    x, res, gamma = rows_of(T, H, BF16, 1), rows_of(T, H, BF16, 2), gamma_of(H, F32)
    y0, h0, y = (torch.empty(T, H, dtype=BF16, device="cuda") for _ in range(3))
    bqe.moe_norm_rows(x, gamma, y0, 1e-6, res, h0)
    stream = res.clone()
    bqe.moe_norm_rows(x, gamma, y, 1e-6, stream, stream)
    assert torch.equal(stream, h0) and torch.equal(y, y0)


# Rows of 129 to 1024 chunks of 16 bytes, more of them than fit at once: the last rows of each group of threads
@pytest.mark.parametrize("T,H,pad", [(457, 2048, 0), (611, 1096, 8), (913, 1536, 0), (500, 4088, 8), (610, 2056, 0),
                                     (458, 8192, 0), (760, 4096, 0)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_backward_of_many_rows(T, H, pad, dtype):
    test_norm_rows_backward(T, H, pad, dtype, F32, True)
    test_norm_rows_backward(T, H, pad, dtype, dtype, False)
