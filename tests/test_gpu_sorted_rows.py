"""moe_dispatch, moe_combine, their gradients and the router's gradient against
their definitions in 64 bits.

Tolerances: a copy is exact.  A sum of k products in fp32 is within
(k + 1) 2^-24 of the sum of the terms' absolute values, a dot product of H terms
within (H + 1) 2^-24 of it, whatever the order.  Rounding to the output's type is
monotonic: the output lies between the rounded ends of that interval.
"""
import numpy as np
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from tests import _sorted as S

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rows_of(n, width, dtype, seed, pad=0):
    """Random rows with `pad` unused elements between them (NaN)."""
    g = torch.Generator().manual_seed(seed)
    t = torch.full((n, width + pad), float("nan"))
    t[:, :width] = torch.randn(n, width, generator=g)
    return t.to(dtype).cuda()[:, :width]


def f64(t):
    return t.double().cpu().numpy()


def between(got, want, bound, dtype):
    """got is some value of want +- bound, rounded to dtype (the ends' own
    rounding to fp32 on the way is half a unit, 2^-24)."""
    bound = bound + EPS * np.abs(want)
    lo, hi = (f64(torch.from_numpy(v).float().to(dtype)) for v in (want - bound, want + bound))
    g = f64(got)
    bad = ~((lo <= g) & (g <= hi))
    assert not bad.any(), (np.argwhere(bad)[:4], g[bad][:4], want[bad][:4], bound[bad][:4])


def within(got, want, mag, terms, dtype):
    between(got, want, terms * EPS * mag, dtype)


# T, k, E, H, drop, padding between rows
SHAPES = [(1, 1, 1, 1, 0.0, 0), (1, 6, 256, 4096, 0.0, 0), (1, 8, 8, 2, 0.0, 0), (3, 2, 16, 7, 0.4, 1),
          (33, 8, 1024, 128, 0.3, 3), (257, 3, 5, 1030, 0.2, 0), (64, 6, 256, 4096, 0.0, 8), (130, 4, 64, 2047, 0.5, 2),
          (19, 5, 9, 8200, 0.9, 0), (1000, 6, 256, 256, 0.0, 0)]
TYPES = [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)]


@pytest.mark.parametrize("T,k,E,H,drop,pad", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_dispatch(T, k, E, H, drop, pad, dtype):
    _, _, _, offsets, row_src, row_dst = S.routing(T, k, E, 11 * T + k, drop)
    x = rows_of(T, H, dtype, 1, pad)
    xs = rows_of(T * k, H, dtype, 2, pad)
    bqe.moe_dispatch(x, dev(offsets), dev(row_dst), xs)
    n = offsets[-1]
    want = torch.zeros(T * k, H, dtype=dtype, device="cuda")
    want[:n] = x[dev(row_src[:n].astype(np.int64) // k)]
    assert torch.equal(xs, want)


@pytest.mark.parametrize("T,k,E,H,drop,pad", SHAPES)
@pytest.mark.parametrize("dtype,out_dtype", TYPES)
def test_combine_and_dispatch_backward(T, k, E, H, drop, pad, dtype, out_dtype):
    _, _, w, offsets, _, row_dst = S.routing(T, k, E, 7 * T + k, drop)
    y = rows_of(T * k, H, dtype, 3, pad)
    y[offsets[-1]:] = float("nan")           # positions that hold nothing are not read
    w_dev = dev(np.where(row_dst.reshape(T, k) < 0, np.nan, w).astype(np.float32))  # nor the weights of empty slots
    out = rows_of(T, H, out_dtype, 4, pad)
    bqe.moe_combine(y, w_dev, dev(row_dst), out)
    want, mag = S.combine64(f64(y), w, row_dst, T, k)
    within(out, want, mag, k + 1, out_dtype)
    again = torch.empty_like(out)
    bqe.moe_combine(y, w_dev, dev(row_dst), again)
    assert torch.equal(out, again)
    dx = rows_of(T, H, out_dtype, 5, pad)
    bqe.moe_dispatch_backward(y, dev(row_dst), dx)
    want, mag = S.combine64(f64(y), None, row_dst, T, k)
    within(dx, want, mag, k + 1, out_dtype)


@pytest.mark.parametrize("T,k,E,H,drop,pad", SHAPES)
@pytest.mark.parametrize("dtype,out_dtype", TYPES)
def test_combine_backward(T, k, E, H, drop, pad, dtype, out_dtype):
    _, _, w, offsets, row_src, row_dst = S.routing(T, k, E, 5 * T + k, drop)
    n = offsets[-1]
    y, dout = rows_of(T * k, H, dtype, 6, pad), rows_of(T, H, out_dtype, 7, pad)
    y[n:] = float("nan")
    dy, dw = rows_of(T * k, H, dtype, 8, pad), torch.full((T, k), float("nan"), device="cuda")
    bqe.moe_combine_backward(dout, y, dev(w), dev(offsets), dev(row_dst), dy, dw)
    d64, y64 = f64(dout), f64(y)
    want = np.zeros((T * k, H))
    src = row_src[:n].astype(np.int64)
    want[:n] = w.reshape(-1)[src, None].astype(np.float64) * d64[src // k]
    within(dy, want, np.abs(want), 1, dtype)
    terms = d64[:, None, :] * np.where(row_dst.reshape(T, k, 1) >= 0, y64[np.maximum(row_dst, 0)].reshape(T, k, H), 0)
    within(dw, terms.sum(2), np.abs(terms).sum(2), H + 1, F32)


def test_combine_gradient_against_differences():
    """dy and dw are the differences of moe_combine's own definition."""
    T, k, E, H = 5, 3, 7, 10
    _, _, w, offsets, _, row_dst = S.routing(T, k, E, 3, 0.3)
    y, dout = rows_of(T * k, H, F32, 9), rows_of(T, H, F32, 10)
    dy, dw = torch.empty_like(y), torch.empty(T, k, device="cuda")
    bqe.moe_combine_backward(dout, y, dev(w), dev(offsets), dev(row_dst), dy, dw)
    d64, y64 = f64(dout), f64(y)

    def loss(yy, ww):
        return (S.combine64(yy, ww, row_dst, T, k)[0] * d64).sum()

    h = 1e-6  # the loss is linear in each: a difference is exact but for its own rounding
    w64 = w.astype(np.float64)
    for i in np.ndindex(y64.shape):
        e = np.zeros_like(y64)
        e[i] = h
        diff = (loss(y64 + e, w64) - loss(y64 - e, w64)) / (2 * h)
        assert abs(diff - f64(dy)[i]) <= 1e-6 * (1 + abs(diff))
    for i in np.ndindex(w64.shape):
        if row_dst.reshape(T, k)[i] < 0:
            assert dw[i] == 0
            continue
        e = np.zeros_like(w64)
        e[i] = h
        diff = (loss(y64, w64 + e) - loss(y64, w64 - e)) / (2 * h)
        assert abs(diff - f64(dw)[i]) <= 1e-5 * (1 + abs(diff))


# Per value: two fp32 transcendentals of at most 2 units (2^-22 together, halved by the square root), a sum of k terms
# of s, once squared, and under twenty further roundings: (2 k + 40) 2^-24 of the terms' absolute values.
@pytest.mark.parametrize("T,k,E,drop", [(1, 1, 1, 0.0), (1, 6, 256, 0.0), (5, 8, 8, 0.5), (300, 6, 256, 0.2),
                                        (77, 3, 1023, 0.9), (129, 4, 33, 0.0)])
def test_route_backward(T, k, E, drop):
    logits, ids, _, _, _, _ = S.routing(T, k, E, 13 * T + k, drop)
    logits = logits * np.float32(4)
    dw = np.random.default_rng(T).standard_normal((T, k)).astype(np.float32)
    got = torch.full((T, E), float("nan"), device="cuda")
    bqe.moe_route_backward(dev(logits), dev(ids), dev(dw), got, S.W_SCALE)
    want, mag = S.route_grad64(logits, ids, dw.astype(np.float64))
    assert np.all(np.abs(f64(got) - want) <= (2 * k + 40) * EPS * mag)
    if k == 1:
        assert not got.any()


def test_route_backward_against_differences():
    T, k, E = 6, 4, 9
    logits, ids, _, _, _, _ = S.routing(T, k, E, 21, 0.2)
    dw = np.random.default_rng(2).standard_normal((T, k))
    got = torch.empty(T, E, device="cuda")
    bqe.moe_route_backward(dev(logits), dev(ids), dev(dw.astype(np.float32)), got, S.W_SCALE)
    l, h = logits.astype(np.float64), 1e-5
    for i in np.ndindex(l.shape):
        e = np.zeros_like(l)
        e[i] = h
        diff = ((S.route_weights64(l + e, ids) - S.route_weights64(l - e, ids)) * dw).sum() / (2 * h)
        assert abs(diff - f64(got)[i]) <= 1e-6
    # and its weights are those of moe_route's definition where nothing is pruned
    assert np.allclose(S.route_weights64(l, np.abs(ids)).sum(1), S.W_SCALE)


def test_route_backward_extreme_logits():
    """Very negative and very positive logits give finite gradients: s is 0 (and
    the gradient with it) only where exp underflows."""
    logits = np.array([[-30.0, -31.0, -29.5, 0.0], [80.0, 79.0, 60.0, 0.0], [-300.0, -301.0, -302.0, 0.0]], np.float32)
    ids = np.tile(np.array([0, 1, 2], np.int32), (3, 1))
    dw = np.array([[1.0, -2.0, 0.5]] * 3, np.float32)
    got = torch.empty(3, 4, device="cuda")
    bqe.moe_route_backward(dev(logits), dev(ids), dev(dw), got, S.W_SCALE)
    want, mag = S.route_grad64(logits[:2], ids[:2], dw[:2].astype(np.float64))
    # log1p(exp(l)) at l = -30 is exp(l) to 2^-43: the same bound
    assert np.all(np.abs(f64(got)[:2] - want) <= 46 * EPS * mag)
    assert not got[2].any()


def test_bad_positions_are_empty_slots():
    """Positions outside [0, R) and ids outside [0, E) are skipped."""
    T, k, H = 4, 2, 16
    row_dst = np.array([0, 8, -5, 1, 2, 2 ** 31 - 1, 3, -2 ** 31], np.int32)
    x, y = rows_of(T, H, F32, 1), rows_of(T * k, H, F32, 2)
    xs = torch.full((T * k, H), 5.0, device="cuda")
    offsets = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    bqe.moe_dispatch(x, offsets, dev(row_dst), xs)
    assert torch.equal(xs[:4], x) and not xs[4:].any()
    out = torch.empty(T, H, device="cuda")
    bqe.moe_combine(y, torch.ones(T, k, device="cuda"), dev(row_dst), out)
    assert torch.equal(out, y[:4])
    dw = torch.empty(T, k, device="cuda")
    dy = torch.empty_like(y)
    bqe.moe_combine_backward(x, y, torch.ones(T, k, device="cuda"), offsets, dev(row_dst), dy, dw)
    assert torch.equal(dy[:4], x) and not dy[4:].any()
    assert [bool(v) for v in dw.reshape(-1)] == [True, False, False, True, True, False, True, False]
    dl = torch.empty(1, 4, device="cuda")
    bqe.moe_route_backward(torch.zeros(1, 4, device="cuda"), torch.tensor([[7, 2]], dtype=torch.int32, device="cuda"),
                           torch.ones(1, 2, device="cuda"), dl)
    assert not dl.any()


def test_infinities_and_nan_reach_only_their_own_rows():
    T, k, E, H = 8, 2, 4, 24
    _, _, w, offsets, _, row_dst = S.routing(T, k, E, 1)
    y = rows_of(T * k, H, BF16, 3)
    y[row_dst[0], 3], y[row_dst[3], 5] = float("nan"), float("inf")  # slots 0 of token 0 and 1 of token 1
    out = torch.empty(T, H, device="cuda")
    bqe.moe_combine(y, dev(w), dev(row_dst), out)
    bad = ~torch.isfinite(out)
    assert bad.sum() == 2 and bad[0, 3] and bad[1, 5]


def test_no_tokens():
    none = torch.empty(0, 8, device="cuda")
    i32 = torch.empty(0, dtype=torch.int32, device="cuda")
    offsets = torch.zeros(5, dtype=torch.int32, device="cuda")
    bqe.moe_dispatch(none, offsets, i32, none)
    bqe.moe_dispatch_backward(none, i32, none)
    bqe.moe_combine(none, none[:, :2], i32, none)
    bqe.moe_combine_backward(none, none, none[:, :2], offsets, i32, none, none[:, :2])
    bqe.moe_route_backward(none, i32.view(0, 2), none[:, :2], none)


def test_another_stream_and_a_graph():
    T, k, E, H = 40, 6, 64, 512
    _, _, w, offsets, _, row_dst = S.routing(T, k, E, 4, 0.1)
    y, dst, wd = rows_of(T * k, H, BF16, 3), dev(row_dst), dev(w)
    want = torch.empty(T, H, device="cuda")
    bqe.moe_combine(y, wd, dst, want)
    torch.cuda.synchronize()
    side, out = torch.cuda.Stream(), torch.zeros(T, H, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    bqe.moe_combine(y, wd, dst, out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bqe.moe_combine(y, wd, dst, out)
        bqe.moe_dispatch_backward(y, dst, out)
        bqe.moe_combine(y, wd, dst, out)
    y.mul_(2)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, 2 * want)


def test_offsets_past_32_bits():
    """2.2e9 elements on the sorted side: rows at the far end land where they should."""
    T, k, H = 33000, 8, 8336
    row_dst = torch.arange(T * k, dtype=torch.int32, device="cuda").flip(0)
    offsets = torch.tensor([0, T * k], dtype=torch.int32, device="cuda")
    x = torch.randn(T, H, device="cuda").to(BF16)
    xs = torch.empty(T * k, H, dtype=BF16, device="cuda")
    assert xs.numel() > 2 ** 31
    bqe.moe_dispatch(x, offsets, row_dst, xs)
    for t in (0, 1, T // 2, T - 1):
        for j in (0, k - 1):
            assert torch.equal(xs[T * k - 1 - (t * k + j)], x[t])
    out = torch.empty(T, H, dtype=torch.float32, device="cuda")
    bqe.moe_combine(xs, torch.full((T, k), 0.25, device="cuda"), row_dst, out)
    assert torch.equal(out, x.float() * 2)
    dw = torch.empty(T, k, device="cuda")
    bqe.moe_combine_backward(x, xs, torch.full((T, k), 0.25, device="cuda"), offsets, row_dst, xs.clone(), dw)
    norm = x.double().square().sum(1, keepdim=True)
    assert torch.all((dw.double() - norm).abs() <= (H + 1) * EPS * norm)


@pytest.mark.parametrize("T,H", [(4, 512), (64, 256), (700, 1024)])
def test_calls_in_a_row_read_what_the_last_one_wrote(T, H):
    """Each call's kernel may start before the one in front of it ends: its rows
    must be the new ones all the same, also where the buffer was read before."""
    k, E, n = 3, 4, 60
    _, _, _, offsets, _, row_dst = S.routing(T, k, E, 5)
    off, dst, w = dev(offsets), dev(row_dst), torch.ones(T, k, device="cuda")
    xs, outs = torch.zeros(T * k, H, device="cuda"), torch.empty(n, T, H, device="cuda")
    x = torch.arange(1.0, n + 1, device="cuda")[:, None, None].expand(n, T, H).contiguous()
    graph = torch.cuda.CUDAGraph()
    bqe.moe_dispatch(x[0], off, dst, xs)
    with torch.cuda.graph(graph):
        for i in range(n):
            bqe.moe_dispatch(x[i], off, dst, xs)
            bqe.moe_combine(xs, w, dst, outs[i])
    for _ in range(5):
        outs.zero_()
        graph.replay()
        assert torch.equal(outs, k * x)
