"""The 4-bit experts and the norm as they are used: a served layer against its definition in
64 bits, weights for moe_create, a training step with the norm in front, chains of calls.

Tolerances.  With fp32 rows between the products a gated value is within 20 * 2^-24 = d of its
own.  It has another code where it is within d of one of seven ties, a share of 7 d of the codes,
each off by at most half its value, and another block scale where the block's maximum is, 32 d of
the blocks, off by an eighth: relative L2 below sqrt(7 d) / 2 + sqrt(32 d) / 8 = 2.3e-3.
Gradients run in fp32 through sums of a few thousand terms: relative L2 below 1e-5.
"""
import numpy as np
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from block_quantized_expert_gb300 import sorted_experts as se
from tests import _blocks as B
from tests.test_gpu_block_product import FMTS, values
from tests.test_gpu_sorted_experts import routed, weights
from tests.test_gpu_sorted_rows import BF16, F32, f64
from workloads.generate import encode_mxfp4_rows, encode_nvfp4_rows

pytestmark = pytest.mark.gpu


def scaled(blocks, fmt):
    q, s, g = blocks
    v = values(q, s, fmt)
    return v if g is None else v * g.double()[..., None]


@pytest.mark.parametrize("T,k,E,H,I,drop", [(1, 6, 64, 1024, 512, 0.0), (33, 4, 16, 256, 128, 0.3), (700, 6, 24, 512, 288, 0.1)])
@pytest.mark.parametrize("fmt", FMTS)
def test_block_layer(T, k, E, H, I, drop, fmt):
    gate, up, down = weights(E, H, I)
    layer = se.BlockExperts(gate, up, down, fmt, rows=F32)
    logits, ids = routed(T, k, E, drop)
    s = se.sort_tokens(ids, E)
    w = se.router_weights(logits, ids)
    x = torch.randn(T, H, device="cuda").to(BF16)
    got = layer(x, s, w)
    bqe.moe_check_product()
    x64, gu64, d64 = scaled(layer.blocks(x), fmt), scaled(layer.gate_up, fmt), scaled(layer.down, fmt)
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        gu = x64[t] @ gu64[e].T
        h = f64(torch.nn.functional.silu(gu[:, :I]) * gu[:, I:])
        g = B.row_scale(h) if fmt == B.NVFP4 else None
        sb = B.scale_bytes(h, fmt, g)
        v = B.values(B.pack(B.codes(h, B.scale_values(sb, fmt), g)), sb, fmt) * (1 if g is None else g[:, None])
        want.index_add_(0, t, (torch.from_numpy(v).cuda() @ d64[e].T) * w[t, j].double()[:, None])
    assert float((got.double() - want).norm()) <= 2.3e-3 * float(want.norm())
    assert not got[(ids < 0).all(1)].any()
    # bf16 rows, the default, stay near the same layer: at most their own rounding moves a share of 7 * 2^-8 of the codes
    near = se.BlockExperts(gate, up, down, fmt)(x, s, w)
    assert float((near.double() - want).norm()) <= (7 * 2.0 ** -8) ** 0.5 * float(want.norm())


@pytest.mark.parametrize("E,N,K", [(3, 128, 256), (2, 256, 128)])
def test_layer_weights_are_the_encoders(E, N, K):
    """The bytes that the workloads' encoders make of the same matrices, for moe_create."""
    w = (np.random.default_rng(K).standard_normal((E, N, K)) / np.sqrt(K)).astype(np.float32)
    x = torch.from_numpy(w).cuda()
    q, s, none = se.quantize_layer_weights(x, bqe.MOE_WEIGHTS_MXFP4)
    q4, s4, g4 = se.quantize_layer_weights(x, bqe.MOE_WEIGHTS_NVFP4)
    assert none is None
    for e in range(E):
        want = encode_mxfp4_rows(w[e])
        assert np.array_equal(q[e].cpu().numpy(), want[0]) and np.array_equal(s[e].cpu().numpy(), want[1])
        want = encode_nvfp4_rows(w[e])
        assert np.array_equal(q4[e].cpu().numpy(), want[0]) and np.array_equal(s4[e].cpu().numpy(), want[1])
        assert g4[e].item() == want[2]


@pytest.mark.parametrize("fmt", FMTS)
def test_a_layer_of_ones_own_weights(fmt):
    """moe_create on weights made here: the layer is near the 4-bit experts of the same weights (they
    differ in the activations' 8 or 4 bits and, for NVFP4, in the scales of a matrix or a channel)."""
    T, k, E, H, I = 16, 2, 8, 256, 128
    gate, up, down = weights(E, H, I)
    parts = {}
    for name, m in (("gate", gate), ("up", up), ("down", down)):
        parts[name + "_q"], parts[name + "_s"], g = se.quantize_layer_weights(m, fmt)
        if g is not None:
            parts[name + "_g"] = g
    layer = bqe.moe_create(bqe.MoeConfig(H, I, E, k, T, weight_format=fmt), parts)
    logits, ids = routed(T, k, E, 0.0)
    w = se.router_weights(logits, ids)
    x = torch.randn(T, H, device="cuda").to(BF16)
    out = torch.empty(T, H, device="cuda")
    bqe.moe_forward(layer, x, ids, w, out)
    bqe.moe_check(layer)
    layer.close()
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            g, u, d = (scaled((parts[n + "_q"][e], parts[n + "_s"][e], None), fmt) * (parts[n + "_g"][e].double() if n + "_g" in parts else 1)
                       for n in ("gate", "up", "down"))
            h = torch.nn.functional.silu(g @ x[t].double()) * (u @ x[t].double())
            want[t] += w[t, j].double() * (d @ h)
    # e4m3 activations, twice: half a step is 2^-4 of a value, spread evenly 2^-4 / sqrt(3) in the
    # mean square, twice for x (gate and up), once for h
    assert float((out.double() - want).norm()) <= 3 * 2.0 ** -4 / 3 ** 0.5 * float(want.norm())


def test_norm_codes_feed_the_int8_experts():
    T, k, E, H, I = 50, 3, 8, 512, 256
    layer = se.Int8Experts(*weights(E, H, I))
    logits, ids = routed(T, k, E, 0.0)
    s, w = se.sort_tokens(ids, E), se.router_weights(logits, ids)
    x, stream = (torch.randn(T, H, device="cuda").to(BF16) for _ in range(2))
    gamma = torch.rand(H, device="cuda") + 0.5
    y, h, codes = se.norm_codes(x, gamma, stream)
    assert torch.equal(h, (x.float() + stream.float()).to(BF16))
    assert torch.equal(layer(y, s, w, codes), layer(y, s, w))
    alone, same, _ = se.norm_codes(h, gamma)
    assert torch.equal(alone, y) and same is h


# ----------------------------------------------------------------- training --
def norm64(x, gamma, residual, eps=1e-6):
    h = x if residual is None else x + residual
    return h * (h.square().mean(1, keepdim=True) + eps).rsqrt() * gamma, h


@pytest.mark.parametrize("T,H", [(1, 64), (90, 136), (300, 1030), (5, 9000)])
@pytest.mark.parametrize("uses", ["y", "h", "both"])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_is_differentiable(T, H, uses, residual):
    if uses != "y" and not residual:
        return  # h is x itself
    g = torch.Generator("cuda").manual_seed(T)
    leaves = [torch.randn(T, H, generator=g, device="cuda"), torch.rand(H, generator=g, device="cuda") + 0.5]
    if residual:
        leaves.append(torch.randn(T, H, generator=g, device="cuda"))
    a, b = torch.randn(T, H, generator=g, device="cuda"), torch.randn(T, H, generator=g, device="cuda")
    mine = [t.clone().requires_grad_() for t in leaves]
    ref = [t.double().requires_grad_() for t in leaves]
    for f, ts, c, d in ((se.norm, mine, a, b), (norm64, ref, a.double(), b.double())):
        y, h = f(ts[0], ts[1], ts[2] if residual else None)
        loss = 0
        if uses in ("y", "both"):
            loss = loss + (y * c).sum()
        if uses in ("h", "both"):
            loss = loss + (h * d).sum()
        loss.backward()
    for m, r in zip(mine, ref):
        if r.grad is None:
            assert m.grad is None
        else:
            assert float((m.grad.double() - r.grad).norm()) <= 1e-5 * float(r.grad.norm())


def test_norm_types_strides_and_refusals():
    x = torch.randn(64, 40, device="cuda").to(BF16).t()  # not dense
    gamma = (torch.rand(64, device="cuda") + 0.5).to(BF16).requires_grad_()
    y, h = se.norm(x, gamma, x)
    (y.float().square().sum() + h.float().sum()).backward()
    assert gamma.grad.dtype == BF16 and y.dtype == BF16 and torch.equal(h, (x.float() * 2).to(BF16))
    with pytest.raises(ValueError, match="residual"):
        se.norm(x, gamma, x.float())
    with pytest.raises(ValueError, match="residual"):
        se.norm(x, gamma, x[:10])
    with pytest.raises(ValueError, match="gamma"):
        se.norm(x, gamma[:10], x)


def test_a_penalty_on_the_norms_gradient_raises():
    x = torch.randn(4, 32, device="cuda", requires_grad=True)
    y, _ = se.norm(x, torch.ones(32, device="cuda"))
    (grad,) = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grad.square().sum().backward()


def test_training_step_with_the_norm():
    T, k, E, H, I = 90, 3, 8, 136, 72
    gate, up, down = weights(E, H, I)
    logits, ids = routed(T, k, E, 0.2)
    x, stream, gamma = torch.randn(T, H, device="cuda"), torch.randn(T, H, device="cuda"), torch.rand(H, device="cuda") + 0.5
    c = torch.randn(T, H, device="cuda")
    s = se.sort_tokens(ids, E)
    ends = s.offsets.tolist()
    leaves = (x, stream, gamma, gate, up, down, logits)
    mine = [t.clone().requires_grad_() for t in leaves]
    y, h = se.norm(mine[0], mine[2], mine[1])
    xs, rows = se.dispatch(y, s), []
    for e in range(E):
        r = xs[ends[e]:ends[e + 1]]
        rows.append((torch.nn.functional.silu(r @ mine[3][e].T) * (r @ mine[4][e].T)) @ mine[5][e].T)
    out = h + se.combine(torch.cat(rows + [xs[ends[E]:]]), se.router_weights(mine[6], ids), s)
    (out * c).sum().backward()

    ref = [t.double().requires_grad_() for t in leaves]
    y, h = norm64(ref[0], ref[2], ref[1])
    kept = ids >= 0
    sp = torch.nn.functional.softplus(ref[6].gather(1, ids.long().clamp(min=0)), threshold=1e9).sqrt() * kept
    w = se.W_SCALE * sp / sp.sum(1, keepdim=True).clamp(min=1e-300)
    out = h
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        f = torch.nn.functional.silu(y[t] @ ref[3][e].T) * (y[t] @ ref[4][e].T)
        out = out.index_add(0, t, (f @ ref[5][e].T) * w[t, j, None])
    (out * c.double()).sum().backward()
    for a, b in zip(mine, ref):
        assert float((a.grad.double() - b.grad).norm()) <= 1e-5 * float(b.grad.norm())


# ------------------------------------------------------------ calls in a row --
@pytest.mark.parametrize("T,k,E,K,I", [(1, 1, 4, 128, 64), (3, 2, 4, 128, 64), (40, 3, 8, 256, 128), (700, 4, 6, 512, 256), (30, 2, 4, 96, 32)])
@pytest.mark.parametrize("fmt", FMTS)
def test_chain_of_calls(T, k, E, K, I, fmt):
    """Norm, blocks, product, gated blocks, product, each step over the same buffers, captured back to
    back: the bits of the same calls made one at a time."""
    from tests.test_gpu_chained_calls import N, compare, routed as routes_of

    R, routes = T * k, routes_of(T, k, E, T)
    x, stream = torch.randn(N, T, K, device="cuda").to(BF16), torch.randn(N, T, K, device="cuda").to(BF16)
    gamma = torch.rand(K, device="cuda") + 0.5
    gate, up, down = weights(E, K, I)
    layer = se.BlockExperts(gate, up, down, fmt)
    y, h, rstd = torch.empty(T, K, dtype=BF16, device="cuda"), torch.empty(T, K, dtype=BF16, device="cuda"), torch.empty(T, device="cuda")
    q, s, g = layer.blocks(x[0])
    gu = torch.empty(R, 2 * I, dtype=BF16, device="cuda")
    hq, hs, hg = layer.blocks(gu.zero_(), gated=True)
    (wq, ws, wg), (dq, ds, dg) = layer.gate_up, layer.down

    def step(i, out, done):
        _, _, _, off, src, _ = routes[i]
        bqe.moe_norm_rows(x[i], gamma, y, 1e-6, stream[i], h, rstd)
        done()
        bqe.moe_quantize_blocks(y, q, s, g, fmt)
        done()
        bqe.moe_block_product(q, s, wq, ws, gu, off, src, k, g, wg, fmt)
        done()
        bqe.moe_quantize_blocks(gu, hq, hs, hg, fmt, gated=True)
        done()
        bqe.moe_block_product(hq, hs, dq, ds, out[0], off, None, 1, hg, dg, fmt)
        done()
        bqe.moe_norm_rows_backward(y, h, gamma, rstd, out[1], dh=stream[i])
        done()

    compare(step, lambda: [torch.empty(N, R, K, dtype=BF16, device="cuda"), torch.empty(N, T, K, dtype=BF16, device="cuda")])


def test_two_streams_at_once():
    """Products and norms that overlap share nothing."""
    T, k, E, H, I = 300, 4, 16, 512, 256
    layer = se.BlockExperts(*weights(E, H, I))
    logits, ids = routed(T, k, E, 0.0)
    s, w = se.sort_tokens(ids, E), se.router_weights(logits, ids)
    xs = [torch.randn(T, H, device="cuda").to(BF16) for _ in range(2)]
    gamma = torch.rand(H, device="cuda") + 0.5
    call = lambda x: layer(se.norm_codes(x, gamma)[0], s, w)  # noqa: E731
    want = [call(x) for x in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(20):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(call(xs[i]))
    torch.cuda.synchronize()
    bqe.moe_check_product()
    for i in (0, 1):
        assert all(torch.equal(g, want[i]) for g in got[i])


def small():
    f = lambda *n: torch.zeros(*n, device="cuda")  # noqa: E731
    u = lambda *n: torch.zeros(*n, dtype=torch.uint8, device="cuda")  # noqa: E731
    T, H, E, N = 4, 64, 3, 8
    return {"moe_norm_rows": (f(T, H), f(H), f(T, H)),
            "moe_norm_rows_backward": (f(T, H), f(T, H), f(H), f(T), f(T, H)),
            "moe_quantize_blocks": (f(T, H), u(T, H // 2), u(T, H // 16), f(T)),
            "moe_dequantize_blocks": (u(T, H // 2), u(T, H // 16), f(T, H), f(T)),
            "moe_block_product": (u(T, H // 2), u(T, H // 16), u(E, N, H // 2), u(E, N, H // 16), f(T, N),
                                  torch.zeros(E + 1, dtype=torch.int32, device="cuda"))}


@pytest.mark.parametrize("name", ["moe_norm_rows", "moe_norm_rows_backward", "moe_quantize_blocks", "moe_dequantize_blocks",
                         "moe_block_product"])
def test_tensors_of_another_device_are_refused(name, monkeypatch):
    args = small()[name]
    getattr(bqe, name)(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_cuda_getDevice", lambda: 1)
        with pytest.raises(ValueError, match="cuda:0.*current device.*cuda:1"):
            getattr(bqe, name)(*args)
        with pytest.raises(ValueError, match="cuda:0.*current device.*cuda:1"):
            getattr(bqe, name)(*args, stream=side)
    getattr(bqe, name)(*args, stream=side)
    side.synchronize()


@pytest.mark.parametrize("M", [100, 1000])
def test_a_wait_that_runs_out_is_reported(M):
    K, N = 512, 256
    q, s = torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda"), torch.zeros(M, K // 16, dtype=torch.uint8, device="cuda")
    wq, ws = torch.zeros(1, N, K // 2, dtype=torch.uint8, device="cuda"), torch.zeros(1, N, K // 16, dtype=torch.uint8, device="cuda")
    out, want = torch.empty(M, N, device="cuda"), torch.zeros(M, N, device="cuda")
    bqe.moe_block_product(q, s, wq, ws, out)
    bqe.moe_check_product()
    bqe.moe_test_stall_next_product()
    bqe.moe_block_product(q, s, wq, ws, out)
    with pytest.raises(bqe.MoeError, match="moe_block_product") as e:
        bqe.moe_check_product()
    assert e.value.status == bqe.MOE_ERR_TIMEOUT
    out.fill_(7)
    bqe.moe_block_product(q, s, wq, ws, out)
    bqe.moe_check_product()
    assert torch.equal(out, want)
