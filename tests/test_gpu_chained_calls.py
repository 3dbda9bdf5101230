"""Chains of calls over the same buffers: every kernel may start while the one in
front of it still writes what it reads, so each link is captured back to back,
many times over, with buffers that are written again at every step, and must
give the bits of the same calls made one at a time."""
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from tests.test_gpu_sorted_rows import BF16, F16, F32

pytestmark = pytest.mark.gpu
N = 24


def compare(step, outputs):
    """step(i, out) for i < N: apart and synchronised, then in one graph."""
    want, got = outputs(), outputs()
    for i in range(N):
        step(i, [o[i] for o in want], torch.cuda.synchronize)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(N):
            step(i, [o[i] for o in got], lambda: None)
    for _ in range(5):
        for o in got:
            o.fill_(7)
        graph.replay()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def routed(T, k, E, seed):
    """N routings of T tokens, sorted: lists of (logits, ids, w, offsets, row_src, row_dst)."""
    out = []
    for i in range(N):
        g = torch.Generator("cuda").manual_seed(1000 * seed + i)
        logits = torch.randn(T, E, generator=g, device="cuda")
        ids = logits.topk(k, dim=1).indices.int()
        ids[torch.rand(T, k, generator=g, device="cuda") < 0.1] = -1
        off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        src, dst = (torch.empty(T * k, dtype=torch.int32, device="cuda") for _ in range(2))
        bqe.moe_permute_noalloc(ids, E, off, src, dst)
        out.append((logits, ids, torch.rand(T, k, generator=g, device="cuda"), off, src, dst))
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("T,k,E,K,I", [(3, 2, 4, 128, 64), (40, 3, 8, 256, 128), (700, 4, 6, 512, 256), (30, 2, 4, 100, 36)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_product_then_gated_quantisation(T, k, E, K, I, dtype):
    R = T * k
    routes = routed(T, k, E, T)
    x = torch.randn(N, T, K, device="cuda")
    wq = torch.randint(-127, 128, (E, 2 * I, K), dtype=torch.int8, device="cuda")
    ws = torch.rand(E, 2 * I, device="cuda") * 1e-3 + 1e-4
    q, s = torch.empty(T, K, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    gu = torch.empty(R, 2 * I, dtype=dtype, device="cuda")

    def step(i, out, done):
        _, _, _, off, src, _ = routes[i]
        bqe.moe_quantize_rows(x[i], q, s)
        done()
        bqe.moe_expert_product(q, s, wq, ws, gu, off, src, k)
        done()
        bqe.moe_quantize_rows(gu, out[0], out[1], gated=True)
        done()

    compare(step, lambda: [torch.empty(N, R, I, dtype=torch.int8, device="cuda"), torch.empty(N, R, device="cuda")])


@pytest.mark.parametrize("T,k,E,H", [(4, 3, 8, 512), (200, 6, 32, 257), (900, 6, 64, 1024)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_combine_gradient_then_router_gradient(T, k, E, H, dtype):
    R = T * k
    routes = routed(T, k, E, T + 1)
    x = torch.randn(N, T, H, device="cuda").to(dtype)
    y, dy = (torch.empty(R, H, dtype=dtype, device="cuda") for _ in range(2))
    dout, dw = torch.empty(T, H, device="cuda"), torch.empty(T, k, device="cuda")

    def step(i, out, done):
        logits, ids, w, off, _, dst = routes[i]
        bqe.moe_dispatch(x[i], off, dst, y)          # y of this step
        done()
        bqe.moe_combine(y, w, dst, dout)             # and its dout
        done()
        bqe.moe_combine_backward(dout, y, w, off, dst, dy, dw)
        done()
        bqe.moe_route_backward(logits, ids, dw, out[0])
        done()
        bqe.moe_dispatch_backward(dy, dst, out[1])
        done()

    compare(step, lambda: [torch.empty(N, T, E, device="cuda"), torch.empty(N, T, H, dtype=dtype, device="cuda")])


@pytest.mark.parametrize("T,k,E,H", [(5, 2, 4, 256), (300, 6, 64, 512)])
def test_sort_then_dispatch_and_product(T, k, E, H):
    """The positions, sources and offsets are those of this step's sort."""
    R = T * k
    routes = routed(T, k, E, T + 2)
    x = torch.randn(T, H, device="cuda")
    q = torch.randint(-127, 128, (T, H), dtype=torch.int8, device="cuda")
    wq = torch.randint(-127, 128, (E, 64, H), dtype=torch.int8, device="cuda")
    s, ws = torch.rand(T, device="cuda"), torch.rand(E, 64, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    src, dst = (torch.empty(R, dtype=torch.int32, device="cuda") for _ in range(2))

    def step(i, out, done):
        bqe.moe_permute_noalloc(routes[i][1], E, off, src, dst)
        done()
        bqe.moe_dispatch(x, off, dst, out[0])
        done()
        bqe.moe_expert_product(q, s, wq, ws, out[1], off, src, k)
        done()

    compare(step, lambda: [torch.empty(N, R, H, device="cuda"), torch.empty(N, R, 64, device="cuda")])


@pytest.mark.parametrize("tokens", [3, 40, 300, 5000])
def test_the_layer_step_by_step(tokens):
    """Route, sort, quantisation and layer over the same ids, weights and positions;
    the layer's own buffers are written again by every call."""
    from tests import _gpu as G

    cfg = G.CONFIGS[0]
    layer = G.make_layer(cfg, G.weights_np(0), tokens)
    R = tokens * cfg.k
    g = torch.Generator("cuda").manual_seed(tokens)
    logits = torch.randn(N, tokens, cfg.E, generator=g, device="cuda")
    x = torch.randn(N, tokens, cfg.H, generator=g, device="cuda").to(BF16).view(torch.int16)
    ids, w = torch.empty(tokens, cfg.k, dtype=torch.int32, device="cuda"), torch.empty(tokens, cfg.k, device="cuda")
    off = torch.empty(cfg.E + 1, dtype=torch.int32, device="cuda")
    src, dst = (torch.empty(R, dtype=torch.int32, device="cuda") for _ in range(2))

    def step(i, out, done):
        bqe.moe_route(layer, logits[i], ids, w)
        done()
        bqe.moe_permute(layer, ids, off, src, dst)
        done()
        bqe.moe_dispatch(x[i].view(BF16), off, dst, out[0])
        done()
        bqe.moe_forward(layer, x[i], ids, w, out[1])
        done()

    compare(step, lambda: [torch.empty(N, R, cfg.H, dtype=BF16, device="cuda"),
                           torch.empty(N, tokens, cfg.H, device="cuda")])
    bqe.moe_check(layer)
    layer.close()
