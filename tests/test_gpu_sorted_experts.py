"""The sorted-row operators together: the 8-bit expert layer against its
definition in 64 bits on its own codes, and a training step's gradients against
autograd in 64 bits.

Tolerances.  The layer's codes of x are compared exactly by using them; gu and y are
rounded to bf16 (2^-8 of a value, independent over thousands of them), and a
code of h moves by at most one step of 1/127 of its row's maximum where gu's
rounding crosses a boundary: relative L2 below 2^-8 + 1/127.  The gradients run
in fp32 through sums of at most a few thousand terms: relative L2 below 1e-5.
"""
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from block_quantized_expert_gb300 import sorted_experts as se

pytestmark = pytest.mark.gpu


def weights(E, H, I):
    g = torch.Generator("cuda").manual_seed(5)
    gate, up = (torch.randn(E, I, H, generator=g, device="cuda") / H ** 0.5 for _ in range(2))
    return gate, up, torch.randn(E, H, I, generator=g, device="cuda") / I ** 0.5


def routed(T, k, E, drop):
    g = torch.Generator("cuda").manual_seed(T)
    logits = torch.randn(T, E, generator=g, device="cuda")
    ids = logits.topk(k, dim=1).indices.int()
    keep = torch.rand(T, k, generator=g, device="cuda").sort(dim=1, descending=True).values >= drop
    return logits, torch.where(keep, ids, -1)


@pytest.mark.parametrize("T,k,E,H,I,drop", [(1, 6, 64, 1024, 512, 0.0), (33, 4, 16, 256, 128, 0.3), (700, 6, 24, 512, 272, 0.1)])
def test_int8_layer(T, k, E, H, I, drop):
    gate, up, down = weights(E, H, I)
    layer = se.Int8Experts(gate, up, down)
    logits, ids = routed(T, k, E, drop)
    s = se.sort_tokens(ids, E)
    w = se.router_weights(logits, ids)
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    got = layer(x, s, w)
    bqe.moe_check_product()
    q, scale = torch.empty(T, H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    bqe.moe_quantize_rows(x, q, scale)
    x64 = q.double() * scale.double()[:, None]
    gu64 = layer.gate_up.double() * layer.gate_up_scale.double()[:, :, None]
    d64 = layer.down.double() * layer.down_scale.double()[:, :, None]
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if e >= 0:
                gu = gu64[e] @ x64[t]
                h = torch.nn.functional.silu(gu[:I]) * gu[I:]
                m = h.abs().max()
                want[t] += w[t, j].double() * (d64[e] @ (torch.round(127 * h / m) * m / 127))
    assert float((got.double() - want).norm()) <= (2.0 ** -8 + 1 / 127) * float(want.norm())
    assert not got[(ids < 0).all(1)].any()


def test_training_step_gradients():
    T, k, E, H, I = 90, 3, 8, 136, 72
    gate, up, down = weights(E, H, I)
    logits, ids = routed(T, k, E, 0.2)
    x = torch.randn(T, H, device="cuda")
    s = se.sort_tokens(ids, E)
    ends = s.offsets.tolist()

    mine = [t.clone().requires_grad_() for t in (x, gate, up, down, logits)]
    xs, rows = se.dispatch(mine[0], s), []
    for e in range(E):
        r = xs[ends[e]:ends[e + 1]]
        rows.append((torch.nn.functional.silu(r @ mine[1][e].T) * (r @ mine[2][e].T)) @ mine[3][e].T)
    y = torch.cat(rows + [xs[ends[E]:]])
    g = torch.randn(T, H, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    (se.combine(y, se.router_weights(mine[4], ids), s) * g).sum().backward()

    ref = [t.double().clone().requires_grad_() for t in (x, gate, up, down, logits)]
    kept = ids >= 0
    sp = torch.nn.functional.softplus(ref[4].gather(1, ids.long().clamp(min=0)), threshold=1e9).sqrt() * kept
    w = se.W_SCALE * sp / sp.sum(1, keepdim=True).clamp(min=1e-300)
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        h = torch.nn.functional.silu(ref[0][t] @ ref[1][e].T) * (ref[0][t] @ ref[2][e].T)
        out = out.index_add(0, t, (h @ ref[3][e].T) * w[t, j, None])
    (out * g.double()).sum().backward()
    for a, b in zip(mine, ref):
        assert float((a.grad.double() - b.grad).norm()) <= 1e-5 * float(b.grad.norm())
