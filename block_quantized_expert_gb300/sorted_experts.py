"""Experts of the caller's own around the sorted-row operators: a served expert
layer with 8-bit integer weights, and the pieces of a training step.

The layer of moe_create holds 4-bit experts and only runs forward.  This module
is the same path (route, sort, SwiGLU experts, combine: "DeepSeek-V4-Flash 284B -
Deep-Dive Mathematical & Kernel Guide", sections 1 to 4) for experts it does not
hold:

* Int8Experts: per-channel 8-bit weights, tokens quantised per row.  A call is
  five operators: moe_quantize_rows on the tokens, moe_expert_product (gate and
  up in one, each sorted position gathering its token), moe_quantize_rows with the
  gate, moe_expert_product (down), moe_combine.
* dispatch, combine and router_weights: differentiable forms of moe_dispatch,
  moe_combine and the router's weights, for products that run in between.  They
  are differentiable once: a gradient of their gradient raises.

    python -m block_quantized_expert_gb300.sorted_experts

runs both on random weights and prints how far they are from plain PyTorch.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch
from torch.autograd.function import once_differentiable

import block_quantized_expert_gb300 as bqe

W_SCALE = 1.5


@dataclass
class Sorted:
    """A routing in the experts' order: what moe_permute gives, with the ids."""
    ids: torch.Tensor       # int32 [T][k], -1: empty slot
    offsets: torch.Tensor   # int32 [E + 1]
    row_src: torch.Tensor   # int32 [T * k], unset from offsets[E] on
    row_dst: torch.Tensor   # int32 [T * k]


def sort_tokens(ids: torch.Tensor, n_experts: int) -> Sorted:
    """The stable sort of the (token, expert) rows, at most 2^20 of them, on the
    current stream.  Each call has its own scratch."""
    T, k = ids.shape
    new = lambda n: torch.empty(n, dtype=torch.int32, device=ids.device)  # noqa: E731
    s = Sorted(ids, new(n_experts + 1), new(T * k), new(T * k))
    scratch = torch.empty(bqe.moe_permute_scratch_bytes(T, k, n_experts), dtype=torch.uint8, device=ids.device)
    bqe.moe_permute_scratch(ids, n_experts, s.offsets, s.row_src, s.row_dst, scratch)
    return s


def quantize_weights(w: torch.Tensor):
    """[E][N][K] weights to int8 with one scale an output channel."""
    E, N, K = w.shape
    wq = torch.empty((E, N, K), dtype=torch.int8, device=w.device)
    scale = torch.empty((E, N), dtype=torch.float32, device=w.device)
    bqe.moe_quantize_rows(w.reshape(E * N, K), wq.view(E * N, K), scale.view(E * N))
    return wq, scale


class Int8Experts:
    """SwiGLU experts with 8-bit integer weights: gate and up [E][I][H], down [E][H][I].

    `rows` is the type of the rows between the products (gate and up, and the experts'
    outputs before they are combined).  bf16, the default, halves their traffic against
    fp32, and its rounding (2^-9 of a value) is below a code's half step (1/254 of a
    row's maximum); fp32 leaves the codes as the only rounding.
    """

    def __init__(self, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor, rows: torch.dtype = torch.bfloat16):
        if rows not in (torch.float32, torch.bfloat16, torch.float16):
            raise ValueError(f"rows must be float32, bfloat16 or float16, got {rows}")
        self.rows = rows
        self.E, self.I, self.H = gate.shape
        self.gate_up, self.gate_up_scale = quantize_weights(torch.cat([gate, up], dim=1))
        self.down, self.down_scale = quantize_weights(down)

    def __call__(self, x: torch.Tensor, s: Sorted, w: torch.Tensor) -> torch.Tensor:
        """x [T][H] in bf16, fp16 or fp32; w [T][k] the routing weights; fp32 [T][H].

        Asynchronous: whether a device-side wait of the products ran out, which leaves
        the output undefined, is what moe_check_product tells, and the caller asks it."""
        T, k = w.shape
        R, dev = T * k, x.device
        q = torch.empty((T, self.H), dtype=torch.int8, device=dev)
        scale = torch.empty(T, dtype=torch.float32, device=dev)
        gu = torch.empty((R, 2 * self.I), dtype=self.rows, device=dev)
        h = torch.empty((R, self.I), dtype=torch.int8, device=dev)
        h_scale = torch.empty(R, dtype=torch.float32, device=dev)
        y = torch.empty((R, self.H), dtype=self.rows, device=dev)
        out = torch.empty((T, self.H), dtype=torch.float32, device=dev)
        bqe.moe_quantize_rows(x, q, scale)
        bqe.moe_expert_product(q, scale, self.gate_up, self.gate_up_scale, gu, s.offsets, s.row_src, k)
        bqe.moe_quantize_rows(gu, h, h_scale, gated=True)
        bqe.moe_expert_product(h, h_scale, self.down, self.down_scale, y, s.offsets)
        bqe.moe_combine(y, w, s.row_dst, out)
        return out


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, offsets, row_dst):
        ctx.save_for_backward(row_dst)
        ctx.T = x.shape[0]
        xs = torch.empty((row_dst.numel(), x.shape[1]), dtype=x.dtype, device=x.device)
        bqe.moe_dispatch(x, offsets, row_dst, xs)
        return xs

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs):
        (row_dst,) = ctx.saved_tensors
        dx = torch.empty((ctx.T, dxs.shape[1]), dtype=dxs.dtype, device=dxs.device)
        bqe.moe_dispatch_backward(dxs.contiguous(), row_dst, dx)
        return dx, None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, w, offsets, row_dst):
        ctx.save_for_backward(y, w, offsets, row_dst)
        out = torch.empty((w.shape[0], y.shape[1]), dtype=torch.float32, device=y.device)
        bqe.moe_combine(y, w, row_dst, out)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        y, w, offsets, row_dst = ctx.saved_tensors
        dy, dw = torch.empty_like(y), torch.empty_like(w)
        bqe.moe_combine_backward(dout.contiguous(), y, w, offsets, row_dst, dy, dw)
        return dy, dw, None, None


class _RouterWeights(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, w_scale):
        ctx.save_for_backward(logits, ids)
        ctx.w_scale = w_scale
        kept = (ids >= 0) & (ids < logits.shape[1])  # the others are empty slots, whose logits are not read
        l = logits.gather(1, torch.where(kept, ids, 0).long())
        # as in moe_route_backward: below -17 s is exp(l / 2) to fp32's rounding, and 0 below -174
        s = torch.where(l < -17.0, torch.exp(0.5 * l), (l.clamp(min=0) + torch.log1p(torch.exp(-l.abs()))).sqrt())
        s = torch.where(kept & ~(l < -174.0), s, 0.0)
        total = s.sum(1, keepdim=True)
        return w_scale * (s / torch.where(total == 0, 1.0, total))

    @staticmethod
    @once_differentiable
    def backward(ctx, dw):
        logits, ids = ctx.saved_tensors
        dlogits = torch.empty_like(logits)
        bqe.moe_route_backward(logits, ids, dw.contiguous(), dlogits, ctx.w_scale)
        return dlogits, None, None


def dispatch(x: torch.Tensor, s: Sorted) -> torch.Tensor:
    """[T][H] tokens to the [T * k][H] sorted rows; differentiable in x."""
    return _Dispatch.apply(x, s.offsets, s.row_dst)


def combine(y: torch.Tensor, w: torch.Tensor, s: Sorted) -> torch.Tensor:
    """Sorted rows back to [T][H] with the weights [T][k]; differentiable in y and w."""
    return _Combine.apply(y, w, s.offsets, s.row_dst)


def router_weights(logits: torch.Tensor, ids: torch.Tensor, w_scale: float = W_SCALE) -> torch.Tensor:
    """The weights [T][k] of moe_route, in fp32, for logits [T][E] of any floating type
    and whole-number ids [T][k]; differentiable in the logits.  Ids outside [0, E)
    are empty slots with weight 0.  A logit below -174 counts as
    weight 0.  (moe_route itself takes exp(l), which loses bits below l = -87 and
    is 0 below -104.)"""
    if logits.dim() != 2 or not logits.is_floating_point():
        raise ValueError(f"logits must be a 2-D floating tensor, got {logits.dtype} {tuple(logits.shape)}")
    if ids.dim() != 2 or ids.shape[0] != logits.shape[0] or ids.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"ids must be int32 or int64 of shape ({logits.shape[0]}, top_k), got {ids.dtype} {tuple(ids.shape)}")
    if not 1 <= ids.shape[1] <= min(8, logits.shape[1]):
        raise ValueError(f"top_k must be in [1, 8] and at most the number of experts, got {ids.shape[1]}")
    if ids.dtype == torch.int64:  # an id past 32 bits is an empty slot, not what its low bits say
        ids = torch.where((ids >= 0) & (ids < logits.shape[1]), ids, -1).int()
    return _RouterWeights.apply(logits.float().contiguous(), ids.contiguous(), w_scale)


def _example() -> None:
    torch.manual_seed(0)
    T, k, E, H, I = 512, 6, 64, 1024, 512
    dev = "cuda"
    logits = torch.randn(T, E, device=dev)
    ids = logits.topk(k, dim=1).indices.int()
    s = sort_tokens(ids, E)
    gate, up = (torch.randn(E, I, H, device=dev) / H ** 0.5 for _ in range(2))
    down = torch.randn(E, H, I, device=dev) / I ** 0.5
    x = torch.randn(T, H, device=dev)

    def plain(x, gate, up, down, logits):
        sp = torch.nn.functional.softplus(logits.gather(1, ids.long())).sqrt()
        w = W_SCALE * sp / sp.sum(1, keepdim=True)
        out = torch.zeros_like(x)
        for e in range(E):
            t, j = (ids == e).nonzero(as_tuple=True)
            h = torch.nn.functional.silu(x[t] @ gate[e].T) * (x[t] @ up[e].T)
            out = out.index_add(0, t, (h @ down[e].T) * w[t, j, None])
        return out

    want = plain(x, gate, up, down, logits)
    got = Int8Experts(gate, up, down)(x, s, router_weights(logits, ids))
    bqe.moe_check_product()
    print("8-bit experts: relative L2 distance from fp32 experts %.2e" % ((got - want).norm() / want.norm()).item())

    leaves = [t.clone().requires_grad_() for t in (x, gate, up, down, logits)]
    plain(*leaves).square().sum().backward()
    mine = [t.clone().requires_grad_() for t in (x, gate, up, down, logits)]
    xs, rows = dispatch(mine[0], s), []
    ends = s.offsets.tolist()
    for e in range(E):
        r = xs[ends[e]:ends[e + 1]]
        h = torch.nn.functional.silu(r @ mine[1][e].T) * (r @ mine[2][e].T)
        rows.append(h @ mine[3][e].T)
    combine(torch.cat(rows), router_weights(mine[4], ids), s).square().sum().backward()
    for name, a, b in zip(("x", "gate", "up", "down", "logits"), mine, leaves):
        print("training step: d%-6s relative L2 distance %.2e" % (name, ((a.grad - b.grad).norm() / b.grad.norm()).item()))


if __name__ == "__main__":
    _example()
