"""Cases of the sorted-expert operators: dispatch, combine and the product with
8-bit integer experts, each with its plain form in 32 bits and its definition
in 64 bits.

The rows r = t * k + j of T tokens with k experts each are sorted by expert:
`offsets` [E + 1] are the experts' segments, `row_src` [R] the row at a sorted
position, `row_dst` [R] a row's sorted position (-1: the slot is empty, a
pruned expert).  Positions from offsets[E] on hold nothing.

  dispatch        xs[p] = x[row_src[p] / k], zero past offsets[E]
  dispatch_grad   dx[t] = sum_j dxs[row_dst[t, j]]
  combine         out[t] = sum_j w[t, j] y[row_dst[t, j]]
  combine_grad    dy[p] = w[r] dout[r / k] with r = row_src[p];
                  dw[t, j] = <dout[t], y[row_dst[t, j]]>; and through
                  w_j = w_scale s_j / sum_i s_i, s = sqrt(softplus(logit)):
                  dlogits[t, e_j] = (w_scale / S^2) sum_i s_i (dw_j - dw_i)
                                    sigmoid(logit_j) / (2 s_j), else 0
  product         out[p, n] = scale[r] w_scale[e, n] sum_i q[r, i] wq[e, n, i],
                  q and scale the tokens' rows in 8 bits with one scale each:
                  scale = max|x| / 127, q = round(127 x / max|x|), half to even;
                  `gated`: the rows are silu(x[:, :K]) * x[:, K:]
"""
import math

import torch

own = False

W_SCALE = 1.5
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
# The largest pass listed, in bytes and in multiplications of the product.
MOST_BYTES = 1.0e9
MOST_WEIGHTS = 256 * 4096 * 4096
MOST_MACS = 8192 * 6 * 4096 * 4096


def _rows(name, op, tokens, top_k, experts, hidden, dtype, out="", drop=0.0):
    return {"name": name, "op": op, "tokens": tokens, "top_k": top_k, "experts": experts, "hidden": hidden,
            "dtype": dtype, "out": out or dtype, "drop": drop}


def _product(name, tokens, top_k, experts, K, N, out, gated=False, spread=0.5):
    return {"name": name, "op": "product", "tokens": tokens, "top_k": top_k, "experts": experts, "K": K, "N": N,
            "dtype": "bfloat16", "out": out, "gated": gated, "spread": spread}


def listed():
    return [
        # prompt of 8192 tokens spread over the experts' segments
        _rows("dispatch 8192 bf16", "dispatch", 8192, 6, 256, 4096, "bfloat16"),
        # gradient of the spread tokens with pruned slots, an odd width, in fp32
        _rows("dispatch_grad 1501 odd fp32", "dispatch_grad", 1501, 3, 60, 1030, "float32", drop=0.25),
        # the same for the long training batch
        _rows("dispatch_grad 8192 bf16", "dispatch_grad", 8192, 6, 256, 4096, "bfloat16"),
        # one token being decoded: its six experts' rows, latency only
        _rows("combine 1 fp32", "combine", 1, 6, 256, 4096, "float32"),
        # the long prompt's experts joined, fp32 out as the layer gives it
        _rows("combine 8192 bf16", "combine", 8192, 6, 256, 4096, "bfloat16", "float32"),
        # a small training batch through the joined outputs, weights and router
        _rows("combine_grad 509 odd fp16", "combine_grad", 509, 4, 64, 2047, "float16", drop=0.2),
        # the long training batch
        _rows("combine_grad 8192 bf16", "combine_grad", 8192, 6, 256, 4096, "bfloat16"),
        # gate and up matrices of the six experts of one decoded token
        _product("product 1", 1, 6, 256, 4096, 4096, "bfloat16"),
        # down matrices of a decoded batch, after the gate
        _product("product 32 gated", 32, 6, 256, 2048, 4096, "bfloat16", gated=True),
        # a dense (shared) expert with ragged sizes, fp32 out
        _product("product 777 dense ragged fp32", 777, 1, 1, 1104, 1001, "float32"),
        # a short prompt: a dozen rows an expert, every weight read
        _product("product 500", 500, 6, 256, 4096, 4096, "bfloat16"),
        # the long prompt: nearly two hundred rows an expert
        _product("product 8192", 8192, 6, 256, 4096, 4096, "bfloat16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(n):
    return n + 16 if n == 3072 else n


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad", "product", "product"])
    tokens = _log(rng, 1, 8192)
    top_k = rng.randint(1, 8)
    experts = _log(rng, max(8, top_k), 256)
    if op != "product":
        hidden = _width(rng.choice([_log(rng, 128, 8192), 128 * rng.randint(1, 64)]))
        dtype = rng.choice(sorted(DTYPES))
        out = rng.choice([dtype, "float32"]) if op != "dispatch" else dtype
        c = _rows("", op, tokens, top_k, experts, hidden, dtype, out, rng.choice([0.0, round(rng.random() * 0.5, 3)]))
        while work(c)["bytes"] > MOST_BYTES:
            c["tokens"] //= 2
    else:
        if rng.random() < 0.3:
            top_k = experts = 1
        gated = rng.random() < 0.4
        K = _width(16 * _log(rng, 16, 256))
        N = _width(rng.choice([_log(rng, 128, 4096), 128 * rng.randint(1, 32)]))
        while experts > 8 and experts * K * N > MOST_WEIGHTS:
            experts //= 2
        while tokens > 1 and tokens * top_k * K * N > MOST_MACS:
            tokens //= 2
        out = rng.choice(["bfloat16", "float16"] + ["float32"] * (not gated))
        c = _product("", tokens, top_k, experts, K, N, out, gated, rng.choice([0.0, 0.5, 1.0]))
        c["dtype"] = rng.choice(["bfloat16", "float32"])
    del c["name"]
    return c


def work(case):
    T, k, E = case["tokens"], case["top_k"], case["experts"]
    R = T * k
    size = {"float32": 4, "bfloat16": 2, "float16": 2}
    a, o = size[case["dtype"]], size[case["out"]]
    if case["op"] == "product":
        K, N = case["K"], case["N"]
        used = E * (1.0 - (1.0 - 1.0 / E) ** R) if E > 1 else 1.0
        x = (R if case["gated"] else T) * K * a * (2 if case["gated"] else 1)
        return {"bytes": x + used * (K * N + 4 * N) + R * N * o, "flops": 2.0 * R * K * N}
    H, kept = case["hidden"], R * (1.0 - case["drop"])
    if case["op"] == "dispatch":
        return {"bytes": T * H * a + R * H * a + 4 * R, "flops": 0.0}
    if case["op"] == "dispatch_grad":
        return {"bytes": kept * H * a + T * H * o + 4 * R, "flops": kept * H}
    if case["op"] == "combine":
        return {"bytes": kept * H * a + T * H * o + 8 * R, "flops": 2.0 * kept * H}
    return {"bytes": T * H * o + kept * H * a + R * H * a + 4 * T * E + 20 * R, "flops": 3.0 * kept * H}


def _routing(case, g):
    """A router's choice of top_k experts a token, its weights, and the sort by expert; `drop` prunes the tails of that
    share of the slots, whole tokens among them."""
    T, k, E = case["tokens"], case["top_k"], case["experts"]
    R = T * k
    logits = torch.randn(T, E, generator=g, device="cuda") + case.get("spread", 0.5) * torch.randn(E, generator=g, device="cuda")
    top, ids = logits.topk(k, dim=1)
    keep = torch.rand(T, k, generator=g, device="cuda").sort(dim=1, descending=True).values >= case.get("drop", 0.0)
    keep[0, 0] = True
    s = (top.clamp(min=0) + torch.log1p(torch.exp(-top.abs()))).sqrt() * keep
    w = W_SCALE * s / s.sum(1, keepdim=True).clamp(min=1e-20)
    ids = torch.where(keep, ids, -1)
    flat = torch.where(keep, ids, E).reshape(-1)
    order = torch.argsort(flat, stable=True)
    dst = torch.empty_like(order)
    dst[order] = torch.arange(R, device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.bincount(flat, minlength=E + 1)[:E].cumsum(0)
    return {"logits": logits, "ids": ids.int(), "w": w, "offsets": offsets.int(), "row_src": order.int(),
            "row_dst": torch.where(keep.reshape(-1), dst, -1).int()}


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    T, k, E = case["tokens"], case["top_k"], case["experts"]
    R, dt = T * k, DTYPES[case["dtype"]]
    st = {"case": case}
    if case["op"] == "product":
        K, N = case["K"], case["N"]
        if E > 1:
            st.update(_routing(case, g))
            st["most"] = int(st["offsets"].diff().max())
        x = torch.randn(R if case["gated"] else T, K * (2 if case["gated"] else 1), generator=g, device="cuda")
        # a few channels of a trained model's activations are much larger than the rest
        x *= 1.0 + 7.0 * (torch.rand(x.shape[1], generator=g, device="cuda") < 0.01)
        st["x"] = x.to(dt)
        wq = torch.empty(E, N, K, dtype=torch.int8, device="cuda")
        step = max(1, (1 << 28) // (N * K))
        for e in range(0, E, step):
            part = torch.randn(min(step, E - e), N, K, generator=g, device="cuda")
            wq[e:e + step] = part.mul_(32.0).round_().clamp_(-127, 127)
        st["wq"] = wq
        st["w_scale"] = (0.5 + torch.rand(E, N, generator=g, device="cuda")) / (32.0 * math.sqrt(K))
        return st
    H, out = case["hidden"], DTYPES[case["out"]]
    st.update(_routing(case, g))
    if case["op"] == "dispatch":
        st["x"] = torch.randn(T, H, generator=g, device="cuda").to(dt)
    elif case["op"] == "dispatch_grad":
        st["dxs"] = torch.randn(R, H, generator=g, device="cuda").to(dt)
    else:
        st["y"] = torch.randn(R, H, generator=g, device="cuda").to(dt)
    if case["op"] == "combine_grad":
        st["dout"] = torch.randn(T, H, generator=g, device="cuda").to(out)
    return st


# ------------------------------------------------------------- plain forms --
def _gather(rows, dst, k):
    """The sorted rows of every token's slots [T, k, H] in 32 bits; empty slots zero."""
    at = dst.long()
    got = rows.float()[at.clamp(min=0)]
    return torch.where((at >= 0)[:, None], got, 0.0).view(-1, k, rows.shape[1])


def _quantized(x, gated):
    x = x.float()
    if gated:
        g, u = x.chunk(2, dim=1)
        x = g / (1.0 + torch.exp(-g)) * u
    most = x.abs().amax(1, keepdim=True)
    scale = most / torch.full_like(most, 127.0)  # a quotient, not a product with a rounded 1 / 127
    q = torch.where(most > 0, torch.round(x * 127.0 / most), 0.0)
    return q, scale


def _plain_product(st):
    c = st["case"]
    q, scale = _quantized(st["x"], c["gated"])
    if c["experts"] == 1:
        out = (q @ st["wq"][0].float().t()) * scale * st["w_scale"]
        return out.to(DTYPES[c["out"]])
    R, E, k = c["tokens"] * c["top_k"], c["experts"], c["top_k"]
    row = torch.arange(R, device="cuda") if c["gated"] else st["row_src"].long() // k
    offsets, p = st["offsets"].long(), torch.arange(R, device="cuda")
    expert = torch.searchsorted(offsets, p, right=True) - 1
    q, scale = q[row], scale[row]
    if R < E:  # fewer rows than experts: each with its own matrix
        out = torch.bmm(st["wq"][expert].float(), q[:, :, None])[:, :, 0]
    else:  # every expert's rows, padded to the longest segment
        slot = expert * st["most"] + p - offsets[expert]
        rows = q.new_zeros(E * st["most"], c["K"])
        rows[slot] = q
        out = torch.bmm(rows.view(E, st["most"], -1), st["wq"].float().transpose(1, 2)).view(E * st["most"], -1)[slot]
    return (out * scale * st["w_scale"][expert]).to(DTYPES[c["out"]])


def _plain(st):
    c = st["case"]
    k, out = c["top_k"], DTYPES[c["out"]]
    if c["op"] == "product":
        return _plain_product(st)
    if c["op"] == "dispatch_grad":
        return _gather(st["dxs"], st["row_dst"], k).sum(1).to(out)
    if c["op"] == "combine":
        return (_gather(st["y"], st["row_dst"], k) * st["w"][:, :, None]).sum(1).to(out)
    placed = (torch.arange(st["row_src"].shape[0], device="cuda") < st["offsets"][-1])[:, None]
    src = st["row_src"].long()
    if c["op"] == "dispatch":
        return torch.where(placed, st["x"][src // k], 0.0)
    dout = st["dout"].float()
    dy = torch.where(placed, st["w"].reshape(-1)[src][:, None] * dout[src // k], 0.0).to(st["y"].dtype)
    dw = (_gather(st["y"], st["row_dst"], k) * dout[:, None, :]).sum(2)
    return {"dy": dy, "dw": dw, "dlogits": _route_grad(st["logits"], st["ids"], dw)}


def _route_grad(logits, ids, dw):
    kept = ids >= 0
    at = ids.long().clamp(min=0)
    l = logits.gather(1, at)
    s = (l.clamp(min=0) + torch.log1p(torch.exp(-l.abs()))).sqrt()
    total = torch.where(kept, s, 0.0).sum(1, keepdim=True)
    total = torch.where(total > 0, total, 1.0)
    s_kept = torch.where(kept, s, 0.0)
    against = (s_kept[:, None, :] * (dw[:, :, None] - dw[:, None, :])).sum(2)  # sum_i s_i (dw_j - dw_i)
    d = W_SCALE / total / total * against / (1.0 + torch.exp(-l)) / (2.0 * s)
    return torch.zeros_like(logits).scatter_add_(1, at, torch.where(kept, d, 0.0))


# ------------------------------------------------- the framework's operators --
def _framework(st):
    import block_quantized_expert_gb300 as bqe

    c = st["case"]
    T, k, out = c["tokens"], c["top_k"], DTYPES[c["out"]]
    if c["op"] == "product":
        x, K = st["x"], c["K"]
        q = torch.empty(x.shape[0], K, dtype=torch.int8, device="cuda")
        scale = torch.empty(x.shape[0], dtype=torch.float32, device="cuda")
        res = torch.empty(T * k, c["N"], dtype=out, device="cuda")
        bqe.moe_quantize_rows(x, q, scale, gated=c["gated"])
        if c["experts"] == 1:
            bqe.moe_expert_product(q, scale, st["wq"], st["w_scale"], res)
        elif c["gated"]:
            bqe.moe_expert_product(q, scale, st["wq"], st["w_scale"], res, st["offsets"])
        else:
            bqe.moe_expert_product(q, scale, st["wq"], st["w_scale"], res, st["offsets"], st["row_src"], k)
        return res
    H = c["hidden"]
    if c["op"] == "dispatch":
        xs = torch.empty(T * k, H, dtype=out, device="cuda")
        bqe.moe_dispatch(st["x"], st["offsets"], st["row_dst"], xs)
        return xs
    if c["op"] == "dispatch_grad":
        dx = torch.empty(T, H, dtype=out, device="cuda")
        bqe.moe_dispatch_backward(st["dxs"], st["row_dst"], dx)
        return dx
    if c["op"] == "combine":
        res = torch.empty(T, H, dtype=out, device="cuda")
        bqe.moe_combine(st["y"], st["w"], st["row_dst"], res)
        return res
    dy, dw, dlogits = torch.empty_like(st["y"]), torch.empty_like(st["w"]), torch.empty_like(st["logits"])
    bqe.moe_combine_backward(st["dout"], st["y"], st["w"], st["offsets"], st["row_dst"], dy, dw)
    bqe.moe_route_backward(st["logits"], st["ids"], dw, dlogits, W_SCALE)
    return {"dy": dy, "dw": dw, "dlogits": dlogits}


def run(state):
    return _framework(state) if own else _plain(state)


# --------------------------------------------------------- definition, 64 bits --
def _exact_product(st):
    c = st["case"]
    k, E = c["top_k"], c["experts"]
    x = st["x"].double()
    if c["gated"]:
        x = x[:, :c["K"]] * torch.sigmoid(x[:, :c["K"]]) * x[:, c["K"]:]
    most = x.abs().max(dim=1).values
    scale, q = most / 127, torch.round(x * 127 / most.clamp(min=1e-300)[:, None])
    ends = st["offsets"].tolist() if E > 1 else [0, c["tokens"]]
    src = st["row_src"].long() // k if E > 1 and not c["gated"] else torch.arange(c["tokens"] * k, device="cuda")
    out = torch.zeros(c["tokens"] * k, c["N"], dtype=torch.float64, device="cuda")
    for e in range(E):
        rows = src[ends[e]:ends[e + 1]]
        if len(rows):
            dots = q[rows] @ st["wq"][e].double().T
            out[ends[e]:ends[e + 1]] = dots * st["w_scale"][e].double() * scale[rows][:, None]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "product":
        return _exact_product(st)
    T, k = case["tokens"], case["top_k"]
    dst = st["row_dst"].long().view(T, k)
    live = dst >= 0
    rows = dst[live]                              # sorted positions that hold a row
    token = live.nonzero()[:, 0]                  # and the tokens they come from
    if case["op"] == "dispatch":
        xs = torch.zeros(T * k, case["hidden"], dtype=torch.float64, device="cuda")
        xs[rows] = st["x"][token].double()
        return xs
    out = torch.zeros(T, case["hidden"], dtype=torch.float64, device="cuda")
    if case["op"] in ("dispatch_grad", "combine"):
        val = st["dxs" if case["op"] == "dispatch_grad" else "y"].double()
        for j in range(k):
            on = live[:, j]
            f = st["w"][on, j].double()[:, None] if case["op"] == "combine" else 1.0
            out[on] += f * val[dst[on, j]]
        return out
    dout = st["dout"].double()
    dy = torch.zeros(T * k, case["hidden"], dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        on = live[:, j]
        dy[dst[on, j]] = st["w"][on, j].double()[:, None] * dout[on]
        dw[on, j] = (dout[on] * st["y"][dst[on, j]].double()).sum(1)
    # dw_j / dl_i of w_j = w_scale s_j / S over the kept slots, times dw_j, summed
    l = st["logits"].double()
    s = (torch.logaddexp(l, torch.zeros_like(l)).sqrt()).gather(1, st["ids"].long().clamp(min=0)) * live
    slope = torch.sigmoid(l).gather(1, st["ids"].long().clamp(min=0)) / (2 * s.clamp(min=1e-300))
    dlogits = torch.zeros_like(l)
    for j in range(k):
        on = live[:, j]
        ds = sum(s[on, i] * (dw[on, j] - dw[on, i]) * live[on, i] for i in range(k) if i != j) + torch.zeros_like(s[on, j])
        dlogits[on, st["ids"][on, j].long()] = W_SCALE * ds * slope[on, j] / s[on].sum(1) ** 2
    return {"dy": dy, "dw": dw, "dlogits": dlogits}
