"""Cases of the operators around the experts in 4 bits: the norm in front of them
with the residual's addition, its gradient, rows to blocks of 4 bits and back, and
the product of such rows with experts in 4 bits; each with its plain form in 32
bits and its definition in 64 bits.

  norm       h = x + residual, held in the rows' type (x itself without a residual);
             rstd = 1 / sqrt(mean h^2 + eps); y = h rstd gamma, in the rows' type;
             `codes`: y also in 8 bits with one scale a row (scale = max|y| / 127,
             q = round(127 y / max|y|), half to even), on which the shared
             expert's 8-bit integer matrix works
  norm_grad  from dy and, where the residual goes on, dh: with g = dy gamma
             dx = dh + rstd (g - h rstd^2 mean(g h)),  dgamma = sum_t dy h rstd
  requantize rows to 4 bits and back, as a training step that minds the rounding
             sees its weights
  product    out[p, n] = scale[r] w_scale[e, n] sum_i v[r, i] w[e, n, i] over the
             positions p of expert e's segment, v and w being block values; the rows
             are the tokens' (r = row_src[p] / k), or `gated`: silu(x[:, :K]) * x[:, K:]

Blocks: e2m1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two codes a
byte, the even element low, times a scale for each
  mxfp4      32 elements, 2^(floor(log2 max) - 2)
  nvfp4      16 elements, e4m3 of max / 6 / scale; element = value * e4m3 * scale
             with scale the least power of two from (the row's max) / 2688 up, so that
             no e4m3 passes 448 and dividing by it rounds nothing
both rounded to nearest, half to even, up to 6.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
SIZE = {"float32": 4, "bfloat16": 2, "float16": 2}
BLOCK = {"mxfp4": 32, "nvfp4": 16}
# The largest pass listed, in bytes and in multiplications of the product.
MOST_BYTES = 1.2e9
MOST_WEIGHTS = 256 * 4096 * 4096
MOST_MACS = 8192 * 6 * 4096 * 4096


def _norm(name, op, tokens, hidden, dtype, residual=True, codes=0):
    return {"name": name, "op": op, "tokens": tokens, "hidden": hidden, "dtype": dtype, "residual": residual, "codes": codes}


def _requantize(name, rows, K, dtype, form):
    return {"name": name, "op": "requantize", "rows": rows, "K": K, "dtype": dtype, "form": form}


def _product(name, tokens, top_k, experts, K, N, form, out, gated=False, spread=0.5):
    return {"name": name, "op": "product", "tokens": tokens, "top_k": top_k, "experts": experts, "K": K, "N": N,
            "form": form, "dtype": "bfloat16", "out": out, "gated": gated, "spread": spread}


def listed():
    return [
        # one token being decoded, in front of the shared expert's 8-bit gate and up: latency
        _norm("norm 1 codes bf16", "norm", 1, 4096, "bfloat16", codes=4096),
        # a training batch of an odd width in fp32, first layer (no residual yet)
        _norm("norm 1501 odd fp32", "norm", 1501, 1030, "float32", residual=False),
        # the long prompt
        _norm("norm 8192 bf16", "norm", 8192, 4096, "bfloat16"),
        # a small training batch
        _norm("norm_grad 509 odd fp16", "norm_grad", 509, 2047, "float16"),
        # the long training batch
        _norm("norm_grad 8192 bf16", "norm_grad", 8192, 4096, "bfloat16"),
        # one expert's down matrix with ragged sizes, from fp32 master weights
        _requantize("requantize 777 ragged fp32", 777, 1056, "float32", "mxfp4"),
        # gate and up matrices of 16 experts
        _requantize("requantize 65536 bf16", 65536, 4096, "bfloat16", "nvfp4"),
        # gate and up matrices of the six experts of one decoded token
        _product("product 1 nvfp4", 1, 6, 256, 4096, 4096, "nvfp4", "bfloat16"),
        # down matrices of a decoded batch, after the gate
        _product("product 32 gated mxfp4", 32, 6, 256, 2048, 4096, "mxfp4", "bfloat16", gated=True),
        # a dense (shared) expert with ragged sizes, fp32 out
        _product("product 777 dense ragged", 777, 1, 1, 1120, 1001, "nvfp4", "float32"),
        # a short prompt: a dozen rows an expert, every weight read
        _product("product 500 mxfp4", 500, 6, 256, 4096, 4096, "mxfp4", "bfloat16"),
        # the long prompt: nearly two hundred rows an expert
        _product("product 8192 nvfp4", 8192, 6, 256, 4096, 4096, "nvfp4", "bfloat16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "requantize", "product", "product"])
    dtype = rng.choice(sorted(DTYPES))
    form = rng.choice(sorted(BLOCK))
    tokens = _log(rng, 1, 8192)
    if op in ("norm", "norm_grad"):
        hidden = rng.choice([_log(rng, 128, 8192), 128 * rng.randint(1, 64)])
        codes = rng.choice([0, 128 * rng.randint(1, 32)]) if op == "norm" else 0
        c = _norm("", op, tokens, hidden, dtype, rng.random() < 0.7, codes)
        while work(c)["bytes"] > MOST_BYTES or work(c)["flops"] > 2 * MOST_MACS:
            c["tokens"] //= 2
    elif op == "requantize":
        c = _requantize("", _log(rng, 1, 131072), 32 * _log(rng, 1, 256), dtype, form)
        while work(c)["bytes"] > MOST_BYTES:
            c["rows"] //= 2
    else:
        top_k = rng.randint(1, 8)
        experts = _log(rng, max(8, top_k), 256)
        if rng.random() < 0.3:
            top_k = experts = 1
        gated = rng.random() < 0.4
        K = 32 * _log(rng, 8, 128)
        N = rng.choice([_log(rng, 128, 4096), 128 * rng.randint(1, 32)])
        while experts > 8 and experts * K * N > MOST_WEIGHTS:
            experts //= 2
        while tokens > 1 and tokens * top_k * K * N > MOST_MACS:
            tokens //= 2
        out = rng.choice(["bfloat16", "float16"] + ["float32"] * (not gated))
        c = _product("", tokens, top_k, experts, K, N, form, out, gated, rng.choice([0.0, 0.5, 1.0]))
        c["dtype"] = rng.choice(["bfloat16", "float32"])
    del c["name"]
    return c


def work(case):
    a = SIZE[case["dtype"]]
    if case["op"] == "product":
        T, k, E, K, N = case["tokens"], case["top_k"], case["experts"], case["K"], case["N"]
        R = T * k
        used = E * (1.0 - (1.0 - 1.0 / E) ** R) if E > 1 else 1.0
        x = (R if case["gated"] else T) * K * a * (2 if case["gated"] else 1)
        return {"bytes": x + used * N * (K / 2 + K / BLOCK[case["form"]] + 4 * (case["form"] == "nvfp4")) + R * N * SIZE[case["out"]],
                "flops": 2.0 * R * K * N}
    if case["op"] == "requantize":
        n = case["rows"] * case["K"]
        return {"bytes": n * (2 * a + 0.5 + 1 / BLOCK[case["form"]]) + 4 * case["rows"] * (case["form"] == "nvfp4"), "flops": 0.0}
    T, H, N = case["tokens"], case["hidden"], case["codes"]
    if case["op"] == "norm":
        codes = T * (H + 4 + N * a) + N * (H + 4) if N else 0
        return {"bytes": T * H * a * (4 if case["residual"] else 2) + 4 * H + 4 * T + codes, "flops": 4.0 * T * H + 2.0 * T * H * N}
    return {"bytes": T * H * a * (4 if case["residual"] else 3) + 8 * H + 4 * T, "flops": 8.0 * T * H}


def _routing(case, g):
    """A router's choice of top_k experts a token and the sort of the rows t * top_k + j by expert."""
    T, k, E = case["tokens"], case["top_k"], case["experts"]
    logits = torch.randn(T, E, generator=g, device="cuda") + case["spread"] * torch.randn(E, generator=g, device="cuda")
    flat = logits.topk(k, dim=1).indices.reshape(-1)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.bincount(flat, minlength=E).cumsum(0)
    return {"offsets": offsets.int(), "row_src": torch.argsort(flat, stable=True).int(), "most": int(offsets.diff().max())}


def _rows(g, rows, width, dtype):
    """A trained model's activations: a few channels are much larger than the rest."""
    x = torch.randn(rows, width, generator=g, device="cuda")
    return (x * (1.0 + 7.0 * (torch.rand(width, generator=g, device="cuda") < 0.01))).to(DTYPES[dtype])


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    st = {"case": case}
    if case["op"] == "requantize":
        w = torch.randn(case["rows"], case["K"], generator=g, device="cuda") / math.sqrt(case["K"])
        st["x"] = (w * (0.5 + torch.rand(case["rows"], 1, generator=g, device="cuda"))).to(DTYPES[case["dtype"]])
        return st
    if case["op"] == "product":
        T, k, E, K, N = case["tokens"], case["top_k"], case["experts"], case["K"], case["N"]
        if E > 1:
            st.update(_routing(case, g))
        st["x"] = _rows(g, T * k if case["gated"] else T, K * (2 if case["gated"] else 1), case["dtype"])
        wq = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
        ws = torch.empty(E, N, K // BLOCK[case["form"]], dtype=torch.uint8, device="cuda")
        wg = torch.ones(E, N, device="cuda")
        step = max(1, (1 << 28) // (N * K))
        for e in range(0, E, step):
            n = min(step, E - e)
            part = torch.randn(n * N, K, generator=g, device="cuda") / math.sqrt(K)
            part *= 0.5 + torch.rand(n * N, 1, generator=g, device="cuda")
            v, s, scale = _blocks(part, case["form"])
            wq[e:e + n], ws[e:e + n] = _codes(v).view(n, N, -1), _scale_bytes(s, case["form"]).view(n, N, -1)
            if scale is not None:
                wg[e:e + n] = scale.view(n, N)
        st.update(wq=wq, ws=ws, w_scale=wg if case["form"] == "nvfp4" else None)
        return st
    T, H, N, dt = case["tokens"], case["hidden"], case["codes"], DTYPES[case["dtype"]]
    st["gamma"] = 0.5 + torch.rand(H, generator=g, device="cuda")
    x = _rows(g, T, H, case["dtype"])
    residual = (4.0 * torch.randn(T, H, generator=g, device="cuda")).to(dt) if case["residual"] else None
    if case["op"] == "norm":
        st.update(x=x, residual=residual)
        if N:
            st["wq"] = (32.0 * torch.randn(1, N, H, generator=g, device="cuda")).round_().clamp_(-127, 127).to(torch.int8)
            st["w_scale"] = (0.5 + torch.rand(1, N, generator=g, device="cuda")) / (32.0 * math.sqrt(H))
        return st
    st.update(h=x, dy=torch.randn(T, H, generator=g, device="cuda").to(dt), dh=residual,
              rstd=1.0 / (x.float().square().mean(1) + EPS).sqrt())
    return st


# ------------------------------------------------------------- plain forms --
def _e2m1(a):
    """Magnitudes rounded to the nearest e2m1 value, half to even, at most 6."""
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return (torch.round(a / step) * step).clamp(max=6.0)


def _power(e):
    """2^e in 32 bits, for whole -127 <= e <= 127."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).int().view(torch.float32)


def _blocks(x, form):
    """Rows [rows, K] in 32 bits as (e2m1 values [rows, K], block scales, row scales or None)."""
    b = x.view(x.shape[0], -1, BLOCK[form])
    most = b.abs().amax(2)
    if form == "mxfp4":
        e = torch.where(most > 0, torch.frexp(most).exponent - 3, -127).clamp(min=-127)
        s, scale, y = _power(e), None, b * _power(-e)[:, :, None]
    else:
        m, e = torch.frexp(most.amax(1))
        scale = torch.where(m > 0, _power((e - torch.where(m <= 0.65625, 12, 11)).clamp(min=-126)), 0.0)
        # (tensors of sixes: a product with a rounded 1 / 6 is not a quotient)
        t = torch.where(scale[:, None] > 0, most / torch.full_like(most, 6.0) / scale[:, None], 0.0)
        s = t.clamp(max=448.0).to(torch.float8_e4m3fn).float()
        d = (s * scale[:, None])[:, :, None]
        y = torch.where(d > 0, b / d, 0.0)
    return torch.where(torch.signbit(y), -_e2m1(y.abs()), _e2m1(y.abs())).view_as(x), s, scale


def _codes(v):
    """e2m1 values to codes, two a byte."""
    a = v.abs()
    c = torch.where(a <= 2.0, 2.0 * a, torch.where(a <= 4.0, a + 2.0, 7.0)).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    return c[:, 0::2] | (c[:, 1::2] << 4)


def _scale_bytes(s, form):
    return (torch.frexp(s).exponent + 126).to(torch.uint8) if form == "mxfp4" else s.to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes, scales, form):
    """Codes [..., K / 2] and scale bytes to the block values e2m1 * scale [..., K] in 32 bits."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    e, m = (c >> 1) & 3, c & 1
    v = ((m + 2 * (e > 0)) << (e.clamp(min=1) - 1)).float() * 0.5
    v = torch.where(c > 7, -v, v)
    s = _power(scales.int() - 127) if form == "mxfp4" else scales.view(torch.float8_e4m3fn).float()
    return (v.view(*s.shape, BLOCK[form]) * s[..., None]).view_as(v)


def _plain_product(st):
    c = st["case"]
    R, E, k, form = c["tokens"] * c["top_k"], c["experts"], c["top_k"], c["form"]
    x = st["x"].float()
    if c["gated"]:
        g, u = x.chunk(2, dim=1)
        x = g / (1.0 + torch.exp(-g)) * u
    v, s, scale = _blocks(x.contiguous(), form)
    rows = (v.view(*s.shape, -1) * s[:, :, None]).view_as(v)
    if E == 1:
        row, expert = slice(None), slice(None)
        out = rows @ _values(st["wq"][0], st["ws"][0], form).t()
    else:
        offsets, p = st["offsets"].long(), torch.arange(R, device="cuda")
        row = p if c["gated"] else st["row_src"].long() // k
        expert = torch.searchsorted(offsets, p, right=True) - 1
        rows = rows[row]
        if R < E:  # fewer rows than experts: each with its own matrix
            out = torch.bmm(_values(st["wq"][expert], st["ws"][expert], form), rows[:, :, None])[:, :, 0]
        else:  # every expert's rows, padded to the longest segment
            slot = expert * st["most"] + p - offsets[expert]
            padded = rows.new_zeros(E * st["most"], c["K"])
            padded[slot] = rows
            weights = _values(st["wq"], st["ws"], form)
            out = torch.bmm(padded.view(E, st["most"], -1), weights.transpose(1, 2)).view(E * st["most"], -1)[slot]
    if scale is not None:
        out = out * scale[row][:, None] * st["w_scale"][expert]
    return out.to(DTYPES[c["out"]])


def _plain(st):
    c = st["case"]
    dt = DTYPES[c["dtype"]]
    if c["op"] == "product":
        return _plain_product(st)
    if c["op"] == "requantize":
        v, s, scale = _blocks(st["x"].float(), c["form"])
        x = (v.view(*s.shape, -1) * s[:, :, None]).view_as(v)
        return (x if scale is None else x * scale[:, None]).to(dt)
    if c["op"] == "norm":
        h = st["x"] if st["residual"] is None else (st["x"].float() + st["residual"].float()).to(dt)
        rstd = 1.0 / (h.float().square().mean(1) + EPS).sqrt()
        y = (h.float() * rstd[:, None] * st["gamma"]).to(dt)
        out = {"h": h, "y": y, "rstd": rstd}
        if c["codes"]:
            f = y.float()
            most = f.abs().amax(1, keepdim=True)
            q = torch.where(most > 0, torch.round(f * 127.0 / most), 0.0)
            out["z"] = ((q @ st["wq"][0].float().t()) * (most / torch.full_like(most, 127.0)) * st["w_scale"]).to(dt)
        return out
    h, dy, r = st["h"].float(), st["dy"].float(), st["rstd"][:, None]
    g = dy * st["gamma"]
    dx = r * (g - h * r * r * (g * h).mean(1, keepdim=True))
    if st["dh"] is not None:
        dx = dx + st["dh"].float()
    return {"dx": dx.to(dt), "dgamma": (dy * h * r).sum(0)}


# ------------------------------------------------- the framework's operators --
def _framework(st):
    import block_quantized_expert_gb300 as bqe

    c = st["case"]
    new = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    if c["op"] in ("requantize", "product"):
        fmt = bqe.MOE_WEIGHTS_NVFP4 if c["form"] == "nvfp4" else bqe.MOE_WEIGHTS_MXFP4
        x = st["x"]
        rows, K = x.shape[0], c["K"]
        q, s = new(rows, K // 2, dtype=torch.uint8), new(rows, K // BLOCK[c["form"]], dtype=torch.uint8)
        scale = new(rows) if c["form"] == "nvfp4" else None
        bqe.moe_quantize_blocks(x, q, s, scale, fmt, gated=c.get("gated", False))
        if c["op"] == "requantize":
            back = torch.empty_like(x)
            bqe.moe_dequantize_blocks(q, s, back, scale, fmt)
            return back
        out = new(c["tokens"] * c["top_k"], c["N"], dtype=DTYPES[c["out"]])
        if c["experts"] == 1:
            bqe.moe_block_product(q, s, st["wq"], st["ws"], out, None, None, 1, scale, st["w_scale"], fmt)
        elif c["gated"]:
            bqe.moe_block_product(q, s, st["wq"], st["ws"], out, st["offsets"], None, 1, scale, st["w_scale"], fmt)
        else:
            bqe.moe_block_product(q, s, st["wq"], st["ws"], out, st["offsets"], st["row_src"], c["top_k"], scale,
                                  st["w_scale"], fmt)
        return out
    T, H, N, dt = c["tokens"], c["hidden"], c["codes"], DTYPES[c["dtype"]]
    if c["op"] == "norm":
        x, residual = st["x"], st["residual"]
        h = x if residual is None else torch.empty_like(x)
        y, rstd = torch.empty_like(x), new(T)
        q, scale = (new(T, H, dtype=torch.int8), new(T)) if N else (None, None)
        bqe.moe_norm_rows(x, st["gamma"], y, EPS, residual, None if residual is None else h, rstd, q, scale)
        out = {"h": h, "y": y, "rstd": rstd}
        if N:
            out["z"] = new(T, N, dtype=dt)
            bqe.moe_expert_product(q, scale, st["wq"], st["w_scale"], out["z"])
        return out
    dx, dgamma = torch.empty_like(st["h"]), new(H)
    scratch = new(bqe.moe_norm_scratch_bytes(T, H), dtype=torch.uint8)
    bqe.moe_norm_rows_backward(st["dy"], st["h"], st["gamma"], st["rstd"], dx, dgamma, scratch, st["dh"])
    return {"dx": dx, "dgamma": dgamma}


def run(state):
    return _framework(state) if own else _plain(state)


# --------------------------------------------------------- definition, 64 bits --
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_FINE = [b * 2.0 ** -9 if b < 8 else (8 + b % 8) * 2.0 ** (b // 8 - 10) for b in range(127)]  # e4m3 values


def _two(e):
    """2^e in 64 bits, for whole e (pow of a tensor is off by a rounding on some devices)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest(a, grid):
    """The nearest of the grid's values, ties to the one of even place."""
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = torch.searchsorted(mid, a, right=False), torch.searchsorted(mid, a, right=True)
    return grid[torch.where(lo % 2 == 0, lo, hi)]


def _exact_rows(x, form):
    """(block values, row scales) of rows in 64 bits."""
    grid = torch.tensor(_GRID, dtype=torch.float64, device="cuda")
    n = BLOCK[form]
    values, scales = torch.empty_like(x), torch.ones(x.shape[0], dtype=torch.float64, device="cuda")
    if form == "nvfp4":
        fine = torch.tensor(_FINE, dtype=torch.float64, device="cuda")
        m, e = torch.frexp(x.abs().amax(1) / 2688)
        scales = _two(torch.where(m == 0.5, e - 1, e).clamp(min=-126))
    for k in range(0, x.shape[1], n):
        b = x[:, k:k + n]
        most = b.abs().amax(1)
        if form == "mxfp4":
            s = _two(torch.where(most > 0, torch.frexp(most).exponent - 3, -127).clamp(min=-127))
            d = s
        else:
            s = _nearest(most / (6 * scales.clamp(min=1e-300)), fine)
            d = s * scales
        v = _nearest(b.abs() / d.clamp(min=1e-300)[:, None], grid) * (d > 0)[:, None]
        values[:, k:k + n] = torch.sign(b) * v * s[:, None]
    return values, scales


def _exact_product(st):
    c = st["case"]
    K, E, k, form = c["K"], c["experts"], c["top_k"], c["form"]
    x = st["x"].double()
    if c["gated"]:
        x = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:]
    rows, scale = _exact_rows(x, form)
    fine = torch.tensor(_FINE, dtype=torch.float64, device="cuda")
    both = torch.tensor(_GRID + tuple(-v for v in _GRID), dtype=torch.float64, device="cuda")
    ends = st["offsets"].tolist() if E > 1 else [0, c["tokens"]]
    src = st["row_src"].long() // k if E > 1 and not c["gated"] else torch.arange(c["tokens"] * k, device="cuda")
    out = torch.zeros(c["tokens"] * k, c["N"], dtype=torch.float64, device="cuda")
    for e in range(E):
        at = src[ends[e]:ends[e + 1]]
        if not len(at):
            continue
        codes, s = st["wq"][e].long(), st["ws"][e].long()
        s = _two(s - 127) if form == "mxfp4" else fine[s]
        w = torch.empty(c["N"], K, dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = both[codes % 16], both[codes // 16]
        w *= s.repeat_interleave(BLOCK[form], dim=1)
        if st["w_scale"] is not None:
            w *= st["w_scale"][e].double()[:, None]
        out[ends[e]:ends[e + 1]] = (rows[at] * scale[at][:, None]) @ w.T
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "product":
        return _exact_product(st)
    if case["op"] == "requantize":
        v, scale = _exact_rows(st["x"].double(), case["form"])
        return v * scale[:, None]
    if case["op"] == "norm":
        h = st["x"].double() if st["residual"] is None else (st["x"].double() + st["residual"].double())
        held = h.to(DTYPES[case["dtype"]]).double()  # the stream's own type is part of the definition
        rstd = (held.pow(2).mean(1) + EPS).rsqrt()
        y = held * rstd[:, None] * st["gamma"].double()
        out = {"h": h, "y": y, "rstd": rstd}
        if case["codes"]:
            held = y.to(DTYPES[case["dtype"]]).double()
            most = held.abs().max(dim=1).values[:, None]
            q = torch.round(held * 127 / most.clamp(min=1e-300)) * (most / 127)
            out["z"] = q @ (st["wq"][0].double() * st["w_scale"][0].double()[:, None]).T
        return out
    h, dy, r, gamma = st["h"].double(), st["dy"].double(), st["rstd"].double()[:, None], st["gamma"].double()
    # d/dh of y = h rstd(h) gamma, applied to dy, and of the sum that the residual goes on as
    dx = dy * gamma * r - h * r ** 3 * (dy * gamma * h).sum(1, keepdim=True) / h.shape[1]
    if st["dh"] is not None:
        dx += st["dh"].double()
    return {"dx": dx, "dgamma": torch.einsum("th,th,t->h", dy, h, r[:, 0])}
