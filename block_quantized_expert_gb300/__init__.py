"""Python binding of libmoe (include/moe.h): the routed-expert FFN layer of a
DeepSeek-V4-Flash-style MoE on one GB300, MXFP4 experts, MXFP8 activations.

Argument marshalling only: every step runs in libmoe's CUDA kernels.  Tensors
are torch CUDA tensors (device memory and streams come from PyTorch); the
functions check dtype, shape, device and contiguity, pass raw pointers and
the current CUDA stream, and raise MoeError on a non-zero status.  There is no
fallback: if libmoe.so cannot be loaded the import of the functions fails.
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass
from typing import Optional

_HAS_TORCH = True
try:
    import torch
except ModuleNotFoundError as _missing:  # the library, its C entries and sizes do without
    if _missing.name != "torch":
        raise

    class _NoTorch:
        def __getattr__(self, name):
            raise ModuleNotFoundError("calls on tensors need PyTorch (torch)", name="torch")

    torch, _HAS_TORCH = _NoTorch(), False

from . import _build

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_OOM, MOE_ERR_CUDA, MOE_ERR_TIMEOUT = range(6)
_STATUS = {1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_OOM",
           4: "MOE_ERR_CUDA", 5: "MOE_ERR_TIMEOUT"}

# Every symbol include/moe.h declares.
EXPORTS = ("moe_create", "moe_destroy", "moe_route", "moe_route_hash", "moe_permute",
           "moe_quantize", "moe_forward", "moe_forward_host", "moe_hidden", "moe_check",
           "moe_workspace_bytes", "moe_last_error", "moe_set_gemm_path", "moe_set_stage_events",
           "moe_kernel_launches", "moe_permute_noalloc", "moe_set_trace", "moe_route_forward",
           "moe_set_route_prune", "moe_set_wait_limit", "moe_test_stall_next_decode", "moe_test_decode_split",
           "moe_set_decode_kernel", "moe_decode_info", "moe_dispatch", "moe_dispatch_backward",
           "moe_combine", "moe_combine_backward", "moe_route_backward", "moe_quantize_rows",
           "moe_expert_product", "moe_check_product", "moe_test_stall_next_product", "moe_permute_scratch",
           "moe_permute_scratch_bytes")


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_STATUS.get(status, status)}: {msg}")
        self.status = status


class moe_config(C.Structure):
    _fields_ = [("hidden", C.c_int), ("inter", C.c_int), ("n_experts", C.c_int),
                ("top_k", C.c_int), ("max_tokens", C.c_int), ("has_shared", C.c_int),
                ("w_scale", C.c_float), ("weight_format", C.c_int)]


MOE_WEIGHTS_MXFP4, MOE_WEIGHTS_NVFP4 = 0, 1


_WEIGHT_FIELDS = ("gate_q", "gate_s", "up_q", "up_s", "down_q", "down_s",
                  "sh_gate_q", "sh_gate_s", "sh_up_q", "sh_up_s", "sh_down_q", "sh_down_s")


class moe_weights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in _WEIGHT_FIELDS + ("gate_g", "up_g", "down_g")]


_lib = None


def load_library(build: bool = True) -> C.CDLL:
    """Load (building first if stale and `build`) the in-tree libmoe.so."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.build() if build else _build.LIB
    if not path.exists():
        raise ImportError(f"libmoe.so not found at {path}")
    L = C.CDLL(str(path))
    vp, i, f, ll = C.c_void_p, C.c_int, C.c_float, C.c_longlong
    sigs = {
        "moe_create": ([C.POINTER(moe_config), C.POINTER(moe_weights), vp, C.POINTER(vp)], i),
        "moe_destroy": ([vp], i),
        "moe_route": ([vp, vp, i, vp, vp, vp], i),
        "moe_route_hash": ([vp, vp, vp, i, i, vp, vp, vp], i),
        "moe_permute": ([vp, vp, i, vp, vp, vp, vp], i),
        "moe_quantize": ([vp, vp, i, vp, vp, vp], i),
        "moe_forward": ([vp, vp, i, vp, vp, vp, vp], i),
        "moe_forward_host": ([vp, vp, vp, i, vp, vp], i),
        "moe_hidden": ([vp, i, vp, vp, vp], i),
        "moe_check": ([vp, vp], i),
        "moe_workspace_bytes": ([C.POINTER(moe_config)], C.c_size_t),
        "moe_last_error": ([vp], C.c_char_p),
        "moe_set_gemm_path": ([vp, i], i),
        "moe_set_stage_events": ([vp, C.POINTER(vp), i], i),
        "moe_kernel_launches": ([vp], C.c_ulonglong),
        "moe_permute_noalloc": ([vp, i, i, i, vp, vp, vp, vp], i),
        "moe_permute_scratch": ([vp, i, i, i, vp, vp, vp, vp, C.c_size_t, vp], i),
        "moe_permute_scratch_bytes": ([i, i, i], C.c_size_t),
        "moe_set_trace": ([vp, vp, C.c_size_t], i),
        "moe_route_forward": ([vp, vp, vp, i, vp, vp, vp, vp], i),
        "moe_set_route_prune": ([vp, i, f, f], i),
        "moe_set_wait_limit": ([vp, C.c_double], i),
        "moe_test_stall_next_decode": ([vp], i),
        "moe_test_decode_split": ([C.c_int, C.c_int, C.c_int, C.c_int, C.c_int, C.c_int, C.POINTER(C.c_int)], i),
        "moe_set_decode_kernel": ([vp, i], i),
        "moe_decode_info": ([vp, C.POINTER(C.c_int)], i),
        "moe_dispatch": ([vp, i, ll, i, i, i, vp, i, vp, vp, ll, vp], i),
        "moe_dispatch_backward": ([vp, i, ll, i, i, i, vp, vp, i, ll, vp], i),
        "moe_combine": ([vp, i, ll, vp, i, i, i, vp, vp, i, ll, vp], i),
        "moe_combine_backward": ([vp, i, ll, vp, i, ll, vp, i, i, i, vp, i, vp, vp, ll, vp, vp], i),
        "moe_route_backward": ([vp, vp, vp, i, i, i, f, vp, vp], i),
        "moe_quantize_rows": ([vp, i, ll, i, i, i, vp, ll, vp, vp], i),
        "moe_expert_product": ([vp, ll, i, vp, i, vp, vp, i, i, vp, vp, i, i, vp, i, ll, vp], i),
        "moe_check_product": ([vp], i),
        "moe_test_stall_next_product": ([], i),
    }
    for name, (args, res) in sigs.items():
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, res
    _lib = L
    return L


def _check(status: int, layer_ptr=None):
    if status != MOE_OK:
        msg = load_library().moe_last_error(layer_ptr)
        raise MoeError(status, msg.decode() if msg else "")


def _stream(stream) -> int:
    if stream is None:  # torch.cuda.current_stream() without the Stream object around it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t, dtype, shape=None, name="tensor"):
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and (shape is None or t.shape == shape)
            and t.is_contiguous()):
        return t.data_ptr()
    if t is None:
        raise ValueError(f"{name} is None")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


MOE_F32, MOE_BF16, MOE_F16 = range(3)
_ROW_TYPES = {}
if _HAS_TORCH:
    _ROW_TYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float16: MOE_F16, torch.int8: None}


def _rows(t, name, rows=None, width=None):
    """(pointer, moe_dtype, stride) of a 2-D CUDA tensor of rows whose elements
    are adjacent; the moe_dtype of int8 rows is None."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape, code = t.shape, _ROW_TYPES.get(t.dtype, -1)
    if code == -1 or len(shape) != 2:
        raise ValueError(f"{name} must be a 2-D tensor of rows in float32, bfloat16, float16 or int8, "
                         f"got {t.dtype} {tuple(shape)}")
    n, m = shape
    if (rows is not None and n != rows) or (width is not None and m != width):
        raise ValueError(f"{name} must have shape ({n if rows is None else rows}, {m if width is None else width}), "
                         f"got {tuple(shape)}")
    step, inner = t.stride()
    if inner != 1 and m > 1:
        raise ValueError(f"the elements of a row of {name} must be adjacent")
    return t.data_ptr(), code, (step if n > 1 else m)


def _hptr(t, dtype, shape, name):
    if not isinstance(t, torch.Tensor) or t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous host {dtype} tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    return t.data_ptr()


@dataclass
class MoeConfig:
    hidden: int
    inter: int
    n_experts: int
    top_k: int
    max_tokens: int
    has_shared: bool = False
    w_scale: float = 1.5
    weight_format: int = MOE_WEIGHTS_MXFP4

    def c(self) -> moe_config:
        return moe_config(self.hidden, self.inter, self.n_experts, self.top_k, self.max_tokens,
                          int(bool(self.has_shared)), self.w_scale, int(self.weight_format))


class Layer:
    """Owner of a moe_layer*; freed by moe_destroy (or when collected)."""

    def __init__(self, ptr: int, cfg: MoeConfig):
        self.ptr = C.c_void_p(ptr)
        self.cfg = cfg

    def close(self):
        if self.ptr and self.ptr.value:
            moe_destroy(self)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def moe_workspace_bytes(cfg: MoeConfig) -> int:
    return load_library().moe_workspace_bytes(C.byref(cfg.c()))


def moe_create(cfg: MoeConfig, weights: dict, stream=None) -> Layer:
    """weights: dict of CUDA tensors named as the fields of moe_weights (uint8;
    NVFP4 layers also float32 gate_g, up_g, down_g [E])."""
    lib = load_library()
    H, I, E = cfg.hidden, cfg.inter, cfg.n_experts
    nv = cfg.weight_format == MOE_WEIGHTS_NVFP4
    blk = 16 if nv else 32
    shapes = {"gate_q": (E, I, H // 2), "gate_s": (E, I, H // blk), "up_q": (E, I, H // 2),
              "up_s": (E, I, H // blk), "down_q": (E, H, I // 2), "down_s": (E, H, I // blk),
              "sh_gate_q": (I, H), "sh_gate_s": (I // 128, H // 128), "sh_up_q": (I, H),
              "sh_up_s": (I // 128, H // 128), "sh_down_q": (H, I), "sh_down_s": (H // 128, I // 128)}
    wt = moe_weights()
    for n in _WEIGHT_FIELDS:
        if n.startswith("sh_") and not cfg.has_shared:
            setattr(wt, n, None)
            continue
        setattr(wt, n, _ptr(weights.get(n), torch.uint8, shapes[n], n))
    for n in ("gate_g", "up_g", "down_g"):
        setattr(wt, n, _ptr(weights.get(n), torch.float32, (E,), n) if nv else None)
    out = C.c_void_p()
    _check(lib.moe_create(C.byref(cfg.c()), C.byref(wt), _stream(stream), C.byref(out)))
    return Layer(out.value, cfg)


def moe_destroy(layer: Layer):
    lib = load_library()
    st = lib.moe_destroy(layer.ptr)
    layer.ptr = C.c_void_p(None)
    _check(st)


def moe_set_gemm_path(layer: Layer, path: int):
    _check(load_library().moe_set_gemm_path(layer.ptr, int(path)), layer.ptr)


def moe_set_decode_kernel(layer: Layer, kind: int):
    """One-token calls: 0 automatic, 1 the CUDA-core GEMV kernel, 2 the tcgen05 kernel."""
    _check(load_library().moe_set_decode_kernel(layer.ptr, int(kind)), layer.ptr)


def moe_decode_info(layer: Layer) -> int:
    """The whole-layer kernel a one-token call takes: 0 none, 1 CUDA-core GEMV, 2 tcgen05."""
    kind = C.c_int(0)
    _check(load_library().moe_decode_info(layer.ptr, C.byref(kind)), layer.ptr)
    return kind.value


def moe_set_route_prune(layer: Layer, keep: int, min_w: float = 0.0, rho: float = 0.0):
    """Tail pruning of the learned router: keep at most `keep` experts, stop at
    the first weight below `min_w`, rescale the kept weights for correlation
    `rho` (0: L2 quadrature, 1: linear).  keep >= k with min_w <= 0: off."""
    _check(load_library().moe_set_route_prune(layer.ptr, int(keep), float(min_w), float(rho)), layer.ptr)


def moe_set_wait_limit(layer: Layer, seconds: float):
    """Wall-time limit of the layer's device-side waits (default 2 s)."""
    _check(load_library().moe_set_wait_limit(layer.ptr, float(seconds)), layer.ptr)


def moe_test_decode_split(num_sms: int, kept: int, hidden: int, inter: int, nvfp4: bool = False,
                          shared: bool = False) -> list:
    """The CUDA-core decode kernel's down-row cuts (host computation, no GPU)."""
    cut = (C.c_int * (num_sms + 1))()
    _check(load_library().moe_test_decode_split(num_sms, kept, hidden, inter, int(nvfp4), int(shared), cut))
    return list(cut)


def moe_test_stall_next_decode(layer: Layer):
    """Test hook: the next one-token decode-kernel call cannot complete its
    hand-off, runs out its bounded waits and reports MOE_ERR_TIMEOUT."""
    _check(load_library().moe_test_stall_next_decode(layer.ptr), layer.ptr)


def moe_set_stage_events(layer: Layer, events):
    """events: 6 torch.cuda.Event (recorded by the next moe_forward), or None."""
    lib = load_library()
    if events is None:
        _check(lib.moe_set_stage_events(layer.ptr, None, 0), layer.ptr)
        return
    if len(events) != 6:
        raise ValueError("need 6 events")
    for ev in events:  # torch creates the CUDA event lazily
        if ev.cuda_event == 0:
            ev.record()
    arr = (C.c_void_p * 6)(*[ev.cuda_event for ev in events])
    _check(lib.moe_set_stage_events(layer.ptr, arr, 6), layer.ptr)


def moe_route(layer: Layer, logits, ids, w, stream=None):
    T = logits.shape[0]
    c = layer.cfg
    st = load_library().moe_route(layer.ptr, _ptr(logits, torch.float32, (T, c.n_experts), "logits"), T,
                                  _ptr(ids, torch.int32, (T, c.top_k), "ids"),
                                  _ptr(w, torch.float32, (T, c.top_k), "w"), _stream(stream))
    _check(st, layer.ptr)


def moe_route_hash(layer: Layer, token_ids, tid2eid, ids, w, stream=None):
    T = token_ids.shape[0]
    V = tid2eid.shape[0]
    c = layer.cfg
    st = load_library().moe_route_hash(layer.ptr, _ptr(token_ids, torch.int32, (T,), "token_ids"),
                                       _ptr(tid2eid, torch.int32, (V, c.top_k), "tid2eid"), V, T,
                                       _ptr(ids, torch.int32, (T, c.top_k), "ids"),
                                       _ptr(w, torch.float32, (T, c.top_k), "w"), _stream(stream))
    _check(st, layer.ptr)


def moe_permute(layer: Layer, ids, offsets, row_src, row_dst, stream=None):
    T = ids.shape[0]
    c = layer.cfg
    R = T * c.top_k
    st = load_library().moe_permute(layer.ptr, _ptr(ids, torch.int32, (T, c.top_k), "ids"), T,
                                    _ptr(offsets, torch.int32, (c.n_experts + 1,), "offsets"),
                                    _ptr(row_src, torch.int32, (R,), "row_src"),
                                    _ptr(row_dst, torch.int32, (R,), "row_dst"), _stream(stream))
    _check(st, layer.ptr)


def moe_permute_noalloc(ids, n_experts: int, offsets, row_src, row_dst, stream=None):
    """The grouping of moe_permute without a layer and without allocating
    (scratch in a static device array; T * top_k <= 65536)."""
    T, k = ids.shape
    R = T * k
    st = load_library().moe_permute_noalloc(
        _ptr(ids, torch.int32, (T, k), "ids"), T, k, n_experts,
        _ptr(offsets, torch.int32, (n_experts + 1,), "offsets"),
        _ptr(row_src, torch.int32, (R,), "row_src"), _ptr(row_dst, torch.int32, (R,), "row_dst"),
        _stream(stream))
    _check(st)


def moe_permute_scratch_bytes(T: int, top_k: int, n_experts: int) -> int:
    """Bytes of scratch of moe_permute_scratch; 0 for sizes that it does not take."""
    return load_library().moe_permute_scratch_bytes(T, top_k, n_experts)


def moe_permute_scratch(ids, n_experts: int, offsets, row_src, row_dst, scratch, stream=None):
    """The grouping of moe_permute without a layer, in the caller's scratch (a CUDA
    uint8 tensor of moe_permute_scratch_bytes); calls share nothing."""
    T, k = ids.shape
    R = T * k
    st = load_library().moe_permute_scratch(
        _ptr(ids, torch.int32, (T, k), "ids"), T, k, n_experts,
        _ptr(offsets, torch.int32, (n_experts + 1,), "offsets"),
        _ptr(row_src, torch.int32, (R,), "row_src"), _ptr(row_dst, torch.int32, (R,), "row_dst"),
        _ptr(scratch, torch.uint8, None, "scratch"), scratch.numel(),
        _here(stream, ids, offsets, row_src, row_dst, scratch))
    _check(st)


def moe_quantize(layer: Layer, x, q, s, stream=None):
    T = x.shape[0]
    H = layer.cfg.hidden
    st = load_library().moe_quantize(layer.ptr, _ptr(x, torch.int16, (T, H), "x"), T,
                                     _ptr(q, torch.uint8, (T, H), "q"),
                                     _ptr(s, torch.uint8, (T, H // 32), "s"), _stream(stream))
    _check(st, layer.ptr)


def moe_forward(layer: Layer, x, ids, w, out, stream=None):
    """x: int16 CUDA tensor [T][H] holding bf16 bits (or a bfloat16 tensor)."""
    T = x.shape[0]
    c = layer.cfg
    if x.dtype == torch.bfloat16:
        x = x.view(torch.int16)
    st = load_library().moe_forward(layer.ptr, _ptr(x, torch.int16, (T, c.hidden), "x"), T,
                                    _ptr(ids, torch.int32, (T, c.top_k), "ids"),
                                    _ptr(w, torch.float32, (T, c.top_k), "w"),
                                    _ptr(out, torch.float32, (T, c.hidden), "out"), _stream(stream))
    _check(st, layer.ptr)


def moe_route_forward(layer: Layer, logits, x, ids, w, out, stream=None):
    """Routing and layer in one call (ids, w and out are written)."""
    T = x.shape[0]
    c = layer.cfg
    if x.dtype == torch.bfloat16:
        x = x.view(torch.int16)
    st = load_library().moe_route_forward(
        layer.ptr, _ptr(logits, torch.float32, (T, c.n_experts), "logits"),
        _ptr(x, torch.int16, (T, c.hidden), "x"), T, _ptr(ids, torch.int32, (T, c.top_k), "ids"),
        _ptr(w, torch.float32, (T, c.top_k), "w"), _ptr(out, torch.float32, (T, c.hidden), "out"),
        _stream(stream))
    _check(st, layer.ptr)


def moe_forward_host(layer: Layer, x, logits, out, stream=None):
    """Host tensors (pinned for overlap): x int16 [T][H], logits f32 [T][E], out f32 [T][H]."""
    T = x.shape[0]
    c = layer.cfg
    st = load_library().moe_forward_host(layer.ptr, _hptr(x, torch.int16, (T, c.hidden), "x"),
                                         _hptr(logits, torch.float32, (T, c.n_experts), "logits"), T,
                                         _hptr(out, torch.float32, (T, c.hidden), "out"),
                                         _stream(stream))
    _check(st, layer.ptr)


def moe_hidden(layer: Layer, T: int, hq, hs, stream=None):
    c = layer.cfg
    R = T * c.top_k
    st = load_library().moe_hidden(layer.ptr, T, _ptr(hq, torch.uint8, (R, c.inter), "hq"),
                                   _ptr(hs, torch.uint8, (R, c.inter // 32), "hs"), _stream(stream))
    _check(st, layer.ptr)


def moe_check(layer: Layer, stream=None) -> int:
    """Synchronise the stream; raise MoeError if a device-side check fired."""
    st = load_library().moe_check(layer.ptr, _stream(stream))
    _check(st, layer.ptr)
    return st


def moe_set_trace(layer: Layer, buf):
    """buf: CUDA int64 tensor of >= max(48 * num_sms + 4, 8 * num_sms + 1024) entries, or None."""
    if buf is None:
        _check(load_library().moe_set_trace(layer.ptr, None, 0), layer.ptr)
        return
    _check(load_library().moe_set_trace(layer.ptr, _ptr(buf, torch.int64, None, "buf"), buf.numel()),
           layer.ptr)


def moe_kernel_launches(layer: Layer) -> int:
    return int(load_library().moe_kernel_launches(layer.ptr))


def moe_last_error(layer: Optional[Layer] = None) -> str:
    m = load_library().moe_last_error(layer.ptr if layer else None)
    return m.decode() if m else ""


def _here(stream, *tensors) -> int:
    """_stream for calls without a layer, on CUDA tensors: all of them, and the
    stream, must belong to the current device, on which the call launches."""
    dev = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"a tensor of this call is on cuda:{t.get_device()}, the current device is cuda:{dev}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    on = getattr(getattr(stream, "device", None), "index", None)
    if on is not None and on != dev:
        raise ValueError(f"the stream is of cuda:{on}, the current device is cuda:{dev}")
    return _stream(stream)


def _slots(row_dst, T, name="row_dst"):
    """(pointer, top_k) of the slots [T][top_k], also given flat."""
    n = row_dst.numel()
    if T < 1 or n % T or not 1 <= n // T <= 8:
        raise ValueError(f"{name} must hold T * top_k positions with top_k in [1, 8], got {n} for T = {T}")
    return _ptr(row_dst, torch.int32, None, name), n // T


def moe_dispatch(x, offsets, row_dst, xs, stream=None):
    """xs[row_dst[t, j]] = x[t]; zeros past the last placed row.  x [T][H] and
    xs [T * top_k][H] in one of float32, bfloat16, float16; offsets [E + 1] and
    row_dst [T * top_k] as moe_permute writes them."""
    T, H = x.shape
    if T == 0:
        return
    dst, k = _slots(row_dst, T)
    px, dt, sx = _rows(x, "x")
    ps, dts, ss = _rows(xs, "xs", T * k, H)
    if dt is None or dts != dt:
        raise ValueError("x and xs must have one floating dtype")
    lib = _lib or load_library()
    st = lib.moe_dispatch(px, dt, sx, T, k, H, _ptr(offsets, torch.int32, None, "offsets"),
                          offsets.numel() - 1, dst, ps, ss, _here(stream, x, offsets, row_dst, xs))
    if st:
        _check(st)


def moe_dispatch_backward(dxs, row_dst, dx, stream=None):
    """dx[t] = sum_j dxs[row_dst[t, j]]; dx in dxs's dtype or float32."""
    T, H = dx.shape
    if T == 0:
        return
    dst, k = _slots(row_dst, T)
    ps, dts, ss = _rows(dxs, "dxs", T * k, H)
    px, dt, sx = _rows(dx, "dx")
    if dt is None or dts is None:
        raise ValueError("dxs and dx must be floating tensors")
    lib = _lib or load_library()
    st = lib.moe_dispatch_backward(ps, dts, ss, T, k, H, dst, px, dt, sx, _here(stream, dxs, row_dst, dx))
    if st:
        _check(st)


def moe_combine(y, w, row_dst, out, stream=None):
    """out[t] = sum_j w[t, j] * y[row_dst[t, j]]; out in y's dtype or float32."""
    T, H = out.shape
    if T == 0:
        return
    dst, k = _slots(row_dst, T)
    py, dty, sy = _rows(y, "y", T * k, H)
    po, dto, so = _rows(out, "out")
    if dty is None or dto is None:
        raise ValueError("y and out must be floating tensors")
    lib = _lib or load_library()
    st = lib.moe_combine(py, dty, sy, _ptr(w, torch.float32, (T, k), "w"), T, k, H, dst, po, dto, so,
                         _here(stream, y, w, row_dst, out))
    if st:
        _check(st)


def moe_combine_backward(dout, y, w, offsets, row_dst, dy, dw, stream=None):
    """dy[row_dst[t, j]] = w[t, j] * dout[t] (zeros past the last placed row)
    and dw[t, j] = <dout[t], y[row_dst[t, j]]>; dout in y's dtype or float32."""
    T, H = dout.shape
    if T == 0:
        return
    dst, k = _slots(row_dst, T)
    pd, dtd, sd = _rows(dout, "dout")
    py, dty, sy = _rows(y, "y", T * k, H)
    pg, dtg, sg = _rows(dy, "dy", T * k, H)
    if dtd is None or dty is None or dtg != dty:
        raise ValueError("y and dy must have one floating dtype, and dout be a floating tensor")
    lib = _lib or load_library()
    st = lib.moe_combine_backward(pd, dtd, sd, py, dty, sy, _ptr(w, torch.float32, (T, k), "w"), T, k, H,
                                  _ptr(offsets, torch.int32, None, "offsets"), offsets.numel() - 1, dst, pg,
                                  sg, _ptr(dw, torch.float32, (T, k), "dw"),
                                  _here(stream, dout, y, w, offsets, row_dst, dy, dw))
    if st:
        _check(st)


def moe_route_backward(logits, ids, dw, dlogits, w_scale: float = 1.5, stream=None):
    """Gradient of moe_route's weights: dlogits [T][E] from dw [T][k]."""
    T, E = logits.shape
    k = ids.shape[1]
    if T == 0:
        return
    lib = _lib or load_library()
    st = lib.moe_route_backward(_ptr(logits, torch.float32, (T, E), "logits"),
                                _ptr(ids, torch.int32, (T, k), "ids"), _ptr(dw, torch.float32, (T, k), "dw"),
                                T, E, k, float(w_scale), _ptr(dlogits, torch.float32, (T, E), "dlogits"),
                                _here(stream, logits, ids, dw, dlogits))
    if st:
        _check(st)


def moe_quantize_rows(x, q, scale, gated: bool = False, stream=None):
    """x [rows][K] (gated: [rows][2 K], SiLU of the first half times the second)
    to int8 q [rows][K] with one float32 scale a row."""
    rows, K = q.shape
    if rows == 0:
        return
    px, dt, sx = _rows(x, "x", rows, 2 * K if gated else K)
    pq, dtq, sq = _rows(q, "q")
    if dt is None or dtq is not None:
        raise ValueError("x must be a floating tensor and q int8")
    lib = _lib or load_library()
    st = lib.moe_quantize_rows(px, dt, sx, int(bool(gated)), rows, K, pq, sq,
                               _ptr(scale, torch.float32, (rows,), "scale"), _here(stream, x, q, scale))
    if st:
        _check(st)


def moe_expert_product(q, scale, wq, w_scale, out, offsets=None, row_src=None, top_k: int = 1, stream=None):
    """out[p] = scale[r] * w_scale[e] * (wq[e] q[r]) for the positions p of expert
    e's segment; r = row_src[p] // top_k, or p without row_src.  q [rows][K] and
    wq [E][N][K] int8, w_scale [E][N], out [R][N]; offsets [E + 1] may be left
    out with one expert."""
    R, N = out.shape
    if R == 0:
        return
    if wq.dim() != 3:
        raise ValueError(f"wq must have shape (E, N, K), got {tuple(wq.shape)}")
    E, _, K = wq.shape
    pq, dtq, sq = _rows(q, "q", None, K)
    po, dto, so = _rows(out, "out")
    if dtq is not None or dto is None:
        raise ValueError("q must be int8 and out a floating tensor")
    rows = q.shape[0]
    lib = _lib or load_library()
    st = lib.moe_expert_product(pq, sq, rows, _ptr(scale, torch.float32, (rows,), "scale"), K,
                                _ptr(wq, torch.int8, (E, N, K), "wq"),
                                _ptr(w_scale, torch.float32, (E, N), "w_scale"), E, N,
                                None if offsets is None else _ptr(offsets, torch.int32, (E + 1,), "offsets"),
                                None if row_src is None else _ptr(row_src, torch.int32, (R,), "row_src"),
                                int(top_k), R, po, dto, so, _here(stream, q, scale, wq, w_scale, out, offsets, row_src))
    if st:
        _check(st)


def moe_check_product(stream=None):
    """Synchronise the stream; raise MoeError if a wait of moe_expert_product ran out,
    on any stream of the current device, since the last check on any."""
    _check(load_library().moe_check_product(_stream(stream)))


def moe_test_stall_next_product():
    """Test hook: the next tensor-core moe_expert_product runs out its bounded waits."""
    _check(load_library().moe_test_stall_next_product())
