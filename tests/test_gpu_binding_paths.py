"""The norm's and the 4-bit blocks' calls have a short way through the binding for dense tensors on the
current stream: whatever it does not take is refused as the long way (here: a stream given) refuses it."""
import pytest
import torch

import block_quantized_expert_gb300 as bqe

pytestmark = pytest.mark.gpu
T, H, E, N = 4, 64, 3, 8


def f(*n):
    return torch.zeros(*n, device="cuda")


def u(*n):
    return torch.zeros(*n, dtype=torch.uint8, device="cuda")


def i(*n):
    return torch.zeros(*n, dtype=torch.int32, device="cuda")


# positional arguments, then keywords; `need`: arguments that may not be None
CALLS = {
    "moe_norm_rows": (dict(x=f, gamma=f, y=f, residual=f, h=f, rstd=f, q=lambda *n: torch.zeros(*n, dtype=torch.int8, device="cuda"), scale=f),
                      dict(x=(T, H), gamma=(H,), y=(T, H), residual=(T, H), h=(T, H), rstd=(T,), q=(T, H), scale=(T,)), ("gamma",)),
    "moe_norm_rows_backward": (dict(dy=f, h=f, gamma=f, rstd=f, dx=f, dgamma=f, scratch=u, dh=f),
                               dict(dy=(T, H), h=(T, H), gamma=(H,), rstd=(T,), dx=(T, H), dgamma=(H,), scratch=(T * H * 4,), dh=(T, H)),
                               ("dy", "gamma", "rstd", "dx")),
    "moe_quantize_blocks": (dict(x=f, q=u, s=u, scale=f), dict(x=(T, H), q=(T, H // 2), s=(T, H // 16), scale=(T,)), ("s",)),
    "moe_dequantize_blocks": (dict(q=u, s=u, x=f, scale=f), dict(q=(T, H // 2), s=(T, H // 16), x=(T, H), scale=(T,)), ("s",)),
    "moe_block_product": (dict(q=u, s=u, wq=u, ws=u, out=f, offsets=i, row_src=i, scale=f, w_scale=f),
                          dict(q=(T, H // 2), s=(T, H // 16), wq=(E, N, H // 2), ws=(E, N, H // 16), out=(T, N), offsets=(E + 1,),
                               row_src=(T,), scale=(T,), w_scale=(E, N)), ("s", "ws")),
}
CASES = [(name, arg, how) for name, (makers, _, need) in CALLS.items() for arg in makers
         for how in ("dtype", "shape", "host") + (("None",) if arg in need else ())]


def arguments(name):
    makers, shapes, _ = CALLS[name]
    return {a: makers[a](*shapes[a]) for a in makers}


def outcome(call, args, **more):
    try:
        call(**args, **more)
    except Exception as e:  # noqa: BLE001 (what is raised is what is compared)
        return type(e), str(e)
    return None, ""


@pytest.mark.parametrize("name,arg,how", CASES)
def test_both_ways_refuse(name, arg, how):
    call, args = getattr(bqe, name), arguments(name)
    call(**args)
    t = args[arg]
    if how == "dtype":
        args[arg] = t.to(torch.float64)
    elif how == "shape":
        args[arg] = t.new_zeros((t.shape[0] - 1, *t.shape[1:]))
    elif how == "host":
        args[arg] = t.cpu()
    else:
        args[arg] = None
    short, long = outcome(call, args), outcome(call, args, stream=torch.cuda.current_stream())
    assert short[0] in (ValueError, bqe.MoeError), short
    assert short == long


def test_whole_numbers_of_any_kind():
    """top_k as numpy and torch hold it."""
    import numpy as np

    a = arguments("moe_block_product")
    q, w = torch.zeros(T, H, dtype=torch.int8, device="cuda"), torch.zeros(E, N, H, dtype=torch.int8, device="cuda")
    for k in (np.int64(1), torch.tensor(1), 1):
        bqe.moe_block_product(**a, top_k=k)
        bqe.moe_block_product(**a, top_k=k, stream=torch.cuda.current_stream())
        bqe.moe_expert_product(q, f(T), w, f(E, N), f(T, N), a["offsets"], a["row_src"], k)
    torch.cuda.synchronize()
