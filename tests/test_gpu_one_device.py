"""The calls without a layer launch on the current device: tensors and streams of
another one are refused before anything is enqueued.  (One GPU is enough: the
current device's number is what the test changes.)"""
import pytest
import torch

import block_quantized_expert_gb300 as bqe
from block_quantized_expert_gb300 import sorted_experts as se

pytestmark = pytest.mark.gpu


def calls():
    T, k, E, H = 4, 2, 3, 32
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    b = lambda *s: torch.zeros(*s, dtype=torch.int8, device="cuda")  # noqa: E731
    R, off, dst, ids = T * k, i(E + 1), i(T * k), i(T, k)
    return {
        "moe_dispatch": (f(T, H), off, dst, f(R, H)),
        "moe_dispatch_backward": (f(R, H), dst, f(T, H)),
        "moe_combine": (f(R, H), f(T, k), dst, f(T, H)),
        "moe_combine_backward": (f(T, H), f(R, H), f(T, k), off, dst, f(R, H), f(T, k)),
        "moe_route_backward": (f(T, E), ids, f(T, k), f(T, E)),
        "moe_quantize_rows": (f(T, H), b(T, H), f(T)),
        "moe_expert_product": (b(T, H), f(T), b(E, 8, H), f(E, 8), f(R, 8), off, i(R), k),
        "moe_permute_scratch": (ids, E, off, i(R), dst, torch.zeros(4096, dtype=torch.uint8, device="cuda")),
    }


@pytest.mark.parametrize("name", ["moe_dispatch", "moe_dispatch_backward", "moe_combine",
                         "moe_combine_backward", "moe_route_backward", "moe_quantize_rows", "moe_expert_product",
                         "moe_permute_scratch"])
def test_tensors_of_another_device_are_refused(name, monkeypatch):
    args = calls()[name]
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


class OtherStream:
    """What a stream of another device says of itself."""
    cuda_stream, device = 0, torch.device("cuda", 1)


@pytest.mark.parametrize("name", ["moe_combine", "moe_expert_product", "moe_permute_scratch"])
def test_streams_of_another_device_are_refused(name):
    with pytest.raises(ValueError, match="stream.*cuda:1"):
        getattr(bqe, name)(*calls()[name], stream=OtherStream())


def test_the_differentiable_forms_refuse_too(monkeypatch):
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    s, x = se.sort_tokens(ids, 3), torch.zeros(4, 8, device="cuda")
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_cuda_getDevice", lambda: 1)
        for call in (lambda: se.dispatch(x, s), lambda: se.combine(torch.zeros(8, 8, device="cuda"), torch.zeros(4, 2, device="cuda"), s)):
            with pytest.raises(ValueError, match="current device"):
                call()
