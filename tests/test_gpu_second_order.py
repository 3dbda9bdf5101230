"""The gradients of dispatch, combine and router_weights are values without a graph
of their own: differentiating them again raises instead of leaving terms out."""
import pytest
import torch

from block_quantized_expert_gb300 import sorted_experts as se

pytestmark = pytest.mark.gpu


def pieces():
    T, k, E, H = 6, 2, 4, 8
    g = torch.Generator("cuda").manual_seed(1)
    logits = torch.randn(T, E, generator=g, device="cuda")
    ids = logits.topk(k, dim=1).indices.int()
    s = se.sort_tokens(ids, E)
    x = torch.randn(T, H, generator=g, device="cuda")
    return {"dispatch": (lambda v: se.dispatch(v, s), x),
            "combine y": (lambda v: se.combine(v, torch.ones(T, k, device="cuda"), s), se.dispatch(x, s)),
            "combine w": (lambda v: se.combine(se.dispatch(x, s), v, s), torch.rand(T, k, device="cuda")),
            "router": (lambda v: se.router_weights(v, ids), logits)}


@pytest.mark.parametrize("name", ["dispatch", "combine y", "combine w", "router"])
def test_a_penalty_on_a_gradient_raises(name):
    f, v = pieces()[name]
    v = v.detach().clone().requires_grad_()
    loss = f(v).square().sum()
    (grad,) = torch.autograd.grad(loss, v, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (loss + grad.square().sum()).backward()


@pytest.mark.parametrize("name", ["dispatch", "combine y", "combine w", "router"])
def test_the_first_order_is_as_before(name):
    f, v = pieces()[name]
    a, b = v.detach().clone().requires_grad_(), v.detach().clone().requires_grad_()
    f(a).square().sum().backward()
    (grad,) = torch.autograd.grad(f(b).square().sum(), b, create_graph=True)
    assert torch.equal(a.grad, grad) and a.grad.any()
