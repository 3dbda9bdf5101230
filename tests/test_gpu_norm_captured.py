"""norm and its gradient captured as a training step captures them: the bits of eager calls, replayed on other inputs."""
import pytest
import torch

from block_quantized_expert_gb300 import sorted_experts as se
from tests.test_gpu_sorted_rows import BF16, F32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [(1, 64), (300, 1030), (500, 4096), (5, 33001)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_captured_step(T, H, dtype):
    draw = lambda: [torch.randn(T, H, device="cuda").to(dtype) for _ in range(4)]  # noqa: E731
    x, r, a, b = static = draw()
    gamma = (torch.rand(H, device="cuda") + 0.5).requires_grad_()

    def step():
        leaves = [x.detach().requires_grad_(), r.detach().requires_grad_(), gamma]
        y, h = se.norm(leaves[0], gamma, leaves[1])
        return (y.detach(), h.detach(), *torch.autograd.grad((y, h), leaves, (a, b)))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t, new in zip(static, draw()):
            t.copy_(new)
        graph.replay()
        want = step()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
