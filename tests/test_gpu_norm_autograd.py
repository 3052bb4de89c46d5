"""The example's norm under automatic differentiation where its gradient comes
in other forms than a whole matrix: broadcast (a sum over the rows), absent
(one output unused), shared with other uses of the leaves, and asked for
again (a second derivative, which the library does not have).
"""
import pytest
import torch

from . import op_ref as ref
from .test_gpu_feed_forward import ff

pytestmark = pytest.mark.gpu
M, N = 33, 200


def leaves(dtype=torch.float32):
    return [torch.randn(s, generator=ref.rng(i)).to(dtype) for i, s in enumerate(((M, N), (M, N), (N,)))]


def formula(x, r, w):
    h = x + r
    return h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + ff.EPS) * w, h


LOSSES = {
    "rows summed": lambda y, h, x: (y.sum(0) * torch.arange(N, device=y.device) / N).sum(),
    "only the sum": lambda y, h, x: (h * h).sum(),
    "only the norm": lambda y, h, x: (y * y * y).sum(),
    "all summed": lambda y, h, x: y.sum() + 2 * h.sum(),
    "x used again": lambda y, h, x: (y * x).sum() + (h * x).sum(),
}


@pytest.mark.parametrize("loss", sorted(LOSSES))
def test_gradients(loss):
    mine = [t.cuda().requires_grad_() for t in leaves()]
    LOSSES[loss](*ff.RmsNorm.apply(*mine), mine[0]).backward()
    exact = [t.double().requires_grad_() for t in leaves()]
    LOSSES[loss](*formula(*exact), exact[0]).backward()
    # fp32 throughout: sums of 200 and of 33 terms, a few roundings each, of values up to a few tens
    for a, b in zip(mine, exact):
        want = torch.zeros_like(b) if b.grad is None else b.grad
        assert (a.grad.cpu().double() - want).abs().max() < 2.0 ** -24 * 256 * (1 + want.abs().max())


def test_a_second_derivative_is_refused():
    x, r, w = (t.cuda().requires_grad_() for t in leaves())
    y, h = ff.RmsNorm.apply(x, r, w)
    (dx,) = torch.autograd.grad((y * y * y).sum() + (h * h).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (dx * dx).sum().backward()
