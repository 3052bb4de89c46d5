"""examples/feed_forward.py on the device: its decode and prompt paths against
the block computed in 64 bits from the same 4-bit weights, and its norm under
automatic differentiation against torch's own gradients of the formula.
"""
import importlib.util
import os

import pytest
import torch

from . import op_ref as ref

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")
spec = importlib.util.spec_from_file_location("feed_forward", PATH)
ff = importlib.util.module_from_spec(spec)
spec.loader.exec_module(ff)


def block64(b, x, r):
    h, _, n = ref.rmsnorm(x.cpu(), r.cpu(), b.norm.cpu(), ff.EPS)
    gu, dn = (ref.w4_weights(q.cpu(), s.cpu(), 2 * q.shape[1], "int4", ff.GROUP) for q, s in (b.gate_up, b.down))
    gu = n @ gu.t()
    act = torch.nn.functional.silu(gu[:, :b.hidden]) * gu[:, b.hidden:]
    return act @ dn.t(), h


@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_both_paths(tokens):
    b = ff.FeedForward(512, 1024, seed=3)
    x, r = (ref.loud(tokens, 512, 70 + i).to(torch.bfloat16).cuda() for i in range(2))
    want, h = block64(b, x, r)
    for path, rel in ((b.decode, 2.0 ** -4), (b.prompt, 2.0 ** -7)):
        # the rows' own rounding (e4m3 2^-4, bf16 2^-8) dominates and averages out over a sum: a whole
        # half step of relative error in the norm of the result is far more than the paths can make
        y, s = path(x, r.clone())
        assert ((y.double().cpu() - want).norm() / want.norm()).item() < rel
        ref.check(s.cpu(), h, h.abs() * ref.U, "residual")


def test_norm_under_autograd():
    g = ref.rng(5)
    x, r, dy, dh = (torch.randn(33, 200, generator=g) for _ in range(4))
    w = torch.randn(200, generator=g)
    leaves = [t.cuda().requires_grad_() for t in (x, r, w)]
    y, h = ff.RmsNorm.apply(*leaves)
    (y * dy.cuda()).sum().add((h * dh.cuda()).sum()).backward()
    ls = [t.double().requires_grad_() for t in (x, r, w)]
    h64 = ls[0] + ls[1]
    y64 = h64 * torch.rsqrt((h64 * h64).mean(dim=1, keepdim=True) + ff.EPS) * ls[2]
    (y64 * dy.double()).sum().add((h64 * dh.double()).sum()).backward()
    # fp32 throughout: sums of 200 and of 33 terms, a few roundings each
    for a, b in zip(leaves, ls):
        assert (a.grad.cpu().double() - b.grad).abs().max() < 2.0 ** -24 * 64 * (1 + b.grad.abs().max())


def test_command_runs(capsys):
    apart = ff.main(4, 512, 1024)
    assert apart < 2.0 ** -4 and "decode path" in capsys.readouterr().out
