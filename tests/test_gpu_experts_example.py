"""examples/experts.py on the device: each step of the block against the 64-bit
formula of what it read, and the whole of it in a graph.
"""
import importlib.util
import os

import pytest
import torch

from . import beside_ref as br
from . import op_ref as ref

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "experts.py")
spec = importlib.util.spec_from_file_location("experts", PATH)
ex = importlib.util.module_from_spec(spec)
spec.loader.exec_module(ex)


@pytest.mark.parametrize("tokens", [1, 6, 40])
def test_the_block_step_by_step(tokens):
    K, E, k = 256, 6, 3
    block = ex.Block(K, 128, E, k, 3, 8, seed=2)
    x, r = (ref.loud(tokens, K, 60 + i).bfloat16() for i in range(2))
    adapter = torch.arange(tokens, dtype=torch.int32) % 4 - 1
    t, R = block.buffers(tokens), r.cuda()
    y = block(x.cuda(), adapter.cuda(), R, t)
    torch.cuda.synchronize()
    assert y is R
    proj, far = ref.w4_matmul(x, block.proj[0].cpu(), block.proj[1].cpu(), "int4", ex.GROUP)
    # the projection is rounded to bf16 before the adapters add to it: half a step of 2^-8
    o, far_o = br.lora(x, adapter, block.a.cpu(), block.b.cpu(), block.scale.cpu(), proj.clone())
    ref.check(t["o"].cpu(), o, far_o + far + 2.0 ** -8 * (proj.abs() + far), "projection")
    h, _, n = ref.rmsnorm(t["o"].cpu(), r, block.norm.cpu(), ex.EPS)
    ref.check(t["n"].cpu(), n, n.abs() * (ref.norm_rel(K) + 8 * ref.U), "norm")
    N = t["n"].cpu().double()
    logits = N @ block.router.cpu().double().t()
    ref.check(t["logits"].cpu(), logits, K * ref.U * (N.abs() @ block.router.cpu().double().abs().t()), "logits")
    index, weight = br.route(t["logits"].cpu(), k)
    assert torch.equal(t["index"].cpu(), index)
    assert ((t["weight"].cpu().double() - weight).abs() <= weight * 60 * br.U).all()
    base = h.to(torch.bfloat16)
    want, far = br.moe(t["n"].cpu(), index, t["weight"].cpu(), block.gate_up[0].cpu(), block.down[0].cpu(), block.gate_up[1].cpu(),
                       block.down[1].cpu(), "int4", ex.GROUP, base=base)
    # h itself is rounded to bf16 from fp32 sums: where the two roundings differ it is a step (2^-7 of it at most) away
    ref.check(y.cpu(), want, far + h.abs() * ref.U * 2, "y")


def test_command_runs(capsys):
    y = ex.main(5, 256, 128, 8, 2, 3, 8)
    out = capsys.readouterr().out
    assert torch.isfinite(y.float()).all() and "called" in out and "replayed" in out
