"""A gated feed-forward block of a language model on the library's operators:
one path for a decode batch (norm to e4m3 rows, products with 4-bit weights),
one for a prompt (norm, weights expanded once, tuned products), and the norm's
gradients for training.

    python examples/feed_forward.py [tokens]

Both paths start from the same residual stream and 4-bit weights; the script
prints how far they are apart and the time of one block.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_autotuning_amd as gt  # noqa: E402

GROUP, EPS = 128, 1e-6


def quantise(w):
    """N x K weights as two's complement nibbles (even k low) and bf16 scales per group of k."""
    N, K = w.shape
    g = w.float().reshape(N, K // GROUP, GROUP)
    s = (g.abs().amax(dim=2) / 7.0).clamp(min=1e-8).bfloat16()
    q = (g / s.float()[:, :, None]).round().clamp(-8, 7).to(torch.int8).reshape(N, K)
    return ((q[:, 0::2] & 15) | (q[:, 1::2] << 4)).view(torch.uint8).contiguous(), s


class FeedForward:
    """y = down(silu(gate(n)) * up(n)), n = norm(x + residual); gate and up are one matrix."""

    def __init__(self, width, hidden, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.width, self.hidden = width, hidden
        self.norm = (1 + 0.1 * torch.randn(width, generator=g, device=device)).bfloat16()
        self.gate_up = quantise(torch.randn(2 * hidden, width, generator=g, device=device) * width ** -0.5)
        self.down = quantise(torch.randn(width, hidden, generator=g, device=device) * hidden ** -0.5)
        self.wide = None

    def decode(self, x, residual):
        """A few rows: (y, the new residual)."""
        M, dev = x.shape[0], x.device
        st = torch.cuda.current_stream().cuda_stream
        n = torch.empty(M, self.width, dtype=torch.float8_e4m3fn, device=dev)
        scale = torch.empty(M, device=dev)
        gt.gt_rmsnorm(gt.make_rmsnorm_desc(x, self.norm, n, residual=residual, sum_out=residual, row_scale=scale, quant="row",
                                           eps=EPS, stream=st))
        gu = torch.empty(M, 2 * self.hidden, dtype=torch.bfloat16, device=dev)
        gt.gt_w4_matmul(gt.make_w4_desc(n, *self.gate_up, gu, group=GROUP, row_scale=scale, stream=st))
        act = torch.nn.functional.silu(gu[:, :self.hidden].float()).mul_(gu[:, self.hidden:]).bfloat16()
        y = torch.empty(M, self.width, dtype=torch.bfloat16, device=dev)
        gt.gt_w4_matmul(gt.make_w4_desc(act, *self.down, y, group=GROUP, stream=st))
        return y, residual

    def prompt(self, x, residual):
        """Many rows: (y, the new residual).  The first call expands the weights."""
        M, dev = x.shape[0], x.device
        st = torch.cuda.current_stream().cuda_stream
        gt.gt_set_stream(st)
        if self.wide is None:
            self.wide = []
            for q, s in (self.gate_up, self.down):
                w = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.bfloat16, device=dev)
                gt.gt_w4_expand(gt.make_w4_expand_desc(q, s, w, group=GROUP, stream=st))
                self.wide.append(w)
        n = torch.empty(M, self.width, dtype=torch.bfloat16, device=dev)
        gt.gt_rmsnorm(gt.make_rmsnorm_desc(x, self.norm, n, residual=residual, sum_out=residual, eps=EPS, stream=st))
        gu = torch.empty(M, 2 * self.hidden, dtype=torch.bfloat16, device=dev)
        gt.gemm_tuned(n, self.wide[0], gu, M, 2 * self.hidden, self.width, "NT", "bf16")
        act = torch.nn.functional.silu(gu[:, :self.hidden].float()).mul_(gu[:, self.hidden:]).bfloat16()
        y = torch.empty(M, self.width, dtype=torch.bfloat16, device=dev)
        gt.gemm_tuned(act, self.wide[1], y, M, self.width, self.hidden, "NT", "bf16")
        return y, residual


class RmsNorm(torch.autograd.Function):
    """(norm(x + residual), x + residual) with the library's backward pass,
    which has no derivative of its own."""

    @staticmethod
    def forward(ctx, x, residual, weight):
        y, h = torch.empty_like(x), torch.empty_like(x)
        rstd = torch.empty(x.shape[0], device=x.device)
        gt.gt_rmsnorm(gt.make_rmsnorm_desc(x, weight, y, residual=residual, sum_out=h, rstd=rstd, eps=EPS,
                                           stream=torch.cuda.current_stream().cuda_stream))
        ctx.save_for_backward(h, weight, rstd)
        return y, h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dh):
        h, weight, rstd = ctx.saved_tensors
        dx, dw = torch.empty_like(h), torch.empty_like(weight)
        gt.gt_rmsnorm_backward(gt.make_rmsnorm_bwd_desc(dy.contiguous(), h, weight, rstd, dx, dw, dsum=dh.contiguous(),
                                                        stream=torch.cuda.current_stream().cuda_stream))
        return dx, dx, dw


def main(tokens=16, width=4096, hidden=16384):
    ff = FeedForward(width, hidden)
    x = torch.randn(tokens, width, device="cuda").bfloat16()
    r = torch.randn(tokens, width, device="cuda").bfloat16()
    few, _ = ff.decode(x, r.clone())
    many, _ = ff.prompt(x, r.clone())
    apart = ((few.float() - many.float()).norm() / many.float().norm()).item()
    print("%d tokens, %d -> 2 x %d -> %d: the two paths are %.3f %% apart (e4m3 rows)" % (tokens, width, hidden, width, 100 * apart))
    for name, path in (("decode", ff.decode), ("prompt", ff.prompt)):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        for _ in range(3):
            path(x, r)
        a.record()
        for _ in range(20):
            path(x, r)
        b.record()
        b.synchronize()
        print("%s path: %.1f us a block" % (name, a.elapsed_time(b) / 20 * 1e3))
    return apart


if __name__ == "__main__":
    main(*(int(v) for v in sys.argv[1:]))
