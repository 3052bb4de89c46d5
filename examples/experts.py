"""A block of a mixture-of-experts model for a decode batch whose requests have
adapters of their own, on the library's operators: a projection with 4-bit
weights, the requests' adapters beside it, the norm, the router's product, the
choice of experts and their layer.

    python examples/experts.py [tokens]

The block can be captured into a graph (one call before makes the stream's
workspaces and tunes the router's product); the script prints the time of one
block, called and replayed.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_autotuning_amd as gt  # noqa: E402

GROUP, EPS = 128, 1e-6


def quantise(w):
    """Rows of K as two's complement nibbles (even k low) and bf16 scales per group of k."""
    g = w.float().unflatten(-1, (-1, GROUP))
    s = (g.abs().amax(dim=-1) / 7.0).clamp(min=1e-8).bfloat16()
    q = (g / s.float()[..., None]).round().clamp(-8, 7).to(torch.int8).flatten(-2)
    return ((q[..., 0::2] & 15) | (q[..., 1::2] << 4)).view(torch.uint8).contiguous(), s


class Block:
    """h = residual + proj(x) + adapter(x); y = h + experts(norm(h)), written over the residual."""

    def __init__(self, width, hidden, experts, topk, adapters, rank, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5

        self.width, self.experts, self.topk = width, experts, topk
        self.proj = quantise(normal(width, width))
        self.a, self.b = normal(adapters, rank, width).bfloat16(), normal(adapters, width, rank).bfloat16()
        self.scale = torch.rand(adapters, generator=g, device=device)
        self.norm = (1 + 0.1 * torch.randn(width, generator=g, device=device)).bfloat16()
        self.router = normal(experts, width).bfloat16()
        self.gate_up = quantise(normal(experts, 2 * hidden, width))
        self.down = quantise(normal(experts, width, hidden))

    def buffers(self, tokens):
        """What a block of so many tokens writes, kept by the caller over calls and replays."""
        dev, wide = self.norm.device, (tokens, self.width)
        return dict(o=torch.empty(wide, dtype=torch.bfloat16, device=dev), n=torch.empty(wide, dtype=torch.bfloat16, device=dev),
                    logits=torch.empty(tokens, self.experts, dtype=torch.bfloat16, device=dev),
                    index=torch.empty(tokens, self.topk, dtype=torch.int32, device=dev),
                    weight=torch.empty(tokens, self.topk, device=dev))

    def __call__(self, x, adapter, residual, t):
        """x and residual tokens x width, adapter (int32) each token's own or -1; the block's result replaces residual."""
        st = torch.cuda.current_stream().cuda_stream
        gt.gt_w4_matmul(gt.make_w4_desc(x, *self.proj, t["o"], group=GROUP, stream=st))
        gt.gt_lora(gt.make_lora_desc(x, adapter, self.a, self.b, t["o"], base=t["o"], scale=self.scale, stream=st))
        gt.gt_rmsnorm(gt.make_rmsnorm_desc(t["o"], self.norm, t["n"], residual=residual, sum_out=residual, eps=EPS, stream=st))
        gt.gemm_tuned_ex(gt.make_desc(t["n"], self.router, t["logits"], x.shape[0], self.experts, self.width, "NT", "bf16", stream=st))
        gt.gt_route(gt.make_route_desc(t["logits"], t["index"], t["weight"], stream=st))
        gt.gt_moe(gt.make_moe_desc(t["n"], t["index"], t["weight"], self.gate_up[0], self.down[0], residual, base=residual,
                                   gate_up_scales=self.gate_up[1], down_scales=self.down[1], format="int4", group=GROUP, stream=st))
        return residual


def main(tokens=16, width=2048, hidden=768, experts=128, topk=8, adapters=8, rank=16):
    block = Block(width, hidden, experts, topk, adapters, rank)
    x = torch.randn(tokens, width, device="cuda").bfloat16()
    adapter = torch.arange(tokens, device="cuda", dtype=torch.int32) % (adapters + 1) - 1
    start = torch.randn(tokens, width, device="cuda").bfloat16()
    r, t = start.clone(), block.buffers(tokens)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        called = block(x, adapter, r, t).clone()
        st.synchronize()
        with torch.cuda.graph(graph, stream=st):
            block(x, adapter, r, t)
        r.copy_(start)
        graph.replay()
        st.synchronize()
        assert torch.equal(called, r)
        for name, run in (("called", lambda: block(x, adapter, r, t)), ("replayed", graph.replay)):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            for _ in range(3):
                run()
            a.record()
            for _ in range(20):
                run()
            b.record()
            b.synchronize()
            print("%d tokens, %d of %d experts %d x %d, %s: %.1f us a block" % (
                tokens, topk, experts, width, hidden, name, a.elapsed_time(b) / 20 * 1e3))
    return called


if __name__ == "__main__":
    main(*(int(v) for v in sys.argv[1:]))
