"""Measured cases of the operators around the matrix product: the RMS norm with
the residual's addition (in the product's types, or in e4m3 with scales), its
backward pass, the product of a few rows with 4-bit weights and group scales,
and the expansion of such weights for gemm_tuned.

Plain form (own = False): elementary torch operations in 32 bits, rounded once
at the end.  The library's form (own = True): the calls of its Python binding
on the descriptors a serving or training program keeps.
"""
import math

import torch

own = False

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
E4M3_MAX = 448.0
AMAX_LEAST = 2.0 ** -100  # a row of smaller values is scaled as if its largest were this
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def norm(name, M, N, dtype, out, quant="none", residual=True, weight="same", offset=0.0, pad=0):
    return dict(name=name, op="norm", M=M, N=N, dtype=dtype, out=out, quant=quant, residual=residual,
                weight=dtype if weight == "same" else weight, offset=offset, pad=pad)


def grad(name, M, N, dtype, dsum=True, weight="same", offset=0.0, pad=0):
    return dict(name=name, op="norm_grad", M=M, N=N, dtype=dtype, dsum=dsum,
                weight=dtype if weight == "same" else weight, offset=offset, pad=pad)


def w4(name, M, N, K, x, out, fmt, group, scales, pad=0):
    return dict(name=name, op="w4", M=M, N=N, K=K, x=x, out=out, format=fmt, group=group, scales=scales, pad=pad)


def expand(name, N, K, out, fmt, group, scales):
    return dict(name=name, op="expand", N=N, K=K, out=out, format=fmt, group=group, scales=scales)


def listed():
    return [
        # one token of a serving loop: the residual stream's addition and the e4m3 row of the next product
        norm("norm_token", 1, 4096, "bf16", "e4m3", "row"),
        # a ragged batch of requests, the activation scale fixed by calibration, rows inside a wider buffer
        norm("norm_batch", 37, 5001, "f16", "e4m3", "tensor", pad=7),
        # a prompt, or a training step's forward pass
        norm("norm_prompt", 8192, 4096, "bf16", "bf16"),
        # the gradient for a few sequences of a small model
        grad("grad_small", 500, 1000, "f16", dsum=False, weight="f32"),
        # a training step: the residual path's gradient joins in the same pass
        grad("grad_train", 8192, 4096, "bf16"),
        # the smallest projection: one token, where the launch and the latency count
        w4("w4_token_small", 1, 1024, 1024, "bf16", "bf16", "int4", 128, "bf16"),
        # one token through a feed-forward projection
        w4("w4_token", 1, 16384, 4096, "bf16", "bf16", "int4", 128, "f16"),
        # a decode batch on e4m3 rows (as the norm writes them) with small-group floating 4-bit weights
        w4("w4_batch_e4m3", 16, 8192, 8192, "e4m3", "bf16", "e2m1", 32, "bf16"),
        # a large decode batch, sizes that no tile divides
        w4("w4_rows_odd", 61, 11001, 4100, "f16", "f32", "int4", 64, "f32", pad=3),
        # the largest: the projection to the vocabulary for a few requests
        w4("w4_head", 4, 65536, 8192, "bf16", "f32", "int4", 128, "bf16"),
        # a small odd matrix laid out for a prompt's product
        expand("expand_small", 1001, 999, "f16", "e2m1", 32, "f16"),
        # a feed-forward projection laid out for a prompt's product
        expand("expand_large", 16384, 8192, "bf16", "int4", 128, "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "w4", "w4", "expand"])
    c = {"op": op}
    if op in ("norm", "norm_grad"):
        c["N"] = _log(rng, 32, 16384)
        c["M"] = _log(rng, 1, min(16384, (1 << 25) // c["N"]))
        c["dtype"] = rng.choice(["bf16", "f16", "f32"])
        if c["dtype"] == "f32":
            c["M"] = max(1, c["M"] // 2)
        c["weight"] = rng.choice([c["dtype"], c["dtype"], "f32", "none"])
        c["offset"] = rng.choice([0.0, 0.0, 1.0]) if c["weight"] != "none" else 0.0
        c["pad"] = rng.choice([0, 0, 1, 8])
        if op == "norm":
            c["residual"] = rng.choice([True, True, False])
            c["quant"] = rng.choice(["none", "row", "tensor"])
            c["out"] = c["dtype"] if c["quant"] == "none" else "e4m3"
        else:
            c["dsum"] = rng.choice([True, False])
        return c
    c["K"] = _log(rng, 32, 16384)
    c["N"] = _log(rng, 16, min(65536, (1 << 29) // c["K"] // (1 if op == "w4" else 4)))
    c["format"] = rng.choice(["int4", "int4", "e2m1"])
    c["group"] = rng.choice([32, 64, 128, 128])
    c["scales"] = rng.choice(["bf16", "f16", "f32"])
    if op == "w4":
        c["M"] = _log(rng, 1, 64)
        if c["M"] * c["N"] * c["K"] > 1 << 32:
            c["M"] = max(1, (1 << 32) // (c["N"] * c["K"]))
        c["x"] = rng.choice(["bf16", "f16", "e4m3"])
        c["out"] = rng.choice(["bf16", "f16", "f32"] if c["x"] == "e4m3" else [c["x"], "f32"])
        c["pad"] = rng.choice([0, 0, 3, 16])
    else:
        c["out"] = rng.choice(["bf16", "f16", "f32"])
    return c


# ---- inputs


def _rows(g, M, N, pad, std=1.0):
    """M x N rows with a row stride of N + pad: normal values, and a few columns much larger than the rest."""
    x = torch.randn(M, N + pad, generator=g, device="cuda") * std
    loud = torch.randint(0, N, (max(1, N // 256),), generator=g, device="cuda")
    x[:, loud] *= 12.0
    return x


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("norm", "norm_grad"):
        M, N, pad, dt = c["M"], c["N"], c["pad"], TORCH[c["dtype"]]
        w = None
        if c["weight"] != "none":
            w = (torch.randn(N, generator=g, device="cuda") * 0.2 + (1.0 - c["offset"])).to(TORCH[c["weight"]])
        s["w"] = w
        x = _rows(g, M, N, pad).to(dt)[:, :N]
        if c["op"] == "norm":
            s["x"] = x
            s["r"] = _rows(g, M, N, pad, 3.0).to(dt)[:, :N] if c["residual"] else None
            s["scale"] = 0.05 if c["quant"] == "tensor" else 1.0
            s["eps"] = 1e-6
            # the buffers that a serving loop keeps for its results
            s["sum"] = torch.empty(M, N, dtype=dt, device="cuda") if c["residual"] else None
            s["y"] = torch.empty(M, N, dtype=TORCH[c["out"]], device="cuda")
            s["rstd"] = torch.empty(M, device="cuda")
            s["scales"] = torch.empty(M, device="cuda") if c["quant"] == "row" else None
        else:
            s["h"] = x
            h = x.float()
            s["rstd"] = torch.rsqrt((h * h).mean(dim=1) + 1e-6)
            s["dy"] = (torch.randn(M, N + pad, generator=g, device="cuda") * 0.1).to(dt)[:, :N]
            s["dsum"] = (torch.randn(M, N + pad, generator=g, device="cuda") * 0.1).to(dt)[:, :N] if c["dsum"] else None
            s["dx"] = torch.empty(M, N, dtype=dt, device="cuda")
            s["dw"] = torch.empty(N, device="cuda") if w is not None else None
    else:
        N, K, G = c["N"], c["K"], -(-c["K"] // c["group"])
        s["q"] = torch.randint(0, 256, (N, -(-K // 2)), generator=g, device="cuda", dtype=torch.uint8)
        s["s"] = (torch.exp(torch.randn(N, G, generator=g, device="cuda") * 0.3) * (0.25 / math.sqrt(K))).to(
            TORCH[c["scales"]])
        if c["op"] == "w4":
            x = _rows(g, c["M"], K, c["pad"])
            s["rs"] = None
            if c["x"] == "e4m3":
                s["rs"] = x[:, :K].abs().amax(dim=1) / E4M3_MAX
                x = (x / s["rs"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
            s["x"] = x.to(TORCH[c["x"]])[:, :K]
            s["y"] = torch.empty(c["M"], N, dtype=TORCH[c["out"]], device="cuda")
        else:
            s["y"] = torch.empty(N, K, dtype=TORCH[c["out"]], device="cuda")
    if own:  # the descriptors that a user's program builds once for its buffers; no data is read or written here
        import gemm_autotuning_amd as gt

        if c["op"] == "norm":
            s["desc"] = gt.make_rmsnorm_desc(s["x"], s["w"], s["y"], residual=s["r"], sum_out=s["sum"], rstd=s["rstd"],
                                             row_scale=s["scales"], quant=c["quant"], eps=s["eps"], scale=s["scale"],
                                             weight_offset=c["offset"])
        elif c["op"] == "norm_grad":
            s["desc"] = gt.make_rmsnorm_bwd_desc(s["dy"], s["h"], s["w"], s["rstd"], s["dx"], dweight=s["dw"],
                                                 dsum=s["dsum"], weight_offset=c["offset"])
        elif c["op"] == "w4":
            s["desc"] = gt.make_w4_desc(s["x"], s["q"], s["s"], s["y"], format=c["format"], group=c["group"],
                                        row_scale=s["rs"])
        else:
            s["desc"] = gt.make_w4_expand_desc(s["q"], s["s"], s["y"], format=c["format"], group=c["group"])
    return s


# ---- one pass


def _values(q, K, fmt, dtype):
    """The N x K values that the nibbles stand for: the low one of a byte is the even k."""
    code = torch.stack((q & 15, q >> 4), dim=2).reshape(q.shape[0], -1)[:, :K]
    if fmt == "int4":
        v = code.to(dtype)
        return torch.where(v >= 8, v - 16, v)
    mag = torch.tensor(E2M1, dtype=dtype, device=q.device)[(code & 7).int()]
    return torch.where(code >= 8, -mag, mag)


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        h = s["x"].float()
        if s["r"] is not None:
            h = h + s["r"].float()
        rstd = 1.0 / torch.sqrt((h * h).mean(dim=1) + s["eps"])
        y = h * rstd[:, None]
        if s["w"] is not None:
            y = y * (s["w"].float() + c["offset"])
        out = {"rstd": rstd}
        if s["r"] is not None:
            out["sum"] = h.to(s["x"].dtype)
        if c["quant"] == "row":
            out["scales"] = y.abs().amax(dim=1).clamp(min=AMAX_LEAST) / E4M3_MAX
            y = y / out["scales"][:, None]
        elif c["quant"] == "tensor":
            y = (y / s["scale"]).clamp(-E4M3_MAX, E4M3_MAX)
        out["y"] = y.to(TORCH[c["out"]])
        return out
    if c["op"] == "norm_grad":
        dy, xh = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
        g = dy * (s["w"].float() + c["offset"]) if s["w"] is not None else dy
        dx = s["rstd"][:, None] * (g - xh * (g * xh).mean(dim=1, keepdim=True))
        if s["dsum"] is not None:
            dx = dx + s["dsum"].float()
        out = {"dx": dx.to(s["h"].dtype)}
        if s["w"] is not None:
            out["dw"] = (dy * xh).sum(dim=0)
        return out
    w = _values(s["q"], c["K"], c["format"], torch.float32)
    w = w * s["s"].float().repeat_interleave(c["group"], dim=1)[:, :c["K"]]
    if c["op"] == "expand":
        return {"y": w.to(TORCH[c["out"]])}
    y = s["x"].float() @ w.t()
    if s["rs"] is not None:
        y = y * s["rs"][:, None]
    return {"y": y.to(TORCH[c["out"]])}


def run(state):
    if not own:
        return _plain(state)
    import gemm_autotuning_amd as gt

    c = state["case"]
    if c["op"] == "norm":
        gt.gt_rmsnorm(state["desc"])
        return {k: state[k] for k in ("rstd", "sum", "scales", "y") if state[k] is not None}
    if c["op"] == "norm_grad":
        gt.gt_rmsnorm_backward(state["desc"])
        return {k: state[k] for k in ("dx", "dw") if state[k] is not None}
    if c["op"] == "w4":
        gt.gt_w4_matmul(state["desc"])
    else:
        gt.gt_w4_expand(state["desc"])
    return {"y": state["y"]}


def work(case):
    c = case
    if c["op"] in ("norm", "norm_grad"):
        M, N, e = c["M"], c["N"], BYTES[c["dtype"]]
        wb = N * BYTES[c["weight"]] if c["weight"] != "none" else 0
        if c["op"] == "norm":
            per = e + (2 * e if c["residual"] else 0) + BYTES[c["out"]]
            return {"bytes": M * N * per + wb + 4 * M * (2 if c["quant"] == "row" else 1), "flops": 5 * M * N}
        return {"bytes": M * N * e * (4 if c["dsum"] else 3) + wb + (4 * N if wb else 0) + 4 * M, "flops": 9 * M * N}
    N, K = c["N"], c["K"]
    weights = N * -(-K // 2) + N * -(-K // c["group"]) * BYTES[c["scales"]]
    if c["op"] == "expand":
        return {"bytes": weights + N * K * BYTES[c["out"]], "flops": N * K}
    M = c["M"]
    rows = M * K * BYTES[c["x"]] + (4 * M if c["x"] == "e4m3" else 0)
    return {"bytes": weights + rows + M * N * BYTES[c["out"]], "flops": 2 * M * N * K}


# ---- the definition in 64 bits, written with a table of the codes' values and sums taken group by group


def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    d = torch.float64
    if c["op"] == "norm":
        h = s["x"].to(d) if s["r"] is None else s["x"].to(d).add(s["r"].to(d))
        rstd = (h.square().sum(dim=1) / c["N"] + s["eps"]).pow(-0.5)
        gain = torch.ones(c["N"], dtype=d, device="cuda") if s["w"] is None else s["w"].to(d) + c["offset"]
        y = torch.einsum("mn,m,n->mn", h, rstd, gain)
        out = {"rstd": rstd}
        if s["r"] is not None:
            out["sum"] = h
        if c["quant"] == "row":
            out["scales"] = torch.maximum(y.abs().max(dim=1).values, torch.full_like(rstd, AMAX_LEAST)) / E4M3_MAX
            y = y / out["scales"].unsqueeze(1)
        elif c["quant"] == "tensor":
            y = torch.minimum(torch.maximum(y / s["scale"], torch.full_like(y, -E4M3_MAX)), torch.full_like(y, E4M3_MAX))
        out["y"] = y
        return out
    if c["op"] == "norm_grad":
        # y_j = h_j r gain_j with r = (mean h^2 + eps)^(-1/2): dy_j/dh_i = r gain_j (i == j) - h_j gain_j h_i r^3 / N
        h, r, dy = s["h"].to(d), s["rstd"].to(d).unsqueeze(1), s["dy"].to(d)
        gain = torch.ones(c["N"], dtype=d, device="cuda") if s["w"] is None else s["w"].to(d) + c["offset"]
        dot = (dy * h) @ gain
        dx = dy * gain * r - h * (r.pow(3) * dot.unsqueeze(1) / c["N"])
        out = {"dx": dx if s["dsum"] is None else dx + s["dsum"].to(d)}
        if s["w"] is not None:
            out["dw"] = torch.mv((dy * h).t(), r.squeeze(1))
        return out
    table = [float(v) for v in range(8)] + [float(v - 16) for v in range(8, 16)]
    if c["format"] == "e2m1":
        table = list(E2M1) + [-v for v in E2M1]
    table = torch.tensor(table, dtype=d, device="cuda")
    N, K, G = c["N"], c["K"], c["group"]
    out = torch.zeros(c["M"] if c["op"] == "w4" else N, N if c["op"] == "w4" else K, dtype=d, device="cuda")
    for g in range(-(-K // G)):
        k0, k1 = g * G, min(K, g * G + G)
        b = s["q"][:, k0 // 2:(k1 + 1) // 2].long()
        v = torch.empty(N, 2 * b.shape[1], dtype=d, device="cuda")
        v[:, 0::2] = table[b % 16]
        v[:, 1::2] = table[b // 16]
        v = v[:, :k1 - k0] * s["s"][:, g].to(d).unsqueeze(1)
        if c["op"] == "w4":
            out += s["x"][:, k0:k1].to(d) @ v.t()
        else:
            out[:, k0:k1] = v
    if c["op"] == "w4" and s["rs"] is not None:
        out = out * s["rs"].to(d).unsqueeze(1)
    return {"y": out}
