"""Measured cases of what a decode batch meets beside its products: the choice
of experts from a router's logits, a whole layer of gated experts for a few
tokens (16-bit or 4-bit weights), and the low-rank adapters of many requests
beside a shared projection.

Plain form (own = False): elementary torch operations in 32 bits, rounded once
at the end.  The library's form (own = True): the calls of its Python binding
on the descriptors a serving program keeps.
"""
import math

import torch

own = False

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def route(name, M, E, k, dtype, score="softmax", normalise=True, scale=1.0, masked=False, pad=0):
    return dict(name=name, op="route", M=M, E=E, k=k, dtype=dtype, score=score, normalise=normalise, scale=scale,
                masked=masked, pad=pad)


def moe(name, T, E, k, K, H, dtype, out, fmt="none", group=128, scales="bf16", act="silu", base=True, absent=False, pad=0):
    return dict(name=name, op="moe", T=T, E=E, k=k, K=K, H=H, dtype=dtype, out=out, format=fmt, group=group, scales=scales,
                act=act, base=base, absent=absent, pad=pad)


def lora(name, M, L, r, K, N, dtype, out, requests="rows", base=True, scaled=True, pad=0):
    return dict(name=name, op="lora", M=M, L=L, r=r, K=K, N=N, dtype=dtype, out=out, requests=requests, base=base,
                scaled=scaled, pad=pad)


def listed():
    return [
        # one token's experts, from a router's product in fp32
        route("route_token", 1, 128, 8, "f32"),
        # a ragged batch, sigmoid scores, experts masked out (a device that is full, or absent)
        route("route_odd", 513, 77, 3, "f16", score="sigmoid", scale=2.5, masked=True, pad=3),
        # a prompt's tokens over many experts
        route("route_prompt", 8192, 256, 8, "bf16", normalise=False),
        # one token through a layer of many small experts
        moe("moe_token", 1, 128, 8, 2048, 768, "bf16", "bf16"),
        # one token through a layer of fewer, larger experts with 4-bit weights
        moe("moe_token_int4", 1, 64, 4, 4096, 2048, "bf16", "bf16", fmt="int4", scales="f16"),
        # a decode batch: most experts have a row or two
        moe("moe_batch", 16, 32, 4, 4096, 1024, "bf16", "bf16"),
        # sizes that no tile divides, small groups of floating 4-bit weights, slots that another device serves
        moe("moe_odd", 37, 20, 3, 1001, 999, "f16", "f32", fmt="e2m1", group=32, scales="f32", act="gelu", base=False,
            absent=True, pad=3),
        # the largest: a large decode batch over large 4-bit experts, about eight rows to each
        moe("moe_large", 64, 64, 8, 4096, 2048, "bf16", "bf16", fmt="int4", group=64),
        # one token of one request beside an attention projection
        lora("lora_token", 1, 8, 16, 4096, 4096, "bf16", "bf16"),
        # a decode batch of requests with adapters of their own beside a feed-forward projection
        lora("lora_batch", 48, 64, 64, 4096, 16384, "bf16", "bf16"),
        # odd sizes, some requests without an adapter, the adapters' part alone
        lora("lora_odd", 77, 5, 12, 1001, 999, "f16", "f32", base=False, scaled=False, pad=5),
        # prompts of several requests: long runs of rows with one adapter
        lora("lora_prompt", 4096, 6, 32, 4096, 4096, "bf16", "bf16", requests="runs"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    case = _draw(rng)
    del case["name"]
    return case


def _draw(rng):
    op = rng.choice(["route", "moe", "moe", "lora", "lora"])
    if op == "route":
        E = _log(rng, 4, 512)
        return route("", _log(rng, 1, 16384), E, _log(rng, 1, min(E, 16)), rng.choice(["f32", "bf16", "f16"]),
                     rng.choice(["softmax", "softmax", "sigmoid"]), rng.choice([True, False]), rng.choice([1.0, 2.5]),
                     rng.choice([True, False]), rng.choice([0, 0, 1, 8]))
    dt = rng.choice(["bf16", "bf16", "f16"])
    out, base, pad = rng.choice([dt, dt, "f32"]), rng.choice([True, False]), rng.choice([0, 0, 3, 16])
    if op == "moe":
        K, H = _log(rng, 64, 8192), _log(rng, 64, 8192)
        most = (1 << 29) // (3 * K * H)  # experts of at most half a billion weights together
        E = _log(rng, 1, max(1, min(256, most)))
        return moe("", _log(rng, 1, 128), E, _log(rng, 1, min(E, 8)), K, H, dt, out, rng.choice(["none", "none", "int4", "e2m1"]),
                   rng.choice([32, 64, 128]), rng.choice(["bf16", "f16", "f32"]), rng.choice(["silu", "silu", "gelu"]), base,
                   rng.choice([True, False]), pad)
    K, N, r = _log(rng, 64, 16384), _log(rng, 64, 16384), _log(rng, 4, 128)
    M = _log(rng, 1, min(4096, (1 << 25) // max(K, N)))
    return lora("", M, _log(rng, 1, 64), r, K, N, dt, out, rng.choice(["rows", "runs"]), base, rng.choice([True, False]), pad)


# ---- inputs


def _rows(g, M, N, pad):
    """M x N rows with a row stride of N + pad: normal values, and a few columns much larger than the rest."""
    x = torch.randn(M, N + pad, generator=g, device="cuda")
    loud = torch.randint(0, N, (max(1, N // 256),), generator=g, device="cuda")
    x[:, loud] *= 12.0
    return x


def _nibbles(g, E, N, K, c):
    """E matrices N x K in 4 bits, and their scales per group of k."""
    q = torch.randint(0, 256, (E, N, -(-K // 2)), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.exp(torch.randn(E, N, -(-K // c["group"]), generator=g, device="cuda") * 0.3) * (0.25 / math.sqrt(K))
    return q, s.to(TORCH[c["scales"]])


def _normal(g, shape, std, dtype):
    """Normal values, matrix by matrix (no fp32 copy of the whole)."""
    out = torch.empty(shape, dtype=TORCH[dtype], device="cuda")
    for m in out:
        m.copy_(torch.randn(m.shape, generator=g, device="cuda") * std)
    return out


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "route":
        l = torch.randn(c["M"], c["E"] + c["pad"], generator=g, device="cuda") * 2.0
        l = l + torch.randn(c["E"] + c["pad"], generator=g, device="cuda")  # experts are not equally popular
        if c["masked"]:
            l[torch.rand(l.shape, generator=g, device="cuda") < 0.25] = -math.inf
            l[: max(1, c["M"] // 64)] = -math.inf  # rows whose mask leaves nothing
        s["logits"] = l.to(TORCH[c["dtype"]])[:, :c["E"]]
        s["index"] = torch.empty(c["M"], c["k"], dtype=torch.int32, device="cuda")
        s["weight"] = torch.empty(c["M"], c["k"], device="cuda")
    elif c["op"] == "moe":
        T, E, k, K, H, dt = c["T"], c["E"], c["k"], c["K"], c["H"], c["dtype"]
        s["x"] = _rows(g, T, K, c["pad"]).to(TORCH[dt])[:, :K]
        score = torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
        top = torch.sort(torch.softmax(score, dim=1), dim=1, descending=True, stable=True)
        s["weight"] = (top.values[:, :k] / top.values[:, :k].sum(dim=1, keepdim=True)).contiguous()
        s["index"] = top.indices[:, :k].int().contiguous()
        if c["absent"]:
            s["index"][torch.rand(T, k, generator=g, device="cuda") < 0.2] = -1
        s["gs"] = s["ds"] = None
        if c["format"] == "none":
            s["gate_up"] = _normal(g, (E, 2 * H, K), K ** -0.5, dt)
            s["down"] = _normal(g, (E, K, H), H ** -0.5, dt)
        else:
            s["gate_up"], s["gs"] = _nibbles(g, E, 2 * H, K, c)
            s["down"], s["ds"] = _nibbles(g, E, K, H, c)
        s["base"] = torch.randn(T, K, generator=g, device="cuda").to(TORCH[c["out"]]) if c["base"] else None
        s["y"] = torch.empty(T, K, dtype=TORCH[c["out"]], device="cuda")
    else:
        M, L, r, K, N, dt = c["M"], c["L"], c["r"], c["K"], c["N"], c["dtype"]
        s["x"] = _rows(g, M, K, c["pad"]).to(TORCH[dt])[:, :K]
        s["a"] = _normal(g, (L, r, K), K ** -0.5, dt)
        s["b"] = _normal(g, (L, N, r), r ** -0.5, dt)
        s["scale"] = torch.rand(L, generator=g, device="cuda") * 1.5 + 0.5 if c["scaled"] else None
        # an adapter of each request, and for about one in eight none
        n = M if c["requests"] == "rows" else min(M, 8)
        of = torch.randint(0, L, (n,), generator=g, device="cuda", dtype=torch.int32)
        of[torch.rand(n, generator=g, device="cuda") < 0.125] = -1
        s["index"] = of if n == M else of.repeat_interleave(-(-M // n))[:M].contiguous()
        s["base"] = torch.randn(M, N, generator=g, device="cuda").to(TORCH[c["out"]]) if c["base"] else None
        s["y"] = torch.empty(M, N, dtype=TORCH[c["out"]], device="cuda")
    if own:  # the descriptors that a user's program builds once for its buffers; no data is read or written here
        import gemm_autotuning_amd as gt

        if c["op"] == "route":
            s["desc"] = gt.make_route_desc(s["logits"], s["index"], s["weight"], score=c["score"], normalise=c["normalise"],
                                           scale=c["scale"])
        elif c["op"] == "moe":
            s["desc"] = gt.make_moe_desc(s["x"], s["index"], s["weight"], s["gate_up"], s["down"], s["y"], base=s["base"],
                                         gate_up_scales=s["gs"], down_scales=s["ds"], format=c["format"], group=c["group"],
                                         activation=c["act"])
        else:
            s["desc"] = gt.make_lora_desc(s["x"], s["index"], s["a"], s["b"], s["y"], base=s["base"], scale=s["scale"])
    return s


# ---- one pass


def _values(q, scales, K, fmt, group):
    """The E x N x K weights in 32 bits: the low nibble of a byte is the even k."""
    if fmt == "none":
        return q.float()
    code = torch.stack((q & 15, q >> 4), dim=3).reshape(q.shape[0], q.shape[1], -1)[:, :, :K]
    if fmt == "int4":
        v = ((code ^ 8).float()) - 8.0
    else:
        v = torch.tensor(list(E2M1) + [-m for m in E2M1], device=q.device)[code.int()]
    return v * scales.float().repeat_interleave(group, dim=2)[:, :, :K]


def _activated(g, u, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g)) * u
    # the tanh form: g (1 + tanh z) / 2 = g / (1 + exp(-2 z)), z = sqrt(2 / pi) (g + 0.044715 g^3)
    return g / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g))) * u


def _plain(s):
    c = s["case"]
    if c["op"] == "route":
        l = s["logits"].float()
        top = torch.sort(l, dim=1, descending=True, stable=True)
        chosen, index = top.values[:, :c["k"]], top.indices[:, :c["k"]].int()
        left = chosen > -math.inf
        if c["score"] == "softmax":
            most = top.values[:, :1].clamp(min=torch.finfo(torch.float32).min)
            w = torch.exp(chosen - most)
            total = w.sum(dim=1, keepdim=True) if c["normalise"] else torch.exp(l - most).sum(dim=1, keepdim=True)
            w = w / total
        else:
            w = 1.0 / (1.0 + torch.exp(-chosen))
            if c["normalise"]:
                w = w / w.sum(dim=1, keepdim=True)
        return {"index": torch.where(left, index, -1), "weight": torch.where(left, w * c["scale"], 0.0)}
    if c["op"] == "moe":
        T, E, k, K, H = c["T"], c["E"], c["k"], c["K"], c["H"]
        x, here = s["x"].float(), (s["index"] >= 0) & (s["index"] < E)
        if T * k <= E:  # the slots' own experts; each row of x meets its k of them
            e = s["index"].clamp(min=0).flatten().long()
            gu = _values(s["gate_up"][e], None if s["gs"] is None else s["gs"][e], K, c["format"], c["group"])
            h = torch.bmm(gu, x.repeat_interleave(k, dim=0).unsqueeze(2)).squeeze(2)
            h = _activated(h[:, :H], h[:, H:], c["act"])
            dn = _values(s["down"][e], None if s["ds"] is None else s["ds"][e], H, c["format"], c["group"])
            w = torch.where(here, s["weight"], 0.0)
            y = (torch.bmm(dn, h.unsqueeze(2)).reshape(T, k, K) * w.unsqueeze(2)).sum(dim=1)
        else:  # every expert on every row, and the weights of those that are not chosen are zero
            w = torch.zeros(T, E, device=x.device).scatter_add_(1, s["index"].clamp(min=0).long(),
                                                                torch.where(here, s["weight"], 0.0))
            h = (x @ _values(s["gate_up"], s["gs"], K, c["format"], c["group"]).reshape(E * 2 * H, K).t()).reshape(T, E, 2 * H)
            h = _activated(h[:, :, :H], h[:, :, H:], c["act"]) * w.unsqueeze(2)
            dn = _values(s["down"], s["ds"], H, c["format"], c["group"])
            y = h.reshape(T, E * H) @ dn.transpose(1, 2).reshape(E * H, K)
    else:
        M, L, r, K, N = c["M"], c["L"], c["r"], c["K"], c["N"]
        mine = (s["index"].unsqueeze(1) == torch.arange(L, device=s["x"].device)).float()
        if s["scale"] is not None:
            mine = mine * s["scale"]
        h = (s["x"].float() @ s["a"].float().reshape(L * r, K).t()).reshape(M, L, r) * mine.unsqueeze(2)
        y = h.reshape(M, L * r) @ s["b"].float().transpose(1, 2).reshape(L * r, N)
    if s["base"] is not None:
        y = y + s["base"].float()
    return {"y": y.to(TORCH[c["out"]])}


def run(state):
    if not own:
        return _plain(state)
    import gemm_autotuning_amd as gt

    op = state["case"]["op"]
    if op == "route":
        gt.gt_route(state["desc"])
        return {"index": state["index"], "weight": state["weight"]}
    if op == "moe":
        gt.gt_moe(state["desc"])
    else:
        gt.gt_lora(state["desc"])
    return {"y": state["y"]}


def _active(n, draws, each=1):
    """How many of n experts are expected to be met by so many draws of `each` different ones."""
    return n * (1.0 - (1.0 - each / n) ** draws)


def work(case):
    c = case
    if c["op"] == "route":
        return {"bytes": c["M"] * (c["E"] * BYTES[c["dtype"]] + 8 * c["k"]), "flops": 4 * c["M"] * c["E"]}
    if c["op"] == "moe":
        T, K, H = c["T"], c["K"], c["H"]
        pairs = T * c["k"] * (0.8 if c["absent"] else 1.0)
        met = _active(c["E"], T * (0.8 if c["absent"] else 1.0), c["k"])
        if c["format"] == "none":
            each = 3 * K * H * BYTES[c["dtype"]]
        else:
            each = 2 * H * (-(-K // 2)) + K * (-(-H // 2))
            each += (2 * H * -(-K // c["group"]) + K * -(-H // c["group"])) * BYTES[c["scales"]]
        rows = T * K * (BYTES[c["dtype"]] + BYTES[c["out"]] * (2 if c["base"] else 1)) + 8 * T * c["k"]
        return {"bytes": int(met * each) + rows, "flops": int(6 * pairs * K * H)}
    M, K, N, r = c["M"], c["K"], c["N"], c["r"]
    met = _active(c["L"], 0.875 * (M if c["requests"] == "rows" else min(M, 8)))
    rows = M * (int(0.875 * K) * BYTES[c["dtype"]] + N * BYTES[c["out"]] * (2 if c["base"] else 1)) + 4 * M
    return {"bytes": int(met * r * (K + N) * BYTES[c["dtype"]]) + rows, "flops": int(1.75 * M * r * (K + N))}


# ---- the definition in 64 bits, one expert or adapter after another


def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    d = torch.float64
    if c["op"] == "route":
        # one choice after another: the first of the largest that is left
        l = s["logits"].to(d)
        at, index, weight = torch.arange(c["M"], device="cuda"), [], []
        rest = l.clone()
        taken = torch.zeros_like(l, dtype=torch.bool)
        for _ in range(c["k"]):
            most = rest.max(dim=1, keepdim=True).values
            i = ((rest == most) & ~taken).int().argmax(dim=1)
            gone = most.squeeze(1) == -math.inf
            index.append(torch.where(gone, -1, i).int())
            weight.append(torch.where(gone, -math.inf, l[at, i]))
            rest[at, i] = -math.inf
            taken[at, i] = True
        index, chosen = torch.stack(index, dim=1), torch.stack(weight, dim=1)
        if c["score"] == "softmax":
            w = (chosen - torch.logsumexp(chosen if c["normalise"] else l, dim=1, keepdim=True)).exp()
        else:
            w = torch.special.expit(chosen)
            if c["normalise"]:
                w = w / w.sum(dim=1, keepdim=True)
        return {"index": index, "weight": torch.where(index < 0, 0.0, w * c["scale"])}
    table = torch.tensor([float(v if v < 8 else v - 16) for v in range(16)] if c.get("format") == "int4" else
                         list(E2M1) + [-v for v in E2M1], dtype=d, device="cuda")

    def matrix(w, sc, e, K):
        if c["op"] == "lora" or c["format"] == "none":
            return w[e].to(d)
        v = torch.empty(w.shape[1], 2 * w.shape[2], dtype=d, device="cuda")
        v[:, 0::2] = table[(w[e] % 16).long()]
        v[:, 1::2] = table[(w[e] // 16).long()]
        k = torch.arange(K, device="cuda") // c["group"]
        return v[:, :K] * sc[e].to(d)[:, k]

    x = s["x"].to(d)
    y = torch.zeros(s["y"].shape, dtype=d, device="cuda") if s["base"] is None else s["base"].to(d).clone()
    for e in range(c["E"] if c["op"] == "moe" else c["L"]):
        if c["op"] == "lora":
            rows = torch.nonzero(s["index"] == e).squeeze(1)
            f = 1.0 if s["scale"] is None else s["scale"][e].to(d)
            if rows.numel():
                y[rows] += f * (x[rows] @ s["a"][e].to(d).t()) @ s["b"][e].to(d).t()
            continue
        rows, slot = torch.nonzero(s["index"] == e, as_tuple=True)
        if not rows.numel():
            continue
        gu = x[rows] @ matrix(s["gate_up"], s["gs"], e, c["K"]).t()
        a, u = gu[:, :c["H"]], gu[:, c["H"]:]
        if c["act"] == "silu":
            h = a * torch.special.expit(a) * u
        else:
            h = 0.5 * a * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (a + 0.044715 * a ** 3))) * u
        y.index_add_(0, rows, (h @ matrix(s["down"], s["ds"], e, c["H"]).t()) * s["weight"][rows, slot].to(d).unsqueeze(1))
    return {"y": y}
