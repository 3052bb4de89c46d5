"""Experts and adapters beside the product in 64 bits, on the CPU, with how far
a result computed as the library does may be from them (u = 2^-24, fp32's
half step).

A dot product of n terms summed in fp32 in any of the kernels' orders is off
by at most dot(n) u times the sum of the terms' magnitudes: the matrix core
adds 32 products at a time, so that no chain is longer than n / 32 + 200.
Between two products a value v is taken as two 16-bit parts, off by 2^-16 |v|
(bf16: 8 and 8 bits), or by 2^-21 |v| and 2^-37 of its row's largest (f16
under the row's power of two, the second part down to its least subnormal).
"""
import math

import torch

from . import op_ref as ref

U = ref.U


def dot(n):
    return (n / 32 + 200) * U


def split(v, dtype):
    if dtype == torch.bfloat16:
        return v.abs() * 2.0 ** -16
    return v.abs() * 2.0 ** -21 + v.abs().amax(dim=-1, keepdim=True) * 2.0 ** -37


def shifted(v, over):
    """exp(v) / sum exp(over), both less the largest: a logarithm of the sum
    would be lost beside values like 3e38."""
    most = over.max()
    return torch.exp(v - most) / torch.exp(over - most).sum()


def route(logits, k, score="softmax", normalise=True, scale=1.0):
    """(index, weight): one choice after another, the first of the largest that is left."""
    l = logits.double()
    M, E = l.shape
    index = torch.full((M, k), -1, dtype=torch.int32)
    weight = torch.zeros(M, k, dtype=torch.float64)
    for m in range(M):
        row = l[m].tolist()
        order = sorted((i for i in range(E) if row[i] != -math.inf),
                       key=lambda i: (0 if math.isnan(row[i]) else 1, 0.0 if math.isnan(row[i]) else -row[i], i))
        top = order[:k]
        if not top:
            continue
        index[m, :len(top)] = torch.tensor(top, dtype=torch.int32)
        chosen = l[m, top]
        if score == "softmax":
            w = shifted(chosen, chosen if normalise else l[m])
        elif normalise:  # by their logarithms, which do not run out of range
            log = torch.nn.functional.logsigmoid(chosen)
            w = shifted(log, log)
        else:
            w = torch.sigmoid(chosen)
        weight[m, :len(top)] = w * scale
    return index, weight


def weights(w, s, K, fmt, group):
    """A matrix N x K in 64 bits."""
    return w.double() if fmt == "none" else ref.w4_weights(w, s, K, fmt, group)


def activation(g, act):
    z = g if act == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
    return g * torch.special.expit(z)


def moe(x, index, weight, gate_up, down, gs=None, ds=None, fmt="none", group=128, act="silu", base=None):
    """(y, bound before the store).  An activation's slope is at most 1.13; its
    exponential, quotient and the cubic of its argument cost at most 8 u of |g|
    (an argument off by a few u moves g * sigmoid(z) by |g| |z| / (2 + 2 cosh z)
    of them, and |z| / (2 + 2 cosh z) < 0.23)."""
    T, K = x.shape
    H = gate_up.shape[1] // 2
    y = torch.zeros(T, K, dtype=torch.float64) if base is None else base.double()
    far = 2 * U * y.abs()
    for t in range(T):
        for j in range(index.shape[1]):
            e = int(index[t, j])
            if not 0 <= e < gate_up.shape[0]:
                continue
            wgu = weights(gate_up[e], None if gs is None else gs[e], K, fmt, group)
            wd = weights(down[e], None if ds is None else ds[e], H, fmt, group)
            xt = x[t].double()
            gu, mag = wgu @ xt, wgu.abs() @ xt.abs()
            g, u, a = gu[:H], gu[H:], activation(gu[:H], act)
            h = a * u
            dg, du = dot(K) * mag[:H], dot(K) * mag[H:]
            dh = (1.13 * dg + 8 * U * g.abs()) * (u.abs() + du) + a.abs() * du + 4 * U * h.abs()
            w = float(weight[t, j])
            y[t] += w * (wd @ h)
            m = wd.abs() @ h.abs()
            far[t] += abs(w) * (wd.abs() @ (dh + split(h, x.dtype)) + (dot(H) + 8 * U) * m) + 4 * U * y[t].abs()
    return y, far


def lora(x, index, a, b, scale=None, base=None):
    """(y, bound before the store)."""
    M, K = x.shape
    r = a.shape[1]
    y = torch.zeros(M, b.shape[1], dtype=torch.float64) if base is None else base.double()
    far = torch.zeros_like(y)
    for m in range(M):
        e = int(index[m])
        if not 0 <= e < a.shape[0]:
            continue
        A, B, xm = a[e].double(), b[e].double(), x[m].double()
        h, dh = A @ xm, dot(K) * (A.abs() @ xm.abs())
        f = 1.0 if scale is None else float(scale[e])
        d = B @ h
        far[m] = abs(f) * (B.abs() @ (dh + split(h, x.dtype)) + (dot(r) + 4 * U) * (B.abs() @ h.abs())) + 2 * U * y[m].abs()
        y[m] += f * d
        far[m] += 2 * U * y[m].abs()
    return y, far


# ---- inputs
def nibbles(E, N, K, group, scales, seed, codes=None):
    """Bytes of two codes each (any, or of the listed ones), and scales."""
    g = ref.rng(seed)
    if codes is None:
        q = torch.randint(0, 256, (E, N, -(-K // 2)), generator=g, dtype=torch.uint8)
    else:
        t = torch.tensor(codes, dtype=torch.uint8)
        n = t[torch.randint(0, len(codes), (2, E, N, -(-K // 2)), generator=g)]
        q = n[0] | (n[1] << 4)
    s = torch.exp(torch.randn(E, N, -(-K // group), generator=g) * 0.3) * (0.25 / math.sqrt(K))
    return q, s.to(ref.DT[scales])


def normal(shape, std, dtype, seed):
    return (torch.randn(shape, generator=ref.rng(seed)) * std).to(dtype)


def choices(T, E, k, seed, absent=False):
    """k different experts of E for each of T tokens, and their weights."""
    g = ref.rng(seed)
    index = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    if absent:
        index[torch.rand(T, k, generator=g) < 0.25] = -1
    return index, torch.rand(T, k, generator=g)
