"""The operators around the product in 64 bits, on the CPU, and how far a
result computed in fp32 and rounded once may be from them.

Bounds.  u = 2^-24 is fp32's half step.  A sum of n terms in any order is off
by at most (n - 1) u times the sum of the terms' magnitudes; where the terms
are first added in parts the largest chain counts, and the chains assumed here
(CHAIN terms per part) are longer than any the kernels form.  A store rounds
by at most finfo(t).eps / 2 of the value, or half the least subnormal.
"""
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134,
        torch.float8_e4m3fn: 2.0 ** -10}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def chain(n):
    """Longest chain of additions of a row sum: 1/64 of the row in one lane, then the joins."""
    return n / 64 + 32


def rmsnorm(x, r, w, eps=1e-6, offset=0.0):
    """(h, rstd, y) in 64 bits."""
    h = x.double() if r is None else x.double() + r.double()
    rstd = 1.0 / torch.sqrt((h * h).mean(dim=1) + eps)
    y = h * rstd[:, None]
    if w is not None:
        y = y * (w.double() + offset)
    return h, rstd, y


def norm_rel(n):
    """Relative error of rstd, and of y before its store: the sum of squares
    (halved by the root), the root, the quotient and three products."""
    return (chain(n) / 2 + 8) * U


def row_scale(y):
    return torch.clamp(y.abs().amax(dim=1), min=2.0 ** -100) / 448.0


def rmsnorm_backward(dy, h, w, rstd, dsum=None, offset=0.0):
    """(dx, dw, bound of dx before its store, bound of dw before its store)."""
    dy, h, rstd = dy.double(), h.double(), rstd.double()[:, None]
    M, N = h.shape
    gain = torch.ones(N, dtype=torch.float64) if w is None else w.double() + offset
    g, n = dy * gain, h * rstd
    dx = rstd * (g - n * (g * n).mean(dim=1, keepdim=True))
    far = 8 * U * rstd * g.abs() + rstd * n.abs() * ((chain(N) + 8) * U * (g * n).abs().mean(dim=1, keepdim=True))
    if dsum is not None:
        dx = dx + dsum.double()
        far = far + 2 * U * (dx.abs() + dsum.double().abs())
    dw = (dy * n).sum(dim=0)
    return dx, dw, far + 4 * U * dx.abs(), (M + 8) * U * (dy * n).abs().sum(dim=0)


def codes(q, K):
    """The N x K nibbles: the low one of a byte is the even k."""
    return torch.stack((q & 15, q >> 4), dim=2).reshape(q.shape[0], -1)[:, :K].long()


def w4_values(q, K, fmt):
    c = codes(q, K)
    if fmt == "int4":
        return torch.where(c >= 8, c - 16, c).double()
    v = torch.tensor(E2M1, dtype=torch.float64)[c & 7]
    return torch.where(c >= 8, -v, v)


def w4_weights(q, s, K, fmt, group):
    return w4_values(q, K, fmt) * s.double().repeat_interleave(group, dim=1)[:, :K]


def w4_matmul(x, q, s, fmt, group, rs=None, x_scale=1.0):
    """(y, bound before the store)."""
    K = x.shape[1]
    w = w4_weights(q, s, K, fmt, group)
    y, mag = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    f = x_scale if rs is None else x_scale * rs.double()[:, None]
    return y * f, (128 + K / 32 + 64 + 8) * U * (mag * f).abs()


def check(got, ref, far, what=""):
    """Every element within its bound: far (before the store) and the store's own rounding."""
    got, dt = got.double().cpu(), got.dtype
    ref = ref.double()
    if dt == torch.float8_e4m3fn:
        ref = ref.clamp(-448.0, 448.0)
    bad = torch.isfinite(ref) != torch.isfinite(got)
    ok = torch.isfinite(ref) & torch.isfinite(got)
    tol = (ref.abs() + far) * HALF[dt] + far + TINY[dt]
    over = torch.where(ok, (got - ref).abs() - tol, torch.zeros_like(ref))
    assert not bad.any(), "%s: finite and not, first at %s" % (what, torch.nonzero(bad)[0].tolist())
    same = torch.where(ok, torch.zeros_like(ref), torch.where(torch.isnan(ref), torch.isnan(got), got == ref).double() - 1)
    assert (same == 0).all(), "%s: another infinity or NaN" % what
    worst = over.max().item() if over.numel() else -1.0
    assert worst <= 0, "%s: over its bound by %g at %s (%g, not %g)" % (
        what, worst, torch.nonzero(over == over.max())[0].tolist(), got.flatten()[over.argmax()], ref.flatten()[over.argmax()])


def padded(t, pad, device="cuda", fill=float("nan")):
    """The matrix inside a buffer whose rows are `pad` elements longer (pads hold `fill`), and that buffer."""
    M, N = t.shape
    buf = torch.full((M, N + pad), fill, dtype=torch.float32).to(t.dtype) if t.dtype.is_floating_point else \
        torch.full((M, N + pad), int(fill), dtype=t.dtype)
    buf[:, :N] = t
    buf = buf.to(device)
    return buf[:, :N], buf


def rng(seed):
    return torch.Generator().manual_seed(seed)


def loud(M, N, seed, std=1.0):
    """Normal rows with a few columns an order larger."""
    g = rng(seed)
    x = torch.randn(M, N, generator=g) * std
    x[:, torch.randint(0, N, (max(1, N // 256),), generator=g)] *= 12.0
    return x
