"""A layer of gated experts on the device against the 64-bit formula: formats,
types, sizes, tokens, strides, absent experts, experts named twice, bases,
non-finite values; whole-number inputs bit for bit.
"""
import math

import pytest
import torch

import gemm_autotuning_amd as gt

from . import beside_ref as br
from . import op_ref as ref

pytestmark = pytest.mark.gpu


def layer(E, H, K, dtype, fmt, group, scales, seed):
    if fmt == "none":
        return dict(gate_up=br.normal((E, 2 * H, K), K ** -0.5, dtype, seed), down=br.normal((E, K, H), H ** -0.5, dtype, seed + 1))
    (gu, gs), (dn, ds) = br.nibbles(E, 2 * H, K, group, scales, seed), br.nibbles(E, K, H, group, scales, seed + 1)
    return dict(gate_up=gu, gs=gs, down=dn, ds=ds)


def run(x, index, weight, w, fmt="none", group=128, act="silu", base=None, out=None, pad=0, spread=False, in_place=False):
    """y on the CPU.  pad: every operand's rows lie inside wider ones; spread:
    so do the experts' matrices, and the scales are stored groups first."""
    T, K = x.shape
    c = {}
    for n, t in w.items():
        E, N, last = t.shape
        if n in ("gs", "ds"):
            c[n] = t.permute(0, 2, 1).contiguous().cuda().permute(0, 2, 1) if spread else t.cuda()
        elif spread:
            big = torch.full((E, N + 1, last + pad), 255 if t.dtype == torch.uint8 else math.nan, dtype=t.dtype, device="cuda")
            c[n] = big[:, :N, :last]
            c[n].copy_(t)
        else:
            c[n] = t.cuda()
    xc, _ = ref.padded(x, pad)
    odt = out or x.dtype
    buf = torch.full((T, K + pad), math.nan, device="cuda").to(odt)
    y = buf[:, :K]
    b = None
    if base is not None:
        b = ref.padded(base, pad)[0]
        if in_place:
            y.copy_(b)
            b = y
    gt.gt_moe(gt.make_moe_desc(xc, index.cuda(), weight.cuda(), c["gate_up"], c["down"], y, base=b, gate_up_scales=c.get("gs"),
                               down_scales=c.get("ds"), format=fmt, group=group, activation=act,
                               stream=torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert torch.isnan(buf[:, K:].float()).all(), "pads written"
    return y.cpu()


def same(T, E, k, K, H, dtype, fmt="none", group=128, scales="bf16", act="silu", out=None, absent=False, base=False, seed=0, **kw):
    x = ref.loud(T, K, seed + 5).to(dtype)
    index, weight = br.choices(T, E, k, seed + 6, absent)
    w = layer(E, H, K, dtype, fmt, group, scales, seed)
    b = br.normal((T, K), 1.0, out or dtype, seed + 7) if base else None
    got = run(x, index, weight, w, fmt, group, act, b, out, **kw)
    want, far = br.moe(x, index, weight, w["gate_up"], w["down"], w.get("gs"), w.get("ds"), fmt, group, act, b)
    ref.check(got, want, far, "y")


BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("fmt", ["none", "int4", "e2m1"])
@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (3, 8, 3), (16, 3, 2), (17, 2, 1), (40, 5, 4)])
def test_tokens(fmt, dtype, T, E, k):
    same(T, E, k, 256, 128, dtype, fmt, base=T != 3, out=F32 if T == 40 else None, seed=T)


@pytest.mark.parametrize("fmt,group,scales", [("none", 128, "bf16"), ("int4", 32, "f32"), ("e2m1", 64, "f16"), ("int4", 128, "bf16")])
@pytest.mark.parametrize("K,H", [(1, 1), (2, 3), (7, 9), (8, 8), (15, 17), (31, 33), (32, 64), (63, 65), (100, 129), (127, 130),
                                 (257, 255), (300, 511), (520, 70)])
def test_sizes(fmt, group, scales, K, H):
    same(5, 4, 2, K, H, BF if K % 2 else F16, fmt, group, scales, act="gelu" if H % 2 else "silu", out=F32 if K % 3 else None, pad=3,
         spread=True, absent=True, base=bool(K % 2), seed=K)


@pytest.mark.parametrize("fmt,group,scales", [("none", 128, "bf16"), ("int4", 32, "f32"), ("e2m1", 64, "f16"), ("int4", 128, "bf16")])
@pytest.mark.parametrize("K,H", [(1, 1), (2, 3), (7, 9), (8, 8), (15, 17), (31, 33), (32, 64), (63, 65), (100, 129), (127, 130),
                                 (257, 255), (300, 511), (520, 70)])
def test_sizes_of_more_tokens(fmt, group, scales, K, H):
    same(11, 4, 2, K, H, BF if K % 2 else F16, fmt, group, scales, act="gelu" if H % 2 else "silu", out=F32 if K % 3 else None, pad=3,
         spread=True, absent=True, base=bool(K % 2), seed=K)


@pytest.mark.parametrize("fmt", ["none", "int4", "e2m1"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (2, 64, 8), (4, 40, 3), (8, 300, 2), (8, 9, 9)])
def test_few_tokens_of_many_experts(fmt, T, E, k):
    same(T, E, k, 72, 40, F16 if T % 4 else BF, fmt, 32, "f16", absent=T > 1, base=E > 40, out=F32 if k == 9 else None, pad=T, spread=E < 40,
         seed=E)


@pytest.mark.parametrize("fmt", ["none", "int4"])
def test_long_rows_of_more_tokens(fmt):
    same(9, 2, 2, 1100, 1500, BF, fmt, 64, seed=1)
    same(9, 2, 1, 5000, 40, F16, fmt, 32, seed=2)
    same(10, 2, 1, 40, 9001, BF, fmt, 128, seed=3)


@pytest.mark.parametrize("fmt", ["none", "int4"])
def test_long_rows(fmt):
    same(2, 3, 2, 1100, 1500, BF, fmt, 64, seed=1)
    same(2, 2, 1, 5000, 40, F16, fmt, 32, seed=2)
    same(2, 2, 1, 40, 9001, BF, fmt, 128, seed=3)


@pytest.mark.parametrize("fmt", ["none", "int4", "e2m1"])
@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("T,E,k,K,H", [(1, 6, 3, 96, 80), (9, 3, 2, 100, 100), (70, 2, 2, 128, 100), (33, 7, 5, 64, 33)])
def test_whole_numbers(fmt, dtype, T, E, k, K, H):
    # gates of at least 32: the activation is the gate itself (its exponential is below fp32's half step);
    # every value and sum is a whole number, or a half or quarter, within 2^24 of its steps, and the
    # values between the products take at most 16 bits
    g = ref.rng(T + K)
    x = torch.randint(1, 3, (T, K), generator=g).to(dtype)
    index, _ = br.choices(T, E, k, 3)
    weight = 2.0 ** torch.randint(-1, 2, (T, k), generator=g).float()
    few = [0, 1, 2, 10]  # 0, .5, 1, -1 in e2m1
    if fmt == "none":
        gate = torch.randint(1, 3, (E, H, K), generator=g)
        up = torch.randint(0, 12, (E, H, K), generator=g)
        up = torch.where(up < 3, up - 1, 0)
        w = dict(gate_up=torch.cat([gate, up], 1).to(dtype), down=torch.randint(-1, 2, (E, K, H), generator=g).to(dtype))
    else:
        pos, sparse = ([1, 2], [0] * 12 + [1, 15]) if fmt == "int4" else ([1, 2], [0] * 12 + [2, 10])
        gq = br.nibbles(E, H, K, 32, "f32", 1, pos)[0]
        uq = br.nibbles(E, H, K, 32, "f32", 2, sparse)[0]
        dq = br.nibbles(E, K, H, 32, "f32", 3, [0, 1, 15, 2] if fmt == "int4" else few)[0]
        w = dict(gate_up=torch.cat([gq, uq], 1), down=dq, gs=torch.ones(E, 2 * H, -(-K // 32)), ds=torch.ones(E, K, -(-H // 32)))
    want, _ = br.moe(x, index, weight, w["gate_up"], w["down"], w.get("gs"), w.get("ds"), fmt, 32)
    assert want.abs().max() < 2 ** 21
    got = run(x, index, weight, w, fmt, 32, out=F32)
    assert torch.equal(got.double(), want)


@pytest.mark.parametrize("times", [1, 4])
def test_an_expert_named_twice_and_indices_out_of_range(times):
    x = ref.loud(4 * times, 96, 1).to(BF)
    w = layer(3, 64, 96, BF, "none", 128, "bf16", 2)
    index = torch.tensor([[1, 1, 1], [0, 3, 0], [-1, -7, 2 ** 31 - 1], [2, -2 ** 31, 0]], dtype=torch.int32)
    weight = torch.rand(4, 3, generator=ref.rng(3))
    weight[1, 1] = math.nan  # of a slot that is never followed
    index, weight = index.repeat(times, 1), weight.repeat(times, 1)
    base = br.normal((4 * times, 96), 1.0, BF, 4)
    for b in (None, base):
        got = run(x, index, weight, w, base=b)
        want, far = br.moe(x, index, weight, w["gate_up"], w["down"], base=b)
        ref.check(got, want, far)
        assert torch.equal(got[2].double(), want[2])


@pytest.mark.parametrize("T", [6, 11])
def test_in_place(T):
    x = ref.loud(T, 100, 1).to(F16)
    w = layer(3, 50, 100, F16, "none", 128, "bf16", 2)
    index, weight = br.choices(T, 3, 2, 3)
    base = br.normal((T, 100), 1.0, F16, 4)
    a = run(x, index, weight, w, base=base, pad=5)
    assert torch.equal(a, run(x, index, weight, w, base=base, pad=5, in_place=True))


@pytest.mark.parametrize("T", [7, 9])
@pytest.mark.parametrize("dtype", [BF, F16])
def test_non_finite_rows_stay_their_own(dtype, T):
    # an infinity or NaN in a row makes that row's results what the formula gives and leaves the others
    x = ref.loud(T, 200, 1).to(dtype)
    w = layer(2, 70, 200, dtype, "none", 128, "bf16", 2)
    index, weight = br.choices(T, 2, 2, 3)
    clean = run(x, index, weight, w)
    x[3, 17], x[5, 199] = math.inf, math.nan
    got = run(x, index, weight, w)
    keep = [m for m in range(T) if m not in (3, 5)]
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[5].float()).all()
    assert not torch.isfinite(got[3].float()).any()


@pytest.mark.parametrize("T", [2, 10])
def test_infinite_results_have_their_sign(T):
    # an activation past every number, times weights of one sign: an infinity, not a NaN
    x = torch.full((T, 64), 1.0).to(BF)
    gate_up = torch.ones(1, 2 * 32, 64).to(BF) * 2.0 ** 70
    down = torch.ones(1, 64, 32).to(BF)
    down[0, 1::2] = -1.0
    got = run(x, torch.zeros(T, 1, dtype=torch.int32), torch.ones(T, 1), dict(gate_up=gate_up, down=down))
    assert (got[:, 0::2] == math.inf).all() and (got[:, 1::2] == -math.inf).all()


@pytest.mark.parametrize("T", [3, 12])
def test_large_and_small_activations_of_f16(T):
    # values between the products far outside f16's own range, above and below
    for big in (2.0 ** 9, 2.0 ** -9):
        x = (ref.loud(T, 128, 1) * big).to(F16)
        w = layer(2, 96, 128, F16, "none", 128, "bf16", 2)
        index, weight = br.choices(T, 2, 2, 3)
        if big > 1:
            weight *= 2.0 ** -14
        got = run(x, index, weight, w, out=F32)
        want, far = br.moe(x, index, weight, w["gate_up"], w["down"])
        ref.check(got, want, far)


@pytest.mark.parametrize("T", [2, 12])
def test_weights_that_nothing_reads(T):
    # experts that no token names may hold anything
    x = ref.loud(T, 64, 1).to(BF)
    w = layer(5, 32, 64, BF, "none", 128, "bf16", 2)
    index = torch.tensor([[1, 3], [3, 1]], dtype=torch.int32).repeat(T // 2, 1)
    weight = torch.rand(T, 2, generator=ref.rng(1))
    clean = run(x, index, weight, w)
    for e in (0, 2, 4):
        w["gate_up"][e], w["down"][e] = math.nan, math.nan
    assert torch.equal(run(x, index, weight, w), clean)


def test_many_tokens_run_in_ranges():
    # more pairs than one launch takes
    T, E, k = 1500, 4, 3
    x = torch.randint(1, 3, (T, 64), generator=ref.rng(1)).to(BF)
    index, weight = br.choices(T, E, k, 2, absent=True)
    weight = torch.ones(T, k)
    g = ref.rng(5)
    up = torch.randint(0, 12, (E, 40, 64), generator=g)
    w = dict(gate_up=torch.cat([torch.randint(1, 3, (E, 40, 64), generator=g), torch.where(up < 3, up - 1, 0)], 1).to(BF),
             down=torch.randint(-1, 2, (E, 64, 40), generator=g).to(BF))
    got = run(x, index, weight, w, out=F32)
    xs, want = x.double(), torch.zeros(T, 64, dtype=torch.float64)
    for e in range(E):
        gu = xs @ w["gate_up"][e].double().t()
        want += ((gu[:, :40] * gu[:, 40:]) @ w["down"][e].double().t()) * (index == e).sum(dim=1, keepdim=True)
    assert torch.equal(got.double(), want)


@pytest.mark.parametrize("none", ["H", "E", "topk"])
def test_nothing_to_add(none):
    T, K, H, E, k = 5, 33, 16, 2, 2
    H, E, k = (0 if none == "H" else H), (0 if none == "E" else E), (0 if none == "topk" else k)
    x = torch.ones(T, K).to(BF)
    base = br.normal((T, K), 1.0, BF, 1)
    index, weight = torch.zeros(T, k, dtype=torch.int32), torch.ones(T, k)
    w = dict(gate_up=torch.ones(E, 2 * H, K).to(BF), down=torch.ones(E, K, H).to(BF))
    assert torch.equal(run(x, index, weight, w, base=base, pad=2), base)
    assert (run(x, index, weight, w, pad=2) == 0).all()


@pytest.mark.parametrize("T,E,k,K,H", [(1, 5, 3, 64, 48), (9, 300, 40, 33, 17), (700, 3, 3, 64, 32), (1400, 2, 2, 16, 8), (3, 2, 2, 4, 4)])
def test_the_callers_workspace_is_enough_and_not_left(T, E, k, K, H):
    x = ref.loud(T, K, 1).to(BF)
    w = layer(E, H, K, BF, "none", 128, "bf16", 2)
    index, weight = br.choices(T, E, k, 3)
    y = torch.empty(T, K, device="cuda").bfloat16()
    args = (x.cuda(), index.cuda(), weight.cuda(), w["gate_up"].cuda(), w["down"].cuda(), y)
    n = gt.gt_moe_workspace(gt.make_moe_desc(*args))
    buf = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    gt.gt_moe(gt.make_moe_desc(*args, workspace=buf[:n], stream=torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert (buf[n:] == 0x5A).all(), "written past the workspace"
    assert torch.equal(y.cpu(), run(x, index, weight, w))


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("T,E,k,K,H", [(16, 1, 1, 96, 40), (63, 2, 1, 257, 130), (64, 1, 1, 128, 256), (65, 1, 1, 500, 9), (33, 2, 2, 8, 8),
                                       (129, 3, 2, 100, 300), (150, 2, 2, 640, 17), (40, 2, 2, 1100, 600), (17, 1, 1, 31, 1500)])
def test_many_rows_of_an_expert(dtype, T, E, k, K, H):
    same(T, E, k, K, H, dtype, act="gelu" if T % 2 else "silu", out=F32 if T % 3 else None, absent=T > 100, base=T > 64,
         pad=3 * (T % 2), spread=bool(T % 2), seed=T)


def test_the_rows_of_one_expert_among_many():
    # on average 16 rows to an expert and more, and all of them name one
    T, E, K, H = 200, 5, 130, 70
    x = ref.loud(T, K, 1).to(BF)
    w = layer(E, H, K, BF, "none", 128, "bf16", 2)
    weight = torch.rand(T, 1, generator=ref.rng(3))
    index = torch.full((T, 1), 3, dtype=torch.int32)
    index[77] = -1
    for e in (0, 1, 2, 4):
        w["gate_up"][e], w["down"][e] = math.nan, math.nan
    got = run(x, index, weight, w)
    want, far = br.moe(x, index, weight, w["gate_up"], w["down"])
    ref.check(got, want, far, "y")


@pytest.mark.parametrize("dtype", [BF, F16])
def test_non_finite_rows_among_many_stay_their_own(dtype):
    T = 90
    x = ref.loud(T, 200, 1).to(dtype)
    w = layer(2, 70, 200, dtype, "none", 128, "bf16", 2)
    index, weight = br.choices(T, 2, 2, 3)
    clean = run(x, index, weight, w)
    x[3, 17], x[70, 199] = math.inf, math.nan
    got = run(x, index, weight, w)
    keep = [m for m in range(T) if m not in (3, 70)]
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[70].float()).all()
    assert not torch.isfinite(got[3].float()).any()


def test_large_and_small_activations_of_many_f16_rows():
    for big in (2.0 ** 9, 2.0 ** -9):
        x = (ref.loud(80, 128, 1) * big).to(F16)
        w = layer(2, 300, 128, F16, "none", 128, "bf16", 2)
        index, weight = br.choices(80, 2, 2, 3)
        if big > 1:
            weight *= 2.0 ** -14
        got = run(x, index, weight, w, out=F32)
        want, far = br.moe(x, index, weight, w["gate_up"], w["down"])
        ref.check(got, want, far)
