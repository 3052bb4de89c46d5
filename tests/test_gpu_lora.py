"""Adapters of many requests on the device against the 64-bit formula: types,
ranks, sizes, rows in any order of adapters, rows without one, strides, in
place; whole-number inputs bit for bit.
"""
import math

import pytest
import torch

import gemm_autotuning_amd as gt

from . import beside_ref as br
from . import op_ref as ref

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def run(x, index, a, b, scale=None, base=None, out=None, pad=0, spread=False, in_place=False):
    M, N = x.shape[0], b.shape[1]

    def inside(t):
        if not spread:
            return t.cuda()
        E, R, C = t.shape
        big = torch.full((E, R + 1, C + pad), math.nan, dtype=t.dtype, device="cuda")
        big[:, :R, :C].copy_(t)
        return big[:, :R, :C]

    xc, _ = ref.padded(x, pad)
    buf = torch.full((M, N + pad), math.nan, device="cuda").to(out or x.dtype)
    y = buf[:, :N]
    bc = None
    if base is not None:
        bc = ref.padded(base, pad)[0]
        if in_place:
            y.copy_(bc)
            bc = y
    gt.gt_lora(gt.make_lora_desc(xc, index.cuda(), inside(a), inside(b), y, base=bc, scale=None if scale is None else scale.cuda(),
                                 stream=torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert torch.isnan(buf[:, N:].float()).all(), "pads written"
    return y.cpu()


def same(M, L, r, K, N, dtype, out=None, base=True, scaled=True, seed=0, index=None, **kw):
    x = ref.loud(M, K, seed).to(dtype)
    a, b = br.normal((L, r, K), K ** -0.5, dtype, seed + 1), br.normal((L, N, r), r ** -0.5, dtype, seed + 2)
    g = ref.rng(seed + 3)
    if index is None:
        index = torch.randint(-1, L, (M,), generator=g, dtype=torch.int32)
    scale = torch.randn(L, generator=g) if scaled else None
    bs = br.normal((M, N), 1.0, out or dtype, seed + 4) if base else None
    got = run(x, index, a, b, scale, bs, out, **kw)
    want, far = br.lora(x, index, a, b, scale, bs)
    ref.check(got, want, far, "y")
    none = (index < 0) | (index >= L)
    assert torch.equal(got[none], bs[none] if base else torch.zeros_like(got[none])), "rows without an adapter"


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 130])
def test_rows(dtype, M):
    same(M, 6, 16, 256, 192, dtype, out=F32 if M % 2 else None, base=M != 2, seed=M)


@pytest.mark.parametrize("r", [1, 2, 3, 4, 7, 8, 9, 15, 16, 17, 24, 31, 32, 33, 40, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256])
def test_ranks(r):
    same(9, 3, r, 130, 70, BF if r % 2 else F16, seed=r, pad=r % 3, spread=bool(r % 2), scaled=r % 5 != 0)


@pytest.mark.parametrize("K", [1, 2, 7, 8, 9, 31, 63, 64, 100, 127, 128, 129, 255, 257, 1000, 1025, 4100, 9000])
def test_lengths(K):
    same(5, 3, 12, K, 50, BF if K % 2 else F16, seed=K, pad=1, spread=True)


@pytest.mark.parametrize("N", [1, 2, 3, 8, 15, 16, 17, 63, 64, 65, 127, 129, 500, 1023, 4097])
def test_columns(N):
    same(20, 4, 8, 96, N, BF if N % 2 else F16, seed=N, pad=3, out=F32 if N % 3 == 0 else None)


@pytest.mark.parametrize("r", [1, 4, 7, 8, 9, 15, 16, 17, 24, 31, 32])
def test_ranks_of_many_rows(r):
    for M in (700, 1100):
        same(M, 7, r, 72, 40, BF if r % 2 else F16, out=F32 if r > 8 else None, pad=r % 4, spread=r > 4, seed=r)


@pytest.mark.parametrize("r", [130, 200, 256])
@pytest.mark.parametrize("K", [8, 31, 100, 129, 1000, 2051])
def test_lengths_of_high_ranks(r, K):
    same(128, 5, r, K, 33, F16 if K % 2 else BF, out=F32, pad=K % 2, spread=K > 100, seed=K)


@pytest.mark.parametrize("K", [8, 9, 31, 100, 127, 128, 129, 300, 1000, 2050])
def test_lengths_of_many_rows(K):
    same(1100, 9, 20, K, 30, F16 if K % 2 else BF, out=F32, pad=K % 2, spread=K > 128, seed=K)


def test_long_rows_of_a_batch():
    same(64, 6, 64, 16500, 70, BF, out=F32, seed=1)
    same(24, 6, 100, 20001, 70, F16, out=F32, seed=2, spread=True)


@pytest.mark.parametrize("r,K,N", [(8, 8, 5), (9, 130, 64), (16, 100, 70), (31, 257, 33), (32, 1290, 65), (33, 128, 100), (40, 31, 9),
                                   (64, 600, 130)])
def test_thousands_of_rows(r, K, N):
    M = 2100
    runs = torch.div(torch.arange(M), 300, rounding_mode="floor").int() - 1
    same(M, 8 if K < 100 else 5, r, K, N, BF if r % 2 else F16, out=F32 if r > 16 else None, pad=r % 4, spread=r > 16, seed=r,
         index=runs if r % 3 else None, in_place=r == 32)


@pytest.mark.parametrize("K", [8, 9, 31, 100, 127, 128, 129, 300, 1000, 2050])
def test_lengths_of_wide_results(K):
    same(90, 7, 16, K, 2100, F16 if K % 2 else BF, out=F32, pad=K % 2, spread=K > 128, seed=K)


@pytest.mark.parametrize("r,K", [(32, 4096), (32, 4097), (33, 64), (16, 8193), (20, 520), (1, 1 << 17)])
@pytest.mark.parametrize("M", [2, 19])
def test_ranks_and_lengths_of_few_rows(M, r, K):
    same(M, 3, r, K, 1030, BF if M == 2 else F16, out=F32, seed=r)


@pytest.mark.parametrize("N", [80, 2700])
@pytest.mark.parametrize("order", ["one", "runs", "each", "none", "alternate", "out of range"])
def test_orders(order, N):
    M, L = 100, 100
    index = {"one": torch.full((M,), 7), "runs": torch.arange(M) // 30, "each": torch.randperm(L, generator=ref.rng(1)),
             "none": torch.full((M,), -1), "alternate": torch.arange(M) % 2 * 50,
             "out of range": torch.where(torch.arange(M) % 3 == 0, 2 ** 31 - 1, torch.where(torch.arange(M) % 3 == 1, -2 ** 31, 3))}[order]
    for in_place in (False, True):
        same(M, L, 8, 64, N, BF, index=index.int(), in_place=in_place, pad=2)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("M,L,r,K,N", [(1, 1, 16, 100, 100), (50, 7, 12, 130, 200), (700, 5, 64, 64, 129), (40, 40, 130, 300, 64)])
def test_whole_numbers(dtype, M, L, r, K, N):
    g = ref.rng(M + K)
    x = torch.randint(-2, 3, (M, K), generator=g).to(dtype)
    a = torch.randint(-1, 2, (L, r, K), generator=g).to(dtype)
    b = torch.randint(-2, 3, (L, N, r), generator=g).to(dtype)
    index = torch.randint(-1, L, (M,), generator=g, dtype=torch.int32)
    scale = 2.0 ** torch.randint(-2, 3, (L,), generator=g).float()
    base = torch.randint(-50, 50, (M, N), generator=g).float()
    want = base.double()
    for e in range(L):
        m = index == e
        want[m] += scale[e].double() * (x[m].double() @ a[e].double().t()) @ b[e].double().t()
    got = run(x, index, a, b, scale, base, out=F32)
    assert torch.equal(got.double(), want)


@pytest.mark.parametrize("r", [8, 40])
@pytest.mark.parametrize("dtype", [BF, F16])
def test_non_finite_rows_stay_their_own(dtype, r):
    x = ref.loud(20, 100, 1).to(dtype)
    a, b = br.normal((3, r, 100), 0.1, dtype, 2), br.normal((3, 60, r), 0.3, dtype, 3)
    index = torch.arange(20).int() % 4 - 1
    clean = run(x, index, a, b)
    x[5, 3], x[6, 99], x[4, 0] = math.inf, math.nan, math.inf  # row 4 has no adapter
    got = run(x, index, a, b)
    keep = [m for m in range(20) if m not in (5, 6)]
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[6].float()).all() and not torch.isfinite(got[5].float()).any()


@pytest.mark.parametrize("r", [8, 40])
def test_a_base_that_is_not_finite(r):
    x = ref.loud(4, 64, 1).to(BF)
    a, b = br.normal((2, r, 64), 0.1, BF, 2), br.normal((2, 40, r), 0.3, BF, 3)
    base = torch.zeros(4, 40).to(BF)
    base[0, 0], base[1, 39], base[3, 5] = math.inf, math.nan, -math.inf
    got = run(x, torch.tensor([0, 1, -1, -1], dtype=torch.int32), a, b, base=base)
    assert got[0, 0] == math.inf and torch.isnan(got[1, 39].float()) and got[3, 5] == -math.inf
    assert torch.isfinite(got.float()).sum() == 4 * 40 - 3


@pytest.mark.parametrize("r", [8, 40])
def test_large_and_small_values_of_f16(r):
    for big in (2.0 ** 9, 2.0 ** -12):
        x = (ref.loud(6, 200, 1) * big).to(F16)
        a = (br.normal((2, r, 200), big, F32, 2)).to(F16)
        b = br.normal((2, 30, r), 0.3, F16, 3)
        index = torch.arange(6).int() % 2
        got = run(x, index, a, b, out=F32)
        want, far = br.lora(x, index, a, b)
        ref.check(got, want, far)


def test_many_rows():
    M, L, r, K, N = 9000, 9, 16, 128, 96
    g = ref.rng(3)
    x = torch.randint(-2, 3, (M, K), generator=g).to(BF)
    a, b = torch.randint(-1, 2, (L, r, K), generator=g).to(BF), torch.randint(-2, 3, (L, N, r), generator=g).to(BF)
    for index in (torch.randint(-1, L, (M,), generator=g, dtype=torch.int32), (torch.arange(M) // 1001).int() - 1):
        want = torch.zeros(M, N, dtype=torch.float64)
        for e in range(L):
            m = index == e
            want[m] = (x[m].double() @ a[e].double().t()) @ b[e].double().t()
        assert torch.equal(run(x, index, a, b, out=F32).double(), want)


@pytest.mark.parametrize("r,L,out,base", [(8, 3, F32, True), (40, 90, BF, True), (130, 5, F32, False), (3, 4, F16, True), (200, 3, F32, True)])
def test_results_past_the_caches(r, L, out, base):
    M, K, N = 2300, 72, 5001
    g = ref.rng(r)
    dt = F16 if out == F16 else BF
    x, a = torch.randint(-1, 2, (M, K), generator=g).to(dt), torch.randint(-1, 2, (L, r, K), generator=g).to(dt)
    b = torch.randint(-1, 2, (L, N, r), generator=g).to(dt)
    b[:, :, 2:] = 0  # sums that 8 bits hold
    a[:, :, 30:] = 0
    bs = torch.randint(-40, 41, (M, N), generator=g).to(out) if base else None
    index = torch.randint(-1, L, (M,), generator=g, dtype=torch.int32)
    want = bs.double() if base else torch.zeros(M, N, dtype=torch.float64)
    for e in range(L):
        m = index == e
        want[m] += (x[m].double() @ a[e].double().t()) @ b[e].double().t()
    assert want.abs().max() < 256
    assert torch.equal(run(x, index, a, b, base=bs, out=out, pad=5).double(), want)


@pytest.mark.parametrize("none", ["K", "adapters", "rank"])
def test_nothing_to_add(none):
    M, L, r, K, N = 5, 2, 4, 32, 33
    K, L, r = (0 if none == "K" else K), (0 if none == "adapters" else L), (0 if none == "rank" else r)
    x, a, b = torch.ones(M, K).to(BF), torch.ones(L, r, K).to(BF), torch.ones(L, N, r).to(BF)
    base, index = br.normal((M, N), 1.0, BF, 1), torch.zeros(M, dtype=torch.int32)
    assert torch.equal(run(x, index, a, b, base=base, pad=2), base)
    assert (run(x, index, a, b, pad=2) == 0).all()


@pytest.mark.parametrize("M,L,r,K", [(1, 1, 16, 4096), (3, 2, 40, 9000), (500, 1, 8, 5000), (4096, 3, 16, 256), (4097, 1, 16, 4096), (4596, 1, 16, 8192),
                                     (9000, 9, 12, 2000), (5, 2, 7, 4), (4096 + 2047, 2, 64, 4000),
                                     (4096 + 200, 3, 40, 9000), (2048, 1, 8, 3000)])
def test_the_callers_workspace_is_enough_and_not_left(M, L, r, K):
    g = ref.rng(M)
    x = torch.randint(-1, 2, (M, K), generator=g).to(BF)
    a, b = torch.randint(-1, 2, (L, r, K), generator=g).to(BF), torch.randint(-2, 3, (L, 64, r), generator=g).to(BF)
    index = torch.randint(-1, L, (M,), generator=g, dtype=torch.int32)
    y = torch.empty(M, 64, device="cuda")
    args = (x.cuda(), index.cuda(), a.cuda(), b.cuda(), y)
    n = gt.gt_lora_workspace(gt.make_lora_desc(*args))
    buf = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    gt.gt_lora(gt.make_lora_desc(*args, workspace=buf[:n], stream=torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert (buf[n:] == 0x5A).all(), "written past the workspace"
    want = torch.zeros(M, 64, dtype=torch.float64)
    for e in range(L):
        m = index == e
        want[m] = (x[m].double() @ a[e].double().t()) @ b[e].double().t()
    assert torch.equal(y.cpu().double(), want)
