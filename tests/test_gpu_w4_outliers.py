"""4-bit weight products of rows whose large elements meet zero or small
weights: what an element adds to a sum is its product, so an element of any
size at a weight of zero leaves the others' sum as accurate as it is without
it (the bound of tests/op_ref.py, which holds the products' magnitudes and
nothing else), and huge elements overflow only where their products do.
"""
import itertools

import pytest
import torch

import gemm_autotuning_amd as gt

from . import op_ref as ref

pytestmark = pytest.mark.gpu

LARGEST = {"bf16": 2.0 ** 126, "f16": 2.0 ** 15, "e4m3": 448.0}


def product(v, q, s, fmt, group):
    y = torch.empty(v.shape[0], q.shape[0], device="cuda")
    gt.gt_w4_matmul(gt.make_w4_desc(v.cuda(), q.cuda(), s.cuda(), y, fmt, group))
    torch.cuda.synchronize()
    return y.cpu()


def zero_at(q, k):
    q[:, k // 2] &= 0x0F if k % 2 else 0xF0


@pytest.mark.parametrize("x,fmt,group", list(itertools.product(("bf16", "f16", "e4m3"), ("int4", "e2m1"), (32, 64, 128))))
@pytest.mark.parametrize("M,N,K", [(1, 40, 256), (4, 64, 2048), (16, 33, 4100), (20, 48, 1024), (61, 100, 640), (3, 17, 20001)])
def test_an_outlier_at_a_zero_weight_adds_nothing(M, N, K, x, fmt, group):
    g = ref.rng(M + K)
    for size in (1e3, 1e5, 2.0 ** 40, 2.0 ** 100, LARGEST[x]):
        if size > LARGEST[x]:
            continue
        v = torch.randn(M, K, generator=g).to(ref.DT[x])
        q = torch.randint(0, 256, (N, -(-K // 2)), generator=g, dtype=torch.uint8)
        s = torch.rand(N, -(-K // group), generator=g) + 0.5
        for i, k in enumerate((5, 100, K // 2, K - 1)):
            v[:, k] = (size if i % 2 else -size / 2)
            zero_at(q, k)
        want, far = ref.w4_matmul(v, q, s, fmt, group)
        ref.check(product(v, q, s, fmt, group), want, far, "y, elements of %g" % size)


@pytest.mark.parametrize("M", [1, 20, 50])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("K", [256, 4096, 9000])
def test_huge_elements_of_opposite_signs(M, group, K):
    # products of up to 10.5 * 2^124 that a row's signed sum does not show: every product and sum is finite
    N, big = 32, 1.5 * 2.0 ** 124
    v = torch.zeros(M, K).bfloat16()
    v[:, 0], v[:, 8] = big, -big
    v[M // 2, 16], v[M // 2, 24] = 1.9375 * 2.0 ** 122, -1.9375 * 2.0 ** 122
    v[0, K - 1] = 1.0
    codes = torch.zeros(N, K, dtype=torch.uint8)
    codes[:, 0], codes[:, 16] = 7, 7
    codes[:, K - 1] = 9
    codes[1::2, 0] = 0
    codes[1::2, 8] = 7
    q = codes[:, 0::2] | codes[:, 1::2] << 4
    s = torch.full((N, -(-K // group)), 2.0 ** -3)
    want, far = ref.w4_matmul(v, q, s, "int4", group)
    assert torch.isfinite(want).all()
    ref.check(product(v, q, s, "int4", group), want, far, "y")


@pytest.mark.parametrize("x", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", ["int4", "e2m1"])
def test_subnormal_elements_count(x, fmt):
    # 16-bit rows below the least normal value: their products are exact in fp32 (f16) or at its far end (bf16)
    M, N, K = 5, 40, 640
    least = 2.0 ** -24 if x == "f16" else 2.0 ** -133
    v = (torch.randint(-100, 101, (M, K), generator=ref.rng(3)).double() * least).to(ref.DT[x])
    q = torch.randint(0, 256, (N, K // 2), generator=ref.rng(4), dtype=torch.uint8)
    s = torch.full((N, K // 128), 1.0 if x == "f16" else 2.0 ** 20)
    want, far = ref.w4_matmul(v, q, s, fmt, 128)
    ref.check(product(v, q, s, fmt, 128), want, far, "y")


def test_a_row_does_not_depend_on_the_rows_beside_it():
    # the same row alone and among others, with integer weights in groups of 32 and 128: exact sums, equal bits
    N, K = 100, 1024
    v = torch.randint(-4, 5, (64, K), generator=ref.rng(5)).float().bfloat16()
    q = torch.randint(0, 256, (N, K // 2), generator=ref.rng(6), dtype=torch.uint8)
    for group in (32, 128):
        s = torch.full((N, K // group), 0.5)
        all_rows = product(v, q, s, "int4", group)
        for m in (0, 17, 63):
            assert torch.equal(product(v[m:m + 1], q, s, "int4", group)[0], all_rows[m])
