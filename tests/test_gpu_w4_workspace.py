"""The workspace of a 4-bit weight product whose K takes several slices: it
stays within a bound whatever the sizes, and a product that needs more runs
in ranges of columns and rows that meet without a gap.
"""
import pytest
import torch

import gemm_autotuning_amd as gt

from . import op_ref as ref

pytestmark = pytest.mark.gpu

MOST = 64 << 20  # of partial sums


def integers(M, N, K, group, seed, rare=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-4, 5, (M, K), generator=g, device="cuda", dtype=torch.int8)
    if rare:
        for m in range(M):
            x[m] *= torch.randint(0, 200, (K,), generator=g, device="cuda", dtype=torch.uint8) == 0
    q = torch.randint(0, 256, (N, -(-K // 2)), generator=g, device="cuda", dtype=torch.uint8)
    s = 2.0 ** torch.randint(-2, 1, (N, -(-K // group)), generator=g, device="cuda").float()
    return x.bfloat16(), q, s


def product_of(x, q, s, group):
    """The same sums, all exact in fp32, from the expanded weights: 2^20 of K at a time."""
    M, K = x.shape
    y = torch.zeros(M, q.shape[0], device="cuda")
    step = 1 << 20
    for k in range(0, K, step):
        n = min(step, K - k)
        w = torch.empty(q.shape[0], n, device="cuda")
        gt.gt_w4_expand(gt.make_w4_expand_desc(q[:, k // 2:(k + n + 1) // 2], s[:, k // group:-(-(k + n) // group)], w, "int4", group,
                                               stream=torch.cuda.current_stream().cuda_stream))
        y += x[:, k:k + n].float() @ w.t()
    return y


def took(call):
    """Device memory that the call itself allocates."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.mem_get_info()[0]
    call()
    torch.cuda.synchronize()
    return before - torch.cuda.mem_get_info()[0]


@pytest.mark.parametrize("M,N,K,rare", [(300, 30011, 4192, False), (256, 65536, 8192, False), (20, 600000, 4161, False),
                                        (257, 300, (1 << 23) + (1 << 18) + 33, True)])
def test_partial_sums_stay_within_their_bound(M, N, K, rare):
    x, q, s = integers(M, N, K, 64, M + N, rare)
    out = torch.full((M, N + 5), float("nan"), device="cuda")
    st = torch.cuda.Stream()
    d = gt.make_w4_desc(x, q, s, out[:, :N], group=64, stream=st.cuda_stream)
    # a buffer grows to twice its size at least, so up to twice the bound, and the counters beside them
    assert took(lambda: gt.gt_w4_matmul(d)) <= 2 * MOST + (4 << 20)
    assert torch.equal(out[:, :N], product_of(x, q, s, 64))
    assert torch.isnan(out[:, N:]).all(), "pads written"


def test_row_scales_and_strides_across_the_ranges():
    M, N, K, group = 300, 30011, 4192, 32
    x, q, s = integers(M, N, K, group, 9)
    rs = 2.0 ** torch.randint(-3, 4, (M,), device="cuda").float()
    S = s.t().contiguous().t()  # groups outermost
    out = torch.full((M, N + 3), float("nan"), device="cuda").bfloat16()
    gt.gt_w4_matmul(gt.make_w4_desc(x, q, S, out[:, :N], group=group, row_scale=rs, x_scale=0.5))
    torch.cuda.synchronize()
    assert torch.equal(out[:, :N], (product_of(x, q, s, group) * 0.5 * rs[:, None]).bfloat16())
    assert torch.isnan(out[:, N:].float()).all()
