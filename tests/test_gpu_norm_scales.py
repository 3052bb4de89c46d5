"""The RMS norm's e4m3 output over one given scale, anywhere in fp32's range:
the formula is a quotient, so a scale whose reciprocal passes the range of
normal numbers must not turn zeros into NaN or cost the quotient its bits.
"""
import pytest
import torch

import gemm_autotuning_amd as gt

from . import op_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [300, 5000, 16390, 33000])  # f32 rows past 16384 elements, bf16 ones past 32768 are read again
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [2.0 ** -149, 1e-39, 2.0 ** -129, 2.0 ** -128, 2.0 ** -127, 2.0 ** -126, 1e-30, 2.0 ** -100,
                                   2.0 ** 100, 1e30, 2.0 ** 126, 2.0 ** 127, 3.4e38])
def test_any_finite_scale(N, dtype, scale):
    M = 5
    x = ref.loud(M, N, 1).to(ref.DT[dtype])
    x[2] = 0
    x[3, ::2] = 0
    # outputs between 2^-8 and 2^9, both sides of e4m3's range, as far as fp32 holds them
    gain = min(max(scale * 4, 2.0 ** -126), 2.0 ** 122)
    w = (torch.rand(N, generator=ref.rng(2)) + 1.0).double().mul(gain).float()
    y = torch.full((M, N), float("nan"), dtype=torch.float8_e4m3fn, device="cuda")
    gt.gt_rmsnorm(gt.make_rmsnorm_desc(x.cuda(), w.cuda(), y, quant="tensor", scale=scale))
    torch.cuda.synchronize()
    _, _, want = ref.rmsnorm(x, None, w)
    real = float(torch.tensor(scale, dtype=torch.float32).double())
    # the norm's own bound, and half a step of fp32's least value where the weighted element is subnormal
    far = want.abs() * (ref.norm_rel(N) + 8 * ref.U) + 2 * 2.0 ** -150
    ref.check(y.cpu(), want / real, far / real, "y")
    assert (y[2].float() == 0).all() and (y[3, ::2].float() == 0).all()
