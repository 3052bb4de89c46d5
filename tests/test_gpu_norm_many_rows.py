"""The RMS norm of more rows than one launch has workgroups."""
import pytest
import torch

import gemm_autotuning_amd as gt

from . import op_ref as ref

pytestmark = pytest.mark.gpu


def test_many_long_rows():
    # 2^22 + 3 rows of a workgroup of 1024 threads each (a launch takes fewer than 2^32 threads), in place
    M, N = (1 << 22) + 3, 16392
    if torch.cuda.mem_get_info()[0] < 3 * M * N:
        pytest.skip("needs %d GB free" % (3 * M * N >> 30))
    x = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, 4095, 1 << 20, 1 << 21, (1 << 22) - 1, 1 << 22, M - 1]
    v = ref.loud(len(rows), N, 5).bfloat16()
    for i, m in enumerate(rows):
        x[m] = v[i].cuda()
    gt.gt_rmsnorm(gt.make_rmsnorm_desc(x, None, x))
    torch.cuda.synchronize()
    _, _, want = ref.rmsnorm(v, None, None)
    got = torch.stack([x[m] for m in rows]).cpu()
    del x
    torch.cuda.empty_cache()
    ref.check(got, want, want.abs() * (ref.norm_rel(N) + 8 * ref.U), "y")
