"""An operator whose workspace cannot be allocated: its status says so, and
nothing of it is left for the next check after a launch, the program's own or
torch's, to find; the call works once there is memory again.
"""
import pytest
import torch

import gemm_autotuning_amd as gt

from . import op_ref as ref

pytestmark = pytest.mark.gpu
OOM = 7


@pytest.mark.parametrize("op", ["w4", "gradient"])
def test_a_failed_workspace_leaves_nothing_behind(op):
    st = torch.cuda.Stream()
    if op == "w4":  # 60 MiB of partial sums: more than any stream has before
        M, N, K = 60, 16384, 32768
        q = torch.full((N, K // 2), 0x11, dtype=torch.uint8, device="cuda")
        d = gt.make_w4_desc(torch.ones(M, K, device="cuda").bfloat16(), q, torch.ones(N, K // 128, device="cuda"),
                            torch.zeros(M, N, device="cuda"), stream=st.cuda_stream)
        out, want, call = d.tensors[3], float(K), gt.gt_w4_matmul
    else:  # 64 rows of partial sums of 65536 columns
        M, N = 70, 65536
        h = torch.ones(M, N, device="cuda")
        d = gt.make_rmsnorm_bwd_desc(h, h, None, torch.ones(M, device="cuda"), None, torch.zeros(N, device="cuda"),
                                     stream=st.cuda_stream)
        out, want, call = d.tensors[6], float(M), gt.gt_rmsnorm_backward
    torch.cuda.synchronize()
    gt.gt_test_fail_allocs(1)
    try:
        with pytest.raises(gt.GemmTuneError) as e:
            call(d)
    finally:
        gt.gt_test_fail_allocs(0)
    assert e.value.status == OOM
    x = torch.randn(4, 64, device="cuda") + 1  # torch checks after its own launches
    y = torch.empty_like(x)
    gt.gt_rmsnorm(gt.make_rmsnorm_desc(x, None, y))
    torch.cuda.synchronize()
    _, _, y64 = ref.rmsnorm(x.cpu(), None, None)
    ref.check(y.cpu(), y64, y64.abs() * (ref.norm_rel(64) + 8 * ref.U), "y")
    assert (out == 0).all()
    call(d)
    st.synchronize()
    assert (out == want).all()
