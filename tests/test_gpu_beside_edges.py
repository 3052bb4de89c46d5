"""Experts and adapters beside the product at the edges of what their calls
take: default strides of scales.
"""
import pytest
import torch

import gemm_autotuning_amd as gt

from . import beside_ref as br
from . import op_ref as ref

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("T", [2, 11])
@pytest.mark.parametrize("first", [True, False])
def test_scales_one_matrix_after_another_by_default(T, first):
    # lde <= 0: the experts' scales follow each other, whether a row's groups or a group's rows are neighbours
    E, k, K, H, group = 3, 2, 130, 96, 32
    (gu, gs), (dn, ds) = br.nibbles(E, 2 * H, K, group, "f32", 1), br.nibbles(E, K, H, group, "f32", 2)
    x, (index, weight) = ref.loud(T, K, 3).to(BF), br.choices(T, E, k, 4)
    y = torch.empty(T, K, device="cuda")

    def stored(t):
        return t.permute(0, 2, 1).contiguous().cuda().permute(0, 2, 1) if first else t.cuda()

    d = gt.make_moe_desc(x.cuda(), index.cuda(), weight.cuda(), gu.cuda(), dn.cuda(), y, gate_up_scales=stored(gs), down_scales=stored(ds),
                         format="int4", group=group, stream=stream())
    assert (d.gate_up_scale_ldn, d.gate_up_scale_ldg) == ((1, 2 * H) if first else (5, 1))
    d.gate_up_scale_lde = d.down_scale_lde = 0
    gt.gt_moe(d)
    torch.cuda.synchronize()
    want, far = br.moe(x, index, weight, gu, dn, gs, ds, "int4", group)
    ref.check(y.cpu(), want, far, "y")
