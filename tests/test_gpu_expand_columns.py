"""Expanded 4-bit weights at the numbers of columns where the threads of a
row change: a power of two of pieces, one more and one less, a row's rest
alone, and rows that need several workgroups.
"""
import pytest
import torch

import gemm_autotuning_amd as gt

from . import op_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [1, 3, 4, 5, 7, 8, 9, 63, 64, 65, 71, 127, 128, 512, 1023, 1024, 1025, 1031, 2047, 2048, 2049, 2055,
                               4096, 4103, 8192, 8193])
@pytest.mark.parametrize("N", [1, 70, 2100])
@pytest.mark.parametrize("out,fmt,group", [("bf16", "int4", 128), ("f16", "e2m1", 32), ("f32", "int4", 64)])
def test_columns(N, K, out, fmt, group):
    q = torch.randint(0, 256, (N, -(-K // 2)), generator=ref.rng(K), dtype=torch.uint8)
    s = (torch.rand(N, -(-K // group), generator=ref.rng(N)) + 0.5).half()
    y = torch.full((N, K + 3), float("nan"), device="cuda").to(ref.DT[out])
    gt.gt_w4_expand(gt.make_w4_expand_desc(q.cuda(), s.cuda(), y[:, :K], fmt, group))
    torch.cuda.synchronize()
    # a 16-bit scale times a code is exact in fp32: rounded once
    want = (ref.w4_values(q, K, fmt).float() * s.float().repeat_interleave(group, dim=1)[:, :K]).to(ref.DT[out])
    assert torch.equal(y[:, :K].cpu(), want)
    assert torch.isnan(y[:, K:].float()).all(), "pads written"
