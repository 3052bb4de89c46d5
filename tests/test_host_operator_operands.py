"""What the binding of the operators around the product refuses of a tensor
before its address reaches the library: rows that lie over each other
(broadcast ones among them, whose stride of 0 would read as "dense").
"""
import pytest
import torch

import gemm_autotuning_amd as gt

BF, M, N, K = torch.bfloat16, 3, 10, 64


def norm(**t):
    a = {k: torch.zeros(M, t.get("N", N), dtype=BF) for k in ("x", "residual", "sum_out", "y")}
    a.update((k, v) for k, v in t.items() if k != "N")
    return gt.make_rmsnorm_desc(a["x"], None, a["y"], residual=a["residual"], sum_out=a["sum_out"])


def bwd(**t):
    a = {k: torch.zeros(M, t.get("N", N), dtype=BF) for k in ("dy", "h", "dsum", "dx")}
    a.update((k, v) for k, v in t.items() if k != "N")
    return gt.make_rmsnorm_bwd_desc(a["dy"], a["h"], None, torch.zeros(M), a["dx"], dsum=a["dsum"])


def w4(**t):
    a = dict(x=torch.zeros(M, K, dtype=BF), qweight=torch.zeros(N, K // 2, dtype=torch.uint8), y=torch.zeros(M, N, dtype=BF))
    a.update(t)
    return gt.make_w4_desc(a["x"], a["qweight"], torch.zeros(N, 1), a["y"], group=64)


def expand(**t):
    a = dict(qweight=torch.zeros(N, K // 2, dtype=torch.uint8), out=torch.zeros(N, K, dtype=BF))
    a.update(t)
    return gt.make_w4_expand_desc(a["qweight"], torch.zeros(N, 1), a["out"], group=64)


OPERANDS = [(norm, "x", (M, N), BF), (norm, "residual", (M, N), BF), (norm, "sum_out", (M, N), BF), (norm, "y", (M, N), BF),
            (bwd, "dy", (M, N), BF), (bwd, "h", (M, N), BF), (bwd, "dsum", (M, N), BF), (bwd, "dx", (M, N), BF),
            (w4, "x", (M, K), BF), (w4, "qweight", (N, K // 2), torch.uint8), (w4, "y", (M, N), BF),
            (expand, "qweight", (N, K // 2), torch.uint8), (expand, "out", (N, K), BF)]
IDS = ["%s-%s" % (f.__name__, k) for f, k, _, _ in OPERANDS]


@pytest.mark.parametrize("make,name,shape,dtype", OPERANDS, ids=IDS)
def test_rows_over_each_other_are_refused(make, name, shape, dtype):
    rows, cols = shape
    make()  # dense operands are taken
    with pytest.raises(ValueError, match=name):
        make(**{name: torch.zeros(cols, dtype=dtype).expand(rows, cols)})
    for stride in (1, cols - 1):  # windows
        with pytest.raises(ValueError, match=name):
            make(**{name: torch.zeros(rows * cols, dtype=dtype).as_strided(shape, (stride, 1))})
    make(**{name: torch.zeros(rows, cols + 3, dtype=dtype)[:, :cols]})


@pytest.mark.parametrize("make,name", [(norm, n) for n in ("x", "residual", "sum_out", "y")] + [
    (bwd, n) for n in ("dy", "h", "dsum", "dx")])
def test_a_broadcast_column_is_refused(make, name):
    # rows of one element: the stride along them says nothing, the one between them does
    make(N=1)
    make(N=1, **{name: torch.zeros(M, 4, dtype=BF)[:, 1:2]})
    with pytest.raises(ValueError, match=name):
        make(N=1, **{name: torch.zeros(1, 1, dtype=BF).expand(M, 1)})


def test_the_gradient_of_a_sum_over_rows_is_refused():
    # what automatic differentiation hands over for y.sum(0): one row for all
    y = torch.zeros(M, N, requires_grad=True)
    seen = []
    y.register_hook(seen.append)
    (y.sum(0) * torch.ones(N)).sum().backward()
    assert seen[0].stride(0) == 0
    with pytest.raises(ValueError, match="dy"):
        gt.make_rmsnorm_bwd_desc(seen[0], torch.zeros(M, N), None, torch.zeros(M), torch.zeros(M, N))


def test_one_row_may_have_any_stride():
    x = torch.zeros(1, N, dtype=BF)
    one = torch.zeros(4, N, dtype=BF).as_strided((1, N), (0, 1))
    d = gt.make_rmsnorm_desc(one, None, x)
    assert d.ldx == N and d.ldy == N


def test_vectors_must_not_be_broadcast():
    with pytest.raises(ValueError, match="weight"):
        gt.make_rmsnorm_desc(torch.zeros(M, N), torch.zeros(1).expand(N), torch.zeros(M, N))
    with pytest.raises(ValueError, match="rstd"):
        gt.make_rmsnorm_bwd_desc(torch.zeros(M, N), torch.zeros(M, N), None, torch.zeros(1).expand(M), torch.zeros(M, N))
    with pytest.raises(ValueError, match="row_scale"):
        gt.make_w4_desc(torch.zeros(M, K, dtype=BF), torch.zeros(N, K // 2, dtype=torch.uint8), torch.zeros(N, 1),
                        torch.zeros(M, N), group=64, row_scale=torch.zeros(1).expand(M))


@pytest.mark.parametrize("op", ["norm", "bwd", "w4", "expand"])
def test_host_tensors_are_refused_before_a_launch(op):
    # the stand-in device takes every call that reaches the library
    make, call = {"norm": (norm, gt.gt_rmsnorm), "bwd": (bwd, gt.gt_rmsnorm_backward), "w4": (w4, gt.gt_w4_matmul),
                  "expand": (expand, gt.gt_w4_expand)}[op]
    gt.gt_test_fake_device(True, "f32", [1.0])
    try:
        with pytest.raises(ValueError, match="cpu"):
            call(make())
    finally:
        gt.gt_test_fake_device(False)


def test_tensors_of_two_devices_are_refused():
    with pytest.raises(ValueError, match="meta"):
        norm(residual=torch.zeros(M, N, dtype=BF, device="meta"))
