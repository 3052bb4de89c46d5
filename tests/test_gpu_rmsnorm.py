"""The RMS norm with the residual's addition and its backward pass on the
device, against the 64-bit formulas with derived bounds (tests/op_ref.py):
types, e4m3 outputs with both kinds of scale, ragged sizes and row strides,
rows of one element and of the most, zero and non-finite rows, results
written over their inputs, another stream, and graph replays.
"""
import pytest
import torch

import gemm_autotuning_amd as gt

from . import op_ref as ref

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 7), (3, 64), (4, 129), (5, 1000), (2, 4096), (37, 5001), (130, 2048), (1, 65536), (3, 40007),
          (2, 16384), (600, 100)]


def weight_of(kind, dtype, N, offset, seed):
    if kind == "none":
        return None
    w = torch.randn(N, generator=ref.rng(seed)) * 0.3 + 1.0 - offset
    return w.to(ref.DT[dtype if kind == "same" else kind])


def forward(M, N, dtype, out, quant, residual, wkind, offset=0.0, pad=0, eps=1e-6, scale=0.05, x=None, r=None, w=None):
    """Runs the call; (outputs on the CPU, inputs) with the pads checked."""
    x = ref.loud(M, N, 11).to(ref.DT[dtype]) if x is None else x
    if r is None and residual:
        r = ref.loud(M, N, 12, 3.0).to(ref.DT[dtype])
    w = weight_of(wkind, dtype, N, offset, 13) if w is None else w
    X, _ = ref.padded(x, pad)
    R = ref.padded(r, pad)[0] if r is not None else None
    S, sbuf = ref.padded(torch.zeros(M, N, dtype=x.dtype), pad)
    Y, ybuf = ref.padded(torch.zeros(M, N).to(ref.DT[out]), pad)
    rstd = torch.full((M,), -1.0, device="cuda")
    scales = torch.full((M,), -1.0, device="cuda")
    d = gt.make_rmsnorm_desc(X, None if w is None else w.cuda(), Y, residual=R, sum_out=S, rstd=rstd, row_scale=scales,
                             quant=quant, eps=eps, scale=scale, weight_offset=offset,
                             stream=torch.cuda.current_stream().cuda_stream)
    gt.gt_rmsnorm(d)
    torch.cuda.synchronize()
    if pad:
        assert torch.isnan(sbuf[:, N:].float()).all() and torch.isnan(ybuf[:, N:].float()).all(), "pads written"
    return (S.cpu(), Y.cpu(), rstd.cpu(), scales.cpu()), (x, r, w)


def check_forward(M, N, dtype, out, quant, residual, wkind, offset=0.0, pad=0, eps=1e-6, scale=0.05, **given):
    (S, Y, rstd, scales), (x, r, w) = forward(M, N, dtype, out, quant, residual, wkind, offset, pad, eps, scale, **given)
    h, r64, y = ref.rmsnorm(x, r, w, eps, offset)
    rel = ref.norm_rel(N)
    ref.check(S, h, h.abs() * ref.U, "sum")
    ref.check(rstd, r64, r64 * rel, "rstd")
    if quant == "row":
        sc = ref.row_scale(y)
        ref.check(scales, sc, sc * (rel + 4 * ref.U), "row scale")
        y = y / sc[:, None]
    elif quant == "tensor":
        y = y / scale
    if quant != "row":
        assert (scales == -1).all()
    ref.check(Y, y, y.abs() * (rel + 8 * ref.U), "y")


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("dtype,out,quant", [("bf16", "bf16", "none"), ("f16", "e4m3", "tensor"), ("f32", "f32", "none"),
                                             ("bf16", "e4m3", "row"), ("f32", "bf16", "none"), ("f16", "f32", "none"),
                                             ("f32", "e4m3", "row"), ("bf16", "f16", "none")])
def test_forward(M, N, dtype, out, quant):
    check_forward(M, N, dtype, out, quant, residual=(M + N) % 2 == 1 or N > 1000, wkind="same", pad=(M * 3 + N) % 5)


@pytest.mark.parametrize("wkind", ["none", "f32", "f16", "bf16"])
@pytest.mark.parametrize("offset", [0.0, 1.0])
@pytest.mark.parametrize("residual", [True, False])
def test_forward_weights(wkind, offset, residual):
    check_forward(9, 1537, "bf16", "bf16", "none", residual, wkind, offset, pad=8)


@pytest.mark.parametrize("pad", [0, 1, 2, 3, 4, 8])
@pytest.mark.parametrize("dtype,out,quant", [("bf16", "e4m3", "row"), ("f32", "f32", "none")])
def test_forward_strides(pad, dtype, out, quant):
    check_forward(33, 2040 + pad, dtype, out, quant, True, "f32", pad=pad)


def test_zero_rows():
    x = ref.loud(5, 300, 1).to(torch.bfloat16)
    x[2] = 0
    check_forward(5, 300, "bf16", "e4m3", "row", False, "same", x=x)
    (_, Y, rstd, scales), _ = forward(5, 300, "bf16", "e4m3", "row", False, "same", x=x)
    assert (Y[2].float() == 0).all() and abs(rstd[2].item() - 1000.0) < 1e-3
    assert scales[2].item() == pytest.approx(2.0 ** -100 / 448, rel=1e-6)


@pytest.mark.parametrize("dtype,out,quant", [("bf16", "bf16", "none"), ("f32", "f32", "none"), ("bf16", "e4m3", "row"),
                                             ("f16", "e4m3", "tensor")])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_row_stays_alone(dtype, out, quant, bad):
    x = ref.loud(6, 777, 2).to(ref.DT[dtype])
    x[3, 500] = bad
    (S, Y, rstd, scales), (_, r, w) = forward(6, 777, dtype, out, quant, True, "same", x=x)
    (S0, Y0, rstd0, scales0), _ = forward(6, 777, dtype, out, quant, True, "same", x=ref.loud(6, 777, 2).to(ref.DT[dtype]))
    rows = [0, 1, 2, 4, 5]
    assert torch.equal(Y[rows].float(), Y0[rows].float()) and torch.equal(rstd[rows], rstd0[rows])
    assert torch.equal(scales[rows], scales0[rows])
    # inf * (1 / inf) and anything times NaN: the formula's NaN, at the bad place at least
    assert torch.isnan(Y[3, 500].float())
    if quant == "row":
        assert torch.isnan(scales[3]) and torch.isnan(Y[3].float()).all()
    elif bad != bad:
        assert torch.isnan(Y[3].float()).all()
    else:
        assert (torch.cat((Y[3, :500], Y[3, 501:])).float() == 0).all() and rstd[3] == 0


def test_large_and_small_values():
    # sums of squares far from 1, inside fp32's range
    for std in (1e-12, 1e12):
        x = ref.loud(4, 512, 5, std)
        check_forward(4, 512, "f32", "f32", "none", False, "none", eps=0.0, x=x)


def test_saturation():
    x = ref.loud(4, 512, 6).to(torch.bfloat16)
    check_forward(4, 512, "bf16", "e4m3", "tensor", False, "same", scale=1e-3, x=x)


@pytest.mark.parametrize("N", [300, 4096, 30001])
@pytest.mark.parametrize("over", ["residual", "x", "y"])
def test_results_over_inputs(N, over):
    M = 7
    x, r = ref.loud(M, N, 21).to(torch.bfloat16), ref.loud(M, N, 22).to(torch.bfloat16)
    w = weight_of("same", "bf16", N, 0.0, 23)
    X, R, W = x.cuda(), r.cuda(), w.cuda()
    S = {"residual": R, "x": X, "y": torch.empty_like(X)}[over]
    Y = X if over == "y" else torch.empty_like(X)
    gt.gt_rmsnorm(gt.make_rmsnorm_desc(X, W, Y, residual=R, sum_out=S))
    h, _, y = ref.rmsnorm(x, r, w)
    ref.check(S.cpu(), h, h.abs() * ref.U, "sum")
    ref.check(Y.cpu(), y, y.abs() * (ref.norm_rel(N) + 8 * ref.U), "y")


def test_empty():
    x = torch.zeros(0, 16, device="cuda", dtype=torch.float16)
    gt.gt_rmsnorm(gt.make_rmsnorm_desc(x, None, x.clone()))


# ---- backward
def backward(M, N, dtype, dyt, dsum, wkind, dwt, offset=0.0, pad=0, want=("dx", "dw"), h=None):
    dt = ref.DT[dtype]
    h = ref.loud(M, N, 31).to(dt) if h is None else h
    dy = (torch.randn(M, N, generator=ref.rng(32)) * 0.1).to(ref.DT[dyt])
    ds = (torch.randn(M, N, generator=ref.rng(33)) * 0.1).to(dt) if dsum else None
    w = weight_of(wkind, dtype, N, offset, 34)
    rstd = ref.rmsnorm(h, None, None)[1].float()
    DX, buf = ref.padded(torch.zeros(M, N, dtype=dt), pad)
    DW = torch.full((N,), float("nan")).to(ref.DT[dwt]).cuda()
    d = gt.make_rmsnorm_bwd_desc(ref.padded(dy, pad)[0], ref.padded(h, pad)[0], None if w is None else w.cuda(), rstd.cuda(),
                                 DX if "dx" in want else None, DW if "dw" in want else None,
                                 dsum=None if ds is None else ref.padded(ds, pad)[0], weight_offset=offset)
    gt.gt_rmsnorm_backward(d)
    torch.cuda.synchronize()
    if pad:
        assert torch.isnan(buf[:, N:].float()).all(), "pads written"
    return DX.cpu(), DW.cpu(), ref.rmsnorm_backward(dy, h, w, rstd, ds, offset)


@pytest.mark.parametrize("M,N", SHAPES + [(4097, 64), (2000, 257), (300, 1031)])
@pytest.mark.parametrize("dtype,dyt", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
def test_backward(M, N, dtype, dyt):
    DX, DW, (dx, dw, fx, fw) = backward(M, N, dtype, dyt, (M + N) % 2 == 0, "same", "f32", pad=(M + N) % 4)
    ref.check(DX, dx, fx, "dx")
    ref.check(DW, dw, fw, "dw")


@pytest.mark.parametrize("wkind,dwt", [("none", "f32"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("offset", [0.0, 1.0])
@pytest.mark.parametrize("want", [("dx", "dw"), ("dx",), ("dw",)])
def test_backward_weights(wkind, dwt, offset, want):
    DX, DW, (dx, dw, fx, fw) = backward(70, 1537, "bf16", "f32", True, wkind, dwt, offset, 8, want)
    if "dx" in want:
        ref.check(DX, dx, fx, "dx")
    else:
        assert (DX == 0).all()
    if "dw" in want:
        ref.check(DW, dw, fw, "dw")
    else:
        assert torch.isnan(DW.float()).all()


def test_backward_of_no_rows_clears_the_weight_gradient():
    z = torch.zeros(0, 33, device="cuda")
    dw = torch.ones(33, device="cuda")
    gt.gt_rmsnorm_backward(gt.make_rmsnorm_bwd_desc(z, z, None, torch.zeros(0, device="cuda"), None, dw))
    assert (dw == 0).all()


@pytest.mark.parametrize("over", ["dy", "h", "dsum"])
@pytest.mark.parametrize("N", [640, 20001])
def test_gradient_over_its_inputs(over, N):
    M = 19
    t = {k: torch.randn(M, N, generator=ref.rng(i)).to(torch.bfloat16) for i, k in enumerate(("dy", "h", "dsum"))}
    w = weight_of("same", "bf16", N, 0.0, 4)
    rstd = ref.rmsnorm(t["h"], None, None)[1].float()
    dev = {k: v.cuda() for k, v in t.items()}
    dw = torch.empty(N, device="cuda")
    gt.gt_rmsnorm_backward(gt.make_rmsnorm_bwd_desc(dev["dy"], dev["h"], w.cuda(), rstd.cuda(), dev[over], dw, dev["dsum"]))
    dx, dw64, fx, fw = ref.rmsnorm_backward(t["dy"], t["h"], w, rstd, t["dsum"])
    ref.check(dev[over].cpu(), dx, fx, "dx")
    ref.check(dw.cpu(), dw64, fw, "dw")


def test_bad_gradient_row_stays_alone():
    h = ref.loud(40, 500, 31)
    DX, _, (dx, _, fx, _) = backward(40, 500, "f32", "f32", False, "same", "f32", h=h)
    bad = h.clone()
    bad[7, 3] = float("nan")
    DB, _, _ = backward(40, 500, "f32", "f32", False, "same", "f32", h=bad)
    keep = [i for i in range(40) if i != 7]
    assert torch.equal(DX[keep], DB[keep]) and torch.isnan(DB[7]).all()


def test_gradient_against_differences():
    # a loss of the device's own fp32 forward pass, central differences along random directions: truncation is
    # O(step^2), rounding about 2^-24 of the sum's terms over the step
    M, N, step = 4, 96, 2.0 ** -6
    g = ref.rng(41)
    x, dy = torch.randn(M, N, generator=g), torch.randn(M, N, generator=g)
    w = torch.randn(N, generator=g)

    def loss(x, w):
        y, rstd = torch.empty(M, N, device="cuda"), torch.empty(M, device="cuda")
        gt.gt_rmsnorm(gt.make_rmsnorm_desc(x.cuda(), w.cuda(), y, rstd=rstd))
        return (y.cpu().double() * dy.double()).sum().item(), rstd

    rstd = loss(x, w)[1]
    dx, dw = torch.empty(M, N, device="cuda"), torch.empty(N, device="cuda")
    gt.gt_rmsnorm_backward(gt.make_rmsnorm_bwd_desc(dy.cuda(), x.cuda(), w.cuda(), rstd, dx, dw))
    for t, grad in ((x, dx), (w, dw)):
        for i in range(3):
            e = torch.randn(t.shape, generator=ref.rng(50 + i))
            e /= e.norm()
            up, down = (loss(x + step * e, w), loss(x - step * e, w)) if t is x else (loss(x, w + step * e), loss(x, w - step * e))
            diff = (up[0] - down[0]) / (2 * step)
            want = (grad.cpu().double() * e.double()).sum().item()
            assert abs(diff - want) < 2e-3 * (1 + abs(want))


# ---- streams and graphs
def test_another_stream():
    M, N = 64, 4096
    s = torch.cuda.Stream()
    x = ref.loud(M, N, 61).to(torch.bfloat16)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    X = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    src = x.pin_memory()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        big = torch.ones(4096, 4096, device="cuda")
        for _ in range(4):
            big = big @ big * 1e-4
        X.copy_(src, non_blocking=True)
        gt.gt_rmsnorm(gt.make_rmsnorm_desc(X, None, y, stream=s.cuda_stream))
    s.synchronize()
    _, _, want = ref.rmsnorm(x, None, None)
    ref.check(y.cpu(), want, want.abs() * (ref.norm_rel(N) + 8 * ref.U), "y")


def test_graph_replays():
    M, N = 50, 1000
    x = torch.empty(M, N, device="cuda")
    y, dx, dw, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(N, device="cuda"), torch.empty(M, device="cuda")
    w = weight_of("same", "f32", N, 0.0, 3).cuda()
    dy = ref.loud(M, N, 4).cuda()

    def step(stream):
        gt.gt_rmsnorm(gt.make_rmsnorm_desc(x, w, y, rstd=rstd, stream=stream.cuda_stream))
        gt.gt_rmsnorm_backward(gt.make_rmsnorm_bwd_desc(dy, x, w, rstd, dx, dw, dsum=y, stream=stream.cuda_stream))

    s = torch.cuda.Stream()
    x.copy_(ref.loud(M, N, 70))
    torch.cuda.synchronize()
    step(s)  # the stream's workspace is made outside the capture
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step(s)
    for i in range(4):
        x.copy_(ref.loud(M, N, 71 + i))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, rstd, dx, dw)]
        step(torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, rstd, dx, dw)))
