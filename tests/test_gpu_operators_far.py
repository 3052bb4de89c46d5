"""The operators around the product where offsets, sizes and values are far
out: matrices past 2^31 elements and 2^32 bytes, rows longer than a
workgroup's registers, results stored past the caches, strides too wide for
the tiles, huge bf16 rows, strides and graphs of the two-launch forms.
References are computed on sampled rows and columns only.
"""
import pytest
import torch

import gemm_autotuning_amd as gt

from . import op_ref as ref

pytestmark = pytest.mark.gpu


def made(M, N, seed, dt=torch.bfloat16, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(M, N, dtype=dt, device="cuda")
    for m in range(0, M, 4096):  # in parts: the generator's fp32 values stay small
        t[m:m + 4096] = torch.randn(min(4096, M - m), N, generator=g, device="cuda") * std
    return t


@pytest.mark.parametrize("N", [65536, 32768, 16384])
def test_norm_and_gradient_past_31_bits_of_elements(N):
    # a norm and its gradient over 2.3 * 2^30 elements: the last rows start past 2^32 bytes
    M = (2 ** 31 + 2 ** 28) // N
    x, w = made(M, N, 1), made(1, N, 2)[0]
    y, rstd = torch.empty_like(x), torch.empty(M, device="cuda")
    gt.gt_rmsnorm(gt.make_rmsnorm_desc(x, w, y, rstd=rstd))
    rows = [0, 1, M // 2, M - 2, M - 1]
    xs, ws = x[rows].cpu(), w.cpu()
    _, r64, y64 = ref.rmsnorm(xs, None, ws)
    ref.check(y[rows].cpu(), y64, y64.abs() * (ref.norm_rel(N) + 8 * ref.U), "y")
    ref.check(rstd[rows].cpu(), r64, r64 * ref.norm_rel(N), "rstd")
    dy, dw = y, torch.empty(N, device="cuda")  # any dy will do
    dx = torch.empty_like(x)
    gt.gt_rmsnorm_backward(gt.make_rmsnorm_bwd_desc(dy, x, w, rstd, dx, dw))
    d64, _, far, _ = ref.rmsnorm_backward(dy[rows].cpu(), xs, ws, rstd[rows].cpu())
    ref.check(dx[rows].cpu(), d64, far, "dx")
    cols = slice(N - 64, N)
    n = x[:, cols].double() * rstd.double()[:, None]
    want = (dy[:, cols].double() * n).sum(dim=0).cpu()
    bound = ((M + 8) * ref.U * (dy[:, cols].double() * n).abs().sum(dim=0)).cpu()
    ref.check(dw[cols].cpu(), want, bound, "dw")


@pytest.mark.parametrize("dtype,N", [("bf16", 32769), ("f32", 16385), ("f32", 65536), ("f16", 65536)])
@pytest.mark.parametrize("quant", ["none", "row", "tensor"])
def test_rows_longer_than_the_registers_hold(dtype, N, quant):
    M, dt = 5, ref.DT[dtype]
    x, r = ref.loud(M, N, 3).to(dt), ref.loud(M, N, 4).to(dt)
    w = torch.randn(N, generator=ref.rng(5)).to(dt)
    X, R = x.cuda(), r.cuda()
    Y = torch.empty(M, N, dtype=dt if quant == "none" else torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(M, device="cuda") if quant == "row" else None
    gt.gt_rmsnorm(gt.make_rmsnorm_desc(X, w.cuda(), Y, residual=R, sum_out=R, row_scale=sc, quant=quant, scale=0.05))
    h, _, y = ref.rmsnorm(x, r, w)
    rel = ref.norm_rel(N)
    ref.check(R.cpu(), h, h.abs() * ref.U, "sum")
    if quant == "row":
        s = ref.row_scale(y)
        ref.check(sc.cpu(), s, s * (rel + 4 * ref.U), "scale")
        y = y / s[:, None]
    elif quant == "tensor":
        y = y / 0.05
    ref.check(Y.cpu(), y, y.abs() * (rel + 8 * ref.U), "y")


@pytest.mark.parametrize("pad", [0, 3])
def test_results_past_the_caches(pad):
    # enough bytes for the stores that bypass the caches, pads untouched
    M, N = 9001, 4100
    x, r, w = made(M, N + pad, 1)[:, :N], made(M, N + pad, 2)[:, :N], made(1, N, 3)[0]
    s, y = (torch.full((M, N + pad), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rstd = torch.empty(M, device="cuda")
    gt.gt_rmsnorm(gt.make_rmsnorm_desc(x, w, y[:, :N], residual=r, sum_out=s[:, :N], rstd=rstd))
    rows = [0, 1, 17, 4500, 8999, 9000]
    h, _, y64 = ref.rmsnorm(x[rows].cpu(), r[rows].cpu(), w.cpu())
    ref.check(s[rows, :N].cpu(), h, h.abs() * ref.U, "sum")
    ref.check(y[rows, :N].cpu(), y64, y64.abs() * (ref.norm_rel(N) + 8 * ref.U), "y")
    dx = torch.full((M, N + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
    gt.gt_rmsnorm_backward(gt.make_rmsnorm_bwd_desc(y[:, :N], s[:, :N], w, rstd, dx[:, :N], dsum=r))
    d64, _, far, _ = ref.rmsnorm_backward(y[rows, :N].cpu(), s[rows, :N].cpu(), w.cpu(), rstd[rows].cpu(), r[rows].cpu())
    ref.check(dx[rows, :N].cpu(), d64, far, "dx")
    for t in (s, y, dx):
        assert not torch.isnan(t[:, :N]).any()
        if pad:
            assert torch.isnan(t[:, N:].float()).all(), "pads written"


@pytest.mark.parametrize("fmt,out,pad", [("int4", "bf16", 0), ("e2m1", "f32", 5)])
def test_expansion_past_the_caches(fmt, out, pad):
    N, K = 13001, 9999
    q = torch.randint(0, 256, (N, K // 2 + 1), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda",
                      dtype=torch.uint8)
    s = torch.rand(N, -(-K // 64), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(torch.float16)
    y = torch.full((N, K + pad), float("nan"), device="cuda").to(ref.DT[out])
    gt.gt_w4_expand(gt.make_w4_expand_desc(q, s, y[:, :K], fmt, 64))
    rows = [0, 1, 2, 6500, 12999, 13000]
    want = ref.w4_weights(q[rows].cpu(), s[rows].cpu(), K, fmt, 64).float().to(ref.DT[out])
    assert torch.equal(y[rows, :K].cpu(), want)
    assert not torch.isnan(y[:, :K]).any() and (not pad or torch.isnan(y[:, K:].float()).all())


@pytest.mark.parametrize("x,fmt,group", [("bf16", "int4", 128), ("e4m3", "e2m1", 32)])
@pytest.mark.parametrize("M", [2, 40])
def test_weights_past_32_bits_of_bytes(x, fmt, group, M):
    # 5.2 GB of weights: the last columns start past 2^32 bytes
    N, K = 160001, 65536
    g = torch.Generator(device="cuda").manual_seed(7)
    q = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
    for n in range(0, N, 16384):
        q[n:n + 16384] = torch.randint(0, 256, (min(16384, N - n), K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (2.0 ** torch.randint(-9, -5, (N, K // group), generator=g, device="cuda").float()).bfloat16()
    v = torch.randint(-2, 3, (M, K), generator=ref.rng(8)).float().to(ref.DT[x])
    y = torch.empty(M, N, device="cuda")
    gt.gt_w4_matmul(gt.make_w4_desc(v.cuda(), q, s, y, fmt, group))
    cols = [0, 1, 15, 16, 80000, 131071, 131072, 131073, 159998, 160000]
    want, far = ref.w4_matmul(v, q[cols].cpu(), s[cols].cpu(), fmt, group)
    ref.check(y[:, cols].cpu(), want, far, "y")
    assert torch.isfinite(y).all()


def test_weight_rows_too_far_apart_for_the_tiles():
    # a row stride past the tiles' 32-bit offsets, over memory that is there
    N, K, ldq = 18, 96, 1 << 27
    buf = torch.zeros((N - 1) * ldq + K // 2, dtype=torch.uint8, device="cuda")
    q = torch.randint(0, 256, (N, K // 2), generator=ref.rng(9), dtype=torch.uint8)
    Q = buf.as_strided((N, K // 2), (ldq, 1))
    Q.copy_(q.cuda())
    s = torch.rand(N, 3, generator=ref.rng(10)) + 0.5
    v = torch.randint(-4, 5, (3, K), generator=ref.rng(11)).float().bfloat16()
    y = torch.empty(3, N, device="cuda")
    gt.gt_w4_matmul(gt.make_w4_desc(v.cuda(), Q, s.cuda(), y, "int4", 32))
    want, far = ref.w4_matmul(v, q, s, "int4", 32)
    ref.check(y.cpu(), want, far, "y")
    out = torch.empty(N, K, device="cuda")
    gt.gt_w4_expand(gt.make_w4_expand_desc(Q, s.cuda(), out, "int4", 32))
    w = ref.w4_weights(q, s, K, "int4", 32)
    ref.check(out.cpu(), w, w.abs() * ref.U, "w")


@pytest.mark.parametrize("M", [1, 13, 33])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("K", [640, 4096 + 96])
def test_huge_bf16_rows(M, group, K):
    # elements of 2^110..2^124 with integers: eight times an element must not overflow on the way
    N = 50
    g = ref.rng(12)
    v = torch.randn(M, K, generator=g).bfloat16()
    v[M // 2, 5] = 2.0 ** 124
    v[M // 2, K - 1] = -(2.0 ** 110)
    q = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    s = torch.full((N, -(-K // group)), 2.0 ** -3)
    y = torch.empty(M, N, device="cuda")
    gt.gt_w4_matmul(gt.make_w4_desc(v.cuda(), q.cuda(), s.cuda(), y, "int4", group))
    want, far = ref.w4_matmul(v, q, s, "int4", group)
    ref.check(y.cpu(), want, far, "y")


def test_outlier_with_a_zero_weight():
    # the largest element meets weights of zero: what is left must keep fp32's accuracy of its own terms and
    # of the element's part in the sums (eight times it, over a group)
    M, N, K = 4, 64, 2048
    v = torch.randn(M, K, generator=ref.rng(13)).bfloat16()
    v[:, 100] = 1000.0
    q = torch.randint(0, 256, (N, K // 2), generator=ref.rng(14), dtype=torch.uint8)
    q[:, 50] &= 0xF0  # k = 100
    s = torch.ones(N, K // 128)
    y = torch.empty(M, N, device="cuda")
    gt.gt_w4_matmul(gt.make_w4_desc(v.cuda(), q.cuda(), s.cuda(), y))
    want, far = ref.w4_matmul(v, q, s, "int4", 128)
    ref.check(y.cpu(), want, far + 16 * ref.U * 8 * 1000.0, "y")


@pytest.mark.parametrize("M,N,dtype", [(1500, 700, "bf16"), (3000, 130, "f32"), (700, 9000, "f16"), (1200, 16384, "f32"),
                                       (64, 20000, "bf16"), (1025, 33, "f16")])
def test_gradient_in_two_launches_into_a_graph(M, N, dtype):
    dt = ref.DT[dtype]
    h, dy, ds = (ref.loud(M, N, 20 + i).to(dt) for i in range(3))
    w = torch.randn(N, generator=ref.rng(23)).to(dt)
    rstd = ref.rmsnorm(h, None, None)[1].float()
    H, DY, DS, W, R = (t.cuda() for t in (h, dy, ds, w, rstd))
    DX, DW = torch.empty_like(H), torch.empty(N, device="cuda")
    st = torch.cuda.Stream()
    d = gt.make_rmsnorm_bwd_desc(DY, H, W, R, DX, DW, DS, stream=st.cuda_stream)
    torch.cuda.synchronize()
    gt.gt_rmsnorm_backward(d)
    st.synchronize()
    dx, dw, fx, fw = ref.rmsnorm_backward(dy, h, w, rstd, ds)
    ref.check(DX.cpu(), dx, fx, "dx")
    ref.check(DW.cpu(), dw, fw, "dw")
    first = DX.clone(), DW.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        gt.gt_rmsnorm_backward(d)
    for _ in range(3):
        DX.zero_()
        DW.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(DX, first[0]) and torch.equal(DW, first[1])


@pytest.mark.parametrize("M,N", [(100, 700), (513, 1000), (2000, 64)])
def test_the_gradients_forms_agree(M, N):
    # dx over dy takes two launches, dx beside it one where the rows are few: the same dx, and dw within its bound
    h, dy = ref.loud(M, N, 31).half(), ref.loud(M, N, 32).half()
    w = torch.randn(N, generator=ref.rng(33)).half()
    rstd = ref.rmsnorm(h, None, None)[1].float()
    H, W, R = h.cuda(), w.cuda(), rstd.cuda()
    out = []
    for over in (False, True):
        DY = dy.cuda()
        DX, DW = DY if over else torch.empty_like(DY), torch.empty(N, device="cuda")
        gt.gt_rmsnorm_backward(gt.make_rmsnorm_bwd_desc(DY, H, W, R, DX, DW))
        out.append((DX.cpu(), DW.cpu()))
    assert torch.equal(out[0][0], out[1][0])
    _, dw, _, fw = ref.rmsnorm_backward(dy, h, w, rstd)
    for _, DW in out:
        ref.check(DW, dw, fw, "dw")


def test_growing_the_workspace_under_capture_is_refused():
    # 64 rows of 32 slices: a workspace larger than any other test's, so that the stream cannot have it yet
    M, N, K = 64, 8192, 65536
    q = torch.full((N, K // 2), 0x11, dtype=torch.uint8, device="cuda")
    s = torch.ones(N, K // 128, device="cuda")
    x, y = torch.ones(M, K, device="cuda").bfloat16(), torch.zeros(M, N, device="cuda")
    st = torch.cuda.Stream()
    d = gt.make_w4_desc(x, q, s, y, stream=st.cuda_stream)
    marker = torch.zeros(1, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        marker.add_(1)
        with pytest.raises(gt.GemmTuneError, match="captur"):
            gt.gt_w4_matmul(d)
    graph.replay()
    torch.cuda.synchronize()
    assert marker.item() == 1.0 and (y == 0).all()
    gt.gt_w4_matmul(d)  # outside the capture the workspace is made
    st.synchronize()
    assert (y == float(K)).all()
