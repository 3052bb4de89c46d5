"""The experts' choice on the device against the 64-bit definition: every
width of row and number of choices, ties, masks, rows that nothing is left
of, NaN and infinities, strides, weights that underflow.
"""
import math

import pytest
import torch

import gemm_autotuning_amd as gt

from . import beside_ref as br
from . import op_ref as ref

pytestmark = pytest.mark.gpu


def run(logits, k, score="softmax", normalise=True, scale=1.0, pad=0):
    """(index, weight) on the CPU; inputs and outputs inside wider buffers."""
    x, _ = ref.padded(logits, pad)
    M = logits.shape[0]
    ib = torch.full((M, k + pad), 77, dtype=torch.int32, device="cuda")
    wb = torch.full((M, k + pad), 77.0, device="cuda")
    gt.gt_route(gt.make_route_desc(x, ib[:, :k], wb[:, :k], score=score, normalise=normalise, scale=scale,
                                   stream=torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert (ib[:, k:] == 77).all() and (wb[:, k:] == 77).all(), "pads written"
    return ib[:, :k].cpu(), wb[:, :k].cpu()


def same(logits, k, score="softmax", normalise=True, scale=1.0, pad=0):
    got_i, got_w = run(logits, k, score, normalise, scale, pad)
    want_i, want_w = br.route(logits, k, score, normalise, scale)
    assert torch.equal(got_i, want_i)
    # an exponential of an argument of magnitude a is off by (a + 2) u (a sum of positive terms by no
    # more, relatively, and its chain of at most 24 additions), a quotient and two products by 3 u more;
    # what is below fp32's range may be nothing
    fin = logits.double()[torch.isfinite(logits)]
    a = 2 * fin.abs().max().item() if fin.numel() else 0.0
    ref.check(got_w, want_w, want_w.abs() * (2 * a + 40) * br.U + 2.0 ** -126, "weights")


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (5, 3), (16, 16), (17, 8), (63, 4), (64, 8), (65, 17), (77, 3), (128, 8), (129, 1),
                                 (256, 16), (256, 17), (257, 8), (512, 8), (513, 2), (1024, 64), (1000, 6)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_sizes_and_types(E, k, dtype):
    g = ref.rng(E * 64 + k)
    for M, score, normalise in ((1, "softmax", True), (7, "sigmoid", True), (19, "softmax", False), (3, "sigmoid", False)):
        logits = (torch.randn(M, E, generator=g) * 3).to(ref.DT[dtype])  # 16-bit logits hold ties
        same(logits, k, score, normalise, 2.5 if normalise else 1.0, pad=M % 4)


@pytest.mark.parametrize("E,k", [(6, 4), (40, 8), (200, 8), (300, 20)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masks(E, k, score):
    g = ref.rng(E)
    for dtype in (torch.float32, torch.float16):
        logits = torch.randn(33, E, generator=g).to(dtype)
        logits[torch.rand(33, E, generator=g) < 0.5] = -math.inf
        logits[0] = -math.inf  # nothing is left
        logits[1] = -math.inf
        logits[1, E - 1] = torch.finfo(dtype).min  # the type's lowest value is a number
        logits[2] = torch.finfo(dtype).min
        for normalise in (True, False):
            same(logits, k, score, normalise)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_ties_go_to_the_lowest_index(dtype):
    for E in (10, 64, 100, 256, 1000):
        logits = torch.zeros(5, E)
        logits[1, 1::2] = -0.0  # the same number
        logits[2, E // 2:] = 1.0
        logits[3] = torch.arange(E) % 3
        logits[4] = torch.arange(E) // 2
        same(logits.to(ref.DT[dtype]), min(E, 16))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_nan_and_infinity(dtype):
    logits = torch.randn(6, 50, generator=ref.rng(1)).to(ref.DT[dtype])
    logits[0, 7] = math.nan
    logits[1, 7], logits[1, 30] = -math.nan, math.nan
    logits[2, 9] = math.inf
    logits[3] = math.nan
    logits[4, 20:] = -math.inf
    logits[4, 3] = math.nan
    for score in ("softmax", "sigmoid"):
        for normalise in (True, False):
            i, w = run(logits, 8, score, normalise)
            want_i, want_w = br.route(logits, 8, score, normalise)
            assert torch.equal(i, want_i)
            if score == "softmax":
                assert torch.isnan(w[:5]).any(dim=1).all()
            for m in (0, 1, 3, 4):
                assert torch.isnan(w[m, 0])
            clean = w[5]
            ref.check(clean, want_w[5], want_w[5].abs() * 60 * br.U)
    i, w = run(logits, 8, "sigmoid", False)
    assert w[2, 0] == 1.0 and not torch.isnan(w[0, 1:]).any()


def test_weights_far_out():
    # softmax of very different logits, and sigmoids that all underflow but for their quotients
    logits = torch.tensor([[1000.0, 0.0, -1000.0, 999.0], [-200.0, -201.0, -300.0, -200.5], [3e38, -3e38, 0.0, 3e38],
                           [-3e38, -3e38, -3e38, -3e38]])
    for score in ("softmax", "sigmoid"):
        i, w = run(logits, 4, score, True)
        want_i, want_w = br.route(logits, 4, score, True)
        assert torch.equal(i, want_i)
        assert ((w.double() - want_w).abs() <= want_w * 2.0 ** -10 + 2.0 ** -100).all(), (score, w, want_w)


def test_many_rows_and_a_graph():
    g = ref.rng(4)
    logits = torch.randn(20011, 96, generator=g)
    x = logits.cuda()
    index = torch.empty(20011, 6, dtype=torch.int32, device="cuda")
    weight = torch.empty(20011, 6, device="cuda")
    st = torch.cuda.Stream()
    d = gt.make_route_desc(x, index, weight, stream=st.cuda_stream)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        gt.gt_route(d)
    for turn in range(3):
        x.copy_(torch.roll(logits, turn, 1).cuda())
        index.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = torch.sort(x, dim=1, descending=True, stable=True)
        assert torch.equal(index.long(), want.indices[:, :6])
        w = torch.softmax(want.values[:, :6].double(), dim=1)
        assert ((weight.double() - w).abs() <= w * 60 * br.U).all()
