"""Host side of the operators around the product: what they refuse, what they
take, and the 64-bit references the GPU tests compare with (the gradient
against differences and against automatic differentiation).
"""
import ctypes

import pytest
import torch

import gemm_autotuning_amd as gt

from . import op_ref as ref

P = 0x10000  # an aligned address that nothing reads: every call here ends before a launch


@pytest.fixture
def stand_in():
    gt.gt_test_fake_device(True, "f32", [1.0])
    yield
    gt.gt_test_fake_device(False)


def norm_desc(**kw):
    d = gt.RmsNormDesc(x=P, residual=P, weight=P, sum_out=P, y=P, rstd=P, row_scale=P, M=4, N=8, in_dtype=gt.BF16,
                       weight_dtype=-1, out_dtype=-1, quant=0, eps=1e-6, weight_offset=0.0, scale=1.0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def bwd_desc(**kw):
    d = gt.RmsNormBwdDesc(dy=P, h=P, weight=P, rstd=P, dsum=P, dx=P, dweight=P, M=4, N=8, in_dtype=gt.F16, dy_dtype=-1,
                          weight_dtype=-1, dweight_dtype=-1)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def w4_desc(**kw):
    d = gt.W4Desc(x=P, row_scale=None, qweight=P, scales=P, y=P, M=4, N=8, K=64, x_dtype=gt.BF16, out_dtype=-1, format=0,
                  scale_dtype=gt.BF16, group=32, x_scale=1.0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def expand_desc(**kw):
    d = gt.W4ExpandDesc(qweight=P, scales=P, out=P, N=8, K=64, out_dtype=gt.BF16, format=0, scale_dtype=gt.F16, group=128)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


CALLS = {"norm": (gt.gt_rmsnorm, norm_desc), "bwd": (gt.gt_rmsnorm_backward, bwd_desc),
         "w4": (gt.gt_w4_matmul, w4_desc), "expand": (gt.gt_w4_expand, expand_desc)}
INVALID, UNSUPPORTED = 1, 2
REFUSED = [
    ("norm", dict(x=None), INVALID), ("norm", dict(y=None), INVALID), ("norm", dict(M=-1), INVALID),
    ("norm", dict(N=-3), INVALID), ("norm", dict(in_dtype=9), INVALID), ("norm", dict(in_dtype=-1), INVALID),
    ("norm", dict(in_dtype=gt.FP8_E4M3), UNSUPPORTED), ("norm", dict(weight_dtype=gt.FP8_E4M3), UNSUPPORTED),
    ("norm", dict(weight_dtype=4), INVALID), ("norm", dict(out_dtype=7), INVALID),
    ("norm", dict(out_dtype=gt.FP8_E4M3), INVALID), ("norm", dict(out_dtype=gt.BF16, quant=1), INVALID),
    ("norm", dict(quant=3), INVALID), ("norm", dict(quant=-1), INVALID), ("norm", dict(quant=2, row_scale=None), INVALID),
    ("norm", dict(quant=1, scale=0.0), INVALID), ("norm", dict(quant=1, scale=-1.0), INVALID),
    ("norm", dict(quant=1, scale=float("nan")), INVALID), ("norm", dict(quant=1, scale=float("inf")), INVALID),
    ("norm", dict(eps=-1e-6), INVALID), ("norm", dict(eps=float("nan")), INVALID), ("norm", dict(eps=float("inf")), INVALID),
    ("norm", dict(weight_offset=float("inf")), INVALID), ("norm", dict(ldx=7), INVALID), ("norm", dict(ldr=7), INVALID),
    ("norm", dict(lds=7), INVALID), ("norm", dict(ldy=7), INVALID), ("norm", dict(N=65537), UNSUPPORTED),
    ("norm", dict(x=P + 1), INVALID), ("norm", dict(residual=P + 1), INVALID), ("norm", dict(rstd=P + 2), INVALID),
    ("norm", dict(ldx=1 << 62), INVALID),
    ("bwd", dict(dy=None), INVALID), ("bwd", dict(h=None), INVALID), ("bwd", dict(rstd=None), INVALID),
    ("bwd", dict(dx=None, dweight=None), INVALID), ("bwd", dict(M=-1), INVALID), ("bwd", dict(N=65537), UNSUPPORTED),
    ("bwd", dict(in_dtype=gt.FP8_E4M3), UNSUPPORTED), ("bwd", dict(dy_dtype=gt.BF16), UNSUPPORTED),
    ("bwd", dict(dweight_dtype=gt.FP8_E4M3), UNSUPPORTED), ("bwd", dict(weight_dtype=5), INVALID),
    ("bwd", dict(lddx=3), INVALID), ("bwd", dict(ldds=3), INVALID), ("bwd", dict(dsum=P + 1), INVALID),
    ("bwd", dict(dweight=P + 2), INVALID), ("bwd", dict(weight_offset=float("nan")), INVALID),
    ("w4", dict(x=None), INVALID), ("w4", dict(qweight=None), INVALID), ("w4", dict(scales=None), INVALID),
    ("w4", dict(y=None), INVALID), ("w4", dict(M=-1), INVALID), ("w4", dict(N=-1), INVALID), ("w4", dict(K=-1), INVALID),
    ("w4", dict(x_dtype=gt.F32), UNSUPPORTED), ("w4", dict(x_dtype=4), INVALID), ("w4", dict(x_dtype=-1), INVALID),
    ("w4", dict(out_dtype=gt.FP8_E4M3), UNSUPPORTED), ("w4", dict(scale_dtype=gt.FP8_E4M3), UNSUPPORTED),
    ("w4", dict(scale_dtype=-1), INVALID), ("w4", dict(format=2), INVALID), ("w4", dict(format=-1), INVALID),
    ("w4", dict(group=0), INVALID), ("w4", dict(group=16), INVALID), ("w4", dict(group=256), INVALID),
    ("w4", dict(ldx=63), INVALID), ("w4", dict(ldq=31), INVALID), ("w4", dict(ldy=7), INVALID),
    ("w4", dict(K=65, ldq=32), INVALID), ("w4", dict(x=P + 1), INVALID), ("w4", dict(scales=P + 1), INVALID),
    ("w4", dict(row_scale=P + 2), INVALID), ("w4", dict(x_scale=float("inf")), INVALID), ("w4", dict(ldq=1 << 62), INVALID),
    ("expand", dict(qweight=None), INVALID), ("expand", dict(scales=None), INVALID), ("expand", dict(out=None), INVALID),
    ("expand", dict(out_dtype=gt.FP8_E4M3), UNSUPPORTED), ("expand", dict(out_dtype=-1), INVALID),
    ("expand", dict(ldo=63), INVALID), ("expand", dict(group=1), INVALID), ("expand", dict(N=-1), INVALID),
    ("expand", dict(out=P + 1), INVALID),
]


@pytest.mark.parametrize("op,change,status", REFUSED, ids=["%s-%s" % (o, "-".join(c)) + str(i) for i, (o, c, _) in enumerate(REFUSED)])
def test_refused(stand_in, op, change, status):
    call, make = CALLS[op]
    with pytest.raises(gt.GemmTuneError) as e:
        call(make(**change))
    assert e.value.status == status
    assert gt.gt_last_error()


def test_null_descriptors_are_refused():
    L = gt.lib()
    for f in (L.gt_rmsnorm, L.gt_rmsnorm_backward, L.gt_w4_matmul, L.gt_w4_expand):
        assert f(None) == INVALID


TAKEN = [
    ("norm", {}), ("norm", dict(quant=1)), ("norm", dict(quant=2)), ("norm", dict(out_dtype=gt.F32)),
    ("norm", dict(residual=None, weight=None, sum_out=None, rstd=None, row_scale=None)), ("norm", dict(N=65536)),
    ("norm", dict(M=0, x=None, y=None)), ("norm", dict(N=0, x=None, y=None)), ("norm", dict(ldx=9, ldy=1000)),
    ("bwd", {}), ("bwd", dict(dx=None)), ("bwd", dict(dweight=None, dsum=None, weight=None)), ("bwd", dict(dy_dtype=gt.F32)),
    ("bwd", dict(M=0, dy=None, h=None, rstd=None)), ("bwd", dict(N=0)),
    ("w4", {}), ("w4", dict(x_dtype=gt.FP8_E4M3, row_scale=P)), ("w4", dict(K=1)), ("w4", dict(K=0, x=None, qweight=None)),
    ("w4", dict(M=0)), ("w4", dict(N=0)), ("w4", dict(qweight=P + 1, ldq=33)), ("w4", dict(scale_ldn=1, scale_ldg=8)),
    ("expand", {}), ("expand", dict(K=0)), ("expand", dict(N=0)), ("expand", dict(K=63, out_dtype=gt.F32)),
]


@pytest.mark.parametrize("op,change", TAKEN, ids=["%s-%d" % (o, i) for i, (o, _) in enumerate(TAKEN)])
def test_taken(stand_in, op, change):
    call, make = CALLS[op]
    call(make(**change))


def test_descriptor_sizes_match_the_header():
    # the C structs have no padding but the tail's, so the sizes pin the layout
    assert ctypes.sizeof(gt.RmsNormDesc) == 7 * 8 + 6 * 8 + 4 * 4 + 3 * 4 + 4 + 8
    assert ctypes.sizeof(gt.RmsNormBwdDesc) == 7 * 8 + 6 * 8 + 4 * 4 + 4 + 4 + 8
    assert ctypes.sizeof(gt.W4Desc) == 5 * 8 + 8 * 8 + 5 * 4 + 4 + 8
    assert ctypes.sizeof(gt.W4ExpandDesc) == 3 * 8 + 6 * 8 + 4 * 4 + 8


# ---- the binding's own checks
def test_binding_reads_shapes_strides_and_types():
    x = torch.zeros(3, 20, dtype=torch.bfloat16)[:, :10]
    y = torch.zeros(3, 10, dtype=torch.float8_e4m3fn)
    rs = torch.zeros(3)
    d = gt.make_rmsnorm_desc(x, torch.ones(10), y, row_scale=rs, quant="row")
    assert (d.M, d.N, d.ldx, d.ldy, d.in_dtype, d.weight_dtype, d.out_dtype, d.quant) == (3, 10, 20, 10, 2, 0, 3, 2)
    s = torch.zeros(2, 16, dtype=torch.float16)
    q = torch.zeros(16, 40, dtype=torch.uint8)[:, :33]
    w = gt.make_w4_desc(torch.zeros(1, 65, dtype=torch.float16), q, s.t(), torch.zeros(1, 16), group=64)
    assert (w.M, w.N, w.K, w.ldq, w.scale_ldn, w.scale_ldg, w.out_dtype) == (1, 16, 65, 40, 1, 16, 0)


@pytest.mark.parametrize("wrong", ["shape", "type", "stride", "scales", "vector", "group", "bytes", "broadcast"])
def test_binding_refuses(wrong):
    x, y = torch.zeros(3, 10, dtype=torch.bfloat16), torch.zeros(3, 10, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 5, dtype=torch.uint8), torch.zeros(4, 1)
    with pytest.raises(ValueError):
        if wrong == "shape":
            gt.make_rmsnorm_desc(x, None, y[:2])
        elif wrong == "type":
            gt.make_rmsnorm_desc(x, None, y, residual=x.float())
        elif wrong == "stride":
            gt.make_rmsnorm_desc(torch.zeros(10, 3, dtype=torch.bfloat16).t(), None, y)
        elif wrong == "scales":
            gt.make_w4_desc(x, q, torch.zeros(4, 2), torch.zeros(3, 4))
        elif wrong == "vector":
            gt.make_rmsnorm_desc(x, torch.ones(9), y)
        elif wrong == "group":
            gt.make_w4_desc(x, q, s, torch.zeros(3, 4), group=48)
        elif wrong == "bytes":
            gt.make_w4_expand_desc(q.int(), s, torch.zeros(4, 10))
        else:
            gt.make_w4_expand_desc(q, torch.zeros(1, 1).expand(4, 1), torch.zeros(4, 10))


# ---- the references
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_reference_gradient_against_differentiation(offset):
    g = ref.rng(3)
    M, N = 3, 7
    x = torch.randn(M, N, generator=g, dtype=torch.float64)
    w = torch.randn(N, generator=g, dtype=torch.float64)
    dy = torch.randn(M, N, generator=g, dtype=torch.float64)
    ds = torch.randn(M, N, generator=g, dtype=torch.float64)

    def value(x, w):
        h, _, y = ref.rmsnorm(x, None, w, 1e-3, offset)
        return (y * dy).sum() + (h * ds).sum()

    rstd = ref.rmsnorm(x, None, w, 1e-3, offset)[1]
    dx, dw, _, _ = ref.rmsnorm_backward(dy, x, w, rstd, ds, offset)
    xa, wa = x.clone().requires_grad_(), w.clone().requires_grad_()
    value(xa, wa).backward()
    assert torch.allclose(dx, xa.grad, rtol=1e-12, atol=1e-13) and torch.allclose(dw, wa.grad, rtol=1e-12, atol=1e-13)
    step = 1e-5
    for t, grad in ((x, dx), (w, dw)):
        for i in range(t.numel()):
            e = torch.zeros(t.numel(), dtype=torch.float64)
            e[i] = step
            e = e.reshape(t.shape)
            up = value(x + e, w) if t is x else value(x, w + e)
            down = value(x - e, w) if t is x else value(x, w - e)
            assert abs((up - down) / (2 * step) - grad.flatten()[i]) < 1e-7


def test_reference_nibbles():
    q = torch.tensor([[0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE]], dtype=torch.uint8)
    assert ref.w4_values(q, 16, "int4")[0].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1]
    assert ref.w4_values(q, 15, "e2m1")[0].tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4]
