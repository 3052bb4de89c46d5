"""Host side of experts and adapters beside the product: what the entry points
and the binding refuse and take (nothing launched), their workspaces' sizes,
and the 64-bit references against plain torch.
"""
import ctypes
import math

import pytest
import torch

import gemm_autotuning_amd as gt

from . import beside_ref as br
from . import op_ref as ref

P = 0x10000  # an aligned address that nothing reads: every call here ends before a launch


@pytest.fixture
def stand_in():
    gt.gt_test_fake_device(True, "f32", [1.0])
    yield
    gt.gt_test_fake_device(False)


def make(cls, kw, change):
    d = cls(**kw)
    for k, v in change.items():
        setattr(d, k, v)
    return d


def route_desc(**c):
    return make(gt.RouteDesc, dict(logits=P, index=P, weight=P, M=4, E=16, topk=2, dtype=gt.F32, scale=1.0), c)


def moe_desc(**c):
    return make(gt.MoeDesc, dict(x=P, index=P, weight=P, gate_up=P, gate_up_scales=P, down=P, down_scales=P, base=P, y=2 * P, M=4, K=64,
                                 H=32, E=8, topk=2, x_dtype=gt.BF16, out_dtype=-1, format=-1, scale_dtype=gt.BF16, group=32), c)


def lora_desc(**c):
    return make(gt.LoraDesc, dict(x=P, index=P, a=P, b=P, scale=P, base=P, y=2 * P, M=4, K=64, N=32, adapters=8, rank=16,
                                  x_dtype=gt.F16, out_dtype=-1), c)


CALLS = {"route": (gt.gt_route, route_desc), "moe": (gt.gt_moe, moe_desc), "lora": (gt.gt_lora, lora_desc)}
INVALID, UNSUPPORTED = 1, 2
FAR = 1 << 62
REFUSED = [
    ("route", dict(logits=None), INVALID), ("route", dict(index=None), INVALID), ("route", dict(weight=None), INVALID),
    ("route", dict(M=-1), INVALID), ("route", dict(E=-1), INVALID), ("route", dict(topk=0), INVALID), ("route", dict(topk=-1), INVALID),
    ("route", dict(topk=17), INVALID), ("route", dict(E=0), INVALID), ("route", dict(E=1025), UNSUPPORTED),
    ("route", dict(E=100, topk=65), UNSUPPORTED), ("route", dict(dtype=gt.FP8_E4M3), UNSUPPORTED), ("route", dict(dtype=-1), INVALID),
    ("route", dict(dtype=4), INVALID), ("route", dict(score=2), INVALID), ("route", dict(score=-1), INVALID),
    ("route", dict(normalise=2), INVALID), ("route", dict(scale=math.nan), INVALID), ("route", dict(scale=math.inf), INVALID),
    ("route", dict(ldl=15), INVALID), ("route", dict(ldi=1), INVALID), ("route", dict(ldw=1), INVALID),
    ("route", dict(logits=P + 2), INVALID), ("route", dict(index=P + 2), INVALID), ("route", dict(weight=P + 1), INVALID),
    ("route", dict(ldl=FAR), INVALID),
    ("moe", dict(x=None), INVALID), ("moe", dict(index=None), INVALID), ("moe", dict(weight=None), INVALID),
    ("moe", dict(gate_up=None), INVALID), ("moe", dict(down=None), INVALID), ("moe", dict(y=None), INVALID),
    ("moe", dict(M=-1), INVALID), ("moe", dict(K=-1), INVALID), ("moe", dict(H=-1), INVALID), ("moe", dict(E=-1), INVALID),
    ("moe", dict(topk=-1), INVALID), ("moe", dict(E=4097), UNSUPPORTED), ("moe", dict(topk=65), UNSUPPORTED),
    ("moe", dict(K=(1 << 30) + 1), UNSUPPORTED), ("moe", dict(H=(1 << 30) + 1), UNSUPPORTED),
    ("moe", dict(K=(1 << 24) + 1), UNSUPPORTED), ("moe", dict(H=(1 << 24) + 1), UNSUPPORTED),
    ("moe", dict(x_dtype=gt.F32), UNSUPPORTED), ("moe", dict(x_dtype=gt.FP8_E4M3), UNSUPPORTED), ("moe", dict(x_dtype=-1), INVALID),
    ("moe", dict(out_dtype=gt.FP8_E4M3), UNSUPPORTED), ("moe", dict(out_dtype=7), INVALID), ("moe", dict(format=2), INVALID),
    ("moe", dict(format=-2), INVALID), ("moe", dict(activation=2), INVALID), ("moe", dict(activation=-1), INVALID),
    ("moe", dict(format=0, group=16), INVALID), ("moe", dict(format=0, scale_dtype=gt.FP8_E4M3), UNSUPPORTED),
    ("moe", dict(format=0, scale_dtype=-1), INVALID), ("moe", dict(format=0, gate_up_scales=None), INVALID),
    ("moe", dict(format=1, down_scales=None), INVALID), ("moe", dict(format=0, gate_up_scales=P + 1), INVALID),
    ("moe", dict(format=1, scale_dtype=gt.F32, down_scales=P + 2), INVALID),
    ("moe", dict(ldx=63), INVALID), ("moe", dict(ldi=1), INVALID), ("moe", dict(ldw=1), INVALID), ("moe", dict(ldb=63), INVALID),
    ("moe", dict(ldy=63), INVALID), ("moe", dict(gate_up_ld=63), INVALID), ("moe", dict(down_ld=31), INVALID),
    ("moe", dict(gate_up_stride=63), INVALID), ("moe", dict(down_stride=31), INVALID), ("moe", dict(format=0, gate_up_ld=31), INVALID),
    ("moe", dict(format=0, down_ld=15), INVALID), ("moe", dict(gate_up_ld=FAR), INVALID), ("moe", dict(gate_up_stride=FAR), INVALID),
    ("moe", dict(format=0, gate_up_scale_ldn=FAR), INVALID), ("moe", dict(format=0, down_scale_lde=FAR), INVALID),
    ("moe", dict(format=0, down_scale_ldg=FAR), INVALID), ("moe", dict(ldy=FAR), INVALID),
    ("moe", dict(x=P + 1), INVALID), ("moe", dict(gate_up=P + 1), INVALID), ("moe", dict(down=P + 1), INVALID),
    ("moe", dict(index=P + 2), INVALID), ("moe", dict(weight=P + 2), INVALID), ("moe", dict(base=P + 1), INVALID),
    ("moe", dict(y=P, base=P, ldb=70), INVALID), ("moe", dict(workspace=P, workspace_bytes=16), INVALID),
    ("moe", dict(workspace=P + 8, workspace_bytes=1 << 30), INVALID), ("moe", dict(workspace=None, workspace_bytes=1 << 30), INVALID),
    ("moe", dict(workspace=P, workspace_bytes=-1), INVALID),
    ("lora", dict(x=None), INVALID), ("lora", dict(index=None), INVALID), ("lora", dict(a=None), INVALID), ("lora", dict(b=None), INVALID),
    ("lora", dict(y=None), INVALID), ("lora", dict(M=-1), INVALID), ("lora", dict(K=-1), INVALID), ("lora", dict(N=-1), INVALID),
    ("lora", dict(adapters=-1), INVALID), ("lora", dict(rank=-1), INVALID), ("lora", dict(adapters=4097), UNSUPPORTED),
    ("lora", dict(rank=257), UNSUPPORTED), ("lora", dict(K=(1 << 30) + 1), UNSUPPORTED), ("lora", dict(N=(1 << 30) + 1), UNSUPPORTED),
    ("lora", dict(K=(1 << 24) + 1), UNSUPPORTED), ("lora", dict(N=(1 << 24) + 1), UNSUPPORTED),
    ("lora", dict(x_dtype=gt.F32), UNSUPPORTED), ("lora", dict(x_dtype=9), INVALID), ("lora", dict(out_dtype=gt.FP8_E4M3), UNSUPPORTED),
    ("lora", dict(ldx=63), INVALID), ("lora", dict(ldb=31), INVALID), ("lora", dict(ldy=31), INVALID), ("lora", dict(a_ld=63), INVALID),
    ("lora", dict(b_ld=15), INVALID), ("lora", dict(a_stride=63), INVALID), ("lora", dict(b_stride=15), INVALID),
    ("lora", dict(a_ld=FAR), INVALID), ("lora", dict(b_stride=FAR), INVALID), ("lora", dict(ldx=FAR), INVALID),
    ("lora", dict(y=P), INVALID), ("lora", dict(x=P + 1), INVALID), ("lora", dict(a=P + 1), INVALID), ("lora", dict(b=P + 1), INVALID), ("lora", dict(scale=P + 2), INVALID),
    ("lora", dict(index=P + 1), INVALID), ("lora", dict(y=P, base=P, ldy=40), INVALID), ("lora", dict(workspace=P, workspace_bytes=16), INVALID),
    ("lora", dict(workspace=P + 4, workspace_bytes=1 << 30), INVALID),
]


@pytest.mark.parametrize("op,change,status", REFUSED, ids=["%s-%s%d" % (o, "-".join(c), i) for i, (o, c, _) in enumerate(REFUSED)])
def test_refused(stand_in, op, change, status):
    call, desc = CALLS[op]
    with pytest.raises(gt.GemmTuneError) as e:
        call(desc(**change))
    assert e.value.status == status
    assert gt.gt_last_error()


TAKEN = [
    ("route", {}), ("route", dict(M=0, logits=None, index=None, weight=None)), ("route", dict(E=1024, topk=64)),
    ("route", dict(E=1, topk=1, dtype=gt.F16)), ("route", dict(ldl=20, ldi=3, ldw=5, score=1, normalise=1)),
    ("moe", {}), ("moe", dict(base=None)), ("moe", dict(base=P, y=P)), ("moe", dict(format=0)), ("moe", dict(format=1, group=128)),
    ("moe", dict(M=0, x=None, y=None, index=None)), ("moe", dict(K=0, x=None, gate_up=None, down=None, y=None)),
    ("moe", dict(H=0, gate_up=None, down=None)), ("moe", dict(E=0, gate_up=None, down=None)), ("moe", dict(topk=0, index=None, weight=None)),
    ("moe", dict(E=4096, topk=64, x_dtype=gt.F16, out_dtype=gt.F32)), ("moe", dict(workspace=P, workspace_bytes=1 << 26)),
    ("moe", dict(gate_up_ld=8 * 64, gate_up_stride=64)), ("moe", dict(format=0, gate_up=P + 1, down=P + 3)),
    ("moe", dict(gate_up_scales=None, down_scales=None)),
    ("lora", {}), ("lora", dict(base=None, scale=None)), ("lora", dict(base=2 * P, y=2 * P)), ("lora", dict(M=0, x=None, y=None)),
    ("lora", dict(N=0, b=None, y=None)), ("lora", dict(rank=0, a=None, b=None)), ("lora", dict(K=0, x=None)),
    ("lora", dict(adapters=0, a=None, b=None)), ("lora", dict(adapters=4096, rank=256)), ("lora", dict(workspace=P, workspace_bytes=1 << 26)),
]


@pytest.mark.parametrize("op,change", TAKEN, ids=["%s-%d" % (o, i) for i, (o, _) in enumerate(TAKEN)])
def test_taken(stand_in, op, change):
    call, desc = CALLS[op]
    call(desc(**change))


def test_x_that_is_y(stand_in):
    gt.gt_moe(moe_desc(x=2 * P, y=2 * P))
    gt.gt_moe(moe_desc(x=2 * P, y=2 * P, base=2 * P, ldx=70, ldy=70, ldb=70))
    gt.gt_moe(moe_desc(x=2 * P, y=2 * P, E=0, out_dtype=gt.F32))  # x is not read
    for change in (dict(out_dtype=gt.F32), dict(out_dtype=gt.F16), dict(ldy=70), dict(ldx=70)):
        with pytest.raises(gt.GemmTuneError) as e:
            gt.gt_moe(moe_desc(x=2 * P, y=2 * P, **change))
        assert e.value.status == INVALID


def test_null_arguments_are_refused(stand_in):
    L = gt.lib()
    n = ctypes.c_int64(7)
    for f in (L.gt_route, L.gt_moe, L.gt_lora):
        assert f(None) == INVALID
    for f, d in ((L.gt_moe_workspace, moe_desc()), (L.gt_lora_workspace, lora_desc())):
        assert f(None, ctypes.byref(n)) == INVALID and f(ctypes.byref(d), None) == INVALID


def test_workspaces(stand_in):
    # enough is enough, a byte less is refused; bounded however many rows there are, pointers not looked at
    for size, (call, desc) in ((gt.gt_moe_workspace, CALLS["moe"]), (gt.gt_lora_workspace, CALLS["lora"])):
        n = size(desc(x=None, y=None, index=None))
        assert 0 < n < 1 << 20
        call(desc(workspace=P, workspace_bytes=n))
        with pytest.raises(gt.GemmTuneError):
            call(desc(workspace=P, workspace_bytes=n - 1))
        assert size(desc(M=0)) == 0
        most = size(desc(M=1 << 40))
        assert n < most <= (64 << 20) + (2 << 20)
        call(desc(M=1 << 20, workspace=P, workspace_bytes=most))
    assert gt.gt_moe_workspace(moe_desc(H=0)) == 0 and gt.gt_lora_workspace(lora_desc(rank=0)) == 0
    with pytest.raises(gt.GemmTuneError):
        gt.gt_moe_workspace(moe_desc(x_dtype=gt.F32))


def test_a_layers_workspace_is_what_its_kernels_use(stand_in):
    # without tiles (one token, few that hardly share experts, rows shorter than 16 bytes, rows too far
    # apart) only the activations
    for change in (dict(M=1, K=65536, H=65536, E=64, topk=64, format=0), dict(M=1, K=4096, H=2048, E=4, topk=64),
                   dict(M=3, K=2048, H=768, E=128, topk=8), dict(M=100, K=4, H=24), dict(M=20, gate_up_ld=1 << 28)):
        d = moe_desc(**{**change, "gate_up": None, "gate_up_scales": None})
        assert gt.gt_moe_workspace(d) == d.M * d.topk * d.H * 4, change
    # about 64 MiB however long the rows, or one token's activations
    for K in (64, 4096, 65536, 1 << 24):
        for H in (64, 14336, 65536, 1 << 24):
            for topk in (1, 8, 64):
                for f in (-1, 0):
                    for M in (1, 7, 64, 1000, 1 << 20):
                        d = moe_desc(M=M, K=K, H=H, E=64, topk=topk, format=f)
                        assert 0 < gt.gt_moe_workspace(d) <= max(81 << 20, topk * H * 4), (M, K, H, topk, f)
    for bad in (dict(gate_up_stride=63), dict(down_ld=31), dict(format=0, down_scale_ldg=FAR)):
        with pytest.raises(gt.GemmTuneError):
            gt.gt_moe_workspace(moe_desc(**bad))


def test_descriptor_sizes_match_the_header():
    assert ctypes.sizeof(gt.RouteDesc) == 3 * 8 + 6 * 8 + 3 * 4 + 4 + 8
    assert ctypes.sizeof(gt.MoeDesc) == 10 * 8 + 21 * 8 + 6 * 4 + 8
    assert ctypes.sizeof(gt.LoraDesc) == 8 * 8 + 13 * 8 + 2 * 4 + 8


# ---- the binding's own checks
def tensors(**change):
    T, K, H, E, k = 3, 40, 16, 4, 2
    t = dict(x=torch.zeros(T, K, dtype=torch.bfloat16), index=torch.zeros(T, k, dtype=torch.int32), weight=torch.zeros(T, k),
             gate_up=torch.zeros(E, 2 * H, K, dtype=torch.bfloat16), down=torch.zeros(E, K, H, dtype=torch.bfloat16),
             y=torch.zeros(T, K, dtype=torch.bfloat16))
    t.update(change)
    return t


def test_binding_reads_shapes_strides_and_types():
    big = torch.zeros(4, 33, 50, dtype=torch.bfloat16)
    d = gt.make_moe_desc(**tensors(gate_up=big[:, :32, :40], down=torch.zeros(40, 4, 16, dtype=torch.bfloat16).permute(1, 0, 2)))
    assert (d.M, d.K, d.H, d.E, d.topk, d.gate_up_ld, d.gate_up_stride, d.down_ld, d.down_stride) == (3, 40, 16, 4, 2, 50, 1650, 64, 16)
    q = tensors(gate_up=torch.zeros(4, 32, 20, dtype=torch.uint8), down=torch.zeros(4, 40, 8, dtype=torch.uint8))
    d = gt.make_moe_desc(**q, gate_up_scales=torch.zeros(4, 2, 32).permute(0, 2, 1), down_scales=torch.zeros(4, 40, 1), format="int4", group=32)
    assert (d.gate_up_ld, d.gate_up_stride, d.gate_up_scale_lde, d.gate_up_scale_ldn, d.gate_up_scale_ldg) == (20, 640, 64, 1, 32)
    assert (d.format, d.scale_dtype, d.group, d.down_scale_lde, d.down_scale_ldn) == (0, gt.F32, 32, 40, 1)
    a, b = torch.zeros(5, 8, 40, dtype=torch.float16), torch.zeros(5, 24, 8, dtype=torch.float16)
    y = torch.zeros(3, 30)[:, :24]
    ws = torch.zeros(1024)
    d = gt.make_lora_desc(torch.zeros(3, 40, dtype=torch.float16), torch.zeros(3, dtype=torch.int32), a, b, y, base=y, workspace=ws)
    assert (d.M, d.K, d.N, d.adapters, d.rank, d.ldy, d.ldb, d.a_ld, d.a_stride, d.b_ld, d.b_stride) == (3, 40, 24, 5, 8, 30, 30, 40, 320, 8, 192)
    assert d.workspace_bytes == 4096 and d.out_dtype == gt.F32 and d.base == d.y
    d = gt.make_route_desc(torch.zeros(3, 20)[:, :16], torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2), score="sigmoid")
    assert (d.M, d.E, d.topk, d.ldl, d.score, d.normalise) == (3, 16, 2, 20, 1, 1)


BAD = dict(
    index_type=dict(index=torch.zeros(3, 2, dtype=torch.int64)), index_shape=dict(index=torch.zeros(2, 2, dtype=torch.int32)),
    weight_type=dict(weight=torch.zeros(3, 2, dtype=torch.float16)), weight_shape=dict(weight=torch.zeros(3, 3)),
    odd=dict(gate_up=torch.zeros(4, 31, 40, dtype=torch.bfloat16)), experts=dict(down=torch.zeros(3, 40, 16, dtype=torch.bfloat16)),
    types=dict(gate_up=torch.zeros(4, 32, 40, dtype=torch.float16)), columns=dict(gate_up=torch.zeros(4, 40, 32, dtype=torch.bfloat16).transpose(1, 2)),
    shared=dict(gate_up=torch.zeros(1, 32, 40, dtype=torch.bfloat16).expand(4, 32, 40)),
    one_row=dict(down=torch.zeros(4, 1, 16, dtype=torch.bfloat16).expand(4, 40, 16)),
    base=dict(base=torch.zeros(3, 40)), base_row=dict(base=torch.zeros(1, 40, dtype=torch.bfloat16).expand(3, 40)),
    y=dict(y=torch.zeros(3, 41, dtype=torch.bfloat16)), scales=dict(gate_up_scales=torch.zeros(4, 32, 2)),
    no_scales=dict(format="int4", gate_up=torch.zeros(4, 32, 20, dtype=torch.uint8), down=torch.zeros(4, 40, 8, dtype=torch.uint8)),
    bytes=dict(format="e2m1"), workspace=dict(workspace=torch.zeros(8, 8).t()),
)


@pytest.mark.parametrize("what", sorted(BAD))
def test_binding_refuses(what):
    gt.make_moe_desc(**tensors())
    with pytest.raises(ValueError):
        gt.make_moe_desc(**tensors(**BAD[what]))


def test_binding_refuses_more():
    x, i = torch.zeros(3, 40, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
    a, b, y = torch.zeros(5, 8, 40, dtype=torch.float16), torch.zeros(5, 24, 8, dtype=torch.float16), torch.zeros(3, 24)
    gt.make_lora_desc(x, i, a, b, y)
    for bad in (dict(a=a.float()), dict(b=b[:4]), dict(index=i.long()), dict(index=i[:2]), dict(y=y[:, :23]), dict(scale=torch.zeros(4)),
                dict(a=a[:1].expand(5, 8, 40)), dict(b=b[:, :, :7]), dict(base=y.half()), dict(index=torch.zeros(1, dtype=torch.int32).expand(3))):
        with pytest.raises(ValueError):
            gt.make_lora_desc(**{**dict(x=x, index=i, a=a, b=b, y=y), **bad})
    l, w = torch.zeros(3, 16), torch.zeros(3, 2)
    i = torch.zeros(3, 2, dtype=torch.int32)
    for bad in (dict(index=i.long()), dict(weight=w.half()), dict(weight=w[:2]), dict(logits=l[:1].expand(3, 16)),
                dict(index=torch.zeros(1, 2, dtype=torch.int32).expand(3, 2))):
        with pytest.raises(ValueError):
            gt.make_route_desc(**{**dict(logits=l, index=i, weight=w), **bad})


def test_whether_matrices_meet():
    # against every byte, for views of one buffer
    g = ref.rng(1)
    seen = {True: 0, False: 0}
    buf = torch.zeros(400)
    for _ in range(4000):
        views, places = [], []
        for t in (buf, buf):
            n, c, at = (int(torch.randint(1, hi, (1,), generator=g)) for hi in (7, 9, 120))
            s = c + int(torch.randint(0, 30, (1,), generator=g))
            views.append(t.as_strided((n, c), (s, 1), at))
            places.append({at + i * s + j for i in range(n) for j in range(c)})
        want = bool(places[0] & places[1])
        assert gt._meet(*views) == want and gt._meet(*views[::-1]) == want
        if int(torch.randint(0, 2, (1,), generator=g)):  # rows of one length apart
            a, b = views[0], buf.as_strided(tuple(views[1].shape), (views[0].stride(0), 1), views[1].storage_offset())
            if b.stride(0) >= b.shape[1]:
                want = bool(places[0] & {b.storage_offset() + i * b.stride(0) + j for i in range(b.shape[0]) for j in range(b.shape[1])})
                assert gt._meet(a, b) == want
        seen[want] += 1
    assert min(seen.values()) > 500


def test_binding_refuses_operands_that_overlap_the_result():
    x, w = torch.zeros(3, 40, dtype=torch.bfloat16), tensors()
    big = torch.zeros(8, 100, dtype=torch.bfloat16)
    flat = torch.zeros(1000, dtype=torch.bfloat16)
    for y in (x, big[:3, 40:80]):
        gt.make_moe_desc(**{**w, "x": x, "y": y})
    gt.make_moe_desc(**{**w, "x": big[:3, :40], "y": big[:3, 40:80], "base": big[:3, 40:80]})
    gt.make_moe_desc(**{**w, "x": big[:3, :40], "y": big[3:6, :40], "base": big[:3, :40]})
    gt.make_moe_desc(**{**w, "x": big[:3, :40], "y": big[:3, :40], "base": big[:3, :40]})
    over = [dict(x=big[:3, :40], y=big[1:4, :40]), dict(x=big[:3, :40], y=big[:3, 39:79]),
            dict(x=flat[:120].view(3, 40), y=flat.as_strided((3, 40), (50, 1), 0)),
            dict(x=flat[:120].view(3, 40), y=flat.view(torch.float32)[:120].view(3, 40)),
            dict(y=big[:3, :40], base=big[1:4, :40]), dict(y=big[:3, :40], base=big[:3, 1:41])]
    for bad in over:
        with pytest.raises(ValueError, match="overlaps y"):
            gt.make_moe_desc(**{**w, **bad})
    a, b, i = torch.zeros(2, 8, 40, dtype=torch.bfloat16), torch.zeros(2, 40, 8, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    gt.make_lora_desc(big[:3, :40], i, a, b, big[:3, 40:80], base=big[:3, 40:80])
    for bad in over + [dict(x=x, y=x)]:
        with pytest.raises(ValueError, match="overlaps y"):
            gt.make_lora_desc(bad.get("x", x), i, a, b, bad["y"], base=bad.get("base"))


def test_host_tensors_are_refused(stand_in):
    for call, d in ((gt.gt_moe, gt.make_moe_desc(**tensors())), (gt.gt_route, gt.make_route_desc(torch.zeros(3, 16), torch.zeros(
            3, 2, dtype=torch.int32), torch.zeros(3, 2)))):
        with pytest.raises(ValueError, match="GPU"):
            call(d)


# ---- the references
def test_reference_route():
    l = torch.randn(6, 20, generator=ref.rng(1))
    i, w = br.route(l, 4, "softmax", False)
    p = torch.softmax(l.double(), 1).sort(1, descending=True)
    assert torch.equal(i.long(), p.indices[:, :4]) and torch.allclose(w, p.values[:, :4])
    i, w = br.route(l, 4, "sigmoid", True, 3.0)
    s = torch.sigmoid(l.double()).gather(1, i.long())
    assert torch.allclose(w, 3.0 * s / s.sum(1, keepdim=True))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_reference_layer(act):
    x, w = ref.loud(3, 20, 1), dict(gate_up=br.normal((4, 12, 20), 0.2, torch.float32, 2), down=br.normal((4, 20, 6), 0.4, torch.float32, 3))
    index, weight = br.choices(3, 4, 2, 4)
    y, far = br.moe(x, index, weight, w["gate_up"], w["down"], act=act)
    f = torch.nn.functional.silu if act == "silu" else lambda v: torch.nn.functional.gelu(v, approximate="tanh")
    for t in range(3):
        want = 0
        for j in range(2):
            e = index[t, j]
            gu = w["gate_up"][e].double() @ x[t].double()
            want = want + weight[t, j].double() * (w["down"][e].double() @ (f(gu[:6]) * gu[6:]))
        assert torch.allclose(y[t], want, rtol=1e-12) and (far[t] > 0).all()


def test_reference_adapters():
    x, a, b = ref.loud(5, 20, 1), br.normal((3, 4, 20), 0.2, torch.float32, 2), br.normal((3, 7, 4), 0.5, torch.float32, 3)
    base, scale = br.normal((5, 7), 1.0, torch.float32, 4), torch.tensor([2.0, -1.0, 0.5])
    index = torch.tensor([0, 2, -1, 1, 3], dtype=torch.int32)
    y, _ = br.lora(x, index, a, b, scale, base)
    for m in range(5):
        want = base[m].double()
        if 0 <= index[m] < 3:
            e = index[m]
            want = want + scale[e].double() * (x[m].double() @ a[e].double().t() @ b[e].double().t())
        assert torch.allclose(y[m], want, rtol=1e-12)
