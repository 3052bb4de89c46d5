"""Experts and adapters beside the product at the edges of what their calls
take: default strides of scales, infinities between the
products and in scales, values between the products that take all of fp32's
bits, exponentials far from 0,
more rows than a launch,
results over the rows themselves, NaN among the logits, one token's experts
named many times.
"""
import math

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


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("T", [3, 10, 40])
def test_an_infinite_activation_beside_large_ones(dtype, T):
    # one row of gate is infinite, the others give values that f16 does not hold: the result is the
    # infinity, of the sign that down gives it
    K, H, n = 64, 40, 5
    x = torch.full((T, K), 16.0).to(dtype)
    gate_up = torch.full((1, 2 * H, K), 16.0).to(dtype)
    gate_up[0, n] = math.inf
    down = torch.ones(1, K, H).to(dtype)
    down[0, :, n] = -1.0
    down[0, 1::2] *= -1.0
    y = torch.empty(T, K, device="cuda")
    gt.gt_moe(gt.make_moe_desc(x.cuda(), torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.ones(T, 1, device="cuda"), gate_up.cuda(),
                               down.cuda(), y, stream=stream()))
    torch.cuda.synchronize()
    assert (y[:, 0::2] == -math.inf).all() and (y[:, 1::2] == math.inf).all()


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("M", [2, 40, 2100])
@pytest.mark.parametrize("r", [12, 40])
def test_an_infinite_value_of_an_adapter_beside_large_ones(dtype, r, M):
    K, N = 64, 70
    x = torch.full((M, K), 64.0).to(dtype)
    a = torch.full((1, r, K), 64.0).to(dtype)
    a[0, 3] = math.inf
    b = torch.ones(1, N, r).to(dtype)
    b[0, :, 3] = -1.0
    b[0, 1::2] *= -1.0
    y = torch.empty(M, N, device="cuda")
    gt.gt_lora(gt.make_lora_desc(x.cuda(), torch.zeros(M, dtype=torch.int32, device="cuda"), a.cuda(), b.cuda(), y, stream=stream()))
    torch.cuda.synchronize()
    assert (y[:, 0::2] == -math.inf).all() and (y[:, 1::2] == math.inf).all()


@pytest.mark.parametrize("fmt,scales", [("int4", "f32"), ("e2m1", "bf16")])
@pytest.mark.parametrize("T", [1, 3, 12])
@pytest.mark.parametrize("where", ["gate", "down"])
def test_an_infinite_scale_of_the_last_group(where, T, fmt, scales):
    # positive codes under it: the results are infinite, and no NaN comes from what lies past the row's end
    E, K, H, group = 1, 100, 72, 32
    gu, gs = br.nibbles(E, 2 * H, K, group, scales, 1, codes=[1, 2, 3])
    dn, ds = br.nibbles(E, K, H, group, scales, 2, codes=[1, 2, 3])
    if where == "gate":
        gs[:, :H, -1] = math.inf
    else:
        ds[:, :, -1] = math.inf
    x = (ref.loud(T, K, 3).abs() + 0.5).to(BF)
    y = torch.empty(T, K, device="cuda")
    gt.gt_moe(gt.make_moe_desc(x.cuda(), torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.ones(T, 1, device="cuda"), gu.cuda(),
                               dn.cuda(), y, gate_up_scales=gs.cuda(), down_scales=ds.cuda(), format=fmt, group=group, stream=stream()))
    torch.cuda.synchronize()
    assert (y == math.inf).all()


@pytest.mark.parametrize("fmt", ["none", "int4", "e2m1"])
@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("T,E,k,H", [(1, 2, 2, 40), (12, 3, 2, 40), (12, 2, 2, 1100), (9, 1, 1, 2300), (50, 2, 2, 130), (20, 1, 1, 2300)])
def test_activations_of_23_bits(fmt, dtype, T, E, k, H):
    # gates above 32 are their own activation, so that the values between the products are whole numbers
    # below 2^23, and a row of down names one of them: every result is exact
    K, g = 256, ref.rng(T + H)
    x = torch.randint(1, 4, (T, K), generator=g).to(dtype)
    index, _ = br.choices(T, E, k, 3)
    at, sign = torch.randint(0, H, (E, K), generator=g), torch.randint(0, 2, (E, K), generator=g) * 2 - 1
    down = torch.zeros(E, K, H, dtype=torch.int8).scatter_(2, at.unsqueeze(2), sign.unsqueeze(2).to(torch.int8))
    if fmt == "none":
        w = dict(gate_up=torch.randint(1, 9, (E, 2 * H, K), generator=g).to(dtype), down=down.to(dtype), gs=None, ds=None)
    else:
        few = [1, 2, 3, 4, 5, 6, 7] if fmt == "int4" else [2, 4, 5, 6, 7]  # whole numbers of 1 to 7, or 6
        one = torch.where(down == 0, 0, torch.where(down > 0, 1, 15) if fmt == "int4" else torch.where(down > 0, 2, 10)).to(torch.uint8)
        w = dict(gate_up=br.nibbles(E, 2 * H, K, 64, "f32", 1, few)[0], down=one[:, :, 0::2] | one[:, :, 1::2] << 4,
                 gs=torch.ones(E, 2 * H, K // 64), ds=torch.ones(E, K, -(-H // 64)))
    want, _ = br.moe(x, index, torch.ones(T, k), w["gate_up"], w["down"], w["gs"], w["ds"], fmt, 64)
    assert 2 ** 20 < want.abs().max() < 2 ** 24
    y = torch.empty(T, K, device="cuda")
    c = {n: t.cuda() for n, t in w.items() if t is not None}
    gt.gt_moe(gt.make_moe_desc(x.cuda(), index.cuda(), torch.ones(T, k, device="cuda"), c["gate_up"], c["down"], y,
                               gate_up_scales=c.get("gs"), down_scales=c.get("ds"), format=fmt, group=64, stream=stream()))
    torch.cuda.synchronize()
    assert torch.equal(y.cpu().double(), want)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("M,r,K", [(5, 12, 4096), (40, 40, 4096), (2100, 40, 4096), (600, 7, 4100), (300, 130, 4096), (90, 256, 3900)])
def test_an_adapters_values_of_23_bits(dtype, M, r, K):
    # whole numbers below 2^23 between the products, of which a row of b names one: every result is exact
    L, N, g = 2, 90, ref.rng(M + r)
    x, a = torch.randint(1, 65, (M, K), generator=g).to(dtype), torch.randint(1, 65, (L, r, K), generator=g).to(dtype)
    at, sign = torch.randint(0, r, (L, N), generator=g), torch.randint(0, 2, (L, N), generator=g) * 2 - 1
    b = torch.zeros(L, N, r).scatter_(2, at.unsqueeze(2), sign.unsqueeze(2).float()).to(dtype)
    index = torch.randint(-1, L, (M,), generator=g, dtype=torch.int32)
    want = torch.zeros(M, N, dtype=torch.float64)
    for e in range(L):
        m = index == e
        want[m] = (x[m].double() @ a[e].double().t()) @ b[e].double().t()
    assert 2 ** 21 < want.abs().max() < 2 ** 23
    y = torch.empty(M, N, device="cuda")
    gt.gt_lora(gt.make_lora_desc(x.cuda(), index.cuda(), a.cuda(), b.cuda(), y, stream=stream()))
    torch.cuda.synchronize()
    assert torch.equal(y.cpu().double(), want)


@pytest.mark.parametrize("T", [1, 12, 40])
def test_activations_of_gates_far_below_zero(T):
    # an activation to each result.  Relatively: the exponential is off by 2 u (an ulp), the sum and the
    # quotient by u each; bf16's parts are all of it
    K = H = 256
    x = torch.zeros(T, K)
    x[:, 0] = 1.0
    gates = torch.linspace(-70.0, 70.0, H).to(BF)
    gate_up = torch.zeros(1, 2 * H, K)
    gate_up[0, :H, 0], gate_up[0, H:, 0] = gates.float(), 1.0
    y = torch.empty(T, K, device="cuda")
    gt.gt_moe(gt.make_moe_desc(x.to(BF).cuda(), torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.ones(T, 1, device="cuda"),
                               gate_up.to(BF).cuda(), torch.eye(K, dtype=BF).unsqueeze(0).cuda(), y, stream=stream()))
    torch.cuda.synchronize()
    want = br.activation(gates.double(), "silu")
    far = (y.cpu().double() - want).abs() / want.abs()
    assert far.max() <= 5 * br.U, far.max() / br.U


@pytest.mark.parametrize("E,k,M", [(17, 17, (1 << 25) + 4097), (4, 2, (1 << 26) + 5)])
def test_choices_of_more_rows_than_one_launch_takes(E, k, M):
    # the rows repeat every 4099, and so do their choices
    part = torch.randn(4099, E, generator=ref.rng(E)).half()
    logits = part.cuda().repeat(-(-M // 4099), 1)[:M]
    index, weight = torch.full((M, k), -7, dtype=torch.int32, device="cuda"), torch.full((M, k), -7.0, device="cuda")
    gt.gt_route(gt.make_route_desc(logits, index, weight, stream=stream()))
    torch.cuda.synchronize()
    want, w = br.route(part, k)
    # an exponential of an argument of magnitude a is off by (a + 2) u, the sum of positive ones and the
    # quotient by 40 u more
    assert ((weight[:4099].cpu().double() - w).abs() <= w * (4 * part.abs().max().item() + 40) * br.U).all()
    for t, first in ((index, want.cuda()), (weight, weight[:4099])):
        whole = M // 4099 * 4099
        assert (t[:whole].view(-1, 4099, k) == first).all() and (t[whole:] == first[:M - whole]).all()


@pytest.mark.parametrize("T,E,k", [(1, 3, 2), (7, 200, 3), (30, 4, 3), (1500, 4, 3)])
def test_results_over_the_rows_themselves(T, E, k):
    # x is y, and is the base too; many tokens run in several ranges
    K, H = 72, 40
    x, (index, weight) = ref.loud(T, K, 1).to(BF).cuda(), br.choices(T, E, k, 2)
    gate_up, down = br.normal((E, 2 * H, K), K ** -0.5, BF, 3).cuda(), br.normal((E, K, H), H ** -0.5, BF, 4).cuda()
    for base in (False, True):
        here, there = x.clone(), torch.empty_like(x)
        for xs, y in ((x, there), (here, here)):
            gt.gt_moe(gt.make_moe_desc(xs, index.cuda(), weight.cuda(), gate_up, down, y, base=xs if base else None, stream=stream()))
        torch.cuda.synchronize()
        assert torch.equal(here, there)


@pytest.mark.parametrize("dtype", [F32, F16, BF])
@pytest.mark.parametrize("E", [50, 400])
def test_a_nan_is_in_all_weights_that_are_divided(dtype, E):
    # with a softmax or normalise a NaN makes all weights of its row NaN, and +infinity does with a softmax;
    # a sigmoid by itself leaves the others
    k = 8
    logits = torch.randn(6, E, generator=ref.rng(1)).to(dtype)
    logits[0, 7] = math.nan
    logits[1, 7], logits[1, 30] = -math.nan, math.nan
    logits[2, 9] = math.inf
    logits[3] = math.nan
    logits[4, 20:] = -math.inf
    logits[4, 3] = math.nan
    for score in ("softmax", "sigmoid"):
        for normalise in (True, False):
            index, weight = torch.empty(6, k, dtype=torch.int32, device="cuda"), torch.empty(6, k, device="cuda")
            gt.gt_route(gt.make_route_desc(logits.cuda(), index, weight, score=score, normalise=normalise, stream=stream()))
            torch.cuda.synchronize()
            i, w = index.cpu(), weight.cpu()
            want_i, want_w = br.route(logits, k, score, normalise)
            assert torch.equal(i, want_i)
            nan = torch.isnan(w)
            if score == "softmax":
                assert nan[:5].all() and not nan[5].any()
            elif normalise:
                assert nan[[0, 1, 3, 4]].all() and not nan[[2, 5]].any()
            else:
                assert torch.equal(nan, torch.isnan(logits.gather(1, i.long())))
            # arguments up to 12: exponentials off by 2 u, a sum of up to 1024 and the quotients by 60 u together
            ok = ~nan
            assert ((w.double() - want_w)[ok].abs() <= 100 * br.U * want_w[ok]).all()


@pytest.mark.parametrize("fmt", ["none", "int4"])
@pytest.mark.parametrize("dtype", [BF, F16])
def test_one_token_that_names_its_experts_many_times(dtype, fmt):
    E, k, K, H = 2, 11, 100, 72
    g = ref.rng(1)
    if fmt == "none":
        c = dict(gate_up=br.normal((E, 2 * H, K), K ** -0.5, dtype, 2), down=br.normal((E, K, H), H ** -0.5, dtype, 3), gs=None, ds=None)
    else:
        (gu, gs), (dn, ds) = br.nibbles(E, 2 * H, K, 32, "f16", 2), br.nibbles(E, K, H, 32, "f16", 3)
        c = dict(gate_up=gu, down=dn, gs=gs, ds=ds)
    x, index, weight = ref.loud(1, K, 4).to(dtype), torch.randint(-1, E, (1, k), generator=g, dtype=torch.int32), torch.rand(1, k, generator=g)
    y = torch.empty(1, K, device="cuda")
    d = {n: t if t is None else t.cuda() for n, t in c.items()}
    gt.gt_moe(gt.make_moe_desc(x.cuda(), index.cuda(), weight.cuda(), d["gate_up"], d["down"], y, gate_up_scales=d["gs"],
                               down_scales=d["ds"], format=fmt, group=32, stream=stream()))
    torch.cuda.synchronize()
    want, far = br.moe(x, index, weight, c["gate_up"], c["down"], c["gs"], c["ds"], fmt, 32)
    ref.check(y.cpu(), want, far, "y")
