"""The experts' choice, layer and adapters in a program: other streams, several
threads, graphs that are captured once and replayed, workspaces shared and
not, operands far apart in memory, the same bits every time.
"""
import ctypes
import threading

import pytest
import torch

import gemm_autotuning_amd as gt

from . import beside_ref as br
from . import op_ref as ref

pytestmark = pytest.mark.gpu
HIP = ctypes.CDLL("libamdhip64.so")
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


class Layer:
    """The choice and the layer of one set of experts, with the reference's results."""

    def __init__(self, T, E, k, K, H, dtype, fmt, seed):
        self.fmt, self.k = fmt, k
        if fmt == "none":
            self.w = dict(gate_up=br.normal((E, 2 * H, K), K ** -0.5, dtype, seed), down=br.normal((E, K, H), H ** -0.5, dtype, seed + 1))
        else:
            (gu, gs), (dn, ds) = br.nibbles(E, 2 * H, K, 64, "bf16", seed), br.nibbles(E, K, H, 64, "bf16", seed + 1)
            self.w = dict(gate_up=gu, gs=gs, down=dn, ds=ds)
        self.x = ref.loud(T, K, seed + 2).to(dtype)
        self.logits = torch.randn(T, E, generator=ref.rng(seed + 3))
        self.dev = {n: t.cuda() for n, t in self.w.items()}
        self.X, self.L = self.x.cuda(), self.logits.cuda()
        self.index = torch.empty(T, k, dtype=torch.int32, device="cuda")
        self.weight = torch.empty(T, k, device="cuda")
        self.y = torch.zeros(T, K, dtype=dtype, device="cuda")

    def descs(self, stream, workspace=None):
        c = self.dev
        return (gt.make_route_desc(self.L, self.index, self.weight, stream=stream),
                gt.make_moe_desc(self.X, self.index, self.weight, c["gate_up"], c["down"], self.y, gate_up_scales=c.get("gs"),
                                 down_scales=c.get("ds"), format=self.fmt, group=64, workspace=workspace, stream=stream))

    def run(self, d):
        gt.gt_route(d[0])
        gt.gt_moe(d[1])

    def check(self):
        i, w = br.route(self.L.cpu(), self.k)
        assert torch.equal(self.index.cpu(), i)
        want, far = br.moe(self.X.cpu(), i, self.weight.cpu(), self.w["gate_up"], self.w["down"], self.w.get("gs"), self.w.get("ds"),
                           self.fmt, 64)
        ref.check(self.y.cpu(), want, far, "y")

    def change(self, turn):
        self.L.copy_(torch.roll(self.logits, turn, 1).cuda())
        self.X.copy_(torch.roll(self.x, turn, 0).cuda())
        self.y.zero_()
        self.index.fill_(-1)


LAYERS = [(1, 9, 3, 200, 96, BF, "none"), (13, 5, 2, 256, 130, F16, "int4"), (70, 2, 2, 130, 72, BF, "none"), (150, 4, 2, 64, 64, F16, "e2m1")]


@pytest.mark.parametrize("case", LAYERS)
def test_another_stream_and_a_graph(case):
    layer = Layer(*case, seed=3)
    st = torch.cuda.Stream()
    d = layer.descs(st.cuda_stream)
    torch.cuda.synchronize()
    layer.run(d)
    st.synchronize()
    layer.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        layer.run(d)
    for turn in range(1, 4):
        layer.change(turn)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            graph.replay()
        st.synchronize()
        layer.check()
        if turn == 2:  # the program's own call between the replays, on the same stream and workspace
            layer.y.zero_()
            torch.cuda.synchronize()
            layer.run(d)
            st.synchronize()
            layer.check()


def test_two_graphs_at_once_on_workspaces_of_their_own():
    layers = [Layer(*LAYERS[1], seed=5), Layer(*LAYERS[2], seed=6)]
    streams, graphs, keep = [torch.cuda.Stream() for _ in layers], [], []
    for layer, st in zip(layers, streams):
        ws = torch.empty(gt.gt_moe_workspace(layer.descs(0)[1]), dtype=torch.uint8, device="cuda")
        d = layer.descs(streams[0].cuda_stream, ws)  # both captured on one stream, which never gets a workspace
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=streams[0]):
            layer.run(d)
        graphs.append(g)
        keep.append((ws, d))
    for turn in range(1, 4):
        for layer in layers:
            layer.change(turn)
        torch.cuda.synchronize()
        for _ in range(5):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for layer in layers:
            layer.check()


def test_a_first_call_under_capture_is_refused():
    layer = Layer(2, 4, 2, 64, 64, BF, "none", seed=8)
    a, b = torch.ones(1, 32, 64, device="cuda").bfloat16(), torch.ones(1, 128, 32, device="cuda").bfloat16()
    x, y = torch.ones(5, 64, device="cuda").bfloat16(), torch.zeros(5, 128, device="cuda")
    handle = ctypes.c_void_p()  # a stream that no other test can have had
    assert HIP.hipStreamCreate(ctypes.byref(handle)) == 0
    st = torch.cuda.ExternalStream(handle.value)
    d = layer.descs(handle.value)
    lora = gt.make_lora_desc(x, torch.zeros(5, dtype=torch.int32, device="cuda"), a, b, y, stream=handle.value)
    marker = torch.zeros(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        marker.add_(1)
        for call, desc in ((gt.gt_lora, lora), (gt.gt_moe, d[1])):
            with pytest.raises(gt.GemmTuneError, match="captur"):
                call(desc)
    graph.replay()
    torch.cuda.synchronize()
    assert marker.item() == 1.0 and (y == 0).all()
    layer.run(d)  # outside the capture the workspace is made
    gt.gt_lora(lora)
    st.synchronize()
    layer.check()
    assert (y == 64.0 * 32).all()


@pytest.mark.parametrize("shared", [False, True])
def test_threads(shared):
    # eight threads, on streams of their own or all on one (whose calls take its workspace in turn)
    layers = [Layer(*LAYERS[i % 4], seed=20 + i) for i in range(8)]
    one = torch.cuda.Stream()
    streams = [one if shared else torch.cuda.Stream() for _ in layers]
    descs = [layer.descs(st.cuda_stream) for layer, st in zip(layers, streams)]
    torch.cuda.synchronize()
    start, errors = threading.Barrier(8), []

    def work(i):
        try:
            start.wait()
            for _ in range(10):
                layers[i].run(descs[i])
        except Exception as e:
            errors.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for layer in layers:
        layer.check()


def test_the_same_bits_every_time():
    for case in LAYERS:
        layer = Layer(*case, seed=9)
        d = layer.descs(torch.cuda.current_stream().cuda_stream)
        seen = []
        for _ in range(4):
            layer.y.zero_()
            layer.run(d)
            torch.cuda.synchronize()
            seen.append(layer.y.clone())
        assert all(torch.equal(seen[0], s) for s in seen[1:])


@pytest.mark.parametrize("T,k", [(1, 1), (3, 2), (20, 1), (60, 1)])
def test_experts_past_32_bits_of_bytes(T, k):
    # two experts of 2.7 GB each, 5.4 GB in all: the second one's down matrix and its last rows of gate and up
    # start past 2^32 bytes
    E, K, H = 2, 65536, 6800
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(1)
    gate_up = torch.zeros(E, 2 * H, K, dtype=BF, device=dev)
    down = torch.zeros(E, K, H, dtype=BF, device=dev)
    some = [0, 1, H // 2, H - 2, H - 1]
    rows = [0, 1, K // 2, K - 2, K - 1]
    for e in range(E):
        for n in some + [H + s for s in some]:
            gate_up[e, n] = torch.randn(K, generator=g, device=dev).mul_(K ** -0.5).bfloat16()
        for n in rows:
            down[e, n] = torch.randn(H, generator=g, device=dev).bfloat16()
    x = torch.randn(T, K, generator=g, device=dev).bfloat16()
    index = torch.tensor([[(t + j) % 2 for j in range(k)] for t in range(T)], dtype=torch.int32)
    weight = torch.rand(T, k, generator=ref.rng(2))
    y = torch.full((T, K), 7.0, device=dev)
    gt.gt_moe(gt.make_moe_desc(x, index.to(dev), weight.to(dev), gate_up, down, y, stream=torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    keep = torch.cat([torch.tensor(some), H + torch.tensor(some)])
    small = gate_up[:, keep.to(dev)].cpu()  # the other rows of gate and up give nothing
    sd = down[:, rows][:, :, some].cpu()
    # the formula over what is not zero; its activations are the same values
    want = torch.zeros(T, len(rows), dtype=torch.float64)
    far = torch.zeros_like(want)
    xs = x.cpu().double()
    for t in range(T):
        for j in range(k):
            e, w = int(index[t, j]), float(weight[t, j])
            gu, mag = small[e].double() @ xs[t], small[e].double().abs() @ xs[t].abs()
            gg, u = gu[:5], gu[5:]
            a = br.activation(gg, "silu")
            h = a * u
            dg, du = br.dot(K) * mag[:5], br.dot(K) * mag[5:]
            dh = (1.13 * dg + 8 * br.U * gg.abs()) * (u.abs() + du) + a.abs() * du + 4 * br.U * h.abs()
            D = sd[e].double()
            want[t] += w * (D @ h)
            far[t] += abs(w) * (D.abs() @ (dh + br.split(h, BF)) + (br.dot(H) + 8 * br.U) * (D.abs() @ h.abs())) + 4 * br.U * want[t].abs()
    ref.check(y[:, rows].cpu(), want, far, "y")
    others = torch.ones(K, dtype=torch.bool)
    others[rows] = False
    assert (y.cpu()[:, others] == 0).all()


@pytest.mark.parametrize("M", [1, 5, 70])
def test_adapters_past_31_bits_of_elements(M):
    # matrices half of 2^32 bytes apart, over memory that is there: the third one starts at 2^32
    L, r, K, N = 3, 16, 300, 200
    far = 1 << 30  # elements
    g = ref.rng(4)
    a, b = br.normal((L, r, K), K ** -0.5, BF, 1), br.normal((L, N, r), r ** -0.5, BF, 2)
    bufs = [torch.zeros((L - 1) * far + t[0].numel(), dtype=BF, device="cuda") for t in (a, b)]
    A = bufs[0].as_strided((L, r, K), (far, K, 1))
    B = bufs[1].as_strided((L, N, r), (far, r, 1))
    A.copy_(a.cuda())
    B.copy_(b.cuda())
    x = ref.loud(M, K, 5).to(BF)
    index = torch.randint(0, L, (M,), generator=g, dtype=torch.int32)
    index[0] = L - 1
    y = torch.empty(M, N, device="cuda")
    gt.gt_lora(gt.make_lora_desc(x.cuda(), index.cuda(), A, B, y, stream=torch.cuda.current_stream().cuda_stream))
    want, bound = br.lora(x, index, a, b)
    ref.check(y.cpu(), want, bound, "y")


def test_rows_of_the_index_far_apart():
    # the choices, their weights, x, base and y as columns of wide buffers
    T, E, k, K, H = 6, 4, 3, 72, 40
    x = ref.loud(T, K, 1).to(F16)
    w = dict(gate_up=br.normal((E, 2 * H, K), K ** -0.5, F16, 2), down=br.normal((E, K, H), H ** -0.5, F16, 3))
    index, weight = br.choices(T, E, k, 4)
    base = br.normal((T, K), 1.0, F16, 5)

    def wide(t, fill, by):
        buf = torch.full((T, by), fill, dtype=t.dtype, device="cuda")
        buf[:, :t.shape[1]].copy_(t)
        return buf[:, :t.shape[1]]

    y = wide(torch.zeros(T, K, dtype=F16), float("nan"), 1 << 20)
    gt.gt_moe(gt.make_moe_desc(wide(x, float("nan"), 1 << 21), wide(index, 1, 1001), wide(weight, float("nan"), 77), w["gate_up"].cuda(),
                               w["down"].cuda(), y, base=wide(base, float("nan"), 12345), stream=torch.cuda.current_stream().cuda_stream))
    want, far = br.moe(x, index, weight, w["gate_up"], w["down"], base=base)
    ref.check(y.cpu(), want, far, "y")


def test_the_layer_on_the_default_stream_after_gt_set_stream():
    layer = Layer(*LAYERS[0], seed=12)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    gt.gt_set_stream(st.cuda_stream)
    try:
        layer.run(layer.descs(0))
        st.synchronize()
        layer.check()
    finally:
        gt.gt_set_stream(0)
