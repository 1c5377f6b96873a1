"""The new operators as they are used: routed experts on 8-bit rows with a shared
expert beside them, forward and data gradient; on several streams at once, and
captured into a graph that is replayed."""
import pytest
import torch

import block_ref as bref
import expert_ref as ref
from gpu_util import announce
from test_gpu_expert_linear import DEV, routing

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


class Layer:
    """One mixture-of-experts layer: E routed experts in 8 bits, a shared one in bf16."""

    def __init__(self, gpu, E, H, inter, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        self.E, self.inter = E, inter
        self.w1, self.w1_t = gpu.ep_cast_fp8_blocks((n(E, 2 * inter, H) * H ** -0.5).to(BF16), transposed=True)
        self.w2, self.w2_t = gpu.ep_cast_fp8_blocks((n(E, H, inter) * inter ** -0.5).to(BF16), transposed=True)
        self.s1, self.s2 = (n(2 * inter, H) * H ** -0.5).to(BF16), (n(H, inter) * inter ** -0.5).to(BF16)

    def forward(self, gpu, x, idx, wts):
        lay = gpu.ep_get_layout(idx, self.E, 16)
        rx, rs, _ = gpu.ep_dispatch(x, lay, wts, recv_fp8=True)
        h = gpu.ep_block_linear((rx, rs), self.w1, lay, activation="swiglu")
        y = gpu.ep_block_linear(gpu.ep_cast_fp8(h, 128), self.w2, lay)
        shared, _ = gpu.ep_gated_ffn(x, self.s1, self.s2, residual=x)
        return lay, (rx, rs), h, y, gpu.ep_combine(y, lay, wts, bias=shared)[0]


@pytest.mark.parametrize("T,E,K", [(1, 4, 2), (50, 8, 2), (700, 4, 2)])
def test_forward_and_data_gradient(gpu, T, E, K):
    announce("block chain", T, E, K)
    H, inter = 512, 256
    layer = Layer(gpu, E, H, inter, T)
    g = torch.Generator(device=DEV).manual_seed(T + 1)
    x = torch.randn((T, H), generator=g, device=DEV).to(BF16)
    idx = routing(T, E, K, T)
    wts = torch.rand((T, K), generator=g, device=DEV)
    lay, recv, h, y, out = layer.forward(gpu, x, idx, wts)
    assert lay.check() == 0
    sp = ref.spans(lay, lay.max_recv_rows)
    for rows, want, err in bref.block_linear(recv, layer.w1, None, "swiglu", None, sp):
        ref.assert_near(h[rows], want, err, what="h")
    for rows, want, err in bref.block_linear(gpu.ep_cast_fp8(h, 128), layer.w2, None, "none", None, sp):
        ref.assert_near(y[rows], want, err, what="y")
    shared, _ = gpu.ep_gated_ffn(x, layer.s1, layer.s2, residual=x)
    _, _, want, err = bref.ffn(x, layer.s1, layer.s2, "swiglu", x)
    ref.assert_near(shared, want, err, what="shared")
    total, dst = shared.double(), lay.dst_slot.long()
    size = total.abs()
    for k in range(K):
        part = torch.where((dst[:, k] >= 0)[:, None], y[dst[:, k].clamp(min=0)].double() * wts[:, k, None].double(), 0.0)
        total, size = total + part, size + part.abs()
    ref.assert_near(out, total, (K + 1) * ref.U * size, what="out")

    # the gradient of the receive rows: dh = dy W2, in 8 bits, against the transposed codes
    dy, _, _ = gpu.ep_dispatch(torch.randn((T, H), generator=g, device=DEV).to(BF16), lay)
    d8 = gpu.ep_cast_fp8(dy, 128)
    dh = gpu.ep_block_linear(d8, layer.w2_t, lay)
    dv, w2 = bref.rows_value(*d8), bref.weights_value(*layer.w2)
    for (rows, want, err), (e, a, b) in zip(bref.block_linear(d8, layer.w2_t, None, "none", None, sp),
                                            [s for s in sp if s[1] < s[2]]):
        ref.assert_near(dh[rows], want, err, what="dh")
        # the transposed codes stand for the same matrix
        assert torch.allclose(want, dv[a:b] @ w2[e], rtol=1e-12, atol=1e-12)


def step(gpu, layer, x, idx, wts, dout):
    """A serving pass of the layer, and a training step of its shared expert."""
    out = layer.forward(gpu, x, idx, wts)[-1]
    y, z = gpu.ep_gated_ffn(x, layer.s1, layer.s2, save=True)
    return [out, y, *gpu.ep_gated_ffn_backward(dout, x, z, layer.s1, layer.s2)]


@pytest.mark.parametrize("T", [6, 300])
def test_graph_replays_match_eager(gpu, T):
    """Replays with other inputs in the same buffers, eager work and synchronisations
    between them."""
    announce("block chain, graph", T)
    layer = Layer(gpu, 4, 256, 128, T)
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn((T, 256), generator=g, device=DEV).to(BF16)
    idx, wts = routing(T, 4, 2, T), torch.rand((T, 2), generator=g, device=DEV)
    dout = torch.randn((T, 256), generator=g, device=DEV).to(BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(gpu, layer, x, idx, wts, dout)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(gpu, layer, x, idx, wts, dout)
    for i in range(4):
        x.copy_(torch.randn((T, 256), generator=g, device=DEV))
        idx.copy_(routing(T, 4, 2, T + i))
        dout.copy_(torch.randn((T, 256), generator=g, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step(gpu, layer, x, idx, wts, dout)):
            assert torch.equal(a, b)


def test_streams_at_once(gpu):
    """Two callers at the same time: nothing is shared between their calls."""
    announce("block chain, streams")
    jobs = []
    for i, T in enumerate((40, 260)):
        layer = Layer(gpu, 4, 256, 128, i)
        g = torch.Generator(device=DEV).manual_seed(i)
        x = torch.randn((T, 256), generator=g, device=DEV).to(BF16)
        dout = torch.randn((T, 256), generator=g, device=DEV).to(BF16)
        args = (layer, x, routing(T, 4, 2, i), torch.rand((T, 2), generator=g, device=DEV), dout)
        jobs.append((torch.cuda.Stream(), args, step(gpu, *args)))
    torch.cuda.synchronize()
    runs = []
    for _ in range(5):
        for stream, args, want in jobs:
            with torch.cuda.stream(stream):
                runs.append((step(gpu, *args), want))
    torch.cuda.synchronize()
    for got, want in runs:
        for a, b in zip(got, want):
            assert torch.equal(a, b)
