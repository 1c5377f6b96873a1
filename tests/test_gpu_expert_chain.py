"""The expert operators together, as they are used: a training step of the
experts between dispatch and combine against the formulas in 64 bits, and the
operators captured into a HIP graph against eager calls, bit for bit."""
import pytest
import torch

import expert_ref as ref
from gpu_util import announce
from test_gpu_expert_linear import DEV, routing

pytestmark = pytest.mark.gpu


class Bounded:
    """A value in 64 bits with a bound on the error of its stored counterpart."""

    def __init__(self, v, e=None):
        self.v, self.e = v, torch.zeros_like(v) if e is None else e

    def rounded(self):
        """Stored in bf16."""
        return Bounded(self.v, self.e + ref.BF16_HALF * (self.v.abs() + self.e))

    def product(self, w):
        """self @ w with exact w, summed in fp32."""
        a = w.abs()
        return Bounded(self.v @ w, self.e @ a + w.shape[0] * ref.U * ((self.v.abs() + self.e) @ a))

    def times(self, o):
        return Bounded(self.v * o.v, self.e * o.v.abs() + self.v.abs() * o.e + self.e * o.e
                       + 2 * ref.U * (self.v * o.v).abs())


@pytest.mark.parametrize("T,E,K,A", [(150, 4, 2, 16), (900, 3, 2, 128)])
def test_training_step(gpu, T, E, K, A):
    announce("chain", T, E, K, A)
    H, inter = 256, 192
    g = torch.Generator(device=DEV).manual_seed(T)
    idx = routing(T, E, K, T)
    w = torch.rand((T, K), generator=g, device=DEV)
    x = torch.randn((T, H), generator=g, device=DEV).bfloat16()
    w1 = (torch.randn((E, 2 * inter, H), generator=g, device=DEV) * H ** -0.5).bfloat16()
    w2 = (torch.randn((E, H, inter), generator=g, device=DEV) * inter ** -0.5).bfloat16()
    dout = torch.randn((T, H), generator=g, device=DEV).bfloat16()

    lay = gpu.ep_get_layout(idx, E, A)
    recv, _, rw = gpu.ep_dispatch(x, lay, w)
    h, kept = gpu.ep_expert_linear(recv, w1, lay, activation="swiglu", checkpoint=True)
    y, _ = gpu.ep_expert_linear(h, w2, lay)
    out, _ = gpu.ep_combine(y, lay, w)
    # backward: the combine's is a dispatch, the dispatch's a combine
    drow, _, _ = gpu.ep_dispatch(dout, lay)
    dh, _ = gpu.ep_expert_linear(drow, w2, lay, transposed=True)
    dz, hw, dweights = gpu.ep_expert_activation_backward(dh, kept, lay, "swiglu", rw)
    dw2, _ = gpu.ep_expert_wgrad(drow, hw, lay)
    dw1, _ = gpu.ep_expert_wgrad(dz, recv, lay)
    drecv, _ = gpu.ep_expert_linear(dz, w1, lay, transposed=True)
    dx, _ = gpu.ep_combine(drecv, lay, None)
    assert lay.check() == 0

    # the formulas, with the checkpoint as it was kept (its own error is
    # test_gpu_expert_linear's subject)
    z8 = ref.value(kept)
    want_out, want_dx = (Bounded(torch.zeros((T, H), dtype=torch.float64, device=DEV)) for _ in "ab")
    src = lay.src_of_slot.long()
    for e, a, b in ref.spans(lay, lay.max_recv_rows):
        if a == b:
            continue
        pair = src[a:b]
        t, wt = pair // K, w.flatten()[pair].double().unsqueeze(1)
        assert (idx.flatten()[pair] == e).all()
        xe, v1, v2 = x[t].double(), w1[e].double(), w2[e].double()
        z = Bounded(xe).product(v1.T)
        f, fe = ref.activate(z.v, "swiglu", z.e)
        ye = Bounded(f, fe).rounded().product(v2.T).rounded()
        want_out.v.index_add_(0, t, wt * ye.v)
        want_out.e.index_add_(0, t, wt * (ye.e + K * ref.U * ye.v.abs()))

        de = Bounded(dout[t].double())
        dhe = de.product(v2).rounded()
        gate, up = z8[a:b].chunk(2, dim=1)
        f, df = ref.f_df(gate, "swiglu")
        hq = Bounded(f * up, 4 * ref.ACT_U * (f * up).abs())
        ref.assert_near(dweights[a:b], (dhe.v * hq.v).sum(1),
                        dhe.times(hq).e.sum(1) + inter * ref.U * (dhe.v * hq.v).abs().sum(1), ref.U)
        one = Bounded(wt.expand_as(dhe.v).contiguous())
        d = dhe.times(one)
        slope = 1 + f.abs() * (1 + 0.25 * gate * gate)
        dze = Bounded(torch.cat([d.v * up * df, d.v * f], 1),
                      torch.cat([d.e * (up * df).abs() + 4 * ref.ACT_U * (d.v * up).abs() * slope,
                                 d.e * f.abs() + 4 * ref.ACT_U * (d.v * f).abs()], 1)).rounded()
        hwe = hq.times(one).rounded()
        n = b - a
        ref.assert_near(dw2[e], de.v.T @ hwe.v,
                        de.v.abs().T @ hwe.e + n * ref.U * (de.v.abs().T @ (hwe.v.abs() + hwe.e)), ref.U)
        ref.assert_near(dw1[e], dze.v.T @ xe,
                        dze.e.T @ xe.abs() + n * ref.U * ((dze.v.abs() + dze.e).T @ xe.abs()), ref.U)
        dr = dze.product(v1).rounded()
        want_dx.v.index_add_(0, t, dr.v)
        want_dx.e.index_add_(0, t, dr.e + K * ref.U * dr.v.abs())
    ref.assert_near(out, want_out.v, want_out.e, what="out")
    ref.assert_near(dx, want_dx.v, want_dx.e, what="dx")


def test_fp8_rows_through_dispatch_and_back(gpu):
    """The fp8 dispatch's rows go into the product as they are, and, kept in 8
    bits, into the weight gradient: the same as of the rows they stand for."""
    T, E, K, H, N = 400, 4, 2, 512, 256
    g = torch.Generator(device=DEV).manual_seed(1)
    idx = routing(T, E, K, 1)
    x = torch.randn((T, H), generator=g, device=DEV).bfloat16()
    lay = gpu.ep_get_layout(idx, E, 16)
    q, s, _ = gpu.ep_dispatch(x, lay, recv_fp8=True, scale_fmt="ue8m0")
    wc, ws = gpu.ep_cast_fp8(torch.randn((E * N, H), generator=g, device=DEV).bfloat16(), 128,
                             scale_fmt="ue8m0")
    w = (wc.view(E, N, H), ws.view(E, N, -1))
    out, _ = gpu.ep_expert_linear((q, s), w, lay, activation="silu")
    for rs, z, dz, y, dy in ref.linear((q, s), w, None, "silu", None, False,
                                       ref.spans(lay, lay.max_recv_rows)):
        ref.assert_near(out[rs], y, dy)
    dy = torch.randn((lay.max_recv_rows, N), generator=g, device=DEV).bfloat16()
    dw, _ = gpu.ep_expert_wgrad(dy, (q, s), lay)
    # the scales are powers of two: the rows that hold a pair are bf16 numbers
    rows = ref.value((q, s)).bfloat16()
    for _, a, b in ref.spans(lay, lay.max_recv_rows):
        assert torch.equal(rows[a:b].double(), ref.value((q[a:b], s[a:b])))
    dw2, _ = gpu.ep_expert_wgrad(dy, rows, lay)
    assert torch.equal(dw, dw2)


def test_graph_replays_match_eager(gpu):
    """Layout, products, gradients and the decode layer in one graph, replayed on
    new inputs with eager work of the same shapes in between."""
    T, E, K, H, inter = 300, 4, 2, 256, 128
    st = dict(idx=torch.zeros((T, K), dtype=torch.int64, device=DEV),
              x=torch.zeros((T, H), dtype=torch.bfloat16, device=DEV),
              w=torch.zeros((T, K), device=DEV))
    g = torch.Generator(device=DEV).manual_seed(0)
    w1 = (torch.randn((E, 2 * inter, H), generator=g, device=DEV) * H ** -0.5).bfloat16()
    w2 = (torch.randn((E, H, inter), generator=g, device=DEV) * inter ** -0.5).bfloat16()

    def fill(seed):
        gg = torch.Generator(device=DEV).manual_seed(seed)
        st["idx"].copy_(routing(T, E, K, seed))
        st["x"].copy_(torch.randn((T, H), generator=gg, device=DEV))
        st["w"].copy_(torch.rand((T, K), generator=gg, device=DEV))

    def run(lay=None):
        lay = gpu.ep_get_layout(st["idx"], E, 16, layout=lay)
        rows = lay.max_recv_rows
        new = lambda c, dt=torch.bfloat16: torch.zeros((rows, c) if c else rows, dtype=dt, device=DEV)  # noqa: E731
        recv, _, rw = gpu.ep_dispatch(st["x"], lay, st["w"], zero_padding=True)
        h, kept = gpu.ep_expert_linear(recv, w1, lay, activation="swiglu", out=new(inter),
                                       checkpoint=(new(2 * inter, torch.uint8), new(2 * inter // 32, torch.uint8)))
        y, _ = gpu.ep_expert_linear(h, w2, lay, out=new(H))
        out, _ = gpu.ep_combine(y, lay, st["w"])
        dh, _ = gpu.ep_expert_linear(recv, w2, lay, transposed=True, out=new(inter))
        dz, hw, dw = gpu.ep_expert_activation_backward(
            dh, kept, lay, "swiglu", rw, out=(new(2 * inter), new(inter), new(0, torch.float32)))
        dw1, db1 = gpu.ep_expert_wgrad(dz, recv, lay, bias_grad=True)
        dec = gpu.ep_moe_decode(st["x"][:40], st["idx"][:40], st["w"][:40], w1, w2)
        return [h, *kept, y, out, dh, dz, hw, dw, dw1, db1, dec]

    fill(1)
    lay = gpu.ep_get_layout(st["idx"], E, 16)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run(lay)
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(lay)
    for seed in (2, 3, 4, 5):
        announce("expert graph replay", seed)
        fill(seed)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        seen = [t.clone() for t in got]
        want = run()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(seen, want)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i


@pytest.mark.parametrize("T,E,K,A", [(150, 4, 2, 16), (900, 3, 2, 128)])
def test_gradients_behind_a_down_bias(gpu, T, E, K, A):
    """out = sum_k w (W2 h + b2): the routing weights' gradient needs b2's term, and
    b2's own is the column sum of the weighted gradient rows."""
    announce("chain with a down bias", T, E, K, A)
    H, inter = 256, 192
    g = torch.Generator(device=DEV).manual_seed(T)
    idx = routing(T, E, K, T)
    w = torch.rand((T, K), generator=g, device=DEV)
    x = torch.randn((T, H), generator=g, device=DEV).bfloat16()
    w1 = (torch.randn((E, 2 * inter, H), generator=g, device=DEV) * H ** -0.5).bfloat16()
    w2 = (torch.randn((E, H, inter), generator=g, device=DEV) * inter ** -0.5).bfloat16()
    b2 = torch.randn((E, H), generator=g, device=DEV).bfloat16()
    dout = torch.randn((T, H), generator=g, device=DEV).bfloat16()

    lay = gpu.ep_get_layout(idx, E, A)
    recv, _, rw = gpu.ep_dispatch(x, lay, w, zero_padding=True)
    _, kept = gpu.ep_expert_linear(recv, w1, lay, activation="swiglu", checkpoint=True)
    drow, _, _ = gpu.ep_dispatch(dout, lay, zero_padding=True)
    dh, _ = gpu.ep_expert_linear(drow, w2, lay, transposed=True)
    _, _, dweights = gpu.ep_expert_activation_backward(dh, kept, lay, "swiglu", rw)
    weighted = (drow.float() * rw.unsqueeze(1)).bfloat16()
    _, db2 = gpu.ep_expert_wgrad(weighted, recv, lay, bias_grad=True)

    z8 = ref.value(kept)
    missing = 0.0
    for e, a, b in ref.spans(lay, lay.max_recv_rows):
        pair = lay.src_of_slot.long()[a:b]
        t, wt = pair // K, w.flatten()[pair].double().unsqueeze(1)
        de, bias = dout[t].double(), b2[e].double()
        f = ref.f_df(z8[a:b, :inter], "swiglu")[0]
        h = f * z8[a:b, inter:]
        # L = sum_r w_r dout_r . (W2 h_r + b2)
        want = (de * (h @ w2[e].double().T + bias)).sum(1)
        dhe = Bounded(de).product(w2[e].double()).rounded()
        err = dhe.times(Bounded(h, 4 * ref.ACT_U * h.abs())).e.sum(1)
        err += inter * ref.U * (dhe.v * h).abs().sum(1) + (H + 2) * ref.U * (de * bias).abs().sum(1)
        term = (drow[a:b].float() * b2[e].float()).sum(1)
        # the sum of the two: one more rounding, of the first relative to itself
        err += ref.U * ((dhe.v * h).sum(1).abs() + (de * bias).sum(1).abs())
        ref.assert_near(dweights[a:b] + term, want, err, ref.U, "routing weights")
        missing = max(missing, ((dweights[a:b].double() - want).abs() - err).max().item() if b > a else 0.0)
        ref.assert_near(db2[e], (wt * de).sum(0),
                        (ref.BF16_HALF + (b - a + 1) * ref.U) * (wt * de).abs().sum(0) * (1 + ref.BF16_HALF),
                        ref.U, "db2")
    assert missing > 1.0                               # the term matters here


@pytest.mark.parametrize("byte", [10, 30, 220, 246])
def test_scales_near_the_ends(gpu, byte):
    """fp8 values that pass through bf16 on their way (checkpoint, weight gradient,
    decode): smallest and largest codes under the smallest and largest scales that
    keep them normal numbers."""
    announce("expert scales near the ends", byte)
    T, E, K, k, n = 300, 3, 2, 256, 128
    g = torch.Generator(device=DEV).manual_seed(byte)
    back = 2.0 ** (127 - byte)

    def fp8(shape, b):
        c = torch.randint(0, 127, shape, generator=g, device=DEV, dtype=torch.uint8)
        c = c | torch.randint(0, 2, shape, generator=g, device=DEV, dtype=torch.uint8) << 7
        return c, torch.full((*shape[:-1], shape[-1] // 128), b, device=DEV, dtype=torch.uint8)

    idx = routing(T, E, K, byte)
    lay = gpu.ep_get_layout(idx, E)
    rows = lay.max_recv_rows
    x, w = fp8((rows, k), byte), fp8((E, n, k), 254 - byte)
    out, ck = gpu.ep_expert_linear(x, w, lay, checkpoint=True)
    for rs, _, _, y, _ in ref.linear(x, w, None, "none", None, False, ref.spans(lay, rows)):
        e = next(e for e, a, b in ref.spans(lay, rows) if a == rs.start and b > a)
        err = (k + 1) * ref.U * (ref.value(x)[rs].abs() @ ref.value(w)[e].T.abs())
        ref.assert_near(out[rs], y, err, what="linear")
        ref.assert_checkpoint(ck[0][rs], ck[1][rs], y, err)

    dy = (torch.randn((rows, n), generator=g, device=DEV) * back).bfloat16()
    dw, _ = gpu.ep_expert_wgrad(dy, x, lay)
    for e, a, b in ref.spans(lay, rows):
        yv, xv = dy[a:b].double(), ref.value(x)[a:b]
        ref.assert_near(dw[e], yv.T @ xv, (b - a) * ref.U * (yv.abs().T @ xv.abs()), ref.U, "dw")

    xt = (torch.randn((20, k), generator=g, device=DEV) * back * 2.0 ** -12).bfloat16()
    w1, w2 = fp8((E, n, k), byte), fp8((E, k, n), 112)
    few = gpu.ep_moe_decode(xt, idx[:20], None, w1, w2, "none")
    want, err = (torch.zeros((20, k), dtype=torch.float64, device=DEV) for _ in "ab")
    for e in range(E):
        t, _ = (idx[:20] == e).nonzero(as_tuple=True)
        v1, v2, xv = ref.value(w1)[e], ref.value(w2)[e], xt[t].double()
        h = xv @ v1.T
        dh = (k + 1) * ref.U * (xv.abs() @ v1.T.abs())
        dh = dh + ref.BF16_HALF ** 2 * (h.abs() + dh)
        y = h @ v2.T
        want.index_add_(0, t, y)
        err.index_add_(0, t, (dh + (n + 1) * ref.U * (h.abs() + dh)) @ v2.T.abs() + (K + 2) * ref.U * y.abs())
    ref.assert_near(few, want, err, what="decode")
