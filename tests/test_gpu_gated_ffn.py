"""ep_gated_ffn and ep_gated_ffn_backward against the formulas in 64 bits, and
the gradients against differences."""
import pytest
import torch

import block_ref as bref
import expert_ref as ref
from gpu_util import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


def make(T, H, inter, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    return (n(T, H).to(BF16), (n(2 * inter, H) * H ** -0.5).to(BF16), (n(H, inter) * inter ** -0.5).to(BF16),
            n(T, H).to(BF16), g)


def check(gpu, T, H, inter, act="swiglu", residual=True):
    announce("gated ffn", T, H, inter, act, residual)
    x, w1, w2, r, _ = make(T, H, inter, T + H)
    r = r if residual else None
    z, dz, want, err = bref.ffn(x, w1, w2, act, r)
    out, none = gpu.ep_gated_ffn(x, w1, w2, act, residual=r)
    assert none is None
    ref.assert_near(out, want, err, what="out")
    saved, kept = gpu.ep_gated_ffn(x, w1, w2, act, residual=r, save=True)
    ref.assert_near(saved, want, err, what="out beside z")
    ref.assert_near(kept, z, dz, what="z")


# few rows (three groups), tiles of 64, 128, 192 and 256 rows
@pytest.mark.parametrize("T", [1, 2, 16, 17, 33, 64, 65, 100, 129, 160, 161, 300, 1000])
@pytest.mark.parametrize("H,inter,act", [(256, 128, "swiglu"), (520, 264, "geglu"), (1024, 1408, "swiglu")])
def test_forward(gpu, T, H, inter, act):
    check(gpu, T, H, inter, act, residual=T % 2 == 0)


@pytest.mark.parametrize("H,inter", [(8, 8), (8, 1000), (1000, 8), (24, 40), (72, 24)])
@pytest.mark.parametrize("T", [1, 50, 200, 600])
def test_forward_odd_sizes(gpu, T, H, inter):
    check(gpu, T, H, inter)


# products whole and in parts in tiles of each size
@pytest.mark.parametrize("T,H,inter", [(100, 4096, 256), (512, 4096, 1024), (512, 2048, 4096), (640, 128, 1696),
                                       (640, 3392, 64), (1024, 2048, 1280), (1024, 2560, 2048), (2100, 3584, 72),
                                       (2100, 2048, 2048)])
def test_forward_tiles(gpu, T, H, inter):
    check(gpu, T, H, inter)


def check_backward(gpu, T, H, inter, act, seed=0):
    announce("gated ffn backward", T, H, inter, act)
    x, w1, w2, dout, g = make(T, H, inter, T + H + seed)
    z = torch.randn((T, 2 * inter), generator=g, device=DEV).to(BF16)
    want = bref.ffn_backward(dout, x, z, w1, w2, act)
    start = [torch.randn(w.shape, generator=g, device=DEV) for w in (w1, w2)]
    for dt, half in ((torch.float32, ref.U), (BF16, ref.BF16_HALF)):
        got = gpu.ep_gated_ffn_backward(dout, x, z, w1, w2, act, dtype=dt)
        assert [t.dtype for t in got] == [BF16, dt, dt]
        for name, v, (y, e), h in zip(("dx", "dw1", "dw2"), got, want, (ref.BF16_HALF, half, half)):
            ref.assert_near(v, y, e, h, name)
        add = [s.to(dt) for s in start]
        more = gpu.ep_gated_ffn_backward(dout, x, z, w1, w2, act, dtype=dt, accumulate=add,
                                         out=(None, add[0].clone(), add[1].clone()))
        in_place = [s.clone() for s in add]
        gpu.ep_gated_ffn_backward(dout, x, z, w1, w2, act, dtype=dt, accumulate=in_place, out=(None, *in_place))
        for i in (1, 2):
            y, e = want[i]
            ref.assert_near(more[i], y + add[i - 1].double(), e + ref.U * (y.abs() + add[i - 1].double().abs()), half)
            assert torch.equal(more[i], in_place[i - 1])
        assert torch.equal(more[0], got[0])


@pytest.mark.parametrize("T", [1, 16, 63, 64, 65, 130, 161, 500, 1300])
@pytest.mark.parametrize("H,inter,act", [(256, 128, "swiglu"), (520, 264, "geglu"), (1024, 1408, "geglu")])
def test_backward(gpu, T, H, inter, act):
    check_backward(gpu, T, H, inter, act)


@pytest.mark.parametrize("H,inter", [(8, 8), (8, 1000), (1000, 8), (24, 40)])
@pytest.mark.parametrize("T", [1, 200, 600])
def test_backward_odd_sizes(gpu, T, H, inter):
    check_backward(gpu, T, H, inter, "swiglu")


def test_backward_many_rows(gpu):
    check_backward(gpu, 2500, 4096, 1536, "swiglu")


# sizes whose products take every pair of tiles: weight gradients in 128 x 128 tiles,
# in runs of rows, in 256 x 256 tiles; dx whole and in parts of each tile
@pytest.mark.parametrize("T,H,inter", [(700, 2048, 1024), (1500, 4096, 512), (1100, 512, 2048), (600, 4096, 2048),
                                       (5000, 256, 512), (3000, 1024, 264), (2000, 136, 1400),
                                       (1024, 2560, 1024), (4096, 1792, 64), (4096, 128, 1792)])
def test_backward_tiles(gpu, T, H, inter):
    check_backward(gpu, T, H, inter, "geglu")


@pytest.mark.parametrize("rows", [4000, 9000])
def test_backward_of_many_rows_and_few_weights(gpu, rows):
    check_backward(gpu, rows, 128, 136, "swiglu")


@pytest.mark.parametrize("act", ["swiglu", "geglu"])
def test_gradients_against_differences(gpu, act):
    """Forward and backward pass together, along random directions.  x and w1 are
    small whole numbers (over 8), so that z is a bf16 number and nothing is lost
    where it is kept; the difference of the formula in 64 bits is off by its step
    squared, and the gradients by their bounds."""
    announce("gated ffn, differences", act)
    T, H, inter = 40, 64, 48
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randint(-2, 3, (T, H), generator=g, device=DEV).to(BF16)
    w1 = (torch.randint(-1, 2, (2 * inter, H), generator=g, device=DEV) / 8).to(BF16)
    w2 = torch.randn((H, inter), generator=g, device=DEV).to(BF16)
    dout = torch.randn((T, H), generator=g, device=DEV).to(BF16)
    _, z = gpu.ep_gated_ffn(x, w1, w2, act, save=True)
    assert torch.equal(z.double(), x.double() @ w1.double().T)
    got = gpu.ep_gated_ffn_backward(dout, x, z, w1, w2, act)
    bounds = bref.ffn_backward(dout, x, z, w1, w2, act)

    def loss(a, b, c):
        gate, up = (a @ b.T).chunk(2, dim=1)
        return (dout.double() * ((ref.f_df(gate, act)[0] * up) @ c.T)).sum()

    at = [x.double(), w1.double(), w2.double()]
    eps = 1e-5
    for i in range(3):
        d = torch.randn(at[i].shape, generator=g, device=DEV, dtype=torch.float64)
        hi, lo = ([v + s * eps * d if j == i else v for j, v in enumerate(at)] for s in (1, -1))
        diff = (loss(*hi) - loss(*lo)) / (2 * eps)
        y, e = bounds[i]
        half = ref.BF16_HALF if i == 0 else ref.U
        room = ((e + half * (y.abs() + e)) * d.abs()).sum() + 1e-6 * (y * d).abs().sum()
        assert abs((got[i].double() * d).sum() - diff) <= room
        assert room < 0.5 * (y * d).abs().sum()            # the bound tells a gradient from none


def test_no_tokens(gpu):
    announce("gated ffn, no tokens")
    x, w1, w2, _, _ = make(0, 64, 32, 0)
    out, z = gpu.ep_gated_ffn(x, w1, w2, save=True)
    assert out.shape == (0, 64) and z.shape == (0, 64)
    one = [torch.ones_like(w, dtype=torch.float32) for w in (w1, w2)]
    dx, d1, d2 = gpu.ep_gated_ffn_backward(out, x, z, w1, w2)
    assert dx.shape == (0, 64) and not d1.any() and not d2.any()
    _, d1, d2 = gpu.ep_gated_ffn_backward(out, x, z, w1, w2, accumulate=one)
    assert (d1 == 1).all() and (d2 == 1).all()


def test_one_gradient_to_add_to(gpu):
    announce("gated ffn, one gradient to add to")
    x, w1, w2, dout, _ = make(70, 64, 32, 1)
    _, z = gpu.ep_gated_ffn(x, w1, w2, save=True)
    a = gpu.ep_gated_ffn_backward(dout, x, z, w1, w2)
    b = gpu.ep_gated_ffn_backward(dout, x, z, w1, w2, accumulate=(None, torch.ones_like(a[2])))
    assert torch.equal(a[1], b[1]) and not torch.equal(a[2], b[2])


def test_weight_gradients_alone(gpu):
    """Without dx (the C entry point's NULL)."""
    announce("gated ffn, no dx")
    import ctypes

    from combine_ep_get_layout_amd import _abi
    lib = _abi.load()
    V = ctypes.c_void_p
    for T, H, inter in ((20, 64, 32), (900, 256, 512), (2500, 4096, 1536)):
        x, w1, w2, dout, g = make(T, H, inter, 6)
        z = torch.randn((T, 2 * inter), generator=g, device=DEV).to(BF16)
        want = gpu.ep_gated_ffn_backward(dout, x, z, w1, w2)
        d1, d2 = torch.zeros_like(want[1]), torch.zeros_like(want[2])
        n = lib.ep_gated_ffn_workspace_bytes(T, H, inter, 1)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        p = [V(t.data_ptr()) for t in (dout, x, z, w1, w2, ws, d1, d2)]
        rc = lib.ep_gated_ffn_backward(p[0], p[1], p[2], T, H, inter, p[3], p[4], _abi.EP_ACT_SWIGLU, None, None,
                                       p[5], n, None, p[6], p[7], 0, V(torch.cuda.current_stream().cuda_stream))
        assert rc == 0
        torch.cuda.synchronize()
        assert torch.equal(d1, want[1]) and torch.equal(d2, want[2])


def test_rows_do_not_mix(gpu):
    """A row of infinities or NaN reaches its own output row alone."""
    announce("gated ffn, non-finite rows")
    for T in (40, 300):
        x, w1, w2, _, _ = make(T, 128, 72, 2)
        want, _ = gpu.ep_gated_ffn(x, w1, w2)
        x[5], x[9] = float("nan"), float("inf")
        out, _ = gpu.ep_gated_ffn(x, w1, w2)
        keep = torch.arange(T, device=DEV)
        keep = keep[(keep != 5) & (keep != 9)]
        assert torch.equal(out[keep], want[keep]) and out[5].isnan().all() and not out[9].isfinite().any()


def test_huge_gates_stay_finite_in_the_gradients(gpu):
    announce("gated ffn, huge gates")
    for act in ("swiglu", "geglu"):
        x, w1, w2, dout, _ = make(100, 64, 32, 3)
        z = torch.full((100, 64), 1.0, device=DEV, dtype=BF16)
        z[:50, :32], z[50:, :32] = 3e4, -3e4
        for t in gpu.ep_gated_ffn_backward(dout, x, z, w1, w2, act):
            assert t.isfinite().all()


def test_residual_in_place(gpu):
    announce("gated ffn, residual in place")
    for T in (30, 300):
        x, w1, w2, r, _ = make(T, 128, 64, 4)
        want, _ = gpu.ep_gated_ffn(x, w1, w2, residual=r)
        out, _ = gpu.ep_gated_ffn(x, w1, w2, residual=r, out=r)
        assert out is r and torch.equal(out, want)


def test_binding_checks(gpu):
    announce("gated ffn, binding")
    x, w1, w2, r, _ = make(10, 64, 32, 5)
    _, z = gpu.ep_gated_ffn(x, w1, w2, save=True)
    for bad in (lambda: gpu.ep_gated_ffn(x, w1[:62].contiguous(), w2), lambda: gpu.ep_gated_ffn(x, w1, w2.t()),
                lambda: gpu.ep_gated_ffn(x.float(), w1, w2), lambda: gpu.ep_gated_ffn(x, w1, w2, residual=r[:9]),
                lambda: gpu.ep_gated_ffn(x, w1, w2, save=z[:9]), lambda: gpu.ep_gated_ffn(x, w1, w2, out=r[:9]),
                lambda: gpu.ep_gated_ffn(x, w1, w2, "silu"),
                lambda: gpu.ep_gated_ffn_backward(r, x, z[:, :32].contiguous(), w1, w2),
                lambda: gpu.ep_gated_ffn_backward(r[:9], x, z, w1, w2),
                lambda: gpu.ep_gated_ffn_backward(r, x, z, w1, w2, accumulate=(w1, w2)),
                lambda: gpu.ep_gated_ffn_backward(r, x, z, w1, w2, out=(r, None, w2))):
        with pytest.raises(ValueError):
            bad()


def test_offsets_past_32_bits(gpu):
    """4.4 million rows of 1024 bytes: rows around byte 2^31 and 2^32 of x, dout, out and
    dx, the first and the last ones.  The other rows' dout is zero, so that the weight
    gradients are those of these rows."""
    T, H, inter = 4_400_000, 512, 64
    announce("gated ffn", T, H, inter)
    g = torch.Generator(device=DEV).manual_seed(5)
    n = lambda *s: torch.empty(s, device=DEV, dtype=BF16).normal_(generator=g)  # noqa: E731
    x, w1, w2 = n(T, H), (n(2 * inter, H) * H ** -0.5), (n(H, inter) * inter ** -0.5)
    at = torch.cat([torch.arange(b - 40, b + 40, device=DEV) for b in (40, 1 << 21, 1 << 22, T - 40)])
    dout = torch.zeros(T, H, device=DEV, dtype=BF16)
    dout[at] = n(len(at), H)
    out, z = gpu.ep_gated_ffn(x, w1, w2, save=True)
    zv, dz, want, err = bref.ffn(x[at], w1, w2, "swiglu", None)
    ref.assert_near(out[at], want, err, what="out")
    ref.assert_near(z[at], zv, dz, what="z")
    del out
    got = gpu.ep_gated_ffn_backward(dout, x, z, w1, w2)
    want = bref.ffn_backward(dout[at], x[at], z[at], w1, w2, "swiglu")
    for name, v, (y, e), h in zip(("dx", "dw1", "dw2"), (got[0][at], *got[1:]), want,
                                  (ref.BF16_HALF, ref.U, ref.U)):
        ref.assert_near(v, y, e, h, name)
    live = torch.zeros(T, device=DEV, dtype=torch.bool)
    live[at] = True
    assert not (got[0] != 0).any(dim=1)[~live].any()
