"""ep_expert_wgrad and ep_expert_activation_backward against their definitions
in 64 bits, and against differences."""
import pytest
import torch

import expert_ref as ref
from gpu_util import announce
from test_gpu_expert_linear import DEV, make, routing

pytestmark = pytest.mark.gpu


def held_rows(lay, rows):
    held = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for _, a, b in ref.spans(lay, rows):
        held[a:b] = True
    return held


@pytest.mark.parametrize("T,E,K,A", [(1, 4, 1, 1), (40, 8, 2, 16), (300, 3, 2, 1), (900, 2, 1, 128)])
@pytest.mark.parametrize("n,k", [(8, 8), (256, 256), (264, 136), (520, 1000)])
def test_wgrad(gpu, T, E, K, A, n, k):
    announce("wgrad", T, E, K, A, n, k)
    lay, rows, x, _, g = make(gpu, T, E, K, k, 8, A)
    dy = torch.randn((rows, n), generator=g, device=DEV).bfloat16()
    check_wgrad(gpu, lay, rows, dy, x, g)


@pytest.mark.parametrize("T,E,K", [(5, 4, 1), (130, 3, 2), (700, 2, 2)])
@pytest.mark.parametrize("n,k", [(64, 128), (328, 640)])
def test_wgrad_fp8_rows(gpu, T, E, K, n, k):
    announce("wgrad fp8", T, E, K, n, k)
    lay, rows, x, _, g = make(gpu, T, E, K, k, 8)
    x = (x.float() * torch.exp2(torch.randint(-30, 30, (rows, k // 128), generator=g, device=DEV)
                                .float()).repeat_interleave(128, dim=1)).bfloat16()
    dy = torch.randn((rows, n), generator=g, device=DEV).bfloat16()
    check_wgrad(gpu, lay, rows, dy, gpu.ep_cast_fp8(x, 128, scale_fmt="ue8m0"), g)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,k", [(2056, 1000), (1024, 2176)])
def test_wgrad_of_large_outputs(gpu, n, k, fp8):
    """At least 256 tiles of 256 x 256, of experts with no, one, and many rows."""
    if fp8:
        k = (k + 127) // 128 * 128
    announce("wgrad large", n, k, fp8)
    counts = [0, 1, 63, 64, 65, 400, 1000, 1700]
    idx = torch.cat([torch.full((c,), e, dtype=torch.int64) for e, c in enumerate(counts)])
    idx = idx[torch.randperm(len(idx), generator=torch.Generator().manual_seed(n))].unsqueeze(1).to(DEV)
    lay, rows, x, _, g = make(gpu, len(idx), len(counts), 1, k, 8, idx=idx)
    if fp8:
        x = gpu.ep_cast_fp8(x, 128, scale_fmt="ue8m0")
    dy = torch.randn((rows, n), generator=g, device=DEV).bfloat16()
    check_wgrad(gpu, lay, rows, dy, x, g)


def check_wgrad(gpu, lay, rows, dy, x, g):
    E, n = lay.num_experts, dy.shape[1]
    k = (x[0] if isinstance(x, tuple) else x).shape[1]
    held = held_rows(lay, rows)
    dy[~held] = float("nan")
    if isinstance(x, tuple):
        x[0].view(torch.uint8)[~held] = 0x7F
    else:
        x[~held] = float("nan")
    yv, xv = dy.double(), ref.value(x)
    want = torch.zeros((E, n, k), dtype=torch.float64, device=DEV)
    err, wb, eb = torch.zeros_like(want), want[:, :, 0].clone(), want[:, :, 0].clone()
    for e, a, b in ref.spans(lay, rows):
        want[e] = yv[a:b].T @ xv[a:b]
        err[e] = (b - a) * ref.U * (yv[a:b].abs().T @ xv[a:b].abs())
        wb[e] = yv[a:b].sum(0)
        eb[e] = (b - a) * ref.U * yv[a:b].abs().sum(0)
    for dt, half in ((torch.float32, ref.U), (torch.bfloat16, ref.BF16_HALF)):
        dw, db = gpu.ep_expert_wgrad(dy, x, lay, bias_grad=True, dtype=dt)
        ref.assert_near(dw, want, err, half, "dw")
        ref.assert_near(db, wb, eb, ref.U, "db")
        only, none = gpu.ep_expert_wgrad(dy, x, lay, dtype=dt)
        assert none is None and torch.equal(only, dw)
        dw0 = torch.randn((E, n, k), generator=g, device=DEV).to(dt)
        db0 = torch.randn((E, n), generator=g, device=DEV)
        w2, b2 = gpu.ep_expert_wgrad(dy, x, lay, bias_grad=True, dtype=dt, accumulate=(dw0, db0))
        ref.assert_near(w2, want + dw0.double(), err, half, "dw + dw0")
        ref.assert_near(b2, wb + db0.double(), eb, ref.U, "db + db0")
        # into the gradients themselves
        gpu.ep_expert_wgrad(dy, x, lay, bias_grad=True, dtype=dt, accumulate=(dw0, db0),
                            out=(dw0, db0))
        assert torch.equal(dw0, w2) and torch.equal(db0, b2)


def test_wgrad_of_experts_without_rows(gpu):
    idx = torch.full((30, 1), 2, device=DEV, dtype=torch.int64)
    lay, rows, x, _, g = make(gpu, 30, 4, 1, 64, 8, idx=idx)
    dy = torch.randn((rows, 32), generator=g, device=DEV).bfloat16()
    dw = torch.full((4, 32, 64), 9.0, device=DEV)
    db = torch.full((4, 32), 9.0, device=DEV)
    gpu.ep_expert_wgrad(dy, x, lay, bias_grad=True, out=(dw, db))
    assert (dw[[0, 1, 3]] == 0).all() and (db[[0, 1, 3]] == 0).all() and (dw[2] != 0).any()
    lay0 = gpu.ep_get_layout(idx[:0], 4)
    dw, db = gpu.ep_expert_wgrad(dy[:0], x[:0], lay0, bias_grad=True)
    assert (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "swiglu", "geglu"])
@pytest.mark.parametrize("T,E,K,A,n,ckpt", [(1, 2, 1, 1, 64, True), (200, 4, 2, 16, 1088, True),
                                            (100, 3, 2, 1, 2112, True), (150, 4, 2, 1, 272, False)])
@pytest.mark.parametrize("weights", [False, True])
def test_activation_backward(gpu, act, T, E, K, A, n, ckpt, weights):
    announce("activation backward", act, T, E, K, A, n, ckpt, weights)
    lay, rows, z, _, g = make(gpu, T, E, K, n, 8, A)
    z = (z.float() * 3).bfloat16()
    m = n // 2 if ref.gated(act) else n
    dh = torch.randn((rows, m), generator=g, device=DEV).bfloat16()
    w = torch.rand((rows,), generator=g, device=DEV) if weights else None
    held = held_rows(lay, rows)
    dh[~held] = float("nan")
    pre = gpu.ep_cast_fp8(z, 32, scale_fmt="ue8m0") if ckpt else z
    out = (torch.full((rows, n), 7.0, device=DEV, dtype=torch.bfloat16),
           torch.full((rows, m), 7.0, device=DEV, dtype=torch.bfloat16),
           torch.full((rows,), 7.0, device=DEV))
    got = gpu.ep_expert_activation_backward(dh, pre, lay, act, w, out=out)
    torch.cuda.synchronize()
    for o in got:
        assert (o[~held] == 7.0).all()
    zv, dv = ref.value(pre)[held], dh[held].double()
    wv = w[held].double().unsqueeze(1) if weights else 1.0
    h, dpre = _gradients(zv, dv, wv, act)
    # each factor is good to ACT_U relative to |z| times its slope, products add 4 u
    tol = 4 * ref.ACT_U
    mag = _magnitudes(zv, dv, wv, act)
    ref.assert_near(got[0][held], dpre, tol * mag[1], what="dpre")
    ref.assert_near(got[1][held], h * wv, tol * (mag[0] * wv), what="h")
    ref.assert_near(got[2][held], (dv * h).sum(1),
                    (tol + m * ref.U) * (dv.abs() * mag[0]).sum(1), ref.U, "dweights")


def _gradients(z, d, w, act):
    if ref.gated(act):
        n = z.shape[1] // 2
        g, u = z[:, :n], z[:, n:]
        f, df = ref.f_df(g, act)
        return f * u, torch.cat([w * d * u * df, w * d * f], dim=1)
    f, df = ref.f_df(z, act)
    return f, w * d * df


def _magnitudes(z, d, w, act):
    """Bounds of |h| and |dpre| by magnitudes of their factors (f' is formed as
    p + f (1 - p) y': terms of at most 1 + |f| (1 + |z|^2))."""
    if ref.gated(act):
        n = z.shape[1] // 2
        g, u = z[:, :n], z[:, n:]
        f = ref.f_df(g, act)[0].abs()
        big = 1 + f * (1 + 0.25 * g * g)
        return f * u.abs(), torch.cat([(w * d * u).abs() * big, (w * d).abs() * f], dim=1)
    f = ref.f_df(z, act)[0].abs()
    return f, (w * d).abs() * (1 + f * (1 + 0.25 * z * z))


@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu", "geglu"])
def test_activation_backward_against_differences(gpu, act):
    """Central differences of the definition, L = sum over rows of w h . c."""
    lay, rows, z, _, g = make(gpu, 60, 3, 2, 128, 8)
    m = 64 if ref.gated(act) else 128
    c = torch.randn((rows, m), generator=g, device=DEV).bfloat16()
    w = torch.rand((rows,), generator=g, device=DEV)
    dpre, _, dw = gpu.ep_expert_activation_backward(c, z, lay, act, w)
    held = held_rows(lay, rows)
    zv, cv, wv = z[held].double(), c[held].double(), w[held].double()
    h = lambda v: ref.activate(v, act, torch.zeros_like(v))[0]  # noqa: E731
    loss = lambda v, s: ((h(v) * cv).sum(1) * s)  # noqa: E731
    step = 1e-4
    for col in (0, 5, 63, 64, 127):
        d = torch.zeros_like(zv)
        d[:, col] = step
        num = (loss(zv + d, wv) - loss(zv - d, wv)) / (2 * step)
        # differences are good to step^2 times the third derivative; bf16 results
        ref.assert_near(dpre[held][:, col], num, 1e-6 * (1 + cv.abs().amax(1) * 8), what=f"col {col}")
    num = (loss(zv, wv + step) - loss(zv, wv - step)) / (2 * step)
    ref.assert_near(dw[held], num, 1e-4 * torch.ones_like(num), ref.U, "dweights")


@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu", "geglu"])
def test_activation_of_huge_values(gpu, act):
    """From about 100 on an activation is z or 0 and its derivative 1 or 0, to the
    last bit of fp32, up to the end of the format."""
    announce("activation of huge values", act)
    lay, rows, _, _, g = make(gpu, 40, 2, 1, 8, 8)
    n, m = 64, 32 if ref.gated(act) else 64
    z = torch.randn((rows, n), generator=g, device=DEV).bfloat16()
    huge = torch.tensor([100.0, 1e10, 2e19, 6e19, 1e20, 1e30, 3e38], device=DEV).bfloat16()
    z[:, :7], z[:, 7:14] = huge, -huge
    dh = (torch.randn((rows, m), generator=g, device=DEV) * 2.0 ** -10).bfloat16()
    if ref.gated(act):
        z[:, 32:46] = 1.0
    dpre, h, dw = gpu.ep_expert_activation_backward(dh, z, lay, act)
    held = held_rows(lay, rows)
    assert torch.equal(dpre[held][:, :7], dh[held][:, :7])
    assert (dpre[held][:, 7:14] == 0).all()
    assert torch.equal(h[held][:, :7], z[held][:, :7]) and (h[held][:, 7:14] == 0).all()
    if ref.gated(act):
        assert torch.equal(dpre[held][:, 32:39], (dh[held][:, :7].double() * huge.double()).bfloat16())
        assert (dpre[held][:, 39:46] == 0).all()
    assert torch.isfinite(dw[held]).all() and torch.isfinite(dpre[held].float()).all()
    # and forward, from the product's sums
    x = torch.zeros((rows, n), device=DEV, dtype=torch.bfloat16)
    x[:] = z
    w = torch.eye(n, device=DEV).bfloat16().expand(2, n, n).contiguous()
    out, _ = gpu.ep_expert_linear(x, w, lay, activation=act)
    assert torch.equal(out[held][:, :7], huge.expand(int(held.sum()), 7)) and (out[held][:, 7:14] == 0).all()
