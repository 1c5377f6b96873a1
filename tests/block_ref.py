"""The block-scaled product and the gated feed-forward block from their
definitions in 64 bits, and the error each output may have (see expert_ref for
the constants and the fp8 instruction's cut)."""
import torch

import expert_ref as ref

B = 128


def rows_value(codes, scales):
    c = codes.view(torch.float8_e4m3fn) if codes.dtype == torch.uint8 else codes
    return c.double() * scales.double().repeat_interleave(B, dim=-1)


def weights_value(codes, scales):
    per = scales.double().repeat_interleave(B, dim=-1).repeat_interleave(B, dim=-2)
    c = codes.view(torch.float8_e4m3fn) if codes.dtype == torch.uint8 else codes
    return c.double() * per[..., :c.shape[-2], :]


def block_linear(x, w, bias, act, residual, sp):
    """Per span (rows, out, its error before the rounding).  One block: 128
    products are added in fp32, each group of 8 cut below 2^-13 of its largest;
    then one rounding of the scales' product, one fused multiply-add a block, and
    at most 8 partial sums."""
    xv = rows_value(*x)
    K = xv.shape[1]
    for e, a, b in sp:
        if a == b:
            continue
        we = weights_value(*(v if e is None else v[e] for v in w)).T
        z = xv[a:b] @ we
        dz = (B + 3 + K // B + 8) * ref.U * (xv[a:b].abs() @ we.abs())
        big = lambda v: v.abs().unflatten(-1, (-1, 8)).amax(-1)  # noqa: E731
        dz = dz + 7 * 2.0 ** -13 * (big(xv[a:b]) @ big(we.T).T)
        if bias is not None:
            bv = (bias if e is None else bias[e]).double()
            z = z + bv
            dz = dz + ref.U * (z.abs() + bv.abs())
        y, dy = ref.activate(z, act, dz)
        if residual is not None:
            y = y + residual[a:b].double()
            dy = dy + ref.U * y.abs()
        yield slice(a, b), y, dy


def rounded(v, dv):
    """The error of bf16(v) where v is off by at most dv."""
    return dv + ref.BF16_HALF * (v.abs() + dv)


def ffn(x, w1, w2, act, residual):
    """(z, its error, out, its error), both errors before their rounding."""
    xv, v1, v2 = x.double(), w1.double(), w2.double()
    z = xv @ v1.T
    dz = (xv.shape[1] + 9) * ref.U * (xv.abs() @ v1.abs().T)
    h, dh = ref.activate(z, act, dz)
    dh = rounded(h, dh)
    out = h @ v2.T
    err = dh @ v2.abs().T + (h.shape[1] + 9) * ref.U * ((h.abs() + dh) @ v2.abs().T)
    if residual is not None:
        out = out + residual.double()
        err = err + ref.U * out.abs()
    return z, dz, out, err


def ffn_backward(dout, x, z, w1, w2, act):
    """((dx, error), (dw1, error), (dw2, error)) before the last rounding."""
    d, xv, v1, v2 = dout.double(), x.double(), w1.double(), w2.double()
    g, u = z.double().chunk(2, dim=1)
    f, df = ref.f_df(g, act)
    dh = d @ v2
    e = (d.shape[1] + 1) * ref.U * (d.abs() @ v2.abs())
    # the value to a few u of itself; the derivative p + f (1 - p) (2 y')' of the
    # terms' sizes: |p| <= 1 and a second term under 1.13 + 1
    ef, edf = ref.ACT_U * f.abs(), ref.ACT_U * 2.2
    dg, du = dh * u * df, dh * f
    eg = rounded(dg, e * u.abs() * (df.abs() + edf) + dh.abs() * u.abs() * edf + 2 * ref.U * dg.abs())
    eu = rounded(du, e * (f.abs() + ef) + dh.abs() * ef + ref.U * du.abs())
    h = f * u
    eh = rounded(h, ef * u.abs() + ref.U * h.abs())
    dz, ez = torch.cat([dg, du], 1), torch.cat([eg, eu], 1)
    T = x.shape[0]

    def product(a, ea, b, n):
        return a @ b, ea @ b.abs() + (n + 2) * ref.U * ((a.abs() + ea) @ b.abs())

    dx = product(dz, ez, v1, dz.shape[1])
    dw1 = [v.T for v in product(xv.T, torch.zeros_like(xv.T), dz, T)]
    dw1[1] = dw1[1] + (xv.abs().T @ ez).T * (1 + (T + 2) * ref.U)
    dw2 = [d.T @ h, (d.abs().T @ eh) + (T + 2) * ref.U * (d.abs().T @ (h.abs() + eh))]
    return dx, tuple(dw1), tuple(dw2)
