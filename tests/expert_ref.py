"""The expert operators from their definition in 64 bits, and the error each
output may have.

u = 2^-24 bounds one fp32 rounding relative to the value, 2^-8 one bf16
rounding and 2^-4 one e4m3 rounding (half a step).  Products of bf16 or fp8
values are exact in fp32, and a sum of K of them in any order is off by at
most K u sum |x w|.  The fp8 matrix instruction adds less exactly: it aligns
the products of 8 consecutive channels to the largest of them and cuts each off
below 2^-13 of that one's power of two before it adds them to the fp32 sum
(seen by adding one product 2^-s of another: kept to s = 13, and to s = 23 from
another 8 channels).  A product so loses less than 2^-13 of the largest, which
is at most max |x| max |w| of the 8 channels, and the largest itself, with its 8
significant bits, nothing: 7 2^-13 max |x| max |w| per 8 channels.  Every bound
below carries these through the formula (the activations' derivatives are at
most 1.13 in magnitude) and adds the last rounding.  The exponential and the reciprocal behind the activations are good
to a few u; 32 u covers them."""
import math

import torch

U = 2.0 ** -24
BF16_HALF = 2.0 ** -8
SLOPE = 1.13
ACT_U = 32 * U
# The hardware's exponential and reciprocal may flush a gate under 2^-126 to 0;
# the factors a gate meets here (z, z^2, u, d, w with |z|, |u|, |d| under 2^5,
# w at most 1) multiply that to less than 2^-126 2^25 < 2^-100.
TINY = 2.0 ** -100


def value(v):
    """Rows or weights in float64; (codes, UE8M0 scales) as the values they stand for."""
    if not isinstance(v, tuple):
        return v.double()
    codes, scales = v
    g = codes.shape[-1] // scales.shape[-1]
    c = codes.view(torch.float8_e4m3fn) if codes.dtype == torch.uint8 else codes
    return c.double() * torch.exp2(scales.double() - 127).repeat_interleave(g, dim=-1)


def gated(act):
    return act in ("swiglu", "geglu")


def f_df(z, act):
    if act in ("silu", "swiglu"):
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))
    if act in ("gelu", "geglu"):
        c = math.sqrt(2 / math.pi)
        # (1 + tanh y) / 2 = sigmoid(2 y), which keeps its digits where tanh y is near -1
        p = torch.sigmoid(2 * c * (z + 0.044715 * z ** 3))
        return z * p, p + z * p * (1 - p) * 2 * c * (1 + 0.134145 * z * z)
    return z, torch.ones_like(z)


def activate(z, act, dz):
    """(act(z), its error when z is off by at most dz)."""
    if gated(act):
        n = z.shape[-1] // 2
        g, u, dg, du = z[..., :n], z[..., n:], dz[..., :n], dz[..., n:]
        f = f_df(g, act)[0]
        df = SLOPE * dg + ACT_U * f.abs()
        return f * u, df * u.abs() + f.abs() * du + df * du
    f = f_df(z, act)[0]
    return f, SLOPE * dz + (ACT_U * f.abs() if act != "none" else 0)


def spans(lay, num_rows):
    """(expert, first row, one past the last row) of the rows that hold a pair."""
    off, cnt = lay.expert_offset.tolist(), lay.num_tokens_per_expert.tolist()
    return [(e, off[e], max(off[e], min(off[e] + min(cnt[e], off[e + 1] - off[e]), num_rows)))
            for e in range(len(cnt))]


def linear(x, w, bias, act, residual, transposed, sp):
    """Per span (rows, z, z's error, out, out's error before its rounding)."""
    xv, wv = value(x), value(w)
    for e, a, b in sp:
        if a == b:
            continue
        we = wv[e] if transposed else wv[e].T
        z = xv[a:b] @ we
        dz = (xv.shape[1] + 1) * U * (xv[a:b].abs() @ we.abs())
        if isinstance(x, tuple):
            big = lambda v: v.abs().unflatten(-1, (-1, 8)).amax(-1)  # noqa: E731
            dz = dz + 7 * 2.0 ** -13 * (big(xv[a:b]) @ big(we.T).T)
        if bias is not None:
            z = z + bias[e].double()
            dz = dz + U * z.abs() + U * bias[e].double().abs()
        y, dy = activate(z, act, dz)
        if residual is not None:
            y = y + residual[a:b].double()
            dy = dy + U * y.abs()
        yield slice(a, b), z, dz, y, dy


def assert_near(got, want, err, half=BF16_HALF, what=""):
    got = got.double()
    bad = ~((got - want).abs() <= err + half * (want.abs() + err) + TINY)
    if bad.any():
        i = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{got[tuple(i)].item()} for {want[tuple(i)].item()}")


def assert_checkpoint(codes, scales, z, dz):
    """codes and scales hold z (off by at most dz) to half an e4m3 step, under
    the smallest power of two s with amax <= 448 s."""
    s = torch.exp2(scales.double() - 127).repeat_interleave(32, dim=-1)
    got = value((codes, scales))
    # half a step: 2^-4 of a normal value, 2^-10 s below 2^-6 s
    half = torch.maximum(z.abs() * 2.0 ** -4, s * 2.0 ** -10)
    assert ((got - z).abs() <= half + dz * (1 + 2.0 ** -3)).all()
    amax = z.abs().unflatten(-1, (-1, 32)).amax(-1)
    da = dz.unflatten(-1, (-1, 32)).amax(-1)
    lo = torch.ceil(torch.log2((amax - da).clamp(min=1e-4) / 448 * (1 - 2 * U)))
    hi = torch.ceil(torch.log2((amax + da).clamp(min=1e-4) / 448 * (1 + 2 * U)))
    e = scales.double() - 127
    assert ((e >= lo) & (e <= hi)).all()
