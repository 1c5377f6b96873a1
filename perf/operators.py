"""What the expert operators are measured on: the experts' grouped products over a receive layout
(with bias, activation and residual, the 8-bit checkpoint of their pre-activations, and the
gradients), and the whole mixture-of-experts layer of a few tokens.

`own = False`: the plain forms, elementary torch operations in 32 bits.  `own = True`: the
framework's calls.  8-bit rows are e4m3 codes with one UE8M0 byte (a power of two) per group of
channels, as the framework's fp8 dispatch writes them."""
import math

import torch

own = False

DEV = "cuda:0"
BF16, F32, F64, U8 = torch.bfloat16, torch.float32, torch.float64, torch.uint8
E4M3 = torch.float8_e4m3fn


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # the smallest expert layer of the test workloads: latency of one call
        dict(name="up_tiny", op="linear", T=64, topk=2, E=8, A=1, kin=256, n=512, act="swiglu",
             bias=True, residual=False, fp8=False, transposed=False, checkpoint=True),
        # training, one rank's 8 of 256 experts, 32768 pairs: the gated up projection, its
        # pre-activations kept in 8 bits for the backward pass
        dict(name="up_train", op="linear", T=16384, topk=2, E=8, A=128, kin=7168, n=4096,
             act="swiglu", bias=False, residual=False, fp8=False, transposed=False,
             checkpoint=True),
        # the down projection of the same rank, with a bias and a residual in the rows' order
        dict(name="down_train", op="linear", T=16384, topk=2, E=8, A=128, kin=2048, n=7168,
             act="none", bias=True, residual=True, fp8=False, transposed=False,
             checkpoint=False),
        # the data gradient of the up projection: rows [dg | du] against the weights as they lie
        dict(name="dgrad_train", op="linear", T=16384, topk=2, E=8, A=128, kin=4096, n=7168,
             act="none", bias=False, residual=False, fp8=False, transposed=True,
             checkpoint=False),
        # serving a prefill on fp8 rows and weights
        dict(name="up_fp8", op="linear", T=16384, topk=2, E=8, A=128, kin=7168, n=4096,
             act="swiglu", bias=False, residual=False, fp8=True, transposed=False,
             checkpoint=False),
        # all 256 experts on one GPU: about 128 rows each, bound by reading the weights
        dict(name="up_256_experts", op="linear", T=4096, topk=8, E=256, A=1, kin=7168, n=4096,
             act="swiglu", bias=False, residual=False, fp8=False, transposed=False,
             checkpoint=False),
        # the gated activation's backward from the 8-bit checkpoint, large and odd
        dict(name="act_backward", op="act", T=16384, topk=2, E=8, A=128, n=4096, act="swiglu",
             weights=True),
        dict(name="act_backward_odd", op="act", T=333, topk=3, E=16, A=16, n=1408, act="geglu",
             weights=True),
        # the weight gradient: fp8 receive rows kept from the forward pass, fp32 gradients
        dict(name="wgrad_train", op="wgrad", T=16384, topk=2, E=8, A=128, kin=7168, n=4096,
             fp8=True, bias=False, bf16_out=False, accumulate=False),
        # ragged small experts, bias gradient, gradients accumulated over micro-batches
        dict(name="wgrad_ragged", op="wgrad", T=700, topk=3, E=16, A=1, kin=1024, n=1408,
             fp8=False, bias=True, bf16_out=False, accumulate=True),
        # one token of one sequence
        dict(name="decode_1", op="decode", T=1, topk=8, E=256, hidden=7168, inter=2048,
             act="swiglu", fp8=False, residual=True),
        # the decode batch of the benchmark, on fp8 weights
        dict(name="decode_128_fp8", op="decode", T=128, topk=8, E=256, hidden=7168, inter=2048,
             act="swiglu", fp8=True, residual=False),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step`, spread over the logarithm of [lo, hi]."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "act", "wgrad", "decode", "decode"])
    E = rng.choice([4, 8, 16, 24, 32, 64])
    topk = rng.choice([1, 2, 3, 4])
    T = _log(rng, 1, 16384 // topk)
    A = rng.choice([1, 1, 16, 128])
    acts = ["none", "silu", "gelu", "swiglu", "geglu"]
    if op == "linear":
        fp8 = rng.random() < 0.25
        act = rng.choice(acts)
        transposed = not fp8 and act == "none" and rng.random() < 0.5
        kin = _log(rng, 128, 7168, 128 if fp8 else 8)
        # the weights of all experts stay under those of the largest listed case
        n = _log(rng, 128, 4096, 64)
        return dict(op=op, T=T, topk=topk, E=E, A=A, kin=kin, n=n, act=act,
                    bias=rng.random() < 0.5, residual=rng.random() < 0.3, fp8=fp8,
                    transposed=transposed, checkpoint=act != "none" and rng.random() < 0.5)
    if op == "act":
        return dict(op=op, T=T, topk=topk, E=E, A=A, n=_log(rng, 128, 4096, 64),
                    act=rng.choice(acts[1:]), weights=rng.random() < 0.7)
    if op == "wgrad":
        fp8 = rng.random() < 0.5
        return dict(op=op, T=T, topk=topk, E=E, A=A, kin=_log(rng, 128, 4096, 128 if fp8 else 8),
                    n=_log(rng, 128, 4096, 8), fp8=fp8, bias=rng.random() < 0.5,
                    bf16_out=rng.random() < 0.3, accumulate=rng.random() < 0.3)
    fp8 = rng.random() < 0.5
    return dict(op=op, T=_log(rng, 1, 128), topk=rng.choice([1, 2, 4, 6, 8]),
                E=rng.choice([8, 32, 60, 128]), hidden=_log(rng, 256, 7168, 128),
                inter=_log(rng, 128, 2048, 128), act=rng.choice(["swiglu", "geglu"]), fp8=fp8,
                residual=rng.random() < 0.5)


def _gated(act):
    return act in ("swiglu", "geglu")


# ---- inputs ----------------------------------------------------------------------------------

def _routing(g, T, E, topk, drop):
    """Distinct experts per token in random order; some slots without an expert."""
    idx = torch.rand((T, E), generator=g, device=DEV).argsort(dim=1)[:, :topk].contiguous()
    if drop:
        idx = torch.where(torch.rand((T, topk), generator=g, device=DEV) < 0.02,
                          torch.full_like(idx, -1), idx)
    return idx


def _normal(g, shape, scale, dtype=BF16):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype).mul_(scale)


def _fp8(g, shape, group, top):
    """e4m3 codes of normal values whose groups' largest are near the end of the format, with
    UE8M0 scales a few octaves apart."""
    codes = torch.randn(shape, generator=g, device=DEV, dtype=BF16).mul_(100.0)
    codes = codes.clamp_(-448.0, 448.0).to(E4M3)
    scales = torch.randint(top - 3, top + 1, (*shape[:-1], shape[-1] // group), generator=g,
                           device=DEV, dtype=U8)
    return codes, scales


def _plan(idx, E, A):
    """The receive layout of the routing: per expert the pairs in (token, slot) order, padded to
    A rows; `rows` the rows that hold a pair, `group` their expert, `place` their rank in it."""
    flat = idx.flatten()
    kept = (flat >= 0).nonzero().flatten()
    order = kept[torch.sort(flat[kept], stable=True).indices]
    group = flat[order]
    counts = torch.bincount(group, minlength=E)
    padded = (counts + A - 1) // A * A
    first = torch.cumsum(padded, 0) - padded
    place = torch.arange(group.numel(), device=DEV) - (torch.cumsum(counts, 0) - counts)[group]
    return dict(rows=first[group] + place, group=group, place=place,
                cap=max(1, int(counts.max())), counts=counts.tolist(), first=first.tolist())


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(c)
    T, E, topk = c["T"], c["E"], c["topk"]
    s["idx"] = _routing(g, T, E, topk, c["op"] != "decode")
    if c["op"] == "decode":
        H, inter = c["hidden"], c["inter"]
        s["w"] = torch.softmax(torch.randn((T, topk), generator=g, device=DEV), dim=1)
        s["x"] = _normal(g, (T, H), 1.0)
        s["res"] = _normal(g, (T, H), 1.0) if c["residual"] else None
        if c["fp8"]:
            s["w1"] = _fp8(g, (E, 2 * inter, H), 128, 116)
            s["w2"] = _fp8(g, (E, H, inter), 128, 116)
        else:
            s["w1"] = _normal(g, (E, 2 * inter, H), H ** -0.5)
            s["w2"] = _normal(g, (E, H, inter), inter ** -0.5)
        return s
    # rows of the receive buffer: the worst case of the routing, as a program allocates it
    R = T * topk + min(E, T * topk) * (c["A"] - 1)
    s["R"] = R
    s["plan"] = _plan(s["idx"], E, c["A"])
    n, act = c["n"], c.get("act", "none")
    if c["op"] == "linear":
        k = c["kin"]
        m = n // 2 if _gated(act) else n
        if c["fp8"]:
            s["x"] = _fp8(g, (R, k), 128, 121)
            s["weight"] = _fp8(g, (E, n, k), 128, 116)
        else:
            s["x"] = _normal(g, (R, k), 1.0)
            s["weight"] = _normal(g, (E, k, n) if c["transposed"] else (E, n, k), k ** -0.5)
        s["b"] = _normal(g, (E, n), 0.5) if c["bias"] else None
        s["res"] = _normal(g, (R, m), 1.0) if c["residual"] else None
        s["out"] = torch.zeros((R, m), device=DEV, dtype=BF16)
        if c["checkpoint"]:
            s["codes"] = torch.zeros((R, n), device=DEV, dtype=U8).view(E4M3)
            s["scales"] = torch.zeros((R, n // 32), device=DEV, dtype=U8)
    elif c["op"] == "act":
        m = n // 2 if _gated(act) else n
        s["dh"] = _normal(g, (R, m), 0.02)
        s["pre"] = _fp8(g, (R, n), 32, 121)
        s["w"] = torch.rand((R,), generator=g, device=DEV) if c["weights"] else None
        s["dpre"] = torch.zeros((R, n), device=DEV, dtype=BF16)
        s["h"] = torch.zeros((R, m), device=DEV, dtype=BF16)
        s["dw"] = torch.zeros((R,), device=DEV, dtype=F32)
    else:
        k = c["kin"]
        s["dy"] = _normal(g, (R, n), 0.02)
        s["x"] = _fp8(g, (R, k), 128, 121) if c["fp8"] else _normal(g, (R, k), 1.0)
        dt = BF16 if c["bf16_out"] else F32
        if c["accumulate"]:
            s["dw0"] = _normal(g, (E, n, k), 0.1, dt)
            s["db0"] = _normal(g, (E, n), 0.1, F32) if c["bias"] else None
    if own:
        # the dispatch's handle, which the program has before its experts run
        import combine_ep_get_layout_amd as ep
        s["layout"] = ep.ep_get_layout(s["idx"], E, c["A"])
    return s


# ---- plain forms -----------------------------------------------------------------------------

def _wide(v, dtype=F32):
    """Rows in `dtype`: 8-bit rows as the values they stand for."""
    if v is None:
        return None
    if not isinstance(v, tuple):
        return v.to(dtype)
    codes, scales = v
    grouped = codes.to(dtype).unflatten(-1, (scales.shape[-1], -1))
    return (grouped * torch.exp2(scales.to(dtype) - 127.0).unsqueeze(-1)).flatten(-2)


def _f(z, act):
    if act in ("silu", "swiglu"):
        return z / (1.0 + torch.exp(-z))
    if act in ("gelu", "geglu"):
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _df(z, act):
    if act in ("silu", "swiglu"):
        p = 1.0 / (1.0 + torch.exp(-z))
        return p + z * p * (1.0 - p)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 0.134145 * z * z)


def _activate(z, act):
    if _gated(act):
        gate, up = z.chunk(2, dim=-1)
        return _f(gate, act) * up
    return _f(z, act)


def _packed(x, p, E):
    """The pairs' rows in one block per expert, [E, cap, columns], zeros behind each."""
    out = torch.zeros((E, p["cap"], x.shape[1]), device=DEV, dtype=x.dtype)
    out[p["group"], p["place"]] = x[p["rows"]]
    return out


def _checkpoint(z):
    """z after e4m3 with a power of two per 32 channels, as the values kept: exact in bf16."""
    v = z.unflatten(-1, (-1, 32))
    amax = v.abs().amax(dim=-1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2(torch.clamp(amax, min=1e-4).double() / 448.0))).float()
    return ((v / scale).to(E4M3).to(F32) * scale).flatten(-2).to(BF16)


def _plain_linear(s):
    p, E = s["plan"], s["E"]
    w = _wide(s["weight"])
    z = torch.bmm(_packed(_wide(s["x"]), p, E), w if s["transposed"] else w.transpose(1, 2))
    z = z[p["group"], p["place"]]
    if s["b"] is not None:
        z = z + s["b"].float()[p["group"]]
    y = _activate(z, s["act"])
    if s["res"] is not None:
        y = y + s["res"].float()[p["rows"]]
    out = torch.zeros_like(s["out"])
    out[p["rows"]] = y.to(BF16)
    if not s["checkpoint"]:
        return out
    kept = torch.zeros((s["R"], s["n"]), device=DEV, dtype=BF16)
    kept[p["rows"]] = _checkpoint(z)
    return out, kept


def _plain_act(s):
    p, act = s["plan"], s["act"]
    rows = p["rows"]
    z = _wide((s["pre"][0][rows], s["pre"][1][rows]))
    dh = s["dh"][rows].float()
    h = _activate(z, act)
    dw = (dh * h).sum(dim=1)
    if s["w"] is not None:
        w = s["w"][rows].unsqueeze(1)
        dh, h = dh * w, h * w
    if _gated(act):
        gate, up = z.chunk(2, dim=-1)
        dz = torch.cat([dh * up * _df(gate, act), dh * _f(gate, act)], dim=1)
    else:
        dz = dh * _df(z, act)
    out = [torch.zeros_like(s[name]) for name in ("dpre", "h", "dw")]
    for o, v in zip(out, (dz, h, dw)):
        o[rows] = v.to(o.dtype)
    return out


def _plain_wgrad(s):
    p, E = s["plan"], s["E"]
    dy = _packed(s["dy"].float(), p, E)
    dw = torch.bmm(dy.transpose(1, 2), _packed(_wide(s["x"]), p, E))
    db = dy.sum(dim=1) if s["bias"] else None
    if s["accumulate"]:
        dw = dw + s["dw0"].float()
        db = db + s["db0"] if s["bias"] else None
    return [dw.to(BF16 if s["bf16_out"] else F32)] + ([db] if s["bias"] else [])


def _plain_decode(s):
    x, idx, act, E, K = s["x"].float(), s["idx"], s["act"], s["E"], s["topk"]
    T, flat = x.shape[0], idx.flatten()
    xp = x.repeat_interleave(K, dim=0)
    if flat.numel() <= E:
        # few pairs: each takes its own expert's weights
        take = lambda w: _wide(tuple(v[flat] for v in w) if isinstance(w, tuple) else w[flat])  # noqa: E731
        h = _activate(torch.bmm(take(s["w1"]), xp.unsqueeze(2)).squeeze(2), act)
        y = torch.bmm(take(s["w2"]), h.unsqueeze(2)).squeeze(2)
    else:
        # every expert, a block of at most T rows each (a token's experts are distinct)
        token = torch.arange(T, device=DEV).repeat_interleave(K)
        block = torch.zeros((E, T, x.shape[1]), device=DEV)
        block[flat, token] = xp
        h = _activate(torch.bmm(block, _wide(s["w1"]).transpose(1, 2)), act)
        y = torch.bmm(h, _wide(s["w2"]).transpose(1, 2))[flat, token]
    out = (y.unflatten(0, (T, K)) * s["w"].unsqueeze(2)).sum(dim=1)
    if s["res"] is not None:
        out = out + s["res"].float()
    return out.to(BF16)


# ---- the framework's calls -------------------------------------------------------------------

def _own(s):
    import combine_ep_get_layout_amd as ep
    op = s["op"]
    if op == "decode":
        return ep.ep_moe_decode(s["x"], s["idx"], s["w"], s["w1"], s["w2"], activation=s["act"],
                                bias=s["res"])
    lay = s["layout"]
    if op == "linear":
        kept = (s["codes"], s["scales"]) if s["checkpoint"] else None
        out, kept = ep.ep_expert_linear(s["x"], s["weight"], lay, bias=s["b"],
                                        activation=s["act"], residual=s["res"],
                                        transposed=s["transposed"], checkpoint=kept,
                                        out=s["out"])
        return (out, _wide(kept, BF16)) if s["checkpoint"] else out
    if op == "act":
        return list(ep.ep_expert_activation_backward(
            s["dh"], s["pre"], lay, activation=s["act"], row_weights=s["w"],
            out=(s["dpre"], s["h"], s["dw"])))
    dw, db = ep.ep_expert_wgrad(s["dy"], s["x"], lay, bias_grad=s["bias"],
                                dtype=BF16 if s["bf16_out"] else F32,
                                accumulate=(s["dw0"], s["db0"]) if s["accumulate"] else None)
    return [dw] + ([db] if s["bias"] else [])


def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "act": _plain_act, "wgrad": _plain_wgrad,
            "decode": _plain_decode}[state["op"]](state)


# ---- accounting ------------------------------------------------------------------------------

def work(case):
    c = case
    pairs = c["T"] * c["topk"]
    b = 1 if c.get("fp8") else 2
    if c["op"] == "decode":
        experts = c["E"] * (1.0 - (1.0 - c["topk"] / c["E"]) ** c["T"])
        weights = 3 * c["hidden"] * c["inter"] * experts
        return {"bytes": weights * (b + (1 / 128 if c["fp8"] else 0))
                + c["T"] * c["hidden"] * (6 if c["residual"] else 4) + 12.0 * pairs,
                "flops": 6.0 * pairs * c["hidden"] * c["inter"]}
    rows = 0.98 * pairs
    n, act = c["n"], c.get("act", "none")
    m = n // 2 if _gated(act) else n
    if c["op"] == "act":
        return {"bytes": rows * (2 * m + n * (1 + 1 / 32) + 2 * n + 2 * m + 8),
                "flops": 20.0 * rows * n}
    k = c["kin"]
    xb = k * (b + (1 / 128 if c["fp8"] else 0))
    if c["op"] == "wgrad":
        out = c["E"] * n * k * (2 if c["bf16_out"] else 4) * (2 if c["accumulate"] else 1)
        return {"bytes": rows * (2 * n + xb) + out, "flops": 2.0 * rows * n * k}
    experts = c["E"] * (1.0 - (1.0 - 0.98 * c["topk"] / c["E"]) ** c["T"])
    moved = rows * xb + experts * n * xb + rows * m * (4 if c["residual"] else 2)
    moved += rows * n * (1 + 1 / 32) if c["checkpoint"] else 0
    return {"bytes": moved, "flops": 2.0 * rows * n * k}


# ---- the definition in 64 bits ---------------------------------------------------------------

def _value(v):
    """What stored numbers are, in 64 bits."""
    if not isinstance(v, tuple):
        return v.double()
    codes, scales = v
    per = codes.shape[-1] // scales.shape[-1]
    return codes.double() * torch.pow(2.0, scales.double() - 127).repeat_interleave(per, dim=-1)


def _at(v, i):
    return tuple(t[i] for t in v) if isinstance(v, tuple) else v[i]


def _sigma(z):
    return torch.sigmoid(z)


_G = math.sqrt(2 / math.pi)


def _act64(z, act):
    """(value, derivative) of the activation function."""
    if act in ("silu", "swiglu"):
        q = _sigma(z)
        return z * q, q * (1 + z * (1 - q))
    if act in ("gelu", "geglu"):
        t = torch.tanh(_G * (z + 0.044715 * z ** 3))
        return z * (1 + t) / 2, (1 + t) / 2 + z / 2 * (1 - t ** 2) * _G * (1 + 3 * 0.044715 * z ** 2)
    return z, torch.ones_like(z)


def _halves(z):
    return z[..., :z.shape[-1] // 2], z[..., z.shape[-1] // 2:]


def _through(z, act):
    if _gated(act):
        a, b = _halves(z)
        return _act64(a, act)[0] * b
    return _act64(z, act)[0]


def _kept64(z):
    """The 8-bit checkpoint's values: nearest e4m3 multiples of the groups' powers of two."""
    v = z.reshape(z.shape[0], -1, 32)
    top = torch.clamp(v.abs().max(dim=2, keepdim=True).values, min=float(torch.tensor(1e-4)))
    s = torch.pow(2.0, torch.ceil(torch.log2(top / 448)))
    q = v / s
    step = torch.pow(2.0, torch.clamp(torch.floor(torch.log2(q.abs().clamp(min=1e-30))), min=-6) - 3)
    return (torch.round(q / step) * step * s).reshape(z.shape)


def exact(case, seed):
    s = prepare(case, seed)
    E, act = s["E"], s.get("act", "none")
    if s["op"] == "decode":
        x, out = s["x"].double(), torch.zeros(s["x"].shape, device=DEV, dtype=F64)
        if s["res"] is not None:
            out += s["res"].double()
        for e in range(E):
            t, k = (s["idx"] == e).nonzero(as_tuple=True)
            if t.numel():
                h = _through(x[t] @ _value(_at(s["w1"], e)).T, act)
                out.index_add_(0, t, h @ _value(_at(s["w2"], e)).T * s["w"][t, k, None].double())
        return out
    p = s["plan"]
    spans = [(e, a, a + c) for e, (a, c) in enumerate(zip(p["first"], p["counts"])) if c]
    if s["op"] == "linear":
        out = torch.zeros(s["out"].shape, device=DEV, dtype=F64)
        kept = torch.zeros((s["R"], s["n"]), device=DEV, dtype=F64) if s["checkpoint"] else None
        for e, a, z in spans:
            w = _value(_at(s["weight"], e))
            v = _value(_at(s["x"], slice(a, z))) @ (w if s["transposed"] else w.T)
            if s["b"] is not None:
                v = v + s["b"][e].double()
            out[a:z] = _through(v, act)
            if kept is not None:
                kept[a:z] = _kept64(v)
            if s["res"] is not None:
                out[a:z] += s["res"][a:z].double()
        return (out, kept) if s["checkpoint"] else out
    if s["op"] == "act":
        out = [torch.zeros(s[v].shape, device=DEV, dtype=F64) for v in ("dpre", "h", "dw")]
        for e, a, b in spans:
            z, dh = _value(_at(s["pre"], slice(a, b))), s["dh"][a:b].double()
            w = 1.0 if s["w"] is None else s["w"][a:b, None].double()
            h = _through(z, act)
            if _gated(act):
                g, u = _halves(z)
                f, df = _act64(g, act)
                out[0][a:b] = torch.cat([w * dh * u * df, w * dh * f], dim=1)
            else:
                out[0][a:b] = w * dh * _act64(z, act)[1]
            out[1][a:b] = w * h
            out[2][a:b] = (dh * h).sum(dim=1)
        return out
    k, n = s["kin"], s["n"]
    dw = s["dw0"].double() if s["accumulate"] else torch.zeros((E, n, k), device=DEV, dtype=F64)
    db = torch.zeros((E, n), device=DEV, dtype=F64)
    if s["accumulate"] and s["bias"]:
        db = s["db0"].double()
    for e, a, z in spans:
        dy = s["dy"][a:z].double()
        dw[e] += dy.T @ _value(_at(s["x"], slice(a, z)))
        db[e] += dy.sum(dim=0)
    return [dw] + ([db] if s["bias"] else [])
