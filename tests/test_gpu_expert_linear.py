"""ep_expert_linear against its definition in 64 bits: types, activations,
transposed weights, bias, residual, the 8-bit checkpoint; ragged and empty
experts, odd sizes, padding rows that hold NaN, fixed capacity, short buffers."""
import pytest
import torch

import expert_ref as ref
from gpu_util import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def routing(T, E, K, seed, drop=0.1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    idx = torch.rand((T, E), generator=g, device=DEV).argsort(dim=1)[:, :K].contiguous()
    return torch.where(torch.rand((T, K), generator=g, device=DEV) < drop, -1, idx)


def make(gpu, T, E, K, k, n, A=1, fp8=False, transposed=False, seed=0, idx=None, **kw):
    idx = routing(T, E, K, seed) if idx is None else idx
    lay = gpu.ep_get_layout(idx, E, A, **kw)
    rows = lay.max_recv_rows
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    x = torch.randn((rows, k), generator=g, device=DEV).bfloat16()
    w = (torch.randn((E, k, n) if transposed else (E, n, k), generator=g, device=DEV)
         * k ** -0.5).bfloat16()
    if fp8:
        x = gpu.ep_cast_fp8(x, 128, scale_fmt="ue8m0")
        c, s = gpu.ep_cast_fp8(w.view(E * n, k), 128, scale_fmt="ue8m0")
        w = (c.view(E, n, k), s.view(E, n, k // 128))
    return lay, rows, x, w, g


def check(gpu, lay, rows, x, w, act="none", bias=None, residual=None, transposed=False,
          checkpoint=False):
    n = (w[0] if isinstance(w, tuple) else w).shape[2 if transposed else 1]
    m = n // 2 if ref.gated(act) else n
    # padding rows hold NaN, and no output row of theirs may change
    sp = ref.spans(lay, rows)
    held = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for _, a, b in sp:
        held[a:b] = True
    if isinstance(x, tuple):
        x[0].view(torch.uint8)[~held] = 0x7F
    else:
        x[~held] = float("nan")
    out = torch.full((rows, m), 7.0, device=DEV, dtype=torch.bfloat16)
    kept = None
    if checkpoint:
        kept = (torch.full((rows, n), 3, device=DEV, dtype=torch.uint8),
                torch.full((rows, n // 32), 5, device=DEV, dtype=torch.uint8))
    got, ck = gpu.ep_expert_linear(x, w, lay, bias=bias, activation=act, residual=residual,
                                   transposed=transposed, checkpoint=kept, out=out)
    torch.cuda.synchronize()
    assert got is out
    assert (out[~held] == 7.0).all()
    for rs, z, dz, y, dy in ref.linear(x, w, bias, act, residual, transposed, sp):
        ref.assert_near(out[rs], y, dy, what=f"rows {rs}")
        if checkpoint:
            ref.assert_checkpoint(ck[0][rs], ck[1][rs], z, dz)
    if checkpoint:
        assert (ck[0][~held] == 3).all() and (ck[1][~held] == 5).all()
    return out


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "swiglu", "geglu"])
@pytest.mark.parametrize("T,E,K,k,n", [(64, 8, 2, 256, 512), (700, 3, 2, 200, 320),
                                       (900, 4, 2, 328, 576)])
def test_activations_bias_residual(gpu, act, T, E, K, k, n):
    announce("linear", act, T, E, K, k, n)
    lay, rows, x, w, g = make(gpu, T, E, K, k, n)
    b = torch.randn((E, n), generator=g, device=DEV).bfloat16()
    m = n // 2 if ref.gated(act) else n
    res = torch.randn((rows, m), generator=g, device=DEV).bfloat16()
    check(gpu, lay, rows, x, w, act, b, res, checkpoint=True)
    check(gpu, lay, rows, x, w, act)


@pytest.mark.parametrize("k", [8, 64, 72, 136, 1024])
@pytest.mark.parametrize("n", [8, 256, 264, 1000])
@pytest.mark.parametrize("transposed", [False, True])
def test_odd_sizes(gpu, k, n, transposed):
    announce("linear sizes", k, n, transposed)
    for T, E in ((1, 1), (33, 5), (600, 2)):
        lay, rows, x, w, _ = make(gpu, T, E, 1, k, n, transposed=transposed)
        check(gpu, lay, rows, x, w, transposed=transposed)


@pytest.mark.parametrize("T,E,K,A", [(1, 8, 2, 1), (50, 8, 2, 16), (500, 6, 2, 128),
                                     (1500, 4, 2, 1)])
@pytest.mark.parametrize("k,n", [(128, 64), (640, 448), (1536, 1088)])
def test_fp8(gpu, T, E, K, A, k, n):
    announce("linear fp8", T, E, K, A, k, n)
    for act in ("none", "swiglu"):
        lay, rows, x, w, g = make(gpu, T, E, K, k, n, A, fp8=True)
        b = torch.randn((E, n), generator=g, device=DEV).bfloat16()
        check(gpu, lay, rows, x, w, act, b, checkpoint=True)


@pytest.mark.parametrize("act,n", [("swiglu", 16), ("geglu", 80), ("silu", 8)])
def test_narrow_outputs(gpu, act, n):
    announce("linear narrow", act, n)
    for T, E in ((20, 3), (700, 2)):
        lay, rows, x, w, _ = make(gpu, T, E, 1, 72, n)
        check(gpu, lay, rows, x, w, act)


@pytest.mark.parametrize("T", [60, 700])
def test_transposed_weights_with_every_part_of_the_epilogue(gpu, T):
    announce("linear transposed epilogue", T)
    lay, rows, x, w, g = make(gpu, T, 2, 1, 136, 448, transposed=True)
    b = torch.randn((2, 448), generator=g, device=DEV).bfloat16()
    res = torch.randn((rows, 224), generator=g, device=DEV).bfloat16()
    check(gpu, lay, rows, x, w, "swiglu", b, res, transposed=True, checkpoint=True)


@pytest.mark.parametrize("T", [100, 260, 300, 400])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "transposed"])
def test_rows_per_expert(gpu, T, kind):
    """50, 130, 150 and 200 expected rows an expert (each has its row tile), with
    experts on both sides of it."""
    announce("linear rows per expert", T, kind)
    g = torch.Generator(device=DEV).manual_seed(T)
    # uneven: expert 0 gets twice its share, expert 3 none
    idx = torch.randint(0, 5, (T, 2), generator=g, device=DEV)
    idx = torch.where(idx >= 3, torch.where(idx == 3, 0, -1), idx)
    tr = kind == "transposed"
    for act in ("none", "geglu") if not tr else ("none",):
        lay, rows, x, w, g = make(gpu, T, 4, 2, 640, 704, fp8=kind == "fp8", transposed=tr, idx=idx)
        b = torch.randn((4, 704), generator=g, device=DEV).bfloat16()
        m = 352 if act == "geglu" else 704
        res = torch.randn((rows, m), generator=g, device=DEV).bfloat16()
        check(gpu, lay, rows, x, w, act, b, res, transposed=tr, checkpoint=True)


@pytest.mark.parametrize("T", [100, 260, 300, 400])
@pytest.mark.parametrize("kind,k", [("bf16", 8), ("bf16", 72), ("bf16", 640), ("fp8", 128), ("fp8", 640)])
def test_rows_per_expert_of_many_columns(gpu, T, kind, k):
    """As above with more 64 x 64 tiles than run at once: the larger tiles."""
    announce("linear rows per expert, many columns", T, kind, k)
    g = torch.Generator(device=DEV).manual_seed(T)
    idx = torch.randint(0, 5, (T, 2), generator=g, device=DEV)
    idx = torch.where(idx >= 3, torch.where(idx == 3, 0, -1), idx)
    for act, n in (("none", 8264), ("swiglu", 16448)):
        lay, rows, x, w, g = make(gpu, T, 4, 2, k, n, fp8=kind == "fp8", idx=idx)
        m = n // 2 if act == "swiglu" else n
        b = torch.randn((4, n), generator=g, device=DEV).bfloat16()
        res = torch.randn((rows, m), generator=g, device=DEV).bfloat16()
        check(gpu, lay, rows, x, w, act, b, res, checkpoint=n % 32 == 0)


@pytest.mark.parametrize("E", [1, 300, 700, 4096])
def test_many_experts_most_of_them_empty(gpu, E):
    announce("linear experts", E)
    lay, rows, x, w, _ = make(gpu, 100, E, 1, 64, 128)
    check(gpu, lay, rows, x, w)


def test_one_expert_takes_all(gpu):
    idx = torch.full((1000, 1), 5, device=DEV, dtype=torch.int64)
    lay, rows, x, w, _ = make(gpu, 1000, 16, 1, 192, 512, A=128, idx=idx)
    check(gpu, lay, rows, x, w, "swiglu", checkpoint=True)


def test_no_rows(gpu):
    """All slots without an expert, and a batch of no tokens: nothing is written."""
    idx = torch.full((20, 2), -1, device=DEV, dtype=torch.int64)
    lay, rows, x, w, _ = make(gpu, 20, 4, 2, 64, 64, A=8, idx=idx)
    check(gpu, lay, rows, x, w)
    lay = gpu.ep_get_layout(idx[:0], 4, 8)
    out, _ = gpu.ep_expert_linear(x[:0], w, lay)
    assert out.shape == (0, 64)


def test_fixed_capacity_overflow(gpu):
    """Experts with more pairs than their capacity: the rows they have."""
    idx = torch.zeros((300, 1), device=DEV, dtype=torch.int64)
    idx[200:] = 2
    lay, rows, x, w, _ = make(gpu, 300, 4, 1, 64, 96, A=1, idx=idx, capacity=128)
    assert lay.num_tokens_per_expert.tolist() == [200, 0, 100, 0]
    check(gpu, lay, rows, x, w)


def test_short_buffer_sets_the_overflow_bit(gpu):
    lay, rows, x, w, _ = make(gpu, 400, 4, 2, 64, 96)
    R = lay.num_recv_rows()
    short = R - 37
    guard = torch.full((R, 96), 7.0, device=DEV, dtype=torch.bfloat16)
    out, _ = gpu.ep_expert_linear(x[:short].contiguous(), w, lay, out=guard[:short])
    torch.cuda.synchronize()
    assert (guard[short:] == 7.0).all()
    for rs, z, dz, y, dy in ref.linear(x, w, None, "none", None, False, ref.spans(lay, short)):
        ref.assert_near(out[rs], y, dy)
    with pytest.raises(RuntimeError):
        lay.check()


def test_checkpoint_of_exact_values_is_the_cast(gpu):
    """Identity weights give z = x, so the checkpoint is ep_cast_fp8's, bit for bit."""
    E, k = 3, 256
    lay, rows, x, _, g = make(gpu, 500, E, 2, k, k)
    x = (x.float() * torch.exp2(torch.randint(-20, 20, (rows, 8), generator=g, device=DEV)
                                .float()).repeat_interleave(32, dim=1)).bfloat16()
    w = torch.eye(k, device=DEV).bfloat16().expand(E, k, k).contiguous()
    out, (codes, scales) = gpu.ep_expert_linear(x, w, lay, checkpoint=True)
    q, s = gpu.ep_cast_fp8(x, 32, scale_fmt="ue8m0")
    R = lay.num_recv_rows()
    assert torch.equal(out[:R], x[:R])
    assert torch.equal(codes[:R].view(torch.uint8), q[:R].view(torch.uint8))
    assert torch.equal(scales[:R], s[:R])


def test_infinities_stay_in_their_row(gpu):
    lay, rows, x, w, _ = make(gpu, 300, 2, 1, 128, 256)
    x[7, 5] = float("inf")
    x[9, 3] = float("nan")
    out, _ = gpu.ep_expert_linear(x, w, lay, activation="silu")
    R = lay.num_recv_rows()
    finite = torch.isfinite(out[:R].float()).all(dim=1)
    assert not finite[9] and finite.sum() >= R - 2
    assert torch.isnan(out[9].float()).all()


def test_same_bits_again_and_for_a_part_of_the_batch(gpu):
    """Two calls give the same bits, and an expert's rows do not depend on the others'."""
    lay, rows, x, w, _ = make(gpu, 1200, 4, 2, 320, 512)
    a, _ = gpu.ep_expert_linear(x, w, lay, activation="swiglu")
    b, _ = gpu.ep_expert_linear(x, w, lay, activation="swiglu")
    R = lay.num_recv_rows()
    assert torch.equal(a[:R].view(torch.int16), b[:R].view(torch.int16))
    o = lay.expert_offset.tolist()
    x2 = x.clone()
    x2[o[1]:] = 0
    c, _ = gpu.ep_expert_linear(x2, w, lay, activation="swiglu")
    assert torch.equal(a[:o[1]].view(torch.int16), c[:o[1]].view(torch.int16))


def test_other_streams_at_once(gpu):
    """Calls on two streams with their own buffers overlap freely."""
    jobs = [make(gpu, 800, 4, 2, 512, 512, seed=s) for s in (3, 4)]
    want = [gpu.ep_expert_linear(x, w, lay, activation="geglu")[0] for lay, _, x, w, _ in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [torch.zeros_like(v) for v in want]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o, (lay, _, x, w, _) in zip(streams, got, jobs):
            with torch.cuda.stream(s):
                gpu.ep_expert_linear(x, w, lay, activation="geglu", out=o)
    torch.cuda.synchronize()
    for g, v, (lay, *_) in zip(got, want, jobs):
        R = lay.num_recv_rows()
        assert torch.equal(g[:R].view(torch.int16), v[:R].view(torch.int16))


@pytest.mark.parametrize("T", [100, 260, 400])
@pytest.mark.parametrize("act,n", [("none", 8256), ("swiglu", 16512), ("silu", 64)])
@pytest.mark.parametrize("k", [128, 640])
def test_checkpoint_of_fp8_products_keeps_the_small_ones(gpu, T, act, n, k):
    """One product in 8 is some 2^14 times the others and cancels against the next 8
    channels' one: z is the sum of the small ones.  With a checkpoint the products
    are exact and their sum is off by no more than one of fp32 terms, in every tile."""
    announce("linear fp8 checkpoint, small products", T, act, n, k)
    E = 4
    idx = torch.arange(T, device=DEV).remainder(3).unsqueeze(1)
    lay = gpu.ep_get_layout(idx, E)
    rows = lay.max_recv_rows
    g = torch.Generator(device=DEV).manual_seed(T)

    def codes(shape, sign):
        v = torch.randint(8, 16, shape, generator=g, device=DEV).float() / 4      # 2 to 3.75
        v = v * torch.where(torch.rand(shape, generator=g, device=DEV) < 0.3, -1.0, 1.0)
        v[..., ::8] = 256.0
        if sign:
            v[..., 8::16] = -256.0
        return v.to(torch.float8_e4m3fn)

    def scales(shape):
        return torch.randint(118, 123, shape, generator=g, device=DEV, dtype=torch.uint8)

    x = (codes((rows, k), False), scales((rows, k // 128)))
    w = (codes((E, n, k), True), scales((E, n, k // 128)))
    b = torch.randn((E, n), generator=g, device=DEV).mul_(0.01).bfloat16()
    out, ck = gpu.ep_expert_linear(x, w, lay, bias=b, activation=act, checkpoint=True)
    xv, wv = ref.value(x), ref.value(w)
    for e, lo, hi in ref.spans(lay, rows):
        if lo == hi:
            continue
        z = xv[lo:hi] @ wv[e].T + b[e].double()
        dz = (k + 1) * ref.U * (xv[lo:hi].abs() @ wv[e].T.abs()) + 2 * ref.U * z.abs()
        ref.assert_checkpoint(ck[0][lo:hi], ck[1][lo:hi], z, dz)
        y, dy = ref.activate(z, act, dz)
        ref.assert_near(out[lo:hi], y, dy, what=f"rows {lo} to {hi}")
