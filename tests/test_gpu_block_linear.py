"""ep_cast_fp8_blocks and ep_block_linear against their definitions: exact codes
and scales; products over receive layouts and dense rows, activations, ragged and
empty experts, odd sizes, rows that hold NaN and no pair, scales far apart."""
import pytest
import torch

import block_ref as bref
import expert_ref as ref
from gpu_util import announce
from test_gpu_expert_linear import DEV, routing

pytestmark = pytest.mark.gpu


def cast_blocks_64(w):
    """Codes and scales from the definition: fp32 scale, fp32 quotient (both are
    rounded from 64 bits, which the two roundings do not show), nearest e4m3."""
    n, k = w.shape
    v = torch.nn.functional.pad(w.double(), (0, -k % 128, 0, -n % 128))
    t = v.view(-(-n // 128), 128, -(-k // 128), 128)
    top = t.abs().amax(dim=(1, 3)).clamp(min=float(torch.tensor(1e-4)))
    s = (top / 448).float()
    q = (t / s.double()[:, None, :, None]).float().view(v.shape)[:n, :k]
    return q.to(torch.float8_e4m3fn), s


@pytest.mark.parametrize("shape", [(8, 8), (128, 128), (1, 136, 264), (3, 384, 256), (2, 1000, 1408),
                                   (0, 64, 64), (5, 120, 8), (1, 8, 2056)])
def test_cast(gpu, shape):
    announce("cast blocks", shape)
    g = torch.Generator(device=DEV).manual_seed(sum(shape))
    w = torch.randn(shape, generator=g, device=DEV)
    # blocks of very different sizes, one of zeros, one under the floor
    w = (w * torch.exp2(torch.randint(-20, 20, (*shape[:-1], 1), generator=g, device=DEV).float())).bfloat16()
    if w.numel():
        w.view(-1, *shape[-2:])[0, :128, :128] *= 0
        w.view(-1, *shape[-2:])[-1, -8:, -8:] = -1e-6
    (c, s), (ct, st) = gpu.ep_cast_fp8_blocks(w, transposed=True)
    only, none = gpu.ep_cast_fp8_blocks(w)
    assert none is None and torch.equal(only[0].view(torch.uint8), c.view(torch.uint8))
    assert torch.equal(only[1], s) and c.shape == w.shape
    assert torch.equal(ct.view(torch.uint8), c.view(torch.uint8).transpose(-1, -2))
    assert torch.equal(st, s.transpose(-1, -2))
    for i, m in enumerate(w.view(-1, *shape[-2:])):
        wc, ws = cast_blocks_64(m)
        assert torch.equal(s.view(-1, *s.shape[-2:])[i], ws)
        assert torch.equal(c.view(-1, *shape[-2:])[i].view(torch.uint8), wc.view(torch.uint8))


def test_cast_into_buffers_on_a_stream(gpu):
    announce("cast blocks, buffers")
    w = torch.randn((2, 72, 200), device=DEV).bfloat16()
    want = gpu.ep_cast_fp8_blocks(w, transposed=True)
    bufs = [torch.empty_like(t) for pair in want for t in pair]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = gpu.ep_cast_fp8_blocks(w, transposed=True, out=bufs)
    side.synchronize()
    assert got[0][0] is bufs[0] and got[1][1] is bufs[3]
    for a, b in zip(bufs, [t for pair in want for t in pair]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    with pytest.raises(ValueError):
        gpu.ep_cast_fp8_blocks(w, transposed=True, out=bufs[:2])
    with pytest.raises(gpu.EpError):
        gpu.ep_cast_fp8_blocks(w[:, :, :196].contiguous())


def test_cast_of_infinities_and_nan(gpu):
    """NaN keeps to itself; a block that holds an infinity has a NaN scale and NaN codes."""
    announce("cast blocks, non-finite")
    w = torch.randn((256, 256), device=DEV).bfloat16()
    want, _ = gpu.ep_cast_fp8_blocks(w)
    w[3, 5] = float("nan")
    w[200, 130] = float("-inf")
    (c, s), (ct, st) = gpu.ep_cast_fp8_blocks(w, transposed=True)
    top = w[:128, :128].double().nan_to_num(0.0).abs().max()
    assert s[0, 0].item() == (top / 448).float().item()
    assert torch.equal(s[0, 1], want[1][0, 1]) and torch.equal(s[1, 0], want[1][1, 0]) and s[1, 1].isnan()
    nan = c.float().isnan()
    assert nan[3, 5] and nan[128:, 128:].all() and int(nan.sum()) == 1 + 128 * 128
    assert torch.equal(ct.view(torch.uint8), c.view(torch.uint8).T) and torch.equal(st.view(torch.int32), s.view(torch.int32).T)


def rows(g, n, k):
    x = torch.randn((n, k), generator=g, device=DEV)
    x = x * torch.exp2(torch.randint(-3, 4, (n, k // 128), generator=g, device=DEV).float()).repeat_interleave(128, dim=1)
    return x.bfloat16()


def weights(g, shape):
    n, k = shape[-2:]
    w = torch.randn(shape, generator=g, device=DEV) * k ** -0.5
    w = w * torch.exp2(torch.randint(-2, 3, (*shape[:-1], k // 128), generator=g, device=DEV).float()).repeat_interleave(128, dim=-1)
    return w.bfloat16()


def check(gpu, x, w, lay=None, act="none", bias=None, residual=None):
    """Rows without a pair hold NaN codes and scales, and none of theirs changes."""
    n, m = x[0].shape[0], w[0].shape[-2] // (2 if ref.gated(act) else 1)
    sp = [(None, 0, n)] if lay is None else ref.spans(lay, n)
    held = torch.zeros(n, dtype=torch.bool, device=DEV)
    for _, a, b in sp:
        held[a:b] = True
    x[0].view(torch.uint8)[~held] = 0x7F
    x[1][~held] = float("nan")
    out = torch.full((n + 3, m), 7.0, device=DEV, dtype=torch.bfloat16)
    got = gpu.ep_block_linear(x, w, lay, bias=bias, activation=act, residual=residual, out=out)
    torch.cuda.synchronize()
    assert got is out and (out[n:] == 7.0).all() and (out[:n][~held] == 7.0).all()
    for rs, y, dy in bref.block_linear(x, w, bias, act, residual, sp):
        ref.assert_near(out[rs], y, dy, what=f"rows {rs}")
    return out


def case(gpu, T, E, K, k, n, act="none", A=1, seed=0, bias=False, residual=False, idx=None, **kw):
    announce("block linear", T, E, K, k, n, act, A, bias, residual)
    g = torch.Generator(device=DEV).manual_seed(seed)
    lay, lead, have = None, (), T
    if E:
        lay = gpu.ep_get_layout(routing(T, E, K, seed) if idx is None else idx, E, A, **kw)
        lead, have = (E,), lay.max_recv_rows
    x = gpu.ep_cast_fp8(rows(g, have, k), 128)
    w, _ = gpu.ep_cast_fp8_blocks(weights(g, (*lead, n, k)))
    m = n // 2 if ref.gated(act) else n
    b = torch.randn((*lead, n), generator=g, device=DEV).bfloat16() if bias else None
    r = torch.randn((have, m), generator=g, device=DEV).bfloat16() if residual else None
    check(gpu, x, w, lay, act, b, r)


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "swiglu", "geglu"])
@pytest.mark.parametrize("T,E,K,k,n", [(1, 0, 1, 256, 192), (40, 0, 1, 640, 320), (64, 8, 2, 256, 512),
                                       (700, 3, 2, 384, 704)])
def test_activations_bias_residual(gpu, act, T, E, K, k, n):
    case(gpu, T, E, K, k, n, act, bias=True, residual=True, seed=T)


# every row count's kernel: few rows (three groups), tiles of 64, 128, 192 and 256
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256,
                               257, 513])
@pytest.mark.parametrize("n,k,act", [(4096, 128, "swiglu"), (4104, 1152, "none")])
def test_dense_rows(gpu, T, n, k, act):
    case(gpu, T, 0, 1, k, n, act, seed=T)


@pytest.mark.parametrize("T,k,n,act", [(100, 7168, 512, "swiglu"), (300, 4096, 1032, "none"), (130, 7168, 4096, "swiglu"),
                                       (1000, 2688, 1024, "silu"), (700, 4224, 4096, "geglu"), (65, 5248, 8, "none"),
                                       (512, 7168, 2048, "swiglu"), (512, 7168, 2056, "gelu"), (1024, 4096, 2560, "none"),
                                       (640, 256, 3392, "geglu"), (640, 256, 3400, "none")])
def test_dense_rows_in_parts(gpu, T, k, n, act):
    """Contractions cut into parts, some within a group of four blocks; and whole ones in
    the tiles between."""
    case(gpu, T, 0, 1, k, n, act, bias=True, residual=True, seed=T)


@pytest.mark.parametrize("n,act", [(8, "none"), (24, "none"), (64, "swiglu"), (136, "silu"), (192, "geglu"),
                                   (320, "swiglu"), (1000, "none")])
@pytest.mark.parametrize("T,E", [(3, 0), (100, 0), (300, 4), (2000, 2)])
def test_narrow_and_odd_columns(gpu, n, act, T, E):
    case(gpu, T, E, 1, 384, n, act, seed=n)


@pytest.mark.parametrize("blocks", [1, 2, 3, 4, 5, 6, 7, 8, 9, 13])
@pytest.mark.parametrize("T,E,n", [(5, 0, 128), (200, 2, 256), (300, 2, 4352), (900, 2, 4096)])
def test_contractions_of_few_blocks(gpu, blocks, T, E, n):
    """The rings of steps and of scales at their ends."""
    case(gpu, T, E, 1, 128 * blocks, n, seed=blocks)


@pytest.mark.parametrize("A", [1, 16, 128])
def test_ragged_experts(gpu, A):
    """Experts of no, one and many rows; large enough for tiles of 256 rows."""
    counts = [0, 1, 0, 63, 257, 700, 1200, 3]
    idx = torch.cat([torch.full((c,), e, dtype=torch.int64) for e, c in enumerate(counts)])
    idx = idx[torch.randperm(len(idx), generator=torch.Generator().manual_seed(A))].unsqueeze(1).to(DEV)
    case(gpu, len(idx), len(counts), 1, 640, 4416, "swiglu", A=A, idx=idx, seed=A)


@pytest.mark.parametrize("E,T", [(32, 1600), (16, 1200), (8, 900)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_rows_per_expert(gpu, E, T, act):
    """About 100, 150 and 225 rows an expert of many columns: tiles of 128, 192 and 256 rows."""
    case(gpu, T, E, 2, 896, 4096, act, seed=E, residual=True)


def test_fixed_capacity(gpu):
    idx = torch.zeros((90, 1), dtype=torch.int64, device=DEV)
    idx[60:] = 2
    case(gpu, 90, 4, 1, 256, 256, idx=idx, capacity=32)


def test_no_rows(gpu):
    announce("block linear, no rows")
    g = torch.Generator(device=DEV).manual_seed(0)
    w, _ = gpu.ep_cast_fp8_blocks(weights(g, (64, 128)))
    x = gpu.ep_cast_fp8(rows(g, 0, 128), 128)
    assert gpu.ep_block_linear(x, w).shape == (0, 64)
    w, _ = gpu.ep_cast_fp8_blocks(weights(g, (3, 64, 128)))
    lay = gpu.ep_get_layout(torch.full((20, 2), -1, dtype=torch.int64, device=DEV), 3)
    x = gpu.ep_cast_fp8(rows(g, lay.max_recv_rows, 128), 128)
    check(gpu, x, w, lay)


def test_short_buffer_sets_the_overflow_bit(gpu):
    announce("block linear, short buffer")
    g = torch.Generator(device=DEV).manual_seed(1)
    lay = gpu.ep_get_layout(torch.zeros((300, 1), dtype=torch.int64, device=DEV), 2)
    w, _ = gpu.ep_cast_fp8_blocks(weights(g, (2, 192, 256)))
    check(gpu, gpu.ep_cast_fp8(rows(g, 211, 256), 128), w, lay)
    with pytest.raises(RuntimeError):
        lay.check()


@pytest.mark.parametrize("T", [20, 200])
def test_scales_far_apart_and_not_powers_of_two(gpu, T):
    """Blocks whose scales span the exponents: only a sum in which each block has its
    own scale meets the bound."""
    announce("block linear, scales", T)
    g = torch.Generator(device=DEV).manual_seed(T)
    k, n = 1024, 384

    def codes(shape):
        return torch.randn(shape, generator=g, device=DEV).mul_(90).clamp_(-448, 448).to(torch.float8_e4m3fn)

    def scales(shape, span):
        e = torch.randint(-span, span + 1, shape, generator=g, device=DEV).float()
        return torch.exp2(e) * (1 + torch.rand(shape, generator=g, device=DEV))

    check(gpu, (codes((T, k)), scales((T, k // 128), 30)), (codes((n, k)), scales((3, k // 128), 20)))


@pytest.mark.parametrize("T", [9, 150, 600])
def test_infinities_and_nan_stay_in_their_row(gpu, T):
    announce("block linear, non-finite", T)
    g = torch.Generator(device=DEV).manual_seed(T)
    x = gpu.ep_cast_fp8(rows(g, T, 512), 128)
    w, _ = gpu.ep_cast_fp8_blocks(weights(g, (640, 512)))
    want = gpu.ep_block_linear(x, w)
    x[0].view(torch.uint8)[3, 77] = 0x7F
    x[1][5, 2] = float("inf")
    out = gpu.ep_block_linear(x, w)
    assert out[3].isnan().all() and (~out[5].isfinite()).all()
    keep = torch.arange(T, device=DEV)
    keep = keep[(keep != 3) & (keep != 5)]
    assert torch.equal(out[keep], want[keep])


def test_same_bits_again_and_whatever_the_other_rows_hold(gpu):
    announce("block linear, same bits")
    g = torch.Generator(device=DEV).manual_seed(2)
    w, _ = gpu.ep_cast_fp8_blocks(weights(g, (704, 640)))
    for T in (30, 300):
        x = rows(g, T, 640)
        a = gpu.ep_block_linear(gpu.ep_cast_fp8(x, 128), w, activation="swiglu")
        assert torch.equal(a, gpu.ep_block_linear(gpu.ep_cast_fp8(x, 128), w, activation="swiglu"))
        x[T // 2:] = 5.0
        b = gpu.ep_block_linear(gpu.ep_cast_fp8(x, 128), w, activation="swiglu")
        assert torch.equal(a[:T // 2], b[:T // 2])


def test_residual_in_place_and_pow2_scales(gpu):
    announce("block linear, residual in place")
    g = torch.Generator(device=DEV).manual_seed(3)
    for T in (50, 700):
        x = gpu.ep_cast_fp8(rows(g, T, 256), 128, scale_fmt="pow2")
        w, _ = gpu.ep_cast_fp8_blocks(weights(g, (320, 256)))
        r = torch.randn((T, 320), generator=g, device=DEV).bfloat16()
        want = gpu.ep_block_linear(x, w, residual=r)
        assert torch.equal(gpu.ep_block_linear(x, w, residual=r, out=r), want)
        check(gpu, x, w)


def test_binding_checks(gpu):
    announce("block linear, binding")
    g = torch.Generator(device=DEV).manual_seed(4)
    x = gpu.ep_cast_fp8(rows(g, 10, 256), 128)
    w, _ = gpu.ep_cast_fp8_blocks(weights(g, (64, 256)))
    wl, _ = gpu.ep_cast_fp8_blocks(weights(g, (3, 64, 256)))
    lay = gpu.ep_get_layout(routing(5, 3, 2, 0), 3)
    ue = gpu.ep_cast_fp8(rows(g, 10, 256), 128, scale_fmt="ue8m0")
    for bad in (lambda: gpu.ep_block_linear(ue, w), lambda: gpu.ep_block_linear(x, wl),
                lambda: gpu.ep_block_linear(x, w, lay),
                lambda: gpu.ep_block_linear(x, (w[0], w[1][:, :1].contiguous())),
                lambda: gpu.ep_block_linear((x[0], x[1][:9]), w),
                lambda: gpu.ep_block_linear((x[0], x[1].double()), w),
                lambda: gpu.ep_block_linear(x, w, out=torch.empty((9, 64), device=DEV, dtype=torch.bfloat16)),
                lambda: gpu.ep_block_linear(x, w, bias=torch.zeros(63, device=DEV, dtype=torch.bfloat16)),
                lambda: gpu.ep_block_linear((x[0][:, :192].contiguous(), x[1]), w)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gpu.EpError):                       # halves of 48
        w96, _ = gpu.ep_cast_fp8_blocks(weights(g, (96, 256)))
        gpu.ep_block_linear(x, w96, activation="swiglu")


def test_offsets_past_32_bits(gpu):
    """4.4 million dense rows of 512 codes: rows around byte 2^31 of x and 2^31 and 2^32 of
    out, the first and the last ones."""
    T, k, n = 4_400_000, 512, 512
    announce("block linear", T, n, k)
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.empty(T, k, device=DEV, dtype=torch.bfloat16).normal_(generator=g).to(torch.float8_e4m3fn)
    xs = torch.rand(T, k // 128, generator=g, device=DEV) + 0.5
    w, _ = gpu.ep_cast_fp8_blocks(torch.randn(n, k, generator=g, device=DEV).to(torch.bfloat16))
    out = gpu.ep_block_linear((x, xs), w)
    at = torch.cat([torch.arange(b - 40, b + 40, device=DEV) for b in (40, 1 << 21, 1 << 22, T - 40)])
    some = (x.view(torch.uint8)[at].view(torch.float8_e4m3fn), xs[at])
    for rows, y, dy in bref.block_linear(some, w, None, "none", None, [(None, 0, len(at))]):
        ref.assert_near(out[at][rows], y, dy)
