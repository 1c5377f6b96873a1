"""The block-scaled product, its weights' cast and the gated feed-forward block
refuse bad arguments on the host, before any GPU work (no compute calls; pointers
are never dereferenced)."""
import ctypes
import os

import pytest

from combine_ep_get_layout_amd import _abi, build
from test_expert_abi import PTRS, _params
from test_expert_copies import assembly, check_waits

V = ctypes.c_void_p
INV, UNS, OK, WS = (_abi.EP_ERR_INVALID_ARG, _abi.EP_ERR_UNSUPPORTED, _abi.EP_OK,
                    _abi.EP_ERR_WORKSPACE)
SWIGLU, GELU = _abi.EP_ACT_SWIGLU, _abi.EP_ACT_GELU


def cast(w=16, num=2, n=64, k=64, c=16, s=16, ct=None, st=None):
    return _abi.load().ep_cast_fp8_blocks(V(w), num, n, k, V(c), V(s), V(ct), V(st), None)


@pytest.mark.parametrize("kw,code", [
    (dict(num=-1), INV), (dict(n=0), INV), (dict(n=12), INV), (dict(k=4), INV), (dict(k=-8), INV),
    (dict(w=None), INV), (dict(w=8), INV), (dict(c=None), INV), (dict(s=None), INV),
    (dict(c=None, s=None), INV), (dict(ct=16), INV), (dict(st=16), INV), (dict(c=4), INV),
    (dict(s=2), INV), (dict(ct=4, st=16), INV), (dict(ct=16, st=18), INV),
    (dict(n=(1 << 20) + 8), UNS), (dict(k=(1 << 20) + 8), UNS),
    (dict(num=64, n=1 << 20, k=1 << 20), UNS),
    (dict(num=0, w=None, c=None, s=None), OK),
])
def test_cast(kw, code):
    assert cast(**kw) == code


def linear(x=16, xs=16, w=16, ws=16, n=64, k=128, b=None, act=0, res=None, p=None, lay=None,
           rows=32, wk=None, nb=0, out=16):
    return _abi.load().ep_block_linear(V(x), V(xs), V(w), V(ws), n, k, V(b), act, V(res),
                                       None if p is None else ctypes.byref(p),
                                       None if lay is None else ctypes.byref(lay), rows, V(wk), nb,
                                       V(out), None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=60), INV), (dict(n=0), INV), (dict(k=0), INV), (dict(k=64), INV), (dict(k=192), INV),
    (dict(n=96, act=SWIGLU), INV), (dict(act=5), INV), (dict(act=-1), INV),
    (dict(x=8), INV), (dict(x=None), INV), (dict(xs=None), INV), (dict(xs=18), INV),
    (dict(w=8), INV), (dict(w=None), INV), (dict(ws=None), INV), (dict(ws=18), INV),
    (dict(out=None), INV), (dict(out=8), INV), (dict(b=8), INV), (dict(res=8), INV),
    (dict(rows=-1), INV), (dict(rows=1 << 31), INV),
    (dict(p=_params()), INV), (dict(lay=PTRS), INV),                # one without the other
    (dict(p=_params(P=2, PM=1), lay=PTRS), INV),                    # rows by partition
    (dict(p=_params(), lay=_abi.LayoutPtrs(None, *([16] * 6))), INV),
    (dict(p=_params(), lay=PTRS, rows=-1), INV),
    (dict(n=(1 << 20) + 8), UNS), (dict(k=(1 << 20) + 128), UNS), (dict(n=1 << 20, k=1 << 11), UNS),
    (dict(rows=100, k=8192), WS), (dict(rows=100, k=8192, wk=8, nb=1 << 30), WS),
    (dict(rows=100, k=8192, wk=16, nb=100 * 64 * 4), WS),
    (dict(rows=0, x=None, xs=None, w=None, ws=None, out=None), OK),
    (dict(p=_params(T=0), lay=PTRS, x=None, out=None), OK),
])
def test_linear(kw, code):
    assert linear(**kw) == code


def ffn(x=16, T=4, H=64, I=32, w1=16, w2=16, act=SWIGLU, res=None, z=None, ws=16, nb=1 << 20,
        out=16):
    return _abi.load().ep_gated_ffn(V(x), T, H, I, V(w1), V(w2), act, V(res), V(z), V(ws), nb,
                                    V(out), None)


SIZES = [(dict(T=-1), INV), (dict(T=1 << 31), INV), (dict(H=0), INV), (dict(H=60), INV),
         (dict(I=0), INV), (dict(I=12), INV), (dict(act=0), INV), (dict(act=GELU), INV),
         (dict(act=9), INV), (dict(H=(1 << 20) + 8), UNS), (dict(I=(1 << 19) + 8), UNS),
         (dict(H=1 << 15, I=1 << 14), UNS)]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(x=None), INV), (dict(x=8), INV), (dict(w1=None), INV), (dict(w1=8), INV),
    (dict(w2=None), INV), (dict(w2=8), INV), (dict(res=8), INV), (dict(z=8), INV),
    (dict(out=None), INV), (dict(out=8), INV), (dict(ws=None), WS), (dict(ws=8), WS),
    (dict(nb=16), WS), (dict(T=0, x=None, w1=None, w2=None, ws=None, out=None), OK),
])
def test_ffn(kw, code):
    assert ffn(**kw) == code


def ffn_backward(dout=16, x=16, z=16, T=4, H=64, I=32, w1=16, w2=16, act=SWIGLU, i1=None, i2=None,
                 ws=16, nb=1 << 20, dx=16, d1=16, d2=16, bf=0):
    return _abi.load().ep_gated_ffn_backward(V(dout), V(x), V(z), T, H, I, V(w1), V(w2), act, V(i1),
                                             V(i2), V(ws), nb, V(dx), V(d1), V(d2), bf, None)


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(dout=None), INV), (dict(dout=8), INV), (dict(x=None), INV), (dict(x=8), INV),
    (dict(z=None), INV), (dict(z=8), INV), (dict(w1=None), INV), (dict(w2=None), INV),
    (dict(w1=8), INV), (dict(w2=8), INV), (dict(i1=8), INV), (dict(i2=8), INV), (dict(dx=8), INV),
    (dict(d1=None), INV), (dict(d2=None), INV), (dict(d1=8), INV), (dict(d2=8), INV),
    (dict(bf=2), INV), (dict(ws=None), WS), (dict(ws=8), WS), (dict(nb=16), WS),
])
def test_ffn_backward(kw, code):
    assert ffn_backward(**kw) == code


def test_workspaces():
    f = _abi.load().ep_gated_ffn_workspace_bytes
    for T, H, inter in [(1, 64, 8), (7, 128, 1408), (128, 7168, 2048), (1 << 20, 4096, 4096)]:
        assert f(T, H, inter, 0) >= 2 * T * inter and f(T, H, inter, 1) >= 6 * T * inter
    assert f(0, 8, 8, 0) > 0
    assert ffn(T=7, I=1408, nb=2 * 7 * 1408 - 1) == WS
    assert ffn_backward(T=7, I=1408, nb=6 * 7 * 1408 - 1) == WS
    assert f(-1, 8, 8, 0) == f(1, 8, 0, 0) == f(1, 0, 8, 0) == f(1, 8, 8, 2) == f(1 << 31, 8, 8, 0) == 0
    assert f(1, 8, (1 << 19) + 8, 0) == 0
    g = _abi.load().ep_block_linear_workspace_bytes
    assert g(100, 64, 8192) >= 2 * 100 * 64 * 4 and g(0, 64, 128) == g(100000, 4096, 128) == 0
    assert g(-1, 64, 128) == g(100, 0, 128) == g(100, 64, 0) == g(1 << 31, 64, 128) == 0


# the kernels' 32-bit counts of rows run up to a tile and a ring of steps behind the last
MOST = (1 << 31) - 1024


def test_rows_that_would_pass_the_kernels_counts():
    for rows in (MOST + 1, (1 << 31) - 1):
        assert linear(rows=rows, nb=1 << 60) == INV
        assert ffn(T=rows, nb=1 << 60) == INV
        assert ffn_backward(T=rows, nb=1 << 60) == INV
        assert _abi.load().ep_gated_ffn_workspace_bytes(rows, 8, 8, 0) == 0
        assert _abi.load().ep_block_linear_workspace_bytes(rows, 64, 8192) == 0
    # taken up to there (refused here for its workspace alone, so nothing is launched)
    assert ffn(T=MOST, nb=0) == ffn_backward(T=MOST, nb=0) == WS
    assert _abi.load().ep_gated_ffn_workspace_bytes(MOST, 8, 8, 1) >= 6 * MOST * 8


def test_binding_refuses():
    import torch

    import combine_ep_get_layout_amd as ep
    bf = torch.zeros((8, 128), dtype=torch.bfloat16)
    q = (torch.zeros((8, 128), dtype=torch.uint8), torch.zeros((8, 1)))
    with pytest.raises(ValueError, match="GPU tensor"):
        ep.ep_cast_fp8_blocks(bf)
    with pytest.raises(ValueError, match="GPU tensor"):
        ep.ep_block_linear(q, q)
    with pytest.raises(ValueError, match="codes, float32 scales"):
        ep.ep_block_linear(bf, q)
    with pytest.raises(ValueError, match="activation must be one of"):
        ep.ep_block_linear(q, q, activation="tanh")
    with pytest.raises(ValueError, match="GPU tensor"):
        ep.ep_gated_ffn(bf, bf, bf)
    for act in ("gelu", "none"):
        with pytest.raises(ValueError, match="swiglu"):
            ep.ep_gated_ffn(bf, bf, bf, activation=act)
    with pytest.raises(ValueError, match="GPU tensor"):
        ep.ep_gated_ffn_backward(bf, bf, bf, bf, bf)
    with pytest.raises(ValueError, match="dtype"):
        ep.ep_gated_ffn_backward(bf, bf, bf, bf, bf, dtype=torch.float16)


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")
@pytest.mark.parametrize("name", ["ep_block_linear", "ep_ffn"])
def test_copies_into_lds_wait_for_their_scalars(name, tmp_path):
    code = assembly(os.path.join(build.CSRC, name + ".hip"), tmp_path / "kernels.s")
    assert sum(check_waits(c) for c in code.values()) >= 100
