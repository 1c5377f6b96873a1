"""The expert entry points refuse bad arguments on the host, before any GPU
work (no compute calls; pointers are never dereferenced)."""
import ctypes

import pytest

from combine_ep_get_layout_amd import _abi

V = ctypes.c_void_p
INV, UNS, OK, WS = (_abi.EP_ERR_INVALID_ARG, _abi.EP_ERR_UNSUPPORTED, _abi.EP_OK,
                    _abi.EP_ERR_WORKSPACE)
BF, F8, UE = _abi.EP_DTYPE_BF16, _abi.EP_DTYPE_FP8_E4M3, _abi.EP_DTYPE_FP8_E4M3_UE8M0
PTRS = _abi.LayoutPtrs(*([16] * 7))


def _params(T=16, K=2, E=8, **kw):
    p = _abi.LayoutParams(num_tokens=T, num_topk=K, num_experts=E, expert_alignment=1,
                          num_partitions=kw.get("P", 1), partition_major=kw.get("PM", 0))
    p.max_recv_rows = max(0, T * K)
    return p


def linear(p=None, lay=PTRS, x=16, xd=BF, xs=None, w=16, ws=None, n=64, k=64, tr=0, b=None, act=0,
           res=None, rows=32, out=16, ck=None, cs=None):
    return _abi.load().ep_expert_linear(V(x), xd, V(xs), V(w), V(ws), n, k, tr, V(b), act, V(res),
                                        ctypes.byref(p or _params()),
                                        None if lay is None else ctypes.byref(lay), rows, V(out),
                                        V(ck), V(cs), None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=60), INV), (dict(k=60), INV), (dict(n=0), INV), (dict(k=-8), INV),
    (dict(n=24, act=_abi.EP_ACT_SWIGLU), INV),          # halves of 12
    (dict(act=5), INV), (dict(act=-1), INV), (dict(tr=2), INV),
    (dict(xd=F8, xs=16, ws=16, k=128), INV),            # fp32 scales
    (dict(xd=UE, xs=16, ws=16, k=192), INV),            # k not a multiple of the scale group
    (dict(xd=UE, ws=16, k=128), INV), (dict(xd=UE, xs=16, k=128), INV),   # scales missing
    (dict(xd=UE, xs=16, ws=16, k=128, tr=1), UNS),
    (dict(x=24), INV), (dict(w=8), INV), (dict(out=4), INV), (dict(b=4), INV), (dict(res=4), INV),
    (dict(x=None), INV), (dict(w=None), INV), (dict(out=None), INV),
    (dict(ck=16), INV), (dict(cs=16), INV), (dict(ck=18, cs=16), INV),
    (dict(ck=16, cs=16, n=40), INV), (dict(ck=16, cs=16, n=96, act=_abi.EP_ACT_GEGLU), INV),
    (dict(rows=-1), INV), (dict(rows=1 << 31), INV), (dict(lay=None), INV),
    (dict(lay=_abi.LayoutPtrs(None, *([16] * 6))), INV),
    (dict(lay=_abi.LayoutPtrs(16, None, *([16] * 5))), INV),
    (dict(lay=_abi.LayoutPtrs(*([16] * 6), None)), INV),
    (dict(p=_params(P=2, PM=1)), INV),                  # rows by partition
    (dict(p=_params(T=-1)), INV),
    (dict(n=1 << 20, k=1 << 11), UNS), (dict(n=(1 << 20) + 8), UNS), (dict(k=(1 << 20) + 8), UNS),
    (dict(p=_params(T=0), x=None, w=None, out=None), OK),
    (dict(rows=0, x=None, out=None), OK),
])
def test_linear(kw, code):
    assert linear(**kw) == code


def wgrad(p=None, lay=PTRS, dy=16, x=16, xd=BF, xs=None, n=64, k=64, rows=32, dw0=None, db0=None,
          dw=16, bf=0, db=None):
    return _abi.load().ep_expert_wgrad(V(dy), V(x), xd, V(xs), n, k, ctypes.byref(p or _params()),
                                       ctypes.byref(lay), rows, V(dw0), V(db0), V(dw), bf, V(db),
                                       None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=12), INV), (dict(k=12), INV), (dict(xd=UE, xs=16, k=64), INV), (dict(xd=UE, k=128), INV),
    (dict(xd=F8, xs=16, k=128), INV), (dict(bf=2), INV), (dict(db0=16), INV), (dict(dw=None), INV),
    (dict(dw=8), INV), (dict(dw0=8), INV), (dict(db=18), INV), (dict(dy=8), INV), (dict(x=8), INV),
    (dict(dy=None), INV), (dict(rows=-1), INV), (dict(p=_params(P=2, PM=1)), INV),
    (dict(n=(1 << 20) + 8), UNS),
])
def test_wgrad(kw, code):
    assert wgrad(**kw) == code


def act_backward(p=None, lay=PTRS, dh=16, pre=16, ps=None, n=64, act=1, w=None, rows=32, dpre=16,
                 h=16, dw=16):
    return _abi.load().ep_expert_activation_backward(
        V(dh), V(pre), V(ps), n, act, V(w), ctypes.byref(p or _params()), ctypes.byref(lay), rows,
        V(dpre), V(h), V(dw), None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=12), INV), (dict(n=40, ps=16), INV), (dict(n=96, ps=16, act=3), INV),
    (dict(n=24, act=4), INV), (dict(act=9), INV), (dict(dh=8), INV), (dict(pre=8), INV),
    (dict(pre=4, ps=16), INV), (dict(dpre=8), INV), (dict(h=8), INV), (dict(dw=18), INV),
    (dict(w=18), INV), (dict(dh=None), INV), (dict(pre=None), INV), (dict(dpre=None), INV),
    (dict(rows=-1), INV), (dict(n=(1 << 20) + 64), UNS), (dict(p=_params(P=2, PM=1)), INV),
    (dict(lay=_abi.LayoutPtrs(*([16] * 5), None, 16)), INV),     # no src_of_slot
    (dict(rows=0, dh=None, pre=None, dpre=None), OK),
    (dict(p=_params(T=0), dh=None, pre=None, dpre=None), OK),
])
def test_activation_backward(kw, code):
    assert act_backward(**kw) == code


def decode(x=16, idx=16, w=None, T=4, K=2, E=8, H=128, I=128, wd=BF, w1=16, s1=None, b1=None, w2=16,
           s2=None, b2=None, act=3, r0=None, r1=None, ws=16, nb=1 << 20, st=None, out=16):
    return _abi.load().ep_moe_decode(V(x), V(idx), V(w), T, K, E, H, I, wd, V(w1), V(s1), V(b1),
                                     V(w2), V(s2), V(b2), act, V(r0), V(r1), V(ws), nb, V(st),
                                     V(out), None)


@pytest.mark.parametrize("kw,code", [
    (dict(H=12), INV), (dict(I=12), INV), (dict(T=-1), INV), (dict(K=0), INV), (dict(E=0), INV),
    (dict(act=7), INV), (dict(wd=F8, s1=16, s2=16), INV), (dict(wd=UE, s1=16, s2=16, H=192), INV),
    (dict(wd=UE, s1=16, s2=16, I=64), INV), (dict(wd=UE, s1=16), INV), (dict(wd=UE, s2=16), INV),
    (dict(T=1025, K=1), UNS), (dict(T=300, K=4), UNS), (dict(E=4097), UNS),
    (dict(H=(1 << 20) + 128), UNS), (dict(I=(1 << 20) + 128), UNS),
    (dict(x=8), INV), (dict(x=None), INV), (dict(idx=None), INV), (dict(idx=4), INV),
    (dict(w=18), INV), (dict(w1=8), INV), (dict(w2=None), INV), (dict(b1=17), INV),
    (dict(r0=8), INV), (dict(r1=8), INV), (dict(st=18), INV), (dict(out=8), INV),
    (dict(ws=None), WS), (dict(ws=8), WS), (dict(nb=16), WS),
    (dict(T=0, x=None, idx=None, w1=None, w2=None, out=None, ws=None), OK),
])
def test_decode(kw, code):
    assert decode(**kw) == code


def test_decode_workspace():
    f = _abi.load().ep_moe_decode_workspace_bytes
    assert f(4, 2, 128) >= 4 * 2 * 128 * 2 and f(0, 1, 8) > 0
    assert f(1025, 1, 128) == 0 and f(-1, 1, 128) == 0 and f(1, 0, 128) == 0 and f(1, 1, 0) == 0


def test_binding_refuses_host_tensors():
    import torch

    import combine_ep_get_layout_amd as ep
    p = _params(4, 2, 4)
    lay = ep.Layout(p, torch.device("cpu"))
    x = torch.zeros((8, 64), dtype=torch.bfloat16)
    w = torch.zeros((4, 64, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ep.ep_expert_linear(x, w, lay)
    with pytest.raises(ValueError):
        ep.ep_expert_linear(x, w, lay, activation="tanh")
    with pytest.raises(ValueError):
        ep.ep_expert_wgrad(x, x, lay)
    with pytest.raises(ValueError):
        ep.ep_expert_activation_backward(x, x, lay)
    with pytest.raises(ValueError):
        ep.ep_moe_decode(x, torch.zeros((8, 2), dtype=torch.int64), None, w, w)


def test_decode_workspace_holds_both_parts_of_h():
    """Two bf16 parts an element; sizes whose rounding up cannot hide a missing part."""
    f = _abi.load().ep_moe_decode_workspace_bytes
    for T, K, inter in [(1, 1, 256), (1, 1, 1000), (4, 2, 128), (7, 3, 1408), (128, 8, 2048),
                        (1024, 1, 1 << 20)]:
        assert f(T, K, inter) >= 4 * T * K * inter
        assert decode(T=T, K=K, I=inter // 8 * 8, nb=4 * T * K * (inter // 8 * 8) - 1) in (WS, UNS)


def test_binding_names_the_activation_it_does_not_know():
    import torch

    import combine_ep_get_layout_amd as ep
    lay = ep.Layout(_params(4, 2, 4), torch.device("cpu"))
    x = torch.zeros((8, 64), dtype=torch.bfloat16)
    w = torch.zeros((4, 64, 64), dtype=torch.bfloat16)
    idx = torch.zeros((8, 2), dtype=torch.int64)
    for call in (lambda: ep.ep_expert_linear(x, w, lay, activation="tanh"),
                 lambda: ep.ep_expert_activation_backward(x, x, lay, activation="tanh"),
                 lambda: ep.ep_moe_decode(x, idx, None, w, w, activation="tanh")):
        with pytest.raises(ValueError, match="activation must be one of"):
            call()
    # known names get past that check, to the tensors
    with pytest.raises(ValueError, match="GPU tensor"):
        ep.ep_expert_linear(x, w, lay, activation="gelu")
