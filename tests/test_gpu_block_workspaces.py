"""One workspace, sized for a program's largest batch, under smaller batches that
use more of it (C entry points)."""
import ctypes

import pytest
import torch

from combine_ep_get_layout_amd import _abi
from gpu_util import announce
from test_gpu_block_linear import rows, weights
from test_gpu_expert_linear import DEV
from test_gpu_gated_ffn import make

pytestmark = pytest.mark.gpu
GUARD = 4096


def stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def at(t):
    return ctypes.c_void_p(t.data_ptr())


def workspace(nbytes):
    ws = torch.full((nbytes + GUARD,), 0x5A, dtype=torch.uint8, device=DEV)
    return ws, lambda: bool((ws[nbytes:] == 0x5A).all())


def test_products(gpu):
    lib, n, k, most = _abi.load(), 4096, 7168, 512
    nbytes = lib.ep_block_linear_workspace_bytes(most, n, k)
    ws, whole = workspace(nbytes)
    g = torch.Generator(device=DEV).manual_seed(0)
    w, _ = gpu.ep_cast_fp8_blocks(weights(g, (n, k)))
    for T in (512, 333, 64, 5):
        announce("block linear, one workspace", T)
        x = gpu.ep_cast_fp8(rows(g, T, k), 128)
        want = gpu.ep_block_linear(x, w)
        out = torch.zeros_like(want)
        assert lib.ep_block_linear(at(x[0]), at(x[1]), at(w[0]), at(w[1]), n, k, None, _abi.EP_ACT_NONE, None, None,
                                   None, T, at(ws), nbytes, at(out), stream()) == 0
        torch.cuda.synchronize()
        assert torch.equal(out, want) and whole()


def test_block(gpu):
    lib, H, inter, most = _abi.load(), 4096, 1024, 2000
    sizes = [lib.ep_gated_ffn_workspace_bytes(most, H, inter, b) for b in (0, 1)]
    ws, whole = workspace(max(sizes))
    for T in (2000, 1500, 700, 333, 3):
        announce("gated ffn, one workspace", T)
        x, w1, w2, dout, _ = make(T, H, inter, T)
        out, z = gpu.ep_gated_ffn(x, w1, w2, save=True)
        want = gpu.ep_gated_ffn_backward(dout, x, z, w1, w2)
        o2, z2, got = torch.zeros_like(out), torch.zeros_like(z), [torch.zeros_like(t) for t in want]
        assert lib.ep_gated_ffn(at(x), T, H, inter, at(w1), at(w2), _abi.EP_ACT_SWIGLU, None, at(z2), at(ws),
                                sizes[0], at(o2), stream()) == 0
        assert lib.ep_gated_ffn_backward(at(dout), at(x), at(z2), T, H, inter, at(w1), at(w2), _abi.EP_ACT_SWIGLU,
                                         None, None, at(ws), sizes[1], *[at(t) for t in got], 0, stream()) == 0
        torch.cuda.synchronize()
        assert torch.equal(o2, out) and torch.equal(z2, z) and whole()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
