"""Buffers with fewer rows than the layout: EP_DEV_RECV_OVERFLOW where a row that
holds a pair is missing, and only there, the same for every operator of the
receive segments; the rows that are there are computed, nothing behind them is
touched."""
import pytest
import torch

import expert_ref as ref
from gpu_util import announce
from test_gpu_expert_backward import _gradients
from test_gpu_expert_linear import DEV

pytestmark = pytest.mark.gpu
N, K, A = 96, 64, 16


def layout(gpu, counts):
    idx = torch.cat([torch.full((c,), e, dtype=torch.int64) for e, c in enumerate(counts)])
    idx = idx[torch.randperm(len(idx), generator=torch.Generator().manual_seed(1))].unsqueeze(1)
    return gpu.ep_get_layout(idx.to(DEV), len(counts), A)


def run(gpu, op, lay, rows):
    """The operator on buffers of `rows` rows, its outputs in front of guard rows,
    checked; what the layout's status holds afterwards."""
    g = torch.Generator(device=DEV).manual_seed(2)
    E, most = lay.num_experts, lay.max_recv_rows
    x = torch.randn((most, K), generator=g, device=DEV).bfloat16()[:rows].contiguous()
    w = torch.randn((E, N, K), generator=g, device=DEV).bfloat16()
    y = torch.randn((most, N), generator=g, device=DEV).bfloat16()[:rows].contiguous()
    held = torch.zeros(most, dtype=torch.bool, device=DEV)
    for _, a, b in ref.spans(lay, rows):
        held[a:b] = True
    if op == "linear":
        out = torch.full((most, N), 7.0, device=DEV, dtype=torch.bfloat16)
        gpu.ep_expert_linear(x, w, lay, out=out[:rows])
        for rs, z, dz, want, err in ref.linear(x, w, None, "none", None, False, ref.spans(lay, rows)):
            ref.assert_near(out[rs], want, err)
        assert (out[~held] == 7.0).all()
    elif op == "wgrad":
        dw, db = gpu.ep_expert_wgrad(y, x, lay, bias_grad=True)
        for e, a, b in ref.spans(lay, rows):
            yv, xv = y[a:b].double(), x[a:b].double()
            ref.assert_near(dw[e], yv.T @ xv, (b - a) * ref.U * (yv.abs().T @ xv.abs()), ref.U)
            ref.assert_near(db[e], yv.sum(0), (b - a) * ref.U * yv.abs().sum(0), ref.U)
    else:
        out = [torch.full((most, N), 7.0, device=DEV, dtype=torch.bfloat16) for _ in range(2)]
        dw = torch.full((most,), 7.0, device=DEV)
        z = torch.randn((most, N), generator=g, device=DEV).bfloat16()[:rows].contiguous()
        gpu.ep_expert_activation_backward(y, z, lay, "none", out=(out[0][:rows], out[1][:rows], dw[:rows]))
        for _, a, b in ref.spans(lay, rows):
            h, dpre = _gradients(z[a:b].double(), y[a:b].double(), 1.0, "none")
            assert torch.equal(out[0][a:b].double(), dpre) and torch.equal(out[1][a:b].double(), h)
        for o in (*out, dw):
            assert (o[~held] == 7.0).all()
    return int(lay.status.item())


OPS = ["linear", "wgrad", "act"]


@pytest.mark.parametrize("op", OPS)
def test_buffers_that_end_inside_the_last_padding(gpu, op):
    announce("expert status, cut in the padding", op)
    lay = layout(gpu, [20, 3, 37, 5])
    last = int(lay.expert_offset[3]) + 5
    assert last < lay.num_recv_rows()
    assert run(gpu, op, lay, last) == 0
    assert run(gpu, op, lay, last + 4) == 0
    assert run(gpu, op, lay, lay.max_recv_rows) == 0


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("short", [1, 5, 20, 60])
def test_buffers_that_end_inside_the_pairs(gpu, op, short):
    announce("expert status, cut in the pairs", op, short)
    lay = layout(gpu, [20, 3, 37, 5])
    last = int(lay.expert_offset[3]) + 5
    assert run(gpu, op, lay, last - short) == gpu.EP_DEV_RECV_OVERFLOW


@pytest.mark.parametrize("op", OPS)
def test_experts_without_rows_behind_the_buffers(gpu, op):
    """The last pair is expert 1's; experts 2 and 3 begin behind its padding."""
    announce("expert status, empty experts behind the buffers", op)
    lay = layout(gpu, [20, 3, 0, 0])
    last = int(lay.expert_offset[1]) + 3
    assert last < int(lay.expert_offset[2])
    assert run(gpu, op, lay, last) == 0
    assert run(gpu, op, lay, last - 1) == gpu.EP_DEV_RECV_OVERFLOW


def test_buffers_without_rows(gpu):
    """No rows at all: linear and the activation's backward return at once, the
    status as it was; the weight gradient still writes its zeros, and reports."""
    lay = layout(gpu, [20, 3, 37, 5])
    x = torch.zeros((0, K), device=DEV, dtype=torch.bfloat16)
    y = torch.zeros((0, N), device=DEV, dtype=torch.bfloat16)
    w = torch.zeros((4, N, K), device=DEV, dtype=torch.bfloat16)
    assert gpu.ep_expert_linear(x, w, lay)[0].shape == (0, N)
    assert gpu.ep_expert_activation_backward(y, y, lay, "silu")[0].shape == (0, N)
    assert lay.status.item() == 0
    dw, db = gpu.ep_expert_wgrad(y, x, lay, bias_grad=True)
    assert (dw == 0).all() and (db == 0).all() and lay.status.item() == gpu.EP_DEV_RECV_OVERFLOW


def test_results_into_what_they_add_to(gpu):
    """out may be the residual itself, dpre and h_out the bf16 z and dh."""
    lay = layout(gpu, [200, 3, 0, 137])
    rows = lay.max_recv_rows
    g = torch.Generator(device=DEV).manual_seed(3)
    held = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for _, a, b in ref.spans(lay, rows):
        held[a:b] = True
    new = lambda n: torch.randn((rows, n), generator=g, device=DEV).bfloat16()  # noqa: E731
    for E_n, act in ((96, "none"), (1056, "swiglu"), (8320, "geglu")):
        m = E_n // 2 if ref.gated(act) else E_n
        x, res, w = new(K), new(m), torch.randn((4, E_n, K), generator=g, device=DEV).bfloat16()
        want, _ = gpu.ep_expert_linear(x, w, lay, activation=act, residual=res)
        got, _ = gpu.ep_expert_linear(x, w, lay, activation=act, residual=res, out=res)
        assert got is res and torch.equal(got[held], want[held])
        z, dh = new(E_n), new(m)
        want = gpu.ep_expert_activation_backward(dh, z, lay, act)
        got = gpu.ep_expert_activation_backward(dh, z, lay, act, out=(z, dh, None))
        for p, q in zip(got, want):
            assert torch.equal(p[held], q[held])
