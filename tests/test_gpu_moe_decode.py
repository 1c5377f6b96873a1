"""ep_moe_decode against its definition in 64 bits, and against the path it
stands for (layout, dispatch, two expert products, combine)."""
import pytest
import torch

import expert_ref as ref
from gpu_util import announce
from test_gpu_expert_linear import DEV, routing

pytestmark = pytest.mark.gpu


def weights(gpu, E, n1, H, inter, g, fp8):
    w1 = (torch.randn((E, n1, H), generator=g, device=DEV) * H ** -0.5).bfloat16()
    w2 = (torch.randn((E, H, inter), generator=g, device=DEV) * inter ** -0.5).bfloat16()
    if not fp8:
        return w1, w2
    out = []
    for w in (w1, w2):
        c, s = gpu.ep_cast_fp8(w.view(-1, w.shape[2]), 128, scale_fmt="ue8m0")
        out.append((c.view(w.shape), s.view(*w.shape[:2], -1)))
    return tuple(out)


def reference(x, idx, tw, w1, w2, act, b1, b2, res):
    """(out, the error it may have before its rounding)."""
    T, K = idx.shape
    E, H = b1.shape[0] if b1 is not None else ref.value(w1).shape[0], x.shape[1]
    v1, v2, xv = ref.value(w1), ref.value(w2), x.double()
    inter = v2.shape[2]
    out = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    err, size = torch.zeros_like(out), torch.zeros_like(out)
    for r in res:
        out += r.double()
        size += r.double().abs()
    for k in range(K):
        for e in set(idx[:, k].tolist()):
            if not 0 <= e < E:
                continue
            t = (idx[:, k] == e).nonzero().flatten()
            z = xv[t] @ v1[e].T
            dz = (H + 1) * ref.U * (xv[t].abs() @ v1[e].abs().T)
            if b1 is not None:
                z = z + b1[e].double()
                dz = dz + 2 * ref.U * z.abs()
            h, dh = ref.activate(z, act, dz)
            # h is the sum of two bf16: off by half a step of the second, 2^-8 of
            # at most 2^-8 of h
            dh = dh + ref.BF16_HALF ** 2 * (h.abs() + dh)
            y = h @ v2[e].T
            dy = (dh + (inter + 1) * ref.U * (h.abs() + dh)) @ v2[e].abs().T
            if b2 is not None:
                y = y + b2[e].double()
                dy = dy + 2 * ref.U * y.abs()
            w = tw[t, k].double().unsqueeze(1) if tw is not None else 1.0
            out[t] += w * y
            err[t] += w * dy
            size[t] += w * y.abs()
    return out, err + (K + 2) * ref.U * size


def check(gpu, T, E, K, H, inter, act="swiglu", fp8=False, biases=False, res=0, tw=True, idx=None,
          seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    idx = routing(T, E, K, seed) if idx is None else idx
    n1 = 2 * inter if ref.gated(act) else inter
    w1, w2 = weights(gpu, E, n1, H, inter, g, fp8)
    x = torch.randn((T, H), generator=g, device=DEV).bfloat16()
    w = torch.rand((T, K), generator=g, device=DEV) if tw else None
    b1 = torch.randn((E, n1), generator=g, device=DEV).bfloat16() if biases else None
    b2 = torch.randn((E, H), generator=g, device=DEV).bfloat16() if biases else None
    rs = tuple(torch.randn((T, H), generator=g, device=DEV).bfloat16() for _ in range(res))
    out = gpu.ep_moe_decode(x, idx, w, w1, w2, act, b1, b2, rs or None)
    want, err = reference(x, idx, w, w1, w2, act, b1, b2, rs)
    ref.assert_near(out, want, err)
    return x, idx, w, w1, w2, b1, b2, rs, out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,E,K,H,inter", [(1, 8, 2, 256, 128), (1, 256, 8, 512, 256),
                                           (5, 16, 4, 1280, 384), (32, 8, 2, 256, 128),
                                           (128, 32, 8, 256, 256)])
def test_sizes(gpu, T, E, K, H, inter, fp8):
    announce("decode", T, E, K, H, inter, fp8)
    check(gpu, T, E, K, H, inter, fp8=fp8)


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "swiglu", "geglu"])
def test_activations_biases_residuals(gpu, act):
    announce("decode", act)
    check(gpu, 20, 6, 3, 264, 104, act, biases=True, res=2)
    check(gpu, 3, 6, 2, 264, 104, act, biases=True, res=1, tw=False)


@pytest.mark.parametrize("H,inter", [(8, 8), (72, 40), (1000, 136)])
def test_odd_sizes(gpu, H, inter):
    announce("decode", H, inter)
    check(gpu, 7, 5, 2, H, inter)


@pytest.mark.parametrize("T", [15, 16, 17, 33, 100])
def test_all_tokens_on_one_expert(gpu, T):
    """More pairs of one expert than one pass of 16 takes, and the same expert twice."""
    announce("decode one expert", T)
    idx = torch.full((T, 2), 3, device=DEV, dtype=torch.int64)
    idx[::3, 1] = 1
    check(gpu, T, 5, 2, 256, 128, idx=idx)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("inter", [128, 256, 384, 768])
def test_pairs_per_expert(gpu, inter, fp8):
    """Groups of 8 and 16 pairs, more experts than waves, odd and even numbers of
    steps over the intermediate channels."""
    announce("decode pairs per expert", inter, fp8)
    counts = [0, 1, 7, 8, 9, 15, 16, 17, 1, 0, 24, 25, 32, 33, 2, 8, 9, 16, 3]
    idx = torch.cat([torch.full((n,), e, dtype=torch.int64) for e, n in enumerate(counts)])
    order = torch.randperm(len(idx), generator=torch.Generator().manual_seed(inter))
    x, idx, w, w1, w2, *_, out = check(gpu, len(idx), len(counts), 1, 256, inter, fp8=fp8,
                                       idx=idx[order].unsqueeze(1).to(DEV))
    for t in range(0, len(idx), 29):
        one = gpu.ep_moe_decode(x[t:t + 1], idx[t:t + 1], w[t:t + 1], w1, w2)
        assert torch.equal(one[0].view(torch.int16), out[t].view(torch.int16))


def test_the_most_pairs(gpu):
    check(gpu, 1024, 4, 1, 64, 64)
    check(gpu, 4, 300, 256, 64, 64)
    check(gpu, 128, 4096, 8, 64, 16)


def test_missing_and_invalid_experts(gpu):
    idx = torch.tensor([[-1, -1], [0, -1], [7, 2], [-5, 1], [2 ** 40, 0]], device=DEV)
    x, idx, w, w1, w2, _, _, rs, out = check(gpu, 5, 4, 2, 128, 64, idx=idx, res=1)
    assert torch.equal(out[0], rs[0][0])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    gpu.ep_moe_decode(x, idx, w, w1, w2, status=status)
    assert status.item() == gpu.EP_DEV_BAD_EXPERT
    status.zero_()
    gpu.ep_moe_decode(x[:2], idx[:2], w[:2], w1, w2, status=status)
    assert status.item() == 0
    assert gpu.ep_moe_decode(x[:0], idx[:0], w[:0], w1, w2).shape == (0, 128)


def test_a_token_does_not_depend_on_the_batch(gpu):
    x, idx, w, w1, w2, *_, out = check(gpu, 60, 8, 3, 512, 256)
    for t in (0, 17, 59):
        one = gpu.ep_moe_decode(x[t:t + 1], idx[t:t + 1].contiguous(), w[t:t + 1], w1, w2)
        assert torch.equal(one[0].view(torch.int16), out[t].view(torch.int16))


def test_against_the_dispatched_path(gpu):
    """layout, dispatch, up, down, combine on the same batch: that path also rounds
    h and the expert outputs to bf16."""
    T, E, K, H, inter = 64, 16, 4, 512, 256
    x, idx, w, w1, w2, *_, out = check(gpu, T, E, K, H, inter)
    lay, recv, _, _ = gpu.ep_dispatch_with_layout(x, idx, E, topk_weights=w)
    h, _ = gpu.ep_expert_linear(recv, w1, lay, activation="swiglu")
    y, _ = gpu.ep_expert_linear(h, w2, lay)
    path, _ = gpu.ep_combine(y, lay, w)
    want, err = reference(x, idx, w, w1, w2, "swiglu", None, None, ())
    R = lay.num_recv_rows()
    # a rounded h adds half a step of each of its products; a rounded y half a step
    grow = (h[:R].double().abs().amax() * ref.value(w2).abs().sum(2).amax()
            + 2 * y[:R].double().abs().amax())
    ref.assert_near(path, want, err + ref.BF16_HALF * w.double().sum(1, keepdim=True) * grow)


# From 4104 channels on, the second kernel has more than 128 column tiles and one
# workgroup of it takes every token: an expert's pairs then meet in one wave.
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("inter", [128, 384])
def test_pairs_per_expert_in_one_workgroup(gpu, inter, fp8):
    """No, one, two and three passes of up to 16 pairs of an expert, of one and two
    groups of 8; more experts than waves, some behind each other in one wave."""
    announce("decode pairs per expert, one workgroup", inter, fp8)
    counts = [0, 1, 7, 8, 9, 15, 16, 17, 1, 0, 24, 25, 32, 33, 2, 8, 9, 16, 3]
    idx = torch.cat([torch.full((n,), e, dtype=torch.int64) for e, n in enumerate(counts)])
    order = torch.randperm(len(idx), generator=torch.Generator().manual_seed(inter))
    x, idx, w, w1, w2, *_, out = check(gpu, len(idx), len(counts), 1, 4224 if fp8 else 4104, inter,
                                       fp8=fp8, idx=idx[order].unsqueeze(1).to(DEV))
    for t in range(0, len(idx), 13):
        one = gpu.ep_moe_decode(x[t:t + 1], idx[t:t + 1], w[t:t + 1], w1, w2)
        assert torch.equal(one[0].view(torch.int16), out[t].view(torch.int16))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [4, 8, 9, 17, 100])
def test_all_tokens_on_one_expert_in_one_workgroup(gpu, T, fp8):
    announce("decode one expert, one workgroup", T, fp8)
    idx = torch.full((T, 2), 3, device=DEV, dtype=torch.int64)
    idx[::3, 1] = 1
    x, idx, w, w1, w2, *_, out = check(gpu, T, 5, 2, 4224 if fp8 else 4104, 128, fp8=fp8, idx=idx,
                                       act="geglu")
    for t in (0, T // 2, T - 1):
        one = gpu.ep_moe_decode(x[t:t + 1], idx[t:t + 1], w[t:t + 1], w1, w2, "geglu")
        assert torch.equal(one[0].view(torch.int16), out[t].view(torch.int16))


@pytest.mark.parametrize("T,E,K,inter", [(1024, 4, 1, 64), (128, 4096, 8, 8)])
def test_the_most_pairs_in_one_workgroup(gpu, T, E, K, inter):
    """256 pairs of an expert, and the most local memory that the second kernel takes."""
    announce("decode most pairs, one workgroup", T, E, K, inter)
    x, idx, w, w1, w2, b1, b2, rs, out = check(gpu, T, E, K, 4104, inter, biases=True, res=1)
    for t in (0, T // 2, T - 1):
        one = gpu.ep_moe_decode(x[t:t + 1], idx[t:t + 1], w[t:t + 1], w1, w2, "swiglu", b1, b2,
                                rs[0][t:t + 1])
        assert torch.equal(one[0].view(torch.int16), out[t].view(torch.int16))


@pytest.mark.parametrize("H", [256, 4104])
def test_result_into_a_residual(gpu, H):
    x, idx, w, w1, w2, b1, b2, rs, want = check(gpu, 30, 6, 2, H, 64, biases=True, res=2)
    for i in range(2):
        r = [t.clone() for t in rs]
        got = gpu.ep_moe_decode(x, idx, w, w1, w2, "swiglu", b1, b2, tuple(r), out=r[i])
        assert got is r[i] and torch.equal(got, want)
