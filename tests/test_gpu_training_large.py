"""Routing from logits, gate logits and saved activations on tensors of more
than 2^31 elements: rows before, across and behind that border equal those of
small calls on the same rows (each row's result does not depend on the others).
"""
import pytest
import torch

import fine_grained_moe_gate_b200 as moe

from gpu_harness import DEV, check_status

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _clean():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    moe.moe_get_last_error()
    yield
    torch.cuda.empty_cache()


def shape(T, E, k, d=64, I=128):
    return moe.MoEShape(T, d, E, k, I, 0, 128, moe.MOE_BF16)


def windows(rows, width):
    """Row ranges: the first, the one that crosses 2^31 elements, the last."""
    mid = (1 << 31) // width
    return [(0, 97), (mid - 50, mid + 51), (rows - 101, rows)]


def test_routing_past_32_bit_offsets():
    T, E, k = 8_500_000, 256, 2
    assert T * E > 1 << 31
    g = torch.Generator(device=DEV).manual_seed(1)
    z = torch.randn((T, E), generator=g, device=DEV)
    bias = (torch.rand(E, generator=g, device=DEV) - 0.5) * 0.1
    dw = torch.randn((T, k), generator=g, device=DEV)
    o = moe.route_opts(groups=8, top_groups=4, group_top=2)
    full = moe.route_opts("softmax", renormalize=False)
    idx = torch.empty((T, k), dtype=torch.int32, device=DEV)
    w = torch.empty((T, k), device=DEV)
    counts = torch.empty(E, dtype=torch.int32, device=DEV)
    moe.moe_route_logits(z, bias, shape(T, E, k), o, idx, w, counts)
    assert int(counts.sum()) == T * k and int(idx.min()) >= 0
    assert torch.equal(counts.long(), torch.bincount(idx.view(-1).long(), minlength=E))
    dz = torch.empty((T, E), device=DEV)
    for opts in (o, full):  # the chosen logits alone, and all of them
        moe.moe_route_logits_backward(z, idx, dw, None, shape(T, E, k), opts, dz)
        for lo, hi in windows(T, E):
            n = hi - lo
            zs, i2, w2, c2 = z[lo:hi].clone(), torch.empty_like(idx[:n]), torch.empty_like(w[:n]), counts.clone()
            moe.moe_route_logits(zs, bias, shape(n, E, k), o, i2, w2, c2)
            assert torch.equal(i2, idx[lo:hi]) and torch.equal(w2, w[lo:hi])
            d2 = torch.empty_like(zs)
            moe.moe_route_logits_backward(zs, i2, dw[lo:hi].clone(), None, shape(n, E, k), opts, d2)
            assert torch.equal(d2, dz[lo:hi])
    check_status()


def test_gate_logits_past_32_bit_offsets():
    T, d, E = 8_500_000, 64, 256
    g = torch.Generator(device=DEV).manual_seed(2)
    x = (torch.round(torch.randn((T, d), generator=g, device=DEV) * 16) / 16).to(BF)
    w = (torch.round(torch.randn((E, d), generator=g, device=DEV) * 25) / 1024).to(BF)
    z = torch.empty((T, E), device=DEV)
    moe.moe_gate_logits(x, w, shape(T, E, 1, d), z)
    for lo, hi in windows(T, E):
        assert torch.equal(z[lo:hi].double(), x[lo:hi].double() @ w.double().t())
    check_status()


def test_saved_activations_past_32_bit_offsets():
    T, d, E, k, I = 1_000_000, 64, 2, 1, 2304
    sh = shape(T, E, k, d, I)
    assert T * k * I > 1 << 31
    g = torch.Generator(device=DEV).manual_seed(3)
    x = (torch.round(torch.randn((T, d), generator=g, device=DEV) * 16) / 16).to(BF)
    w1, w3 = ((torch.round(torch.randn((E, I, d), generator=g, device=DEV) * 20) / 1024).to(BF) for _ in range(2))
    cut = T // 3
    offsets = torch.tensor([0, cut, T], dtype=torch.int32, device=DEV)
    h = torch.empty((T, I), dtype=BF, device=DEV)
    buf = moe.saved_act_buffers(sh, DEV)
    moe.moe_ffn_up_save(x, offsets, w1, w3, None, None, None, sh, h, None, moe.saved_acts(buf))
    check_status()
    u = torch.randn((T, I), generator=g, device=DEV)
    perm = torch.arange(T, dtype=torch.int32, device=DEV)
    w = torch.rand(T, generator=g, device=DEV)
    dadg = torch.empty((T, 2 * I), dtype=BF, device=DEV)
    dw = torch.empty(T, device=DEV)
    h2 = torch.empty_like(h)
    moe.moe_swiglu_backward_saved(moe.saved_acts(buf), sh, moe.MOE_ROUTED, u, perm, w, dadg, h2, dw)
    check_status()
    for lo, hi in windows(T, I) + [(cut - 50, cut + 50)]:
        n = hi - lo
        s2 = shape(n, E, k, d, I)
        off2 = (offsets.clamp(lo, hi) - lo).to(torch.int32)
        b2, hs = moe.saved_act_buffers(s2, DEV), torch.empty((n, I), dtype=BF, device=DEV)
        moe.moe_ffn_up_save(x[lo:hi].clone(), off2, w1, w3, None, None, None, s2, hs, None, moe.saved_acts(b2))
        assert torch.equal(hs, h[lo:hi])
        words = lambda b, rows: b.view(I // 128, rows, 4)
        for name in ("a", "g"):
            assert torch.equal(b2[name], buf[name][lo:hi])
            assert torch.equal(words(b2[name + "_scale"], n), words(buf[name + "_scale"], T)[:, lo:hi])
        d2, h3, dw2 = torch.empty((n, 2 * I), dtype=BF, device=DEV), torch.empty_like(hs), torch.empty(n, device=DEV)
        moe.moe_swiglu_backward_saved(moe.saved_acts(b2), s2, moe.MOE_ROUTED, u[lo:hi].clone(), perm[:n].clone(),
                                      w[lo:hi].clone(), d2, h3, dw2)
        assert torch.equal(d2, dadg[lo:hi]) and torch.equal(h3, h2[lo:hi]) and torch.equal(dw2, dw[lo:hi])
    check_status()
