"""Pins for oracle/training.py, CPU only: the choice against a brute force in
torch float64, the gradients against central differences and torch autograd,
the 8-bit tiles against the C oracle's quantizer.

Pages cited (title, section): "DeepSeek V3 From Scratch", "In code" (route)
and "The idea" (fine-grained quantization tiles); "Scaling Efficiency: A Deep
Dive into the DeepSeek-V3 Architecture", DeepSeekMoE sketch (softmax gate).
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import training as ot

OPTS = [
    ot.Opts(),
    ot.Opts(score="softmax"),
    ot.Opts(score="softmax", renormalize=False, scale=16.0),
    ot.Opts(renormalize=False, scale=2.5),
    ot.Opts(groups=4, top_groups=2, group_top=2, scale=2.5),
    ot.Opts(score="softmax", groups=3, top_groups=1, group_top=1),
]


def _weights(z, idx, o):
    """The weights and scores of a fixed choice, torch float64."""
    s = torch.sigmoid(z) if o.score == "sigmoid" else torch.softmax(z, dim=1)
    w = s.gather(1, idx)
    if o.renormalize:
        w = w / w.sum(dim=1, keepdim=True)
    return w * o.scale, s


@pytest.mark.parametrize("o", OPTS)
def test_choice_is_the_sorted_order(o):
    rng = np.random.default_rng(1)
    z, bias, k = rng.normal(size=(40, 12)), rng.uniform(-0.05, 0.05, size=12), 3
    idx, w, counts, short = ot.route(z, bias, k, o)
    s = ot.scores(z, o.score)
    for t in range(40):
        allowed = range(12)
        if o.top_groups < o.groups:
            per = 12 // o.groups
            val = [sum(sorted((s[t] + bias)[g * per:(g + 1) * per])[::-1][:o.group_top]) for g in range(o.groups)]
            allowed = [e for e in range(12) if np.sum(np.array(val) > val[e // per]) < o.top_groups]
        best = sorted(allowed, key=lambda e: -(s[t, e] + bias[e]))[:k]
        assert idx[t].tolist() == best
    assert not short.any() and counts.sum() == 120
    ref, _ = _weights(torch.from_numpy(z), torch.from_numpy(idx).long(), o)
    np.testing.assert_allclose(w, ref.numpy(), rtol=1e-13)
    if o.renormalize:
        np.testing.assert_allclose(w.sum(axis=1), o.scale, rtol=1e-13)


def test_ties_masks_and_short_rows():
    z = np.zeros((4, 6))
    z[1, 0] = z[1, 3] = -np.inf
    z[2, :] = -np.inf
    z[3, 1:] = [np.nan, -np.inf, 2.0, -np.inf, -np.inf]
    idx, w, counts, short = ot.route(z, None, 3, ot.Opts())
    assert idx.tolist() == [[0, 1, 2], [1, 2, 4], [-1, -1, -1], [3, 0, -1]]
    assert short.tolist() == [False, False, True, True]
    assert (w[2] == 0).all() and w[3, 2] == 0 and abs(w[3].sum() - 1) < 1e-15
    assert counts.tolist() == [2, 2, 2, 1, 1, 0]
    # a group whose experts are all masked is never kept
    z = np.zeros((1, 6))
    z[0, :2] = -np.inf
    idx, _, _, _ = ot.route(z, np.array([0, 0, 0, 0, 0.5, -2.0]), 2, ot.Opts(groups=3, top_groups=1, group_top=2))
    assert idx.tolist() == [[2, 3]]


@pytest.mark.parametrize("aux", [False, True])
@pytest.mark.parametrize("o", OPTS)
def test_gradient_against_differences_and_autograd(o, aux):
    rng = np.random.default_rng(2)
    T, E, k = 5, 12, 3
    z = rng.normal(size=(T, E)) * 1.5
    idx, _, _, _ = ot.route(z, None, k, o)
    dw = rng.normal(size=(T, k))
    ds = rng.normal(size=(T, E)) if aux else None
    got = ot.route_backward(z, idx, dw, ds, o)

    def value(zt):
        w, s = _weights(zt, torch.from_numpy(idx).long(), o)
        out = (w * torch.from_numpy(dw)).sum()
        return out + (s * torch.from_numpy(ds)).sum() if aux else out

    zt = torch.from_numpy(z).requires_grad_()
    value(zt).backward()
    np.testing.assert_allclose(got, zt.grad.numpy(), rtol=1e-10, atol=1e-12)
    h = 1e-5
    for t, e in [(0, 0), (1, int(idx[1, 0])), (4, int(idx[4, 2])), (3, 7)]:
        d = np.zeros_like(z)
        d[t, e] = h
        num = (value(torch.from_numpy(z + d)) - value(torch.from_numpy(z - d))).item() / (2 * h)
        # central differences: truncation ~ h^2 |f'''| / 6 and rounding ~ 2^-53 |f| / h, scale factors up to 16 * 3
        assert abs(num - got[t, e]) <= 1e-7


def test_underflowing_scores_keep_their_ratios():
    z = np.full((1, 4), -np.inf)
    z[0, :3] = [-900.0, -901.0, -2000.0]
    idx, w, _, _ = ot.route(z, None, 3, ot.Opts())
    assert idx.tolist() == [[0, 1, 2]]  # equal scores (0): lower index first
    np.testing.assert_allclose(w[0], np.exp([0.0, -1.0, -1100.0]) / (1 + np.exp(-1.0)), rtol=1e-12)


def test_tiles_match_the_quantizer():
    rng = np.random.default_rng(3)
    v = (rng.normal(size=(7, 256)) * np.exp2(rng.integers(-20, 20, size=(7, 1)))).astype(np.float32)
    v[2, :32] = 0.0
    v[3, 32:64] = 448.0
    v[3, 64:96] = np.nextafter(np.float32(448.0), np.float32(1e9))
    codes, eb = oracle.quantize_mx(v)
    assert (ot.tile_exponents(v) + 127 == eb.astype(np.int64)).all()
    words = np.transpose(eb.reshape(7, 2, 4), (1, 0, 2)).copy()
    np.testing.assert_array_equal(ot.dequantize(codes, words), oracle.mx_dequantize(codes, eb))


def test_swiglu_gradient_against_autograd_and_differences():
    rng = np.random.default_rng(4)
    a, g, u = (rng.normal(size=(3, 8)) * 2 for _ in range(3))
    wt = rng.uniform(size=3)
    da, dg, h, dw = ot.swiglu_backward(a, g, u, wt)
    at, gt, wtt = (torch.from_numpy(x).requires_grad_() for x in (a, g, wt))
    ht = torch.nn.functional.silu(at) * gt
    (wtt[:, None] * torch.from_numpy(u) * ht).sum().backward()
    np.testing.assert_allclose(h, ht.detach().numpy(), rtol=1e-12)
    np.testing.assert_allclose(da, at.grad.numpy(), rtol=1e-11, atol=1e-13)
    np.testing.assert_allclose(dg, gt.grad.numpy(), rtol=1e-11, atol=1e-13)
    np.testing.assert_allclose(dw, wtt.grad.numpy(), rtol=1e-11)
    f = lambda x: (wt[:, None] * u * x / (1 + np.exp(-x)) * g).sum()
    d = np.zeros_like(a)
    d[1, 3] = 1e-5
    assert abs((f(a + d) - f(a - d)) / 2e-5 - da[1, 3]) <= 1e-7
