"""GPU parity of moe_gate_logits, moe_route_logits and
moe_route_logits_backward against oracle/training.py (float64).

Pages cited (title, section): "DeepSeek V3 From Scratch", "In code" (route);
"Scaling Efficiency: A Deep Dive into the DeepSeek-V3 Architecture",
DeepSeekMoE sketch (softmax gate).

Indices and counts are equal: the order is the 64-bit values'.
Weights: u = 2^-24.  A 32-bit score carries the exponential's two ulps (4u),
the rounding of its argument (softmax: D u relative, D the spread of the
token's logits), the sums over at most 256 experts (8 additions in a lane, 5
across lanes: 13u) or 1 + e (u), a division (2u) and the weight's own
division, scale and rounding (4u); numerator and sum together (32 + 2D) u.
Gradients: the same relative error in p or s, twice, and differences G - <G, p>
formed in 32 bits: (128 + 8D) u of the terms' magnitudes (``_grad_bound``).
Results below 2^-120 may underflow.
"""
import numpy as np
import pytest
import torch

import fine_grained_moe_gate_b200 as moe
from oracle import training as ot

from gpu_harness import DEV, check_status

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -120


@pytest.fixture(autouse=True)
def _clean_status():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    moe.moe_get_last_error()
    yield


def shape(T, E, k, d=64, dtype=moe.MOE_BF16):
    return moe.MoEShape(T, d, E, k, 128, 0, 128, dtype)


def c_opts(o):
    return moe.route_opts(o.score, o.groups, o.top_groups, o.group_top, o.renormalize, o.scale)


def run_route(z, bias, k, o, stream=None):
    T, E = z.shape
    idx = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), float("nan"), device=DEV)
    counts = torch.full((E,), -7, dtype=torch.int32, device=DEV)
    moe.moe_route_logits(z, bias, shape(T, E, k), c_opts(o), idx, w, counts, stream)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy(), counts.cpu().numpy()


def spread(z):
    f = np.where(np.isfinite(z), z, np.nan)
    f = np.where(np.isfinite(f).any(axis=1, keepdims=True), f, 0.0)
    return (np.nanmax(f, axis=1) - np.nanmin(f, axis=1))[:, None]


def check_route(z, bias, k, o, got=None):
    idx, w, counts = got or run_route(z, bias, k, o)
    zn = z.cpu().numpy()
    ri, rw, rc, short = ot.route(zn, None if bias is None else bias.cpu().numpy(), k, o)
    assert (idx == ri).all(), np.argwhere(idx != ri)[:5]
    assert (counts == rc).all()
    tol = (32 + (2 * spread(zn) if o.score == "softmax" else 0)) * U
    assert (np.abs(w - rw) <= tol * np.abs(rw) + TINY * abs(o.scale)).all(), np.max(np.abs(w - rw) / (np.abs(rw) + 1e-30))
    return short


OPTS = {
    "sigmoid": ot.Opts(),
    "softmax": ot.Opts(score="softmax"),
    "softmax_as_scored": ot.Opts(score="softmax", renormalize=False, scale=16.0),
    "sigmoid_as_scored": ot.Opts(renormalize=False, scale=-0.5),
    "groups2": ot.Opts(groups=4, top_groups=2, group_top=2, scale=2.5),
    "groups1_softmax": ot.Opts(score="softmax", groups=4, top_groups=3, group_top=1, renormalize=False),
}
SHAPES = [(1, 4, 1), (3, 8, 2), (65, 12, 3), (129, 60, 4), (200, 64, 6), (77, 132, 16), (300, 160, 6), (257, 256, 8),
          (40, 252, 5)]


def make(T, E, seed, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    z = torch.randn((T, E), generator=g, device=DEV) * std
    bias = (torch.rand(E, generator=g, device=DEV) * 2 - 1) * 0.05
    return z, bias


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("name", list(OPTS))
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_route_matches_oracle(T, E, k, name, with_bias):
    o = OPTS[name]
    z, bias = make(T, E, T * 1000 + E, 1.5)
    if o.groups > 1 and o.top_groups * (E // o.groups) < k:
        pytest.skip("fewer experts kept than chosen")
    assert not check_route(z, bias if with_bias else None, k, o).any()
    check_status()


@pytest.mark.parametrize("groups,per,top,gtop", [(32, 8, 5, 2), (8, 32, 4, 2), (6, 42, 1, 2), (2, 128, 1, 1), (3, 5, 2, 2),
                                                 (16, 1, 9, 1), (7, 9, 7, 2), (5, 50, 2, 2)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_group_shapes(groups, per, top, gtop, score):
    z, bias = make(130, groups * per, groups * 100 + per, 2.0)
    k = min(8, top * per)
    check_route(z, bias, k, ot.Opts(score=score, groups=groups, top_groups=top, group_top=gtop))
    check_status()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("grouped", [False, True])
def test_ties_go_to_the_lower_index(score, grouped):
    """Logits on a coarse grid: nearly every row has equal values at the border."""
    g = torch.Generator(device=DEV).manual_seed(5)
    z = torch.randint(-2, 3, (500, 256), generator=g, device=DEV).float() * 0.5
    o = ot.Opts(score=score, groups=8, top_groups=3, group_top=2) if grouped else ot.Opts(score=score)
    check_route(z, None, 8, o)
    check_route(z, torch.full((256,), 0.25, device=DEV), 8, o)
    check_route(torch.zeros((33, 256), device=DEV), None, 8, o)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_values_closer_than_their_32_bit_error(score):
    """Neighbouring scores differ by a few 2^-40 through the bias: only their 64-bit values order them."""
    T, E = 64, 96
    rng = np.random.default_rng(6)
    z = torch.from_numpy(rng.normal(size=(T, E)).astype(np.float32)).to(DEV)
    # experts in pairs: the same logit up to one ulp, in either order
    z[:, 1::2] = torch.nextafter(z[:, ::2], torch.from_numpy(np.where(rng.random((T, E // 2)) < 0.5, -9.0, 9.0)
                                                               .astype(np.float32)).to(DEV))
    for o in (ot.Opts(score=score), ot.Opts(score=score, groups=6, top_groups=3, group_top=2),
              ot.Opts(score=score, groups=32, top_groups=9, group_top=2)):
        check_route(z, None, 8, o)
        check_route(z, torch.full((E,), 0.03125, device=DEV), 8, o)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_large_logits(score):
    """Saturated scores (ties in 64 bits), the type's largest and lowest values."""
    z, bias = make(200, 64, 7, 30.0)
    z[0, :] = torch.finfo(torch.float32).min
    z[1, ::2] = torch.finfo(torch.float32).min
    z[2, :5] = torch.finfo(torch.float32).max
    z[3, 4:7] = float("inf")
    z[4, :] = -300.0
    z[4, 9] = -301.0
    for b in (None, bias, bias * 1e6):
        for renorm in (True, False):
            idx, w, counts = run_route(z, b, 6, ot.Opts(score=score, renormalize=renorm))
            ri, rw, rc, _ = ot.route(z.cpu().numpy(), None if b is None else b.cpu().numpy(), 6,
                                     ot.Opts(score=score, renormalize=renorm))
            assert (idx == ri).all() and (counts == rc).all()
            # |z - m| is up to 2^24 here: hold the weights to the part that the exponential's argument keeps
            d = np.minimum(spread(z.cpu().numpy()), 110.0)
            tol = (32 + 2 * d) * U
            assert (np.abs(w - rw) <= tol * np.abs(rw) + 2.0 ** -118).all()
    check_status()


def test_masked_experts_and_empty_rows():
    z, bias = make(300, 60, 8)
    z[:, 10:20] = float("-inf")
    check_route(z, bias, 4, ot.Opts())
    check_status()
    b = bias.clone()
    b[3] = float("-inf")   # masked through the bias
    b[5] = 1e30            # forced
    check_route(z, b, 4, ot.Opts(score="softmax"))
    check_status()
    z[7, :] = float("-inf")
    z[8, 4:] = float("-inf")
    z[9, 2:] = float("-inf")
    z[10, 30] = float("nan")
    for o in (ot.Opts(), ot.Opts(score="softmax"), ot.Opts(score="softmax", renormalize=False),
              ot.Opts(groups=6, top_groups=2, group_top=2)):
        short = check_route(z, bias, 4, o)
        assert short[7] and short[9]
        assert moe.moe_get_last_error() == 6
    # the same with one bad token per call: each is reported on its own
    ok, _ = make(64, 60, 9)
    for t, fill in ((5, float("-inf")), (63, float("nan"))):
        y = ok.clone()
        y[t, :58 if fill != fill else 60] = fill
        check_route(y, None, 4, ot.Opts())
        assert moe.moe_get_last_error() == 6


def test_nan_bias_masks_and_reports():
    z, bias = make(16, 8, 10)
    bias[2] = float("nan")
    check_route(z, bias, 3, ot.Opts())
    assert moe.moe_get_last_error() == 6


def test_no_tokens_clears_counts():
    z = torch.empty((0, 16), device=DEV)
    _, _, counts = run_route(z, None, 2, ot.Opts())
    assert (counts == 0).all()


def test_a_tokens_result_does_not_depend_on_the_batch():
    z, bias = make(5000, 256, 11)
    o = OPTS["groups2"]
    idx, w, counts = run_route(z, bias, 8, o)
    for lo, hi in ((0, 1), (17, 81), (4000, 5000)):
        i2, w2, _ = run_route(z[lo:hi].contiguous(), bias, 8, o)
        assert (i2 == idx[lo:hi]).all() and (w2.view(np.uint32) == w[lo:hi].view(np.uint32)).all()
    again = run_route(z, bias, 8, o)
    assert (again[0] == idx).all() and (again[1].view(np.uint32) == w.view(np.uint32)).all()
    assert (again[2] == counts).all() and counts.sum() == 40000


def test_route_agrees_with_moe_route():
    """The layer's own gate from its logits: where moe_route's 32-bit choice is clear, the two agree."""
    T, d, E, k = 512, 256, 64, 6
    g = torch.Generator(device=DEV).manual_seed(12)
    x = (torch.round(torch.randn((T, d), generator=g, device=DEV) * 16) / 16).bfloat16()
    wg = (torch.round(torch.randn((E, d), generator=g, device=DEV) * 0.06 * 1024) / 1024).bfloat16()
    bias = (torch.rand(E, generator=g, device=DEV) - 0.5) * 0.04
    sh = shape(T, E, k, d)
    i1 = torch.empty((T, k), dtype=torch.int32, device=DEV)
    w1 = torch.empty((T, k), device=DEV)
    c1 = torch.empty(E, dtype=torch.int32, device=DEV)
    moe.moe_route(x, wg, bias, sh, i1, w1, c1)
    z = torch.empty((T, E), device=DEV)
    moe.moe_gate_logits(x, wg, sh, z)
    i2, w2, c2 = run_route(z, bias, k, ot.Opts())
    s = ot.scores(z.cpu().numpy(), "sigmoid") + bias.cpu().numpy()
    top = -np.sort(-s, axis=1)[:, :k + 1]
    clear = (top[:, :-1] - top[:, 1:]).min(axis=1) > 1e-6
    assert clear.mean() > 0.9
    assert (i1.cpu().numpy()[clear] == i2[clear]).all()
    assert np.allclose(w1.cpu().numpy()[clear], w2[clear], rtol=64 * U, atol=0)


# ---------------------------------------------------------------- gate logits

@pytest.mark.parametrize("T,d,E,dtype", [(1, 64, 8, "bf16"), (5, 128, 17, "bf16"), (64, 7168, 256, "bf16"),
                                         (130, 192, 60, "bf16"), (300, 2048, 64, "bf16"), (1000, 512, 255, "bf16"),
                                         (5000, 1024, 250, "bf16"), (20000, 256, 256, "bf16"), (700, 7168, 64, "bf16"),
                                         (127, 320, 31, "bf16"), (129, 448, 129, "bf16"), (256, 64, 256, "bf16"),
                                         (2368, 512, 256, "bf16"), (2369, 512, 256, "bf16"), (3001, 1344, 200, "bf16"),
                                         (4096, 576, 256, "bf16"), (6143, 320, 33, "bf16"), (9473, 192, 256, "bf16"),
                                         (40000, 128, 16, "bf16"),
                                         (1, 8, 1, "f32"), (33, 40, 5, "f32"), (128, 256, 256, "f32"),
                                         (257, 72, 100, "f32")])
def test_gate_logits_exact_on_a_grid(T, d, E, dtype):
    """Inputs of few bits: every partial sum is exact, so the product has to be too."""
    g = torch.Generator(device=DEV).manual_seed(T + d + E)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = (torch.round(torch.randn((T, d), generator=g, device=DEV) * 16) / 16).to(dt)
    w = (torch.round(torch.randn((E, d), generator=g, device=DEV) * 25) / 1024).to(dt)
    z = torch.full((T, E), float("nan"), device=DEV)
    moe.moe_gate_logits(x, w, shape(T, E, 1, d, moe.MOE_BF16 if dtype == "bf16" else moe.MOE_F32), z)
    ref = x.double() @ w.double().t()
    assert torch.equal(z.double(), ref)
    check_status()


@pytest.mark.parametrize("T,d,E", [(64, 7168, 256), (513, 2048, 64), (9000, 7168, 128)])
def test_gate_logits_random(T, d, E):
    """Any bf16 inputs: products are exact in 32 bits, each of the d additions of a sum of magnitude up to A =
    sum |x w| loses at most 2^-23 of it (truncating adders): d * 2^-23 * A."""
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn((T, d), generator=g, device=DEV).bfloat16()
    w = (torch.randn((E, d), generator=g, device=DEV) * 0.02).bfloat16()
    z = torch.empty((T, E), device=DEV)
    moe.moe_gate_logits(x, w, shape(T, E, 1, d), z)
    ref = x.double() @ w.double().t()
    mag = x.double().abs() @ w.double().abs().t()
    assert bool(((z.double() - ref).abs() <= d * 2.0 ** -23 * mag).all())
    # and as a whole: the additions' errors mostly cancel; one per 16 products, each half an ulp of |z|-sized sums
    rel = float((z.double() - ref).norm() / ref.norm())
    assert rel <= d / 16 * 2.0 ** -24, rel


# ---------------------------------------------------------------- backward

def _grad_bound(z, idx, dw, ds, o):
    """(128 + 8D) u of the magnitude of the terms of each dz."""
    T, E = z.shape
    s = ot.scores(z, o.score)
    sp = spread(z) if o.score == "softmax" else np.zeros((T, 1))
    mag = np.zeros((T, E))
    ok = (idx >= 0) & (idx < E)
    G = np.where(ok, np.abs(dw), 0.0) * abs(o.scale)
    dsm = np.zeros((T, E)) if ds is None else np.abs(np.where(s > 0, ds, 0.0))
    for t in range(T):
        e = idx[t][ok[t]]
        if o.renormalize:
            p = ot.chosen_weights(z[t, e].astype(np.float64), s[t, e], ot.Opts(score=o.score))
            np.add.at(mag[t], e, p * 2 * G[t].max(initial=0.0))
        else:
            np.add.at(dsm[t], e, G[t][ok[t]])
    if o.score == "sigmoid":
        az = np.exp(-np.abs(np.where(s > 0, z, 0.0).astype(np.float64)))
        mag += dsm * az / (1 + az) ** 2
    else:
        mag += s * (dsm + (dsm * s).sum(axis=1, keepdims=True))
    return (128 + 8 * np.minimum(sp, 110.0)) * U * mag + TINY


def run_bwd(z, idx, dw, ds, o):
    T, E = z.shape
    dz = torch.full((T, E), float("nan"), device=DEV)
    moe.moe_route_logits_backward(z, idx, dw, ds, shape(T, E, idx.shape[1]), c_opts(o), dz)
    torch.cuda.synchronize()
    return dz.cpu().numpy()


def check_bwd(z, idx, dw, ds, o):
    got = run_bwd(z, idx, dw, ds, o)
    zn, di, dwn = z.cpu().numpy(), idx.cpu().numpy(), dw.cpu().numpy().astype(np.float64)
    dsn = None if ds is None else ds.cpu().numpy().astype(np.float64)
    ref = ot.route_backward(zn, di, dwn, dsn, o)
    tol = _grad_bound(zn, di, dwn, dsn, o)
    nan = np.isnan(ref)  # a NaN gradient of a score in use reaches the logits
    assert (np.isnan(got) == nan).all()
    assert (nan | (np.abs(got - ref) <= tol)).all(), np.nanmax(np.abs(got - ref) / tol)
    return got


@pytest.mark.parametrize("aux", [False, True])
@pytest.mark.parametrize("name", list(OPTS))
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_backward_matches_oracle(T, E, k, name, aux):
    o = OPTS[name]
    if o.groups > 1 and (E % o.groups or o.top_groups * (E // o.groups) < k):
        pytest.skip("fewer experts kept than chosen")
    z, _ = make(T, E, T + E, 2.0)
    g = torch.Generator(device=DEV).manual_seed(E)
    idx = z.topk(k, dim=1).indices.to(torch.int32)
    dw = torch.randn((T, k), generator=g, device=DEV)
    ds = torch.randn((T, E), generator=g, device=DEV) * 0.1 if aux else None
    check_bwd(z, idx, dw, ds, o)
    check_status()


@pytest.mark.parametrize("name", ["sigmoid", "softmax", "softmax_as_scored", "sigmoid_as_scored"])
def test_backward_skipped_slots_masks_and_repeats(name):
    o = OPTS[name]
    T, E, k = 70, 60, 4
    z, _ = make(T, E, 13, 2.0)
    z[:, 3] = float("-inf")
    g = torch.Generator(device=DEV).manual_seed(14)
    idx = z.topk(k, dim=1).indices.to(torch.int32)
    dw = torch.randn((T, k), generator=g, device=DEV)
    ds = torch.randn((T, E), generator=g, device=DEV)
    ds[:, 3] = float("nan")      # behind the mask (row 7 lifts it: its NaN shows)
    idx[0, 1] = -1               # an empty slot
    dw[0, 1] = float("nan")
    idx[1, :] = -1               # a token without experts
    idx[2, 1] = idx[2, 0]        # listed twice
    idx[3, :] = idx[3, 0]        # four times
    idx[4, 2] = 3                # a masked expert
    z[5, :] = float("-inf")
    ds[5, :] = float("inf")
    z[6, int(idx[6, 1])] = float("nan")
    z[7, :] = -250.0             # every score underflows in 32 bits
    z[7, 11] = -251.0
    idx[7] = torch.tensor([11, 12, 13, 14], dtype=torch.int32)
    for d in (None, ds):
        got = check_bwd(z, idx, dw, d, o)
        assert (np.delete(got[:, 3], 7) == 0).all() and (got[5] == 0).all()
        check_status()
    # an index outside the experts: skipped and reported
    idx[9, 0] = E
    check_bwd(z, idx, dw, None, o)
    assert moe.moe_get_last_error() == 6
    idx[9, 0] = -2
    check_bwd(z, idx, dw, ds, o)
    assert moe.moe_get_last_error() == 6


def test_backward_against_differences():
    """The forward's own weights, moved by +-h in one logit: <dw, w> changes by dlogits.  h = 2^-7: truncation
    h^2 / 6 |f'''| <= 1.1e-5 |G|, rounding 2 * 2^-22 |w G| / 2h <= 4e-5 |G|; |G| <= 4 over k = 4 terms."""
    T, E, k = 1, 24, 4
    for o in (ot.Opts(), ot.Opts(score="softmax"), ot.Opts(score="softmax", renormalize=False)):
        z, _ = make(T, E, 15, 1.0)
        z[0, :k] += 6.0  # the choice stays the same under the moves
        idx, _, _ = run_route(z, None, k, o)
        dw = torch.randn((T, k), generator=torch.Generator(device=DEV).manual_seed(16), device=DEV)
        dz = run_bwd(z, torch.from_numpy(idx).to(DEV), dw, None, o)
        for e in list(idx[0]) + [10]:
            val = []
            for sgn in (1, -1):
                y = z.clone()
                y[0, e] += sgn * 2.0 ** -7
                i2, w2, _ = run_route(y, None, k, o)
                by = dict(zip(i2[0].tolist(), w2[0].tolist()))
                val.append(sum(by[int(i)] * float(dw[0, j]) for j, i in enumerate(idx[0])))
            num = (val[0] - val[1]) / 2 ** -6
            assert abs(num - dz[0, e]) <= 4 * 4 * 5.1e-5, (o, e, num, dz[0, e])


def test_other_stream_and_graph_replay():
    """The calls run on the stream they are given, and can be captured and replayed on new inputs."""
    T, E, k = 333, 256, 8
    o = OPTS["groups2"]
    z, bias = make(T, E, 17)
    idx = torch.empty((T, k), dtype=torch.int32, device=DEV)
    w = torch.empty((T, k), device=DEV)
    counts = torch.empty(E, dtype=torch.int32, device=DEV)
    dw = torch.randn((T, k), device=DEV)
    dz = torch.empty((T, E), device=DEV)
    sh, co = shape(T, E, k), c_opts(o)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        moe.moe_route_logits(z, bias, sh, co, idx, w, counts)
        moe.moe_route_logits_backward(z, idx, dw, None, sh, co, dz)
    for seed in (18, 19):
        z.copy_(make(T, E, seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        check_route(z, bias, k, o, (idx.cpu().numpy(), w.cpu().numpy(), counts.cpu().numpy()))
        ref = ot.route_backward(z.cpu().numpy(), idx.cpu().numpy(), dw.cpu().numpy().astype(np.float64), None, o)
        tol = _grad_bound(z.cpu().numpy(), idx.cpu().numpy(), dw.cpu().numpy().astype(np.float64), None, o)
        assert (np.abs(dz.cpu().numpy() - ref) <= tol).all()
    check_status()


def test_streams_and_strided_inputs():
    """A stream of the caller's; two batches on two streams at once; a strided tensor is refused."""
    o = OPTS["groups2"]
    co = c_opts(o)
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = []
    for i, st in enumerate(streams):
        T, E, k = 3000 + i, 256, 8
        z, bias = make(T, E, 30 + i)
        runs.append((z, bias, torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV),
                     torch.empty(E, dtype=torch.int32, device=DEV)))
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (z, bias, idx, w, counts) in zip(streams, runs):
            moe.moe_route_logits(z, bias, shape(z.shape[0], 256, 8), co, idx, w, counts, stream=st)
    with torch.cuda.stream(streams[0]):  # the current stream, when none is given
        moe.moe_route_logits(runs[0][0], runs[0][1], shape(3000, 256, 8), co, *runs[0][2:])
    torch.cuda.synchronize()
    for z, bias, idx, w, counts in runs:
        check_route(z, bias, 8, o, (idx.cpu().numpy(), w.cpu().numpy(), counts.cpu().numpy()))
    check_status()
    z, bias, idx, w, counts = runs[0]
    wide = torch.empty((3000, 512), device=DEV)
    with pytest.raises(moe.MoEError, match="contiguous"):
        moe.moe_route_logits(wide[:, :256], bias, shape(3000, 256, 8), co, idx, w, counts)


# ---------------------------------------------------------------- batches large enough for four tokens per warp

BATCHES = [(131, 5, 2), (300, 16, 8), (901, 60, 4), (835, 63, 7), (1031, 64, 6), (1709, 130, 8), (2083, 160, 6), (3350, 251, 8),
           (3331, 256, 1), (3400, 256, 8), (3329, 256, 9)]


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("name", ["sigmoid", "softmax_as_scored", "softmax"])
@pytest.mark.parametrize("T,E,k", BATCHES)
def test_batch_matches_oracle(T, E, k, name, with_bias):
    z, bias = make(T, E, T + E, 1.5)
    assert not check_route(z, bias if with_bias else None, k, OPTS[name]).any()
    check_status()


@pytest.mark.parametrize("groups,per,top,k", [(8, 32, 4, 8), (8, 20, 3, 6), (6, 42, 3, 8), (6, 9, 2, 7), (8, 31, 4, 8), (3, 5, 2, 8),
                                              (2, 128, 1, 8), (4, 63, 2, 8), (8, 2, 4, 8), (7, 36, 5, 8), (8, 1, 8, 8),
                                              (8, 1, 3, 3), (5, 4, 2, 8), (4, 16, 1, 8)])
@pytest.mark.parametrize("score,gtop", [("sigmoid", 1), ("sigmoid", 2), ("softmax", 1)])
def test_batch_group_shapes(groups, per, top, k, score, gtop):
    E = groups * per
    z, bias = make(max(13 * E, 129) + 2, E, groups * 100 + per, 2.0)
    o = ot.Opts(score=score, groups=groups, top_groups=top, group_top=gtop, scale=2.5)
    check_route(z, bias if score == "sigmoid" else None, k, o)
    check_route(z, None, k, o)
    check_status()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("gtop", [0, 1, 2])
def test_batch_ties_go_to_the_lower_index(score, gtop):
    g = torch.Generator(device=DEV).manual_seed(15)
    z = torch.randint(-2, 3, (3333, 256), generator=g, device=DEV).float() * 0.5
    o = ot.Opts(score=score, groups=8, top_groups=3, group_top=gtop) if gtop else ot.Opts(score=score)
    check_route(z, None, 8, o)
    check_route(z, torch.full((256,), 0.25, device=DEV), 8, o)
    z[:, ::3] += torch.randint(-99, 99, (3333, 86), generator=g, device=DEV).float() / 64  # some ties, most rows without
    check_route(z, None, 7, o)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_batch_values_closer_than_their_32_bit_error(score):
    T, E = 1250, 96
    rng = np.random.default_rng(16)
    z = torch.from_numpy(rng.normal(size=(T, E)).astype(np.float32)).to(DEV)
    z[:, 1::2] = torch.nextafter(z[:, ::2], torch.from_numpy(np.where(rng.random((T, E // 2)) < 0.5, -9.0, 9.0)
                                                               .astype(np.float32)).to(DEV))
    for o in (ot.Opts(score=score), ot.Opts(score=score, groups=6, top_groups=3, group_top=2),
              ot.Opts(score=score, groups=6, top_groups=3, group_top=1)):
        for k in (7, 8):
            check_route(z, None, k, o)
            check_route(z, torch.full((E,), 0.03125, device=DEV), k, o)
    # groups whose values differ by an ulp of one logit
    z[:, 16:32], z[:, 48:64] = z[:, :16], z[:, 32:48]
    z[:, 16::32] = torch.nextafter(z[:, ::32], torch.tensor(9.0, device=DEV))
    for gtop in (1, 2):
        check_route(z, None, 8, ot.Opts(score=score, groups=6, top_groups=3, group_top=gtop))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("kind", ["saturated", "beyond", "tiny", "wide", "huge"])
def test_batch_logits_whose_scores_lie_close(score, kind):
    T, E = 515, 32
    g = torch.Generator(device=DEV).manual_seed(17)
    u = torch.rand((T, E), generator=g, device=DEV)
    z = {"saturated": 12 + 10 * u, "beyond": 25 + 25 * u, "tiny": (u - 0.5) * 1e-12, "wide": (u - 0.5) * 3000,
         "huge": (u - 0.5) * 6e38}[kind]
    if kind == "huge" and score == "softmax":
        z = z.clamp(min=-1e37)  # rows of +inf (6e38 is past the type) beside one low value
    for o in (ot.Opts(score=score), ot.Opts(score=score, groups=4, top_groups=2, group_top=1)):
        idx, w, counts = run_route(z, None, 6, o)
        zn = z.cpu().numpy()
        ri, rw, rc, _ = ot.route(zn, None, 6, o)
        if kind == "tiny":
            # Logits closer than 2^-52: their order is that of two libraries' exp, each within an ulp.  Around
            # s = 1/2 (e^-z = 1, ulp 2^-52): e off by 2^-52, 1 + e rounded by 2^-53, s = 1 / (1 + e) off by a quarter
            # of their sum and 2^-54: D = 1.5 x 2^-53.  Softmax, s = y / sum = 1/32: y off by its ulp 2^-53, the quotient
            # rounded by 2^-53 of it: D = 2^-57.  The r-th largest of values off by at most
            # D is within D of the r-th largest, so the oracle's scores of both choices differ by at most 4 D, 6 x 2^-53
            # and 2^-55 (2^-54 with the sums' own rounding).  Groups as close as that may be exchanged.
            s, near = ot.scores(zn, score), 6 * 2.0 ** -53 if score == "sigmoid" else 2.0 ** -54
            sure = np.ones(T, bool)
            if o.groups > 1:
                gv = np.sort(s.reshape(T, o.groups, -1).max(axis=2), axis=1)[:, ::-1]
                sure = gv[:, o.top_groups - 1] - gv[:, o.top_groups] > near
            at = lambda i: np.take_along_axis(s, i, axis=1)
            assert (np.abs(at(idx) - at(ri)) <= near)[sure].all() and sure.mean() > 0.9
            assert (np.diff(np.sort(idx, axis=1), axis=1) > 0).all()
            rw = np.stack([ot.chosen_weights(zn[t, i].astype(np.float64), s[t, i], o) for t, i in enumerate(idx)])
            rc = np.bincount(idx.reshape(-1), minlength=E)
        else:
            assert (idx == ri).all(), np.argwhere(idx != ri)[:5]
        assert (counts == rc).all()
        # e^x for |x| up to 87 (what is smaller underflows): 2 x 87 u of the argument's rounding
        assert (np.abs(w - rw) <= (32 + 2 * 87) * U * np.abs(rw) + TINY).all()


@pytest.mark.parametrize("name", ["sigmoid", "softmax", "softmax_as_scored"])
def test_batch_best_experts_in_one_lane(name):
    """Experts 32 apart in chunks of four are one lane's: 4, 5 .. 20 of the best lie there."""
    T, E, k = 3400, 256, 8
    g = torch.Generator(device=DEV).manual_seed(18)
    z, bias = make(T, E, 18)
    lane = torch.randint(0, 8, (T, 1), generator=g, device=DEV)
    many = 3 + torch.arange(T, device=DEV)[:, None] % 18
    e = torch.arange(E, device=DEV)[None]
    here = (e // 4 % 8 == lane) & ((e // 32) * 4 + e % 4 < many)
    z = torch.where(here, z.abs() + 4.0, z)
    check_route(z, None, k, OPTS[name])
    check_route(z, bias, k, OPTS[name])
    check_route(z, None, k, ot.Opts(score=OPTS[name].score, groups=8, top_groups=5, group_top=1))
    check_status()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_batch_masks_infinities_and_nan(score):
    T, E, k = 1003, 60, 6
    z, bias = make(T, E, 19)
    inf = float("inf")
    z[:, 7] = -inf
    z[0:40, : E - k] = -inf  # exactly k left
    z[100:103, : E - k + 2] = -inf  # too few
    z[200] = -inf  # none
    z[300:303, 11] = inf
    z[301, 12] = inf
    z[400, 13] = float("nan")
    z[401] = float("nan")
    z[T - 1, 5:] = -inf
    bias[3] = -inf
    bias[4] = 2e38
    for b in (None, bias):
        for o in (ot.Opts(score=score), ot.Opts(score=score, groups=5, top_groups=2, group_top=1)):
            moe.moe_get_last_error()
            assert check_route(z, b, k, o).any()
            assert moe.moe_get_last_error() == 6


@pytest.mark.parametrize("T", [8, 9, 31, 32, 33, 64, 65, 97, 127, 128, 129, 131, 193, 255, 256, 257])
def test_small_batches_at_each_form(T):
    for E, k, o, with_bias in ((256, 8, OPTS["groups2"], True), (64, 6, OPTS["softmax_as_scored"], False),
                               (60, 5, OPTS["sigmoid"], True), (96, 8, ot.Opts(score="softmax", groups=6, top_groups=3), False),
                               (256, 8, OPTS["softmax"], False), (252, 7, OPTS["sigmoid"], True)):
        z, bias = make(T, E, T + E)
        if E == 96:
            z[:, 5] = float("-inf")
        check_route(z, bias if with_bias else None, k, o)
    check_status()


@pytest.mark.parametrize("T", [5, 100, 700])
def test_rows_of_equal_values(T):
    """Every expert a candidate: zeros (a padded batch), a coarse grid, rows of either kind in turn."""
    g = torch.Generator(device=DEV).manual_seed(T)
    for E, k in ((256, 8), (256, 12), (60, 4), (96, 16)):
        z = torch.randint(-1, 2, (T, E), generator=g, device=DEV).float()
        z[::2] = 0.0
        z[1::4] += torch.randn((z[1::4].shape), generator=g, device=DEV)
        bias = torch.full((E,), 0.125, device=DEV)
        for o in (ot.Opts(score="softmax"), ot.Opts(), ot.Opts(groups=4, top_groups=3, group_top=2),
                  ot.Opts(score="softmax", groups=4, top_groups=2, group_top=2, renormalize=False)):
            check_route(z, bias, k, o)
            check_route(z, None, k, o)
    check_status()


def test_graphs_replayed_on_two_streams_at_once():
    """Gate logits, routing and its gradient of several sizes, one graph per size, replayed in turn on two streams."""
    o = OPTS["groups2"]
    co, runs = c_opts(o), []
    for i, (T, d, E, k) in enumerate(((5, 512, 256, 8), (40, 256, 64, 6), (100, 128, 60, 4), (600, 512, 160, 6), (3000, 64, 256, 8))):
        g = torch.Generator(device=DEV).manual_seed(50 + i)
        x = (torch.round(torch.randn((T, d), generator=g, device=DEV) * 16) / 16).to(torch.bfloat16)
        wg = (torch.round(torch.randn((E, d), generator=g, device=DEV) * 25) / 1024).to(torch.bfloat16)
        r = dict(x=x, wg=wg, bias=make(T, E, 60 + i)[1], z=torch.empty((T, E), device=DEV),
                 idx=torch.empty((T, k), dtype=torch.int32, device=DEV), w=torch.empty((T, k), device=DEV),
                 counts=torch.empty(E, dtype=torch.int32, device=DEV), dw=torch.randn((T, k), generator=g, device=DEV),
                 dz=torch.empty((T, E), device=DEV), stream=torch.cuda.Stream(), graph=torch.cuda.CUDAGraph())
        sh = shape(T, E, k, d)

        def calls(r=r, sh=sh):
            moe.moe_gate_logits(r["x"], r["wg"], sh, r["z"])
            moe.moe_route_logits(r["z"], r["bias"], sh, co, r["idx"], r["w"], r["counts"])
            moe.moe_route_logits_backward(r["z"], r["idx"], r["dw"], None, sh, co, r["dz"])
        calls()
        torch.cuda.synchronize()
        r["want"] = [r[n].clone() for n in ("z", "idx", "w", "counts", "dz")]
        with torch.cuda.graph(r["graph"], stream=r["stream"]):
            calls()
        runs.append(r)
    for r in runs:
        for n in ("z", "w", "dz"):
            r[n].fill_(float("nan"))
        r["idx"].fill_(-7)
        r["counts"].fill_(-7)
    torch.cuda.synchronize()
    two = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i, r in enumerate(runs):
            with torch.cuda.stream(two[i % 2]):
                r["graph"].replay()
    torch.cuda.synchronize()
    for r in runs:
        for n, want in zip(("z", "idx", "w", "counts", "dz"), r["want"]):
            assert torch.equal(r[n], want), n
        check_route(r["z"], r["bias"], r["idx"].shape[1], o, tuple(r[n].cpu().numpy() for n in ("idx", "w", "counts")))
    check_status()
