"""GPU parity of moe_ffn_up_save and moe_swiglu_backward_saved against
oracle/training.py and the C oracle's quantizer.

Pages cited (title, section): "DeepSeek V3 From Scratch", "The idea" (FP8 with
fine-grained quantization tiles); "Scaling Efficiency: A Deep Dive into the
DeepSeek-V3 Architecture", DeepSeekMoE sketch (SwiGLU experts).

On inputs of few bits every partial sum of a and g is exact, and the codes and
scales equal the quantizer's bit for bit; h and hs are moe_ffn_up's bits always.
SwiGLU backward, u = 2^-24: outputs are rounded to bf16 (half a step: 2^-8
relative); before that the sigmoid carries the exponential's two ulps, an
addition and a division (8u) and the products a few u more; 1 + a (1 - s)
cancels, so da is held to 2^-8 |da| + 32u |dh g s| (1 + |a|), dg and h to
(2^-8 + 32u).  dw: 32u per product, and a lane's n / 32 additions and 5 across
lanes: (n / 32 + 48) u sum |u h|.  Results below 2^-120 may underflow.
"""
import numpy as np
import pytest
import torch

import fine_grained_moe_gate_b200 as moe
import oracle
from oracle import training as ot

from gpu_harness import DEV, check_status

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -120
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _clean_status():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    moe.moe_get_last_error()
    yield


def make_rows(T, E, k, seed, only=None):
    """offsets, perm_tok of an uneven routing (only: every token to these experts)."""
    rng = np.random.default_rng(seed)
    pick = np.arange(E) if only is None else np.asarray(only)
    idx = np.stack([rng.permutation(pick)[:k] for _ in range(T)]).reshape(-1) if T else np.zeros(0, np.int64)
    perm = np.argsort(idx, kind="stable").astype(np.int32)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(idx, minlength=E))]).astype(np.int32)
    return torch.from_numpy(offsets).to(DEV), torch.from_numpy(perm).to(DEV)


def grid(shape, g, mul, step):
    return (torch.round(torch.randn(shape, generator=g, device=DEV) * mul) * step).to(BF)


def make_up(T, d, E, k, I, S, Is, seed, on_grid=True, only=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    sh = moe.MoEShape(T, d, E, k, I, S, Is, moe.MOE_BF16)
    offsets, perm = make_rows(T, E, k, seed, only)
    new = (lambda s, m, st: grid(s, g, m, st)) if on_grid else (
        lambda s, m, st: (torch.randn(s, generator=g, device=DEV) * m * st).to(BF))
    x = new((T, d), 16, 2.0 ** -4)
    w = {n: new(s, 20, 2.0 ** -10) for n, s in (("w1", (E, I, d)), ("w3", (E, I, d)), ("ws1", (S * Is, d)),
                                                ("ws3", (S * Is, d)))}
    return sh, offsets, perm, x, x[perm.long() // k], w


def run_up(sh, offsets, x, x_perm, w, shared=True):
    rows, SI = sh.T * sh.k, sh.S * sh.Is
    nan = lambda r, c: torch.full((r, c), float("nan"), device=DEV, dtype=BF)
    h, hs = nan(rows, sh.I), nan(sh.T, SI)
    buf = moe.saved_act_buffers(sh, DEV)
    for t in buf.values():
        t.fill_(0xAB)
    shared = shared and sh.S > 0
    sx = (x, w["ws1"], w["ws3"]) if shared else (None, None, None)
    moe.moe_ffn_up_save(x_perm, offsets, w["w1"], w["w3"], *sx, sh, h, hs if shared else None, moe.saved_acts(buf))
    torch.cuda.synchronize()
    check_status()
    h2, hs2 = torch.empty_like(h), torch.empty_like(hs)
    moe.moe_ffn_up(x_perm, offsets, w["w1"], w["w3"], *sx, sh, h2, hs2 if shared else None)
    torch.cuda.synchronize()
    assert torch.equal(h.view(torch.int16), h2.view(torch.int16))
    if shared:
        assert torch.equal(hs.view(torch.int16), hs2.view(torch.int16))
    return h, hs, buf


def preact(sh, offsets, x, x_perm, w):
    """a, g of the routed and of the shared rows, float64."""
    off = offsets.tolist()
    xp, xd = x_perm.double(), x.double()
    out = {}
    for n, wn in (("a", "w1"), ("g", "w3")):
        out[n] = torch.cat([xp[off[e]:off[e + 1]] @ w[wn][e].double().t() for e in range(sh.E)]).cpu().numpy()
        out["s" + n] = (xd @ w["ws" + wn[1]].double().t()).cpu().numpy()
    return out


UP = {
    "one_token": dict(T=1, d=64, E=4, k=2, I=128, S=1, Is=128),
    "ragged": dict(T=37, d=192, E=16, k=4, I=256, S=2, Is=128),
    "odd_halves": dict(T=130, d=128, E=12, k=3, I=384, S=0, Is=128),
    "several_tiles": dict(T=700, d=256, E=4, k=2, I=256, S=1, Is=384),
    "wide": dict(T=96, d=2048, E=64, k=6, I=1408, S=2, Is=1408),
}


@pytest.mark.parametrize("name", list(UP))
def test_up_save_codes_equal_the_quantizers(name):
    c = UP[name]
    sh, offsets, perm, x, x_perm, w = make_up(seed=c["T"], **c)
    _, _, buf = run_up(sh, offsets, x, x_perm, w)
    ref = preact(sh, offsets, x, x_perm, w)
    for n in ("a", "g") + (("sa", "sg") if sh.S else ()):
        codes, eb = oracle.quantize_mx(ref[n].astype(np.float32))
        rows, cols = codes.shape
        words = np.transpose(eb.reshape(rows, cols // 128, 4), (1, 0, 2))
        assert (buf[n].cpu().numpy() == codes).all(), n
        assert (buf[n + "_scale"].cpu().numpy().reshape(cols // 128, rows, 4) == words).all(), n


def test_up_save_empty_experts_and_routed_only():
    c = dict(T=50, d=128, E=8, k=2, I=128, S=1, Is=128)
    sh, offsets, perm, x, x_perm, w = make_up(seed=3, only=[1, 6], **c)
    _, _, buf = run_up(sh, offsets, x, x_perm, w, shared=False)
    ref = preact(sh, offsets, x, x_perm, w)
    codes, _ = oracle.quantize_mx(ref["a"].astype(np.float32))
    assert (buf["a"].cpu().numpy() == codes).all()
    assert (buf["sa"] == 0xAB).all() and (buf["sg_scale"] == 0xAB).all()  # left as they were


@pytest.mark.parametrize("name", ["ragged", "several_tiles"])
def test_up_save_random_inputs(name):
    """Any bf16 inputs: the values stand within half a code step of a (2^-4 relative, or half the smallest step
    2^-9 of the tile's scale) plus the sums' error, d * 2^-23 * sum |x w| (truncating adders)."""
    c = UP[name]
    sh, offsets, perm, x, x_perm, w = make_up(seed=7, on_grid=False, **c)
    _, _, buf = run_up(sh, offsets, x, x_perm, w)
    ref = preact(sh, offsets, x, x_perm, w)
    mag = preact(sh, offsets, x.abs(), x_perm.abs(), {n: t.abs() for n, t in w.items()})
    for n in ("a", "g", "sa", "sg"):
        rows, cols = ref[n].shape
        words = buf[n + "_scale"].cpu().numpy()
        val = ot.dequantize(buf[n].cpu().numpy(), words)
        acc = sh.d * 2.0 ** -23 * mag[n]
        e = np.transpose(words.reshape(cols // 128, rows, 4), (1, 0, 2)).reshape(rows, cols // 32).astype(int) - 127
        step = np.repeat(np.ldexp(1.0, e - 10), 32, axis=1)
        assert (np.abs(val - ref[n]) <= np.maximum(2.0 ** -4 * (np.abs(ref[n]) + acc), step) + acc).all()
        lim = np.abs(ref[n]).reshape(rows, -1, 32).max(axis=2)
        slack = acc.reshape(rows, -1, 32).max(axis=2)
        assert (lim <= np.ldexp(448.0, e) + slack).all() and (lim >= np.ldexp(224.0, e) - slack).all()


def test_up_save_no_tokens():
    c = dict(T=0, d=128, E=4, k=2, I=128, S=0, Is=128)
    sh, offsets, perm, x, x_perm, w = make_up(seed=1, **c)
    moe.moe_ffn_up_save(None, offsets, w["w1"], w["w3"], None, None, None, sh, None, None, moe.MoESavedActs())
    check_status()


# ---------------------------------------------------------------- SwiGLU backward

def make_saved(rows, n, seed, std=2.0):
    rng = np.random.default_rng(seed)
    out = {}
    for name in ("a", "g"):
        v = (rng.normal(size=(rows, n)) * std).astype(np.float32)
        if rows:
            v[0, :32] = 0.0                      # an all-zero tile
            v[rows // 2, 32:64] *= 1e3           # saturated gates
            v[rows - 1, -32:] *= 1e-30
        codes, eb = oracle.quantize_mx(v)
        words = np.transpose(eb.reshape(rows, n // 128, 4), (1, 0, 2)).copy()
        out[name], out[name + "_scale"] = codes, words
    return out


def check_bwd(sh, expert_set, seed, want_h=True, std=2.0, bad=None):
    shared = expert_set == moe.MOE_SHARED
    rows, n = (sh.T, sh.S * sh.Is) if shared else (sh.T * sh.k, sh.I)
    sv = make_saved(rows, n, seed, std)
    pre = "s" if shared else ""
    dev = {pre + k_: torch.from_numpy(v).to(DEV) for k_, v in sv.items()}
    rng = np.random.default_rng(seed + 1)
    un = rng.normal(size=(rows, n)).astype(np.float32)
    perm = rng.permutation(rows).astype(np.int32)
    wn = rng.uniform(size=rows).astype(np.float32)
    if bad is not None:
        perm[bad[0]] = bad[1]
    u, pt, w = (torch.from_numpy(v).to(DEV) for v in (un, perm, wn))
    dadg = torch.full((rows, 2 * n), float("nan"), device=DEV, dtype=BF)
    h = torch.full((rows, n), float("nan"), device=DEV, dtype=BF) if want_h else None
    dw = torch.full((rows,), -7.0, device=DEV)
    moe.moe_swiglu_backward_saved(moe.saved_acts(dev), sh, expert_set, u, None if shared else pt,
                                  None if shared else w, dadg, h, None if shared else dw)
    torch.cuda.synchronize()
    a, g = (ot.dequantize(sv[x], sv[x + "_scale"]) for x in ("a", "g"))
    ok = (perm >= 0) & (perm < rows)
    wt = np.ones(rows) if shared else np.where(ok, wn[np.where(ok, perm, 0)], 0.0)
    da, dg, hr, dot = ot.swiglu_backward(a, g, un, wt)
    s = 1 / (1 + np.exp(-np.clip(a, -700, 700)))
    got = dadg.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    base = np.abs(wt[:, None] * un * g * s) * (1 + np.abs(a))
    assert (np.abs(got[:, :n] - da) <= 2.0 ** -8 * np.abs(da) + 32 * U * base + TINY).all()
    assert (np.abs(got[:, n:] - dg) <= (2.0 ** -8 + 32 * U) * np.abs(dg) + TINY).all()
    if want_h:
        hh = h.float().cpu().numpy().astype(np.float64)
        assert (np.abs(hh - hr) <= (2.0 ** -8 + 32 * U) * np.abs(hr) + TINY).all()
    if not shared:
        d = dw.cpu().numpy()
        mag = np.abs(un * hr).sum(axis=1)
        for r in range(rows):
            if ok[r]:
                assert abs(d[perm[r]] - dot[r]) <= (n / 32 + 48) * U * mag[r] + TINY, r
    return got, dw.cpu().numpy(), perm


@pytest.mark.parametrize("T,k,I", [(1, 1, 128), (3, 2, 128), (9, 3, 256), (50, 4, 384), (40, 6, 1408), (33, 8, 2048)])
@pytest.mark.parametrize("want_h", [True, False])
def test_swiglu_backward_routed(T, k, I, want_h):
    check_bwd(moe.MoEShape(T, 128, 16, k, I, 0, 128, moe.MOE_BF16), moe.MOE_ROUTED, T + I, want_h)
    check_status()


@pytest.mark.parametrize("T,S,Is", [(1, 1, 128), (50, 2, 384), (130, 1, 1408)])
def test_swiglu_backward_shared(T, S, Is):
    check_bwd(moe.MoEShape(T, 128, 16, 2, 128, S, Is, moe.MOE_BF16), moe.MOE_SHARED, T + Is)
    check_status()


def test_swiglu_backward_small_and_large_values():
    sh = moe.MoEShape(20, 128, 16, 2, 256, 0, 128, moe.MOE_BF16)
    check_bwd(sh, moe.MOE_ROUTED, 1, std=2.0 ** -100)
    check_bwd(sh, moe.MOE_ROUTED, 2, std=40.0)
    check_status()


def test_swiglu_backward_bad_permutation_entry():
    sh = moe.MoEShape(20, 128, 16, 2, 128, 0, 128, moe.MOE_BF16)
    for v in (-1, 40):
        got, _, _ = check_bwd(sh, moe.MOE_ROUTED, 5, bad=(3, v))
        assert (got[3] == 0).all()
        assert moe.moe_get_last_error() == 6


def test_swiglu_backward_against_differences():
    """L = sum_q w_q <u_r, h(a, g)> with the saved a moved by one code: dL / da from dadg within the second
    difference.  The move is one step up and one down of the same code, h evaluated in 64 bits."""
    sh = moe.MoEShape(2, 128, 4, 1, 128, 0, 128, moe.MOE_BF16)
    sv = make_saved(2, 128, 9)
    a, g = (ot.dequantize(sv[x], sv[x + "_scale"]) for x in ("a", "g"))
    u = np.random.default_rng(10).normal(size=(2, 128)).astype(np.float32)
    w = np.array([0.75, 0.5], np.float32)
    dev = {k_: torch.from_numpy(v).to(DEV) for k_, v in sv.items()}
    dadg = torch.empty((2, 256), device=DEV, dtype=BF)
    dw = torch.empty(2, device=DEV)
    moe.moe_swiglu_backward_saved(moe.saved_acts(dev), sh, moe.MOE_ROUTED, torch.from_numpy(u).to(DEV),
                                  torch.arange(2, dtype=torch.int32, device=DEV), torch.from_numpy(w).to(DEV), dadg,
                                  None, dw)
    got = dadg.float().cpu().numpy()
    f = lambda x, y: w[:, None] * u * y * x / (1 + np.exp(-x))
    e = 1e-4
    num = (f(a + e, g) - f(a - e, g)) / (2 * e)
    numg = (f(a, g + e) - f(a, g - e)) / (2 * e)
    # truncation e^2 / 6 |f'''| <= 1e-8 |u g| (|silu'''| <= 0.6); bf16 half a step
    np.testing.assert_array_less(np.abs(got[:, :128] - num), 2.0 ** -8 * np.abs(num) + 1e-6 * np.abs(u * g) + 1e-9)
    np.testing.assert_array_less(np.abs(got[:, 128:] - numg), 2.0 ** -8 * np.abs(numg) + 1e-6 * np.abs(u * a) + 1e-9)
