"""GPU parity of the layer with routing from logits (moe_layer_forward_logits,
moe_layer_backward_logits): the operators run together as a training step runs
them, in every form of the gate, with activations saved in 8 bits or recomputed.

Pages cited (title, section): "DeepSeek V3 From Scratch", "In code" (route) and
"The idea" (fine-grained FP8 tiles); "Scaling Efficiency: A Deep Dive into the
DeepSeek-V3 Architecture", DeepSeekMoE sketch; kbwen.com DeepSeek tag page,
"A bias term for each expert" (the complementary balance loss).

Bars, as the layer's own parity tests derive them: the bf16 output 5e-3
relative Frobenius; gradients 2e-5 (fp32 layer), 5e-3 (bf16 on the tensor
cores: operands rounded to bf16, 2^-9 RMS each, twice for dx).  The reference
of a backward with saved activations uses the values the codes stand for, so
the bar stays the same: only the rounding of the operands is left.
"""
import dataclasses

import numpy as np
import pytest
import torch

import fine_grained_moe_gate_b200 as moe
import oracle
from fine_grained_moe_gate_b200.inputs import CONFIGS, make_layer, make_tokens, to_numpy
from oracle import backward as ob
from oracle import training as ot

from gpu_harness import DEV, as_f64, check_status, rel_fro

pytestmark = pytest.mark.gpu

NAMES = ("dx", "dw_gate", "dw1", "dw3", "dw2", "dws1", "dws3", "dws2")
OPTS = {
    "sigmoid": ot.Opts(),
    "groups": ot.Opts(groups=4, top_groups=2, group_top=2, scale=2.5),
    "softmax": ot.Opts(score="softmax"),
    "softmax_as_scored": ot.Opts(score="softmax", renormalize=False, scale=4.0),
    "sigmoid_as_scored": ot.Opts(renormalize=False, scale=1.5),
}
SHAPES = {
    "tc": dict(dtype="bf16", T=200, d=256, E=16, k=4, I=256, S=2, Is=128),
    "tc_no_shared": dict(dtype="bf16", T=130, d=128, E=12, k=3, I=128, S=0, Is=128),
    "simt_bf16": dict(dtype="bf16", T=96, d=192, E=8, k=2, I=128, S=1, Is=128),
    "f32": dict(dtype="f32", T=50, d=40, E=8, k=3, I=24, S=1, Is=16),
}


@pytest.fixture(autouse=True)
def _clean_status():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    moe.moe_get_last_error()
    yield


def c_opts(o):
    return moe.route_opts(o.score, o.groups, o.top_groups, o.group_top, o.renormalize, o.scale)


class Layer:
    """A layer's inputs, and one forward and backward through the calls."""

    def __init__(self, shape, o, save, seed=3, bias=True):
        self.o, self.c = o, c_opts(o)
        self.cfg = CONFIGS["small_bf16"].scaled(name="logits", w_std=0.05, bias_kind="uniform", bias_range=0.02, seed=seed,
                                                **shape)
        self.sh = moe.shape_of(self.cfg)
        self.p = make_layer(self.cfg, DEV)
        self.x = make_tokens(self.cfg, DEV)
        self.bias = self.p["bias"] if bias else None
        T, E, k, d = self.cfg.T, self.cfg.E, self.cfg.k, self.cfg.d
        self.y = torch.full((T, d), float("nan"), dtype=self.x.dtype, device=DEV)
        self.logits = torch.full((T, E), float("nan"), device=DEV)
        self.idx = torch.empty((T, k), dtype=torch.int32, device=DEV)
        self.w = torch.empty((T, k), device=DEV)
        self.counts = torch.empty(E, dtype=torch.int32, device=DEV)
        self.buf = moe.saved_act_buffers(self.sh, DEV) if save else None
        self.saved = moe.saved_acts(self.buf) if save else None
        self.ws = torch.empty(moe.moe_workspace_size(self.sh), dtype=torch.uint8, device=DEV)
        self.dy = torch.randn((T, d), generator=torch.Generator(device=DEV).manual_seed(seed + 101), device=DEV)

    def shared(self):
        return [self.p[n] if self.cfg.S else None for n in ("ws1", "ws3", "ws2")]

    def forward(self):
        p = self.p
        moe.moe_layer_forward_logits(self.x, p["w_gate"], self.bias, p["w1"], p["w3"], p["w2"], *self.shared(), self.sh,
                                     self.c, self.y, self.logits, self.idx, self.w, self.counts, self.saved, self.ws)

    def alloc_backward(self, alpha, L):
        T, d, E, I, S, Is = (getattr(self.cfg, n) for n in ("T", "d", "E", "I", "S", "Is"))
        f = lambda *s: torch.full(s, float("nan"), device=DEV)  # poisoned: every element must be written
        self.g = dict(dx=f(T, d), dw_gate=f(E, d), dw1=f(E, I, d), dw3=f(E, I, d), dw2=f(E, d, I),
                      dws1=f(S, Is, d) if S else None, dws3=f(S, Is, d) if S else None, dws2=f(S, d, Is) if S else None)
        self.loss = f(1)
        n = moe.moe_backward_logits_workspace_size(self.sh, L if alpha > 0 else 0, self.saved is not None)
        self.wsb = torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV)

    def backward(self, alpha=0.0, L=0, dscores=None):
        p = self.p
        moe.moe_layer_backward_logits(self.x, p["w_gate"], p["w1"], p["w3"], p["w2"], *self.shared(), self.sh, self.c,
                                      self.saved, self.logits, self.idx, self.w, self.counts, dscores, self.dy, alpha, L,
                                      *(self.g[n] for n in NAMES), self.loss, self.wsb)

    # ---- the oracle's side, from the tensors the calls produced

    def saved_values(self):
        out = {}
        for n in ("a", "g", "sa", "sg"):
            if self.buf is not None and n in self.buf:
                out[n] = ot.dequantize(self.buf[n].cpu().numpy(), self.buf[n + "_scale"].cpu().numpy())
        return out

    def reference(self, alpha, L, dscores):
        """Gradients by the chain rule in float64; a and g of the saved codes where there are any."""
        f64 = {n: ob.to_f64(to_numpy(t)) for n, t in self.p.items()}
        X, dY = ob.to_f64(to_numpy(self.x)), self.dy.cpu().numpy().astype(np.float64)
        idx, w = self.idx.cpu().numpy(), self.w.cpu().numpy().astype(np.float64)
        z = self.logits.cpu().numpy()
        sv = self.saved_values()
        T, k = idx.shape
        bf = self.cfg.dtype == "bf16"
        rnd = (lambda v: ob.round_like(v, True)) if bf else (lambda v: v)
        out = {n: np.zeros(f64[m].shape) for n, m in (("dw1", "w1"), ("dw3", "w3"), ("dw2", "w2"))}
        dX, dw, row = np.zeros_like(X), np.zeros((T, k)), 0
        for e in range(self.cfg.E):
            tt, jj = np.nonzero(idx == e)
            n = tt.size
            a, g = X[tt] @ f64["w1"][e].T, X[tt] @ f64["w3"][e].T
            if sv:
                a, g = sv["a"][row:row + n], sv["g"][row:row + n]
            row += n
            u = dY[tt] @ f64["w2"][e]
            da, dg, h, dot = ot.swiglu_backward(a, g, u, w[tt, jj])
            # recomputed, h is rounded as the forward rounds it; saved, it is a s g of the codes
            dw[tt, jj] = dot if sv else (u * rnd(h)).sum(axis=1)
            out["dw2"][e] = (w[tt, jj][:, None] * dY[tt]).T @ rnd(h)
            out["dw1"][e], out["dw3"][e] = da.T @ X[tt], dg.T @ X[tt]
            np.add.at(dX, tt, da @ f64["w1"][e] + dg @ f64["w3"][e])
        S, Is = self.cfg.S, self.cfg.Is
        if S:
            out.update({n: np.zeros(f64[m].shape) for n, m in (("dws1", "ws1"), ("dws3", "ws3"), ("dws2", "ws2"))})
        for s in range(S):
            a, g = X @ f64["ws1"][s].T, X @ f64["ws3"][s].T
            if sv:
                a, g = sv["sa"][:, s * Is:(s + 1) * Is], sv["sg"][:, s * Is:(s + 1) * Is]
            da, dg, h, _ = ot.swiglu_backward(a, g, dY @ f64["ws2"][s], np.ones(T))
            out["dws2"][s] = dY.T @ rnd(h)
            out["dws1"][s], out["dws3"][s] = da.T @ X, dg.T @ X
            dX += da @ f64["ws1"][s] + dg @ f64["ws3"][s]
        ds, loss = (np.zeros((T, self.cfg.E)) if dscores is None else dscores.cpu().numpy().astype(np.float64)), 0.0
        if alpha > 0:
            loss, dsb = ob.balance_loss(ot.scores(z, self.o.score), idx, alpha, L)
            ds = ds + dsb
        dz = ot.route_backward(z, idx, dw, ds, self.o)
        out["dx"], out["dw_gate"] = dX + dz @ f64["w_gate"], dz.T @ X
        return out, loss

    def check(self, alpha=0.0, L=0, dscores=None):
        ref, loss = self.reference(alpha, L, dscores)
        c = self.cfg
        tc = c.dtype == "bf16" and all(v % 128 == 0 for v in (c.d, c.I, c.Is))
        tol = 5e-3 if tc else 2e-4 if c.dtype == "bf16" else 2e-5
        for n in NAMES:
            if self.g[n] is None:
                continue
            got = self.g[n].cpu().numpy().astype(np.float64)
            assert np.isfinite(got).all(), n
            assert rel_fro(got, ref[n]) < tol, (n, rel_fro(got, ref[n]))
        assert abs(float(self.loss.item()) - loss) <= 1e-5 * abs(loss)

    def check_forward(self):
        z = self.logits.cpu().numpy()
        zr = ob.to_f64(to_numpy(self.x)) @ ob.to_f64(to_numpy(self.p["w_gate"])).T
        assert rel_fro(z, zr) < 2e-6
        ri, rw, rc, short = ot.route(z, None if self.bias is None else self.bias.cpu().numpy(), self.cfg.k, self.o)
        assert (self.idx.cpu().numpy() == ri).all() and (self.counts.cpu().numpy() == rc).all()
        np.testing.assert_allclose(self.w.cpu().numpy(), rw, rtol=1e-5)
        n = {k_: to_numpy(t) for k_, t in self.p.items()}
        ref = oracle.layer_output(to_numpy(self.x), ri, self.w.cpu().numpy(),
                                  *(n[m] for m in ("w1", "w3", "w2", "ws1", "ws3", "ws2")))
        ref = ob.to_f64(ref)
        assert rel_fro(as_f64(self.y), ref) < (5e-3 if self.cfg.dtype == "bf16" else 1e-5)
        return short


CASES = [(s, o, save) for s in SHAPES for o in OPTS for save in (False, True) if not save or s.startswith("tc")]


@pytest.mark.parametrize("shape,name,save", CASES)
def test_training_step(shape, name, save):
    """Forward, then backward with a loss on the scores."""
    o = OPTS[name]
    L = Layer(SHAPES[shape], o, save)
    L.forward()
    torch.cuda.synchronize()
    check_status()
    assert not L.check_forward().any()
    ds = torch.randn(L.logits.shape, generator=torch.Generator(device=DEV).manual_seed(9), device=DEV) * 0.1
    L.alloc_backward(0.0, 0)
    L.backward(dscores=ds)
    torch.cuda.synchronize()
    check_status()
    L.check(dscores=ds)


@pytest.mark.parametrize("name", ["groups", "softmax_as_scored"])
@pytest.mark.parametrize("save", [False, True])
def test_balance_loss_and_score_gradient_together(name, save):
    L = Layer(SHAPES["tc"], OPTS[name], save, seed=5)
    L.forward()
    ds = torch.randn(L.logits.shape, generator=torch.Generator(device=DEV).manual_seed(9), device=DEV) * 0.1
    for d in (None, ds):
        L.alloc_backward(0.05, 20)
        L.backward(0.05, 20, d)
        torch.cuda.synchronize()
        check_status()
        L.check(0.05, 20, d)


def test_default_form_is_the_layers_own():
    """route_opts() without arguments: the same selection (where clear), output and gradients as the layer calls."""
    L = Layer(SHAPES["tc"], ot.Opts(), False, seed=6)
    L.forward()
    y, p = torch.empty_like(L.y), L.p
    idx, w, counts = torch.empty_like(L.idx), torch.empty_like(L.w), torch.empty_like(L.counts)
    moe.moe_layer_forward(L.x, p["w_gate"], L.bias, p["w1"], p["w3"], p["w2"], p["ws1"], p["ws3"], p["ws2"], L.sh, y, idx,
                          w, counts, L.ws)
    torch.cuda.synchronize()
    assert torch.equal(idx, L.idx) and torch.equal(counts, L.counts)
    assert rel_fro(as_f64(y), as_f64(L.y)) < 1e-3


def test_tokens_with_fewer_experts():
    """Experts masked through the bias until some groups are short: the tokens keep what they have, the step is
    reported, and nothing else changes."""
    o = dataclasses.replace(OPTS["groups"], top_groups=1)   # 4 groups of 4, one kept, k = 4
    for save in (False, True):
        L = Layer(SHAPES["tc"], o, save, seed=7)
        L.bias = L.bias.clone()
        L.bias[[1, 6]] = float("-inf")       # groups 0 and 1 have three experts left
        L.ws.fill_(0x5A)
        L.forward()
        torch.cuda.synchronize()
        assert moe.moe_get_last_error() == 6
        short = L.check_forward_short()
        assert short.any() and not short.all()
        L.alloc_backward(0.0, 0)
        L.backward()
        torch.cuda.synchronize()
        assert moe.moe_get_last_error() == 6
        L.check()


def _check_forward_short(self):
    z = self.logits.cpu().numpy()
    ri, rw, rc, short = ot.route(z, self.bias.cpu().numpy(), self.cfg.k, self.o)
    assert (self.idx.cpu().numpy() == ri).all() and (self.counts.cpu().numpy() == rc).all()
    f64 = {n: ob.to_f64(to_numpy(t)) for n, t in self.p.items()}
    X = ob.to_f64(to_numpy(self.x))
    swiglu = lambda x, w1, w3, w2: (lambda a, g: (a / (1 + np.exp(-a)) * g) @ w2.T)(x @ w1.T, x @ w3.T)
    y = sum(swiglu(X, f64["ws1"][s], f64["ws3"][s], f64["ws2"][s]) for s in range(self.cfg.S))
    for e in range(self.cfg.E):
        tt, jj = np.nonzero(ri == e)
        if tt.size:
            np.add.at(y, tt, rw[tt, jj][:, None] * swiglu(X[tt], f64["w1"][e], f64["w3"][e], f64["w2"][e]))
    assert rel_fro(as_f64(self.y), y) < 5e-3
    return short


Layer.check_forward_short = _check_forward_short


def test_step_in_a_graph():
    """A captured forward and backward replayed on new tokens, with another step captured beside it."""
    steps = [Layer(SHAPES["tc"], OPTS["groups"], True, seed=s) for s in (8, 9)]
    graphs = []
    for L in steps:
        L.alloc_backward(0.0, 0)
        L.forward()
        L.backward()
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            L.forward()
            L.backward()
        graphs.append(g)
    for L, n in zip(steps, (1, 2)):
        L.x.copy_(make_tokens(L.cfg, DEV, step=n))
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    check_status()
    for L in steps:
        assert not L.check_forward().any()
        L.check()


def test_no_tokens():
    L = Layer(dict(SHAPES["tc"], T=0), ot.Opts(), True)
    L.forward()
    L.alloc_backward(0.0, 0)
    L.backward()
    torch.cuda.synchronize()
    check_status()
    assert (L.counts == 0).all()
    for n in NAMES[1:5]:
        assert (L.g[n] == 0).all(), n
