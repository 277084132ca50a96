"""Host-side checks of the routing-from-logits and saved-activation calls: every
refusal comes back before anything reaches a device."""
import ctypes
import os

import pytest

import fine_grained_moe_gate_b200 as moe

INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 1, 2, 3, 4
FAKE = 1 << 20  # a 16-byte aligned non-null "pointer" never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(moe.LIB_PATH):
        from fine_grained_moe_gate_b200 import build
        build.build()
    return moe.lib()


def shape(**kw):
    base = dict(T=128, d=256, E=16, k=4, I=128, S=1, Is=128, dtype=moe.MOE_BF16)
    base.update(kw)
    return moe.MoEShape(*[base[n] for n, _ in moe.MoEShape._fields_])


def opts(**kw):
    base = dict(score=0, groups=4, top_groups=2, group_top=2, renormalize=1, scale=1.0)
    base.update(kw)
    return moe.MoERouteOpts(*[base[n] for n, _ in moe.MoERouteOpts._fields_])


def c(v):
    return None if v is None else ctypes.c_void_p(v)


def _route(L, sh, o, **ptr):
    p = dict(z=FAKE, bias=FAKE, idx=FAKE, w=FAKE, counts=FAKE)
    p.update(ptr)
    return L.moe_route_logits(c(p["z"]), c(p["bias"]), sh, o, c(p["idx"]), c(p["w"]), c(p["counts"]), None)


def _route_bwd(L, sh, o, **ptr):
    p = dict(z=FAKE, idx=FAKE, dw=FAKE, ds=None, dz=FAKE)
    p.update(ptr)
    return L.moe_route_logits_backward(c(p["z"]), c(p["idx"]), c(p["dw"]), c(p["ds"]), sh, o, c(p["dz"]), None)


BAD_OPTS = [
    (dict(score=2), INVALID), (dict(score=-1), INVALID), (dict(groups=0), INVALID), (dict(groups=5), INVALID),
    (dict(top_groups=0), INVALID), (dict(top_groups=5), INVALID), (dict(group_top=0), INVALID),
    (dict(group_top=3), INVALID), (dict(renormalize=2), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(groups=16, top_groups=3), INVALID),  # 3 experts kept, 4 wanted
]


@pytest.mark.parametrize("bad,code", BAD_OPTS)
def test_route_refuses_bad_options(L, bad, code):
    assert _route(L, shape(), opts(**bad)) == code
    assert _route_bwd(L, shape(), opts(**bad)) == code


def test_route_refuses_too_many_groups(L):
    assert _route(L, shape(E=64), opts(groups=64, top_groups=8)) == UNSUPPORTED


@pytest.mark.parametrize("bad,code", [
    (dict(k=0), INVALID), (dict(k=17, E=32), UNSUPPORTED), (dict(k=5, E=4), INVALID), (dict(E=300), UNSUPPORTED),
    (dict(T=-1), INVALID), (dict(dtype=7), INVALID),
])
def test_route_refuses_bad_shapes(L, bad, code):
    o = opts(groups=1, top_groups=1)
    assert _route(L, shape(**bad), o) == code
    assert _route_bwd(L, shape(**bad), o) == code


@pytest.mark.parametrize("name", ["z", "idx", "w", "counts"])
def test_route_refuses_null_and_misaligned(L, name):
    assert _route(L, shape(), opts(), **{name: None}) == INVALID
    assert _route(L, shape(), opts(), **{name: FAKE + 8}) == ALIGN


@pytest.mark.parametrize("name", ["z", "idx", "dw", "dz"])
def test_route_backward_refuses_null_and_misaligned(L, name):
    assert _route_bwd(L, shape(), opts(), **{name: None}) == INVALID
    assert _route_bwd(L, shape(), opts(), **{name: FAKE + 4}) == ALIGN
    assert _route_bwd(L, shape(), opts(), ds=FAKE + 4) == ALIGN


def test_gate_logits_refusals(L):
    f = lambda sh, x=FAKE, w=FAKE, z=FAKE: L.moe_gate_logits(c(x), c(w), sh, c(z), None)
    assert f(shape(), x=None) == INVALID and f(shape(), w=None) == INVALID and f(shape(), z=None) == INVALID
    assert f(shape(), z=FAKE + 4) == ALIGN and f(shape(), x=FAKE + 2) == ALIGN
    assert f(shape(d=96)) == UNSUPPORTED


def _saved(**kw):
    p = {n: FAKE for n, _ in moe.MoESavedActs._fields_}
    p.update(kw)
    return moe.MoESavedActs(**p)


def _up(L, sh, saved, x=FAKE, h=FAKE, hs=FAKE, ws1=FAKE):
    return L.moe_ffn_up_save(c(FAKE), c(FAKE), c(FAKE), c(FAKE), c(x), c(ws1), c(FAKE), sh, c(h), c(hs),
                             ctypes.byref(saved) if saved is not None else None, None)


def test_up_save_refusals(L):
    assert _up(L, shape(), None) == INVALID
    for name, _ in moe.MoESavedActs._fields_:
        assert _up(L, shape(), _saved(**{name: None})) == INVALID, name
        assert _up(L, shape(), _saved(**{name: FAKE + 8})) == ALIGN, name
    assert _up(L, shape(), _saved(), h=None) == INVALID
    assert _up(L, shape(), _saved(), hs=None) == INVALID
    assert _up(L, shape(), _saved(), ws1=None) == INVALID
    assert _up(L, shape(dtype=moe.MOE_F32), _saved()) == UNSUPPORTED
    assert _up(L, shape(dtype=moe.MOE_FP8_E4M3), _saved()) == UNSUPPORTED
    assert _up(L, shape(I=96), _saved()) == UNSUPPORTED


def _bwd(L, sh, saved, expert_set=0, **ptr):
    p = dict(u=FAKE, perm=FAKE, w=FAKE, dadg=FAKE, h=None, dw=FAKE)
    p.update(ptr)
    return L.moe_swiglu_backward_saved(ctypes.byref(saved) if saved is not None else None, sh, expert_set, c(p["u"]),
                                       c(p["perm"]), c(p["w"]), c(p["dadg"]), c(p["h"]), c(p["dw"]), None)


def test_swiglu_backward_refusals(L):
    assert _bwd(L, shape(), None) == INVALID
    assert _bwd(L, shape(), _saved(), expert_set=2) == INVALID
    assert _bwd(L, shape(S=0), _saved(), expert_set=1) == INVALID
    for name in ("u", "perm", "w", "dadg", "dw"):
        assert _bwd(L, shape(), _saved(), **{name: None}) == INVALID, name
        assert _bwd(L, shape(), _saved(), **{name: FAKE + 8}) == ALIGN, name
    assert _bwd(L, shape(), _saved(), h=FAKE + 8) == ALIGN
    for name in ("a", "a_scale", "g", "g_scale"):
        assert _bwd(L, shape(), _saved(**{name: None})) == INVALID
    for name in ("sa", "sa_scale", "sg", "sg_scale"):
        assert _bwd(L, shape(), _saved(**{name: None}), expert_set=1) == INVALID
    assert _bwd(L, shape(dtype=moe.MOE_F32), _saved()) == UNSUPPORTED


def test_binding_helpers():
    with pytest.raises(ValueError):
        moe.route_opts("relu")
    o = moe.route_opts("softmax", groups=8, top_groups=3, renormalize=False, scale=16.0)
    assert (o.score, o.groups, o.top_groups, o.group_top, o.renormalize, o.scale) == (1, 8, 3, 1, 0, 16.0)
    buf = moe.saved_act_buffers(shape(S=0), "cpu")
    assert set(buf) == {"a", "a_scale", "g", "g_scale"}
    assert buf["a"].shape == (512, 128) and buf["a_scale"].numel() == 512 * 4
    buf = moe.saved_act_buffers(shape(S=2), "cpu")
    assert buf["sg"].shape == (128, 256) and buf["sg_scale"].numel() == 2 * 128 * 4
    s = moe.saved_acts(buf)
    assert s.sa == buf["sa"].data_ptr()


def test_layer_refusals(L):
    sh, need = shape(), moe.moe_workspace_size(shape())

    def fwd(sh=sh, o=opts(), saved=_saved(), bias=FAKE, logits=FAKE, ws=FAKE, n=need, ws1=FAKE):
        return L.moe_layer_forward_logits(c(FAKE), c(FAKE), c(bias), c(FAKE), c(FAKE), c(FAKE), c(ws1), c(FAKE), c(FAKE),
                                          sh, o, c(FAKE), c(logits), c(FAKE), c(FAKE), c(FAKE),
                                          ctypes.byref(saved) if saved is not None else None, c(ws), n, None)

    assert fwd(o=opts(groups=3)) == INVALID
    assert fwd(logits=None) == INVALID and fwd(ws1=None) == INVALID
    assert fwd(logits=FAKE + 4) == ALIGN and fwd(bias=FAKE + 4) == ALIGN
    assert fwd(n=need - 256) == WORKSPACE and fwd(ws=None) == WORKSPACE and fwd(ws=FAKE + 16) == ALIGN
    assert fwd(saved=_saved(sg=None)) == INVALID and fwd(saved=_saved(g_scale=FAKE + 4)) == ALIGN
    assert fwd(sh=shape(dtype=moe.MOE_F32)) == UNSUPPORTED  # saved activations are a bf16 layer's
    assert fwd(sh=shape(dtype=moe.MOE_FP8_E4M3), saved=None) == UNSUPPORTED

    def bwd(sh=sh, o=opts(), saved=_saved(), logits=FAKE, ds=None, alpha=0.0, seq=0, n=None, dx=FAKE):
        if n is None:
            n = moe.moe_backward_logits_workspace_size(sh, seq, saved is not None)
        return L.moe_layer_backward_logits(*[c(FAKE)] * 8, sh, o, ctypes.byref(saved) if saved is not None else None,
                                           c(logits), c(FAKE), c(FAKE), c(FAKE), c(ds), c(FAKE), alpha, seq, c(dx),
                                           *[c(FAKE)] * 7, None, c(FAKE), n, None)

    assert bwd(o=opts(scale=float("inf"))) == INVALID
    assert bwd(logits=None) == INVALID and bwd(dx=None) == INVALID and bwd(saved=_saved(a=None)) == INVALID
    assert bwd(logits=FAKE + 4) == ALIGN and bwd(ds=FAKE + 4) == ALIGN
    assert bwd(alpha=-1.0) == INVALID and bwd(alpha=0.1, seq=0) == INVALID and bwd(alpha=0.1, seq=100) == INVALID
    assert bwd(n=moe.moe_backward_logits_workspace_size(sh, 0, True) - 256) == WORKSPACE
    assert bwd(alpha=0.1, seq=64, n=moe.moe_backward_logits_workspace_size(sh, 0, True)) == WORKSPACE
    assert bwd(sh=shape(d=192)) == UNSUPPORTED  # saved activations need the tensor-core widths
    assert bwd(sh=shape(dtype=moe.MOE_F32)) == UNSUPPORTED
    assert moe.moe_backward_logits_workspace_size(shape(d=192), 0, True) == 0
    assert moe.moe_backward_logits_workspace_size(shape(d=192), 0, False) > 0
    full, less = (moe.moe_backward_logits_workspace_size(sh, 0, f) for f in (False, True))
    assert full - less >= 2 * 4 * (512 * 128 + 128 * 128)  # no fp32 a and g


def test_binding_refuses_wrong_tensors():
    """Type, size, strides and device of the tensors, before the library is called (no GPU needed)."""
    import torch
    sh = shape()
    z, idx, w, n = torch.zeros(128, 16), torch.zeros(128, 4, dtype=torch.int32), torch.zeros(128, 4), 16
    counts = torch.zeros(n, dtype=torch.int32)
    o = moe.route_opts()

    def refused(match, **kw):
        a = dict(logits=z, bias=None, idx=idx, w=w, counts=counts)
        a.update(kw)
        with pytest.raises(moe.MoEError, match=match) as e:
            moe.moe_route_logits(a["logits"], a["bias"], sh, o, a["idx"], a["w"], a["counts"])
        assert e.value.status == INVALID

    refused("logits must be float32", logits=z.double())
    refused("logits must be contiguous", logits=torch.zeros(16, 128).t())
    refused("logits must be contiguous with at least 2048", logits=z[:100])
    refused("logits must be contiguous", logits=torch.zeros(128, 32)[:, :16])
    refused("one CUDA device", logits=z)
    bf = torch.zeros(128 * 256, dtype=torch.bfloat16)
    with pytest.raises(moe.MoEError, match="x must be bfloat16"):
        moe.moe_gate_logits(bf.float(), bf, sh, z)
    with pytest.raises(moe.MoEError, match="dlogits|logits"):
        moe.moe_route_logits_backward(z, idx, w, None, sh, o, z.half())
    with pytest.raises(moe.MoEError, match="x_perm"):
        moe.moe_ffn_up_save(bf, counts, bf, bf, None, None, None, sh, bf, None, _saved())
    with pytest.raises(moe.MoEError, match="u must be float32"):
        moe.moe_swiglu_backward_saved(_saved(), sh, moe.MOE_ROUTED, bf, idx, w, bf, None, w)
    with pytest.raises(moe.MoEError, match="x must be"):
        moe.moe_layer_forward_logits(bf[:5], bf, None, bf, bf, bf, bf, bf, bf, sh, o, bf, z, idx, w, counts, None, bf)
    with pytest.raises(moe.MoEError, match="x must be"):
        moe.moe_layer_backward_logits(bf[:5], *[bf] * 7, sh, o, None, z, idx, w, counts, None, z, 0.0, 0, *[z] * 9, bf)


def test_refuses_more_tokens_than_tiles_can_count(L):
    sh = shape(T=(1 << 31) - 255, E=2, k=1)
    o = opts(groups=1, top_groups=1)
    assert _route(L, sh, o) == UNSUPPORTED
    assert _route_bwd(L, sh, o) == UNSUPPORTED
    assert L.moe_gate_logits(c(FAKE), c(FAKE), sh, c(FAKE), None) == UNSUPPORTED


def test_saved_act_tensors_are_checked():
    import torch
    sh = shape()
    buf = moe.saved_act_buffers(sh, "cpu")
    with pytest.raises(moe.MoEError, match="device"):
        moe.moe_swiglu_backward_saved(moe.saved_acts(buf), sh, moe.MOE_ROUTED, FAKE, FAKE, FAKE, FAKE, None, FAKE, stream=0)
    with pytest.raises(moe.MoEError, match="contiguous"):
        moe.saved_acts({"a": torch.empty((4, 8), dtype=torch.uint8).t()})
    # buffers of a smaller layer, taken for ones on a device
    small = moe.saved_acts(moe.saved_act_buffers(shape(I=128, T=127), "cpu"))
    small.device = 0
    for part in (moe.MOE_SHARED, moe.MOE_ROUTED):
        with pytest.raises(moe.MoEError, match="need"):
            moe.moe_swiglu_backward_saved(small, sh, part, FAKE, FAKE, FAKE, FAKE, None, FAKE, stream=0)
    with pytest.raises(moe.MoEError, match="need"):
        moe.moe_ffn_up_save(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, sh, FAKE, FAKE, small, stream=0)
    # one short scale buffer
    buf["sg_scale"] = buf["sg_scale"][:-1]
    short = moe.saved_acts(buf)
    short.device = 0
    with pytest.raises(moe.MoEError, match="need"):
        moe.moe_swiglu_backward_saved(short, sh, moe.MOE_SHARED, FAKE, None, None, FAKE, None, None, stream=0)
