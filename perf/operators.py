"""What the layer's training operators are measured on.

Five operators of one training or serving step of the fine-grained MoE layer:

  gate      gate logits z = x W_gate^T in fp32                      (moe_gate_logits)
  route     experts from logits: sigmoid or softmax scores, bias,
            groups, top-k, weights, load histogram                  (moe_route_logits)
  route_bwd the gradient of the logits                              (moe_route_logits_backward)
  up_save   gate/up projections with SwiGLU, the pre-activations
            kept in 8 bits for the backward                         (moe_ffn_up_save)
  act_bwd   the SwiGLU backward from those 8 bits                   (moe_swiglu_backward_saved)

``run`` computes them in elementary torch operations, or, with ``own`` true,
through the framework's calls.  Token and weight values of the contractions
lie on a grid of a few bits (x in steps of 2^-4, weights of 2^-10 or 2^-12),
so every partial sum is exact in 32 bits whatever its order, and what is
rounded to 8 bits after it can be compared value for value.
"""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # gate: one decoding step of 64 sequences; a prefill batch; the fp32 layer
        dict(name="gate decode", op="gate", T=64, d=7168, E=256, dtype="bf16"),
        dict(name="gate prefill", op="gate", T=8192, d=7168, E=256, dtype="bf16"),
        # route: a decoding step with group-limited sigmoid routing; the same for a prefill batch;
        # a long batch with softmax scores that are not renormalised, in groups ranked by their best expert;
        # plain softmax top-k on a small layer with experts taken out of service
        dict(name="route decode", op="route", T=64, E=256, k=8, score="sigmoid", groups=8, top_groups=4, group_top=2,
             renorm=True, scale=2.5, bias=True, masked=0, spread=1.0),
        dict(name="route prefill", op="route", T=8192, E=256, k=8, score="sigmoid", groups=8, top_groups=4,
             group_top=2, renorm=True, scale=2.5, bias=True, masked=0, spread=1.0),
        dict(name="route softmax groups", op="route", T=32768, E=160, k=6, score="softmax", groups=8, top_groups=3,
             group_top=1, renorm=False, scale=16.0, bias=False, masked=0, spread=1.5),
        dict(name="route softmax masked", op="route", T=4099, E=60, k=4, score="softmax", groups=1, top_groups=1,
             group_top=1, renorm=True, scale=1.0, bias=False, masked=7, spread=1.0),
        # route_bwd: a training batch with an auxiliary loss on the scores; a long sigmoid batch
        dict(name="route_bwd aux", op="route_bwd", T=4096, E=64, k=6, score="softmax", renorm=False, scale=1.0,
             aux=True, spread=1.0),
        dict(name="route_bwd long", op="route_bwd", T=32768, E=256, k=8, score="sigmoid", renorm=True, scale=2.5,
             aux=False, spread=1.0),
        # up_save: a small and a whole training batch of the small layer
        dict(name="up_save microbatch", op="up_save", T=96, d=2048, E=64, k=6, I=1408, S=2, Is=1408),
        dict(name="up_save batch", op="up_save", T=4096, d=2048, E=64, k=6, I=1408, S=2, Is=1408),
        # act_bwd: the routed rows of a microbatch of the small layer; of a large layer's batch
        dict(name="act_bwd microbatch", op="act_bwd", T=96, E=64, k=6, I=1408),
        dict(name="act_bwd batch", op="act_bwd", T=8192, E=256, k=8, I=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "route", "route", "route_bwd", "up_save", "act_bwd"])
    if op == "gate":
        if rng.random() < 0.25:  # the fp32 layer is a small one
            return dict(op=op, T=_log(rng, 1, 512), d=8 * rng.randint(4, 64), E=rng.randint(4, 256), dtype="f32")
        return dict(op=op, T=_log(rng, 1, 8192), d=64 * rng.randint(4, 112), E=rng.randint(8, 256), dtype="bf16")
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 6, 8])
        per = rng.randint(max(1, 16 // groups), 256 // groups)
        E = groups * per
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, top_groups * per))
        masked = rng.randint(0, E // 8) if groups == 1 and E - E // 8 >= k else 0
        return dict(op=op, T=_log(rng, 1, 32768), E=E, k=k, score=rng.choice(["sigmoid", "softmax"]), groups=groups,
                    top_groups=top_groups, group_top=rng.choice([1, 2]) if per > 1 else 1, renorm=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5, 16.0]), bias=rng.random() < 0.6, masked=masked,
                    spread=rng.choice([0.5, 1.0, 3.0]))
    if op == "route_bwd":
        E = rng.randint(8, 256)
        return dict(op=op, T=_log(rng, 1, 32768), E=E, k=rng.randint(1, min(16, E)),
                    score=rng.choice(["sigmoid", "softmax"]), renorm=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5, 16.0]), aux=rng.random() < 0.5, spread=rng.choice([0.5, 1.0, 3.0]))
    E = rng.choice([8, 16, 33, 64])
    k = rng.randint(1, 8)
    I = 128 * rng.randint(1, 11)
    if op == "up_save":
        S = rng.randint(0, 2)
        return dict(op=op, T=_log(rng, 1, 4096), d=64 * rng.randint(2, 32), E=E, k=min(k, 6), I=I, S=S,
                    Is=128 * rng.randint(1, 11))
    return dict(op=op, T=_log(rng, 1, 8192), E=E, k=k, I=I)


def work(case):
    c = dict(case)
    op, T = c["op"], c["T"]
    if op == "gate":
        eb = 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=eb * (T * c["d"] + c["E"] * c["d"]) + 4 * T * c["E"], flops=2 * T * c["d"] * c["E"])
    if op == "route":
        E, k = c["E"], c["k"]
        return dict(bytes=4 * T * E + 8 * T * k + 4 * E * (2 if c["bias"] else 1), flops=8 * T * E)
    if op == "route_bwd":
        E, k = c["E"], c["k"]
        rows = 1  # dlogits; the scores are needed whole only where a sum runs over all experts
        if c["aux"]:
            rows += 2
        elif c["score"] == "softmax" and not c["renorm"]:
            rows += 1
        return dict(bytes=4 * T * E * rows + (8 if rows > 1 else 12) * T * k, flops=(8 if rows > 1 else 1) * T * E)
    R = T * c["k"]
    if op == "up_save":
        d, E, I, SI = c["d"], c["E"], c["I"], c["S"] * c["Is"]
        hit = min(E, R)  # experts without tokens are not read
        out = (2 + 2 + 2 / 32) * (R * I + T * SI)
        return dict(bytes=2 * (R * d + (T * d if SI else 0) + 2 * d * (hit * I + SI)) + out,
                    flops=4 * d * (R * I + T * SI))
    return dict(bytes=R * c["I"] * (2 + 2 / 32 + 4 + 4 + 2) + 12 * R, flops=16 * R * c["I"])


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _grid(t, step):
    return torch.round(t / step) * step


def _tokens(g, T, d, dtype):
    return _grid(_randn(g, T, d), 2.0 ** -4).to(dtype)


def _weights(g, rows, d, dtype):
    std, step = (0.02, 2.0 ** -10) if d <= 2048 else (0.006, 2.0 ** -12)
    return _grid(_randn(g, rows, d) * std, step).to(dtype)


def _empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device=DEV)


def _assignment(g, T, E, k):
    """Routing of T tokens to k of E experts with uneven popularity: the rows
    in expert order, as moe_permute lays them out (offsets, perm_tok)."""
    z = _randn(g, T, E) + 0.5 * _randn(g, E)
    idx = z.topk(k, dim=1).indices.reshape(-1)
    perm = torch.sort(idx, stable=True).indices
    counts = torch.bincount(idx, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return offsets, perm, int(counts.max())


def _buffers(rows, n):
    """8-bit codes and tile scales of a saved [rows][n] matrix."""
    return _empty(rows, n, dtype=torch.uint8), _empty(n // 128, rows, 4, dtype=torch.uint8)


def prepare(case, seed):
    c = dict(case)
    op, T = c["op"], c["T"]
    g = _gen(seed)
    s = dict(c=c)
    if op == "gate":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s.update(x=_tokens(g, T, c["d"], dt), w_gate=_weights(g, c["E"], c["d"], dt), logits=_empty(T, c["E"]))
    elif op == "route":
        z = _randn(g, T, c["E"]) * c["spread"]
        if c["masked"]:  # experts that are out of service for the whole batch
            out = torch.randperm(c["E"], generator=g, device=DEV)[:c["masked"]]
            z[:, out] = -math.inf
        bias = (torch.rand(c["E"], generator=g, device=DEV) * 2 - 1) * 0.05 if c["bias"] else None
        s.update(logits=z, bias=bias, idx=_empty(T, c["k"], dtype=torch.int32), w=_empty(T, c["k"]),
                 counts=_empty(c["E"], dtype=torch.int32))
    elif op == "route_bwd":
        z = _randn(g, T, c["E"]) * c["spread"]
        s.update(logits=z, idx=z.topk(c["k"], dim=1).indices.to(torch.int32), dw=_randn(g, T, c["k"]),
                 dscores=_randn(g, T, c["E"]) * 0.01 if c["aux"] else None, dlogits=_empty(T, c["E"]))
    elif op == "up_save":
        d, E, k, I, SI = c["d"], c["E"], c["k"], c["I"], c["S"] * c["Is"]
        bf = torch.bfloat16
        offsets, perm, cap = _assignment(g, T, E, k)
        x = _tokens(g, T, d, bf)
        s.update(x=x, x_perm=x[torch.div(perm, k, rounding_mode="floor")], offsets=offsets.to(torch.int32), cap=cap,
                 w1=_weights(g, E * I, d, bf).view(E, I, d), w3=_weights(g, E * I, d, bf).view(E, I, d),
                 ws1=_weights(g, SI, d, bf), ws3=_weights(g, SI, d, bf), h=_empty(T * k, I, dtype=bf),
                 hs=_empty(T, SI, dtype=bf))
        for n, rows, cols in (("a", T * k, I), ("g", T * k, I), ("sa", T, SI), ("sg", T, SI)):
            s[n], s[n + "_scale"] = _buffers(rows, cols)
    else:
        R, I = T * c["k"], c["I"]
        _, perm, _ = _assignment(g, T, c["E"], c["k"])
        a, up = _randn(g, R, I), _randn(g, R, I)
        s.update(u=_randn(g, R, I), perm=perm.to(torch.int32),
                 w=torch.rand(T, c["k"], generator=g, device=DEV), dadg=_empty(R, 2 * I, dtype=torch.bfloat16),
                 h=_empty(R, I, dtype=torch.bfloat16), dw=_empty(T, c["k"]))
        s["a"], s["a_scale"] = _quantize(a)
        s["g"], s["g_scale"] = _quantize(up)
    return s


# ---------------------------------------------------------------- plain forms

def _quantize(v):
    """E4M3 codes of v [rows][n] with a power-of-two scale per 32 columns: 2^e, e the smallest integer with
    amax <= 448 * 2^e; the scale bytes (e + 127) as [n / 128][rows][4]."""
    rows, n = v.shape
    t = v.view(rows, n // 32, 32)
    amax = t.abs().amax(dim=2)
    m, q = torch.frexp(amax)  # amax = m 2^q, 448 = 0.875 * 2^9
    e = torch.where(amax > 0, q - 9 + (m > 0.875), torch.zeros_like(q)).clamp(min=-127)
    codes = torch.ldexp(t, -e.unsqueeze(2)).to(torch.float8_e4m3fn).view(torch.uint8).view(rows, n)
    scale = (e + 127).to(torch.uint8).view(rows, n // 128, 4).transpose(0, 1).contiguous()
    return codes, scale


def _values(codes, scale):
    rows, n = codes.shape
    e = scale.transpose(0, 1).reshape(rows, n // 32, 1).to(torch.int32) - 127
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float().view(rows, n // 32, 32), e).view(rows, n)


def _eights(codes, scale):
    """8-bit codes and scales as the values they stand for."""
    return codes.view(torch.float8_e4m3fn), scale.view(torch.float8_e8m0fnu)


def _scores(z, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    e = torch.exp(z - z.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _plain_route(s):
    c = s["c"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    z = s["logits"].double()  # scores next to each other decide the choice
    sc = _scores(z, c["score"])
    v = sc + s["bias"].double() if c["bias"] else sc
    v = torch.where(z == -math.inf, -math.inf, v)
    if c["top_groups"] < G:
        best = torch.sort(v.view(T, G, E // G), dim=2, descending=True).values[:, :, :c["group_top"]].sum(dim=2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=z.device).scatter_(1, kept, True)
        v = torch.where(keep.repeat_interleave(E // G, dim=1), v, -math.inf)
    idx = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :k]
    w = sc.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    counts = torch.zeros(E, dtype=torch.int32, device=z.device)
    counts.index_add_(0, idx.reshape(-1), torch.ones(T * k, dtype=torch.int32, device=z.device))
    return dict(idx=idx.to(torch.int32), w=(w * c["scale"]).float(), counts=counts)


def _plain_route_bwd(s):
    c = s["c"]
    sc = _scores(s["logits"], c["score"])
    idx = s["idx"].long()
    G = s["dw"] * c["scale"]
    if c["renorm"]:
        chosen = sc.gather(1, idx)
        total = chosen.sum(dim=1, keepdim=True)
        G = (G - (G * chosen).sum(dim=1, keepdim=True) / total) / total
    ds = torch.zeros_like(sc).scatter_add_(1, idx, G)
    if c["aux"]:
        ds = ds + s["dscores"]
    if c["score"] == "sigmoid":
        return ds * sc * (1 - sc)
    return sc * (ds - (ds * sc).sum(dim=1, keepdim=True))


def _silu(a):
    return a / (1 + torch.exp(-a))


def _plain_up_save(s):
    c = s["c"]
    E, d = c["E"], c["d"]
    off = s["offsets"].long()
    # the experts' rows side by side, each padded to the longest
    row = off[:-1, None] + torch.arange(s["cap"], device=DEV)
    x = s["x_perm"][row.clamp(max=s["x_perm"].shape[0] - 1).view(-1)].float().view(E, s["cap"], d)
    r = torch.arange(s["x_perm"].shape[0], device=DEV)
    e = torch.searchsorted(off, r, right=True) - 1
    back = e * s["cap"] + r - off[e]
    a, g = (torch.matmul(x, w.float().transpose(1, 2)).view(-1, c["I"])[back] for w in (s["w1"], s["w3"]))
    out = dict(h=(_silu(a) * g).to(torch.bfloat16), a=_eights(*_quantize(a)), g=_eights(*_quantize(g)))
    if c["S"]:
        a, g = (torch.matmul(s["x"].float(), w.float().t()) for w in (s["ws1"], s["ws3"]))
        out.update(hs=(_silu(a) * g).to(torch.bfloat16), sa=_eights(*_quantize(a)), sg=_eights(*_quantize(g)))
    return out


def _plain_act_bwd(s):
    a, g, u = _values(s["a"], s["a_scale"]), _values(s["g"], s["g_scale"]), s["u"]
    perm = s["perm"].long()
    sig = 1 / (1 + torch.exp(-a))
    h = a * sig * g
    dh = s["w"].view(-1)[perm].unsqueeze(1) * u
    dadg = torch.cat([dh * g * sig * (1 + a * (1 - sig)), dh * a * sig], dim=1)
    dw = torch.empty_like(s["w"].view(-1))
    dw[perm] = (u * h).sum(dim=1)
    return dict(dadg=dadg.to(torch.bfloat16), h=h.to(torch.bfloat16), dw=dw.view_as(s["w"]))


def _plain(s):
    op = s["c"]["op"]
    if op == "gate":
        return torch.matmul(s["x"].float(), s["w_gate"].float().t())
    return {"route": _plain_route, "route_bwd": _plain_route_bwd, "up_save": _plain_up_save,
            "act_bwd": _plain_act_bwd}[op](s)


# ---------------------------------------------------------------- the framework's calls

def _handles(s):
    """The shape, options and buffer handles that a program makes once."""
    import fine_grained_moe_gate_b200 as moe
    c = s["c"]
    dt = moe.MOE_F32 if c.get("dtype") == "f32" else moe.MOE_BF16
    s["moe"] = moe
    s["sh"] = moe.MoEShape(c["T"], c.get("d", 128), c["E"], c.get("k", 1), c.get("I", 128), c.get("S", 0),
                           c.get("Is", 128), dt)
    if "score" in c:
        s["opts"] = moe.route_opts(c["score"], groups=c.get("groups", 1), top_groups=c.get("top_groups", 1),
                                   group_top=c.get("group_top", 1), renormalize=c["renorm"], scale=c["scale"])
    if "a" in s:
        s["saved"] = moe.saved_acts(dict(a=s["a"], a_scale=s["a_scale"], g=s["g"], g_scale=s["g_scale"],
                                         sa=s.get("sa"), sa_scale=s.get("sa_scale"), sg=s.get("sg"),
                                         sg_scale=s.get("sg_scale")))


def _own(s):
    if "moe" not in s:
        _handles(s)
    moe, c, sh = s["moe"], s["c"], s["sh"]
    op = c["op"]
    if op == "gate":
        moe.moe_gate_logits(s["x"], s["w_gate"], sh, s["logits"])
        return s["logits"]
    if op == "route":
        moe.moe_route_logits(s["logits"], s["bias"], sh, s["opts"], s["idx"], s["w"], s["counts"])
        return dict(idx=s["idx"], w=s["w"], counts=s["counts"])
    if op == "route_bwd":
        moe.moe_route_logits_backward(s["logits"], s["idx"], s["dw"], s["dscores"], sh, s["opts"], s["dlogits"])
        return s["dlogits"]
    if op == "up_save":
        shared = c["S"] > 0
        moe.moe_ffn_up_save(s["x_perm"], s["offsets"], s["w1"], s["w3"], s["x"] if shared else None,
                            s["ws1"] if shared else None, s["ws3"] if shared else None, sh, s["h"],
                            s["hs"] if shared else None, s["saved"])
        out = dict(h=s["h"], a=_eights(s["a"], s["a_scale"]), g=_eights(s["g"], s["g_scale"]))
        if shared:
            out.update(hs=s["hs"], sa=_eights(s["sa"], s["sa_scale"]), sg=_eights(s["sg"], s["sg_scale"]))
        return out
    moe.moe_swiglu_backward_saved(s["saved"], sh, moe.MOE_ROUTED, s["u"], s["perm"], s["w"], s["dadg"], s["h"],
                                  s["dw"])
    return dict(dadg=s["dadg"], h=s["h"], dw=s["dw"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64-bit answers

def _exact_saved(v):
    """What the codes and the scales stand for before the codes' rounding: v / scale and the scale, by the
    definition (the smallest power of two that keeps a tile within 448)."""
    rows, n = v.shape
    amax = v.abs().view(rows, n // 32, 32).amax(dim=2)
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, 448.0) / 448))
    e = torch.where(torch.exp2(e - 1) * 448 >= amax, e - 1, e)  # log2's rounding
    e = torch.where(torch.exp2(e) * 448 < amax, e + 1, e)
    e = torch.where(amax > 0, e, 0.0).clamp(min=-127)
    codes = (v.view(rows, n // 32, 32) / torch.exp2(e).unsqueeze(2)).view(rows, n)
    return codes, torch.exp2(e).view(rows, n // 128, 4).transpose(0, 1)


def _exact_route(s):
    c = s["c"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    bias = s["bias"].double() if c["bias"] else torch.zeros(E, dtype=torch.float64, device=DEV)
    idx = torch.empty(T, k, dtype=torch.int64, device=DEV)
    w = torch.empty(T, k, dtype=torch.float64, device=DEV)
    lower = torch.ones(E, E, device=DEV).tril(-1).bool()          # [i][j]: j < i
    glower = torch.ones(G, G, device=DEV).tril(-1).bool()
    for t in range(0, T, 1024):
        z = s["logits"][t:t + 1024].double()
        sc = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, dim=1)
        v = (sc + bias).masked_fill(z.isinf(), -math.inf)
        if c["top_groups"] < G:
            best = v.view(-1, G, E // G).topk(c["group_top"], dim=2).values.sum(dim=2)
            ahead = (best.unsqueeze(1) > best.unsqueeze(2)) | ((best.unsqueeze(1) == best.unsqueeze(2)) & glower)
            keep = ahead.sum(dim=2) < c["top_groups"]
            v = v.masked_fill(~keep.unsqueeze(2).expand(-1, -1, E // G).reshape(-1, E), -math.inf)
        # an expert's place: how many are ahead of it
        ahead = (v.unsqueeze(1) > v.unsqueeze(2)) | ((v.unsqueeze(1) == v.unsqueeze(2)) & lower)
        place = ahead.sum(dim=2)
        row, expert = torch.nonzero(place < k, as_tuple=True)
        idx[t + row, place[row, expert]] = expert
        w[t + row, place[row, expert]] = sc[row, expert]
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return dict(idx=idx.to(torch.int32), w=w * c["scale"], counts=torch.bincount(idx.view(-1), minlength=E).to(torch.int32))


def _exact_route_bwd(s):
    """By the chain rule through the scores' Jacobian, written out."""
    c = s["c"]
    z = s["logits"].double()
    idx, dw = s["idx"].long(), s["dw"].double() * c["scale"]
    sc = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, dim=1)
    picked = torch.gather(sc, 1, idx)
    if c["renorm"]:
        p = picked / picked.sum(dim=1, keepdim=True)
        dpick = (dw - (dw * p).sum(dim=1, keepdim=True)) / picked.sum(dim=1, keepdim=True)
    else:
        dpick = dw
    up = s["dscores"].double() if c["aux"] else torch.zeros_like(sc)
    up = up.scatter_add(1, idx, dpick)
    if c["score"] == "sigmoid":
        return up * torch.exp(-z.abs()) / (1 + torch.exp(-z.abs())) ** 2
    return sc * up - sc * (sc * up).sum(dim=1, keepdim=True)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    op = c["op"]
    if op == "gate":
        return s["x"].double() @ s["w_gate"].double().t()
    if op == "route":
        return _exact_route(s)
    if op == "route_bwd":
        return _exact_route_bwd(s)
    if op == "up_save":
        off = s["offsets"].tolist()
        x = s["x_perm"].double()
        a = torch.cat([x[off[e]:off[e + 1]] @ s["w1"][e].double().t() for e in range(c["E"])])
        g = torch.cat([x[off[e]:off[e + 1]] @ s["w3"][e].double().t() for e in range(c["E"])])
        out = dict(h=a * torch.sigmoid(a) * g, a=_exact_saved(a), g=_exact_saved(g))
        if c["S"]:
            x = s["x"].double()
            a, g = x @ s["ws1"].double().t(), x @ s["ws3"].double().t()
            out.update(hs=a * torch.sigmoid(a) * g, sa=_exact_saved(a), sg=_exact_saved(g))
        return out
    rows, n = s["a"].shape
    two = lambda b: torch.exp2(b.permute(1, 0, 2).reshape(rows, n // 32).double() - 127).repeat_interleave(32, dim=1)
    a = s["a"].view(torch.float8_e4m3fn).double() * two(s["a_scale"])
    g = s["g"].view(torch.float8_e4m3fn).double() * two(s["g_scale"])
    u, perm = s["u"].double(), s["perm"].long()
    sig = torch.sigmoid(a)
    wu = s["w"].double().view(-1)[perm].unsqueeze(1) * u
    slope = sig + a * sig * (1 - sig)  # of a sigmoid(a)
    dw = torch.zeros(rows, dtype=torch.float64, device=DEV).scatter_(0, perm, torch.einsum("rn,rn->r", u, a * sig * g))
    return dict(dadg=torch.cat([wu * g * slope, wu * a * sig], dim=1), h=a * sig * g, dw=dw.view(c["T"], c["k"]))
