"""Oracle of routing from logits and of the saved activations (numpy float64)
-- TEST INFRASTRUCTURE, plain loops over the definitions in moe_gate.h.

Sources, by page title and section:
  * "DeepSeek V3 From Scratch", "In code" (scores, biased choice, weights
    from the unbiased scores), "The idea" (FP8 with fine-grained tiles).
  * "Scaling Efficiency: A Deep Dive into the DeepSeek-V3 Architecture",
    DeepSeekMoE sketch (softmax gating, SwiGLU experts).
"""
from __future__ import annotations

import dataclasses

import numpy as np


@dataclasses.dataclass(frozen=True)
class Opts:
    score: str = "sigmoid"
    groups: int = 1
    top_groups: int = 1
    group_top: int = 1
    renormalize: bool = True
    scale: float = 1.0


def scores(z: np.ndarray, score: str) -> np.ndarray:
    """s [T][E] of logits z (float64); masked logits (-inf, NaN) score 0."""
    z = np.asarray(z, np.float64)
    masked = np.isnan(z) | (z == -np.inf)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-z))
        else:
            m = np.where(masked, -np.inf, z).max(axis=1, keepdims=True)
            e = np.where(z == m, 1.0, np.exp(z - m))
            e = np.where(masked, 0.0, e)
            tot = e.sum(axis=1, keepdims=True)
            s = e / np.where(tot > 0, tot, 1.0)
    return np.where(masked, 0.0, s)


def route(z: np.ndarray, bias, k: int, o: Opts):
    """(idx, w, counts, short): the choice by the definition; short[t]: fewer than k experts to choose from."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    s = scores(z, o.score)
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    v = s + b
    v = np.where(np.isnan(v) | np.isnan(z) | (z == -np.inf), -np.inf, v)
    per = E // o.groups
    idx = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        vt = v[t].copy()
        if o.top_groups < o.groups:
            gv = np.full(o.groups, -np.inf)
            for g in range(o.groups):
                best = sorted((x for x in vt[g * per:(g + 1) * per] if x > -np.inf), reverse=True)[:o.group_top]
                if best:
                    gv[g] = sum(best)
            kept = sorted(range(o.groups), key=lambda g: (-gv[g], g))[:o.top_groups]
            for g in range(o.groups):
                if g not in kept:
                    vt[g * per:(g + 1) * per] = -np.inf
        order = [e for e in sorted(range(E), key=lambda e: (-vt[e], e)) if vt[e] > -np.inf][:k]
        idx[t, :len(order)] = order
        w[t, :len(order)] = chosen_weights(z[t, order], s[t, order], o)
    counts = np.bincount(idx[idx >= 0].reshape(-1), minlength=E).astype(np.int32)
    return idx, w, counts, (idx < 0).any(axis=1)


def chosen_weights(z, s, o: Opts):
    if not o.renormalize or len(s) == 0:
        return s * o.scale
    if s.sum() < 1e-200:  # every score underflows: sigmoid and softmax ratios are those of e^z
        s = np.exp(z - z.max()) if np.isfinite(z.max()) else np.zeros_like(s)
    tot = s.sum()
    return o.scale * s / tot if tot > 0 else np.zeros_like(s)


def route_backward(z, idx, dw, dscores, o: Opts) -> np.ndarray:
    """d/dz of <dw, w> + <dscores, s> for the choice idx (slots outside [0, E) skipped)."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    s = scores(z, o.score)
    masked = np.isnan(z) | (z == -np.inf)
    dz = np.zeros((T, E))
    for t in range(T):
        slots = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E and not masked[t, idx[t, j]]]
        e = [int(idx[t, j]) for j in slots]
        G = np.array([float(dw[t, j]) for j in slots]) * o.scale
        ds = np.zeros(E) if dscores is None else np.where(masked[t], 0.0, np.asarray(dscores[t], np.float64))
        if e:
            st = s[t, e]
            if o.renormalize:
                p = chosen_weights(z[t, e], st, dataclasses.replace(o, scale=1.0))
                c = p * (G - (G * p).sum())
                if o.score == "sigmoid":
                    c = c * np.where(z[t, e] > 0, np.exp(-np.abs(z[t, e])), 1.0) / (1.0 + np.exp(-np.abs(z[t, e])))
                np.add.at(dz[t], e, c)
            else:
                np.add.at(ds, e, G)
        if o.score == "sigmoid":
            az = np.exp(-np.abs(np.where(masked[t], 0.0, z[t])))
            dz[t] += np.where(masked[t], 0.0, ds * az / (1.0 + az) ** 2)
        else:
            dz[t] += s[t] * (ds - (ds * s[t]).sum())
    return dz


def tile_exponents(v: np.ndarray) -> np.ndarray:
    """e [rows][n/32]: the smallest integer with amax <= 448 * 2^e (0 for an all-zero tile, at least -127)."""
    rows, n = v.shape
    amax = np.abs(np.asarray(v, np.float64)).reshape(rows, n // 32, 32).max(axis=2)
    m, q = np.frexp(amax)
    e = q - 9 + (m > 0.875)
    return np.maximum(np.where(amax > 0, e, 0), -127)


def dequantize(codes: np.ndarray, words: np.ndarray) -> np.ndarray:
    """Values of E4M3 codes [rows][n] with token-layout scale bytes [n/128][rows][4]."""
    import oracle
    rows, n = codes.shape
    e = np.transpose(words.reshape(n // 128, rows, 4), (1, 0, 2)).reshape(rows, n // 32).astype(np.int64) - 127
    val = np.asarray(oracle.fp8_decode(codes), np.float64).reshape(rows, n // 32, 32)
    return np.ldexp(val, e[:, :, None]).reshape(rows, n)


def swiglu_backward(a, g, u, wt):
    """(da, dg, h, <u, h>) of rows with weights wt, float64."""
    a, g, u = (np.asarray(x, np.float64) for x in (a, g, u))
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-a))
    h = a * s * g
    dh = np.asarray(wt, np.float64)[:, None] * u
    return dh * g * s * (1.0 + a * (1.0 - s)), dh * a * s, h, (u * h).sum(axis=1)
