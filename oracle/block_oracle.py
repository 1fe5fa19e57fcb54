"""Plain NumPy forms, in 64 bits, of the operators around a block's linears: routing to experts,
low-rank adapters, and the fused residual and norm. None shares code with the GPU path.

Each returns, beside the exact value, how far a result may be from it: the roundings that the
operator's definition allows, counted one by one (u = 2^-24 is half a step of fp32, B = 2^-8 of
bf16, both relative)."""
import math

import numpy as np

U, B = 2.0**-24, 2.0**-8


# ---- routing -----------------------------------------------------------------------------


def route(logits, top_k, bias=None, scores="softmax", groups=1, top_groups=None, group_best=1, renormalize=True,
          scale=1.0):
    """ids [T, top_k] and float64 weights, a token and an expert at a time."""
    logits = np.asarray(logits, dtype=np.float32).astype(np.float64)
    T, E = logits.shape
    size, keep = E // groups, groups if top_groups is None else top_groups
    ids, weights = np.full((T, top_k), -1, np.int32), np.zeros((T, top_k))

    def rank(v):  # NaN first, then falling; ties to the lowest index
        return lambda e: (0, 0.0, e) if math.isnan(v[e]) else (1, -v[e], e)

    for t in range(T):
        l = logits[t]
        there = [e for e in range(E) if l[e] != -np.inf]
        if not there:
            continue
        top = max((l[e] for e in there if not math.isnan(l[e])), default=-np.inf)
        with np.errstate(all="ignore"):
            if scores == "softmax":
                p = {e: np.exp(l[e] - top) for e in there}
                total = sum(p.values())
                score = {e: p[e] / total for e in there}
            else:
                score = {e: 1.0 / (1.0 + np.exp(-l[e])) for e in there}
            key = {e: score[e] + (0.0 if bias is None else float(np.float32(bias[e]))) for e in there}
        there = [e for e in there if key[e] != -np.inf]
        if keep < groups:
            of = {}
            for g in range(groups):
                mine = sorted((e for e in there if e // size == g), key=rank(key))
                if mine and bias is None and group_best == 1:  # their largest alone: the order of the logits
                    of[g] = max((l[e] for e in mine if not math.isnan(l[e])), default=math.nan)
                    of[g] = math.nan if any(math.isnan(l[e]) for e in mine) else of[g]
                elif mine:
                    of[g] = sum(key[e] for e in mine[:group_best])
            kept = sorted(of, key=rank(of))[:keep]
            there = [e for e in there if e // size in kept]
        chosen = sorted(there, key=rank(key if bias is not None else l))[:top_k]
        if not chosen:
            continue
        with np.errstate(all="ignore"):
            w = np.array([score[e] for e in chosen])
            if renormalize:
                # shares of the chosen ones, in a range that holds them
                m = max((l[e] for e in chosen if not math.isnan(l[e])), default=-np.inf)
                if scores == "softmax":
                    w = np.array([np.exp(l[e] - m) for e in chosen])
                elif m < 0:
                    w = np.array([np.exp(l[e] - m) / (1.0 + np.exp(l[e])) for e in chosen])
                w = w / w.sum()
        ids[t, : len(chosen)] = chosen
        weights[t, : len(chosen)] = np.float64(np.float32(scale)) * w
    return ids, weights


def route_tol(weights):
    """One rounding to fp32; the 64-bit steps before it are some 2^-40 of a value at most."""
    return np.abs(weights) * (U + 2.0**-40) + 2.0**-149


# ---- low-rank adapters -------------------------------------------------------------------


def lora(y, x, a, b, adapters, scales=None):
    """out [T, N] in float64 before its rounding to bf16, and the tolerance of the rounded one.

    v = A x: any order of K fp32 products and sums, relative to the sum of magnitudes (K + 8) u; its
    scale one rounding more; its three bf16 parts add up to it. B v: 3R products (each exact: 8 by 8
    bits) and their sums, the addition of y; then half a step of bf16."""
    T, N = y.shape
    L, R, K = a.shape
    out, tol = y.astype(np.float64), np.zeros((T, N))
    for i in range(L):
        rows = np.flatnonzero(adapters == i)
        if rows.size == 0:
            continue
        s = 1.0 if scales is None else float(np.float32(scales[i]))
        A, Bm, X = a[i].astype(np.float64), b[i].astype(np.float64), x[rows].astype(np.float64)
        v, va = s * (X @ A.T), abs(s) * (np.abs(X) @ np.abs(A).T)
        off = (K + 9) * U * va + 2.0**-134
        d, da, do = v @ Bm.T, np.abs(v) @ np.abs(Bm).T, off @ np.abs(Bm).T
        exact = out[rows] + d
        err = 1.01 * do + (3 * R + 2) * U * 1.01 * (da + np.abs(out[rows]))
        out[rows] = exact
        tol[rows] = err + B * (np.abs(exact) + err)
    return out, tol + 2.0**-133


# ---- residual and norm -------------------------------------------------------------------

# Additions that a value passes through in a row's sum: 32 in its thread, 6 in its wave, 16 waves.
_PATH = 64


def _norm(v, kind, eps):
    """norm(v) in float64 and how far the kernel's may be from it.

    Layer: the mean as summed is off by `miss`, _PATH u of the mean magnitude and a rounding. Elements less
    that mean are rounded once; their own mean takes the miss back but for its sum, _PATH u of the elements'
    mean magnitude, and three roundings; the elements are rounded once more. The sum of their squares holds the
    miss's until it is taken off: its _PATH u of both stays."""
    if kind == "layer":
        mean = v.mean(1, keepdims=True)
        d = v - mean
        miss = (_PATH + 1) * U * np.abs(v).mean(1, keepdims=True)
        off = (_PATH + 4) * U * (np.abs(d).mean(1, keepdims=True) + miss) + 2 * U * np.abs(d) + U * miss
    else:
        d, off, miss = v, np.zeros_like(v), 0.0
    sd = np.sqrt((d * d).mean(1, keepdims=True) + eps)
    n = d / sd
    worst = off.max(1, keepdims=True) / sd + _PATH * U * (miss / sd) ** 2
    return n, off / sd + np.abs(n) * (worst + (_PATH / 2 + 8) * U), sd


def residual(x, y, kind, eps, post=None, gate=None, c=1.0):
    """h before its rounding, and the tolerance of the rounded one. ``gate`` by row."""
    x, z = x.astype(np.float64), y.astype(np.float64)
    off = np.zeros_like(z)
    if post is not None:
        z, off, _ = _norm(z, kind, eps)
        z, off = z * post, off * np.abs(post) + U * np.abs(z * post)
    if gate is not None:
        z, off = z * gate, off * np.abs(gate) + U * np.abs(z * gate)
    c = float(np.float32(c))
    h = x + c * z
    off = abs(c) * off * 1.01 + U * (np.abs(x) + abs(c) * np.abs(z))
    return h, off + B * (np.abs(h) + off) + 2.0**-133


def normed(h, kind, eps, weight=None, bias=None, scale=None, shift=None):
    """n of the stored h before its rounding, and the tolerance of the rounded one."""
    n, off, _ = _norm(h.astype(np.float64), kind, eps)
    if weight is not None:
        n, off = n * weight, off * np.abs(weight) + U * np.abs(n * weight)
    if bias is not None:
        n = n + bias
        off = off + U * (np.abs(n) + off)
    if scale is not None:
        n, off = n * (1.0 + scale), off * np.abs(1.0 + scale) + 2 * U * np.abs(n) * (1.0 + np.abs(scale))
    if shift is not None:
        n = n + shift
        off = off + U * (np.abs(n) + off)
    off = 1.01 * off
    return n, off + B * (np.abs(n) + off) + 2.0**-133
