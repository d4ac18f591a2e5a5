"""Float64 oracle of the routed side path: gate, experts' products and their gradients, and
of the 4-bit base weights under them.

LoRASpace (the arXiv listing's abstract): static and dynamic composition of a pool's LoRAs;
"Compress then Serve" (academ.us/article/2407.00066), section 3: (W0 + B A) x."""
from __future__ import annotations

import numpy as np


def scores(logits, score):
    """s of every expert (T x E); -inf logits score 0."""
    l = np.asarray(logits, dtype=np.float64)
    if score == "sigmoid":
        return np.where(l > 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
    m = np.max(l, axis=1, keepdims=True)
    m = np.where(np.isneginf(m), 0.0, m)
    e = np.exp(l - m)
    d = e.sum(axis=1, keepdims=True)
    return e / np.where(d > 0, d, 1.0)


def choose(logits, top_k, score, bias=None, n_groups=1, top_groups=1, group_top=1):
    """ids (T x top_k, -1 = empty): row by row, by the definition."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    s = scores(l, score)
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    n = E // n_groups
    out = np.full((T, top_k), -1, dtype=np.int32)
    for t in range(T):
        key = l[t] if bias is None else s[t] + b
        c = s[t] + b
        open_ = [e for e in range(E) if l[t, e] > -np.inf and b[e] > -np.inf]
        if n_groups > 1:
            ranked = []
            for g in range(n_groups):
                # one best without a bias is ordered by the logit, as the experts are
                by = key if bias is None and group_top == 1 else c
                best = sorted((by[e] for e in open_ if e // n == g), reverse=True)[:group_top]
                if best:
                    ranked.append((-sum(best), g))
            keep = {g for _, g in sorted(ranked)[:top_groups]}
            open_ = [e for e in open_ if e // n in keep]
        order = sorted(open_, key=lambda e: (-key[e], e))[:top_k]
        out[t, :len(order)] = order
    return out


def weights(logits, ids, score, renorm, scale=1.0):
    """The chosen experts' weights (T x K), by ratios where renormalised."""
    l = np.asarray(logits, dtype=np.float64)
    on = ids >= 0
    at = np.where(on, ids, 0)
    lj = np.take_along_axis(l, at, axis=1)
    if not renorm:
        return scale * np.where(on, np.take_along_axis(scores(l, score), at, axis=1), 0.0)
    m = np.max(np.where(on, lj, -np.inf), axis=1, keepdims=True, initial=-np.inf)
    m = np.where(np.isneginf(m), 0.0, m)
    r = np.exp(np.where(on, lj, m) - m)
    if score == "sigmoid":
        r = sigmoid_ratios(lj, m, on)
    r = np.where(on, r, 0.0)
    d = r.sum(axis=1, keepdims=True)
    return scale * r / np.where(d > 0, d, 1.0)


def sigmoid_ratios(lj, m, on):
    """sigmoid(l_j) up to a common factor per row: e^-m sigmoid when every chosen l < 0."""
    l = np.where(on, lj, 0.0)
    plain = np.where(l > 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
    low = np.exp(np.minimum(l - m, 0)) / (1 + np.exp(np.minimum(l, 0)))
    return np.where(m < 0, low, plain)


def route_grad(logits, ids, gw, score, renorm, scale=1.0):
    """d sum(gw * weights) / d logits at fixed ids (T x E)."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    s = scores(l, score)
    out = np.zeros((T, E))
    for t in range(T):
        js = [j for j in range(ids.shape[1]) if ids[t, j] >= 0]
        if not js:
            continue
        e = [int(ids[t, j]) for j in js]
        g = np.array([gw[t, j] for j in js], dtype=np.float64)
        w = weights(l[t:t + 1], ids[t:t + 1], score, renorm, 1.0)[0, js]
        if renorm:
            v = scale * w * (g - (g * w).sum())
            if score == "sigmoid":
                v = v * (1 - s[t, e])
            for ej, vj in zip(e, v):
                out[t, ej] += vj
        elif score == "sigmoid":
            for ej, gj in zip(e, g):
                out[t, ej] += scale * gj * s[t, ej] * (1 - s[t, ej])
        else:
            out[t] -= scale * s[t] * (g * s[t, e]).sum()
            for ej, gj in zip(e, g):
                out[t, ej] += scale * gj * s[t, ej]
    return out


def _factors(e, ranks, off_A, off_Bt, A_pool, Bt_pool, d_in, d_out):
    k = int(ranks[e])
    A = np.asarray(A_pool[int(off_A[e]):int(off_A[e]) + k * d_in], dtype=np.float64).reshape(k, d_in)
    Bt = np.asarray(Bt_pool[int(off_Bt[e]):int(off_Bt[e]) + k * d_out], dtype=np.float64).reshape(k, d_out)
    return A, Bt


def mixture(x, base, ids, w, ranks, off_A, off_Bt, A_pool, Bt_pool, scale, adapter_scale=None):
    """(y, magnitude): y = base + sum_j w_j s_j B' (A' x); magnitude = the same sum of
    absolute values of every product, for error bounds."""
    x, y = np.asarray(x, dtype=np.float64), np.array(base, dtype=np.float64)
    mag = np.abs(y)
    for e in range(len(ranks)):
        tok, slot = np.nonzero(ids == e)
        if not len(tok):
            continue
        A, Bt = _factors(e, ranks, off_A, off_Bt, A_pool, Bt_pool, x.shape[1], y.shape[1])
        c = (np.ones(len(tok)) if w is None else np.asarray(w, dtype=np.float64)[tok, slot])
        c = c * (scale if adapter_scale is None else float(adapter_scale[e]))
        np.add.at(y, tok, c[:, None] * ((x[tok] @ A.T) @ Bt))
        np.add.at(mag, tok, np.abs(c)[:, None] * ((np.abs(x[tok]) @ np.abs(A).T) @ np.abs(Bt)))
    return y, mag


def mixture_grad(x, dy, ids, w, ranks, off_A, off_Bt, A_pool, Bt_pool, scale, adapter_scale=None):
    """(dx, dx magnitude, dw, dw magnitude) of sum(dy * y)."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    dx, dxm = np.zeros_like(x), np.zeros_like(x)
    dw, dwm = np.zeros(ids.shape), np.zeros(ids.shape)
    for e in range(len(ranks)):
        tok, slot = np.nonzero(ids == e)
        if not len(tok):
            continue
        A, Bt = _factors(e, ranks, off_A, off_Bt, A_pool, Bt_pool, x.shape[1], dy.shape[1])
        s = scale if adapter_scale is None else float(adapter_scale[e])
        c = s * (np.ones(len(tok)) if w is None else np.asarray(w, dtype=np.float64)[tok, slot])
        u, um = dy[tok] @ Bt.T, np.abs(dy[tok]) @ np.abs(Bt).T
        np.add.at(dx, tok, c[:, None] * (u @ A))
        np.add.at(dxm, tok, np.abs(c)[:, None] * (um @ np.abs(A)))
        dw[tok, slot] = s * (u * (x[tok] @ A.T)).sum(axis=1)
        dwm[tok, slot] = abs(s) * (um * (np.abs(x[tok]) @ np.abs(A).T)).sum(axis=1)
    return dx, dxm, dw, dwm


# ---- 4-bit base weights ---------------------------------------------------------------------

def bf16(v):
    """bf16 value of float64 values in its normal range, by way of fp32 (halves to even, twice)."""
    u = np.asarray(v, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & np.uint64(0xFFFF0000)
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def w4_quantize(W, group, zero_points):
    """(codes d_out x d_in, scales d_out x ng, zeros d_out x ng) of the definition."""
    W = np.asarray(W, dtype=np.float64)
    d_out, d_in = W.shape
    ng = -(-d_in // group)
    codes, sc, zs = np.zeros((d_out, d_in), np.uint8), np.zeros((d_out, ng)), np.full((d_out, ng), 8.0)
    for g in range(ng):
        p = W[:, g * group:(g + 1) * group]
        lo, hi = np.minimum(p.min(axis=1), 0), np.maximum(p.max(axis=1), 0)
        s = bf16((hi - lo) / 15) if zero_points else bf16(np.maximum(hi, -lo) / 7)
        safe = np.where(s > 0, s, 1.0)
        z = np.where(s > 0, np.clip(np.rint(-lo / safe), 0, 15), 0.0) if zero_points else np.full(d_out, 8.0)
        q = np.where(s[:, None] > 0, np.rint(p / safe[:, None]), 0.0)
        codes[:, g * group:(g + 1) * group] = np.clip(q + z[:, None], 0, 15)
        sc[:, g], zs[:, g] = s, z
    return codes, sc, zs


def w4_pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def w4_unpack(q):
    out = np.empty((q.shape[0], 2 * q.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out


def w4_matrix(q, scales, zeros, group):
    """The matrix the codes stand for, float64."""
    c = w4_unpack(q).astype(np.float64)
    at = np.arange(c.shape[1]) // group
    z = 8.0 if zeros is None else (np.asarray(zeros) & 15).astype(np.float64)[:, at]
    return (c - z) * np.asarray(scales, dtype=np.float64)[:, at]
