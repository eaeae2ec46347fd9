"""CPU oracle for expert routing, the grouped layouts, dispatch, combine and the
8-bit activation checkpoints: plain numpy in float64, written from the
definitions (test infrastructure only, like the rest of this package).

bf16 tensors are uint16 bit patterns, E4M3 tensors uint8 codes.
"""
from __future__ import annotations

import numpy as np

from . import TILE, e4m3_decode_table, e4m3_encode_array

NEG = -np.inf
FLT_MAX = float(np.finfo(np.float32).max)


def bf16_to_f32(bits):
    with np.errstate(invalid="ignore"):
        return (np.asarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32)


def f32_to_bf16(v):
    """float32 -> bf16 bits, round to nearest even (finite values)."""
    u = np.ascontiguousarray(v, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def _clean(logits):
    """Logits as float64; NaN and -inf become -inf (never chosen), +inf the largest finite float."""
    l = np.asarray(logits, dtype=np.float64)
    l = np.where(np.isnan(l), NEG, l)
    return np.minimum(l, FLT_MAX)


def _scores(l, score):
    ok = l > NEG
    if score == "softmax":
        m = np.where(ok.any(axis=1, keepdims=True), l.max(axis=1, keepdims=True, initial=NEG), 0.0)
        e = np.where(ok, np.exp(l - m), 0.0)
        return e / np.maximum(e.sum(axis=1, keepdims=True), np.finfo(np.float64).tiny)
    with np.errstate(over="ignore"):
        return np.where(ok, 1.0 / (1.0 + np.exp(-l)), 0.0)


def _chosen_weights(l, score, renorm, full):
    """Weights of one row's chosen logits `l` (all finite) before the scale; `full` the softmax denominators' row."""
    if l.size == 0:
        return l
    if score == "softmax":
        if renorm:
            e = np.exp(l - l.max())
            return e / e.sum()
        f = full[full > NEG]
        return np.exp(l - f.max()) / np.exp(f - f.max()).sum()
    log_p = -np.logaddexp(0.0, -l)
    if renorm:
        e = np.exp(log_p - log_p.max())
        return e / e.sum()
    return np.exp(log_p)


def route(logits, top_k, bias=None, score="softmax", n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0):
    """(ids [T,k] int32, weights [T,k] float64)."""
    l = _clean(logits)
    T, E = l.shape
    ok = l > NEG
    key = _scores(l, score)
    b = None
    if bias is not None:
        b = np.asarray(bias, dtype=np.float64)
        ok &= ~(np.isnan(b) | (b == NEG))[None, :]
        key = key + np.where(np.isnan(b), 0.0, b)[None, :]
    key = np.where(ok, key, NEG)
    order = key if bias is not None else np.where(ok, l, NEG)
    ids = np.full((T, top_k), -1, dtype=np.int32)
    w = np.zeros((T, top_k))
    size = E // n_group
    for t in range(T):
        o = order[t].copy()
        if n_group > 1:
            totals = []
            for g in range(n_group):
                # single keys without a bias compare as their logits (order)
                by = key if group_top == 2 else order
                k = np.sort(by[t, g * size:(g + 1) * size])[::-1][:group_top]
                k = k[k > NEG]
                totals.append(k.sum() if k.size else NEG)
            best = sorted(range(n_group), key=lambda g: (-totals[g], g))[:topk_group]
            for g in range(n_group):
                if g not in best:
                    o[g * size:(g + 1) * size] = NEG
        at = np.lexsort((np.arange(E), -o))[:top_k]
        at = at[o[at] > NEG]
        ids[t, :at.size] = at
        w[t, :at.size] = scale * _chosen_weights(l[t, at], score, renorm, l[t])
    return ids, w


def route_bwd(logits, ids, dweights, score="softmax", renorm=True, scale=1.0):
    """dlogits [T,E] float64, and the magnitudes the terms of each element had (for error bounds)."""
    l = _clean(logits)
    T, E = l.shape
    out = np.zeros((T, E))
    mag = np.zeros((T, E))
    g_all = np.asarray(dweights, dtype=np.float64)
    for t in range(T):
        js = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E and l[t, ids[t, j]] > NEG]
        at = np.array([ids[t, j] for j in js], dtype=np.int64)
        g = g_all[t, js]
        if score == "softmax" and not renorm:
            p = _scores(l[t:t + 1], score)[0]
            d, da = np.zeros(E), np.zeros(E)
            np.add.at(d, at, g)
            np.add.at(da, at, np.abs(g))
            out[t] = scale * p * (d - (d * p).sum())
            mag[t] = scale * p * (da + (da * p).sum())
            continue
        ls = l[t, at]
        p = np.exp(-np.logaddexp(0.0, -ls))
        not_p = np.exp(-np.logaddexp(0.0, ls))
        r = _chosen_weights(ls, score, renorm, l[t])
        if renorm:
            v = scale * r * (g - (g * r).sum())
            a = scale * r * (np.abs(g) + (np.abs(g) * r).sum())
            if score == "sigmoid":
                v, a = v * not_p, a * not_p
        else:
            v = scale * g * p * not_p
            a = np.abs(v)
        np.add.at(out[t], at, v)
        np.add.at(mag[t], at, a)
    return out, mag


def layout_contiguous(ids, E):
    """(slots, m_indices, counts): entries in order within each expert, experts' runs on 128-row blocks."""
    flat = np.asarray(ids).reshape(-1)
    n = flat.size
    B = (n + 127 * min(n, E)) // 128
    slots = np.full(n, -1, dtype=np.int32)
    m_indices = np.full(B, -1, dtype=np.int32)
    counts = np.zeros(E, dtype=np.int32)
    block = 0
    for e in range(E):
        mine = np.flatnonzero(flat == e)
        counts[e] = mine.size
        slots[mine] = block * 128 + np.arange(mine.size)
        nb = -(-mine.size // 128)
        m_indices[block:block + nb] = e
        block += nb
    return slots.reshape(np.shape(ids)), m_indices, counts


def layout_masked(ids, E, cap):
    flat = np.asarray(ids).reshape(-1)
    slots = np.full(flat.size, -1, dtype=np.int32)
    masked_m = np.zeros(E, dtype=np.int32)
    for e in range(E):
        mine = np.flatnonzero(flat == e)[:cap]
        masked_m[e] = mine.size
        slots[mine] = e * cap + np.arange(mine.size)
    return slots.reshape(np.shape(ids)), masked_m


def pad_rows(m_indices, counts):
    """Rows of used blocks that no entry fills."""
    pad = np.zeros(len(m_indices) * 128, dtype=bool)
    for e, c in enumerate(counts):
        at = np.flatnonzero(np.asarray(m_indices) == e)
        if at.size:
            pad[at[0] * 128 + c:(at[-1] + 1) * 128] = True
    return pad


def combine(y, slots, weights=None):
    """(out [T,D] float64, sum of |terms|) for y [rows,D] float64."""
    T, k = slots.shape
    out = np.zeros((T, y.shape[1]))
    mag = np.zeros_like(out)
    for t in range(T):
        for j in range(k):
            if 0 <= slots[t, j] < y.shape[0]:
                v = y[slots[t, j]] * (1.0 if weights is None else float(weights[t, j]))
                out[t] += v
                mag[t] += np.abs(v)
    return out, mag


def combine_dweights(dout, y, slots):
    """(dw [T,k] float64, sum of |terms|)."""
    T, k = slots.shape
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if 0 <= slots[t, j] < y.shape[0]:
                v = dout[t] * y[slots[t, j]]
                dw[t, j], mag[t, j] = v.sum(), np.abs(v).sum()
    return dw, mag


def quant_f32(v):
    """E4M3 codes and scales of float32 groups along the last axis: s = fl32(amax/448), codes of fl32(v/s)."""
    v = np.asarray(v, dtype=np.float32)
    amax = np.abs(v).max(axis=-1)
    s = (amax / np.float32(448.0)).astype(np.float32)
    s = np.where(s == 0, np.float32(1.0), s)
    q = e4m3_encode_array((v / s[..., None]).astype(np.float32).reshape(-1)).reshape(v.shape)
    return q, s


def dequant_1x128(q, s):
    """fl32(code * s) of 1x128 tiles, float32."""
    v = e4m3_decode_table().astype(np.float32)[np.asarray(q, dtype=np.uint8)]
    M, K = v.shape
    return (v.reshape(M, K // TILE, TILE) * np.asarray(s, dtype=np.float32).reshape(M, K // TILE, 1)).astype(
        np.float32).reshape(M, K)


def ckpt_128x1_t(q, s, Mp):
    """1x128 tiles regrouped along tokens: (qt [K,Mp], st [Mp/128,K])."""
    M, K = q.shape
    v = np.zeros((Mp, K), dtype=np.float32)
    v[:M] = dequant_1x128(q, s)
    qt, st = quant_f32(v.T.reshape(K, Mp // TILE, TILE))
    return qt.reshape(K, Mp), np.ascontiguousarray(st.T)


def swiglu_bwd(dh, qc, sc):
    """(d [rows,2I] float64, magnitude of its terms) from dh float64 and the checkpoint."""
    v = dequant_1x128(qc, sc).astype(np.float64)
    n = v.shape[1] // 2
    g, u = v[:, :n], v[:, n:]
    p = np.exp(-np.logaddexp(0.0, -g))
    not_p = np.exp(-np.logaddexp(0.0, g))
    f = 1.0 + g * not_p
    d = np.concatenate([dh * u * p * f, dh * g * p], axis=1)
    mag = np.concatenate([np.abs(dh * u) * p * (np.abs(g) * not_p + np.abs(f)), np.abs(dh * g * p)], axis=1)
    return d, mag
