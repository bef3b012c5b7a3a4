"""CPU oracle for the operators around the grouped GEMM (include/nvfp4_moe.h).

TEST INFRASTRUCTURE ONLY, NumPy in float64, written from the definitions in the
header; it shares no code with the HIP path. Each function returns what the
operator would give if it rounded nothing but its stored results, and where a
test needs it the sum of the terms' magnitudes that its error bound scales with.
"""
from __future__ import annotations

import numpy as np

from .nvfp4_oracle import E2M1_VALUES, decode_e4m3fn, sf_offset

E4M3 = decode_e4m3fn(np.arange(127))          # the positive finite values, rising
E2M1 = E2M1_VALUES[:8]


# ---- routing -------------------------------------------------------------------

def scores(x, kind):
    with np.errstate(all="ignore"):
        if kind == "sigmoid":
            return 1 / (1 + np.exp(-x))
        top = np.max(x, axis=1, keepdims=True)
        top = np.where(np.isneginf(top), 0, top)
        e = np.exp(x - top)
        total = e.sum(1, keepdims=True)
        return e / np.where(total == 0, 1, total)


def route(x, topk, *, score="softmax", bias=None, groups=1, topk_groups=None, group_best=1, renormalize=True, scale=1.0):
    """(ids, weights) of float64 logits [tokens, experts]."""
    x = np.asarray(x, dtype=np.float64)
    tokens, experts = x.shape
    topk_groups = groups if topk_groups is None else topk_groups
    # for the choice, NaN is masked and +inf the largest fp32
    xc = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    s = scores(xc, score)
    v = xc if bias is None and groups == 1 else s if bias is None else s + bias
    v = np.where(np.isneginf(xc) | np.isnan(v), -np.inf, v)
    ids = np.full((tokens, topk), -1, dtype=np.int32)
    w = np.zeros((tokens, topk))
    per = experts // groups
    for t in range(tokens):
        eligible = np.ones(experts, dtype=bool)
        if groups > 1:
            worth = []
            for g in range(groups):
                best = np.sort(v[t, g * per:(g + 1) * per])[::-1][:group_best]
                best = best[best > -np.inf]
                worth.append(best.sum() if best.size else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-worth[g], g))[:topk_groups]
            eligible = np.repeat(np.isin(np.arange(groups), kept), per)
        order = sorted((e for e in range(experts) if eligible[e] and v[t, e] > -np.inf), key=lambda e: (-v[t, e], e))
        chosen = order[:topk]
        ids[t, :len(chosen)] = chosen
        c = s[t, chosen]
        total = c.sum() if renormalize else 1.0
        w[t, :len(chosen)] = c / (total if total != 0 else 1) * scale
        if np.isnan(x[t]).any() or (score == "softmax" and np.isposinf(x[t]).any()):
            w[t, :len(chosen)] = np.nan
    return ids, w


def route_backward(x, ids, dw, *, score="softmax", renormalize=True, scale=1.0):
    """(d logits, magnitude of its terms)."""
    x = np.asarray(x, dtype=np.float64)
    s = scores(x, score)
    d = np.zeros_like(x)
    size = np.zeros_like(x)
    for t in range(x.shape[0]):
        slots = np.flatnonzero(ids[t] >= 0)
        at = ids[t, slots]
        dp = dw[t, slots].astype(np.float64) * scale
        c = s[t, at]
        total = c.sum() if renormalize and c.sum() != 0 else 1.0
        both = np.abs(dp)
        if renormalize:
            both = (both + np.abs(dp * c / total).sum()) / total
            dp = (dp - (dp * c / total).sum()) / total
        ds, dm = np.zeros(x.shape[1]), np.zeros(x.shape[1])
        ds[at], dm[at] = dp, both
        if score == "sigmoid":
            d[t], size[t] = ds * s[t] * (1 - s[t]), dm * s[t]
        else:
            # renormalised, the sum of ds s is zero
            inner = 0.0 if renormalize else (ds * s[t]).sum()
            d[t] = s[t] * (ds - inner)
            size[t] = s[t] * (dm + (0.0 if renormalize else np.abs(ds * s[t]).sum()))
    return d, size


# ---- the plan ----------------------------------------------------------------------

def plan(ids, experts):
    flat = np.asarray(ids).reshape(-1)
    slot_rows = np.full(flat.size, -1, dtype=np.int32)
    row_slots = np.full(flat.size, -1, dtype=np.int32)
    offsets, atoms, row = [0], [0], 0
    for e in range(experts):
        for slot in np.flatnonzero(flat == e):
            slot_rows[slot], row_slots[row] = row, slot
            row += 1
        offsets.append(row)
        atoms.append(atoms[-1] + -(-(offsets[-1] - offsets[-2]) // 128))
    return (np.array(offsets, dtype=np.int32), np.array(atoms, dtype=np.int32), slot_rows.reshape(np.shape(ids)), row_slots)


# ---- NVFP4 -------------------------------------------------------------------------

def _nearest(a, values, unit):
    """Index of the value nearest to a / unit, ties to the even index; the borders are compared exactly (both sides
    are products of few bits)."""
    middle = (values[1:] + values[:-1]) / 2
    a, unit = np.broadcast_arrays(a, unit)
    code = np.zeros(a.shape, dtype=np.int64)
    for i, mid in enumerate(middle):
        code += (a > mid * unit) | ((a == mid * unit) & (i % 2 == 1))
    return code


def quantize(v):
    """(codes [rows, k], scale bytes [rows, k/16]) of fp32 (or float64) rows."""
    v = np.asarray(v)
    blocks = v.reshape(v.shape[0], -1, 16).astype(np.float64)
    top = np.abs(blocks).max(axis=2)
    bad = ~np.isfinite(blocks).all(axis=2)
    scale = _nearest(np.where(bad, 0, top), E4M3, np.float64(6))
    s = E4M3[scale]
    a = np.where(bad[..., None], 0, np.abs(blocks))
    codes = np.where(s[..., None] == 0, 0, _nearest(a, E2M1, np.where(s == 0, 1, s)[..., None]))
    codes = codes + 8 * (np.signbit(blocks) & (s[..., None] != 0) & ~bad[..., None])
    return codes.reshape(v.shape).astype(np.uint8), np.where(bad, 0x7F, scale).astype(np.uint8)


def values(codes, scales):
    return E2M1_VALUES[codes] * np.repeat(decode_e4m3fn(scales), 16, axis=1)


def unpack_rows(a, sfa, rows, k, atom=0):
    """(codes, scale bytes) of `rows` rows whose scale tensor begins at atom row `atom` of sfa."""
    a = np.asarray(a).reshape(-1, k // 2)[:rows]
    codes = np.stack((a & 15, a >> 4), axis=2).reshape(rows, k)
    at = atom * ((k + 63) // 64) * 512 + sf_offset(np.arange(rows)[:, None], np.arange(k // 16)[None, :], max(rows, 1), k)
    return codes, np.asarray(sfa)[at]


def pack(codes, scales):
    """(a [rows, k/2], tiled scales) of codes and scale bytes; padding scales are NaN."""
    rows, k = codes.shape
    a = (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)
    sf = np.full(-(-rows // 128) * 128 * (-(-k // 64)) * 4, 0x7F, dtype=np.uint8)
    sf[sf_offset(np.arange(rows)[:, None], np.arange(k // 16)[None, :], max(rows, 1), k)] = scales
    return a, sf


def swiglu(c, alpha=1.0, scale=1.0):
    with np.errstate(all="ignore"):
        g, u = np.split(np.asarray(c, dtype=np.float64) * np.asarray(alpha, dtype=np.float64), 2, axis=-1)
        return g / (1 + np.exp(-g)) * u * scale


# ---- combine -------------------------------------------------------------------------

def combine(c, weights, rows, alpha=None, ids=None, residual=None):
    """(y, magnitude of its terms)."""
    tokens, topk = rows.shape
    y = np.zeros((tokens, c.shape[1])) if residual is None else residual.astype(np.float64).copy()
    size = np.abs(y)
    for t in range(tokens):
        for j in range(topk):
            if rows[t, j] < 0 or (ids is not None and ids[t, j] < 0):
                continue
            w = float(weights[t, j]) * (1 if alpha is None else float(alpha[ids[t, j]]))
            term = w * c[rows[t, j]].astype(np.float64)
            y[t] += term
            size[t] += np.abs(term)
    return y, size


def combine_backward(dy, c, weights, rows, alpha=None, ids=None):
    """(dc, dweights, magnitude of the terms of dweights); rows that no slot names are NaN in dc."""
    tokens, topk = rows.shape
    dc = np.full(c.shape, np.nan)
    dw, size = np.zeros((tokens, topk)), np.zeros((tokens, topk))
    for t in range(tokens):
        for j in range(topk):
            if rows[t, j] < 0 or (ids is not None and ids[t, j] < 0):
                continue
            f = 1 if alpha is None else float(alpha[ids[t, j]])
            dc[rows[t, j]] = float(weights[t, j]) * f * dy[t].astype(np.float64)
            terms = f * dy[t].astype(np.float64) * c[rows[t, j]].astype(np.float64)
            dw[t, j], size[t, j] = terms.sum(), np.abs(terms).sum()
    return dc, dw, size


# ---- a few tokens --------------------------------------------------------------------

def few(x, ids, w, alpha=None):
    """(products [tokens, topk, n], magnitude of their terms); x [tokens, k] or [tokens, topk, k], w [experts, n, k]."""
    tokens, topk = ids.shape
    y = np.zeros((tokens, topk, w.shape[1]))
    size = np.zeros_like(y)
    for t in range(tokens):
        for j in range(topk):
            e = ids[t, j]
            if 0 <= e < w.shape[0]:
                row = (x[t, j] if x.ndim == 3 else x[t]).astype(np.float64)
                f = 1 if alpha is None else float(alpha[e])
                y[t, j] = w[e] @ row * f
                size[t, j] = np.abs(w[e]) @ np.abs(row) * abs(f)
    return y, size
