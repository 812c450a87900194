"""Plain attention and 8-bit key/value cache, from the definitions.

Attention is computed in float64, one sequence and query at a time, over the
tokens a query may see and no others.  Codes and scales of the cache are
defined in 32-bit arithmetic and computed in numpy float32, so that they can
be compared bit for bit.
"""
from __future__ import annotations

import numpy as np


def attend(q, k, v, scale):
    """One query [dim] over keys and values [tokens][dim] -> (output, the
    weighted mean of |v|, the largest |score|); zeros without tokens."""
    if len(k) == 0:
        z = np.zeros(v.shape[1])
        return z, z, 0.0
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    s = (k @ q) * scale
    w = np.exp(s - s.max())
    w /= w.sum()
    return w @ v, w @ np.abs(v), float(np.abs(s).max())


def prompt(q, k, v, cu_q, cu_k, scale):
    """Causal attention of packed sequences: q [rows][heads][dim], k and v
    [rows][kv heads][dim] -> (outputs, weighted means of |v|, largest |score|
    of each query and head)."""
    rows, heads, dim = q.shape
    group = heads // k.shape[1]
    out, mean, top = np.zeros((rows, heads, dim)), np.zeros((rows, heads, dim)), np.zeros((rows, heads))
    for b in range(len(cu_q) - 1):
        lq, lk = int(cu_q[b + 1] - cu_q[b]), int(cu_k[b + 1] - cu_k[b])
        for i in range(lq):
            n = max(0, i + 1 + lk - lq)
            for h in range(heads):
                ks = slice(int(cu_k[b]), int(cu_k[b]) + n)
                r = int(cu_q[b]) + i
                out[r, h], mean[r, h], top[r, h] = attend(q[r, h], k[ks, h // group], v[ks, h // group], scale)
    return out, mean, top


def grow_page(codes, scale, held, x):
    """One page and head: ``codes`` [rows][dim] hold ``held`` tokens at
    ``scale``, the new tokens ``x`` [n][dim] (float32) go behind them ->
    (codes, scale)."""
    f = np.float32
    codes = codes.copy()
    before = f(scale) if held else f(0)
    finite = np.abs(x[np.isfinite(x)])
    top = f(finite.max()) if finite.size else f(0)
    now = max(before, f(top * f(1.0 / 127.0)))
    tiny = now < np.finfo(np.float32).tiny
    with np.errstate(all="ignore"):
        fresh = f(0) if tiny else f(f(1) / now)
        again = f(0) if tiny else f(before / now)
        y = (x.astype(f) * fresh).astype(f)
    y[np.isnan(y)] = 0
    codes[held: held + len(x)] = np.rint(np.clip(y, -127, 127)).astype(np.int8)
    codes[:held] = np.rint(np.clip(codes[:held].astype(f) * again, -127, 127)).astype(np.int8)
    return codes, now


def store(k_codes, v_codes, k_scales, v_scales, k, v, table, held, cu_new):
    """New tokens k, v [rows][kv heads][dim] (float32) into copies of the
    cache's arrays (layout of entro_attn.h), which are returned."""
    k_codes, v_codes, k_scales, v_scales = (x.copy() for x in (k_codes, v_codes, k_scales, v_scales))
    page = k_codes.shape[2]
    for b in range(len(held)):
        n, at = int(cu_new[b + 1] - cu_new[b]), int(held[b])
        end = at + n
        while at < end:
            p, r = int(table[b][at // page]), at % page
            take = min(page - r, end - at)
            rows = slice(int(cu_new[b]) + at - int(held[b]), int(cu_new[b]) + at - int(held[b]) + take)
            for h in range(k_codes.shape[1]):
                k_codes[p, h], k_scales[p, h] = grow_page(k_codes[p, h], k_scales[p, h], r, k[rows, h])
                c, v_scales[p, h] = grow_page(v_codes[p, h].T, v_scales[p, h], r, v[rows, h])
                v_codes[p, h] = c.T
            at += take
    return k_codes, v_codes, k_scales, v_scales


def rows_of(k_codes, v_codes, k_scales, v_scales, table, first, count):
    """Keys and values [count][kv heads][dim] (float32, code * scale) of one
    sequence's tokens from position ``first`` on; ``table``: its row."""
    page = k_codes.shape[2]
    k = np.zeros((count, k_codes.shape[1], k_codes.shape[3]), np.float32)
    v = np.zeros_like(k)
    for i in range(count):
        p, r = int(table[(first + i) // page]), (first + i) % page
        k[i] = k_codes[p, :, r].astype(np.float32) * k_scales[p][:, None]
        v[i] = v_codes[p, :, :, r].astype(np.float32) * v_scales[p][:, None]
    return k, v
