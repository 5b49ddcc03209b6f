"""Plain fp64 CPU oracle of the softmax decode over a paged KV cache (window
with sinks, shared prefix), of the accumulated attention weights and of the
eviction by them.

TEST INFRASTRUCTURE ONLY: imports nothing from the library.

    z_t = q . k_t over the visible tokens, out = sum_t softmax(z)_t v_t,
    lse = ln sum_t exp(z_t);
    weights of token t: sum over the heads of its KV head of exp(z_t - tau) or
    [(alpha-1) z_t - tau]_+^(1/(alpha-1));
    eviction: the first `sinks`, the last `recent` and the heaviest of the
    tokens between, ties to the lower token.

Pins: tests/test_oracle_softmax.py.
"""
from __future__ import annotations

import math

import numpy as np


def visible(pos: int, length: int, window: int, sinks: int) -> np.ndarray:
    """Tokens that a query at position `pos` sees, ascending."""
    t = np.arange(max(0, min(pos + 1, length)))
    return t[(t > pos - window) | (t < sinks)]


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray):
    """(out, lse) of one query over the rows k, v; (0, -inf) over none."""
    if len(k) == 0:
        return np.zeros(v.shape[1]), -math.inf
    z = k.astype(np.float64) @ q.astype(np.float64)
    m = z.max()
    e = np.exp(z - m)
    return (e / e.sum()) @ v.astype(np.float64), m + math.log(e.sum())


def rows(pool: np.ndarray, table: np.ndarray, kv_head: int, t: np.ndarray) -> np.ndarray:
    """Rows of logical tokens t; pool [pages, kv_heads, page_size, dim]."""
    ps = pool.shape[2]
    return pool[table[t // ps], kv_head, t % ps]


def window_decode(q, k_pool, v_pool, table, lens, window, sinks):
    """q [batch, n, heads, dim] -> out (the same shape) and lse [batch, n, heads]."""
    B, n, H, _ = q.shape
    G = k_pool.shape[1]
    out, lse = np.zeros(q.shape), np.zeros(q.shape[:-1])
    for b in range(B):
        for i in range(n):
            t = visible(int(lens[b]) - n + i, int(lens[b]), window, sinks)
            for h in range(H):
                g = h // (H // G)
                out[b, i, h], lse[b, i, h] = attend(q[b, i, h], rows(k_pool, table[b], g, t),
                                                    rows(v_pool, table[b], g, t))
    return out, lse


def weights(q, k_pool, table, lens, alpha, tau, window, sinks, decay, old):
    """q [batch, heads, dim], old [batch, kv_heads, cells] -> the new sums; cells
    at or past lens stay as in `old`."""
    B, H, _ = q.shape
    G = k_pool.shape[1]
    new = np.array(old, dtype=np.float64)
    for b in range(B):
        L = int(lens[b])
        new[b, :, :L] *= decay
        t = visible(L - 1, L, window, sinks)
        for h in range(H):
            g = h // (H // G)
            z = rows(k_pool, table[b], g, t).astype(np.float64) @ q[b, h].astype(np.float64)
            if np.isneginf(tau[b, h]) if alpha == 1.0 else np.isnan(tau[b, h]):
                continue  # the decode saw nothing
            if alpha == 1.0:
                p = np.exp(z - tau[b, h])
            else:
                p = np.maximum((alpha - 1.0) * z - tau[b, h], 0.0) ** (1.0 / (alpha - 1.0))
            new[b, g, t] += p
    return new


def evict_kept(w: np.ndarray, length: int, keep: int, sinks: int, recent: int) -> np.ndarray:
    """Kept tokens of one row of weights, ascending."""
    if length <= keep:
        return np.arange(length)
    mid = np.arange(sinks, length - recent)
    x = np.where(np.isnan(w[mid]), np.inf, w[mid])
    nan_first = np.lexsort((mid, -x, ~np.isnan(w[mid])))  # a NaN before any number
    best = mid[nan_first[:keep - sinks - recent]]
    return np.sort(np.concatenate([np.arange(sinks), best, np.arange(length - recent, length)]))
