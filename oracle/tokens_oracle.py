"""Plain fp64 CPU oracle of the step that puts new tokens into a paged KV cache
and attends from them: the plan of pages and slots, the norm and rotation of
heads, and the alpha-entmax attention of a ragged chunk.

TEST INFRASTRUCTURE ONLY: imports nothing from the library.

Pins: tests/test_oracle_tokens.py.
"""
from __future__ import annotations

import math

import numpy as np

from oracle import entmax_oracle as O


def plan(seq_lens, new_tokens, free, table, page_size, num_pages, rows):
    """One sequence after the other. free: the free pages, the last one taken
    first. Returns a dict of the call's outputs; `table` is not changed."""
    table = np.array(table, dtype=np.int64)
    most = table.shape[1] * page_size
    stack = list(free)
    wanted = 0
    out = {"new_lens": [], "token_starts": [], "positions": [0] * rows, "slots": [-1] * rows}
    row = 0
    for b, (L, n) in enumerate(zip(seq_lens, new_tokens)):
        L, n = min(max(int(L), 0), most), max(int(n), 0)
        out["token_starts"].append(min(row, rows))
        fits = L + n <= most and row + n <= rows
        held = -(-L // page_size)
        need = -(-(L + n) // page_size) - held if fits else 0
        wanted += need
        granted = fits and (need == 0 or wanted <= len(free))
        if granted:
            for i in range(need):
                table[b, held + i] = stack.pop()
        for i in range(n):
            if row + i >= rows:
                break
            p = L + i
            out["positions"][row + i] = p
            if granted:
                page = table[b, p // page_size]
                if 0 <= page < num_pages:
                    out["slots"][row + i] = int(page) * page_size + p % page_size
        out["new_lens"].append(L + n if granted else L)
        row += n
    out["token_starts"].append(min(row, rows))
    out["free_left"] = len(stack)
    out["block_table"] = table
    return {k: np.array(v) for k, v in out.items()}


def norm(x, weight, eps):
    """x over its last axis by its root mean square; no weight: x itself."""
    x = np.asarray(x, np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def rotate(x, positions, freqs, pair_axis=None, interleaved=False):
    """x [tokens, heads, dim]; positions [axes, tokens]; freqs [half]."""
    x = np.array(x, np.float64)
    for i, f in enumerate(freqs):
        axis = 0 if pair_axis is None else int(pair_axis[i])
        for t in range(x.shape[0]):
            c, s = math.cos(positions[axis][t] * f), math.sin(positions[axis][t] * f)
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + len(freqs))
            u, v = x[t, :, a].copy(), x[t, :, b].copy()
            x[t, :, a], x[t, :, b] = u * c - v * s, u * s + v * c
    return x


def chunk(q, token_starts, k_pool, v_pool, table, seq_lens, alpha, each=None):
    """q [rows, heads, dim]; returns out, tau (NaN for a row that sees nothing),
    support, all of q's rows; rows of no sequence stay NaN. A page outside the
    pool is empty. each(row, head, scores): called for every row that sees a
    token."""
    N, H, D = q.shape
    P, G, ps, _ = k_pool.shape
    out = np.full(q.shape, np.nan)
    tau = np.full((N, H), np.nan)
    support = np.zeros((N, H), np.int64)
    for b, L in enumerate(seq_lens):
        n = token_starts[b + 1] - token_starts[b]
        for i in range(n):
            r = token_starts[b] + i
            t = np.arange(max(0, L - n + i + 1))
            page = table[b][t // ps]
            ok = (page >= 0) & (page < P)
            page, t = page[ok], t[ok]
            for h in range(H):
                g = h // (H // G)
                if len(t) == 0:
                    out[r, h] = 0.0
                    continue
                z = k_pool[page, g, t % ps].astype(np.float64) @ q[r, h].astype(np.float64)
                if each is not None:
                    each(r, h, z)
                tau[r, h] = O.entmax_threshold((alpha - 1.0) * z, alpha)
                p = O.entmax_probs((alpha - 1.0) * z, tau[r, h], alpha)
                live = p > 0
                support[r, h] = live.sum()
                out[r, h] = p[live] @ v_pool[page[live], g, t[live] % ps].astype(np.float64)
    return out, tau, support
