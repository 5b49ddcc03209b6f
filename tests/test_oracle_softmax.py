"""Pins of oracle/softmax_oracle.py: a library softmax, closed forms, the
entmax oracle's own probabilities, and brute force."""
import itertools
import math

import numpy as np
import pytest
import torch

from oracle import entmax_oracle as O
from oracle import softmax_oracle as S


def test_attend_against_torch_and_closed_forms():
    rng = np.random.default_rng(1)
    q, k, v = rng.normal(size=16), rng.normal(size=(37, 16)), rng.normal(size=(37, 16))
    out, lse = S.attend(q, k, v)
    z = torch.from_numpy(k @ q)
    assert np.allclose(out, (torch.softmax(z, 0) @ torch.from_numpy(v)).numpy(), atol=1e-13)
    assert abs(lse - float(torch.logsumexp(z, 0))) < 1e-13
    # equal scores: the mean; one token: its row; none: zero
    out, lse = S.attend(np.zeros(16), k, v)
    assert np.allclose(out, v.mean(0)) and abs(lse - math.log(37)) < 1e-13
    out, lse = S.attend(q, k[:1], v[:1])
    assert np.allclose(out, v[0]) and abs(lse - k[0] @ q) < 1e-13
    out, lse = S.attend(q, k[:0], v[:0])
    assert not out.any() and lse == -math.inf


def test_visible_by_its_definition():
    for pos, length, window, sinks in itertools.product(range(-2, 9), (0, 5, 9), (1, 3, 20),
                                                        (0, 2, 12)):
        want = [t for t in range(length) if t <= pos and (t > pos - window or t < sinks)]
        assert S.visible(pos, length, window, sinks).tolist() == want


def test_window_decode_reads_through_the_table():
    rng = np.random.default_rng(2)
    ps, pages = 16, 5
    k, v = rng.normal(size=(2, pages, 2, ps, 8))
    table = rng.permutation(pages)[None]
    q = rng.normal(size=(1, 2, 4, 8))
    out, lse = S.window_decode(q, k, v, table, [70], 7, 3)
    kk = k[table[0]].transpose(1, 0, 2, 3).reshape(2, -1, 8)
    vv = v[table[0]].transpose(1, 0, 2, 3).reshape(2, -1, 8)
    for i, h in itertools.product(range(2), range(4)):
        pos = 68 + i
        t = [0, 1, 2] + list(range(pos - 6, pos + 1))
        z = kk[h // 2][t] @ q[0, i, h]
        p = np.exp(z) / np.exp(z).sum()
        assert np.allclose(out[0, i, h], p @ vv[h // 2][t], atol=1e-13)
        assert abs(lse[0, i, h] - math.log(np.exp(z).sum())) < 1e-12


@pytest.mark.parametrize("alpha", [1.0, 1.25, 1.5, 2.0])
def test_weights_are_the_decode_probabilities(alpha):
    rng = np.random.default_rng(3)
    k = rng.normal(size=(3, 1, 16, 8))
    q = rng.normal(size=(1, 2, 8))
    L, table = 41, np.array([[2, 0, 1]])
    kk = k[table[0], 0].reshape(-1, 8)[:L]
    tau, want = np.zeros((1, 2)), np.zeros(L)
    for h in range(2):
        z = kk @ q[0, h]
        if alpha == 1.0:
            tau[0, h] = math.log(np.exp(z).sum())
            p = np.exp(z) / np.exp(z).sum()
        else:
            p, tau[0, h] = O.entmax(z, alpha)[:2]
        want += p
    old = rng.random((1, 1, 48))
    new = S.weights(q, k, table, [L], alpha, tau, 1000, 0, 0.5, old)
    assert np.allclose(new[0, 0, :L], 0.5 * old[0, 0, :L] + want, atol=1e-9)
    assert (new[0, 0, L:] == old[0, 0, L:]).all()
    assert abs((new - 0.5 * old)[0, 0, :L].sum() - 2.0) < 1e-9


def test_evict_kept_by_brute_force():
    rng = np.random.default_rng(4)
    for _ in range(60):
        L = int(rng.integers(0, 9))
        w = rng.integers(0, 4, size=12).astype(float)
        sinks, recent = int(rng.integers(0, 3)), int(rng.integers(0, 3))
        keep = sinks + recent + int(rng.integers(0, 4)) or 1
        got = S.evict_kept(w, L, keep, sinks, recent).tolist()
        if L <= keep:
            assert got == list(range(L))
            continue
        forced = set(range(sinks)) | set(range(L - recent, L))
        best = max((sum(w[t] for t in c), [-t for t in c], c)
                   for c in itertools.combinations(sorted(set(range(L)) - forced),
                                                   keep - sinks - recent))
        assert got == sorted(forced | set(best[2]))


def test_evict_kept_nan_first():
    w = np.array([1.0, np.nan, np.inf, 5.0, np.nan, -np.inf])
    assert S.evict_kept(w, 6, 2, 0, 0).tolist() == [1, 4]
    assert S.evict_kept(w, 6, 3, 0, 0).tolist() == [1, 2, 4]
