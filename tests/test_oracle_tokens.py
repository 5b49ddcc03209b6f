"""Pins of oracle/tokens_oracle.py: hand-worked plans, complex rotations,
invariants, and the decode oracle's own attention."""
import math

import numpy as np
import pytest

from oracle import entmax_oracle as O
from oracle import tokens_oracle as T


def test_plan_by_hand():
    # pages of 16: sequence 0 holds one page with 3 tokens, takes 14 more (one
    # page); sequence 1 is new with 33 tokens (three pages); 2 brings none
    table = [[5, -1, -1, -1], [-1] * 4, [7, -1, -1, -1]]
    p = T.plan([3, 0, 16], [14, 33, 0], [10, 11, 12, 13, 14], table, 16, 100, 50)
    assert p["block_table"].tolist() == [[5, 14, -1, -1], [13, 12, 11, -1], [7, -1, -1, -1]]
    assert p["new_lens"].tolist() == [17, 33, 16] and p["free_left"] == 1
    assert p["token_starts"].tolist() == [0, 14, 47, 47]
    assert p["positions"][:15].tolist() == [*range(3, 17), 0] and p["positions"][47:].sum() == 0
    assert p["slots"][12] == 5 * 16 + 15 and p["slots"][13] == 14 * 16
    assert p["slots"][14] == 13 * 16 and p["slots"][46] == 11 * 16
    assert (p["slots"][47:] == -1).all()


def test_plan_refusals():
    # the first wants more than there is, the second would not fit the table,
    # the third needs no page, the fourth is behind the first's want
    table = np.full((4, 2), 3)
    p = T.plan([0, 16, 4, 0], [32, 17, 2, 1], [9], table, 16, 10, 100)
    assert p["new_lens"].tolist() == [0, 16, 6, 0] and p["free_left"] == 1
    assert (p["slots"][:49] == -1).all() and p["slots"][49] == 3 * 16 + 4
    assert (p["block_table"] == 3).all()
    # rows: the second sequence ends behind the last row
    p = T.plan([0, 0, 0], [3, 5, 0], [1, 2], np.full((3, 2), -1), 16, 10, 6)
    assert p["new_lens"].tolist() == [3, 0, 0] and p["token_starts"].tolist() == [0, 3, 6, 6]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product_and_keeps_differences(interleaved):
    rng = np.random.default_rng(3)
    x, y = rng.normal(size=(5, 2, 12)), rng.normal(size=(5, 2, 12))
    f, pos = rng.uniform(size=4), rng.integers(0, 900, (1, 5))
    r = T.rotate(x, pos, f, interleaved=interleaved)
    a, b = (slice(0, 8, 2), slice(1, 8, 2)) if interleaved else (slice(0, 4), slice(4, 8))
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[0][:, None] * f)[:, None]
    assert np.allclose(r[..., a], z.real) and np.allclose(r[..., b], z.imag)
    assert (r[..., 8:] == x[..., 8:]).all()
    # a product depends on the difference of the positions alone
    p = (T.rotate(x, pos + 7, f, interleaved=interleaved)
         * T.rotate(y, pos + 7, f, interleaved=interleaved)).sum(-1)
    assert np.allclose(p, (r * T.rotate(y, pos, f, interleaved=interleaved)).sum(-1))


def test_rotation_on_several_axes():
    rng = np.random.default_rng(4)
    x, f = rng.normal(size=(3, 1, 8)), rng.uniform(size=4)
    pos, axis = rng.integers(0, 99, (3, 3)), [2, 0, 1, 2]
    r = T.rotate(x, pos, f, pair_axis=axis)
    for i in range(4):
        alone = T.rotate(x, pos[axis[i]][None], f)
        assert np.allclose(r[..., [i, i + 4]], alone[..., [i, i + 4]])


def test_norm():
    x = np.array([[3.0, 4.0], [0.0, 0.0]])
    assert np.allclose(T.norm(x, [1.0, 2.0], 0.5)[0], [3 / math.sqrt(13), 8 / math.sqrt(13)])
    assert (T.norm(x, [1.0, 1.0], 1e-6)[1] == 0).all() and (T.norm(x, None, 0.1) == x).all()


@pytest.mark.parametrize("alpha", [1.3, 1.5, 2.0, 3.0])
def test_chunk_rows_are_decodes_of_shorter_sequences(alpha):
    rng = np.random.default_rng(5)
    D, ps, H, G = 8, 4, 4, 2
    k, v = rng.normal(size=(6, G, ps, D)), rng.normal(size=(6, G, ps, D))
    table = np.array([[3, 0, 5], [1, 9, 2]])
    starts, lens = [0, 3, 5], [9, 11]
    q = rng.normal(size=(6, H, D))
    out, tau, sup = T.chunk(q, starts, k, v, table, lens, alpha)
    for r, b, L in [(0, 0, 7), (2, 0, 9), (4, 1, 11)]:
        t = np.array([x for x in range(L) if 0 <= table[b][x // ps] < 6])
        for h in range(H):
            z = np.array([q[r, h] @ k[table[b][x // ps], h // 2, x % ps] for x in t])
            p, th = O.entmax(z, alpha)[:2]
            assert abs(p.sum() - 1) < 1e-9
            vs = np.array([v[table[b][x // ps], h // 2, x % ps] for x in t])
            assert np.allclose(out[r, h], p @ vs) and sup[r, h] == (p > 0).sum()
            assert np.isclose(tau[r, h], th)
    assert np.isnan(out[5]).all()  # a row behind the last sequence


def test_chunk_rows_that_see_nothing():
    k = np.ones((1, 1, 4, 4))
    out, tau, sup = T.chunk(np.ones((3, 1, 4)), [0, 3], k, k, np.array([[0]]), [2], 1.5)
    assert (out[0] == 0).all() and np.isnan(tau[0]) and sup[0] == 0
    assert np.allclose(out[1:], 1) and sup[1:].ravel().tolist() == [1, 2]
