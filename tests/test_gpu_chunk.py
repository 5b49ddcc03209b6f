"""alpha-entmax attention of ragged chunks on the GPU against the float64
oracle.

Tolerances. A score is off by ez = R 2^-24 sum_d |q_d k_d| (R: the chain of
matrix instructions, as for the softmax calls), x = (alpha - 1) z by ex =
(alpha - 1) ez + 2^-22 near the maximum (its difference and product). The
threshold moves by no more than the largest change of an x, and by what the
equation's sum is off, ds, over its slope m sum u^(m-1) >= m: eu = 2 ex + 2^-22
+ ds / m bounds the change of every u = x - tau, and from it each weight's,
numerically: |(u +- eu)_+^m - u_+^m|. Powers by exponential and logarithm are
off by (m |log2 u| + 4) 2^-23 of themselves, the sums of T terms by (T / 16 + 16)
2^-24 of theirs (16 lanes a row and more share the tokens). An output moves by
twice the weights' total change times max |v - out| (numerator and
denominator). A bf16 result adds half a step, its weights 2^-16.
"""
import math

import numpy as np
import pytest
import torch

from oracle import tokens_oracle as T
from parity_util import announce
from test_gpu_softmax import Cache

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def E():
    from sparse_long_context_page_amd import entmaxkv
    return entmaxkv


class Chunk:
    """A paged cache of len(new) sequences, the last new[b] tokens of each with
    queries; rows beyond every length poisoned."""

    def __init__(self, seed, lens, new, Hkv, D, ps, kv, H, q_dtype, spread=2.5, pad=0):
        self.c = Cache(seed, lens, Hkv, D, ps, kv)
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.N, self.H, self.new = int(self.starts[-1]) + pad, H, new
        q = self.c.rng.normal(size=(max(self.N, 1), H, D)) * spread / math.sqrt(D)
        self.q = torch.from_numpy(q.astype(np.float32)).to(BF if q_dtype == "bf16" else F32)

    def run(self, alpha, **kw):
        c = self.c
        k, v, table, lens = c.dev("k", "v", "table", "lens")
        q = self.q.cuda()
        out = torch.full_like(q, 7.0)
        tau = torch.full(q.shape[:2], 7.0, device="cuda")
        sup = torch.full(q.shape[:2], 7, dtype=I32, device="cuda")
        announce(f"chunk lens={c.lens[:6]} new={list(self.new)[:6]} heads={self.H}/{c.Hkv} D={c.D} "
                 f"ps={c.ps} kv={c.kv} q={q.dtype} alpha={alpha}")
        E().entmaxkv_entmax_chunk(c.shape(self.H), q, torch.from_numpy(self.starts).cuda(), k, v,
                                  table, lens, alpha, out, tau=tau, support=sup, **kw)
        torch.cuda.synchronize()
        return out, tau, sup

    def check(self, alpha, got=None, rows=None):
        c, m = self.c, 1.0 / (alpha - 1.0)
        out, tau, sup = (x.double().cpu().numpy() for x in (got or self.run(alpha)))
        q = self.q.double().numpy()
        k, v = c.np64()
        used = self.starts[-1]
        assert (out[used:] == 7).all() and (tau[used:] == 7).all() and (sup[used:] == 7).all()
        R = (12 * c.D // 32 if c.kv == "bf16" else c.D) + 4
        big = np.where(np.isfinite(k), np.abs(k), 0.0).reshape(-1, c.D)
        near = {}

        def each(r, h, z):
            ez = R * 2.0**-24 * float((np.abs(q[r, h]) @ big.T).max())
            near[r, h] = z, ez

        table = np.asarray(c.table)
        with np.errstate(invalid="ignore"):
            ref, rtau, rsup = T.chunk(q[:used], self.starts, k, v, table, c.lens, alpha, each)
        vmax = np.where(np.isfinite(v), np.abs(v), 0.0).max()
        worst = 0.0
        for (r, h), (z, ez) in near.items():
            if rows is not None and r not in rows:
                continue
            x = (alpha - 1.0) * z
            u = x - rtau[r, h]
            p = np.maximum(u, 0.0) ** m
            with np.errstate(divide="ignore"):
                rel = np.where(p > 0, (m * np.abs(np.log2(np.maximum(u, 1e-300))) + 4) * 2.0**-23, 0)
            n = len(z)
            ds = (n / 16 + 16) * 2.0**-24 + float((p * rel).sum())
            ex = (alpha - 1.0) * ez + 2.0**-22
            eu = 2 * ex + 2.0**-22 + ds / m
            dp = np.maximum(np.maximum(u + eu, 0) ** m - p, p - np.maximum(u - eu, 0) ** m)
            change = float(dp.sum()) + 2 * ds
            tol = 2 * change * (vmax + np.abs(ref[r, h]))
            if self.q.dtype == BF:
                tol = tol + 2.0**-8 * np.abs(ref[r, h]) * 1.001 + 2.0**-16 * vmax
            err = np.abs(out[r, h] - ref[r, h])
            assert np.isfinite(out[r, h]).all(), (r, h)
            worst = max(worst, float((err / tol).max()))
            assert (err <= tol).all(), (r, h, float((err / tol).max()))
            tt = ex + eu + 2.0**-22 * (abs(rtau[r, h]) + abs(x.max()))
            assert abs(tau[r, h] - rtau[r, h]) <= tt, (r, h, tau[r, h], rtau[r, h], tt)
            assert abs(sup[r, h] - rsup[r, h]) <= (np.abs(u) <= eu).sum(), (r, h)
        blind = np.isnan(rtau)
        assert (np.isnan(tau[:used]) == blind).all() and (out[:used][blind] == 0).all()
        assert (sup[:used][blind] == 0).all()
        return worst


@pytest.mark.parametrize("kv,q_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ps", [16, 32, 64])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_types_and_shapes(kv, q_dtype, D, ps, G):
    Chunk(ps + G, [77, 33, 140, 16], [5, 1, 40, 16], 2, D, ps, kv, 2 * G, q_dtype).check(1.5)


@pytest.mark.parametrize("alpha", [1.03, 1.1, 1.25, 4 / 3, 1.5, 1.6, 1.9, 2.0])
@pytest.mark.parametrize("spread", [0.01, 0.5, 2.5, 20.0])
def test_alpha_and_spread_of_scores(alpha, spread):
    """From weights on every token (small alpha, flat scores) to one token."""
    Chunk(7, [300, 41], [19, 3], 2, 64, 16, "bf16", 8, "f32", spread).check(alpha)
    Chunk(8, [301, 2], [3, 2], 1, 64, 16, "f32", 2, "f32", spread).check(alpha)


@pytest.mark.parametrize("alpha", [2.5, 3.0, 5.0])
def test_alpha_beyond_two(alpha):
    Chunk(9, [200, 33], [9, 1], 2, 64, 32, "bf16", 4, "f32").check(alpha)
    Chunk(9, [200, 33], [9, 1], 2, 64, 32, "bf16", 4, "f32", 0.3).check(alpha)


@pytest.mark.parametrize("lens,new", [
    ([1], [1]), ([2], [2]), ([0], [0]), ([0, 5, 0], [0, 5, 0]), ([16], [16]), ([17], [17]),
    ([64, 65, 63], [64, 1, 63]), ([128], [100]), ([3] * 70, [1] * 70), ([40] * 3, [0, 7, 0]),
    ([5, 9], [9, 9]), ([0, 4], [6, 2])])
def test_lengths(lens, new):
    """One token, none, whole prompts, sequences without new tokens, and more
    new tokens than the sequence holds (the first rows see nothing)."""
    for G in (1, 4):
        Chunk(len(lens), lens, new, 2, 64, 16, "bf16", 2 * G, "bf16", pad=3).check(1.5)


def test_many_sequences():
    """The search for a block's sequence over more than 64 and 64^2 of them."""
    rng = np.random.default_rng(3)
    new = (rng.random(5000) < 0.1).astype(int)
    lens = [int(x) for x in new * rng.integers(1, 20, 5000)]
    lens = [max(a, b) for a, b in zip(lens, new.tolist())]
    c = Chunk(3, lens, new, 1, 64, 16, "bf16", 1, "bf16")
    c.check(1.5)


def test_equal_scores_and_equal_keys():
    """Ties: all weights alike, at any alpha."""
    for alpha in (1.25, 1.5, 2.0, 3.0):
        c = Chunk(4, [150], [30], 2, 64, 16, "bf16", 4, "f32")
        c.q[:10] = 0.0
        c.c.k[torch.isfinite(c.c.k)] = 0.5
        c.check(alpha)


def test_hidden_rows_have_no_effect():
    """NaN keys and infinite values of tokens that a row does not see, in the
    same tile as those that it does."""
    for kv in ("bf16", "f32"):
        c = Chunk(5, [50], [20], 2, 64, 16, kv, 4, "f32")
        t = 49
        page, row = c.c.table[0][t // 16], t % 16
        clean = c.run(1.5)
        c.c.k[page, :, row], c.c.v[page, :, row] = math.nan, math.inf
        got = c.run(1.5)
        for a, b in zip(clean, got):
            assert torch.equal(a[:19], b[:19])
        assert got[0][19].isnan().all() and got[1][19].isnan().all()


def test_values_of_zero_weight_have_no_effect():
    """A value that is not finite matters to the rows that give it a weight."""
    for kv in ("bf16", "f32"):
        c = Chunk(6, [90], [30], 1, 64, 16, kv, 4, "f32", spread=6.0)
        clean = c.run(1.5)
        k, _ = c.c.np64()
        z = {}
        T.chunk(c.q.double().numpy(), c.starts, k, k, c.c.table, c.c.lens, 1.5,
                lambda r, h, x: z.__setitem__((r, h), x))
        t = 20
        tau = clean[1].double().cpu().numpy()
        weighs = np.array([[0.5 * z[r, h][t] > tau[r, h] for h in range(4)] for r in range(30)])
        assert weighs.any() and not weighs.all()
        c.c.v[c.c.table[0][t // 16], :, t % 16] = math.inf
        got = c.run(1.5)
        live = torch.from_numpy(weighs).cuda()
        assert torch.equal(got[0][~live], clean[0][~live]) and torch.equal(got[1], clean[1])
        assert not got[0][live].isfinite().any()


def test_scores_that_are_no_numbers():
    c = Chunk(7, [40], [4], 2, 64, 16, "f32", 4, "f32")
    c.q[0, 0] = math.nan
    c.q[1, 1] = 3e38  # overflows to +inf somewhere, -inf elsewhere
    c.q[2, 2] = 3e38
    c.c.k[torch.isfinite(c.c.k)] = c.c.k[torch.isfinite(c.c.k)].abs()
    c.c.k[:, 1] = -c.c.k[:, 1].abs()
    out, tau, sup = c.run(1.5)
    for r, h in ((0, 0), (1, 1)):  # NaN, +inf
        assert out[r, h].isnan().all() and tau[r, h].isnan()
    assert (out[2, 2] == 0).all() and tau[2, 2].isnan() and sup[2, 2] == 0  # -inf everywhere
    ok = torch.ones(4, 4, dtype=torch.bool)
    for r, h in ((0, 0), (1, 1), (2, 2)):
        ok[r, h] = False
    assert out[ok.cuda()].isfinite().all()


def test_invalid_pages_are_empty():
    c = Chunk(8, [100, 60, 20], [30, 2, 5], 2, 64, 16, "bf16", 4, "f32")
    c.c.table[0, 1], c.c.table[0, 5], c.c.table[1, 0] = -1, c.c.pages, -7
    c.c.table[2, :] = 2**31 - 1
    c.check(1.5)


def test_token_starts_outside_the_rows_read_and_write_nothing_else():
    c = Chunk(9, [30, 30, 30], [4, 4, 4], 1, 64, 16, "bf16", 2, "bf16")
    for starts in ([0, 4, 8, 999], [-5, 4, 8, 12], [12, 8, 4, 0], [2**31 - 1] * 4, [0, 9, 3, 12]):
        c.starts = np.array(starts, np.int32)
        out, tau, _ = c.run(1.5)  # wrong rows, within the arrays
        assert out.shape == c.q.shape
