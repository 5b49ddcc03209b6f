"""Softmax decode (window with sinks, shared prefix) on the GPU against the
float64 oracle.

Tolerances. A score is a chain of matrix instructions: 3 D/32 of them on bf16
caches (exact products of bf16 parts), D/4 on float32 ones, of up to 4
products that are added with at most 4 roundings each, so
    ez = R 2^-24 max_t sum_d |q_d k_td|,   R = 12 D/32 + 4 or D + 4.
A weight is then off by a factor e^ez, its exponential by 2^-22 more, so an
output by at most 2 (ez + 2^-22) max_t |v_td - out_d| (numerator and
denominator), plus the rounding of the running sums: at most 16 per tile or
part of a row's tokens, each 2^-24 of max |v|. The log of the sum is off by
ez + 2^-22 plus the roundings of the sum and of the result. A bf16 output adds
half a step, 2^-8 of its value. With bf16 queries the weights are used to 16
bits (2^-16 of max |v|), in the many-rows form (from 33 rows of a KV head, and
enough work for it) to 8, each off by at most 2^-8 of itself: 2^-8 of the
weighted mean of |v|. Small cases reach that form among empty sequences.
"""
import math

import numpy as np
import pytest
import torch

from oracle import softmax_oracle as S
from parity_util import announce

pytestmark = pytest.mark.gpu


def E():
    from sparse_long_context_page_amd import entmaxkv
    return entmaxkv


class Cache:
    """A paged cache with rows beyond every length poisoned."""

    def __init__(self, seed, lens, Hkv, D, ps, kv, spare=3, max_pages=None, prefix_pages=0):
        rng = np.random.default_rng(seed)
        self.lens, self.Hkv, self.D, self.ps, self.kv = list(lens), Hkv, D, ps, kv
        B = len(lens)
        self.mp = max_pages or max(1, -(-max(lens) // ps)) + 1
        pages = prefix_pages + B * (self.mp - prefix_pages) + spare
        order = rng.permutation(pages).astype(np.int32)
        self.prefix_table = order[:prefix_pages].copy()
        own = order[prefix_pages:prefix_pages + B * (self.mp - prefix_pages)].reshape(B, -1)
        self.table = np.concatenate([np.tile(self.prefix_table, (B, 1)), own], 1)
        self.pages = pages
        kv_t = torch.bfloat16 if kv == "bf16" else torch.float32
        self.k, self.v = (torch.from_numpy(rng.normal(size=(pages, Hkv, ps, D)).astype(np.float32))
                          .to(kv_t) for _ in range(2))
        used = torch.zeros(pages, ps, dtype=torch.bool)
        for b, L in enumerate(self.lens):
            t = np.arange(L)
            used[self.table[b, t // ps], t % ps] = True
        used[self.prefix_table] = True
        for x, bad in ((self.k, math.nan), (self.v, math.inf)):
            x.transpose(1, 2)[~used] = bad
        self.rng = rng

    def query(self, n, H, q_dtype, scale=2.5):
        q = self.rng.normal(size=(len(self.lens), n, H, self.D)) * scale / math.sqrt(self.D)
        return torch.from_numpy(q.astype(np.float32)).to(
            torch.bfloat16 if q_dtype == "bf16" else torch.float32)

    def shape(self, H):
        return E().make_shape(len(self.lens), H, self.Hkv, self.D, self.ps, self.mp, self.pages,
                              self.kv)

    def dev(self, *names):
        out = []
        for n in names:
            x = getattr(self, n)
            x = torch.from_numpy(np.ascontiguousarray(x)) if isinstance(x, np.ndarray) else x
            out.append((torch.tensor(x, dtype=torch.int32) if isinstance(x, list) else x).cuda())
        return out

    def np64(self):
        return self.k.double().numpy(), self.v.double().numpy()


def check(c, q, out, lse, ref, ref_lse, mean_abs=0.0):
    k, v = c.np64()
    D = c.D
    # sum_d |q_d k_d| row by row would be exact; the largest |q| bounds it
    qn = q.double().numpy()
    finite_k = np.where(np.isfinite(k), np.abs(k), 0.0).reshape(-1, D)
    R = (12 * D // 32 if c.kv == "bf16" else D) + 4
    big = (np.abs(qn).reshape(-1, D) @ finite_k.T).max(-1).reshape(qn.shape[:-1])
    ez = R * 2.0**-24 * big
    vmax = np.where(np.isfinite(v), np.abs(v), 0.0).max()
    tiles = sum(-(-L // 16) for L in c.lens) + 64
    tol = 2 * (ez + 2.0**-22)[..., None] * (vmax + np.abs(ref)) + 16 * tiles * 2.0**-24 * vmax
    if q.dtype == torch.bfloat16:
        tol = tol + 2.0**-8 * np.abs(ref) + 2.0**-16 * vmax + 2.0**-8 * mean_abs
    o = out.double().cpu().numpy()
    assert np.isfinite(o).all()
    err = np.abs(o - ref)
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:4])
    ll = lse.double().cpu().numpy()
    none = np.isneginf(ref_lse)
    assert (np.isneginf(ll) == none).all() and (o[none] == 0).all()
    le = np.abs(np.where(none, 0, ll) - np.where(none, 0, ref_lse))
    lt = ez + 2.0**-22 + 2.0**-23 * np.where(none, 0, np.abs(ref_lse)) + 16 * tiles * 2.0**-24
    assert (le <= lt).all(), float((le / lt).max())


def reference(c, q, lens, window, sinks, rows):
    """out, lse and, where the many-rows form may round weights, the weighted mean of |v|."""
    k, v = c.np64()
    qn = q.double().numpy()
    out, lse = S.window_decode(qn, k, v, c.table, lens, window, sinks)
    rounded = q.dtype == torch.bfloat16 and rows >= 33
    return out, lse, (S.window_decode(qn, k, np.abs(v), c.table, lens, window, sinks)[0]
                      if rounded else 0.0)


def empties(c, q, tiles):
    """Sequences of length 0 that bring a batch over `tiles` tiles of 16 rows
    in the few-rows form (at least 2 tiles a block of rows)."""
    n, H = q.shape[1:3]
    return tiles // (2 * c.Hkv * max(1, n * H // c.Hkv // 16))


def padded(c, q, empty):
    """Shape, q, tables and lengths with `empty` more sequences of length 0."""
    bt, lens, qd = *c.dev("table", "lens"), q.cuda()
    bt = torch.cat([bt, bt.new_full((empty, c.mp), -1)])
    lens = torch.cat([lens, lens.new_zeros(empty)])
    qd = torch.cat([qd, qd[:1].expand(empty, *qd.shape[1:])])
    shape = E().make_shape(len(lens), q.shape[2], c.Hkv, c.D, c.ps, c.mp, c.pages, c.kv)
    return shape, qd, bt, lens


def unpadded(B, out, lse):
    assert (out[B:] == 0).all() and torch.isneginf(lse[B:]).all()
    return out[:B], lse[:B]


def run_window(c, q, window, sinks, empty=0, **kw):
    k, v = c.dev("k", "v")
    shape, qd, bt, lens = padded(c, q, empty)
    out = torch.full_like(qd, float("nan"))
    lse = torch.full(qd.shape[:-1], float("nan"), device="cuda")
    E().entmaxkv_softmax_window(shape, qd, k, v, bt, lens, window, sinks, out, lse,
                                q_tokens=q.shape[1], **kw)
    torch.cuda.synchronize()
    return unpadded(len(q), out, lse)


@pytest.mark.parametrize("kv,qt,D,ps,Hkv,G,n,window,sinks", [
    ("bf16", "bf16", 128, 16, 2, 4, 1, 100, 4),
    ("bf16", "f32", 128, 32, 1, 8, 1, 64, 0),
    ("bf16", "f32", 64, 64, 2, 1, 1, 33, 70),
    ("bf16", "bf16", 64, 16, 1, 2, 3, 17, 1),
    ("f32", "f32", 128, 16, 1, 4, 1, 50, 4),
    ("f32", "f32", 64, 32, 2, 2, 5, 9, 3),
    ("f32", "f32", 64, 64, 1, 8, 1, 2**31 - 1, 0),
    ("bf16", "bf16", 128, 64, 1, 8, 7, 1, 0),
    ("bf16", "f32", 128, 16, 1, 1, 40, 30, 2),
    ("bf16", "bf16", 128, 16, 2, 4, 37, 2**31 - 1, 2**31 - 1),
    ("f32", "f32", 128, 64, 1, 1, 33, 20, 5),
    ("bf16", "bf16", 64, 64, 1, 8, 50, 77, 33),
    ("bf16", "f32", 64, 32, 2, 2, 70, 2**31 - 1, 0),
    ("f32", "f32", 64, 16, 1, 8, 9, 100, 17),
    ("bf16", "bf16", 128, 32, 1, 1, 140, 64, 1),
    # few tokens a block: one part, eight waves
    ("bf16", "bf16", 128, 16, 1, 4, 1, 200, 4),
    ("bf16", "f32", 64, 32, 2, 8, 1, 300, 0),
    ("f32", "f32", 128, 16, 1, 2, 2, 60, 1),
    ("f32", "f32", 64, 64, 1, 4, 1, 1, 0),
])
def test_window(kv, qt, D, ps, Hkv, G, n, window, sinks):
    # lengths of 0 and 1, around a page, a tile and several splits
    lens = (0, 1, ps - 1, ps, ps + 1, 31, 32, 33, 200, 517)
    c = Cache(1, lens, Hkv, D, ps, kv)
    q = c.query(n, Hkv * G, qt)
    announce(f"window {kv}/{qt} D{D} ps{ps} Hkv{Hkv} G{G} n{n} W{window} S{sinks}")
    ref = reference(c, q, lens, window, sinks, n * G)
    for empty in [0] + ([empties(c, q, 4200)] if n * G >= 33 else []):
        announce(f"  and {empty} empty sequences")
        out, lse = run_window(c, q, window, sinks, empty)
        check(c, q, out, lse, *ref)


@pytest.mark.parametrize("kv,qt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("B,lens", [(1, (9000,)), (300, (40, 0, 3, 77))])
def test_window_few_and_many_row_blocks(kv, qt, B, lens):
    """One long sequence (many splits a row block) and many short ones (one
    part a row: the attention kernel writes the result)."""
    lens = [lens[b % len(lens)] for b in range(B)]
    c = Cache(2, lens, 2, 128, 16, kv)
    q = c.query(1, 4, qt)
    announce(f"window blocks {kv}/{qt} B{B}")
    out, lse = run_window(c, q, 5000, 4)
    check(c, q, out, lse, *S.window_decode(q.double().numpy(), *c.np64(), c.table, lens, 5000, 4))


def test_hidden_rows_have_no_effect():
    """Every row that no query sees holds NaN and infinities, inside the pages
    that are read too."""
    lens, window, sinks = (300, 41), 37, 5
    for kv, qt in (("bf16", "bf16"), ("f32", "f32")):
        c = Cache(3, lens, 1, 64, 32, kv)
        q = c.query(2, 4, qt)
        seen = torch.zeros(c.pages, c.ps, dtype=torch.bool)
        for b, L in enumerate(lens):
            for pos in (L - 2, L - 1):
                t = S.visible(pos, L, window, sinks)
                seen[c.table[b, t // c.ps], t % c.ps] = True
        c.k.transpose(1, 2)[~seen] = -math.inf
        c.v.transpose(1, 2)[~seen] = math.nan
        announce(f"window hidden rows {kv}")
        out, lse = run_window(c, q, window, sinks)
        check(c, q, out, lse, *S.window_decode(q.double().numpy(), *c.np64(), c.table, lens,
                                               window, sinks))


@pytest.mark.parametrize("kv,qt,G", [("bf16", "bf16", 4), ("bf16", "f32", 1), ("f32", "f32", 2),
                                     ("bf16", "bf16", 1), ("bf16", "f32", 8)])
def test_infinite_value_reaches_only_the_rows_that_see_it(kv, qt, G):
    """The newest of 24 tokens and the oldest in the first one's window hold
    values that are not finite: the rows between see neither."""
    L, n, window = 130, 24, 40
    c = Cache(4, (L,), 1, 128, 16, kv)
    q = c.query(n, G, qt)
    first = L - n - window + 1
    for t, x in ((L - 1, math.inf), (first, math.nan)):
        c.v[c.table[0, t // 16], :, t % 16, 5] = x
    ref, ref_lse = S.window_decode(q.double().numpy(), *c.np64(), c.table, (L,), window, 0)
    mean_abs = S.window_decode(q.double().numpy(), c.np64()[0], np.abs(c.np64()[1]), c.table,
                               (L,), window, 0)[0] if n * G >= 33 else 0.0
    for empty in [0] + ([empties(c, q, 4200)] if n * G >= 33 else []):
        announce(f"window infinite values {kv} G{G}, {empty} empty sequences")
        out, lse = run_window(c, q, window, 0, empty)
        o = out.double().cpu().numpy()
        bad = np.zeros(o.shape, bool)
        bad[0, 0, :, 5] = bad[0, n - 1, :, 5] = True
        assert not np.isfinite(o[bad]).any()
        assert np.isfinite(o[~bad]).all()
        o[bad] = 0
        check(c, q, torch.from_numpy(o), lse, np.where(bad, 0, ref), ref_lse,
              np.where(bad, 0, mean_abs))


def test_pages_that_are_not_there():
    """Table entries outside the pool: their tokens are hidden."""
    L = 100
    c = Cache(5, (L, L), 1, 64, 16, "bf16")
    c.table[0, 2], c.table[0, 5], c.table[1, :] = -1, c.pages, -7
    q = c.query(1, 2, "f32")
    announce("window invalid pages")
    out, lse = run_window(c, q, 1000, 0)
    t = np.array([t for t in range(L) if t // 16 not in (2, 5)])
    kk, vv = c.np64()
    ref, ref_lse = np.zeros(q.shape), np.full(q.shape[:-1], -np.inf)
    for h in range(2):
        ref[0, 0, h], ref_lse[0, 0, h] = S.attend(q[0, 0, h].double().numpy(),
                                                  S.rows(kk, c.table[0], 0, t),
                                                  S.rows(vv, c.table[0], 0, t))
    check(c, q, out, lse, ref, ref_lse)


@pytest.mark.parametrize("kv,qt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_pages_that_are_not_there_many_rows(kv, qt):
    """The same for a chunk of queries and for a shared prefix."""
    L, n = 150, 40
    c = Cache(8, (L,), 1, 64, 16, kv)
    gone = (1, 4, 8)
    for j, bad in zip(gone, (-1, c.pages, 1 << 30)):
        c.table[0, j] = bad
    q = c.query(n, 1, qt)
    announce(f"window invalid pages, many rows {kv}/{qt}")
    kk, vv = c.np64()
    ref, ref_lse, mean_abs = np.zeros(q.shape), np.zeros(q.shape[:-1]), np.zeros(q.shape)
    for i in range(n):
        t = np.array([t for t in S.visible(L - n + i, L, 90, 3) if t // 16 not in gone])
        k, v = S.rows(kk, c.table[0], 0, t), S.rows(vv, c.table[0], 0, t)
        qi = q[0, i, 0].double().numpy()
        ref[0, i, 0], ref_lse[0, i, 0] = S.attend(qi, k, v)
        mean_abs[0, i, 0] = S.attend(qi, k, np.abs(v))[0]
    for empty in (0, empties(c, q, 4200)):
        out, lse = run_window(c, q, 90, 3, empty)
        check(c, q, out, lse, ref, ref_lse, mean_abs)

    B, P = 36, 6
    c = Cache(9, [P * 16 + 20] * B, 1, 64, 16, kv, prefix_pages=P)
    q = c.query(1, 1, qt)
    c.prefix_table[2], c.prefix_table[5] = -3, c.pages + 5
    kk, vv = c.np64()
    t = np.array([t for t in range(P * 16 + 20) if t // 16 not in (2, 5)])
    ref, ref_lse, mean_abs = np.zeros(q.shape), np.zeros(q.shape[:-1]), np.zeros(q.shape)
    for b in range(B):
        k, v = S.rows(kk, c.table[b], 0, t), S.rows(vv, c.table[b], 0, t)
        qb = q[b, 0, 0].double().numpy()
        ref[b, 0, 0], ref_lse[b, 0, 0] = S.attend(qb, k, v)
        mean_abs[b, 0, 0] = S.attend(qb, k, np.abs(v))[0]
    for empty in (0, 16 * 1100 // 3):
        out, lse = run_prefix(c, q, P, empty)
        check(c, q, out, lse, ref, ref_lse, mean_abs)


def test_extreme_scores():
    """Scores of +-60000 and all equal; a row of zeros."""
    c = Cache(6, (90,), 1, 64, 16, "f32")
    q = c.query(1, 4, "f32")
    q[0, 0, 0] *= 1e4
    q[0, 0, 1] = 0
    q[0, 0, 2] *= -1e4
    q[0, 0, 3] = 1e-30
    announce("window extreme scores")
    out, lse = run_window(c, q, 1000, 0)
    check(c, q, out, lse, *S.window_decode(q.double().numpy(), *c.np64(), c.table, (90,), 1000, 0))


def test_scores_that_rise_late():
    """Keys along q that grow with the position: the running maximum moves in
    every tile, by less and by more than the slack kept."""
    L = 700
    for step in (0.05, 0.5):
        c = Cache(7, (L,), 1, 64, 32, "f32")
        q = c.query(1, 1, "f32")
        u = q[0, 0, 0] / q[0, 0, 0].norm()
        t = np.arange(L)
        ramp = torch.from_numpy(step * t / float(q[0, 0, 0].norm())).float()
        c.k[c.table[0, t // 32], 0, t % 32] = ramp[:, None] * u
        announce(f"window ramp {step}")
        out, lse = run_window(c, q, L, 0)
        check(c, q, out, lse, *S.window_decode(q.double().numpy(), *c.np64(), c.table, (L,), L, 0))


@pytest.mark.parametrize("kv,qt,n", [("bf16", "f32", 1), ("bf16", "bf16", 40), ("f32", "f32", 1),
                                     ("f32", "f32", 35)])
def test_one_long_sequence_among_many_short(kv, qt, n):
    """As many row blocks as workgroups are wanted, so one part each: the long
    one's waves go through their page lists several times."""
    lens = [9001] + [n + b % 3 for b in range(519 if n == 1 else 299)]
    c = Cache(24, lens, 1, 64, 16, kv, max_pages=-(-9001 // 16))
    q = c.query(n, 1, qt)
    announce(f"window long among short {kv}/{qt} n{n}")
    out, lse = run_window(c, q, 1 << 30, 0)
    some = [0, 1, 2, len(lens) - 1]
    few = Cache.__new__(Cache)
    few.__dict__.update(c.__dict__)
    few.lens, few.table = [lens[b] for b in some], c.table[some]
    check(few, q[some], out[some], lse[some], *reference(few, q[some], few.lens, 1 << 30, 0, n))


def test_pool_beyond_32_bits():
    """Pages at the end of a 4.9 GB pool (2.4e9 values a pool)."""
    pages, ps, D, L = 300000, 64, 128, 500
    k, v = (torch.empty(pages, 1, ps, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rng = np.random.default_rng(25)
    c = Cache(25, (L,), 1, D, ps, "bf16")
    far = torch.arange(pages - c.mp, pages, dtype=torch.int32)[None]
    for dst, src in ((k, c.k), (v, c.v)):
        dst[far[0].long().cuda()] = src[torch.from_numpy(c.table[0]).long()].cuda()
    shape = E().make_shape(1, 4, 1, D, ps, c.mp, pages, "bf16")
    bt, lens = far.cuda(), torch.tensor([L], dtype=torch.int32, device="cuda")
    announce("softmax large pool")
    for n, rows in ((1, 4), (20, 80)):
        q = c.query(n, 4, "f32")
        out = torch.empty(q.shape, device="cuda")
        lse = torch.empty(q.shape[:-1], device="cuda")
        E().entmaxkv_softmax_window(shape, q.cuda(), k, v, bt, lens, 300, 4, out, lse, q_tokens=n)
        torch.cuda.synchronize()
        check(c, q, out, lse, *reference(c, q, (L,), 300, 4, rows))


# ---------------------------------------------------------------------------
# shared prefix


def run_prefix(c, q, pages, empty=0, **kw):
    k, v, pt = c.dev("k", "v", "prefix_table")
    shape, qd, bt, lens = padded(c, q, empty)
    bt[:, :pages] = -1  # not read
    qd = qd[:, 0].contiguous()
    out = torch.full_like(qd, float("nan"))
    lse = torch.full(qd.shape[:-1], float("nan"), device="cuda")
    E().entmaxkv_softmax_prefix(shape, qd, k, v, pt, pages, bt, lens, out, lse, **kw)
    torch.cuda.synchronize()
    return unpadded(len(q), out[:, None], lse[:, None])


@pytest.mark.parametrize("kv,qt,D,ps,Hkv,G,B,pages", [
    ("bf16", "bf16", 128, 16, 2, 4, 3, 7),
    ("bf16", "f32", 128, 32, 1, 8, 19, 5),
    ("bf16", "bf16", 64, 64, 2, 2, 33, 3),
    ("bf16", "f32", 64, 16, 1, 1, 50, 20),
    ("f32", "f32", 128, 16, 1, 4, 9, 9),
    ("f32", "f32", 64, 64, 2, 1, 40, 2),
    ("bf16", "bf16", 128, 32, 1, 8, 70, 40),
    ("bf16", "f32", 128, 16, 1, 8, 130, 11),
])
def test_prefix(kv, qt, D, ps, Hkv, G, B, pages):
    P = pages * ps
    # padded, shorter than the prefix, exactly it, one past it, longer ones
    lens = [(P + 37, 0, P, P + 1, P // 2 + 3, 1, P + ps, P + 150)[b % 8] for b in range(B)]
    c = Cache(11, lens, Hkv, D, ps, kv, prefix_pages=pages)
    q = c.query(1, Hkv * G, qt)
    announce(f"prefix {kv}/{qt} D{D} ps{ps} Hkv{Hkv} G{G} B{B} pages{pages}")
    # (as many rows as a KV head needs for the many-rows form, empty sequences)
    rows = 16 * 1100 // (Hkv * max(1, P // 32))
    for empty in (0, rows // G):
        out, lse = run_prefix(c, q, pages, empty)
        check(c, q, out, lse, *reference(c, q, lens, 1 << 30, 0, B * G + empty * G))


@pytest.mark.parametrize("times", [1, 15])
def test_prefix_is_the_whole_table(times):
    P = 4 * 16
    c = Cache(12, [P, P, 20] * times, 1, 64, 16, "bf16", prefix_pages=4, max_pages=4)
    q = c.query(1, 4, "f32")
    announce("prefix whole table")
    out, lse = run_prefix(c, q, 4, 0 if times == 1 else 4 * 1100)
    check(c, q, out, lse, *S.window_decode(q.double().numpy(), *c.np64(), c.table, c.lens,
                                           1 << 30, 0))


@pytest.mark.parametrize("times", [1, 4])
@pytest.mark.parametrize("kv,qt", [("bf16", "bf16"), ("f32", "f32")])
def test_prefix_values_hidden_from_short_sequences(kv, qt, times):
    """A prefix value that is not finite, behind the end of some sequences of
    the batch: only the others' outputs hold it."""
    P = 6 * 16
    lens = [P + 3, 50, P, 0, 60, 61] * times
    c = Cache(13, lens, 1, 64, 16, kv, prefix_pages=6)
    c.v[c.table[0, 60 // 16], 0, 60 % 16, 7] = math.inf
    q = c.query(1, 2, qt)
    announce(f"prefix infinite value {kv}")
    empty = 0 if times == 1 else 16 * 1100 // 3
    out, lse = run_prefix(c, q, 6, empty)
    ref, ref_lse, mean_abs = reference(c, q, lens, 1 << 30, 0, 2 * (len(lens) + empty))
    o = out.double().cpu().numpy()
    sees = np.array(lens) > 60
    assert not np.isfinite(o[sees][..., 7]).any()
    o[sees, ..., 7] = 0
    ref[sees, ..., 7] = 0
    mean_abs = np.nan_to_num(mean_abs, posinf=0.0)
    check(c, q, torch.from_numpy(o), lse, ref, ref_lse, mean_abs)


def test_prefix_equals_window_over_the_same_pages():
    """The batch's shared pages read once give what each sequence gives on its
    own, within both calls' tolerance."""
    lens = [300 + 17 * b for b in range(24)]
    c = Cache(14, lens, 2, 128, 32, "bf16", prefix_pages=8)
    q = c.query(1, 8, "f32")
    announce("prefix against window")
    a, la = run_prefix(c, q, 8)
    b, lb = run_window(c, q, 1 << 30, 0)
    assert torch.allclose(a, b, atol=2e-5, rtol=0) and torch.allclose(la, lb, atol=1e-5, rtol=0)


@pytest.mark.parametrize("qt", ["bf16", "f32"])
def test_long_prefix_for_many(qt):
    """Workgroups of the prefix part go through their page list more than
    once; against the window call over each sequence, within both calls'
    tolerance (bf16: two roundings of the output and one of each weight)."""
    P, B = 6000 if qt == "f32" else 11300, 900
    c = Cache(15, [P * 16 + b % 5 for b in range(2)], 1, 64, 16, "bf16", prefix_pages=P)
    table = np.concatenate([np.tile(c.prefix_table, (B, 1)),
                            np.tile(c.table[:1, P:], (B, 1))], 1)
    lens = torch.tensor([P * 16 - 37 * (b % 7) for b in range(B)], dtype=torch.int32).cuda()
    gen = torch.Generator().manual_seed(3)
    q = (torch.randn(B, 1, 64, generator=gen) * 0.3).to(
        torch.bfloat16 if qt == "bf16" else torch.float32).cuda()
    k, v, pt = c.dev("k", "v", "prefix_table")
    bt = torch.from_numpy(table.astype(np.int32)).cuda()
    shape = E().make_shape(B, 1, 1, 64, 16, c.mp, c.pages, "bf16")
    a, b = torch.empty_like(q), torch.empty_like(q)
    la, lb = (torch.empty(B, 1, device="cuda") for _ in range(2))
    announce(f"prefix long {qt}")
    E().entmaxkv_softmax_prefix(shape, q, k, v, pt, P, bt, lens, a, la)
    E().entmaxkv_softmax_window(shape, q, k, v, bt, lens, 1 << 30, 0, b, lb)
    torch.cuda.synchronize()
    assert torch.allclose(la, lb, atol=2e-5, rtol=0)
    err = (a.double() - b.double()).abs()
    # the outputs average about 1e5 values of size 1: |out| is about 1e-2
    assert err.max() <= (2e-5 if qt == "f32" else 2.0**-7 * b.abs().max().item() + 2.0**-8)


# ---------------------------------------------------------------------------
# how it is called


def test_streams_workspaces_and_repeats():
    c = Cache(21, (900, 40, 1300), 2, 128, 16, "bf16")
    q = c.query(1, 8, "bf16")
    k, v, bt, lens = c.dev("k", "v", "table", "lens")
    s, qd = c.shape(8), q.cuda()
    announce("softmax streams")
    want, want_lse = run_window(c, q, 600, 4)
    # a given workspace, a side stream, a stream handle, no lse
    ws = torch.empty(E().entmaxkv_softmax_window_ws(s, 1, 600, 4), dtype=torch.uint8,
                     device="cuda")
    side = torch.cuda.Stream()
    outs = [torch.empty_like(qd) for _ in range(4)]
    side.wait_stream(torch.cuda.current_stream())
    E().entmaxkv_softmax_window(s, qd, k, v, bt, lens, 600, 4, outs[0], ws=ws)
    torch.cuda.synchronize()
    E().entmaxkv_softmax_window(s, qd, k, v, bt, lens, 600, 4, outs[1], stream=side)
    E().entmaxkv_softmax_window(s, qd, k, v, bt, lens, 600, 4, outs[2], stream=side.cuda_stream)
    torch.cuda.synchronize()
    call = E().Prepared("softmax_window", s, qd, k, v, bt, lens, 600, 4, outs[3])
    call()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_graph_replays_follow_the_inputs():
    """Two captured calls with workspaces of their own, replayed with new
    queries and lengths, eager calls between the replays."""
    c = Cache(22, (900, 40, 1300), 2, 128, 16, "bf16", prefix_pages=2)
    q = c.query(1, 8, "f32").cuda()
    k, v, bt, lens, pt = c.dev("k", "v", "table", "lens", "prefix_table")
    s = c.shape(8)
    out, out2 = torch.empty_like(q), torch.empty_like(q[:, 0])
    announce("softmax graph")
    calls = [E().Prepared("softmax_window", s, q, k, v, bt, lens, 600, 4, out, stream=st)
             for st in (None,)]
    calls.append(E().Prepared("softmax_prefix", s, q, k, v, pt, 2, bt, lens, out2))
    for call in calls:
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        captured = [E().Prepared("softmax_window", s, q, k, v, bt, lens, 600, 4, out),
                    E().Prepared("softmax_prefix", s, q, k, v, pt, 2, bt, lens, out2)]
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            for call in captured:
                call()
    gen = torch.Generator(device="cuda").manual_seed(5)
    for step in range(4):
        q.normal_(0, 0.2, generator=gen)
        lens.copy_(torch.tensor([900 - 31 * step, 40, 1300 - step], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone(), out2.clone()
        for call in calls:
            call()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], out2)


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with a workspace of its own."""
    c = Cache(26, [1200 + 9 * b for b in range(12)], 2, 128, 16, "bf16", prefix_pages=20)
    q = c.query(1, 8, "bf16")
    announce("softmax two streams")
    want, _ = run_window(c, q, 700, 4)
    want2, _ = run_prefix(c, q, 20)
    k, v, bt, lens, pt = c.dev("k", "v", "table", "lens", "prefix_table")
    qd = q.cuda()
    q3 = qd[:, 0].contiguous()
    outs = [(torch.empty_like(qd), torch.empty_like(q3)) for _ in range(6)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for o, o2 in outs:
        E().entmaxkv_softmax_window(c.shape(8), qd, k, v, bt, lens, 700, 4, o, stream=streams[0])
        E().entmaxkv_softmax_prefix(c.shape(8), q3, k, v, pt, 20, bt, lens, o2, stream=streams[1])
    torch.cuda.synchronize()
    for o, o2 in outs:
        assert torch.equal(o, want) and torch.equal(o2, want2[:, 0])


def test_full_window_is_the_softmax_full_decode():
    """window = FULL_WINDOW, no sinks: every valid token."""
    lens = (513, 64, 2000)
    c = Cache(23, lens, 2, 64, 32, "f32")
    q = c.query(1, 4, "f32")
    announce("softmax full")
    out, lse = run_window(c, q, E().FULL_WINDOW, 0)
    check(c, q, out, lse, *S.window_decode(q.double().numpy(), *c.np64(), c.table, lens, 1 << 30, 0))
