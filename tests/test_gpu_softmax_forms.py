"""Softmax decode on the GPU: what must not depend on which form of the
attention kernel a call runs (few rows: 16 rows a workgroup; many rows: row
tiles of their own for every wave)."""
import numpy as np
import pytest
import torch

from oracle import softmax_oracle as S
from parity_util import announce
from test_gpu_softmax import (Cache, E, check, empties, padded, reference, run_prefix, run_window,
                              unpadded)

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


def form(shape, q, window=1 << 30, sinks=0, prefix_pages=0):
    e = E()
    qd = e.ENTMAXKV_BF16 if q.dtype == torch.bfloat16 else e.ENTMAXKV_F32
    got = e.entmaxkv_softmax_form(shape, qd, q.shape[1], window, sinks, prefix_pages)
    return {e.ENTMAXKV_FORM_FEW_ROWS: "few", e.ENTMAXKV_FORM_MANY_ROWS: "many"}[got]


def window_cases(c, q, window=1 << 30, sinks=0):
    """Numbers of empty sequences beside those of c that make the call run each
    form that so many rows can run."""
    out = [0] + ([empties(c, q, 4200)] if q.shape[1] * q.shape[2] // c.Hkv >= 33 else [])
    for empty, want in zip(out, ("few", "many")):
        assert form(padded(c, q, empty)[0], q, window, sinks) == want
    return out


def prefix_empties(c, q, pages):
    """Empty sequences that bring a KV head's rows over 1024 tiles of 16 of
    them and 32 (float32: 16) prefix tokens."""
    G = q.shape[2] // c.Hkv
    return 16 * 1100 // (G * c.Hkv * max(1, pages * c.ps // 32))

# exp of minus these 64ths lies as far as it can (0.57 to 0.79 of 2^-15 of
# itself) above what two cut-off bf16 parts hold of it, and up to 2^-8 away
# from the nearest single bf16
LEVELS = np.array([13, 22, 42, 44, 71, 77, 80, 85, 105, 110, 112, 121]) / 64.0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,L", [(1, 32), (8, 64)])
def test_bf16_queries_lose_nothing_but_the_outputs_rounding(n, L, D):
    """Scores are exact here (every query picks one coordinate of the keys, a
    multiple of 2^-6), and values are 1 or 1 + 2^-7, next to each other in
    bf16: an output is one of them, at most half a step, 2^-8, off plus what
    the weights are off. That is 2^-17 of each (8 bits, then 8 of the rest,
    both to the nearest), 2^-21 for its exponential and as much in the sum l,
    and 60 roundings of 2^-24 of the sums (16 a tile of 32 tokens, two tiles,
    18 of l, the reciprocal and the join)."""
    B, G = 16 // n, 8
    c = Cache(71, (L,) * B, 1, D, 32, "bf16")
    q = torch.zeros(B, n, G, D, dtype=torch.bfloat16)
    for i in range(n):
        for h in range(G):
            q[:, i, h, i * G + h] = 1.0
    t = np.arange(L)
    for b in range(B):
        z = -c.rng.choice(LEVELS, size=(L, D))
        z[0] = 0.0  # the largest score comes first: the weights are exp(z)
        v = 1.0 + 2.0**-7 * c.rng.integers(0, 2, size=(L, D))
        at = c.table[b, t // 32], 0, t % 32
        c.k[at] = torch.from_numpy(z).to(torch.bfloat16)
        c.v[at] = torch.from_numpy(v).to(torch.bfloat16)
    assert (c.k[c.table[0, 0], 0, 1:, 0].double() * 64 % 1 == 0).all()
    ref, ref_lse = S.window_decode(q.double().numpy(), *c.np64(), c.table, c.lens, 1 << 30, 0)
    off = (2.0**-17 + 2 * 2.0**-21 + 60 * 2.0**-24) * ref
    # (64 rows a KV head: also among enough empty sequences for the other form)
    for empty in window_cases(c, q):
        announce(f"bf16 queries' weights n{n} L{L} D{D}, {empty} empty sequences")
        out, lse = run_window(c, q, 1 << 30, 0, empty)
        over = np.abs(out.double().cpu().numpy() - ref) - 2.0**-8 - off
        assert over.max() <= 0, (float(over.max()), int((over > 0).sum()))
        # 2^-21 of the weights, 18 roundings of l, 8 of 2^-23 of the logarithm and 4 + 4 after it
        assert np.abs(lse.double().cpu().numpy() - ref_lse).max() <= 2.0**-21 + 42 * 2.0**-24


# ---------------------------------------------------------------------------
# scores of every size


@pytest.mark.parametrize("kv,qt", TYPES)
@pytest.mark.parametrize("n", [1, 12])
def test_extreme_scores(kv, qt, n):
    """Scores of +-60000 and all equal; a row of zeros; per query token."""
    L = 90
    c = Cache(72, (L,), 1, 64, 16, kv)
    q = c.query(n, 4, qt)
    q[:, :, 0] *= 1e4
    q[:, :, 1] = 0
    q[:, :, 2] *= -1e4
    q[:, :, 3] = 1e-30
    ref = S.window_decode(q.double().numpy(), *c.np64(), c.table, (L,), 1000, 0)
    for empty in window_cases(c, q, 1000):
        announce(f"extreme scores {kv}/{qt} n{n}, {empty} empty sequences")
        out, lse = run_window(c, q, 1000, 0, empty)
        check(c, q, out, lse, *ref)


@pytest.mark.parametrize("kv,qt", TYPES)
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("step", [0.05, 0.5, -0.5])
def test_scores_that_rise_late(kv, qt, n, step):
    """Keys along q that grow (or fall) with the position: the reference of the
    weights moves in every tile, by less and by more than the slack kept, and
    in one of a wave's two row tiles only (every second query is turned
    round)."""
    L = 700
    c = Cache(73, (L,), 1, 64, 32, kv)
    q = c.query(1, 1, "f32")[0, 0, 0]
    u = q / q.norm()
    flip = torch.where(torch.arange(n) // 16 % 2 == 0, 1.0, -1.0)
    qs = (flip[:, None] * q).view(1, n, 1, 64).to(torch.bfloat16 if qt == "bf16" else torch.float32)
    t = np.arange(L)
    ramp = torch.from_numpy(step * t / float(q.norm())).float()
    c.k[c.table[0, t // 32], 0, t % 32] = (ramp[:, None] * u).to(c.k.dtype)
    ref = S.window_decode(qs.double().numpy(), *c.np64(), c.table, (L,), L, 0)
    for empty in window_cases(c, qs, L):
        announce(f"ramp {step} {kv}/{qt} n{n}, {empty} empty sequences")
        out, lse = run_window(c, qs, L, 0, empty)
        check(c, qs, out, lse, *ref)


@pytest.mark.parametrize("kv,qt", TYPES)
def test_rising_and_extreme_scores_over_a_prefix(kv, qt):
    B, P = 12, 20
    c = Cache(74, [P * 16 + 9 * b for b in range(B)], 1, 64, 16, kv, prefix_pages=P)
    q = c.query(1, 4, qt)
    u = q[0, 0, 0].float() / q[0, 0, 0].float().norm()
    t = np.arange(P * 16)
    c.k[c.prefix_table[t // 16], 0, t % 16] = (torch.from_numpy(0.3 * t).float()[:, None]
                                               * u).to(c.k.dtype)
    q[:, :, 1] *= 1e3
    q[:, :, 2] = 0
    ref = S.window_decode(q.double().numpy(), *c.np64(), c.table, c.lens, 1 << 30, 0)
    for empty, want in ((0, "few"), (prefix_empties(c, q, P), "many")):
        assert form(padded(c, q, empty)[0], q, prefix_pages=P) == want
        announce(f"prefix ramp {kv}/{qt}, {empty} empty sequences")
        out, lse = run_prefix(c, q, P, empty)
        check(c, q, out, lse, *ref)


@pytest.mark.parametrize("kv,qt", TYPES)
@pytest.mark.parametrize("L,n,G,window,sinks", [(50001, 40, 1, 1 << 30, 0),
                                                (20011, 33, 4, 19000, 40)])
def test_one_long_chunk(kv, qt, L, n, G, window, sinks):
    """Many rows, few blocks of them: their tokens in many parts, joined."""
    c = Cache(79, (L,), 1, 64, 16, kv)
    q = c.query(n, G, qt)
    shape = padded(c, q, 0)[0]
    assert form(shape, q, window, sinks) == "many"
    assert E().entmaxkv_softmax_window_ws(shape, n, window, sinks) > 0
    announce(f"long chunk {kv}/{qt} L{L} n{n} G{G}")
    out, lse = run_window(c, q, window, sinks)
    check(c, q, out, lse, *S.window_decode(q.double().numpy(), *c.np64(), c.table, (L,), window,
                                           sinks))


# ---------------------------------------------------------------------------
# a large pool


@pytest.mark.parametrize("qt", ["bf16", "f32"])
def test_pool_beyond_32_bits_many_rows(qt):
    """Pages at the end of a 4.9 GB pool, for a chunk of queries and for a
    shared prefix."""
    pages, ps, D, L, P = 300000, 64, 128, 500, 5
    k, v = (torch.empty(pages, 1, ps, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c = Cache(75, (L,), 1, D, ps, "bf16")
    far = np.arange(pages - c.mp, pages, dtype=np.int32)[None]
    for dst, src in ((k, c.k), (v, c.v)):
        dst[torch.from_numpy(far[0]).long().cuda()] = src[torch.from_numpy(c.table[0]).long()].cuda()
    at = Cache.__new__(Cache)
    at.__dict__.update(c.__dict__, table=far, pages=pages)
    q = c.query(20, 4, qt)
    shape, qd, bt, lens = padded(at, q, empties(c, q, 4200))
    assert form(shape, q, 300, 4) == "many"
    announce(f"large pool, many rows {qt}")
    out, lse = torch.empty_like(qd), torch.empty(qd.shape[:-1], device="cuda")
    E().entmaxkv_softmax_window(shape, qd, k, v, bt, lens, 300, 4, out, lse, q_tokens=20)
    torch.cuda.synchronize()
    check(c, q, *unpadded(1, out, lse), *S.window_decode(q.double().numpy(), *c.np64(), c.table,
                                                         (L,), 300, 4))

    q = c.query(1, 4, qt)
    shape, qd, bt, lens = padded(at, q, prefix_empties(c, q, P))
    assert form(shape, q, prefix_pages=P) == "many"
    announce(f"large pool, prefix, many rows {qt}")
    out, lse = torch.empty_like(qd), torch.empty(qd.shape[:-1], device="cuda")
    E().entmaxkv_softmax_prefix(shape, qd, k, v, torch.from_numpy(far[0, :P].copy()).cuda(), P, bt,
                                lens, out, lse)
    torch.cuda.synchronize()
    check(c, q, *unpadded(1, out, lse), *S.window_decode(q.double().numpy(), *c.np64(), c.table,
                                                         (L,), 1 << 30, 0))


# ---------------------------------------------------------------------------
# how the many-rows form is called


class Both:
    """A chunk call and a prefix call of the many-rows form over one cache."""

    def __init__(self, seed, qt):
        c = self.c = Cache(seed, (900, 40, 1300), 2, 128, 16, "bf16", prefix_pages=2)
        chunk, one = c.query(40, 8, qt), c.query(1, 8, qt)
        n = empties(c, chunk, 4200)
        self.wshape, self.q, self.wbt, self.wlens = padded(c, chunk, n)
        assert form(self.wshape, chunk, 600, 4) == "many"
        self.pshape, q1, self.pbt, self.plens = padded(c, one, prefix_empties(c, one, 2))
        assert form(self.pshape, one, prefix_pages=2) == "many"
        self.q1 = q1[:, 0].contiguous()
        self.k, self.v, self.pt = c.dev("k", "v", "prefix_table")

    def outs(self):
        return [torch.full_like(self.q, -7.0), torch.full(self.q.shape[:-1], -7.0, device="cuda"),
                torch.full_like(self.q1, -7.0), torch.full(self.q1.shape[:-1], -7.0, device="cuda")]

    def calls(self, outs, **kw):
        o, e, o1, e1 = outs
        return (E().Prepared("softmax_window", self.wshape, self.q, self.k, self.v, self.wbt,
                             self.wlens, 600, 4, o, lse=e, q_tokens=40, **kw),
                E().Prepared("softmax_prefix", self.pshape, self.q1, self.k, self.v, self.pt, 2,
                             self.pbt, self.plens, o1, lse=e1, **kw))


@pytest.mark.parametrize("qt", ["bf16", "f32"])
def test_graph_replays_of_the_many_rows_form(qt):
    """Captured once, replayed with new queries and lengths, eager calls between
    the replays."""
    x = Both(76, qt)
    outs, got = x.outs(), x.outs()
    announce(f"many rows graph {qt}")
    eager = x.calls(outs)
    for call in eager:
        call()
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        captured = x.calls(got)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            for call in captured:
                call()
    gen = torch.Generator(device="cuda").manual_seed(5)
    for step in range(4):
        x.q.normal_(0, 0.2, generator=gen)
        x.q1.normal_(0, 0.2, generator=gen)
        for lens in (x.wlens, x.plens):
            lens[:3] = torch.tensor([900 - 31 * step, 40 - step, 1300 - step])
        g.replay()
        torch.cuda.synchronize()
        for call in eager:
            call()
        torch.cuda.synchronize()
        for a, b in zip(got, outs):
            assert torch.equal(a, b)
    # and the eager results are right
    c = Cache.__new__(Cache)
    c.__dict__.update(x.c.__dict__, lens=x.wlens[:3].tolist())
    q, q1 = x.q[:3].cpu(), x.q1[:3, None].cpu()
    check(c, q, outs[0][:3], outs[1][:3], *S.window_decode(q.double().numpy(), *c.np64(), c.table,
                                                           c.lens, 600, 4))
    check(c, q1, outs[2][:3, None], outs[3][:3, None],
          *S.window_decode(q1.double().numpy(), *c.np64(), c.table, c.lens, 1 << 30, 0))


@pytest.mark.parametrize("qt", ["bf16", "f32"])
def test_two_streams_of_the_many_rows_form(qt):
    """Chunk and prefix calls that overlap on two streams, each with a
    workspace of its own, against calls one after the other."""
    x = Both(77, qt)
    want = x.outs()
    announce(f"many rows two streams {qt}")
    for call in x.calls(want):
        call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    several = [x.outs() for _ in range(6)]
    pairs = [[x.calls(o, stream=st)[i] for i, st in enumerate(streams)] for o in several]
    torch.cuda.synchronize()
    for pair in pairs:
        for call in pair:
            call()
    torch.cuda.synchronize()
    for outs in several:
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kv,qt", TYPES)
def test_prefix_equals_window_in_both_forms(kv, qt):
    """The batch's shared pages read once give what each sequence gives on its
    own; the oracle stands between the two calls."""
    lens = [300 + 17 * b for b in range(10)]
    c = Cache(78, lens, 2, 64, 32, kv, prefix_pages=8)
    q = c.query(1, 8, qt)
    ref = reference(c, q, lens, 1 << 30, 0, 0)
    announce(f"prefix against window {kv}/{qt}")
    check(c, q, *run_window(c, q, 1 << 30, 0), *ref)
    for empty, want in ((0, "few"), (prefix_empties(c, q, 8), "many")):
        assert form(padded(c, q, empty)[0], q, prefix_pages=8) == want
        check(c, q, *run_prefix(c, q, 8, empty), *ref)
