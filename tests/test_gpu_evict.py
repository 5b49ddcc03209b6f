"""Accumulated attention weights and eviction on the GPU against the float64
oracle, and a run of them together with the decodes.

Tolerance of a weight: the score's error ez (tests/test_gpu_softmax.py) and
that of tau as given (none: the same float32 on both sides) change exp(z -
tau) by a factor e^ez and 2^-22 of its exponential, and [(a-1) z - tau]_+^m by
at most m x^(m-1) ((a-1) ez + 2^-23 |(a-1) z|) with x <= 1, plus m + 2
roundings (2^-20 of a general power); the sum over G heads and the decayed
sum add G + 2 roundings of the total. Kept tokens and copied rows are exact.
"""
import math

import numpy as np
import pytest
import torch

from oracle import entmax_oracle as O
from oracle import softmax_oracle as S
from parity_util import announce
from test_gpu_softmax import Cache, E, check, run_window

pytestmark = pytest.mark.gpu


def taus(c, q, alpha, window=1 << 30, sinks=0):
    """The float32 thresholds that a decode gives, from the float64 oracle."""
    k, _ = c.np64()
    B, H = len(c.lens), q.shape[2]
    out = np.zeros((B, H), np.float32)
    for b, L in enumerate(c.lens):
        t = S.visible(L - 1, L, window, sinks)
        for h in range(H):
            z = S.rows(k, c.table[b], h // (H // c.Hkv), t) @ q[b, 0, h].double().numpy()
            if len(z) == 0:
                out[b, h] = -math.inf if alpha == 1.0 else math.nan
            elif alpha == 1.0:
                out[b, h] = z.max() + math.log(np.exp(z - z.max()).sum())
            else:
                out[b, h] = O.entmax(z, alpha)[1]
    return out


def weight_tolerance(c, q, alpha, ref, old, decay):
    k, _ = c.np64()
    D, G = c.D, q.shape[2] // c.Hkv
    R = (12 * D // 32 if c.kv == "bf16" else D) + 4
    fk = np.where(np.isfinite(k), np.abs(k), 0.0).reshape(-1, D)
    big = (np.abs(q.double().numpy()).reshape(-1, D) @ fk.T).max()
    ez = R * 2.0**-24 * big
    if alpha == 1.0:
        per = ez + 2.0**-22
        return G * per * 1.0 + (G + 2) * 2.0**-24 * np.abs(ref) + 2.0**-24 * np.abs(decay * old)
    m = 1.0 / (alpha - 1.0)
    per = m * ((alpha - 1.0) * ez + 2.0**-23 * (alpha - 1.0) * big) + (m + 2) * 2.0**-20
    return G * per + (G + 2) * 2.0**-24 * np.abs(ref) + 2.0**-24 * np.abs(decay * old)


def run_weights(c, q, alpha, tau, old, decay, window=None, sinks=0, in_place=False):
    k, bt, lens = c.dev("k", "table", "lens")
    w = None if old is None else torch.from_numpy(old).cuda()
    cells = c.mp * c.ps
    new = w if in_place else torch.full((len(c.lens), c.Hkv, cells), -7.0, device="cuda")
    E().entmaxkv_accumulate_weights(c.shape(q.shape[2]), q[:, 0].contiguous().cuda(), k, bt, lens,
                                    alpha, torch.from_numpy(tau).cuda(), decay, w, new,
                                    window=window or E().FULL_WINDOW, sinks=sinks)
    torch.cuda.synchronize()
    return new.double().cpu().numpy()


@pytest.mark.parametrize("kv,qt,D,ps,Hkv,G,alpha", [
    ("bf16", "bf16", 128, 16, 2, 4, 1.0),
    ("bf16", "f32", 128, 32, 1, 8, 1.5),
    ("bf16", "f32", 64, 64, 2, 1, 2.0),
    ("bf16", "f32", 64, 16, 1, 2, 1.25),
    ("bf16", "bf16", 64, 32, 1, 8, 1.7),
    ("f32", "f32", 128, 64, 1, 4, 1.0),
    ("f32", "f32", 64, 16, 2, 2, 4.0 / 3.0),
    ("f32", "f32", 128, 32, 1, 1, 1.5),
])
def test_weights(kv, qt, D, ps, Hkv, G, alpha):
    lens = (0, 1, ps, ps + 1, 31, 33, 600)
    c = Cache(31, lens, Hkv, D, ps, kv)
    q = c.query(1, Hkv * G, qt, 4.0)
    tau = taus(c, q, alpha)
    old = c.rng.random((len(lens), Hkv, c.mp * ps)).astype(np.float32)
    announce(f"weights {kv}/{qt} D{D} ps{ps} G{G} alpha {alpha:.3f}")
    got = run_weights(c, q, alpha, tau, old, 0.75)
    a32 = float(np.float32(alpha))
    ref = S.weights(q[:, 0].double().numpy(), c.np64()[0], c.table, lens, a32,
                    tau.astype(np.float64), 1 << 30, 0, 0.75, old)
    tol = weight_tolerance(c, q, alpha, ref, old, 0.75)
    for b, L in enumerate(lens):
        err = np.abs(got[b, :, :L] - ref[b, :, :L])
        assert (err <= tol[b, :, :L]).all(), (b, float((err / tol[b, :, :L]).max()))
        assert (got[b, :, L:] == -7.0).all()


def test_weights_window_in_place_and_from_nothing():
    lens, window, sinks = (0, 90, 333), 50, 3
    c = Cache(32, lens, 2, 64, 16, "bf16")
    q = c.query(1, 8, "f32")
    tau = taus(c, q, 1.0, window, sinks)
    old = c.rng.random((3, 2, c.mp * 16)).astype(np.float32)
    announce("weights window, in place")
    ref = S.weights(q[:, 0].double().numpy(), c.np64()[0], c.table, lens, 1.0,
                    tau.astype(np.float64), window, sinks, 1.0, old)
    got = run_weights(c, q, 1.0, tau, old, 1.0, window, sinks, in_place=True)
    assert (np.abs(got - ref) <= weight_tolerance(c, q, 1.0, ref, old, 1.0)).all()
    # behind the lengths: untouched, bit for bit
    for b, L in enumerate(lens):
        assert (got[b, :, L:] == old[b, :, L:].astype(np.float64)).all()
    none = run_weights(c, q, 1.0, tau, None, 1.0, window, sinks)
    ref0 = S.weights(q[:, 0].double().numpy(), c.np64()[0], c.table, lens, 1.0,
                     tau.astype(np.float64), window, sinks, 1.0, np.zeros_like(old))
    for b, L in enumerate(lens):
        t = weight_tolerance(c, q, 1.0, ref0, np.zeros_like(old), 1.0)[b, :, :L]
        assert (np.abs(none[b, :, :L] - ref0[b, :, :L]) <= t).all()
        hidden = [x for x in range(L) if x not in S.visible(L - 1, L, window, sinks)]
        assert (none[b][:, hidden] == 0).all()


def test_weights_of_the_librarys_own_decode():
    """tau of decode_full in, total weight G per KV head out (probabilities)."""
    lens = (700, 64)
    c = Cache(33, lens, 2, 128, 32, "bf16")
    q = c.query(1, 8, "f32", 6.0)
    k, v, bt, ln = c.dev("k", "v", "table", "lens")
    out, tau = torch.empty(2, 8, 128, device="cuda"), torch.empty(2, 8, device="cuda")
    qd = q[:, 0].contiguous().cuda()
    announce("weights of decode_full")
    E().entmaxkv_decode_full(c.shape(8), qd, k, v, bt, ln, 1.5, out, tau=tau)
    got = run_weights(c, q, 1.5, tau.cpu().numpy(), None, 1.0)
    for b, L in enumerate(lens):
        total = got[b, :, :L].sum(-1)
        # tau is within 2e-5: a support of n tokens changes by n times that
        assert np.abs(total - 4).max() < 4 * 2 * 4e-5 * L**0.5 + 1e-3


# ---------------------------------------------------------------------------
# eviction


def run_evict(c, w, keep, sinks, recent, fresh=None, with_weights=True):
    B, ps = len(c.lens), c.ps
    need = -(-keep // ps)
    k, v, bt, lens = c.dev("k", "v", "table", "lens")
    if fresh is None:  # fresh pages behind the pool's
        fresh = c.rng.permutation(B * need).reshape(B, need) + c.pages
    grow = torch.full((B * need, *k.shape[1:]), 3.0, dtype=k.dtype, device="cuda")
    k, v = torch.cat([k, grow]), torch.cat([v, grow])
    nt = torch.full((B, c.mp), -1, dtype=torch.int32)
    nt[:, :min(need, c.mp)] = torch.from_numpy(fresh.astype(np.int32))[:, :c.mp]
    shape = E().make_shape(B, c.Hkv, c.Hkv, c.D, ps, c.mp, k.shape[0], c.kv)
    wd = torch.from_numpy(w).cuda()
    kept = torch.full((B, c.Hkv, keep), -9, dtype=torch.int32, device="cuda")
    nl = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    nw = torch.full_like(wd, -9.0) if with_weights else None
    E().entmaxkv_evict(shape, k, v, bt, lens, wd, keep, sinks, recent, nt.cuda(), kept, nl, nw)
    torch.cuda.synchronize()
    return k.cpu(), v.cpu(), nt.numpy(), kept.cpu().numpy(), nl.cpu().numpy(), nw


def check_evict(c, w, keep, sinks, recent):
    k, v, nt, kept, nl, nw = run_evict(c, w, keep, sinks, recent)
    nw = nw.cpu().numpy()
    ps = c.ps
    bits = torch.int16 if c.kv == "bf16" else torch.int32
    kb, vb, k0, v0 = (x.view(bits).numpy() for x in (k, v, c.k, c.v))
    written = np.zeros((k.shape[0], c.Hkv, ps), bool)
    for b, L in enumerate(c.lens):
        n = min(L, keep)
        assert nl[b] == n
        for g in range(c.Hkv):
            want = S.evict_kept(w[b, g], L, keep, sinks, recent)
            assert kept[b, g].tolist() == want.tolist() + [-1] * (keep - n), (b, g)
            i = np.arange(n)
            at = nt[b, i // ps], g, i % ps
            assert (kb[at] == S.rows(k0, c.table[b], g, want)).all()
            assert (vb[at] == S.rows(v0, c.table[b], g, want)).all()
            written[at] = True
            assert (nw[b, g, :n].view(np.int32) == w[b, g, want].view(np.int32)).all()
            assert (nw[b, g, n:] == 0).all()
    # nothing else was written: old pages whole, unused slots as they were
    three = k.new_full((1,), 3.0).view(bits).numpy()[0]
    assert (kb[:c.pages] == k0).all() and (vb[:c.pages] == v0).all()
    rest = ~written[c.pages:]
    assert (kb[c.pages:][rest] == three).all() and (vb[c.pages:][rest] == three).all()


@pytest.mark.parametrize("kv,D,ps,Hkv,keep,sinks,recent", [
    ("bf16", 128, 16, 2, 100, 4, 16),
    ("bf16", 64, 32, 1, 33, 0, 0),
    ("bf16", 128, 64, 3, 1, 0, 1),
    ("f32", 64, 16, 2, 40, 7, 33),     # no places between
    ("f32", 128, 32, 1, 63, 0, 5),
    ("bf16", 64, 64, 1, 640, 65, 1),
    ("bf16", 64, 16, 2, 5000, 3, 100),  # more than the table holds
])
def test_evict(kv, D, ps, Hkv, keep, sinks, recent):
    lens = (0, 1, keep - 1, keep, keep + 1, 5 * keep + 3, 777) if keep < 777 else (0, 1, 450, 777)
    c = Cache(41, lens, Hkv, D, ps, kv)
    w = c.rng.random((len(lens), Hkv, c.mp * ps)).astype(np.float32) ** 8
    announce(f"evict {kv} D{D} ps{ps} Hkv{Hkv} keep{keep} sinks{sinks} recent{recent}")
    check_evict(c, w, keep, sinks, recent)


@pytest.mark.parametrize("kind", ["ties", "zero", "special", "wide"])
def test_evict_weights_of_every_kind(kind):
    lens = (1500, 4100, 90)
    c = Cache(42, lens, 1, 64, 16, "bf16")
    n = c.mp * 16
    w = c.rng.integers(0, 3, size=(3, 1, n)).astype(np.float32)
    if kind == "zero":
        w[:] = 0.0
        w[:, :, ::2] = -0.0
    elif kind == "special":
        for x in (np.nan, np.inf, -np.inf, -3.0, 1e-42, -1e-42):
            w[:, :, c.rng.integers(0, n, size=n // 9)] = x
        w[1, 0, 5] = -np.nan
    elif kind == "wide":
        w = (c.rng.random((3, 1, n)) * 80 - 40).astype(np.float32)
        w = np.exp2(w).astype(np.float32)
    announce(f"evict weights {kind}")
    check_evict(c, w, 300, 4, 20)


@pytest.mark.parametrize("L,keep", [(70000, 9000), (70001, 69999), (40000, 1)])
def test_evict_long(L, keep):
    c = Cache(43, (L,), 1, 64, 64, "bf16")
    w = c.rng.random((1, 1, c.mp * 64)).astype(np.float32) ** 4
    announce(f"evict long {L} keep {keep}")
    check_evict(c, w, keep, 0, 0)


def test_evict_pool_beyond_32_bits():
    """Old pages at the end of a 4.9 GB pool, new ones before them."""
    pages, ps, D, L, keep = 300000, 64, 128, 1000, 200
    k, v = (torch.empty(pages, 1, ps, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c = Cache(45, (L,), 1, D, ps, "bf16")
    far = torch.arange(pages - c.mp, pages, dtype=torch.int32)[None]
    for dst, src in ((k, c.k), (v, c.v)):
        dst[far[0].long().cuda()] = src[torch.from_numpy(c.table[0]).long()].cuda()
    shape = E().make_shape(1, 1, 1, D, ps, c.mp, pages, "bf16")
    nt = torch.full((1, c.mp), -1, dtype=torch.int32)
    nt[0, :4] = torch.arange(pages - c.mp - 9, pages - c.mp - 5)
    w = c.rng.random((1, 1, c.mp * ps)).astype(np.float32)
    kept = torch.empty(1, 1, keep, dtype=torch.int32, device="cuda")
    nl = torch.empty(1, dtype=torch.int32, device="cuda")
    ln = torch.tensor([L], dtype=torch.int32, device="cuda")
    announce("evict large pool")
    q = c.query(1, 1, "f32")
    got = torch.zeros(1, 1, c.mp * ps, device="cuda")
    tau = taus(c, q, 1.0)
    E().entmaxkv_accumulate_weights(shape, q[:, 0].contiguous().cuda(), k, far.cuda(), ln, 1.0,
                                    torch.from_numpy(tau).cuda(), 1.0, None, got)
    E().entmaxkv_evict(shape, k, v, far.cuda(), ln, torch.from_numpy(w).cuda(), keep, 2, 5,
                       nt.cuda(), kept, nl)
    torch.cuda.synchronize()
    ref = S.weights(q[:, 0].double().numpy(), c.np64()[0], c.table, (L,), 1.0,
                    tau.astype(np.float64), 1 << 30, 0, 1.0, np.zeros_like(w))
    assert (np.abs(got.double().cpu().numpy() - ref)
            <= weight_tolerance(c, q, 1.0, ref, np.zeros_like(w), 1.0)).all()
    want = S.evict_kept(w[0, 0], L, keep, 2, 5)
    assert kept[0, 0].tolist() == want.tolist() and nl.tolist() == [keep]
    for x, src in ((k, c.k), (v, c.v)):
        new = x[nt[0, :4].long().cuda(), 0].cpu().reshape(-1, D)[:keep]
        old = src[torch.from_numpy(c.table[0, want // ps]).long(), 0, torch.from_numpy(want % ps)]
        assert torch.equal(new.view(torch.int16), old.view(torch.int16))


def test_weights_many_sequences():
    """More than 64 sequences (the lengths are summed in groups of 64), most of
    them empty or short, a few long: every workgroup's share crosses ends."""
    lens = [0] * 70 + [700] + [b % 4 for b in range(80)] + [333, 0, 1200]
    c = Cache(34, lens, 2, 64, 32, "bf16")
    q = c.query(1, 4, "bf16")
    tau = taus(c, q, 1.0)
    announce("weights many sequences")
    got = run_weights(c, q, 1.0, tau, None, 1.0)
    zero = np.zeros(got.shape)
    ref = S.weights(q[:, 0].double().numpy(), c.np64()[0], c.table, lens, 1.0,
                    tau.astype(np.float64), 1 << 30, 0, 1.0, zero)
    tol = weight_tolerance(c, q, 1.0, ref, zero, 1.0)
    for b, L in enumerate(lens):
        assert (np.abs(got[b, :, :L] - ref[b, :, :L]) <= tol[b, :, :L]).all(), b
        assert (got[b, :, L:] == -7.0).all()


def test_weights_and_evict_in_a_graph():
    """Captured once, replayed with other weights and lengths, eager calls in
    between."""
    c = Cache(35, (300, 80, 511), 2, 64, 16, "bf16")
    B, keep, need = 3, 64, 4
    k, v, bt, ln = c.dev("k", "v", "table", "lens")
    grow = torch.zeros(B * need, *k.shape[1:], dtype=k.dtype, device="cuda")
    k, v = torch.cat([k, grow]), torch.cat([v, grow])
    nt = torch.full((B, c.mp), -1, dtype=torch.int32)
    nt[:, :need] = torch.arange(c.pages, c.pages + B * need).view(B, need)
    nt = nt.cuda()
    shape = E().make_shape(B, 4, 2, 64, 16, c.mp, k.shape[0], "bf16")
    q = c.query(1, 4, "f32")[:, 0].contiguous().cuda()
    tau = torch.full((B, 4), 3.0, device="cuda")
    w = torch.zeros(B, 2, c.mp * 16, device="cuda")
    kept = torch.empty(B, 2, keep, dtype=torch.int32, device="cuda")
    nl, nw = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty_like(w)

    def calls():
        return [E().Prepared("accumulate_weights", shape, q, k, bt, ln, 1.0, tau, 0.5, w, w),
                E().Prepared("evict", shape, k, v, bt, ln, w, keep, 2, 9, nt, kept, nl, nw)]

    announce("weights and evict graph")
    eager = calls()
    for call in eager:
        call()
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        captured = calls()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            for call in captured:
                call()
    gen = torch.Generator(device="cuda").manual_seed(6)
    for step in range(4):
        start = torch.rand(w.shape, device="cuda", generator=gen) * 0.1
        q.normal_(0, 0.3, generator=gen)
        ln.copy_(torch.tensor([300 - step, 80, 511 - 7 * step], dtype=torch.int32))
        got = []
        for run in (g.replay, lambda: [call() for call in eager]):
            w.copy_(start)
            k[c.pages:].zero_()
            v[c.pages:].zero_()
            torch.cuda.synchronize()
            run()
            torch.cuda.synchronize()
            got.append([x.clone() for x in (w, kept, nl, nw, k[c.pages:], v[c.pages:])])
        for a, b in zip(*got):
            assert torch.equal(a, b)


def test_evict_bad_pages_and_no_weights():
    """A table entry outside the pool, old or new: its slots are not copied."""
    c = Cache(44, (100, 100), 1, 64, 16, "f32")
    c.table[0, 2] = c.pages + 1000
    w = np.ones((2, 1, c.mp * 16), np.float32)
    fresh = np.array([[0, 1, 2], [3, 4, 5]]) + c.pages
    fresh[1, 1] = -5
    announce("evict bad pages")
    k, v, nt, kept, nl, nw = run_evict(c, w, 48, 0, 0, fresh, with_weights=False)
    assert nw is None and nl.tolist() == [48, 48]
    assert kept[0, 0].tolist() == kept[1, 0].tolist() == list(range(48))
    for b, i in ((0, 5), (0, 20), (1, 5), (1, 40)):
        assert torch.equal(k[nt[b, i // 16], 0, i % 16], c.k[c.table[b, i // 16], 0, i % 16])
    for p in (fresh[0, 2], fresh[1, 1] + c.pages + 9):
        if p < k.shape[0]:
            assert (k[p] == 3).all() and (v[p] == 3).all()
    assert (k[fresh[0, 2]] == 3).all() and (k[c.pages + 4] == 3).all()


# ---------------------------------------------------------------------------
# together


def test_decode_accumulate_evict_decode():
    """A serving run: softmax and alpha-entmax decodes add up the weights of a
    few steps, the cache is evicted, and both decodes, the page boxes and the
    top-k decode go on over the new pages as over a cache of the kept rows."""
    B, H, Hkv, D, ps, keep = 3, 8, 2, 64, 16, 64
    lens = [200, 60, 131]
    c = Cache(51, lens, Hkv, D, ps, "bf16")
    k, v, bt, ln = c.dev("k", "v", "table", "lens")
    shape0 = c.shape(H)
    w = torch.zeros(B, Hkv, c.mp * ps, device="cuda")
    out, lse = torch.empty(B, 1, H, D, device="cuda"), torch.empty(B, 1, H, device="cuda")
    o2, tau = torch.empty(B, H, D, device="cuda"), torch.empty(B, H, device="cuda")
    announce("decode, accumulate, evict, decode")
    want = np.zeros(w.shape)
    kk, vv = c.np64()
    for step in range(3):
        q = c.query(1, H, "f32", 5.0)
        qd = q.cuda()
        q3 = qd[:, 0].contiguous()
        E().entmaxkv_softmax_window(shape0, qd, k, v, bt, ln, E().FULL_WINDOW, 0, out, lse)
        E().entmaxkv_accumulate_weights(shape0, q3, k, bt, ln, 1.0, lse, 0.9, w, w)
        E().entmaxkv_decode_full(shape0, q3, k, v, bt, ln, 1.5, o2, tau=tau)
        E().entmaxkv_accumulate_weights(shape0, q3, k, bt, ln, 1.5, tau, 1.0, w, w)
        for a, d in ((1.0, 0.9), (1.5, 1.0)):
            want = S.weights(q[:, 0].double().numpy(), kk, c.table, lens, a,
                             taus(c, q, a).astype(np.float64), 1 << 30, 0, d, want)
    torch.cuda.synchronize()
    got = w.double().cpu().numpy()
    # tau itself carries the decode's 2e-5; p <= 1 has slope at most 2
    assert np.abs(got - want).max() < 3 * 4 * (2 * 4e-5 + 1e-4)

    need = -(-keep // ps)
    fresh = torch.arange(c.pages, c.pages + B * need, dtype=torch.int32)
    grow = torch.zeros(B * need, Hkv, ps, D, dtype=k.dtype, device="cuda")
    k, v = torch.cat([k, grow]), torch.cat([v, grow])
    nt = torch.full((B, c.mp), -1, dtype=torch.int32)
    nt[:, :need] = fresh.view(B, need)
    nt = nt.cuda()
    shape1 = E().make_shape(B, H, Hkv, D, ps, c.mp, k.shape[0], "bf16")
    kept = torch.empty(B, Hkv, keep, dtype=torch.int32, device="cuda")
    nl, nw = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty_like(w)
    E().entmaxkv_evict(shape1, k, v, bt, ln, w, keep, 4, 8, nt, kept, nl, nw)
    torch.cuda.synchronize()
    wn, kp = w.cpu().numpy(), kept.cpu().numpy()
    for b, L in enumerate(lens):
        for g in range(Hkv):
            ref = S.evict_kept(wn[b, g], L, keep, 4, 8)
            assert kp[b, g, :len(ref)].tolist() == ref.tolist()
    # the same decodes over a cache that holds the kept rows
    c2 = Cache(52, [min(L, keep) for L in lens], Hkv, D, ps, "bf16", max_pages=c.mp)
    for b, L in enumerate(c2.lens):
        i = np.arange(L)
        for g in range(Hkv):
            src = kp[b, g, :L]
            c2.k[c2.table[b, i // ps], g, i % ps] = c.k[c.table[b, src // ps], g, src % ps]
            c2.v[c2.table[b, i // ps], g, i % ps] = c.v[c.table[b, src // ps], g, src % ps]
    q = c.query(1, H, "f32", 5.0)
    a, la = run_window(c2, q, 20, 4)
    check(c2, q, a, la, *S.window_decode(q.double().numpy(), *c2.np64(), c2.table, c2.lens, 20, 4))
    qd = q.cuda()
    E().entmaxkv_softmax_window(shape1, qd, k, v, nt, nl, 20, 4, out, lse)
    meta = torch.empty(k.shape[0], Hkv, 2, D, dtype=k.dtype, device="cuda")
    E().entmaxkv_build_page_meta(shape1, k, nt, nl, meta)
    sel = torch.empty(B, H, 2, dtype=torch.int32, device="cuda")
    q3 = qd[:, 0].contiguous()
    E().entmaxkv_decode_topk(shape1, q3, meta, k, v, nt, nl, 2, 1.5, sel, o2)
    k2, v2, bt2, ln2 = c2.dev("k", "v", "table", "lens")
    meta2 = torch.empty(c2.pages, Hkv, 2, D, dtype=k.dtype, device="cuda")
    sel2, o3 = torch.empty_like(sel), torch.empty_like(o2)
    E().entmaxkv_build_page_meta(c2.shape(H), k2, bt2, ln2, meta2)
    E().entmaxkv_decode_topk(c2.shape(H), q3, meta2, k2, v2, bt2, ln2, 2, 1.5, sel2, o3)
    torch.cuda.synchronize()
    assert torch.equal(out, a) and torch.equal(lse, la)
    assert torch.equal(sel, sel2) and torch.equal(o2, o3)
