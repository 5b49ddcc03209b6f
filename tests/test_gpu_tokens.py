"""The plan of a step's pages and slots, and the norm, rotation and append of
its tokens, on the GPU against the float64 oracle.

Tolerances of the append. Without a norm a value takes three roundings in
float32 (two products and a sum of a rotation, then the scale of a query), the
sine and cosine beside them are within 4 x 2^-24, all relative to |a| + |b| of
the pair at most: 8 x 2^-24 (|a| + |b|). A norm adds the sum of squares (16
values a lane and 3 steps between lanes, 19 roundings, halved by the root: 10),
the reciprocal root (2), eps (1) and three products: 16 more, 24 in all. A
result is then rounded once to its type: half a step, eps / 2 of the value.
"""
import math

import numpy as np
import pytest
import torch

from oracle import tokens_oracle as T
from parity_util import announce

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def E():
    from sparse_long_context_page_amd import entmaxkv
    return entmaxkv


def dev(x):
    return torch.tensor(np.ascontiguousarray(x), dtype=I32).cuda()


# ---------------------------------------------------------------------------
# plan


def run_plan(lens, new, free, table, ps, pages, rows, capacity=None, **kw):
    """The call on fresh tensors, compared whole with the oracle."""
    B, mp = np.shape(table)
    announce(f"plan B={B} ps={ps} rows={rows} new={sum(new)} free={len(free)}")
    shape = E().make_shape(B, 1, 1, 64, ps, mp, pages, "bf16")
    bt = dev(table)
    stack = dev(list(free) + [77] * (0 if capacity is None else capacity - len(free)))
    o = {"new_lens": dev([9] * B), "token_starts": dev([9] * (B + 1)), "positions": dev([9] * rows),
         "slots": dev([9] * rows), "free_left": dev([9])}
    args = dict(seq_lens=dev(lens), new_tokens=dev(new),
                free_pages=stack if stack.numel() else None, free_count=dev([len(free)]),
                block_table=bt, **o)
    E().entmaxkv_plan_tokens(shape, **args, **kw)
    torch.cuda.synchronize()
    ref = T.plan(lens, new, free, table, ps, pages, rows)
    for k, v in {**o, "block_table": bt}.items():
        assert np.array_equal(v.cpu().numpy().ravel(), ref[k].ravel()), k
    return shape, args, ref


def batch(seed, B, ps, mp, most, empty=0.3):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, mp * ps // 2 + 1, B)
    new = np.where(rng.random(B) < empty, 0, rng.integers(1, most + 1, B))
    order = rng.permutation(3 * B * mp)
    held = -(-lens // ps)
    table = np.where(np.arange(mp) < held[:, None], order[:B * mp].reshape(B, mp), -1)
    return lens.tolist(), new.tolist(), order[B * mp:].tolist(), table, 3 * B * mp


@pytest.mark.parametrize("B,ps,mp,most", [
    (1, 16, 3, 20), (3, 16, 8, 40), (64, 16, 40, 1), (257, 32, 9, 70), (1023, 64, 4, 30),
    (1024, 16, 5, 3), (1025, 16, 5, 33), (3000, 16, 4, 9), (40, 64, 300, 9000)])
def test_plan(B, ps, mp, most):
    lens, new, free, table, pages = batch(B, B, ps, mp, most)
    rows = max(1, sum(new))
    run_plan(lens, new, free, table, ps, pages, rows + 5)
    run_plan(lens, new, free, table, ps, pages, rows)
    # too few pages, none, and too few rows
    run_plan(lens, new, free[:sum(new) // (3 * ps) + 1], table, ps, pages, rows, capacity=len(free))
    run_plan(lens, new, [], table, ps, pages, rows)
    run_plan(lens, new, free, table, ps, pages, max(1, rows // 2))


def test_plan_one_long_prompt_among_empty_sequences():
    # 70000 rows of one sequence over many workgroups, 2999 sequences of none
    lens, new = [0] * 3000, [0] * 3000
    lens[1500], new[1500] = 100, 70001
    table = np.full((3000, 1100), -1)
    table[1500, :2] = [5, 6]
    run_plan(lens, new, list(range(10, 1200)), table, 64, 2000, 70100)


def test_plan_every_row_its_own_sequence():
    n = 5000
    table = np.arange(2 * n).reshape(n, 2)
    run_plan([i % 30 for i in range(n)], [1] * n, list(range(2 * n, 3 * n)), table, 16, 3 * n, n)


def test_plan_bad_values():
    """Lengths outside the table, negative counts, pages outside the pool, more
    free pages said than there are: clamped, refused or without a slot."""
    table = np.array([[0, 1, 2]] * 5)
    table[4, 0] = 999
    lens, new = [-5, 100, 48, 7, 3], [3, 2, 0, -9, 4]
    shape, args, _ = run_plan(lens, new, [-3, 50, 8], table, 16, 40, 12)
    args["free_count"].fill_(2**31 - 1)
    E().entmaxkv_plan_tokens(shape, **args)
    assert int(args["free_left"]) == 3 - 1
    args["free_count"].fill_(-4)
    E().entmaxkv_plan_tokens(shape, **args)
    assert int(args["free_left"]) == 0
    args["new_tokens"].fill_(2**31 - 1)
    E().entmaxkv_plan_tokens(shape, **args)
    assert (args["slots"] == -1).all() and args["token_starts"].tolist() == [0, 12, 12, 12, 12, 12]
    assert args["new_lens"].tolist() == [0, 48, 48, 7, 3]


# ---------------------------------------------------------------------------
# append


class Tokens:
    """Rows of one projection: padding between tokens, junk in it."""

    def __init__(self, seed, n, H, G, D, x, ps=16, pages=None, pad=0):
        rng = np.random.default_rng(seed)
        self.rng, self.n, self.H, self.G, self.D, self.ps = rng, n, H, G, D, ps
        w = (H + 2 * G) * D + pad
        buf = torch.from_numpy(rng.normal(size=(n, w)).astype(np.float32) * 1.7).to(x)
        buf[:, (H + 2 * G) * D:] = math.nan
        self.buf = buf.cuda()
        self.pages = pages or -(-n // ps) + 2
        self.slots = rng.permutation(self.pages * ps)[:n].astype(np.int32)

    def parts(self, buf=None):
        H, G, D, n = self.H, self.G, self.D, self.n
        b = self.buf if buf is None else buf
        cut = (0, H * D, (H + G) * D, (H + 2 * G) * D)
        return [b[:, i:j].view(n, -1, D) for i, j in zip(cut, cut[1:])]


def run_append(c, q_dtype, kv, rot, axes=1, interleaved=False, normed=True, eps=1e-6,
               context=5000, scale=0.3, slots=None, **kw):
    D, n = c.D, c.n
    announce(f"append n={n} heads={c.H}/{c.G} D={D} x={c.buf.dtype} q={q_dtype} kv={kv} rot={rot} "
             f"axes={axes} interleaved={interleaved} norm={normed}")
    rng = c.rng
    q, k, v = c.parts()
    slots = c.slots if slots is None else slots
    pos = rng.integers(0, context, (axes, n))
    freqs = 10000.0 ** -(np.arange(rot // 2) / max(1, rot // 2))
    axis = rng.integers(0, axes, rot // 2) if axes > 1 else None
    qw, kw_ = (rng.normal(size=D).astype(np.float32) if normed else None for _ in range(2))
    kv_t = BF if kv == "bf16" else F32
    k_pool, v_pool = (torch.full((c.pages, c.G, c.ps, D), 7.5, dtype=kv_t).cuda()
                      for _ in range(2))
    q_out = torch.full((n, c.H, D), 7.5, dtype=q_dtype).cuda()
    shape = E().make_shape(1, c.H, c.G, D, c.ps, 1, c.pages, kv)
    w = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
    E().entmaxkv_append_kv(shape, q, k, v, dev(pos), dev(slots), q_out, k_pool, v_pool,
                           freqs=torch.from_numpy(freqs).cuda() if rot else None,
                           pair_axis=None if axis is None else dev(axis), interleaved=interleaved,
                           q_weight=w(qw), k_weight=w(kw_), eps=eps, q_scale=scale, **kw)
    torch.cuda.synchronize()

    def check(got, x, weight, turned, pos, by=1.0):
        f = 1.0
        y = T.norm(x.double().cpu().numpy(), weight, eps)
        ref, mag = y, np.abs(y)
        if turned:
            ref = T.rotate(y, pos, freqs, axis, interleaved)
            # |a| + |b| of every pair: the rotation by 0 of swapped magnitudes
            h = rot // 2
            a, b = ((slice(0, rot, 2), slice(1, rot, 2)) if interleaved
                    else (slice(0, h), slice(h, rot)))
            mag[..., a] = mag[..., b] = mag[..., a] + mag[..., b]
            f = 8.0 if weight is None else 24.0
        elif weight is not None:
            f = 24.0
        tol = (f * 2.0**-24 * mag + torch.finfo(got.dtype).eps / 2 * np.abs(ref)) * by * 1.0001
        err = np.abs(got.double().cpu().numpy() - by * ref)
        assert np.isfinite(err).all() and (err <= tol).all(), float((err / tol.clip(1e-30)).max())

    check(q_out, q, qw, bool(rot), pos, scale)
    live = (slots >= 0) & (slots < c.pages * c.ps)
    at = torch.from_numpy(slots[live].astype(np.int64))
    li = torch.from_numpy(np.flatnonzero(live)).cuda()
    left = torch.ones(c.pages * c.ps, dtype=torch.bool)
    left[at] = False
    for pool, x, weight, turned in ((k_pool, k, kw_, bool(rot)), (v_pool, v, None, False)):
        rows = pool.transpose(1, 2).reshape(-1, c.G, D)
        assert (rows[left.cuda()] == 7.5).all()
        if weight is None and not turned:  # a copy, rounded once or not at all
            assert torch.equal(rows[at.cuda()], x[li].to(kv_t))
        else:
            check(rows[at.cuda()], x[li], weight, turned, pos[:, live])
    return q_out, k_pool, v_pool


@pytest.mark.parametrize("x", [BF, F32])
@pytest.mark.parametrize("q_dtype", [BF, F32])
@pytest.mark.parametrize("kv", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_append_types(x, q_dtype, kv, D):
    run_append(Tokens(1, 13, 8, 2, D, x), q_dtype, kv, D)
    run_append(Tokens(2, 3, 2, 2, D, x, pad=8), q_dtype, kv, 0, normed=False)


@pytest.mark.parametrize("rot", [0, 16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_part_of_a_head_turns(rot, interleaved):
    run_append(Tokens(rot, 5, 4, 1, 128, BF), F32, "bf16", rot, interleaved=interleaved)
    if rot <= 64:
        run_append(Tokens(rot, 5, 4, 1, 64, F32), F32, "f32", rot, interleaved=interleaved,
                   normed=False)


@pytest.mark.parametrize("axes", [1, 2, 3, 8])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_axes(axes, interleaved):
    run_append(Tokens(axes, 21, 8, 8, 128, F32), F32, "f32", 128, axes=axes,
               interleaved=interleaved)


@pytest.mark.parametrize("n,H,G", [(1, 1, 1), (1, 32, 8), (2, 8, 1), (4, 3, 3), (5, 64, 8),
                                   (67, 16, 16), (131, 4, 2)])
def test_append_counts(n, H, G):
    run_append(Tokens(n, n, H, G, 128, BF, ps=32), BF, "bf16", 128)
    run_append(Tokens(n, n, H, G, 64, BF, ps=64), F32, "bf16", 64, normed=False)


def test_append_far_positions():
    """Angles of millions of radians: float32 would be off by tenths."""
    run_append(Tokens(9, 40, 4, 2, 128, F32), F32, "f32", 128, context=2**31 - 1, normed=False)


def test_append_padding_and_bad_slots_write_nothing():
    c = Tokens(5, 50, 4, 2, 64, BF)
    s = c.slots.copy()
    s[::3] = -1
    s[1], s[4], s[7] = c.pages * c.ps, 2**31 - 1, -2**31
    run_append(c, F32, "bf16", 64, slots=s)
    run_append(c, F32, "bf16", 64, slots=np.full(50, -1, np.int32))


def test_append_eps_alone_and_zero_rows():
    c = Tokens(6, 7, 2, 2, 64, F32)
    c.buf[2] = 0.0
    run_append(c, F32, "f32", 64, eps=0.25)


def test_append_keeps_nan_and_infinities_in_their_rows():
    c = Tokens(7, 6, 2, 2, 64, BF)
    q, k, v = c.parts()
    q[1, 0, 5], k[2, 1, 3], v[3, 0, 1] = math.nan, math.inf, math.nan
    pos = dev(np.arange(6))
    pools = [torch.zeros((c.pages, 2, 16, 64), dtype=BF).cuda() for _ in range(2)]
    q_out = torch.zeros((6, 2, 64)).cuda()
    E().entmaxkv_append_kv(E().make_shape(1, 2, 2, 64, 16, 1, c.pages, "bf16"), q, k, v, pos,
                           dev(c.slots), q_out, *pools, q_weight=torch.ones(64).cuda(),
                           k_weight=torch.ones(64).cuda(),
                           freqs=torch.ones(32, dtype=torch.float64).cuda())
    rows = [p.transpose(1, 2).reshape(-1, 2, 64)[torch.from_numpy(c.slots).long().cuda()]
            for p in pools]
    assert q_out[1, 0].isnan().all() and q_out[1, 1].isfinite().all() and q_out[0].isfinite().all()
    bad = ~rows[0].isfinite().all(-1)
    assert bad.nonzero().tolist() == [[2, 1]]
    assert rows[1].isnan().nonzero().tolist() == [[3, 0, 1]]


def test_append_into_a_pool_beyond_32_bits():
    c = Tokens(8, 9, 8, 8, 128, BF, ps=64, pages=40000)  # 5.2 GB a pool
    s = c.slots.copy()
    s[0], s[1] = c.pages * 64 - 1, c.pages * 64 - 65
    D, n = c.D, c.n
    q, k, v = c.parts()
    pools = [torch.empty((c.pages, 8, 64, D), dtype=BF, device="cuda") for _ in range(2)]
    q_out = torch.empty((n, 8, D), dtype=BF, device="cuda")
    E().entmaxkv_append_kv(E().make_shape(1, 8, 8, D, 64, 1, c.pages, "bf16"), q, k, v, None,
                           dev(s), q_out, *pools)
    at = torch.from_numpy(s.astype(np.int64)).cuda()
    for p, x in zip(pools, (k, v)):
        assert torch.equal(p[at // 64, :, at % 64], x)
    assert torch.equal(q_out, q)
