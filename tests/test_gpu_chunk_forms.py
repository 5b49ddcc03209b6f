"""The chunk call where its parts take turns: lists that overflow and are pruned,
rows that go through all of their scores again, parts of long caches, float32
queries looked through by their nearest bf16, large pools; and beside the decode
call. Tolerances as in test_gpu_chunk.py."""
import math

import numpy as np
import pytest
import torch

from parity_util import announce
from test_gpu_chunk import E, Chunk

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def ramp(c, scale, up=True, kinds=((0, 1.0),)):
    """Keys whose scores rise (or fall) with the position, the same direction for
    all rows: every token is above all before it."""
    n = max(c.c.lens)
    t = np.arange(n) if up else np.arange(n)[::-1]
    c.q[:] = 0.0
    c.q[..., 0] = 1.0
    for b, L in enumerate(c.c.lens):
        page = torch.from_numpy(np.asarray(c.c.table)[b][np.arange(L) // c.c.ps].astype(np.int64))
        row = torch.arange(L) % c.c.ps
        c.c.k[page, :, row] = 0.0
        c.c.k[page, :, row, 0] = torch.from_numpy(
            (scale * t[:L, None]).astype(np.float32)).to(c.c.k.dtype)


@pytest.mark.parametrize("kv,q_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("up", [True, False])
@pytest.mark.parametrize("scale", [0.3, 0.01])
def test_rising_and_falling_scores(kv, q_dtype, up, scale):
    """Every token is a hit (rising), or only the first are; supports of a few
    tokens or of hundreds. bf16 keys tie in steps of 2^-8 of themselves."""
    c = Chunk(1, [700], [40], 2, 64, 16, kv, 4, q_dtype)
    ramp(c, scale, up)
    c.check(1.5)


@pytest.mark.parametrize("alpha", [1.25, 1.5])
@pytest.mark.parametrize("spread", [0.3, 1.0])
def test_lists_are_pruned_and_overflow(alpha, spread):
    """Thousands of tokens within the window of a row's maximum: supports about
    and beyond a list's length, in blocks of many rows."""
    Chunk(2, [2500], [24], 1, 64, 32, "bf16", 4, "bf16", spread).check(alpha)
    Chunk(3, [2500], [9], 1, 128, 64, "bf16", 8, "f32", spread).check(alpha)
    Chunk(4, [1500], [20], 1, 64, 16, "f32", 2, "f32", spread).check(alpha)


@pytest.mark.parametrize("kv,q_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("spread", [0.3, 2.5])
def test_single_tokens_over_long_caches(kv, q_dtype, spread):
    """Tokens in many parts, of one row block by several waves."""
    Chunk(5, [9000, 3, 5001], [1, 1, 3], 2, 64, 16, kv, 4, q_dtype, spread).check(1.5)
    Chunk(6, [6000], [1], 1, 128, 64, kv, 8, q_dtype, spread).check(1.25)


def test_prompts_of_several_blocks():
    """More tokens than a block of rows, in parts, beside a single token."""
    for kv, q in (("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")):
        Chunk(7, [300, 77, 130], [300, 1, 129], 1, 64, 16, kv, 4, q).check(1.5)


def test_every_number_of_rows():
    """1 to 300 rows of a KV head: from one row tile by all waves to more than a
    block."""
    for n in (1, 4, 15, 16, 17, 33, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300):
        Chunk(n, [n + 5], [n], 1, 64, 64, "bf16", 1, "bf16").check(1.5)
        Chunk(n, [n + 40], [n], 1, 128, 32, "bf16", 1, "f32").check(2.0)


def test_float32_queries_far_from_bf16_and_large_keys():
    """Queries whose nearest bf16 is as far off as can be, scores of hundreds, and
    keys of very different sizes: the tokens within the rounding's reach are
    taken again exactly."""
    c = Chunk(8, [400], [30], 2, 64, 16, "bf16", 4, "f32")
    c.q = torch.sign(c.q) * (1.0 + 2.0**-8 - 2.0**-20) * 0.5
    c.check(1.5)
    c = Chunk(9, [400], [30], 2, 128, 32, "bf16", 8, "f32", spread=300.0)
    c.check(1.5)
    big = c.c.rng.integers(0, 400, 6)
    for t in big:
        c.c.k[c.c.table[0][t // 32], :, t % 32] *= 64.0
    c.check(1.25)


def test_hidden_values_of_a_block_leave_earlier_rows_alone():
    """What later tokens of the same block hold changes nothing but, with float32
    queries, the last bits (the rounding's reach is taken from the block)."""
    for q in ("bf16", "f32"):
        c = Chunk(10, [90], [40], 1, 64, 16, "bf16", 4, q)
        clean = c.run(1.5)
        for t in (88, 89):
            c.c.k[c.c.table[0][t // 16], :, t % 16] = 1e6
        got = c.run(1.5)
        for a, b in zip(clean, got):
            if q == "bf16":
                assert torch.equal(a[:38], b[:38])
        c.check(1.5, got, rows=set(range(38)))


def test_long_among_short():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(1, 60, 80)]
    new = [int(rng.integers(0, L + 1)) if i % 3 else 1 for i, L in enumerate(lens)]
    lens[40], new[40] = 3000, 20
    Chunk(11, lens, new, 1, 64, 16, "bf16", 2, "bf16").check(1.5)


def test_a_pool_beyond_32_bits():
    """Pages at the end of pools of 5 GB."""
    G, ps, D, pages, L, n = 8, 64, 128, 40000, 150, 20
    k, v = (torch.empty((pages, G, ps, D), dtype=BF, device="cuda") for _ in range(2))
    table = [pages - 1, 7, pages - 2]
    small = torch.randn(3, G, ps, D, generator=torch.Generator().manual_seed(1)).to(BF)
    for x in (k, v):
        x[table] = small.cuda()
    q = (torch.randn(n, 8, D, generator=torch.Generator().manual_seed(2)) * 0.2).to(BF).cuda()
    i32 = lambda x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
    outs = []
    for K, V, bt, P in ((k, v, table, pages), (small.cuda(), small.cuda(), [0, 1, 2], 3)):
        out, tau = torch.empty_like(q), torch.empty((n, 8), device="cuda")
        announce(f"chunk over a pool of {P} pages")
        E().entmaxkv_entmax_chunk(E().make_shape(1, 8, G, D, ps, 3, P, "bf16"), q, i32([0, n]), K, V,
                                  i32([bt]), i32([L]), 1.5, out, tau=tau)
        outs.append((out, tau))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("kv", ["bf16", "f32"])
@pytest.mark.parametrize("alpha", [1.25, 1.5, 2.0])
def test_single_tokens_are_the_full_decode(kv, alpha):
    """One new token a sequence: the full-cache decode call on the same cache,
    both within their own tolerance of the oracle (2e-3 of the output's norm and
    1e-5, as the decode's tests have it)."""
    c = Chunk(12, [700, 33, 1200, 1], [1, 1, 1, 1], 2, 128, 16, kv, 8, "f32")
    got = c.run(alpha)
    k, v, bt, lens = c.c.dev("k", "v", "table", "lens")
    out, tau = torch.empty(4, 8, 128, device="cuda"), torch.empty(4, 8, device="cuda")
    sup = torch.empty(4, 8, dtype=I32, device="cuda")
    shape = E().make_shape(4, 8, 2, 128, 16, c.c.mp, c.c.pages, kv)
    E().entmaxkv_decode_full(shape, c.q.cuda(), k, v, bt, lens, alpha, out, tau, sup)
    torch.cuda.synchronize()
    tol = (2e-3 * out.norm(dim=-1, keepdim=True) if kv == "bf16" else torch.full_like(out, 2e-5))
    assert ((out - got[0]).abs() <= tol).all()
    assert ((tau - got[1]).abs() <= 4e-5 * tau.abs().clamp(min=1)).all()


def test_results_do_not_change_from_run_to_run():
    for q in ("bf16", "f32"):
        c = Chunk(13, [1500, 800], [60, 1], 2, 128, 16, "bf16", 8, q, 1.0)
        first = c.run(1.5)
        for _ in range(3):
            for a, b in zip(first, c.run(1.5)):
                assert torch.equal(a, b)


def test_workspace_of_another_content():
    """The workspace holds nothing that a call needs from before."""
    c = Chunk(14, [500, 1], [40, 1], 2, 64, 16, "bf16", 8, "f32")
    n = E().entmaxkv_entmax_chunk_ws(c.c.shape(8), c.N, 1.5)
    for fill in (0, 255, 127):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        got = c.run(1.5, ws=ws)
        c.check(1.5, got)
