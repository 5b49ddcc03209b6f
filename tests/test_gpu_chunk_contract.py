"""Calls of the chunk that its documentation allows: the output over the queries, a
prompt in slices, and the rows of a sequence that the plan refused."""
import numpy as np
import pytest
import torch

from parity_util import announce
from test_gpu_chunk import Chunk, E
from test_gpu_tokens_run import Server, i32

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


@pytest.mark.parametrize("kv,q_dtype", TYPES)
@pytest.mark.parametrize("spread", [0.05, 2.5])
@pytest.mark.parametrize("lens,new,Hkv", [([500, 40], [1, 3], 2), ([500, 40], [60, 1], 2),
                                          ([400], [400], 8)])
def test_output_over_the_queries(kv, q_dtype, spread, lens, new, Hkv):
    """Short supports and long ones, few blocks (two kernels) and many (three)."""
    c = Chunk(80, lens, new, Hkv, 64, 16, kv, 8 * Hkv, q_dtype, spread)
    want = c.run(1.5)
    q = c.q.cuda()
    k, v, table, cl = c.c.dev("k", "v", "table", "lens")
    tau = torch.empty(q.shape[:2], device="cuda")
    announce("chunk over its queries")
    E().entmaxkv_entmax_chunk(c.c.shape(c.H), q, i32(c.starts.tolist()), k, v, table, cl, 1.5, q,
                              tau=tau)
    torch.cuda.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(tau, want[1])


@pytest.mark.parametrize("kv,q_dtype", TYPES)
@pytest.mark.parametrize("step", [1, 70, 128])
def test_a_prompt_in_slices(kv, q_dtype, step):
    """Each slice with the sequence's length up to its last token; the later tokens'
    keys and values may be in the cache already."""
    L = 200 if step > 1 else 20
    c = Chunk(81, [L], [L], 2, 64, 16, kv, 8, q_dtype)
    k, v, table = c.c.dev("k", "v", "table")
    q = c.q.cuda()
    out, tau = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    sup = torch.full(q.shape[:2], 7, dtype=torch.int32, device="cuda")
    for a in range(0, L, step):
        b = min(a + step, L)
        announce(f"slice {a}..{b} of {L}")
        E().entmaxkv_entmax_chunk(c.c.shape(8), q[a:b], i32([0, b - a]), k, v, table, i32([b]), 1.5,
                                  out[a:b], tau=tau[a:b], support=sup[a:b])
    torch.cuda.synchronize()
    c.check(1.5, (out, tau, sup))


def test_rows_of_a_refused_sequence_with_tokens():
    """They take part as the last tokens of the sequence as it was; nothing of the
    cache, the table or the other sequences changes with them."""
    s = Server(pages=6)
    s.feed([20, 33, 5], 1)  # 2 + 3 + 1 pages: all of them
    s.step()
    s.check()
    s.advance()
    table, k, v = s.table.clone(), s.k.clone(), s.v.clone()
    s.feed([3, 40, 2], 2)  # the second needs two pages more
    s.step()
    torch.cuda.synchronize()
    lens = s.check()  # all rows, the refused ones against the 33 tokens that are there
    assert lens == [23, 33, 7] and s.starts.tolist() == [0, 3, 43, 45]
    assert (s.slots[3:43] == -1).all() and (s.pos[3:43] == torch.arange(33, 73, device="cuda")).all()
    assert (s.out[3:10] == 0).all() and s.tau[3:10].isnan().all()  # 40 rows, 33 tokens
    assert torch.equal(s.table, table)
    pages = table[1, :3].long()
    assert torch.equal(torch.nan_to_num(s.k[pages].float()), torch.nan_to_num(k[pages].float()))
    assert torch.equal(torch.nan_to_num(s.v[pages].float()), torch.nan_to_num(v[pages].float()))
