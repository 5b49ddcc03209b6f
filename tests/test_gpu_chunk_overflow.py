"""A seen score of +inf makes its row's out and tau NaN wherever among the tokens
it lies, in blocks of many rows as of few, and no other row's."""
import numpy as np
import pytest
import torch

from test_gpu_chunk import Chunk

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


@pytest.mark.parametrize("kv,q_dtype", TYPES)
@pytest.mark.parametrize("new", [40, 1])
@pytest.mark.parametrize("at", [0, 3, 70, 127, 128, 290])
def test_one_score_overflows(kv, q_dtype, new, at):
    c = Chunk(20, [340], [new], 2, 64, 16, kv, 8, q_dtype)
    c.q[..., 0] = 0.0
    c.c.k[..., 0][torch.isfinite(c.c.k[..., 0])] = 0.0
    c.c.k[int(c.c.table[0][at // 16]), :, at % 16, 0] = 8.0
    clean = c.run(1.5)
    plain = c.q.clone()
    rows = [(0, 6)] if new == 1 else [(5, 1), (9, 6)]
    for r, h in rows:
        c.q[r, h, 0] = 1e38  # 8e38 at that token, 0 from this coordinate elsewhere
    got = c.run(1.5)
    for r, h in rows:
        assert got[0][r, h].isnan().all() and got[1][r, h].isnan(), (r, h)
        for x, y in zip(got, clean):
            x[r, h] = y[r, h]
    c.q = plain
    c.check(1.5, got)  # the others are what they were
