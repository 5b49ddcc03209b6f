"""The chunk call at the ends of its ranges: so many blocks of rows that the rows
with long supports are a kernel of their own (with few they are not), and alpha
close to 1 and far beyond 2. Tolerances as in test_gpu_chunk.py, which hold for
any alpha: sum u^(m-1) >= 1 for m < 1 as well, as every u <= 1."""
import numpy as np
import pytest
import torch

from test_gpu_chunk import Chunk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv,q_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_long_supports_in_many_blocks(kv, q_dtype):
    """A support takes up to 400 tokens where scores are flat; a sequence of
    peaked scores in between keeps its lists."""
    c = Chunk(1, [400, 30, 500], [390, 30, 500], 2, 64, 16, kv, 16, q_dtype, 0.05)
    c.q[390:420] *= 60.0
    rows = set(range(0, c.N, 7)) | {389, 390, 419, 420, c.N - 1}
    c.check(1.5, rows=rows)


def test_values_that_are_no_numbers_in_many_blocks():
    """NaN and infinities among the values of tokens that every row sees, of no
    weight for most of them."""
    c = Chunk(2, [600], [560], 2, 64, 16, "bf16", 16, "bf16", 0.4)
    t = 7
    page, row = int(np.asarray(c.c.table)[0][t // 16]), t % 16
    c.c.k[page, :, row] = 0.0
    clean = c.run(1.5)
    c.c.v[page, :, row, 3] = float("nan")
    c.c.v[page, :, row, 9] = float("inf")
    c.c.k[page, :, row] = -2.0 * torch.sign(c.q[300, 0].float()).to(c.c.k.dtype)
    got = c.run(1.5)
    k, v = c.c.np64()
    toks = np.asarray(c.c.table)[0][np.arange(600) // 16], np.arange(600) % 16
    q = c.q.double().numpy()
    for r in range(0, 560, 23):
        hi = 40 + r + 1
        for h in range(16):
            z = k[toks[0][:hi], h // 8, toks[1][:hi]] @ q[r, h]
            tau = float(got[1][r, h])
            u = 0.5 * z[t] - tau
            bad = ~torch.isfinite(got[0][r, h].float()).cpu()
            if u < -1e-3:
                assert not bad.any()
            elif u > 1e-3:
                assert bad[3] and bad[9] and int(bad.sum()) == 2
    assert torch.isfinite(clean[0].float()).all()


@pytest.mark.parametrize("alpha", [1.003, 1.01, 12.0, 100.0])
@pytest.mark.parametrize("spread", [0.05, 2.5, 30.0])
def test_alpha_at_its_ends(alpha, spread):
    Chunk(3, [200, 33], [9, 1], 2, 64, 32, "bf16", 4, "bf16", spread).check(alpha)
    Chunk(4, [150, 3], [2, 3], 1, 64, 16, "f32", 2, "f32", spread).check(alpha)
