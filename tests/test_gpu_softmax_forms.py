"""Softmax decode on the GPU: what must not depend on which form of the
attention kernel a call runs (few rows: 16 rows a workgroup; many rows: row
tiles of their own for every wave)."""
import numpy as np
import pytest
import torch

from oracle import softmax_oracle as S
from parity_util import announce
from test_gpu_softmax import Cache, empties, run_window

pytestmark = pytest.mark.gpu

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
    for empty in [0] + ([empties(c, q, 4200)] if n * G >= 33 else []):
        announce(f"bf16 queries' weights n{n} L{L} D{D}, {empty} empty sequences")
        out, lse = run_window(c, q, 1 << 30, 0, empty)
        over = np.abs(out.double().cpu().numpy() - ref) - 2.0**-8 - off
        assert over.max() <= 0, (float(over.max()), int((over > 0).sum()))
        # 2^-21 of the weights, 18 roundings of l, 8 of 2^-23 of the logarithm and 4 + 4 after it
        assert np.abs(lse.double().cpu().numpy() - ref_lse).max() <= 2.0**-21 + 42 * 2.0**-24
