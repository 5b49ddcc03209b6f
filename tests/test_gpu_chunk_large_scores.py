"""Scores so large, or alpha so far above 2, that 1 / (alpha - 1) is lost beside
the largest score: the row's largest token keeps its weight, and those next to it
theirs.

All scores here are exact in float32 (products of one or two coordinates of few
bits), so that the weights follow from their exact differences. A row with one
token in its support returns that token's value, times p / p: two roundings,
2^-23, and half a step of bf16. tau = (alpha - 1) max - 1 by one product and one
sum, its threshold within 2^-22 of -1.
"""
import numpy as np
import pytest
import torch

from oracle import entmax_oracle as O
from test_gpu_chunk import Chunk

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


def one_coordinate(seed, new, kv, q_dtype, scale, sign):
    """Scores scale * sign * (129 .. 255), all different."""
    L = 110
    c = Chunk(seed, [L], [new], 2, 64, 16, kv, 8, q_dtype)
    c.q[:] = 0.0
    c.q[..., 0] = sign
    z = scale * sign * (129.0 + c.c.rng.permutation(127)[:L])
    t = np.arange(L)
    page = torch.from_numpy(np.asarray(c.c.table)[0][t // 16].astype(np.int64))
    c.c.k[page, :, t % 16] = 0.0
    c.c.k[page, :, t % 16, 0] = torch.from_numpy(sign * z)[:, None].to(c.c.k.dtype)
    return c, z


@pytest.mark.parametrize("kv,q_dtype", TYPES)
@pytest.mark.parametrize("new", [40, 1])
@pytest.mark.parametrize("scale,alpha", [(2.0**19, 1.5), (2.0**19, 2.0), (2.0**19, 1.25),
                                         (2.0**30, 1.5), (16.0, 1e4), (0.25, 1e6), (0.25, 1e30)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_the_largest_token_is_the_support(kv, q_dtype, new, scale, alpha, sign):
    """Scores about 1e8 and -1e8, and of tens and thousands with alpha beyond what
    float32 resolves there."""
    c, z = one_coordinate(30, new, kv, q_dtype, scale, sign)
    out, tau, sup = (x.double().cpu().numpy() for x in c.run(alpha))
    v = c.c.np64()[1]
    half = 2.0**-9 * 2 if q_dtype == "bf16" else 0.0
    for r in range(new):
        seen = z[:110 - new + r + 1]
        j = int(seen.argmax())
        ref = v[int(c.c.table[0][j // 16]), :, j % 16].repeat(4, 0)  # [8, 64]
        assert (np.abs(out[r] - ref) <= (2.0**-22 + half) * np.abs(ref)).all(), r
        assert (sup[r] == 1).all(), r
        am1 = float(np.float32(alpha - 1.0))
        if am1 * abs(seen[j]) < 3e38:
            want = am1 * seen[j] - 1.0
            assert (np.abs(tau[r] - want) <= 2.0**-22 * (abs(want) + 1.0)).all(), r


@pytest.mark.parametrize("kv,q_dtype", TYPES)
@pytest.mark.parametrize("new", [40, 1])
@pytest.mark.parametrize("alpha,gap", [(1.9, 1.0), (1.4, 2.0), (1.6, 1.0)])
def test_tokens_near_the_largest_keep_their_weights(kv, q_dtype, new, alpha, gap):
    """Two tokens of scores about 2^23, a whole number apart and less than 1 /
    (alpha - 1), over tokens of score 0. u is exact but for (alpha - 1) * gap and
    the threshold (2^-22 of 1 each), a power's relative error 2^-20 at most here:
    2^-18 of the largest value covers the weights' change on both tokens."""
    L = 90
    c = Chunk(31, [L], [new], 2, 64, 16, kv, 8, q_dtype)
    c.q[:] = 0.0
    c.q[..., :2] = 1.0
    t = np.arange(L)
    page = torch.from_numpy(np.asarray(c.c.table)[0][t // 16].astype(np.int64))
    c.c.k[page, :, t % 16] = 0.0
    top = [7, 33]
    for x, small in zip(top, (8.0, 8.0 - gap)):
        at = int(c.c.table[0][x // 16])
        c.c.k[at, :, x % 16, 0], c.c.k[at, :, x % 16, 1] = 2.0**23, small
    out, _, sup = (x.double().cpu().numpy() for x in c.run(alpha))
    x = (alpha - 1.0) * np.array([0.0, -gap])
    p = O.entmax_probs(x, O.entmax_threshold(x, alpha), alpha)
    assert p[1] > 0.01
    v = c.c.np64()[1]
    rows = np.stack([v[int(c.c.table[0][j // 16]), :, j % 16] for j in top])  # [2, 2, 64]
    ref = np.einsum("t,tgd->gd", p / p.sum(), rows).repeat(4, 0)
    tol = 2.0**-18 * np.abs(rows).max() + (2.0**-8 * np.abs(ref) if q_dtype == "bf16" else 0.0)
    if q_dtype == "bf16":
        tol = tol + 2.0**-16 * np.abs(rows).max()
    assert (sup == 2).all()
    assert (np.abs(out - ref) <= tol).all()
