"""A row whose support is too long for a list shares its tile with rows whose
supports are short: those keep the result of their lists."""
import numpy as np
import pytest
import torch

from test_gpu_chunk import Chunk

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


@pytest.mark.parametrize("kv,q_dtype", TYPES)
@pytest.mark.parametrize("lens,new,Hkv", [([600], [1], 1), ([600], [40], 1), ([1100], [1060], 1),
                                          ([1100], [1060], 2)])
def test_short_supports_beside_long_ones(kv, q_dtype, lens, new, Hkv):
    """Heads of even number look at coordinate 0: three tokens of weight, all others
    far below and falling. Odd heads look at coordinate 1: the same score for
    every token, or what coordinate 0 holds, as the keys are made. What the odd
    heads see is nothing to the even ones, down to the last bit (their lists hold
    the same three tokens either way). Values nearly cancel, so that roundings
    of the weights show in the output."""
    L, n, D, G = lens[0], new[0], 64, 8
    c = Chunk(40, lens, new, Hkv, D, 16, kv, G * Hkv, q_dtype)
    c.q[:] = 0.0
    c.q[:, 0::2, 0] = 1.0
    c.q[:, 1::2, 1] = 1.0
    t = np.arange(L)
    page = torch.from_numpy(np.asarray(c.c.table)[0][t // 16].astype(np.int64))
    z = -20.0 - 10.0 * t
    z[10:13] = 4.0, 3.5, 3.25
    c.c.k[page, :, t % 16] = 0.0
    c.c.k[page, :, t % 16, 0] = torch.from_numpy(z)[:, None].to(c.c.k.dtype)
    v = torch.randn(L, 1, D, generator=torch.Generator().manual_seed(1))
    v[11], v[12] = -0.58406 / 0.26446 * v[10], 0.01 * v[12]  # (the weights at alpha 1.5)
    c.c.v[page, :, t % 16] = v.to(c.c.v.dtype)
    flat = c.run(1.5)
    c.c.k[page, :, t % 16, 1] = c.c.k[page, :, t % 16, 0]
    peaked = c.run(1.5)
    assert (flat[2][:, 0::2] <= 3).all()
    assert (peaked[2] <= 3).all() and int(flat[2][n - 1, 1]) == L
    for a, b in zip(flat, peaked):
        assert torch.equal(a[:, 0::2], b[:, 0::2])
    c.c.k[page, :, t % 16, 1] = 0.0
    c.check(1.5, flat, rows={0, n // 2, n - 1})
