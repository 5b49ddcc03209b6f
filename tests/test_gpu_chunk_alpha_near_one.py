"""The chunk call with alpha close to 1, where all seen tokens have weights that are
nearly those of a softmax, and u = x - tau nearly 1: u^m of a rounded u would be
off by m 2^-24 of itself.

The scores here are exact (sums of four keys of few bits). Tolerances: with d = z -
max z, a weight relative to the largest is (1 + (alpha - 1) d / s)^m, s = max x -
tau: here nearly e^d. In units of 2^-24 of d, alpha - 1, its product, the
reciprocal and the product with it are off by 5, s by 4, the logarithm with its
correction by 6, m and its product by 2, the exponential's argument by 1: 18 |d|,
and the exponential by 2 of itself. An output moves by twice the weights' mean
change times max |v - out|; its sums add (T / 16 + 16) 2^-24 of max |v|, a bf16
result half a step and its weights' 2^-16. s is off by its own rounding and the
rounding of u (2^-24 each) and by those of the step from a sum near 1 (2^-22).
"""
import numpy as np
import pytest
import torch

from oracle import tokens_oracle as T
from test_gpu_chunk import BF, Chunk

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


@pytest.mark.parametrize("kv,q_dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("alpha", [1.01, 1.001, 1.0003, 1.00001, 1.0 + 2.0**-22])
@pytest.mark.parametrize("lens,new", [([60, 7], [1, 3]), ([60, 33], [40, 1]), ([700, 130], [1, 40])])
def test_weights_of_nearly_a_softmax(kv, q_dtype, D, alpha, lens, new):
    """Few tokens (from the lists) and many (from all scores), a few rows of them and
    blocks of many."""
    c = Chunk(70, lens, new, 2, D, 16, kv, 8, q_dtype)
    c.q[..., 4:] = 0.0
    c.q[..., :4] = torch.sign(c.q[..., :4])
    c.c.k = (torch.round(c.c.k.float() * 8) / 8).to(c.c.k.dtype)
    alpha = float(np.float32(alpha))
    out, tau, sup = (x.double().cpu().numpy() for x in c.run(alpha))
    k, v = c.c.np64()
    scores = {}
    ref, rtau, rsup = T.chunk(c.q.double().numpy(), c.starts, k, v, np.asarray(c.c.table), c.c.lens,
                              alpha, lambda r, h, z: scores.__setitem__((r, h), z))
    vmax = np.where(np.isfinite(v), np.abs(v), 0.0).max()
    assert (sup == rsup).all()
    for (r, h), z in scores.items():
        p = np.maximum((alpha - 1.0) * z - rtau[r, h], 0.0) ** (1.0 / (alpha - 1.0))
        change = float((p * (18 * (z.max() - z) + 2)).sum() / p.sum()) * 2.0**-24
        tol = 2 * change * (vmax + np.abs(ref[r, h])) + (len(z) / 16 + 16) * 2.0**-24 * vmax
        if c.q.dtype == BF:
            tol = tol + 2.0**-8 * np.abs(ref[r, h]) + 2.0**-16 * vmax
        err = np.abs(out[r, h] - ref[r, h])
        assert (err <= tol).all(), (r, h, float((err / tol).max()))
        assert abs(tau[r, h] - rtau[r, h]) <= 2.0**-22 + 2.0**-23, (r, h, tau[r, h], rtau[r, h])
