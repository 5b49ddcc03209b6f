"""Attention weights and eviction on the GPU: heads that saw nothing, and rows
beyond what the eviction keeps in registers."""
import numpy as np
import pytest
import torch

from oracle import softmax_oracle as S
from parity_util import announce
from test_gpu_evict import check_evict, run_weights, weight_tolerance
from test_gpu_softmax import Cache, E, run_window

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "f32"])
def test_weights_of_heads_that_saw_nothing(kv):
    """A softmax decode whose visible scores are all -inf gives lse = -inf, a
    sparse decode of no page tau = NaN: such a head gave no token a weight and
    adds nothing, whatever the other heads of its KV head saw."""
    L, H = 70, 4
    c = Cache(36, (L, 5), 1, 64, 16, kv)
    q = c.query(1, H, "f32")
    t = np.arange(L)
    c.k[c.table[0, t // 16], 0, t % 16, 0] = -1e30
    q[0, 0, :2, 0], q[0, 0, 2:, 0] = 1e30, 0.0  # heads 0 and 1: every product overflows
    k, v, bt, ln = c.dev("k", "v", "table", "lens")
    announce(f"weights of heads that saw nothing {kv}")
    out, lse = run_window(c, q, 1000, 0)
    assert torch.isneginf(lse[0, 0, :2]).all() and torch.isfinite(lse[0, 0, 2:]).all()
    assert (out[0, 0, :2] == 0).all()
    tau = lse[:, 0].contiguous().cpu().numpy()
    got = run_weights(c, q, 1.0, tau, None, 1.0)
    rest = S.weights(q[:, 0].double().numpy(), c.np64()[0], c.table, c.lens, 1.0,
                     tau.astype(np.float64), 1 << 30, 0, 1.0, np.zeros(got.shape))
    # the other heads' scores lack the first coordinate
    c.k[c.table[0, t // 16], 0, t % 16, 0] = q[0, 0, :, 0] = 0.0
    tol = weight_tolerance(c, q, 1.0, rest, np.zeros(got.shape), 1.0)
    for b, n in enumerate(c.lens):
        assert (np.abs(got[b, :, :n] - rest[b, :, :n]) <= tol[b, :, :n]).all(), b

    sel = torch.full((2, H, 2), -1, dtype=torch.int32, device="cuda")
    sel[1] = torch.tensor([0, 1], device="cuda")
    q3 = c.query(1, H, "f32")[:, 0].contiguous()
    o, tau = torch.empty(2, H, 64, device="cuda"), torch.empty(2, H, device="cuda")
    E().entmaxkv_decode_sparse(c.shape(H), q3.cuda(), k, v, bt, ln, sel, 2, 1.5, o, tau=tau)
    torch.cuda.synchronize()
    assert torch.isnan(tau[0]).all() and torch.isfinite(tau[1]).all()
    got = run_weights(c, q3[:, None], 1.5, tau.cpu().numpy(), None, 1.0)
    assert (got[0, :, :L] == 0).all() and np.isfinite(got[1, :, :5]).all()
    assert got[1, 0, :5].sum() > H - 1e-3


# ---------------------------------------------------------------------------
# rows whose keys do not fit the registers (over 32768 competing tokens)


def many_kinds(rng, kind, shape):
    """Weights in which the boundary falls among equals, or among values that
    need care."""
    n = shape[-1]
    w = rng.integers(0, 3, size=shape).astype(np.float32)
    if kind == "zero":
        w[:] = 0.0
        w[..., ::2] = -0.0
    elif kind == "special":
        for x in (np.nan, np.inf, -np.inf, -3.0, 1e-42, -1e-42):
            w[..., rng.integers(0, n, size=n // 9)] = x
        w[..., 5] = -np.nan
    elif kind == "wide":
        w = np.exp2((rng.random(shape) * 80 - 40).astype(np.float32)).astype(np.float32)
    elif kind == "few digits":  # many equal keys beside close ones
        w = (1.0 + rng.integers(0, 700, size=shape) * 2.0**-23).astype(np.float32)
    return w


@pytest.mark.parametrize("kind", ["ties", "zero", "special", "wide", "few digits"])
@pytest.mark.parametrize("L,keep,sinks,recent", [(33007, 9001, 3, 17), (70001, 30000, 7, 1),
                                                 (70001, 70000, 6, 300)])
def test_evict_long_rows_of_every_kind(kind, L, keep, sinks, recent):
    """Competing tokens that begin and end inside a lane's four, ranks among
    equals across waves, two KV heads, a short sequence beside."""
    c = Cache(46, (L, 300), 2, 64, 64, "bf16")
    w = many_kinds(c.rng, kind, (2, 2, c.mp * 64))
    announce(f"evict long {kind} L{L} keep{keep} sinks{sinks} recent{recent}")
    check_evict(c, w, keep, sinks, recent)


@pytest.mark.parametrize("sinks", [0, 3, 4])
@pytest.mark.parametrize("over", [-1, 0, 1, 2])
def test_evict_at_the_register_limit(sinks, over):
    """From the multiple of 4 at or below `sinks` to the last of the competing
    tokens: 32768 fit, one more does not."""
    recent = 5
    L = 32768 + over + (sinks & ~3) + recent
    c = Cache(47, (L,), 1, 64, 16, "bf16")
    w = many_kinds(c.rng, "ties", (1, 1, c.mp * 16))
    announce(f"evict register limit {over:+d} sinks{sinks}")
    check_evict(c, w, 12345, sinks, recent)
