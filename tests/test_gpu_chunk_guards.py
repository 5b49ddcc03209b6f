"""What the chunk call writes, held between guards: out, tau, support and the
workspace end where they should, and rows of no sequence keep what they held,
whatever the token starts say."""
import numpy as np
import pytest
import torch

from parity_util import announce
from test_gpu_chunk import Chunk, E

pytestmark = pytest.mark.gpu
I32 = torch.int32
GUARD = 4096  # bytes on either side


class Guarded:
    """n bytes, 256-byte aligned, between guards of 0x5a."""

    def __init__(self, n, fill):
        self.n = n
        self.all = torch.full((n + 2 * GUARD,), 0x5a, dtype=torch.uint8, device="cuda")
        self.mid = self.all[GUARD:GUARD + n]
        self.mid.fill_(fill)

    def view(self, dtype, shape):
        return self.mid.view(dtype).view(shape)

    def whole(self):
        return bool((self.all[:GUARD] == 0x5a).all() and (self.all[GUARD + self.n:] == 0x5a).all())


def run(c, starts, alpha=1.5):
    q = c.q.cuda()
    N, H, D = q.shape
    k, v, table, lens = c.c.dev("k", "v", "table", "lens")
    mem = {"out": Guarded(q.numel() * q.element_size(), 0x11), "tau": Guarded(N * H * 4, 0x11),
           "support": Guarded(N * H * 4, 0x11),
           "ws": Guarded(E().entmaxkv_entmax_chunk_ws(c.c.shape(H), N, alpha), 0xff)}
    out = mem["out"].view(q.dtype, q.shape)
    tau, sup = mem["tau"].view(torch.float32, (N, H)), mem["support"].view(I32, (N, H))
    announce(f"guarded chunk starts={starts} q={q.dtype} kv={c.c.kv}")
    E().entmaxkv_entmax_chunk(c.c.shape(H), q, torch.tensor(starts, dtype=I32, device="cuda"), k, v,
                              table, lens, alpha, out, tau=tau, support=sup, ws=mem["ws"].mid)
    torch.cuda.synchronize()
    for name, m in mem.items():
        assert m.whole(), name
    return mem, (out, tau, sup)


def untouched(x):
    return bool((x.contiguous().view(torch.uint8) == 0x11).all())


TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


@pytest.mark.parametrize("kv,q_dtype", TYPES)
@pytest.mark.parametrize("starts", [[0, 4, 8, 12], [0, 4, 8, 999], [-5, 4, 8, 12]])
def test_starts_beyond_the_rows_are_the_nearest_row(kv, q_dtype, starts):
    c = Chunk(60, [30, 30, 30], [4, 4, 4], 1, 64, 16, kv, 2, q_dtype,
              pad=5 if starts[3] == 12 else 0)
    _, got = run(c, starts)
    for x in got:
        assert untouched(x[12:])
        x[12:] = 7  # as check() has it
    c.check(1.5, got)


@pytest.mark.parametrize("kv,q_dtype", TYPES)
@pytest.mark.parametrize("starts", [[12, 8, 4, 0], [2**31 - 1] * 4, [-2**31] * 4, [5, 5, 5, 5]])
def test_starts_without_rows_write_nothing(kv, q_dtype, starts):
    c = Chunk(61, [30, 30, 30], [4, 4, 4], 1, 64, 16, kv, 2, q_dtype, pad=3)
    _, got = run(c, starts)
    for x in got:
        assert untouched(x)


@pytest.mark.parametrize("kv,q_dtype", TYPES)
@pytest.mark.parametrize("starts", [[0, 9, 3, 12], [0, 12, 0, 12], [3, 15, 1, 2]])
def test_starts_out_of_order_stay_within_their_rows(kv, q_dtype, starts):
    """Sequences that claim the same rows: what those hold is not defined, all
    other rows keep what they held."""
    c = Chunk(62, [30, 30, 30], [4, 4, 4], 1, 64, 16, kv, 2, q_dtype, pad=3)
    _, got = run(c, starts)
    owned = np.zeros(15, bool)
    for a, b in zip(starts, starts[1:]):
        owned[min(a, 15):min(b, 15)] = True
    for x in got:
        assert untouched(x[torch.from_numpy(~owned).cuda()])


@pytest.mark.parametrize("kv,q_dtype", TYPES)
@pytest.mark.parametrize("spread", [0.05, 2.5])
@pytest.mark.parametrize("lens,new,G", [([700, 3], [330, 1], 4), ([900] * 3, [1, 2, 0], 8),
                                        ([1000], [1000], 1)])
def test_guards_of_blocks_and_parts(kv, q_dtype, spread, lens, new, G):
    """Long and short supports, many rows and few, several parts."""
    c = Chunk(63, lens, new, 2, 64, 16, kv, 2 * G, q_dtype, spread, pad=2)
    for alpha in (1.25, 1.5):
        _, got = run(c, c.starts.tolist(), alpha)
        for x in got:
            assert untouched(x[c.starts[-1]:])
            assert not untouched(x[:c.starts[-1]])
