"""Lists of more entries than a row's join holds, among so many blocks of rows that
rows with long supports are a kernel of their own: alpha below 1.5 (lists of 384,
joined to 256) and 1.5 (128). Tolerances as in test_gpu_chunk.py."""
import pytest

from test_gpu_chunk import Chunk, E

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


def many(c, G, one_part, alpha):
    """The plan is of many blocks (more than two of 16 rows a CU), and of one part
    of a row's tokens where asked for."""
    blocks = ((c.N // (16 // G)) + len(c.c.lens)) * c.c.Hkv
    assert blocks > 512
    entries = c.N * c.H * (384 if alpha < 1.5 else 128) * 8
    parts = E().entmaxkv_entmax_chunk_ws(c.c.shape(c.H), c.N, alpha) // entries
    assert (parts == 1) == one_part, parts


@pytest.mark.parametrize("kv,q_dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("alpha", [1.25, 1.5])
@pytest.mark.parametrize("one_part", [True, False])
def test_supports_of_every_length(kv, q_dtype, D, alpha, one_part):
    """Flat scores: the row of position p has a support of p + 1 tokens, 1 to 430
    (lists of one part end at 376 entries, joins at 256; 120 and 128 from 1.5)."""
    lens, new, pad = ([430], [430], 65800) if one_part else ([430] + [0] * 600, [430] + [0] * 600, 0)
    c = Chunk(50, lens, new, 1, D, 16, kv, 1, q_dtype, 0.02, pad=pad)
    many(c, 1, one_part, alpha)
    c.check(alpha)


@pytest.mark.parametrize("kv,q_dtype", TYPES)
@pytest.mark.parametrize("alpha,spread", [(1.25, 0.5), (1.25, 1.0), (1.25, 2.5), (1.5, 0.3)])
def test_supports_about_a_list(kv, q_dtype, alpha, spread):
    """Supports of tens to hundreds of tokens out of thousands, rows of both kinds in
    one tile."""
    for one_part, pad in ((True, 16700), (False, 2100)):
        c = Chunk(51, [2500], [20], 1, 64, 32, kv, 4, q_dtype, spread, pad=pad)
        many(c, 4, one_part, alpha)
        c.check(alpha)
