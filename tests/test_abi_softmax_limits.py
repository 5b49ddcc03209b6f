"""Shapes beyond what one launch holds (2^32 threads) are refused before any
HIP call, at the documented bounds."""
import ctypes

import pytest

from test_abi import ek, shape  # noqa: F401
from test_abi_softmax import UNSUPPORTED, evict, prefix, weights, window


def heads(ek, batch, kv_heads):
    return shape(ek, batch=batch, num_q_heads=kv_heads, num_kv_heads=kv_heads, head_dim=64,
                 page_size=16, max_pages_per_seq=4, num_phys_pages=4)


@pytest.mark.parametrize("batch,kv_heads", [(1 << 24, 1), (1 << 21, 8), (1, 1 << 24)])
def test_two_to_the_24_heads(ek, batch, kv_heads):
    s = heads(ek, batch, kv_heads)
    assert window(ek, s, w=8, sinks=0) == UNSUPPORTED
    assert prefix(ek, s, pages=2) == UNSUPPORTED
    assert evict(ek, s) == UNSUPPORTED
    if batch == 1:
        assert weights(ek, s) == UNSUPPORTED
    n = ctypes.c_size_t()
    assert ek.lib.entmaxkv_softmax_window_ws(ctypes.byref(s), 1, 8, 0,
                                             ctypes.byref(n)) == UNSUPPORTED


def test_below_the_bounds(ek):
    n = ctypes.c_size_t()
    s = heads(ek, (1 << 24) - 1, 1)
    assert ek.lib.entmaxkv_softmax_window_ws(ctypes.byref(s), 1, 8, 0, ctypes.byref(n)) == 0
    assert evict(ek, heads(ek, 1 << 22, 1)) == UNSUPPORTED
    # (a refusal that comes after the bound's: a pointer that is not aligned)
    assert evict(ek, heads(ek, (1 << 22) - 1, 1), k=ctypes.c_void_p(264)) == -1
