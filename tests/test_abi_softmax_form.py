"""The query for the form of the softmax attention kernel: documented answers
and refusals."""
import ctypes

import pytest

from test_abi import ek, shape  # noqa: F401

INVALID, UNSUPPORTED = -1, -2


def test_forms_by_rows_and_work(ek):
    few, many = ek.ENTMAXKV_FORM_FEW_ROWS, ek.ENTMAXKV_FORM_MANY_ROWS
    s = shape(ek)  # a batch of long sequences
    form = ek.entmaxkv_softmax_form
    for qd in (ek.ENTMAXKV_F32, ek.ENTMAXKV_BF16):
        assert form(s, qd) == few
        assert form(s, qd, q_tokens=512, window=4096) == many
        # little work: the rows alone do not decide
        assert form(shape(ek, batch=1, num_q_heads=1, num_kv_heads=1), qd, q_tokens=64,
                    window=16) == few
        assert form(shape(ek, batch=64), qd, prefix_pages=1024) == many
        assert form(shape(ek, batch=1), qd, prefix_pages=1024) == few
        # window arguments say nothing beside a prefix
        assert form(shape(ek, batch=64), qd, 0, 0, -1, 1024) == many


@pytest.mark.parametrize("args,code", [
    ((0, 0, 8, 0, 0), INVALID), ((0, 1, 0, 0, 0), INVALID), ((0, 1, 8, -1, 0), INVALID),
    ((0, 1, 8, 0, -1), INVALID), ((0, 1, 8, 0, 4097), INVALID), ((7, 1, 8, 0, 0), UNSUPPORTED),
    ((7, 1, 8, 0, 4), UNSUPPORTED), ((0, 1 << 20, 8, 0, 0), UNSUPPORTED),
])
def test_refusals(ek, args, code):
    n = ctypes.c_int32(-9)
    s = shape(ek)
    assert ek.lib.entmaxkv_softmax_form(ctypes.byref(s), *args, ctypes.byref(n)) == code
    assert n.value == -9


def test_refusals_of_types_and_pointers(ek):
    s, f, n = shape(ek), shape(ek, kv_dtype="f32"), ctypes.c_int32()
    call = ek.lib.entmaxkv_softmax_form
    assert call(ctypes.byref(f), 1, 1, 8, 0, 0, ctypes.byref(n)) == UNSUPPORTED
    assert call(ctypes.byref(s), 1, 1, 8, 0, 0, None) == INVALID
    assert call(None, 1, 1, 8, 0, 0, ctypes.byref(n)) == INVALID
    with pytest.raises(ValueError, match="int32"):
        ek.entmaxkv_softmax_form(s, 0, 1, 2**31)
