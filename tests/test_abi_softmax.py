"""Refusals of the softmax decode and eviction calls: documented codes from
the C ABI, exceptions from the binding, before any HIP call."""
import ctypes

import pytest
import torch

from test_abi import ek, shape  # noqa: F401

D = ctypes.c_void_p(256)
BIG = 1 << 40
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


def window(ek, s, q=D, qd=1, n=1, k=D, v=D, bt=D, lens=D, w=1024, sinks=4, out=D, ws=D, nws=BIG):
    return ek.lib.entmaxkv_softmax_window(ctypes.byref(s), q, qd, n, k, v, bt, lens, w, sinks,
                                          out, None, ws, nws, None, None)


def prefix(ek, s, q=D, qd=1, pt=D, pages=64, out=D, ws=D, nws=BIG, bt=D):
    return ek.lib.entmaxkv_softmax_prefix(ctypes.byref(s), q, qd, D, D, pt, pages, bt, D, out,
                                          None, ws, nws, None, None)


def weights(ek, s, q=D, qd=0, alpha=1.0, tau=D, w=5, sinks=0, decay=0.9, win=None, wout=D, k=D):
    return ek.lib.entmaxkv_accumulate_weights(ctypes.byref(s), q, qd, k, D, D, alpha, tau, w,
                                              sinks, decay, win, wout, None, None)


def evict(ek, s, k=D, keep=100, sinks=4, recent=10, w=D, new_table=ctypes.c_void_p(512), kept=D,
          new_lens=ctypes.c_void_p(512), new_w=None):
    return ek.lib.entmaxkv_evict(ctypes.byref(s), k, D, D, D, w, keep, sinks, recent, new_table,
                                 kept, new_lens, new_w, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), INVALID), (dict(n=-1), INVALID), (dict(w=0), INVALID), (dict(w=-5), INVALID),
    (dict(sinks=-1), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(bt=None), INVALID), (dict(lens=None), INVALID),
    (dict(out=None), INVALID), (dict(q=ctypes.c_void_p(264)), INVALID),
    (dict(out=ctypes.c_void_p(264)), INVALID), (dict(qd=2), UNSUPPORTED),
    (dict(qd=-1), UNSUPPORTED), (dict(n=1 << 20), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(nws=16), WORKSPACE), (dict(ws=ctypes.c_void_p(16)), INVALID),
])
def test_window_refusals(ek, kw, code):
    assert window(ek, shape(ek), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(pages=0), INVALID), (dict(pages=-1), INVALID), (dict(pages=4097), INVALID),
    (dict(pt=None), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(bt=None), INVALID), (dict(qd=3), UNSUPPORTED), (dict(nws=16), WORKSPACE),
    (dict(q=ctypes.c_void_p(264)), INVALID),
])
def test_prefix_refusals(ek, kw, code):
    assert prefix(ek, shape(ek), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(alpha=0.99), INVALID), (dict(alpha=float("nan")), INVALID),
    (dict(alpha=float("inf")), INVALID), (dict(decay=float("nan")), INVALID),
    (dict(decay=float("inf")), INVALID), (dict(w=0), INVALID), (dict(sinks=-1), INVALID),
    (dict(tau=None), INVALID), (dict(wout=None), INVALID), (dict(q=None), INVALID),
    (dict(qd=5), UNSUPPORTED), (dict(k=ctypes.c_void_p(264)), INVALID),
])
def test_weights_refusals(ek, kw, code):
    assert weights(ek, shape(ek), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(keep=0), INVALID), (dict(keep=-3), INVALID), (dict(sinks=-1), INVALID),
    (dict(recent=-1), INVALID), (dict(keep=13), INVALID), (dict(keep=2**25 + 1), UNSUPPORTED),
    (dict(sinks=2**31 - 1, recent=2**31 - 1), INVALID), (dict(w=None), INVALID),
    (dict(new_table=None), INVALID), (dict(new_table=D), INVALID), (dict(kept=None), INVALID),
    (dict(new_lens=None), INVALID), (dict(new_lens=D), INVALID), (dict(new_w=D), INVALID),
    (dict(w=ctypes.c_void_p(260)), INVALID),
    (dict(k=ctypes.c_void_p(264)), INVALID),
])
def test_evict_refusals(ek, kw, code):
    assert evict(ek, shape(ek), **kw) == code


def test_shapes_are_checked(ek):
    for kw, code in ((dict(head_dim=96), UNSUPPORTED), (dict(batch=0), INVALID),
                     (dict(page_size=8), UNSUPPORTED),
                     (dict(num_q_heads=48, num_kv_heads=3), UNSUPPORTED)):
        s = shape(ek, **kw)
        assert window(ek, s) == prefix(ek, s) == weights(ek, s) == evict(ek, s) == code
    s = shape(ek, kv_dtype="f32")
    assert window(ek, s, qd=1) == prefix(ek, s, qd=1) == weights(ek, s, qd=1) == UNSUPPORTED


def test_workspace_queries(ek):
    s = shape(ek)
    n = ek.entmaxkv_softmax_window_ws(s, 1, 1024, 4)
    assert n > 0 and n % 256 == 0
    # windows and sinks beyond every length are that of the longest sequence
    assert ek.entmaxkv_softmax_window_ws(s, 1, ek.FULL_WINDOW, 2**31 - 1) >= n
    # enough row blocks: no parts to join
    assert ek.entmaxkv_softmax_window_ws(shape(ek, batch=512), 1, 128, 0) == 0
    assert ek.entmaxkv_softmax_prefix_ws(s, 4096) > 0
    for bad in ((0, 1, 0), (1, 0, 0), (1, 1, -1)):
        with pytest.raises(ek.EntmaxKVError):
            ek.entmaxkv_softmax_window_ws(s, *bad)
    with pytest.raises(ek.EntmaxKVError):
        ek.entmaxkv_softmax_prefix_ws(s, 0)
    assert ek.lib.entmaxkv_softmax_window_ws(ctypes.byref(s), 1, 8, 0, None) == INVALID
    assert ek.lib.entmaxkv_softmax_prefix_ws(ctypes.byref(s), 8, None) == INVALID


def _tensors(ek, **kw):
    s = shape(ek, batch=2, num_q_heads=4, num_kv_heads=2, head_dim=64, page_size=16,
              max_pages_per_seq=3, num_phys_pages=9)
    i32 = torch.int32
    t = dict(q=torch.zeros(2, 1, 4, 64), k=torch.zeros(9, 2, 16, 64, dtype=torch.bfloat16),
             v=torch.zeros(9, 2, 16, 64, dtype=torch.bfloat16), bt=torch.zeros(2, 3, dtype=i32),
             lens=torch.zeros(2, dtype=i32), out=torch.zeros(2, 1, 4, 64),
             lse=torch.zeros(2, 1, 4), w=torch.zeros(2, 2, 48), nw=torch.zeros(2, 2, 48),
             kept=torch.zeros(2, 2, 20, dtype=i32), nl=torch.zeros(2, dtype=i32),
             nt=torch.zeros(2, 3, dtype=i32), pt=torch.zeros(2, dtype=i32))
    t.update(kw)
    return s, t


CALLS = {
    "window": lambda E, s, t: E.entmaxkv_softmax_window(s, t["q"], t["k"], t["v"], t["bt"],
                                                        t["lens"], 8, 2, t["out"], t["lse"]),
    "prefix": lambda E, s, t: E.entmaxkv_softmax_prefix(s, t["q"], t["k"], t["v"], t["pt"], 2,
                                                        t["bt"], t["lens"], t["out"], t["lse"]),
    "weights": lambda E, s, t: E.entmaxkv_accumulate_weights(s, t["q"], t["k"], t["bt"], t["lens"],
                                                             1.0, t["lse"], 0.9, t["w"], t["nw"]),
    "evict": lambda E, s, t: E.entmaxkv_evict(s, t["k"], t["v"], t["bt"], t["lens"], t["w"], 20,
                                              2, 3, t["nt"], t["kept"], t["nl"], t["nw"]),
}


@pytest.mark.parametrize("call,bad,error", [
    ("window", dict(q=torch.zeros(2, 1, 4, 64, dtype=torch.float16)), TypeError),
    ("window", dict(q=torch.zeros(2, 1, 4, 63)), ValueError),
    ("window", dict(q=None), TypeError),
    ("window", dict(out=torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16)), TypeError),
    ("window", dict(out=torch.zeros(2, 1, 2, 64)), ValueError),
    ("window", dict(lse=torch.zeros(2, 3)), ValueError),
    ("window", dict(k=torch.zeros(9, 2, 16, 64)), TypeError),
    ("window", dict(v=torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16)), ValueError),
    ("window", dict(k=torch.zeros(9, 2, 64, 16, dtype=torch.bfloat16).transpose(2, 3)),
     ValueError),
    ("window", dict(bt=torch.zeros(2, 3)), TypeError),
    ("window", dict(), ValueError),  # host tensors
    ("prefix", dict(pt=torch.zeros(1, dtype=torch.int32)), ValueError),
    ("prefix", dict(pt=torch.zeros(2)), TypeError),
    ("prefix", dict(), ValueError),
    ("weights", dict(w=torch.zeros(2, 2, 47)), ValueError),
    ("weights", dict(nw=torch.zeros(2, 2, 48, dtype=torch.float64)), TypeError),
    ("weights", dict(), ValueError),
    ("evict", dict(kept=torch.zeros(2, 2, 19, dtype=torch.int32)), ValueError),
    ("evict", dict(nt=torch.zeros(2, 2, dtype=torch.int32)), ValueError),
    ("evict", dict(nl=torch.zeros(2)), TypeError),
    ("evict", dict(), ValueError),
])
def test_binding_refusals(ek, call, bad, error):
    s, t = _tensors(ek, **bad)
    with pytest.raises(error):
        CALLS[call](ek, s, t)


def test_bf16_queries_need_a_bf16_cache(ek):
    s, t = _tensors(ek)
    f = shape(ek, batch=2, num_q_heads=4, num_kv_heads=2, head_dim=64, page_size=16,
              max_pages_per_seq=3, num_phys_pages=9, kv_dtype="f32")
    t.update(q=t["q"].bfloat16(), k=t["k"].float(), v=t["v"].float())
    with pytest.raises(TypeError):
        CALLS["window"](ek, f, t)


@pytest.mark.parametrize("x", [2**31, -2**31 - 1, 2**32 + 8])
def test_numbers_beyond_int32_are_refused(ek, x):
    # (a C argument would hold 2^32 + 8 as a window of 8)
    s = shape(ek)
    for call in (lambda: ek.entmaxkv_softmax_window_ws(s, x, 8, 2),
                 lambda: ek.entmaxkv_softmax_window_ws(s, 1, x, 2),
                 lambda: ek.entmaxkv_softmax_window_ws(s, 1, 8, x),
                 lambda: ek.entmaxkv_softmax_prefix_ws(s, x)):
        with pytest.raises(ValueError, match="int32"):
            call()


@pytest.mark.parametrize("at", [0, 1, 2])
def test_evict_numbers_beyond_int32_are_refused(ek, at, monkeypatch):
    s, t = _tensors(ek)
    monkeypatch.setattr(ek, "_one_device", lambda **kw: None)  # host tensors
    monkeypatch.setattr(ek, "_ptr", lambda *a, **kw: None)
    n = [20, 2, 3]
    n[at] += 2**32
    with pytest.raises(ValueError, match="int32"):
        ek.entmaxkv_evict(s, t["k"], t["v"], t["bt"], t["lens"], t["w"], *n, t["nt"], t["kept"],
                          t["nl"])
