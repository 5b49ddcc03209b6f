"""Refusals of the plan, append and chunk calls: documented codes from the C
ABI, exceptions from the binding, before any HIP call."""
import ctypes

import pytest
import torch

from test_abi import ek, shape  # noqa: F401

D = ctypes.c_void_p(256)
E = ctypes.c_void_p(512)
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


def plan(ek, s, n=64, lens=D, new=D, free=D, cap=100, count=D, table=D, new_lens=E, starts=E,
         pos=E, slots=E, left=E):
    return ek.lib.entmaxkv_plan_tokens(ctypes.byref(s), n, lens, new, free, cap, count, table,
                                       new_lens, starts, pos, slots, left, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), INVALID), (dict(n=-1), INVALID), (dict(n=1 << 24), UNSUPPORTED),
    (dict(lens=None), INVALID), (dict(new=None), INVALID), (dict(free=None), INVALID),
    (dict(cap=-1), INVALID), (dict(count=None), INVALID), (dict(table=None), INVALID),
    (dict(new_lens=None), INVALID), (dict(starts=None), INVALID), (dict(pos=None), INVALID),
    (dict(slots=None), INVALID), (dict(left=None), INVALID), (dict(new_lens=D), INVALID),
    (dict(left=D), INVALID), (dict(free=None, cap=0, left=D), INVALID),
])
def test_plan_refusals(ek, kw, code):
    assert plan(ek, shape(ek), **kw) == code


def test_plan_shape_refusals(ek):
    small = dict(num_q_heads=1, num_kv_heads=1)
    assert plan(ek, shape(ek, batch=65537, **small)) == UNSUPPORTED
    assert plan(ek, shape(ek, batch=0)) == INVALID
    assert plan(ek, shape(ek, page_size=8)) == UNSUPPORTED


def append(ek, s, q=D, k=D, v=D, pos=D, slots=D, freqs=D, axis=None, qw=None, kw_=None, out=E,
           kp=D, vp=D, no_params=False, **p):
    base = dict(num_tokens=10, x_dtype=1, q_dtype=0, rot_dim=128, axes=1, interleaved=0,
                q_stride=6144, k_stride=6144, v_stride=6144, eps=1e-6, q_scale=1.0)
    base.update(p)
    a = ek.Append(**base)
    return ek.lib.entmaxkv_append_kv(ctypes.byref(s), None if no_params else ctypes.byref(a), q, k,
                                     v, pos, slots, freqs, axis, qw, kw_, out, kp, vp, None, None)


BAD = ctypes.c_void_p(264)


@pytest.mark.parametrize("kw,code", [
    (dict(no_params=True), INVALID), (dict(num_tokens=0), INVALID),
    (dict(num_tokens=-7), INVALID), (dict(num_tokens=1 << 24), UNSUPPORTED),
    (dict(x_dtype=2), UNSUPPORTED), (dict(q_dtype=-1), UNSUPPORTED),
    (dict(rot_dim=-16), INVALID), (dict(rot_dim=144), INVALID), (dict(rot_dim=24), UNSUPPORTED),
    (dict(axes=0), INVALID), (dict(axes=9, axis=D), INVALID), (dict(axes=3), INVALID),
    (dict(interleaved=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(q_scale=float("inf")), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(slots=None), INVALID), (dict(out=None), INVALID),
    (dict(kp=None), INVALID), (dict(vp=None), INVALID), (dict(pos=None), INVALID),
    (dict(freqs=None), INVALID), (dict(q=BAD), INVALID), (dict(k=BAD), INVALID),
    (dict(v=BAD), INVALID), (dict(out=BAD), INVALID), (dict(kp=BAD), INVALID),
    (dict(vp=BAD), INVALID), (dict(freqs=ctypes.c_void_p(260)), INVALID),
    (dict(q_stride=4095), INVALID), (dict(q_stride=4088), INVALID), (dict(k_stride=1016), INVALID),
    (dict(v_stride=1028), INVALID), (dict(x_dtype=0, v_stride=1026), INVALID),
    (dict(k_stride=-1024), INVALID), (dict(q_stride=(1 << 32) + 8), INVALID),
])
def test_append_refusals(ek, kw, code):
    assert append(ek, shape(ek), **kw) == code


def small(ek, **kw):
    return shape(ek, **{**dict(batch=2, num_q_heads=4, num_kv_heads=2, head_dim=64, page_size=16,
                               max_pages_per_seq=3, num_phys_pages=9), **kw})


def test_append_binding_refusals(ek):
    bf, i32 = torch.bfloat16, torch.int32
    x = torch.zeros(5, 8 * 64, dtype=bf)
    good = dict(q=x[:, :256].view(5, 4, 64), k=x[:, 256:384].view(5, 2, 64),
                v=x[:, 384:].view(5, 2, 64), positions=torch.zeros(5, dtype=i32),
                slots=torch.zeros(5, dtype=i32), q_out=torch.zeros(5, 4, 64),
                k_pool=torch.zeros(9, 2, 16, 64, dtype=bf), v_pool=torch.zeros(9, 2, 16, 64, dtype=bf),
                freqs=torch.zeros(32, dtype=torch.float64))

    def call(**kw):
        ek.entmaxkv_append_kv(small(ek), **{**good, **kw})

    for kw, e in [(dict(q=good["q"].float()), TypeError), (dict(k=good["q"]), ValueError),
                  (dict(v=good["v"][:4]), ValueError), (dict(q=None), TypeError),
                  (dict(q=good["q"].transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
                  (dict(slots=torch.zeros(4, dtype=i32)), ValueError),
                  (dict(positions=torch.zeros(3, 4, dtype=i32)), ValueError),
                  (dict(positions=torch.zeros(3, 5, dtype=i32)), ValueError),
                  (dict(positions=None), ValueError), (dict(freqs=torch.zeros(32)), TypeError),
                  (dict(q_out=torch.zeros(5, 4, 63)), ValueError),
                  (dict(q_out=torch.zeros(5, 4, 64, dtype=torch.float16)), TypeError),
                  (dict(k_pool=torch.zeros(9, 2, 16, 64)), TypeError),
                  (dict(v_pool=torch.zeros(8, 2, 16, 64, dtype=bf)), ValueError),
                  (dict(q_weight=torch.ones(63)), ValueError),
                  (dict(k_weight=torch.ones(64, dtype=bf)), TypeError),
                  (dict(), ValueError)]:  # all good, but not on a device
        with pytest.raises(e):
            call(**kw)


def test_plan_binding_refusals(ek):
    i32 = torch.int32
    z = lambda n: torch.zeros(n, dtype=i32)  # noqa: E731
    good = dict(seq_lens=z(2), new_tokens=z(2), free_pages=z(4), free_count=z(1),
                block_table=z((2, 3)), new_lens=z(2), token_starts=z(3), positions=z(8),
                slots=z(8), free_left=z(1))
    for kw, e in [(dict(token_starts=z(2)), ValueError), (dict(block_table=z((2, 2))), ValueError),
                  (dict(positions=z(7)), ValueError), (dict(slots=None), TypeError),
                  (dict(new_lens=z(2).long()), TypeError), (dict(free_count=None), ValueError),
                  (dict(seq_lens=z((2, 2))[:, 0]), ValueError), (dict(), ValueError)]:
        with pytest.raises(e):
            ek.entmaxkv_plan_tokens(small(ek), **{**good, **kw})


def chunk(ek, s, q=D, qd=1, n=64, starts=D, k=D, v=D, bt=D, lens=D, alpha=1.5, out=E, ws=D,
          nws=1 << 40):
    return ek.lib.entmaxkv_entmax_chunk(ctypes.byref(s), q, qd, n, starts, k, v, bt, lens, alpha,
                                        out, None, None, ws, nws, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), INVALID), (dict(n=-3), INVALID), (dict(n=1 << 24), UNSUPPORTED),
    (dict(alpha=1.0), INVALID), (dict(alpha=0.5), INVALID), (dict(alpha=float("nan")), INVALID),
    (dict(alpha=float("inf")), INVALID), (dict(qd=2), UNSUPPORTED), (dict(q=None), INVALID),
    (dict(starts=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(bt=None), INVALID), (dict(lens=None), INVALID), (dict(out=None), INVALID),
    (dict(q=BAD), INVALID), (dict(k=BAD), INVALID), (dict(v=BAD), INVALID), (dict(out=BAD), INVALID),
    (dict(ws=None), WORKSPACE), (dict(nws=256), WORKSPACE), (dict(ws=ctypes.c_void_p(16)), INVALID),
])
def test_chunk_refusals(ek, kw, code):
    assert chunk(ek, shape(ek), **kw) == code


def test_chunk_types_and_sizes(ek):
    assert chunk(ek, shape(ek, kv_dtype="f32")) == UNSUPPORTED  # bf16 queries, float32 cache
    assert chunk(ek, shape(ek, head_dim=96)) == UNSUPPORTED
    # more workgroups than a launch holds
    one = dict(num_q_heads=1, num_kv_heads=1, batch=1 << 24)
    assert chunk(ek, shape(ek, **one), n=(1 << 24) - 1) == UNSUPPORTED
    out = ctypes.c_size_t(0)
    ws = ek.lib.entmaxkv_entmax_chunk_ws
    assert ws(ctypes.byref(shape(ek)), 64, 1.5, None) == INVALID
    assert ws(ctypes.byref(shape(ek)), 0, 1.5, ctypes.byref(out)) == INVALID
    assert ws(ctypes.byref(shape(ek)), 64, 1.0, ctypes.byref(out)) == INVALID
    # flat weights take longer lists
    assert ek.entmaxkv_entmax_chunk_ws(shape(ek), 64, 1.25) > ek.entmaxkv_entmax_chunk_ws(
        shape(ek), 64, 1.5) > 0


def test_chunk_binding_refusals(ek):
    bf, i32 = torch.bfloat16, torch.int32
    good = dict(q=torch.zeros(5, 4, 64, dtype=bf), token_starts=torch.zeros(3, dtype=i32),
                k_pool=torch.zeros(9, 2, 16, 64, dtype=bf),
                v_pool=torch.zeros(9, 2, 16, 64, dtype=bf), block_table=torch.zeros(2, 3, dtype=i32),
                seq_lens=torch.zeros(2, dtype=i32), alpha=1.5, out=torch.zeros(5, 4, 64, dtype=bf))
    for kw, e in [(dict(q=torch.zeros(5, 2, 64, dtype=bf)), ValueError),
                  (dict(q=torch.zeros(5, 4 * 64, dtype=bf)), ValueError),
                  (dict(q=torch.zeros(5, 4, 128, dtype=bf)[..., :64]), ValueError),
                  (dict(q=torch.zeros(5, 4, 64, dtype=torch.float16)), TypeError),
                  (dict(token_starts=torch.zeros(2, dtype=i32)), ValueError),
                  (dict(out=torch.zeros(5, 4, 64)), TypeError),
                  (dict(out=torch.zeros(4, 4, 64, dtype=bf)), ValueError),
                  (dict(tau=torch.zeros(5, 3)), ValueError),
                  (dict(support=torch.zeros(5, 4)), TypeError),
                  (dict(k_pool=torch.zeros(8, 2, 16, 64, dtype=bf)), ValueError),
                  (dict(seq_lens=torch.zeros(1, dtype=i32)), ValueError), (dict(), ValueError)]:
        with pytest.raises(e):
            ek.entmaxkv_entmax_chunk(small(ek), **{**good, **kw})
