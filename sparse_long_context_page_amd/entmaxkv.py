"""Python binding of libentmaxkv.so (the C ABI in include/entmaxkv.h).

Argument marshalling only: torch tensors supply device pointers and the
current HIP stream; every step of the decode runs in the library's HIP
kernels. Importing this module loads the library and raises if it is not
built (there is no fallback path).

The function names match the C ABI:
    entmaxkv_build_page_meta, entmaxkv_append_page_meta, entmaxkv_score_select,
    entmaxkv_score_select_noalloc, entmaxkv_decode_sparse, entmaxkv_decode_topk,
    entmaxkv_decode_full, entmaxkv_build_page_moments,
    entmaxkv_append_page_moments, entmaxkv_gauss_select, entmaxkv_softmax_window,
    entmaxkv_softmax_prefix, entmaxkv_accumulate_weights, entmaxkv_evict,
    entmaxkv_plan_tokens, entmaxkv_append_kv, entmaxkv_entmax_chunk, entmaxkv_entmax_chunk_ws,
    entmaxkv_workspace_bytes, entmaxkv_softmax_window_ws, entmaxkv_softmax_prefix_ws,
    entmaxkv_softmax_form, entmaxkv_topk_kernels, entmaxkv_strerror
"""
from __future__ import annotations

import ctypes
import os
from contextlib import nullcontext

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libentmaxkv.so")

ENTMAXKV_OK = 0
ENTMAXKV_ERR_INVALID = -1
ENTMAXKV_ERR_UNSUPPORTED = -2
ENTMAXKV_ERR_WORKSPACE = -3
ENTMAXKV_ERR_HIP = -4

ENTMAXKV_F32 = 0
ENTMAXKV_BF16 = 1

ENTMAXKV_WS_SELECT = 0
ENTMAXKV_WS_SPARSE = 1
ENTMAXKV_WS_FULL = 2
ENTMAXKV_WS_GAUSS = 3
ENTMAXKV_WS_TOPK = 4
ENTMAXKV_FORM_FEW_ROWS = 0
ENTMAXKV_FORM_MANY_ROWS = 1

# kernels each entry point launches (for per-kernel event timing)
KERNELS = {"build_page_meta": 1, "append_page_meta": 1, "score_select": 2,
           "score_select_noalloc": 2, "decode_sparse": 2, "decode_topk": 4,
           "decode_full": 2, "build_page_moments": 1, "append_page_moments": 1,
           "gauss_select": 2, "softmax_window": 2, "softmax_prefix": 2, "accumulate_weights": 1,
           "evict": 1, "plan_tokens": 1, "append_kv": 1, "entmax_chunk": 3}

FULL_WINDOW = 2**31 - 1  # a window that hides no token


class Shape(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32),
        ("num_phys_pages", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
    ]


class Append(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int32),
        ("x_dtype", ctypes.c_int32),
        ("q_dtype", ctypes.c_int32),
        ("rot_dim", ctypes.c_int32),
        ("axes", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64),
        ("eps", ctypes.c_float),
        ("q_scale", ctypes.c_float),
    ]


class EntmaxKVError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {entmaxkv_strerror(code)} (code {code})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python -m sparse_long_context_page_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, F32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    SP = ctypes.POINTER(Shape)
    lib.entmaxkv_build_page_meta.argtypes = [SP, P, P, P, P, P, P]
    lib.entmaxkv_append_page_meta.argtypes = [SP, P, P, P, P, I32, P, P, P]
    lib.entmaxkv_score_select.argtypes = [SP, P, P, P, P, I32, P, P, P, SZ, P, P]
    lib.entmaxkv_score_select_noalloc.argtypes = [SP, P, P, P, P, I32, P, P, P, P]
    lib.entmaxkv_decode_sparse.argtypes = [SP, P, P, P, P, P, P, I32, F32, P, P, P, P, SZ, P, P]
    lib.entmaxkv_decode_topk.argtypes = [SP, P, P, P, P, P, P, I32, F32, P, P, P, P, P, P, SZ,
                                         P, P]
    lib.entmaxkv_decode_full.argtypes = [SP, P, P, P, P, P, F32, P, P, P, P, SZ, P, P]
    lib.entmaxkv_build_page_moments.argtypes = [SP, P, P, P, P, P, P]
    lib.entmaxkv_append_page_moments.argtypes = [SP, P, P, P, P, I32, P, P, P]
    lib.entmaxkv_gauss_select.argtypes = [SP, P, P, P, P, F32, F32, I32, P, P, P, SZ, P, P]
    lib.entmaxkv_softmax_window.argtypes = [SP, P, I32, I32, P, P, P, P, I32, I32, P, P, P, SZ, P,
                                            P]
    lib.entmaxkv_softmax_window_ws.argtypes = [SP, I32, I32, I32, ctypes.POINTER(SZ)]
    lib.entmaxkv_softmax_prefix.argtypes = [SP, P, I32, P, P, P, I32, P, P, P, P, P, SZ, P, P]
    lib.entmaxkv_softmax_prefix_ws.argtypes = [SP, I32, ctypes.POINTER(SZ)]
    lib.entmaxkv_softmax_form.argtypes = [SP, I32, I32, I32, I32, I32, ctypes.POINTER(I32)]
    lib.entmaxkv_accumulate_weights.argtypes = [SP, P, I32, P, P, P, F32, P, I32, I32, F32, P, P,
                                                P, P]
    lib.entmaxkv_evict.argtypes = [SP, P, P, P, P, P, I32, I32, I32, P, P, P, P, P, P]
    lib.entmaxkv_plan_tokens.argtypes = [SP, I32, P, P, P, I32, P, P, P, P, P, P, P, P, P]
    lib.entmaxkv_append_kv.argtypes = [SP, ctypes.POINTER(Append), *[P] * 14]
    lib.entmaxkv_entmax_chunk.argtypes = [SP, P, I32, I32, P, P, P, P, P, F32, P, P, P, P, SZ, P,
                                          P]
    lib.entmaxkv_entmax_chunk_ws.argtypes = [SP, I32, F32, ctypes.POINTER(SZ)]
    lib.entmaxkv_workspace_bytes.argtypes = [SP, I32, I32, ctypes.POINTER(SZ)]
    lib.entmaxkv_topk_kernels.argtypes = [SP, I32, ctypes.POINTER(I32)]
    lib.entmaxkv_strerror.argtypes = [ctypes.c_int]
    lib.entmaxkv_strerror.restype = ctypes.c_char_p
    lib.entmaxkv_version.argtypes = []
    for name in ("entmaxkv_build_page_meta", "entmaxkv_append_page_meta",
                 "entmaxkv_score_select", "entmaxkv_score_select_noalloc",
                 "entmaxkv_decode_sparse", "entmaxkv_decode_topk", "entmaxkv_decode_full",
                 "entmaxkv_build_page_moments", "entmaxkv_append_page_moments",
                 "entmaxkv_gauss_select", "entmaxkv_softmax_window",
                 "entmaxkv_softmax_window_ws", "entmaxkv_softmax_prefix",
                 "entmaxkv_softmax_prefix_ws", "entmaxkv_softmax_form",
                 "entmaxkv_accumulate_weights", "entmaxkv_evict", "entmaxkv_plan_tokens",
                 "entmaxkv_append_kv", "entmaxkv_entmax_chunk", "entmaxkv_entmax_chunk_ws",
                 "entmaxkv_workspace_bytes", "entmaxkv_topk_kernels", "entmaxkv_version"):
        getattr(lib, name).restype = ctypes.c_int
    return lib


lib = _load()


def entmaxkv_strerror(code: int) -> str:
    return lib.entmaxkv_strerror(int(code)).decode()


def make_shape(batch, num_q_heads, num_kv_heads, head_dim, page_size, max_pages_per_seq,
               num_phys_pages, kv_dtype) -> Shape:
    if isinstance(kv_dtype, str):
        kv_dtype = {"f32": ENTMAXKV_F32, "bf16": ENTMAXKV_BF16}[kv_dtype]
    return Shape(int(batch), int(num_q_heads), int(num_kv_heads), int(head_dim), int(page_size),
                 int(max_pages_per_seq), int(num_phys_pages), int(kv_dtype))


# ---------------------------------------------------------------------------
# marshalling helpers


def _ptr(t, name, dtypes=None, nullable=False, numel=None):
    """Pointer of tensor `t` after host-side checks: its dtype, at least
    `numel` elements (the count the shape implies: a shorter tensor would
    make the kernels read or write past its end) and contiguity. Raises
    TypeError / ValueError before any library call. That every tensor lives
    on the GPU is checked afterwards, for all arguments at once
    (_on_device)."""
    if t is None:
        if nullable:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements; the shape needs {numel}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _on_device(**tensors):
    """Every given tensor (None allowed) must be a device tensor."""
    for name, t in tensors.items():
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")


class _Sizes:
    """Element counts the shape implies for each array argument."""

    def __init__(self, shape: Shape):
        B, H, Hkv = shape.batch, shape.num_q_heads, shape.num_kv_heads
        D, ps = shape.head_dim, shape.page_size
        self.q = B * H * D
        self.out = B * H * D
        self.heads = B * H
        self.pool = shape.num_phys_pages * Hkv * ps * D
        self.meta = shape.num_phys_pages * Hkv * 2 * D
        self.block_table = B * shape.max_pages_per_seq
        self.batch = B

    def sel(self, budget):
        return self.heads * max(int(budget), 0)


def _kv_dtypes(shape: Shape):
    return (torch.float32,) if shape.kv_dtype == ENTMAXKV_F32 else (torch.bfloat16, torch.int16)


def _stream(stream, device) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return ctypes.c_void_p(handle)


def _events(events):
    if events is None:
        return None
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(int(e)) for e in events])
    return ctypes.cast(arr, ctypes.c_void_p), arr


def _check(rc: int, where: str):
    if rc != ENTMAXKV_OK:
        raise EntmaxKVError(rc, where)


def entmaxkv_workspace_bytes(shape: Shape, budget_pages: int, which: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib.entmaxkv_workspace_bytes(ctypes.byref(shape), int(budget_pages), int(which),
                                        ctypes.byref(out)), "entmaxkv_workspace_bytes")
    return int(out.value)


def entmaxkv_topk_kernels(shape: Shape, budget_pages: int) -> int:
    """Kernels entmaxkv_decode_topk launches here: 2 (per-head path) or 4."""
    out = ctypes.c_int32(0)
    _check(lib.entmaxkv_topk_kernels(ctypes.byref(shape), int(budget_pages), ctypes.byref(out)),
           "entmaxkv_topk_kernels")
    return int(out.value)


def workspace(shape: Shape, budget_pages: int, which: int, device) -> torch.Tensor:
    """Allocate a workspace tensor of the size the library asks for."""
    n = entmaxkv_workspace_bytes(shape, budget_pages, which)
    return torch.empty(max(n, 1), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------------------
# entry points


def _args_build_page_meta(shape: Shape, k_pool, block_table, seq_lens, meta, stream=None):
    n = _Sizes(shape)
    ptrs = [_ptr(k_pool, "k_pool", _kv_dtypes(shape), numel=n.pool),
            _ptr(block_table, "block_table", (torch.int32,), numel=n.block_table),
            _ptr(seq_lens, "seq_lens", (torch.int32,), numel=n.batch),
            _ptr(meta, "meta", _kv_dtypes(shape), numel=n.meta)]
    _on_device(k_pool=k_pool, block_table=block_table, seq_lens=seq_lens, meta=meta)
    return lib.entmaxkv_build_page_meta, [ctypes.byref(shape), *ptrs,
                                          _stream(stream, k_pool.device), None]


def _args_append(fn, what, shape: Shape, k_pool, block_table, old_lens, new_lens,
                 max_new_tokens, meta, stream=None):
    n = _Sizes(shape)
    ptrs = [_ptr(k_pool, "k_pool", _kv_dtypes(shape), numel=n.pool),
            _ptr(block_table, "block_table", (torch.int32,), numel=n.block_table),
            _ptr(old_lens, "old_lens", (torch.int32,), numel=n.batch),
            _ptr(new_lens, "new_lens", (torch.int32,), numel=n.batch)]
    mp = _ptr(meta, what, _kv_dtypes(shape), numel=n.meta)
    _on_device(k_pool=k_pool, block_table=block_table, old_lens=old_lens, new_lens=new_lens,
               **{what: meta})
    return fn, [ctypes.byref(shape), *ptrs, int(max_new_tokens), mp,
                _stream(stream, k_pool.device), None]


def _args_append_page_meta(shape: Shape, k_pool, block_table, old_lens, new_lens,
                           max_new_tokens, meta, stream=None):
    return _args_append(lib.entmaxkv_append_page_meta, "meta", shape, k_pool, block_table,
                        old_lens, new_lens, max_new_tokens, meta, stream)


def _args_append_page_moments(shape: Shape, k_pool, block_table, old_lens, new_lens,
                              max_new_tokens, moments, stream=None):
    return _args_append(lib.entmaxkv_append_page_moments, "moments", shape, k_pool,
                        block_table, old_lens, new_lens, max_new_tokens, moments, stream)


def _args_build_page_moments(shape: Shape, k_pool, block_table, seq_lens, moments, stream=None):
    n = _Sizes(shape)
    ptrs = [_ptr(k_pool, "k_pool", _kv_dtypes(shape), numel=n.pool),
            _ptr(block_table, "block_table", (torch.int32,), numel=n.block_table),
            _ptr(seq_lens, "seq_lens", (torch.int32,), numel=n.batch),
            _ptr(moments, "moments", _kv_dtypes(shape), numel=n.meta)]
    _on_device(k_pool=k_pool, block_table=block_table, seq_lens=seq_lens, moments=moments)
    return lib.entmaxkv_build_page_moments, [ctypes.byref(shape), *ptrs,
                                             _stream(stream, k_pool.device), None]


def _ws_args(ws, shape, budget, which, device):
    """(pointer, bytes, tensor) of the workspace, allocated when not given."""
    if ws is None:
        ws = workspace(shape, budget, which, device)
    else:
        _ptr(ws, "ws")
        _on_device(ws=ws)
    return ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size(), ws


def _args_gauss_select(shape: Shape, q, moments, block_table, seq_lens, alpha, delta, cap_pages,
                       sel, tau_hat=None, ws=None, stream=None):
    n = _Sizes(shape)
    pq = _ptr(q, "q", (torch.float32,), numel=n.q)
    pm = _ptr(moments, "moments", _kv_dtypes(shape), numel=n.meta)
    pbt = _ptr(block_table, "block_table", (torch.int32,), numel=n.block_table)
    pl = _ptr(seq_lens, "seq_lens", (torch.int32,), numel=n.batch)
    ps_ = _ptr(sel, "sel", (torch.int32,), numel=n.sel(cap_pages))
    pt = _ptr(tau_hat, "tau_hat", (torch.float32,), nullable=True, numel=n.heads)
    _on_device(q=q, moments=moments, block_table=block_table, seq_lens=seq_lens, sel=sel,
               tau_hat=tau_hat)
    pw, nw, ws = _ws_args(ws, shape, cap_pages, ENTMAXKV_WS_GAUSS, q.device)
    return lib.entmaxkv_gauss_select, [
        ctypes.byref(shape), pq, pm, pbt, pl, float(alpha), float(delta), int(cap_pages), ps_,
        pt, pw, nw, _stream(stream, q.device), None], ws


def _args_score_select(shape: Shape, q, meta, block_table, seq_lens, budget_pages, sel,
                       sel_ub=None, ws=None, stream=None):
    n = _Sizes(shape)
    pq = _ptr(q, "q", (torch.float32,), numel=n.q)
    pm = _ptr(meta, "meta", _kv_dtypes(shape), numel=n.meta)
    pbt = _ptr(block_table, "block_table", (torch.int32,), numel=n.block_table)
    pl = _ptr(seq_lens, "seq_lens", (torch.int32,), numel=n.batch)
    ps_ = _ptr(sel, "sel", (torch.int32,), numel=n.sel(budget_pages))
    pu = _ptr(sel_ub, "sel_ub", (torch.float32,), nullable=True, numel=n.sel(budget_pages))
    _on_device(q=q, meta=meta, block_table=block_table, seq_lens=seq_lens, sel=sel,
               sel_ub=sel_ub)
    pw, nw, ws = _ws_args(ws, shape, budget_pages, ENTMAXKV_WS_SELECT, q.device)
    return lib.entmaxkv_score_select, [
        ctypes.byref(shape), pq, pm, pbt, pl, int(budget_pages), ps_, pu, pw, nw,
        _stream(stream, q.device), None], ws


def _args_score_select_noalloc(shape: Shape, q, meta, block_table, seq_lens, budget_pages, sel,
                               sel_ub=None, stream=None):
    n = _Sizes(shape)
    pq = _ptr(q, "q", (torch.float32,), numel=n.q)
    pm = _ptr(meta, "meta", _kv_dtypes(shape), numel=n.meta)
    pbt = _ptr(block_table, "block_table", (torch.int32,), numel=n.block_table)
    pl = _ptr(seq_lens, "seq_lens", (torch.int32,), numel=n.batch)
    ps_ = _ptr(sel, "sel", (torch.int32,), numel=n.sel(budget_pages))
    pu = _ptr(sel_ub, "sel_ub", (torch.float32,), nullable=True, numel=n.sel(budget_pages))
    _on_device(q=q, meta=meta, block_table=block_table, seq_lens=seq_lens, sel=sel,
               sel_ub=sel_ub)
    return lib.entmaxkv_score_select_noalloc, [
        ctypes.byref(shape), pq, pm, pbt, pl, int(budget_pages), ps_, pu,
        _stream(stream, q.device), None]


def _decode_ptrs(shape: Shape, q, k_pool, v_pool, block_table, seq_lens, out, tau, support):
    n = _Sizes(shape)
    return (_ptr(q, "q", (torch.float32,), numel=n.q),
            _ptr(k_pool, "k_pool", _kv_dtypes(shape), numel=n.pool),
            _ptr(v_pool, "v_pool", _kv_dtypes(shape), numel=n.pool),
            _ptr(block_table, "block_table", (torch.int32,), numel=n.block_table),
            _ptr(seq_lens, "seq_lens", (torch.int32,), numel=n.batch),
            _ptr(out, "out", (torch.float32,), numel=n.out),
            _ptr(tau, "tau", (torch.float32,), nullable=True, numel=n.heads),
            _ptr(support, "support", (torch.int32,), nullable=True, numel=n.heads))


def _args_decode_sparse(shape: Shape, q, k_pool, v_pool, block_table, seq_lens, sel,
                        budget_pages, alpha, out, tau=None, support=None, ws=None, stream=None):
    pq, pk, pv, pbt, pl, po, pt, psu = _decode_ptrs(shape, q, k_pool, v_pool, block_table,
                                                     seq_lens, out, tau, support)
    ps_ = _ptr(sel, "sel", (torch.int32,), numel=_Sizes(shape).sel(budget_pages))
    _on_device(q=q, k_pool=k_pool, v_pool=v_pool, block_table=block_table, seq_lens=seq_lens,
               sel=sel, out=out, tau=tau, support=support)
    pw, nw, ws = _ws_args(ws, shape, budget_pages, ENTMAXKV_WS_SPARSE, q.device)
    return lib.entmaxkv_decode_sparse, [
        ctypes.byref(shape), pq, pk, pv, pbt, pl, ps_, int(budget_pages), float(alpha), po, pt,
        psu, pw, nw, _stream(stream, q.device), None], ws


def _args_decode_topk(shape: Shape, q, meta, k_pool, v_pool, block_table, seq_lens,
                      budget_pages, alpha, sel, out, sel_ub=None, tau=None, support=None,
                      ws=None, stream=None):
    pq, pk, pv, pbt, pl, po, pt, psu = _decode_ptrs(shape, q, k_pool, v_pool, block_table,
                                                     seq_lens, out, tau, support)
    n = _Sizes(shape)
    pm = _ptr(meta, "meta", _kv_dtypes(shape), numel=n.meta)
    ps_ = _ptr(sel, "sel", (torch.int32,), numel=n.sel(budget_pages))
    pu = _ptr(sel_ub, "sel_ub", (torch.float32,), nullable=True, numel=n.sel(budget_pages))
    _on_device(q=q, meta=meta, k_pool=k_pool, v_pool=v_pool, block_table=block_table,
               seq_lens=seq_lens, sel=sel, sel_ub=sel_ub, out=out, tau=tau, support=support)
    pw, nw, ws = _ws_args(ws, shape, budget_pages, ENTMAXKV_WS_TOPK, q.device)
    return lib.entmaxkv_decode_topk, [
        ctypes.byref(shape), pq, pm, pk, pv, pbt, pl, int(budget_pages), float(alpha), ps_, pu,
        po, pt, psu, pw, nw, _stream(stream, q.device), None], ws


def _args_decode_full(shape: Shape, q, k_pool, v_pool, block_table, seq_lens, alpha, out,
                      tau=None, support=None, ws=None, stream=None):
    pq, pk, pv, pbt, pl, po, pt, psu = _decode_ptrs(shape, q, k_pool, v_pool, block_table,
                                                     seq_lens, out, tau, support)
    _on_device(q=q, k_pool=k_pool, v_pool=v_pool, block_table=block_table, seq_lens=seq_lens,
               out=out, tau=tau, support=support)
    pw, nw, ws = _ws_args(ws, shape, 0, ENTMAXKV_WS_FULL, q.device)
    return lib.entmaxkv_decode_full, [
        ctypes.byref(shape), pq, pk, pv, pbt, pl, float(alpha), po, pt, psu, pw, nw,
        _stream(stream, q.device), None], ws


def _one_device(**tensors):
    """As _on_device, and all of them on the same device."""
    _on_device(**tensors)
    devices = {t.device for t in tensors.values() if t is not None}
    if len(devices) > 1:
        raise ValueError(f"tensors are on several devices: {sorted(map(str, devices))}")


def _q_dtype(shape: Shape, q) -> int:
    """Query type of the softmax calls: float32, or bfloat16 with a bf16 cache."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch tensor")
    if q.dtype == torch.float32:
        return ENTMAXKV_F32
    if q.dtype == torch.bfloat16 and shape.kv_dtype == ENTMAXKV_BF16:
        return ENTMAXKV_BF16
    raise TypeError(f"q has dtype {q.dtype}; the softmax calls take float32, or bfloat16 with a "
                    "bf16 cache")


def _int32(value) -> int:
    """`value` as an int that the C argument holds (ctypes would wrap it)."""
    value = int(value)
    if not -2**31 <= value < 2**31:
        raise ValueError(f"{value} is beyond int32")
    return value


def _max_tokens(shape: Shape) -> int:
    return shape.max_pages_per_seq * shape.page_size


def entmaxkv_softmax_window_ws(shape: Shape, q_tokens: int, window: int, sinks: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib.entmaxkv_softmax_window_ws(ctypes.byref(shape), _int32(q_tokens), _int32(window),
                                          _int32(sinks), ctypes.byref(out)),
           "entmaxkv_softmax_window_ws")
    return int(out.value)


def entmaxkv_softmax_prefix_ws(shape: Shape, prefix_pages: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib.entmaxkv_softmax_prefix_ws(ctypes.byref(shape), _int32(prefix_pages),
                                          ctypes.byref(out)), "entmaxkv_softmax_prefix_ws")
    return int(out.value)


def entmaxkv_softmax_form(shape: Shape, q_dtype: int, q_tokens: int = 1,
                          window: int = FULL_WINDOW, sinks: int = 0,
                          prefix_pages: int = 0) -> int:
    """ENTMAXKV_FORM_FEW_ROWS or _MANY_ROWS: the form of the attention kernel
    that such a window call (prefix_pages 0) or prefix call runs."""
    out = ctypes.c_int32(0)
    _check(lib.entmaxkv_softmax_form(ctypes.byref(shape), _int32(q_dtype), _int32(q_tokens),
                                     _int32(window), _int32(sinks), _int32(prefix_pages),
                                     ctypes.byref(out)), "entmaxkv_softmax_form")
    return int(out.value)


def _torch_stream(stream, device):
    """The torch stream of a call's `stream` argument, a stream or a handle."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    # (ExternalStream(0) is a new stream, not the null one)
    return torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)


def _given_or_new(ws, nbytes, q, stream):
    """(pointer, bytes, tensor) of a workspace of `nbytes`. One allocated here
    is the allocator's again when the call returns. It is taken on the stream
    that the kernels run on: what that memory held before, and what it holds
    next, follows on the same stream."""
    if ws is None:
        if nbytes == 0:
            return None, 0, None
        on = nullcontext() if stream is None else torch.cuda.stream(_torch_stream(stream, q.device))
        with on:
            ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    else:
        _ptr(ws, "ws")
        _one_device(q=q, ws=ws)
    return ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size(), ws


def _softmax_ptrs(shape: Shape, q, q_tokens, k_pool, v_pool, block_table, seq_lens, out, lse):
    n = _Sizes(shape)
    qd = _q_dtype(shape, q)
    q_tokens = max(int(q_tokens), 0)
    return qd, (_ptr(q, "q", numel=n.q * q_tokens),
                _ptr(k_pool, "k_pool", _kv_dtypes(shape), numel=n.pool),
                _ptr(v_pool, "v_pool", _kv_dtypes(shape), numel=n.pool),
                _ptr(block_table, "block_table", (torch.int32,), numel=n.block_table),
                _ptr(seq_lens, "seq_lens", (torch.int32,), numel=n.batch),
                _ptr(out, "out", (q.dtype,), numel=n.out * q_tokens),
                _ptr(lse, "lse", (torch.float32,), nullable=True, numel=n.heads * q_tokens))


def _args_softmax_window(shape: Shape, q, k_pool, v_pool, block_table, seq_lens, window, sinks,
                         out, lse=None, q_tokens=1, ws=None, stream=None):
    qd, (pq, pk, pv, pbt, pl, po, pe) = _softmax_ptrs(shape, q, q_tokens, k_pool, v_pool,
                                                      block_table, seq_lens, out, lse)
    _one_device(q=q, k_pool=k_pool, v_pool=v_pool, block_table=block_table, seq_lens=seq_lens,
                out=out, lse=lse)
    need = 0 if ws is not None else entmaxkv_softmax_window_ws(shape, q_tokens, window, sinks)
    pw, nw, ws = _given_or_new(ws, need, q, stream)
    return lib.entmaxkv_softmax_window, [
        ctypes.byref(shape), pq, qd, _int32(q_tokens), pk, pv, pbt, pl, _int32(window),
        _int32(sinks), po, pe, pw, nw, _stream(stream, q.device), None], ws


def _args_softmax_prefix(shape: Shape, q, k_pool, v_pool, prefix_table, prefix_pages,
                         block_table, seq_lens, out, lse=None, ws=None, stream=None):
    qd, (pq, pk, pv, pbt, pl, po, pe) = _softmax_ptrs(shape, q, 1, k_pool, v_pool, block_table,
                                                      seq_lens, out, lse)
    ppt = _ptr(prefix_table, "prefix_table", (torch.int32,), numel=max(int(prefix_pages), 0))
    _one_device(q=q, k_pool=k_pool, v_pool=v_pool, prefix_table=prefix_table,
                block_table=block_table, seq_lens=seq_lens, out=out, lse=lse)
    need = 0 if ws is not None else entmaxkv_softmax_prefix_ws(shape, prefix_pages)
    pw, nw, ws = _given_or_new(ws, need, q, stream)
    return lib.entmaxkv_softmax_prefix, [
        ctypes.byref(shape), pq, qd, pk, pv, ppt, _int32(prefix_pages), pbt, pl, po, pe, pw, nw,
        _stream(stream, q.device), None], ws


def _args_accumulate_weights(shape: Shape, q, k_pool, block_table, seq_lens, alpha, tau, decay,
                             weights_in, weights_out, window=FULL_WINDOW, sinks=0, stream=None):
    n = _Sizes(shape)
    cells = shape.batch * shape.num_kv_heads * _max_tokens(shape)
    qd = _q_dtype(shape, q)
    pq = _ptr(q, "q", numel=n.q)
    pk = _ptr(k_pool, "k_pool", _kv_dtypes(shape), numel=n.pool)
    pbt = _ptr(block_table, "block_table", (torch.int32,), numel=n.block_table)
    pl = _ptr(seq_lens, "seq_lens", (torch.int32,), numel=n.batch)
    pt = _ptr(tau, "tau", (torch.float32,), numel=n.heads)
    pi = _ptr(weights_in, "weights_in", (torch.float32,), nullable=True, numel=cells)
    po = _ptr(weights_out, "weights_out", (torch.float32,), numel=cells)
    _one_device(q=q, k_pool=k_pool, block_table=block_table, seq_lens=seq_lens, tau=tau,
                weights_in=weights_in, weights_out=weights_out)
    return lib.entmaxkv_accumulate_weights, [
        ctypes.byref(shape), pq, qd, pk, pbt, pl, float(alpha), pt, _int32(window),
        _int32(sinks), float(decay), pi, po, _stream(stream, q.device), None]


def _args_evict(shape: Shape, k_pool, v_pool, block_table, seq_lens, weights, keep, sinks, recent,
                new_table, kept, new_lens, new_weights=None, stream=None):
    n = _Sizes(shape)
    rows = shape.batch * shape.num_kv_heads
    cells = rows * _max_tokens(shape)
    ptrs = [_ptr(k_pool, "k_pool", _kv_dtypes(shape), numel=n.pool),
            _ptr(v_pool, "v_pool", _kv_dtypes(shape), numel=n.pool),
            _ptr(block_table, "block_table", (torch.int32,), numel=n.block_table),
            _ptr(seq_lens, "seq_lens", (torch.int32,), numel=n.batch),
            _ptr(weights, "weights", (torch.float32,), numel=cells)]
    outs = [_ptr(new_table, "new_table", (torch.int32,), numel=n.block_table),
            _ptr(kept, "kept", (torch.int32,), numel=rows * max(int(keep), 0)),
            _ptr(new_lens, "new_lens", (torch.int32,), numel=n.batch),
            _ptr(new_weights, "new_weights", (torch.float32,), nullable=True, numel=cells)]
    _one_device(k_pool=k_pool, v_pool=v_pool, block_table=block_table, seq_lens=seq_lens,
                weights=weights, new_table=new_table, kept=kept, new_lens=new_lens,
                new_weights=new_weights)
    return lib.entmaxkv_evict, [ctypes.byref(shape), *ptrs, _int32(keep), _int32(sinks),
                                _int32(recent), *outs, _stream(stream, k_pool.device), None]


def _args_plan_tokens(shape: Shape, seq_lens, new_tokens, free_pages, free_count, block_table,
                      new_lens, token_starts, positions, slots, free_left, stream=None):
    n = _Sizes(shape)
    i32 = (torch.int32,)
    tokens = _tensor(slots, "slots").numel()
    capacity = 0 if free_pages is None else _tensor(free_pages, "free_pages").numel()
    ins = [_ptr(seq_lens, "seq_lens", i32, numel=n.batch),
           _ptr(new_tokens, "new_tokens", i32, numel=n.batch)]
    pages = _ptr(free_pages, "free_pages", i32, nullable=True)
    outs = [_ptr(free_count, "free_count", i32, numel=1),
            _ptr(block_table, "block_table", i32, numel=n.block_table),
            _ptr(new_lens, "new_lens", i32, numel=n.batch),
            _ptr(token_starts, "token_starts", i32, numel=n.batch + 1),
            _ptr(positions, "positions", i32, numel=tokens),
            _ptr(slots, "slots", i32), _ptr(free_left, "free_left", i32, numel=1)]
    _one_device(seq_lens=seq_lens, new_tokens=new_tokens, free_pages=free_pages,
                free_count=free_count, block_table=block_table, new_lens=new_lens,
                token_starts=token_starts, positions=positions, slots=slots, free_left=free_left)
    return lib.entmaxkv_plan_tokens, [ctypes.byref(shape), _int32(tokens), *ins, pages,
                                      _int32(capacity), *outs, _stream(stream, slots.device),
                                      None]


def _tensor(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    return t


_DTYPES = {torch.float32: ENTMAXKV_F32, torch.bfloat16: ENTMAXKV_BF16}


def _token_rows(t, name, heads, dim, tokens, dtype):
    """(pointer, values from a token to the next) of [tokens, heads, dim] rows,
    dense within a token."""
    _tensor(t, name)
    if t.dtype != dtype or dtype not in _DTYPES:
        raise TypeError(f"{name} has dtype {t.dtype}; q, k and v are all float32 or all bfloat16")
    if tuple(t.shape) != (tokens, heads, dim):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(tokens, heads, dim)}")
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != dim):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    # one token's stride may be anything; it is never used
    return ctypes.c_void_p(t.data_ptr()), t.stride(0) if tokens > 1 else heads * dim


def _args_append_kv(shape: Shape, q, k, v, positions, slots, q_out, k_pool, v_pool, freqs=None,
                    pair_axis=None, interleaved=False, q_weight=None, k_weight=None, eps=1e-6,
                    q_scale=1.0, stream=None):
    n = _Sizes(shape)
    tokens, D = _tensor(q, "q").shape[0], shape.head_dim
    pq, sq = _token_rows(q, "q", shape.num_q_heads, D, tokens, q.dtype)
    pk, sk = _token_rows(k, "k", shape.num_kv_heads, D, tokens, q.dtype)
    pv, sv = _token_rows(v, "v", shape.num_kv_heads, D, tokens, q.dtype)
    if _tensor(q_out, "q_out").dtype not in _DTYPES:
        raise TypeError(f"q_out has dtype {q_out.dtype}, expected float32 or bfloat16")
    half = 0 if freqs is None else _tensor(freqs, "freqs").numel()
    axes = 1
    if positions is not None:
        axes = 1 if _tensor(positions, "positions").dim() == 1 else positions.shape[0]
    if axes > 1 and half and pair_axis is None:
        raise ValueError("pair_axis is required with several axes")
    i32, f32 = (torch.int32,), (torch.float32,)
    pos = _ptr(positions, "positions", i32, nullable=half == 0, numel=axes * tokens)
    rest = [_ptr(slots, "slots", i32, numel=tokens),
            _ptr(freqs, "freqs", (torch.float64,), nullable=True),
            _ptr(pair_axis, "pair_axis", i32, nullable=True, numel=half),
            _ptr(q_weight, "q_weight", f32, nullable=True, numel=D),
            _ptr(k_weight, "k_weight", f32, nullable=True, numel=D),
            _ptr(q_out, "q_out", numel=tokens * shape.num_q_heads * D),
            _ptr(k_pool, "k_pool", _kv_dtypes(shape), numel=n.pool),
            _ptr(v_pool, "v_pool", _kv_dtypes(shape), numel=n.pool)]
    _one_device(q=q, k=k, v=v, positions=positions, slots=slots, freqs=freqs, pair_axis=pair_axis,
                q_weight=q_weight, k_weight=k_weight, q_out=q_out, k_pool=k_pool, v_pool=v_pool)
    a = Append(_int32(tokens), _DTYPES[q.dtype], _DTYPES[q_out.dtype], 2 * half, axes,
               int(bool(interleaved)), sq, sk, sv, float(eps), float(q_scale))
    return lib.entmaxkv_append_kv, [ctypes.byref(shape), ctypes.byref(a), pq, pk, pv, pos, *rest,
                                    _stream(stream, q.device), None]


def entmaxkv_entmax_chunk_ws(shape: Shape, num_tokens: int, alpha: float) -> int:
    out = ctypes.c_size_t(0)
    _check(lib.entmaxkv_entmax_chunk_ws(ctypes.byref(shape), _int32(num_tokens), float(alpha),
                                        ctypes.byref(out)), "entmaxkv_entmax_chunk_ws")
    return int(out.value)


def _args_entmax_chunk(shape: Shape, q, token_starts, k_pool, v_pool, block_table, seq_lens, alpha,
                       out, tau=None, support=None, ws=None, stream=None):
    n = _Sizes(shape)
    qd = _q_dtype(shape, q)
    H, D = shape.num_q_heads, shape.head_dim
    if q.dim() != 3 or tuple(q.shape[1:]) != (H, D):
        raise ValueError(f"q has shape {tuple(q.shape)}, expected (tokens, {H}, {D})")
    tokens = q.shape[0]
    ptrs = [_ptr(token_starts, "token_starts", (torch.int32,), numel=n.batch + 1),
            _ptr(k_pool, "k_pool", _kv_dtypes(shape), numel=n.pool),
            _ptr(v_pool, "v_pool", _kv_dtypes(shape), numel=n.pool),
            _ptr(block_table, "block_table", (torch.int32,), numel=n.block_table),
            _ptr(seq_lens, "seq_lens", (torch.int32,), numel=n.batch)]
    outs = [_ptr(out, "out", (q.dtype,), numel=tokens * H * D),
            _ptr(tau, "tau", (torch.float32,), nullable=True, numel=tokens * H),
            _ptr(support, "support", (torch.int32,), nullable=True, numel=tokens * H)]
    pq = _ptr(q, "q")
    _one_device(q=q, token_starts=token_starts, k_pool=k_pool, v_pool=v_pool,
                block_table=block_table, seq_lens=seq_lens, out=out, tau=tau, support=support)
    need = 0 if ws is not None else entmaxkv_entmax_chunk_ws(shape, tokens, alpha)
    pw, nw, ws = _given_or_new(ws, need, q, stream)
    return lib.entmaxkv_entmax_chunk, [
        ctypes.byref(shape), pq, qd, _int32(tokens), *ptrs, float(alpha), *outs, pw, nw,
        _stream(stream, q.device), None], ws


def _run(name, fn, args, events):
    if events is not None:
        ev = _events(events)
        args = list(args)
        args[-1] = ev[0]
    _check(fn(*args), name)


def _run_on(device, name, fn, args, events):
    """_run with `device` as the current one (the library launches there)."""
    if device.index is None or device.index == torch.cuda.current_device():
        _run(name, fn, args, events)
    else:
        with torch.cuda.device(device):
            _run(name, fn, args, events)


def entmaxkv_build_page_meta(shape: Shape, k_pool, block_table, seq_lens, meta, stream=None,
                             events=None):
    fn, args = _args_build_page_meta(shape, k_pool, block_table, seq_lens, meta, stream)
    _run("entmaxkv_build_page_meta", fn, args, events)


def entmaxkv_append_page_meta(shape: Shape, k_pool, block_table, old_lens, new_lens,
                              max_new_tokens, meta, stream=None, events=None):
    fn, args = _args_append_page_meta(shape, k_pool, block_table, old_lens, new_lens,
                                      max_new_tokens, meta, stream)
    _run("entmaxkv_append_page_meta", fn, args, events)


def entmaxkv_build_page_moments(shape: Shape, k_pool, block_table, seq_lens, moments,
                                stream=None, events=None):
    fn, args = _args_build_page_moments(shape, k_pool, block_table, seq_lens, moments, stream)
    _run("entmaxkv_build_page_moments", fn, args, events)


def entmaxkv_append_page_moments(shape: Shape, k_pool, block_table, old_lens, new_lens,
                                 max_new_tokens, moments, stream=None, events=None):
    fn, args = _args_append_page_moments(shape, k_pool, block_table, old_lens, new_lens,
                                         max_new_tokens, moments, stream)
    _run("entmaxkv_append_page_moments", fn, args, events)


def entmaxkv_gauss_select(shape: Shape, q, moments, block_table, seq_lens, alpha, delta,
                          cap_pages, sel, tau_hat=None, ws=None, stream=None, events=None):
    fn, args, _ = _args_gauss_select(shape, q, moments, block_table, seq_lens, alpha, delta,
                                     cap_pages, sel, tau_hat, ws, stream)
    _run("entmaxkv_gauss_select", fn, args, events)


def entmaxkv_score_select(shape: Shape, q, meta, block_table, seq_lens, budget_pages, sel,
                          sel_ub=None, ws=None, stream=None, events=None):
    fn, args, _ = _args_score_select(shape, q, meta, block_table, seq_lens, budget_pages, sel,
                                     sel_ub, ws, stream)
    _run("entmaxkv_score_select", fn, args, events)


def entmaxkv_score_select_noalloc(shape: Shape, q, meta, block_table, seq_lens, budget_pages,
                                  sel, sel_ub=None, stream=None, events=None):
    """entmaxkv_score_select with the library's static scratch in place of a
    workspace (allocates nothing; calls overlapping on one GPU race)."""
    fn, args = _args_score_select_noalloc(shape, q, meta, block_table, seq_lens, budget_pages,
                                          sel, sel_ub, stream)
    _run("entmaxkv_score_select_noalloc", fn, args, events)


def entmaxkv_decode_sparse(shape: Shape, q, k_pool, v_pool, block_table, seq_lens, sel,
                           budget_pages, alpha, out, tau=None, support=None, ws=None,
                           stream=None, events=None):
    fn, args, _ = _args_decode_sparse(shape, q, k_pool, v_pool, block_table, seq_lens, sel,
                                      budget_pages, alpha, out, tau, support, ws, stream)
    _run("entmaxkv_decode_sparse", fn, args, events)


def entmaxkv_decode_topk(shape: Shape, q, meta, k_pool, v_pool, block_table, seq_lens,
                         budget_pages, alpha, sel, out, sel_ub=None, tau=None, support=None,
                         ws=None, stream=None, events=None):
    """Bounds, top-k selection and sparse decode in one call (sel is written)."""
    fn, args, _ = _args_decode_topk(shape, q, meta, k_pool, v_pool, block_table, seq_lens,
                                    budget_pages, alpha, sel, out, sel_ub, tau, support, ws,
                                    stream)
    _run("entmaxkv_decode_topk", fn, args, events)


def entmaxkv_decode_full(shape: Shape, q, k_pool, v_pool, block_table, seq_lens, alpha, out,
                         tau=None, support=None, ws=None, stream=None, events=None):
    fn, args, _ = _args_decode_full(shape, q, k_pool, v_pool, block_table, seq_lens, alpha, out,
                                    tau, support, ws, stream)
    _run("entmaxkv_decode_full", fn, args, events)


def entmaxkv_softmax_window(shape: Shape, q, k_pool, v_pool, block_table, seq_lens, window, sinks,
                            out, lse=None, q_tokens=1, ws=None, stream=None, events=None):
    """Softmax attention of every sequence's last q_tokens tokens over a
    window and the first `sinks` tokens. q and out: [batch, q_tokens,
    num_q_heads, head_dim], float32 or (with a bf16 cache) bfloat16; window:
    FULL_WINDOW for all tokens."""
    fn, args, _ = _args_softmax_window(shape, q, k_pool, v_pool, block_table, seq_lens, window,
                                       sinks, out, lse, q_tokens, ws, stream)
    _run_on(q.device, "entmaxkv_softmax_window", fn, args, events)


def entmaxkv_softmax_prefix(shape: Shape, q, k_pool, v_pool, prefix_table, prefix_pages,
                            block_table, seq_lens, out, lse=None, ws=None, stream=None,
                            events=None):
    """Softmax attention of one token per sequence over sequences that share
    their first prefix_pages pages, listed in prefix_table."""
    fn, args, _ = _args_softmax_prefix(shape, q, k_pool, v_pool, prefix_table, prefix_pages,
                                       block_table, seq_lens, out, lse, ws, stream)
    _run_on(q.device, "entmaxkv_softmax_prefix", fn, args, events)


def entmaxkv_accumulate_weights(shape: Shape, q, k_pool, block_table, seq_lens, alpha, tau, decay,
                                weights_in, weights_out, window=FULL_WINDOW, sinks=0, stream=None,
                                events=None):
    """weights_out = decay * weights_in (None: 0) + every cached token's
    attention weight, summed over the query heads of its KV head. tau: the lse
    of a softmax decode (alpha 1) or the tau of an alpha-entmax decode."""
    fn, args = _args_accumulate_weights(shape, q, k_pool, block_table, seq_lens, alpha, tau,
                                        decay, weights_in, weights_out, window, sinks, stream)
    _run_on(q.device, "entmaxkv_accumulate_weights", fn, args, events)


def entmaxkv_evict(shape: Shape, k_pool, v_pool, block_table, seq_lens, weights, keep, sinks,
                   recent, new_table, kept, new_lens, new_weights=None, stream=None, events=None):
    """Keeps `keep` tokens of every (sequence, KV head) by accumulated weight
    and copies them to the pages of new_table."""
    fn, args = _args_evict(shape, k_pool, v_pool, block_table, seq_lens, weights, keep, sinks,
                           recent, new_table, kept, new_lens, new_weights, stream)
    _run_on(k_pool.device, "entmaxkv_evict", fn, args, events)


def entmaxkv_plan_tokens(shape: Shape, seq_lens, new_tokens, free_pages, free_count, block_table,
                         new_lens, token_starts, positions, slots, free_left, stream=None,
                         events=None):
    """Pages of the free list for new_tokens more tokens of every sequence;
    row, position and slot of each. slots' length is the rows of the step."""
    fn, args = _args_plan_tokens(shape, seq_lens, new_tokens, free_pages, free_count, block_table,
                                 new_lens, token_starts, positions, slots, free_left, stream)
    _run_on(slots.device, "entmaxkv_plan_tokens", fn, args, events)


def entmaxkv_append_kv(shape: Shape, q, k, v, positions, slots, q_out, k_pool, v_pool, freqs=None,
                       pair_axis=None, interleaved=False, q_weight=None, k_weight=None, eps=1e-6,
                       q_scale=1.0, stream=None, events=None):
    """Norm and rotation of the heads of q and k; queries to q_out, keys and
    values to their slots. q, k, v: [tokens, heads, head_dim], slices of one
    tensor allowed; positions: [tokens] or [axes, tokens]; freqs: float64, half
    as many as the values rotated (None: no rotation)."""
    fn, args = _args_append_kv(shape, q, k, v, positions, slots, q_out, k_pool, v_pool, freqs,
                               pair_axis, interleaved, q_weight, k_weight, eps, q_scale, stream)
    _run_on(q.device, "entmaxkv_append_kv", fn, args, events)


def entmaxkv_entmax_chunk(shape: Shape, q, token_starts, k_pool, v_pool, block_table, seq_lens,
                          alpha, out, tau=None, support=None, ws=None, stream=None, events=None):
    """alpha-entmax attention of the new tokens of a ragged batch: sequence b's
    are rows token_starts[b] .. token_starts[b + 1] - 1 of q and out, [tokens,
    num_q_heads, head_dim], its last ones in the cache."""
    fn, args, _ = _args_entmax_chunk(shape, q, token_starts, k_pool, v_pool, block_table, seq_lens,
                                     alpha, out, tau, support, ws, stream)
    _run_on(q.device, "entmaxkv_entmax_chunk", fn, args, events)


class Prepared:
    """An entry point with its arguments marshalled once, for tight loops.
    The tensors must stay alive and unchanged in place while it is used.

        call = Prepared("decode_full", shape, q, k, v, bt, lens, 1.5, out, ws=ws)
        call()                 # or call(events=[e0, e1, e2, e3])
    """

    _makers = {"build_page_meta": _args_build_page_meta,
               "append_page_meta": _args_append_page_meta, "score_select": _args_score_select,
               "decode_sparse": _args_decode_sparse, "decode_topk": _args_decode_topk,
               "decode_full": _args_decode_full,
               "build_page_moments": _args_build_page_moments,
               "append_page_moments": _args_append_page_moments,
               "gauss_select": _args_gauss_select,
               "softmax_window": _args_softmax_window,
               "softmax_prefix": _args_softmax_prefix,
               "accumulate_weights": _args_accumulate_weights, "evict": _args_evict,
               "plan_tokens": _args_plan_tokens, "append_kv": _args_append_kv,
               "entmax_chunk": _args_entmax_chunk}

    def __init__(self, name: str, *args, **kwargs):
        r = Prepared._makers[name](*args, **kwargs)
        self.name = "entmaxkv_" + name
        self.fn, self.args = r[0], r[1]
        self.keep = (args, kwargs, r[2:] if len(r) > 2 else ())  # keep tensors alive
        tensors = [t for t in (*args, *kwargs.values()) if isinstance(t, torch.Tensor)]
        # the device that the kernels are launched on (None: there is no other)
        self.device = tensors[0].device.index if torch.cuda.device_count() > 1 else None
        self._ev_cache = {}

    def __call__(self, events=None):
        if self.device is not None and self.device != torch.cuda.current_device():
            with torch.cuda.device(self.device):
                return self(events)
        if events is None:
            rc = self.fn(*self.args)
        else:
            key = tuple(events)
            ev = self._ev_cache.get(key)
            if ev is None:
                ev = self._ev_cache[key] = _events(events)
            self.args[-1] = ev[0]
            rc = self.fn(*self.args)
            self.args[-1] = None
        if rc != ENTMAXKV_OK:
            raise EntmaxKVError(rc, self.name)


# ---------------------------------------------------------------------------
# HIP events for per-kernel timing (plumbing around hipEvent_t)


class HipEvents:
    """A set of timing-enabled hipEvent_t handles, passed as `events=`."""

    _hip = None

    def __init__(self, n: int):
        if HipEvents._hip is None:
            h = ctypes.CDLL("libamdhip64.so")
            h.hipEventCreate.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
            h.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p,
                                              ctypes.c_void_p]
            h.hipEventSynchronize.argtypes = [ctypes.c_void_p]
            h.hipEventDestroy.argtypes = [ctypes.c_void_p]
            h.hipEventRecord.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
            HipEvents._hip = h
        self.handles = []
        for _ in range(n):
            e = ctypes.c_void_p()
            rc = HipEvents._hip.hipEventCreate(ctypes.byref(e))
            if rc != 0:
                raise RuntimeError(f"hipEventCreate failed ({rc})")
            self.handles.append(e.value)

    def record(self, i: int, stream) -> None:
        """Record event i on `stream` (a torch stream or a raw handle)."""
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        rc = HipEvents._hip.hipEventRecord(ctypes.c_void_p(self.handles[i]), ctypes.c_void_p(handle))
        if rc != 0:
            raise RuntimeError(f"hipEventRecord failed ({rc})")

    def __len__(self):
        return len(self.handles)

    def __iter__(self):
        return iter(self.handles)

    def elapsed_ms(self, i: int, j: int) -> float:
        out = ctypes.c_float()
        HipEvents._hip.hipEventSynchronize(ctypes.c_void_p(self.handles[j]))
        rc = HipEvents._hip.hipEventElapsedTime(ctypes.byref(out), ctypes.c_void_p(self.handles[i]),
                                                ctypes.c_void_p(self.handles[j]))
        if rc != 0:
            raise RuntimeError(f"hipEventElapsedTime failed ({rc})")
        return float(out.value)

    def close(self):
        for e in self.handles:
            HipEvents._hip.hipEventDestroy(ctypes.c_void_p(e))
        self.handles = []
