"""Decode benchmark on one MI355X: sparse vs full-cache alpha-entmax decode.

    python bench.py [--gpus 1] [--steps K] [--warmup W] [--workload long_128k]

One step is one pass of the decode hot path over the whole batch (every
sequence, every query head): page bounds + top-k selection, sparse decode
over the selected pages, and the full-cache decode on the same inputs. The
page boxes are built once before timing (they are per-page state, written
when a page is filled) and timed on their own.

Inputs are generated on the host, uploaded, and resident in HBM before any
timing. Each timed step is preceded by an untimed 1 GiB write that evicts the
on-chip caches (L2 + MALL), so the step reads HBM, not a warm cache
(--flush write_read also reads a second 1 GiB buffer afterwards, so the
caches hold clean lines of unrelated data; the times are the same). In the
timed pass HIP events mark only the call boundaries (step start, end of the
sparse path, end of the full path); a second pass over the same steps has
the library record events around every kernel, which gives the per-kernel
durations behind the roofline figures. Prints one JSON line.

The CPU baseline is the float64 oracle run on this host's cores over a
bounded sample of (sequence, query head) decodes of the same workload,
scaled to steps/s.
"""
from __future__ import annotations

import argparse
import hashlib
import json
import math
import multiprocessing as mp
import os
import re
import sys
import time

import numpy as np

ROOT = os.path.dirname(os.path.abspath(__file__))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from sparse_long_context_page_amd import synth  # noqa: E402

METRIC = ("decode steps/s + achieved HBM GB/s (% of peak), sparse vs full entmax, "
          "32K–512K")
PEAK_HBM_GBPS = 8000.0
# kernels of the sparse path (entmaxkv_decode_topk) on its per-head path and
# on its four-kernel path, then those of the full-cache path
SPARSE_KERNELS_HEAD = ["bounds", "select_decode"]
SPARSE_KERNELS_HEAD_SPLIT = ["bounds", "select_score", "tau_pv_sparse"]
SPARSE_KERNELS_SPLIT = ["bounds", "select", "score_sparse", "tau_pv_sparse"]
FULL_KERNELS = ["score_full", "tau_pv_full"]
KERNEL_SOURCES = ["common.hpp", "launch.hpp", "mfma.hpp", "select.hip", "select_impl.hpp",
                  "decode_impl.hpp", "decode_bf16.hip", "decode_f32.hip", "head_impl.hpp",
                  "head_bf16.hip", "meta.hip", "api.hip"]


def sparse_kernels(E, shape, budget) -> list:
    """Names of the kernels entmaxkv_decode_topk runs at this shape and budget."""
    n = E.entmaxkv_topk_kernels(shape, budget)
    return {2: SPARSE_KERNELS_HEAD, 3: SPARSE_KERNELS_HEAD_SPLIT}.get(n, SPARSE_KERNELS_SPLIT)


# ---------------------------------------------------------------------------
# byte accounting (algorithmic bytes: what the method itself must move)


def kv_elem_bytes(w) -> int:
    return 2 if w.kv_dtype == "bf16" else 4


def union_pages(sel: np.ndarray, G: int) -> np.ndarray:
    """Distinct selected pages per (sequence, KV head): [B, H_kv]."""
    B, H, _ = sel.shape
    out = np.zeros((B, H // G), dtype=np.int64)
    for b in range(B):
        for g in range(H // G):
            s = sel[b, g * G:(g + 1) * G].ravel()
            out[b, g] = len(np.unique(s[s >= 0]))
    return out


def algorithmic_bytes(w, lens: np.ndarray, budget: int, sel: np.ndarray, sup_sparse: np.ndarray,
                      sup_full: np.ndarray) -> dict:
    """Per-kernel algorithmic bytes of one step. Workspace traffic (bounds,
    candidate lists) is implementation overhead and is not counted."""
    s = kv_elem_bytes(w)
    B, H, Hkv, D, ps = w.batch, w.num_q_heads, w.num_kv_heads, w.head_dim, w.page_size
    G = H // Hkv
    P = (lens + ps - 1) // ps
    q_b = B * H * D * 4
    out_b = B * H * D * 4
    bt_b = int(P.sum()) * 4
    meta_b = int(P.sum()) * Hkv * 2 * D * s
    k_full_b = int(lens.sum()) * Hkv * D * s
    up = union_pages(sel, G)
    k_sel_b = int(up.sum()) * ps * D * s
    v_sup_sparse = int(sup_sparse.sum()) * D * s
    v_sup_full = int(sup_full.sum()) * D * s
    sel_b = B * H * budget * 4
    return {
        "bounds": meta_b + q_b + bt_b,
        "select": sel_b,
        "score_sparse": k_sel_b + q_b + sel_b + bt_b,
        "tau_pv_sparse": v_sup_sparse + out_b,
        # the per-head kernel: selection written, K of the union pages (each
        # page counted once per KV head, as above), V of the support, outputs
        "select_decode": sel_b + k_sel_b + q_b + bt_b + v_sup_sparse + out_b,
        # its split form: selection, K of the union pages (the threshold
        # kernel then reads the V rows)
        "select_score": sel_b + k_sel_b + q_b + bt_b,
        # what the per-head kernel requests: each selected page once per head
        "_k_per_head": int((sel >= 0).sum()) * ps * D * s,
        "score_full": k_full_b + q_b + bt_b,
        "tau_pv_full": v_sup_full + out_b,
        "_meta_build": int(lens.sum()) * Hkv * D * s + meta_b,
        "_union_pages": int(up.sum()),
        "_union_fraction": float(up.sum()) / float(B * H * min(budget, int(P.max()))),
        # the literal accounting (every V row of the touched pages read, as a
        # decode without the p > 0 skip would): sparse = boxes + K and V of
        # the union pages; full = all of K and V
        "_sparse_all_kv": meta_b + 2 * k_sel_b + 2 * q_b + out_b + sel_b + 2 * bt_b,
        "_full_all_kv": 2 * k_full_b + q_b + out_b + bt_b,
    }


def kernel_source_hash() -> str:
    h = hashlib.sha256()
    for f in KERNEL_SOURCES:
        with open(os.path.join(ROOT, "sparse_long_context_page_amd", "csrc", f), "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()[:16]


def profile_name(w, alpha, budget) -> str:
    """Name of the committed profile summaries of a workload (and, for the
    sweep, of its alpha / budget cell)."""
    if len(w.alphas) > 1 or len(w.budgets) > 1:
        return f"{w.name}_a{alpha}_b{budget}"
    return w.name


def counter_traffic(kernel: str, profile: str):
    """HBM bytes per launch of `kernel` from the committed rocprofv3 counter
    summary of this workload, or None if there is none or the kernel
    sources changed since it was taken."""
    path = os.path.join(ROOT, "profiles", f"counters_{profile}.txt")
    if not os.path.exists(path):
        return None
    text = open(path).read()
    m = re.search(r"source_hash:\s*(\w+)", text)
    t = re.search(r"hbm_bytes_per_launch\[" + re.escape(kernel) + r"\]:\s*([0-9.eE+]+)", text)
    if not m or not t or m.group(1) != kernel_source_hash():
        return None
    return float(t.group(1))


# ---------------------------------------------------------------------------
# CPU baseline: the oracle on the host's cores over sampled heads

_ORACLE_STATE = {}


def _oracle_head(args):
    from oracle import entmax_oracle as O
    b, h, budget, alpha = args
    inp = _ORACLE_STATE["inp"]
    w = inp["workload"]
    g = h // (w.num_q_heads // w.num_kv_heads)
    seq_meta = _ORACLE_STATE["seq_meta"][(b, g)]
    t0 = time.perf_counter()
    _, key, sel = O.select_for_head(inp, b, h, budget, seq_meta=seq_meta)
    sp = O.decode_sparse(inp, b, h, alpha, sel)
    fu = O.decode_full(inp, b, h, alpha)
    dt = time.perf_counter() - t0
    near = sorted(O.near_tie_pages(key, budget))  # (outside the timed region)
    return b, h, dt, sel, sp.out, fu.out, near


ONE_CORE_WORKLOADS = ("tiny_4k_f32", "extreme_512k", "extreme_1m")  # also timed on one core
ONE_CORE_HEADS = 4


def cpu_baseline(inp, budget, alpha, n_heads: int, seed: int = 0):
    """Time the oracle's step (bounds+selection, sparse decode, full decode)
    on a sample of (sequence, head) pairs; page boxes are built before timing,
    as on the GPU."""
    from oracle import entmax_oracle as O
    w = inp["workload"]
    rng = np.random.default_rng(seed)
    pairs = [(int(b), int(h)) for b, h in zip(rng.integers(0, w.batch, n_heads),
                                               rng.integers(0, w.num_q_heads, n_heads))]
    G = w.num_q_heads // w.num_kv_heads
    seq_meta = {}
    for b, h in pairs:
        g = h // G
        if (b, g) not in seq_meta:
            seq_meta[(b, g)] = O.sequence_metadata(inp["k_pool"], inp["block_table"][b],
                                                   inp["seq_lens"][b], w.page_size, g, w.kv_dtype)
    _ORACLE_STATE["inp"] = inp
    _ORACLE_STATE["seq_meta"] = seq_meta
    cores = len(os.sched_getaffinity(0))
    workers = min(cores, n_heads)
    t0 = time.perf_counter()
    ctx = mp.get_context("fork")
    with ctx.Pool(workers, initializer=_pin_blas) as pool:
        results = pool.map(_oracle_head, [(b, h, budget, alpha) for b, h in pairs])
    wall = time.perf_counter() - t0
    step_s = wall * (w.batch * w.num_q_heads) / n_heads
    one_core = None
    if w.name in ONE_CORE_WORKLOADS:
        # the same work on one core, in this process, on the first few pairs
        from threadpoolctl import threadpool_limits
        n1 = min(ONE_CORE_HEADS, n_heads)
        with threadpool_limits(1):
            t1 = time.perf_counter()
            for b, h in pairs[:n1]:
                _oracle_head((b, h, budget, alpha))
            wall1 = time.perf_counter() - t1
        one_core = {"value": 1.0 / (wall1 * (w.batch * w.num_q_heads) / n1), "unit": "steps/s",
                    "cores": 1, "sample": f"{n1} (sequence, head) pairs, scaled per step"}
    return {
        "value": 1.0 / step_s,
        "unit": "steps/s",
        "cores": workers,
        "kind": "oracle",
        "sample": (f"{n_heads} random (sequence, head) pairs of {w.name}: bounds+top-{budget} "
                   f"selection, sparse and full fp64 decode each; wall {wall:.2f} s on {workers} "
                   f"processes, scaled by {w.batch * w.num_q_heads}/{n_heads} heads per step; "
                   f"page boxes prebuilt"),
        "one_core": one_core,
        "_results": results,
    }


def _pin_blas():
    for k in ("OMP_NUM_THREADS", "OPENBLAS_NUM_THREADS", "MKL_NUM_THREADS"):
        os.environ[k] = "1"


# ---------------------------------------------------------------------------


def contained(sup_s, sup_f, tau_s, tau_f, rel: float = 1e-6) -> np.ndarray:
    """Per (sequence, head): did the selection contain the full-cache support?
    When it does, the sparse problem is the full one restricted to a superset
    of the support, so tau and the support size come out the same; a missing
    support token lowers tau and the support size."""
    return (sup_s == sup_f) & (np.abs(tau_s - tau_f) <= rel * np.maximum(1.0, np.abs(tau_f)))


def containment_report(args):
    """Fraction of trials (one trial = one (sequence, query head) decode) whose
    selected pages contain the full-cache support, for every (alpha, budget)
    cell of the workload's sweep; sampled trials are checked against the
    oracle's support pages."""
    import torch
    from oracle import entmax_oracle as O
    from sparse_long_context_page_amd import entmaxkv as E
    w = synth.WORKLOADS[args.workload]
    log = lambda m: (sys.stderr.write(f"[report] {m}\n"), sys.stderr.flush())
    inp = synth.generate(w, synth.WORKLOAD_SEEDS[w.name])
    log(f"generated {w.name}")
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    kv_t = torch.bfloat16 if w.kv_dtype == "bf16" else torch.float32

    def pool(a):
        if w.kv_dtype == "bf16":
            return torch.from_numpy(a.view(np.int16)).to(dev).view(torch.bfloat16)
        return torch.from_numpy(a).to(dev)

    q = torch.from_numpy(inp["q"]).to(dev)
    k, v = pool(inp["k_pool"]), pool(inp["v_pool"])
    bt = torch.from_numpy(inp["block_table"]).to(dev)
    lens = torch.from_numpy(inp["seq_lens"]).to(dev)
    shape = E.make_shape(w.batch, w.num_q_heads, w.num_kv_heads, w.head_dim, w.page_size,
                         inp["max_pages"], inp["num_phys_pages"], w.kv_dtype)
    meta = torch.empty((inp["num_phys_pages"], w.num_kv_heads, 2, w.head_dim), dtype=kv_t,
                       device=dev)
    E.entmaxkv_build_page_meta(shape, k, bt, lens, meta)
    B, H, D = w.batch, w.num_q_heads, w.head_dim
    G = H // w.num_kv_heads
    rng = np.random.default_rng(0)
    n_check = max(0, args.oracle_heads // (len(w.alphas) * len(w.budgets)))
    full = {}
    for alpha in w.alphas:
        out = torch.empty((B, H, D), device=dev)
        tau = torch.empty((B, H), device=dev)
        sup = torch.empty((B, H), dtype=torch.int32, device=dev)
        E.entmaxkv_decode_full(shape, q, k, v, bt, lens, alpha, out, tau, sup)
        torch.cuda.synchronize()
        full[alpha] = (tau.cpu().numpy(), sup.cpu().numpy())
    cells = []
    for budget in w.budgets:
        sel = torch.empty((B, H, budget), dtype=torch.int32, device=dev)
        E.entmaxkv_score_select(shape, q, meta, bt, lens, budget, sel)
        torch.cuda.synchronize()
        sel_np = sel.cpu().numpy()
        for alpha in w.alphas:
            out = torch.empty((B, H, D), device=dev)
            tau = torch.empty((B, H), device=dev)
            sup = torch.empty((B, H), dtype=torch.int32, device=dev)
            E.entmaxkv_decode_sparse(shape, q, k, v, bt, lens, sel, budget, alpha, out, tau, sup)
            torch.cuda.synchronize()
            tau_f, sup_f = full[alpha]
            c = contained(sup.cpu().numpy(), sup_f, tau.cpu().numpy(), tau_f)
            agree = 0
            checks = [(int(rng.integers(0, B)), int(rng.integers(0, H))) for _ in range(n_check)]
            for b, h in checks:
                res = O.decode_full(inp, b, h, alpha)
                ref = set(O.support_pages(res, w.page_size)) <= set(int(j) for j in sel_np[b, h])
                agree += int(ref == bool(c[b, h]))
            cells.append({"alpha": alpha, "budget_pages": budget, "trials": int(c.size),
                          "contained_fraction": round(float(c.mean()), 4),
                          "mean_support_full": round(float(sup_f.mean()), 2),
                          "oracle_checked": len(checks), "oracle_agree": agree})
            log(f"alpha {alpha} budget {budget}: contained {c.mean():.4f}")
    print(json.dumps({"report": "containment", "workload": w.name, "data": "synthetic",
                      "trial": "one (sequence, query head) decode",
                      "criterion": "selected pages contain the full-cache support (GPU: equal "
                                   "support size and tau within 1e-6; sampled trials re-checked "
                                   "against the oracle's support pages)",
                      "cells": cells}))


def sweep_report(args):
    """Times every (alpha, budget) cell of the workload: the sparse path
    (entmaxkv_decode_topk) per cell and the full-cache path per
    alpha, each step after the cache eviction, median of K steps; bytes
    touched and all-K+V bytes against 8 TB/s; per-kernel times from a second
    pass with events around every kernel."""
    import torch
    from sparse_long_context_page_amd import entmaxkv as E
    w = synth.WORKLOADS[args.workload]
    log = lambda m: (sys.stderr.write(f"[report] {m}\n"), sys.stderr.flush())
    inp = synth.generate(w, synth.WORKLOAD_SEEDS[w.name])
    log(f"generated {w.name}")
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    kv_t = torch.bfloat16 if w.kv_dtype == "bf16" else torch.float32

    def pool(a):
        if w.kv_dtype == "bf16":
            return torch.from_numpy(a.view(np.int16)).to(dev).view(torch.bfloat16)
        return torch.from_numpy(a).to(dev)

    q = torch.from_numpy(inp["q"]).to(dev)
    k, v = pool(inp["k_pool"]), pool(inp["v_pool"])
    bt = torch.from_numpy(inp["block_table"]).to(dev)
    lens = torch.from_numpy(inp["seq_lens"]).to(dev)
    shape = E.make_shape(w.batch, w.num_q_heads, w.num_kv_heads, w.head_dim, w.page_size,
                         inp["max_pages"], inp["num_phys_pages"], w.kv_dtype)
    meta = torch.empty((inp["num_phys_pages"], w.num_kv_heads, 2, w.head_dim), dtype=kv_t,
                       device=dev)
    E.entmaxkv_build_page_meta(shape, k, bt, lens, meta)
    B, H, D = w.batch, w.num_q_heads, w.head_dim
    flush_buf = torch.empty(1 << 30, dtype=torch.uint8, device=dev)
    stream = torch.cuda.current_stream(dev)
    K = args.steps
    ev = E.HipEvents(2 * K)
    kev = E.HipEvents(8)

    def timed(calls, nk):
        for i in range(args.warmup):
            flush_buf.fill_(i & 255)
            for c in calls:
                c()
        torch.cuda.synchronize()
        for i in range(K):
            flush_buf.fill_(i & 255)
            ev.record(2 * i, stream)
            for c in calls:
                c()
            ev.record(2 * i + 1, stream)
        torch.cuda.synchronize()
        ms = np.array([ev.elapsed_ms(2 * i, 2 * i + 1) for i in range(K)])
        per_k = []
        for i in range(K):
            flush_buf.fill_(i & 255)
            j = 0
            for c, n in zip(calls, nk):
                c(list(kev)[2 * j:2 * (j + n)])
                j += n
            torch.cuda.synchronize()
            per_k.append([kev.elapsed_ms(2 * t, 2 * t + 1) * 1e3 for t in range(j)])
        return float(np.median(ms)), np.median(np.array(per_k), axis=0)

    out = torch.empty((B, H, D), device=dev)
    tau = torch.empty((B, H), device=dev)
    sup = torch.empty((B, H), dtype=torch.int32, device=dev)
    ws_fu = E.workspace(shape, 0, E.ENTMAXKV_WS_FULL, dev)
    cells, fulls = [], []
    for alpha in w.alphas:
        call = E.Prepared("decode_full", shape, q, k, v, bt, lens, alpha, out, tau, sup,
                          ws=ws_fu, stream=stream)
        ms, kk = timed([call], [2])
        sup_np = sup.cpu().numpy()
        nb = algorithmic_bytes(w, inp["seq_lens"], 1, np.zeros((B, H, 1), np.int32), sup_np,
                               sup_np)
        by = nb["score_full"] + nb["tau_pv_full"]
        fulls.append({"alpha": alpha, "median_us": round(ms * 1e3, 2), "bytes": by,
                      "frac": round(by / (ms * 1e-3) / 1e9 / PEAK_HBM_GBPS, 4),
                      "bytes_all_kv": nb["_full_all_kv"],
                      "frac_all_kv": round(nb["_full_all_kv"] / (ms * 1e-3) / 1e9 /
                                           PEAK_HBM_GBPS, 4),
                      "score_us": round(float(kk[0]), 2), "tau_pv_us": round(float(kk[1]), 2),
                      "mean_support": float(sup_np.mean())})
        log(f"full alpha {alpha}: {ms * 1e3:.1f} us")
    for budget in w.budgets:
        sel = torch.empty((B, H, budget), dtype=torch.int32, device=dev)
        ws_tk = E.workspace(shape, budget, E.ENTMAXKV_WS_TOPK, dev)
        names = sparse_kernels(E, shape, budget)
        for alpha in w.alphas:
            c_tk = E.Prepared("decode_topk", shape, q, meta, k, v, bt, lens, budget, alpha, sel,
                              out, None, tau, sup, ws=ws_tk, stream=stream)
            ms, kk = timed([c_tk], [4])
            sup_np = sup.cpu().numpy()
            nb = algorithmic_bytes(w, inp["seq_lens"], budget, sel.cpu().numpy(), sup_np, sup_np)
            by = sum(nb[n] for n in names)
            cells.append({"alpha": alpha, "budget_pages": budget, "median_us": round(ms * 1e3, 2),
                          "bytes": by, "frac": round(by / (ms * 1e-3) / 1e9 / PEAK_HBM_GBPS, 4),
                          "bytes_all_kv": nb["_sparse_all_kv"],
                          "frac_all_kv": round(nb["_sparse_all_kv"] / (ms * 1e-3) / 1e9 /
                                               PEAK_HBM_GBPS, 4),
                          "union_fraction": round(nb["_union_fraction"], 4),
                          "kernels_us": {n: round(float(x), 2) for n, x in zip(names, kk)},
                          "mean_support": float(sup_np.mean())})
            log(f"sparse alpha {alpha} budget {budget}: {ms * 1e3:.1f} us")
    print(json.dumps({"report": "sweep", "workload": w.name, "data": "synthetic", "steps": K,
                      "cache_flush": args.flush, "timing": "median of the steps",
                      "full": fulls, "sparse": cells}))


def _mass_head(args):
    """Oracle side of the mass report for one (sequence, head): its whole
    cache gathered once, then every (alpha, budget) cell's kept pages."""
    from oracle import entmax_oracle as O
    from oracle import mass_oracle as M
    b, h, cells = args
    inp = _ORACLE_STATE["inp"]
    w = inp["workload"]
    g = h // (w.num_q_heads // w.num_kv_heads)
    K, pos = O.gather_tokens(inp["k_pool"], b, g, inp["block_table"], inp["seq_lens"],
                             w.page_size, w.kv_dtype)
    V, _ = O.gather_tokens(inp["v_pool"], b, g, inp["block_table"], inp["seq_lens"],
                           w.page_size, w.kv_dtype)
    z = K @ inp["q"][b, h].astype(np.float64)
    page = pos // w.page_size
    out = []
    for alpha, budget, sel_row in cells:
        keep = np.isin(page, [int(j) for j in sel_row if j >= 0])
        out.append((alpha, budget, M.mass_comparison(z, V, keep, alpha)))
    return b, h, out


def mass_report(args):
    """Discarded probability mass under the same kept pages (EntmaxKV page,
    sections 3 and 4): for each (alpha, budget) cell of the workload, the
    GPU's top-k selection fixes the kept pages; on sampled heads the oracle
    gives delta (the full-cache mass outside them) for alpha-entmax and for
    softmax over the same scores, the relative output error of each sparse
    output (entmax re-solved on the kept tokens, softmax renormalised), the
    kept share of the entmax support, and checks the 2 B delta bound; over
    every head, the GPU's own sparse-vs-full entmax relative error."""
    import torch
    from sparse_long_context_page_amd import entmaxkv as E
    w = synth.WORKLOADS[args.workload]
    log = lambda m: (sys.stderr.write(f"[report] {m}\n"), sys.stderr.flush())
    inp = synth.generate(w, synth.WORKLOAD_SEEDS[w.name])
    log(f"generated {w.name}")
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    kv_t = torch.bfloat16 if w.kv_dtype == "bf16" else torch.float32

    def pool(a):
        if w.kv_dtype == "bf16":
            return torch.from_numpy(a.view(np.int16)).to(dev).view(torch.bfloat16)
        return torch.from_numpy(a).to(dev)

    q = torch.from_numpy(inp["q"]).to(dev)
    k, v = pool(inp["k_pool"]), pool(inp["v_pool"])
    bt = torch.from_numpy(inp["block_table"]).to(dev)
    lens = torch.from_numpy(inp["seq_lens"]).to(dev)
    shape = E.make_shape(w.batch, w.num_q_heads, w.num_kv_heads, w.head_dim, w.page_size,
                         inp["max_pages"], inp["num_phys_pages"], w.kv_dtype)
    meta = torch.empty((inp["num_phys_pages"], w.num_kv_heads, 2, w.head_dim), dtype=kv_t,
                       device=dev)
    E.entmaxkv_build_page_meta(shape, k, bt, lens, meta)
    B, H, D = w.batch, w.num_q_heads, w.head_dim
    full = {}
    for alpha in w.alphas:
        out = torch.empty((B, H, D), device=dev)
        tau = torch.empty((B, H), device=dev)
        sup = torch.empty((B, H), dtype=torch.int32, device=dev)
        E.entmaxkv_decode_full(shape, q, k, v, bt, lens, alpha, out, tau, sup)
        torch.cuda.synchronize()
        full[alpha] = (out.cpu().numpy(), tau.cpu().numpy(), sup.cpu().numpy())
    rng = np.random.default_rng(0)
    heads = sorted({(int(rng.integers(0, B)), int(rng.integers(0, H)))
                    for _ in range(args.oracle_heads)})
    sels, gpu = {}, {}
    for budget in w.budgets:
        sel = torch.empty((B, H, budget), dtype=torch.int32, device=dev)
        E.entmaxkv_score_select(shape, q, meta, bt, lens, budget, sel)
        torch.cuda.synchronize()
        sels[budget] = sel.cpu().numpy()
        for alpha in w.alphas:
            out = torch.empty((B, H, D), device=dev)
            tau = torch.empty((B, H), device=dev)
            sup = torch.empty((B, H), dtype=torch.int32, device=dev)
            E.entmaxkv_decode_sparse(shape, q, k, v, bt, lens, sel, budget, alpha, out, tau, sup)
            torch.cuda.synchronize()
            of, tf, sf = full[alpha]
            os_ = out.cpu().numpy()
            rel = np.linalg.norm(os_ - of, axis=2) / np.linalg.norm(of, axis=2)
            c = contained(sup.cpu().numpy(), sf, tau.cpu().numpy(), tf)
            gpu[(alpha, budget)] = (rel, c)
    log(f"GPU selections and decodes done; oracle on {len(heads)} heads")
    _ORACLE_STATE["inp"] = inp
    cores = len(os.sched_getaffinity(0))
    tasks = [(b, h, [(alpha, budget, sels[budget][b, h]) for budget in w.budgets
                     for alpha in w.alphas]) for b, h in heads]
    with mp.get_context("fork").Pool(min(cores, len(tasks)), initializer=_pin_blas) as pool_:
        results = pool_.map(_mass_head, tasks)
    stat = lambda x: {"median": float(np.median(x)), "mean": float(np.mean(x)),
                      "min": float(np.min(x)), "max": float(np.max(x))}
    cells = []
    for budget in w.budgets:
        for alpha in w.alphas:
            rs = [r for _, _, res in results for a, bu, r in res if a == alpha and bu == budget]
            de = np.array([r["delta_entmax"] for r in rs])
            ds = np.array([r["delta_softmax"] for r in rs])
            rel_g, c = gpu[(alpha, budget)]
            cells.append({
                "alpha": alpha, "budget_pages": budget, "oracle_heads": len(rs),
                "delta_entmax": stat(de), "delta_softmax": stat(ds),
                "heads_entmax_drops_less": int((de < ds).sum()),
                "heads_entmax_drops_none": int((de == 0.0).sum()),
                "support_kept_fraction": float(np.mean([r["support_kept"] / r["support"]
                                                        for r in rs])),
                "kept_token_fraction": float(np.mean([r["kept_tokens"] / r["tokens"]
                                                      for r in rs])),
                "rel_err_entmax": stat([r["rel_err_entmax"] for r in rs]),
                "rel_err_softmax": stat([r["rel_err_softmax"] for r in rs]),
                "bound_holds": int(sum(r["err_entmax"] <= r["bound_entmax"] + 1e-12
                                       and r["err_softmax"] <= r["bound_softmax"] + 1e-12
                                       for r in rs)),
                "gpu_all_heads": {"heads": int(rel_g.size),
                                  "rel_err_entmax": stat(rel_g.ravel()),
                                  "support_contained_fraction": float(c.mean())}})
            log(f"alpha {alpha} budget {budget}: delta entmax median {np.median(de):.3g}, "
                f"softmax {np.median(ds):.3g}")
    print(json.dumps({"report": "mass", "workload": w.name, "data": "synthetic",
                      "kept_set": "the GPU's top-k page selection (box bound, ties to the "
                                  "lower page)",
                      "softmax": "over the same scores z = q.k; sparse output renormalised "
                                 "over the kept tokens",
                      "cores": min(cores, len(tasks)), "cells": cells}))


def gauss_report(args):
    """Gaussian-aware selection (page moments, tau_hat, pages whose estimated
    maximum clears tau_hat - delta, at most `cap`): for each alpha of the
    workload and each (delta, cap) cell, the pages kept per head, the fraction
    of trials whose kept pages contain the full-cache support (criterion as in
    the containment report, sampled trials re-checked against the oracle), and
    the selection's time; the fixed-budget top-k at the workload's budget for
    comparison."""
    import torch
    from oracle import entmax_oracle as O
    from sparse_long_context_page_amd import entmaxkv as E
    w = synth.WORKLOADS[args.workload]
    log = lambda m: (sys.stderr.write(f"[report] {m}\n"), sys.stderr.flush())
    inp = synth.generate(w, synth.WORKLOAD_SEEDS[w.name])
    log(f"generated {w.name}")
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    kv_t = torch.bfloat16 if w.kv_dtype == "bf16" else torch.float32

    def pool(a):
        if w.kv_dtype == "bf16":
            return torch.from_numpy(a.view(np.int16)).to(dev).view(torch.bfloat16)
        return torch.from_numpy(a).to(dev)

    q = torch.from_numpy(inp["q"]).to(dev)
    k, v = pool(inp["k_pool"]), pool(inp["v_pool"])
    bt = torch.from_numpy(inp["block_table"]).to(dev)
    lens = torch.from_numpy(inp["seq_lens"]).to(dev)
    shape = E.make_shape(w.batch, w.num_q_heads, w.num_kv_heads, w.head_dim, w.page_size,
                         inp["max_pages"], inp["num_phys_pages"], w.kv_dtype)
    B, H, D = w.batch, w.num_q_heads, w.head_dim
    P = int(inp["max_pages"])
    mshape = (inp["num_phys_pages"], w.num_kv_heads, 2, D)
    meta = torch.empty(mshape, dtype=kv_t, device=dev)
    mom = torch.empty(mshape, dtype=kv_t, device=dev)
    E.entmaxkv_build_page_meta(shape, k, bt, lens, meta)
    ev = E.HipEvents(6)
    flush = torch.empty(1 << 30, dtype=torch.uint8, device=dev)

    stream = torch.cuda.current_stream(dev)

    def timed(call, n=7):
        # events at the call's ends only (events between its kernels hold
        # each next launch back)
        ts = []
        for i in range(n):
            flush.fill_(i & 255)
            ev.record(0, stream)
            call()
            ev.record(1, stream)
            torch.cuda.synchronize()
            ts.append(ev.elapsed_ms(0, 1) * 1e3)
        return float(np.median(ts[2:]))

    mom_us = []
    for i in range(5):
        flush.fill_(i)
        E.entmaxkv_build_page_moments(shape, k, bt, lens, mom, events=list(ev)[:2])
        torch.cuda.synchronize()
        mom_us.append(ev.elapsed_ms(0, 1) * 1e3)
    # a decode step's moment maintenance: one appended token per sequence
    # (the touched pages are recomputed to the bits they already hold)
    old_lens = (lens - 1).clamp(min=0)
    mom_app_us = []
    for i in range(5):
        flush.fill_(i)
        E.entmaxkv_append_page_moments(shape, k, bt, old_lens, lens, 1, mom,
                                       events=list(ev)[:2])
        torch.cuda.synchronize()
        mom_app_us.append(ev.elapsed_ms(0, 1) * 1e3)
    rng = np.random.default_rng(0)
    alphas = (args.alpha,) if args.alpha else w.alphas
    budget = args.budget or w.budgets[0]
    cells = []
    for alpha in alphas:
        out = torch.empty((B, H, D), device=dev)
        tau = torch.empty((B, H), device=dev)
        sup = torch.empty((B, H), dtype=torch.int32, device=dev)
        E.entmaxkv_decode_full(shape, q, k, v, bt, lens, alpha, out, tau, sup)
        torch.cuda.synchronize()
        tau_f, sup_f = tau.cpu().numpy(), sup.cpu().numpy()

        def decode_contained(sel_t, cap):
            E.entmaxkv_decode_sparse(shape, q, k, v, bt, lens, sel_t, cap, alpha, out, tau, sup)
            torch.cuda.synchronize()
            return contained(sup.cpu().numpy(), sup_f, tau.cpu().numpy(), tau_f)

        sel_k = torch.empty((B, H, budget), dtype=torch.int32, device=dev)
        E.entmaxkv_score_select(shape, q, meta, bt, lens, budget, sel_k)
        c_k = decode_contained(sel_k, budget)
        cells.append({"policy": "top-k (box bound)", "alpha": alpha, "budget_pages": budget,
                      "contained_fraction": round(float(c_k.mean()), 4)})
        log(f"alpha {alpha} top-{budget}: contained {c_k.mean():.4f}")
        for cap in (budget, P):
            for delta in (0.0, 1.0, 2.0, 3.0, 4.0, 6.0):
                sel = torch.empty((B, H, cap), dtype=torch.int32, device=dev)
                ws = E.workspace(shape, cap, E.ENTMAXKV_WS_GAUSS, dev)
                call = E.Prepared("gauss_select", shape, q, mom, bt, lens, alpha, delta, cap,
                                  sel, None, ws=ws)
                us = timed(call)
                kept = (sel >= 0).sum(dim=2).cpu().numpy()
                c = decode_contained(sel, cap)
                sel_np = sel.cpu().numpy()
                agree = 0
                checks = [(int(rng.integers(0, B)), int(rng.integers(0, H))) for _ in range(2)]
                for b, h in checks:
                    res = O.decode_full(inp, b, h, alpha)
                    ref = set(O.support_pages(res, w.page_size)) <= set(int(j) for j in sel_np[b, h])
                    agree += int(ref == bool(c[b, h]))
                cells.append({"policy": "gaussian", "alpha": alpha, "delta": delta, "cap": cap,
                              "mean_pages": round(float(kept.mean()), 2),
                              "p90_pages": int(np.percentile(kept, 90)),
                              "contained_fraction": round(float(c.mean()), 4),
                              "select_us": round(us, 2), "oracle_checked": len(checks),
                              "oracle_agree": agree})
                log(f"alpha {alpha} delta {delta} cap {cap}: pages {kept.mean():.1f} "
                    f"contained {c.mean():.4f} select {us:.1f} us")
    print(json.dumps({"report": "gauss", "workload": w.name, "data": "synthetic",
                      "page_moments_us": round(float(np.median(mom_us[1:])), 2),
                      "page_moments_append_us": round(float(np.median(mom_app_us[1:])), 2),
                      "trial": "one (sequence, query head) decode",
                      "criterion": "kept pages contain the full-cache support (GPU: equal "
                                   "support size and tau within 1e-6; sampled trials re-checked "
                                   "against the oracle's support pages)",
                      "cells": cells}))


def softmax_report(args):
    """The softmax and eviction calls on a workload's cache: the full-cache
    softmax decode beside the full-cache alpha-entmax decode (the comparison
    the efficiency section of the EntmaxKV page is about), a 4096-token window
    with 4 sinks, the attention weights of both decodes, and the eviction of
    three quarters of every cache by them. A sampled head of each decode is
    re-checked against the oracle."""
    import torch
    from oracle import softmax_oracle as S
    from sparse_long_context_page_amd import entmaxkv as E
    w = synth.WORKLOADS[args.workload]
    log = lambda m: (sys.stderr.write(f"[report] {m}\n"), sys.stderr.flush())
    inp = synth.generate(w, synth.WORKLOAD_SEEDS[w.name])
    log(f"generated {w.name}")
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    bf16 = w.kv_dtype == "bf16"
    B, H, G, D, ps = w.batch, w.num_q_heads, w.num_kv_heads, w.head_dim, w.page_size
    pages, mp = int(inp["num_phys_pages"]), int(inp["max_pages"])
    lens_np = np.asarray(inp["seq_lens"], np.int64)
    keep, sinks, recent = max(int(lens_np.max()) // 4, 8), 4, min(64, int(lens_np.max()) // 8)
    fresh = B * -(-keep // ps)

    def pool(a):
        t = torch.from_numpy(a.view(np.int16)).to(dev).view(torch.bfloat16) if bf16 else \
            torch.from_numpy(a).to(dev)
        return torch.cat([t, torch.zeros((fresh, *t.shape[1:]), dtype=t.dtype, device=dev)])

    q = torch.from_numpy(inp["q"]).to(dev)
    k, v = pool(inp["k_pool"]), pool(inp["v_pool"])
    bt = torch.from_numpy(inp["block_table"]).to(dev)
    lens = torch.from_numpy(inp["seq_lens"]).to(dev)
    nt = torch.full((B, mp), -1, dtype=torch.int32, device=dev)
    nt[:, :fresh // B] = torch.arange(pages, pages + fresh, device=dev).view(B, -1)
    shape = E.make_shape(B, H, G, D, ps, mp, pages + fresh, w.kv_dtype)
    alpha = args.alpha or w.alphas[0]
    out, lse = torch.empty((B, 1, H, D), device=dev), torch.empty((B, 1, H), device=dev)
    oute, tau = torch.empty((B, H, D), device=dev), torch.empty((B, H), device=dev)
    weights = torch.zeros((B, G, mp * ps), device=dev)
    kept = torch.empty((B, G, keep), dtype=torch.int32, device=dev)
    nl, nw = torch.empty((B,), dtype=torch.int32, device=dev), torch.empty_like(weights)
    ws = E.workspace(shape, 0, E.ENTMAXKV_WS_FULL, dev)
    window = 4096
    calls = {
        "entmax_full": E.Prepared("decode_full", shape, q, k, v, bt, lens, alpha, oute, tau, ws=ws),
        "softmax_full": E.Prepared("softmax_window", shape, q, k, v, bt, lens, E.FULL_WINDOW, 0,
                                   out, lse=lse),
        "weights_entmax": E.Prepared("accumulate_weights", shape, q, k, bt, lens, alpha, tau, 1.0,
                                     None, weights),
        "weights_softmax": E.Prepared("accumulate_weights", shape, q, k, bt, lens, 1.0, lse, 1.0,
                                      weights, weights),
        "evict": E.Prepared("evict", shape, k, v, bt, lens, weights, keep, sinks, recent, nt, kept,
                            nl, new_weights=nw),
        "softmax_window_4096": E.Prepared("softmax_window", shape, q, k, v, bt, lens, window, sinks,
                                          out, lse=lse),
    }
    ev = E.HipEvents(2)
    flush = torch.empty(1 << 30, dtype=torch.uint8, device=dev)
    stream = torch.cuda.current_stream(dev)
    rng = np.random.default_rng(0)
    kn, vn = (np.asarray(inp[x]) for x in ("k_pool", "v_pool"))
    if bf16:
        widen = lambda a: (a.astype(np.uint32) << 16).view(np.float32)
    else:
        widen = lambda a: a
    seen = {"softmax_full": (E.FULL_WINDOW, 0), "softmax_window_4096": (window, sinks)}
    us, worst = {}, 0.0
    for name, call in calls.items():
        ts = []
        for i in range(args.warmup + args.steps):
            flush.fill_(i & 255)
            ev.record(0, stream)
            call()
            ev.record(1, stream)
            torch.cuda.synchronize()
            ts.append(ev.elapsed_ms(0, 1) * 1e3)
        us[name] = round(float(np.median(ts[args.warmup:])), 2)
        log(f"{name}: {us[name]} us")
        if name in seen:
            b, h = int(rng.integers(0, B)), int(rng.integers(0, H))
            t = S.visible(int(lens_np[b]) - 1, int(lens_np[b]), *seen[name])
            rows = [widen(S.rows(x, inp["block_table"][b], h // (H // G), t)) for x in (kn, vn)]
            ref, _ = S.attend(inp["q"][b, h], *rows)
            err = float(np.abs(out[b, 0, h].cpu().numpy() - ref).max())
            worst = max(worst, err / float(np.linalg.norm(ref)))
    s = 2 if bf16 else 4
    rows = {"softmax_full": lens_np, "softmax_window_4096": np.minimum(lens_np, window + sinks)}
    print(json.dumps({"report": "softmax", "workload": w.name, "data": "synthetic", "alpha": alpha,
                      "steps": args.steps, "warmup": args.warmup, "us": us,
                      "kv_gbs": {n: round(2 * int(r.sum()) * G * D * s / us[n] / 1e3, 1)
                                 for n, r in rows.items()},
                      "kept_tokens": keep, "worst_error_rel_norm": worst}))


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--warmup", type=int, default=5)
    ap.add_argument("--workload", default="long_128k", choices=sorted(synth.WORKLOADS))
    ap.add_argument("--alpha", type=float, default=None)
    ap.add_argument("--budget", type=int, default=None)
    ap.add_argument("--oracle-heads", type=int, default=64)
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--no-flush", action="store_true", help="hot-cache timing (diagnostic)")
    ap.add_argument("--flush", choices=["write", "write_read"], default="write",
                    help="cache eviction before each timed step: 'write' fills a 1 GiB buffer "
                         "(the caches are left holding its dirty lines); 'write_read' fills it "
                         "and then reads a second 1 GiB buffer (the caches are left holding "
                         "clean lines of unrelated data)")
    ap.add_argument("--report", choices=["containment", "gauss", "mass", "softmax", "sweep"],
                    default=None,
                    help="instead of the timed step: 'containment', the alpha/budget sweep "
                         "report of how often the selected pages contain the full-cache support "
                         "(default workload alpha_sweep_64k); 'gauss', the same for the "
                         "Gaussian-aware selection over a grid of margins and caps, with its "
                         "times (default workload long_128k); 'mass', the probability mass "
                         "alpha-entmax and softmax drop outside the selected pages and their "
                         "output errors, per (alpha, budget) cell; 'softmax', the softmax decode "
                         "(full and windowed), the attention weights and the eviction by them, "
                         "timed beside the full alpha-entmax decode (default workload long_128k); "
                         "'sweep', the sparse path "
                         "timed on every (alpha, budget) cell and the full path on every alpha "
                         "(default workload alpha_sweep_64k); each prints its own JSON line")
    ap.add_argument("--copy-calibration", action="store_true",
                    help="after the steps, run a plain 1 GiB device copy three times (a known-size "
                         "reference for the rocprofv3 FETCH_SIZE / WRITE_SIZE counters)")
    args = ap.parse_args()

    if args.gpus != 1 or int(os.environ.get("WORLD_SIZE", "1")) > 1:
        print("bench.py runs on one GPU only: this build has no multi-GPU path "
              "(collectives and sharding are out of scope).", file=sys.stderr)
        sys.exit(2)

    if args.report == "containment":
        if "--workload" not in sys.argv:
            args.workload = "alpha_sweep_64k"
        containment_report(args)
        return
    if args.report == "gauss":
        gauss_report(args)
        return
    if args.report == "softmax":
        softmax_report(args)
        return
    if args.report == "sweep":
        if "--workload" not in sys.argv:
            args.workload = "alpha_sweep_64k"
        if "--steps" not in sys.argv:
            args.steps = 15
        sweep_report(args)
        return
    if args.report == "mass":
        if "--oracle-heads" not in sys.argv:
            args.oracle_heads = 16
        mass_report(args)
        return

    w = synth.WORKLOADS[args.workload]
    alpha = args.alpha if args.alpha is not None else w.alphas[0]
    budget = args.budget if args.budget is not None else w.budgets[0]
    t_gen = time.perf_counter()
    inp = synth.generate(w, synth.WORKLOAD_SEEDS[w.name])
    t_gen = time.perf_counter() - t_gen
    log = lambda m: (sys.stderr.write(f"[bench] {m}\n"), sys.stderr.flush())
    log(f"generated {w.name} in {t_gen:.1f}s")

    cpu = None
    if not args.no_cpu_baseline:
        cpu = cpu_baseline(inp, budget, alpha, args.oracle_heads)
        log(f"cpu baseline {cpu['value']:.4g} steps/s on {cpu['cores']} cores")

    import torch
    from sparse_long_context_page_amd import entmaxkv as E

    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    kv_t = torch.bfloat16 if w.kv_dtype == "bf16" else torch.float32

    def pool(a):
        if w.kv_dtype == "bf16":
            return torch.from_numpy(a.view(np.int16)).to(dev).view(torch.bfloat16)
        return torch.from_numpy(a).to(dev)

    q = torch.from_numpy(inp["q"]).to(dev)
    k = pool(inp["k_pool"])
    v = pool(inp["v_pool"])
    bt = torch.from_numpy(inp["block_table"]).to(dev)
    lens = torch.from_numpy(inp["seq_lens"]).to(dev)
    shape = E.make_shape(w.batch, w.num_q_heads, w.num_kv_heads, w.head_dim, w.page_size,
                         inp["max_pages"], inp["num_phys_pages"], w.kv_dtype)
    meta = torch.empty((inp["num_phys_pages"], w.num_kv_heads, 2, w.head_dim), dtype=kv_t,
                       device=dev)
    B, H, D = w.batch, w.num_q_heads, w.head_dim
    sel = torch.empty((B, H, budget), dtype=torch.int32, device=dev)
    sel_ub = torch.empty((B, H, budget), dtype=torch.float32, device=dev)
    out_s = torch.empty((B, H, D), device=dev)
    out_f = torch.empty((B, H, D), device=dev)
    tau_s = torch.empty((B, H), device=dev)
    tau_f = torch.empty((B, H), device=dev)
    sup_s = torch.empty((B, H), dtype=torch.int32, device=dev)
    sup_f = torch.empty((B, H), dtype=torch.int32, device=dev)
    ws_tk = E.workspace(shape, budget, E.ENTMAXKV_WS_TOPK, dev)
    ws_fu = E.workspace(shape, budget, E.ENTMAXKV_WS_FULL, dev)
    sp_names = sparse_kernels(E, shape, budget)
    flush_buf = torch.empty(1 << 30, dtype=torch.uint8, device=dev)
    read_buf = (torch.ones(1 << 28, dtype=torch.int32, device=dev)
                if args.flush == "write_read" else None)
    read_sink = torch.empty((), dtype=torch.int64, device=dev)
    stream = torch.cuda.current_stream(dev)

    def flush(i):
        if not args.no_flush:
            flush_buf.fill_(i & 0xFF)
            if read_buf is not None:
                torch.sum(read_buf, dim=0, dtype=torch.int64, out=read_sink)

    # page boxes (per-page state; timed separately)
    n_meta = max(3, min(10, args.steps))
    ev_meta = E.HipEvents(2 * n_meta)
    E.entmaxkv_build_page_meta(shape, k, bt, lens, meta)
    for i in range(n_meta):
        flush(i)
        E.entmaxkv_build_page_meta(shape, k, bt, lens, meta, events=list(ev_meta)[2 * i:2 * i + 2])
    torch.cuda.synchronize()
    meta_ms = float(np.mean([ev_meta.elapsed_ms(2 * i, 2 * i + 1) for i in range(n_meta)]))
    # a decode step's box maintenance: one appended token per sequence (the
    # boxes already hold it, so the update leaves them as they are)
    old_lens = (lens - 1).clamp(min=0)
    ev_app = E.HipEvents(2 * n_meta)
    for i in range(n_meta):
        flush(i)
        E.entmaxkv_append_page_meta(shape, k, bt, old_lens, lens, 1, meta,
                                    events=list(ev_app)[2 * i:2 * i + 2])
    torch.cuda.synchronize()
    append_us = float(np.mean([ev_app.elapsed_ms(2 * i, 2 * i + 1) for i in range(n_meta)])) * 1e3

    call_tk = E.Prepared("decode_topk", shape, q, meta, k, v, bt, lens, budget, alpha, sel, out_s,
                         sel_ub, tau_s, sup_s, ws=ws_tk, stream=stream)
    call_fu = E.Prepared("decode_full", shape, q, k, v, bt, lens, alpha, out_f, tau_f, sup_f,
                         ws=ws_fu, stream=stream)

    def step(kev=None):
        if kev is None:
            call_tk()
            call_fu()
        else:
            call_tk(kev[0:8])
            call_fu(kev[8:12])

    for i in range(args.warmup):
        flush(i)
        step()
    torch.cuda.synchronize()

    # Timed pass: K steps, an event before and after each step only (an event
    # between the two paths holds the next launch back by a few us).
    K = args.steps
    ev_step = E.HipEvents(2 * K)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for i in range(K):
        flush(i)
        ev_step.record(2 * i, stream)
        call_tk()
        call_fu()
        ev_step.record(2 * i + 1, stream)
    torch.cuda.synchronize()
    wall = time.perf_counter() - t0
    step_ms = np.array([ev_step.elapsed_ms(2 * i, 2 * i + 1) for i in range(K)])
    ms_per_step = float(np.median(step_ms))

    # Path pass: the same steps with an event between the sparse and the
    # full path as well, for the per-path times.
    ev_path = E.HipEvents(3 * K)
    for i in range(K):
        flush(i)
        ev_path.record(3 * i, stream)
        call_tk()
        ev_path.record(3 * i + 1, stream)
        call_fu()
        ev_path.record(3 * i + 2, stream)
    torch.cuda.synchronize()
    sparse_ms = np.array([ev_path.elapsed_ms(3 * i, 3 * i + 1) for i in range(K)])
    full_ms = np.array([ev_path.elapsed_ms(3 * i + 1, 3 * i + 2) for i in range(K)])

    # Kernel pass: the same steps with events around every kernel (the library
    # records them on the launch stream), for per-kernel durations.
    ev_kern = E.HipEvents(12 * K)
    hk = list(ev_kern)
    for i in range(K):
        flush(i)
        step(hk[12 * i:12 * (i + 1)])
    torch.cuda.synchronize()
    # event pairs of the step: four for decode_topk (the per-head path fills
    # the first two), two for decode_full
    pairs = list(range(len(sp_names))) + [4, 5]
    kern_ms = np.array([[ev_kern.elapsed_ms(12 * i + 2 * j, 12 * i + 2 * j + 1) for j in pairs]
                        for i in range(K)])
    kernel_names = sp_names + FULL_KERNELS

    # Graph pass: the same step captured once as a HIP graph (on a stream of
    # its own, default priority) and replayed K times, the flush still outside
    # the timed region; every replay must reproduce the eager outputs bitwise.
    eager = [x.clone() for x in (sel, out_s, out_f, tau_s, tau_f)]
    gstream = torch.cuda.Stream(dev)
    g_calls = [
        E.Prepared("decode_topk", shape, q, meta, k, v, bt, lens, budget, alpha, sel, out_s,
                   sel_ub, tau_s, sup_s, ws=ws_tk, stream=gstream),
        E.Prepared("decode_full", shape, q, k, v, bt, lens, alpha, out_f, tau_f, sup_f, ws=ws_fu,
                   stream=gstream)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=gstream):
        for c in g_calls:
            c()
    ev_graph = E.HipEvents(2 * K)
    graph_same = True
    for i in range(K):
        flush(i)
        ev_graph.record(2 * i, stream)
        graph.replay()
        ev_graph.record(2 * i + 1, stream)
        if i == 0:
            torch.cuda.synchronize()
            graph_same = all(torch.equal(a, b) for a, b in
                             zip(eager, (sel, out_s, out_f, tau_s, tau_f)))
    torch.cuda.synchronize()
    graph_ms = np.array([ev_graph.elapsed_ms(2 * i, 2 * i + 1) for i in range(K)])
    graph_same = graph_same and all(torch.equal(a, b) for a, b in
                                    zip(eager, (sel, out_s, out_f, tau_s, tau_f)))
    log(f"graph step {graph_ms.mean():.4f} ms, replays match eager: {graph_same}")

    sel_np = sel.cpu().numpy()
    nbytes = algorithmic_bytes(w, inp["seq_lens"], budget, sel_np, sup_s.cpu().numpy(),
                               sup_f.cpu().numpy())
    kmean = kern_ms.mean(axis=0)
    kernels = {}
    for j, name in enumerate(kernel_names):
        gbps = nbytes[name] / (kmean[j] * 1e-3) / 1e9
        kernels[name] = {"us": round(kmean[j] * 1e3, 2), "bytes": nbytes[name],
                         "GBps": round(gbps, 1), "frac": round(gbps / PEAK_HBM_GBPS, 4)}
    sparse_bytes = sum(nbytes[n] for n in sp_names)
    full_bytes = sum(nbytes[n] for n in FULL_KERNELS)
    paths = {}
    for name, ms, by, by_all in (("sparse", sparse_ms, sparse_bytes, nbytes["_sparse_all_kv"]),
                                 ("full", full_ms, full_bytes, nbytes["_full_all_kv"])):
        med = float(np.median(ms))
        gbps = by / (med * 1e-3) / 1e9
        gbps_all = by_all / (med * 1e-3) / 1e9
        paths[name] = {"median_ms": round(med, 4), "mean_ms": round(float(ms.mean()), 4),
                       "p10_ms": round(float(np.percentile(ms, 10)), 4),
                       "p90_ms": round(float(np.percentile(ms, 90)), 4),
                       "steps_per_s": round(1e3 / med, 1), "bytes": by,
                       "GBps": round(gbps, 1), "frac": round(gbps / PEAK_HBM_GBPS, 4),
                       "bytes_all_kv": by_all, "frac_all_kv": round(gbps_all / PEAK_HBM_GBPS, 4)}
    paths["graph_step"] = {"mean_ms": round(float(graph_ms.mean()), 4),
                           "median_ms": round(float(np.median(graph_ms)), 4),
                           "p10_ms": round(float(np.percentile(graph_ms, 10)), 4),
                           "p90_ms": round(float(np.percentile(graph_ms, 90)), 4),
                           "steps_per_s": round(1e3 / float(np.median(graph_ms)), 1),
                           "matches_eager": bool(graph_same),
                           "note": "the whole step (sparse + full) replayed as one HIP graph"}
    meta_gbps = nbytes["_meta_build"] / (meta_ms * 1e-3) / 1e9
    paths["page_boxes"] = {"ms": round(meta_ms, 4), "bytes": nbytes["_meta_build"],
                           "GBps": round(meta_gbps, 1), "frac": round(meta_gbps / PEAK_HBM_GBPS, 4),
                           "note": "built once per page, outside the step"}
    paths["page_boxes_append"] = {"us": round(append_us, 2),
                                  "note": "box update for one appended token per sequence "
                                          "(a decode step's box maintenance), outside the step"}
    dom = int(np.argmax(kmean))
    dname = kernel_names[dom]
    achieved = nbytes[dname] / (kmean[dom] * 1e-3) / 1e9
    traffic = counter_traffic(dname, profile_name(w, alpha, budget))
    roofline = {"bound": "hbm", "achieved": round(achieved, 1), "peak": PEAK_HBM_GBPS,
                "unit": "GB/s", "frac": round(achieved / PEAK_HBM_GBPS, 4), "traffic": traffic,
                "kernel": dname, "bytes_per_launch": nbytes[dname],
                "launch_us": round(kmean[dom] * 1e3, 2)}
    # each path as a whole against the same peak (bytes touched / the path's
    # median time): the method's own figure, of which the dominant kernel's
    # is an upper bound
    roofline_paths = {name: {"bound": "hbm", "achieved": paths[name]["GBps"],
                             "peak": PEAK_HBM_GBPS, "unit": "GB/s", "frac": paths[name]["frac"],
                             "bytes": paths[name]["bytes"], "median_us": round(
                                 paths[name]["median_ms"] * 1e3, 2)}
                      for name in ("sparse", "full")}

    parity = None
    cpu_line = None
    if cpu is not None:
        errs_s, errs_f, sel_same = [], [], 0
        near_pages = differing = outside = 0
        o_s, o_f = out_s.cpu().numpy(), out_f.cpu().numpy()
        for b, h, _, ref_sel, rs, rf, near in cpu["_results"]:
            sel_same += int(list(sel_np[b, h]) == list(ref_sel))
            diff = set(int(j) for j in sel_np[b, h] if j >= 0) ^ set(j for j in ref_sel if j >= 0)
            near_pages += max(0, len(near) - 1)  # (the budget-th page itself is in the band)
            differing += len(diff)
            outside += len(diff - set(near))
            errs_s.append(float(np.abs(o_s[b, h] - rs).max() / max(1e-30, np.linalg.norm(rs))))
            errs_f.append(float(np.abs(o_f[b, h] - rf).max() / max(1e-30, np.linalg.norm(rf))))
        parity = {"heads": len(cpu["_results"]), "selection_identical": sel_same,
                  "near_tie_pages": near_pages, "differing_pages": differing,
                  "differing_outside_near_ties": outside,
                  "max_rel_err_sparse": max(errs_s), "max_rel_err_full": max(errs_f),
                  "tolerance_rel": 2e-3,
                  "near_tie_band": "pages within 1e-5 relative of the budget-th bound"}
        cpu_line = {k: cpu[k] for k in ("value", "unit", "cores", "kind", "sample")}
        if cpu["one_core"] is not None:
            cpu_line["one_core"] = cpu["one_core"]

    record = {
        "metric": METRIC,
        "value": round(1e3 / ms_per_step, 3),
        "unit": "steps/s",
        "n_gpus": 1,
        "steps": K,
        "warmup": args.warmup,
        "ms_per_step": round(ms_per_step, 4),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "f32",
        "data": "synthetic",
        "config": {"workload": w.name, "batch": B, "q_heads": H, "kv_heads": w.num_kv_heads,
                   "head_dim": D, "context": int(w.context), "page_size": w.page_size,
                   "budget_pages": budget, "alpha": alpha, "kv_dtype": w.kv_dtype,
                   "parallelism": "single GPU", "cache_flush": (args.flush if not args.no_flush else None),
                   "step": "decode_topk (bounds, top-k, sparse decode) + decode_full",
                   "sparse_kernels": sp_names},
        "paths": paths,
        "kernels": kernels,
        "roofline": roofline,
        "roofline_paths": roofline_paths,
        "cpu_baseline": cpu_line,
        "diagnostics": {"union_fraction": round(nbytes["_union_fraction"], 4),
                        "k_bytes_per_head_reads": nbytes["_k_per_head"],
                        "mean_support_sparse": float(sup_s.float().mean()),
                        "mean_support_full": float(sup_f.float().mean()),
                        "wall_s_timed_region": round(wall, 3),
                        "kernel_source_hash": kernel_source_hash()},
        "parity_sample": parity,
    }
    print(json.dumps(record))

    if args.copy_calibration:
        src = torch.empty(1 << 30, dtype=torch.uint8, device=dev).fill_(1)
        dst = torch.empty_like(src)
        for _ in range(3):
            dst.copy_(src)
        torch.cuda.synchronize()
        log("copy calibration: 3 x 1 GiB device-to-device copy done")


if __name__ == "__main__":
    main()
