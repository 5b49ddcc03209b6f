"""Timed cases of the operators that put new tokens into the paged KV cache and
attend from them (the layouts are those of include/entmaxkv.h):

  plan    pages of a free list for the new tokens of every sequence, and the
          position and the cache slot of each token
  append  RMS norm of every head of the new queries and keys, the position
          rotation (one axis or several), keys and values into their slots
  chunk   alpha-entmax attention of the new tokens of a ragged batch (chunks of
          prompts beside single tokens) over all cached tokens up to their own

`run` computes them in elementary torch operations where `own` is false and
with the library where it is true.
"""
import math

import torch

own = False

DEVICE = "cuda"


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # a decode step of a small batch: only the call's latency counts
        {"name": "plan decode 64", "op": "plan", "batch": 64, "page": 16, "context": 32768,
         "chunks": 0, "tokens": 1, "short": 0},
        # a step that mixes prompt chunks with decoding, more wanted than there is room
        {"name": "plan mixed 256 short of pages", "op": "plan", "batch": 256, "page": 16,
         "context": 32768, "chunks": 24, "tokens": 512, "short": 60},
        # many prompts admitted at once
        {"name": "plan prompts 260K tokens", "op": "plan", "batch": 1023, "page": 64,
         "context": 16384, "chunks": 1000, "tokens": 300, "short": 0},
        # a decode step of a small batch, float32 queries for the decode calls
        {"name": "append decode 64", "op": "append", "rows": 64, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "kv": "bf16", "x": "bf16", "q": "f32", "norm": True, "rot": 128,
         "axes": 1, "interleaved": False, "context": 131072},
        # a prompt chunk
        {"name": "append chunk 8192", "op": "append", "rows": 8192, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 32, "kv": "bf16", "x": "bf16", "q": "bf16", "norm": True, "rot": 128,
         "axes": 1, "interleaved": False, "context": 32768},
        # tokens of images and video, their positions on three axes, an odd count
        {"name": "append three axes odd", "op": "append", "rows": 3001, "heads": 16,
         "kv_heads": 8, "dim": 128, "page": 16, "kv": "bf16", "x": "bf16", "q": "bf16",
         "norm": True, "rot": 128, "axes": 3, "interleaved": False, "context": 32768},
        # float32 cache, small heads, half of each rotated in neighbouring pairs, no norm
        {"name": "append f32 partial", "op": "append", "rows": 1777, "heads": 8, "kv_heads": 8,
         "dim": 64, "page": 16, "kv": "f32", "x": "f32", "q": "f32", "norm": False, "rot": 32,
         "axes": 1, "interleaved": True, "context": 9001},
        # a few short chats with a few tokens each: the call's latency counts
        {"name": "chunk short chats", "op": "chunk", "batch": 4, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "kv": "bf16", "q": "bf16", "context": 700, "chunks": 4,
         "tokens": 9, "alpha": 1.5},
        # a prompt from its first token
        {"name": "chunk prompt 2048", "op": "chunk", "batch": 1, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "kv": "bf16", "q": "bf16", "context": 2048, "chunks": 1,
         "tokens": 2048, "alpha": 1.5},
        # prompt chunks beside decoding sequences, float32 queries (the library's own type)
        {"name": "chunk mixed 32", "op": "chunk", "batch": 32, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 32, "kv": "bf16", "q": "f32", "context": 32768, "chunks": 2,
         "tokens": 512, "alpha": 1.5},
        # the last chunk of a long document
        {"name": "chunk 4096 of 32K", "op": "chunk", "batch": 1, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 32, "kv": "bf16", "q": "bf16", "context": 32768, "chunks": 1,
         "tokens": 4096, "alpha": 1.5},
        # float32 cache, small heads, odd lengths, flatter weights
        {"name": "chunk f32 odd", "op": "chunk", "batch": 5, "heads": 16, "kv_heads": 8,
         "dim": 64, "page": 16, "kv": "f32", "q": "f32", "context": 5003, "chunks": 3,
         "tokens": 333, "alpha": 1.25},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "chunk", "chunk", "chunk"])
    case = {"op": op, "page": rng.choice([16, 32, 64])}
    if op == "plan":
        batch = _log_int(rng, 1, 1023)
        tokens = _log_int(rng, 1, min(8192, 260000 // batch))
        case.update(batch=batch, context=max(tokens, _log_int(rng, 64, 32768)),
                    chunks=rng.choice([0, rng.randint(0, batch), batch]), tokens=tokens,
                    short=rng.choice([0, 0, rng.randint(1, batch)]))
        return case
    kv = rng.choice(["bf16", "bf16", "bf16", "f32"])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4] if kv_heads == 8 else [1, 2, 4, 8])
    dim = rng.choice([64, 128])
    case.update(heads=kv_heads * group, kv_heads=kv_heads, dim=dim, kv=kv)
    if op == "append":
        rot = rng.choice([dim, dim, dim // 2, 32, 0])
        case.update(x=rng.choice(["bf16", "f32"]), q=rng.choice(["bf16", "f32"]),
                    rows=_log_int(rng, 1, 8192 if kv == "bf16" else 4096),
                    norm=rng.choice([True, True, False]), rot=rot,
                    axes=rng.choice([1, 1, 2, 3, 4]) if rot else 1,
                    interleaved=rng.choice([False, False, True]),
                    context=_log_int(rng, 64, 1000000))
        if case["x"] == "f32":
            case["rows"] = min(case["rows"], 4096)
    else:
        batch = _log_int(rng, 1, 32)
        chunks = rng.choice([0, 1, rng.randint(0, batch), batch])
        tokens = _log_int(rng, 1, 4096)
        context = max(tokens, _log_int(rng, 64, 32768))
        # no more pairs of a query and a token than the largest listed case (a
        # float32 cache: an eighth, as its products are that much slower)
        most = 4.0e9 if kv == "bf16" else 0.5e9
        while _pairs_bound(batch, chunks, tokens, context) * case["heads"] > most:
            tokens, context = max(1, tokens * 2 // 3), max(1, context * 4 // 5)
            context = max(context, tokens)
        case.update(batch=batch, chunks=chunks, tokens=tokens, context=context,
                    q=rng.choice(["bf16", "f32"]) if kv == "bf16" else "f32",
                    alpha=rng.choice([1.25, 1.5, 1.5, 1.6, 2.0]))
    return case


def _pairs_bound(batch, chunks, tokens, context):
    return (min(chunks, batch) * tokens + batch) * context


# ---------------------------------------------------------------------------
# what a case's sizes imply


def _new_tokens(case):
    """New tokens of each sequence: ragged chunks first, then single tokens."""
    c = case["tokens"]
    return [max(1, c - b * 7919 % (c // 3 + 1)) if b < case["chunks"] else 1
            for b in range(case["batch"])]


def _lens(case):
    """Tokens of each sequence with its new ones: ragged, the first the longest."""
    n = case["context"]
    return [max(t, n - b * 6571 % (n // 2 + 1)) for b, t in enumerate(_new_tokens(case))]


def _max_pages(case):
    return -(-max(_lens(case)) // case["page"])


def _pages_needed(case):
    """New pages of each sequence."""
    ps = case["page"]
    return [-(-L // ps) - -(-(L - n) // ps) for L, n in zip(_lens(case), _new_tokens(case))]


def _bytes(name):
    return 2 if name == "bf16" else 4


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def work(case):
    """plan: every length, free page and table entry in use read once, tokens'
    positions and slots and new pages written once. append: inputs read,
    outputs written. chunk: every cached key read once for its sequence, queries
    read, outputs written; the scores of all pairs (values are read only where a
    weight is not zero, which the sizes do not say)."""
    if case["op"] == "plan":
        new, need = _new_tokens(case), _pages_needed(case)
        return {"bytes": 16 * case["batch"] + 8 * _plan_rows(case) + 8 * sum(need),
                "flops": sum(new)}
    H, G, D = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        n = case["rows"]
        io = (H + 2 * G) * _bytes(case["x"]) + H * _bytes(case["q"]) + 2 * G * _bytes(case["kv"])
        return {"bytes": n * (D * io + 4 * case["axes"] + 4), "flops": 8 * n * (H + G) * D}
    new, lens = _new_tokens(case), _lens(case)
    pairs = sum(n * (2 * L - n + 1) // 2 for n, L in zip(new, lens))
    return {"bytes": sum(lens) * G * D * _bytes(case["kv"])
            + sum(new) * H * (2 * D * _bytes(case["q"]) + 4),
            "flops": 2 * pairs * H * D}


def _plan_rows(case):
    """Token rows of the step's batch: padded, as a captured graph has them."""
    return -(-sum(_new_tokens(case)) // 64) * 64


# ---------------------------------------------------------------------------
# inputs


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    s = {"plan": _prepare_plan, "append": _prepare_append,
         "chunk": _prepare_chunk}[case["op"]](case, gen)
    s["case"] = case
    if own:
        s["call"] = _call(s)
    return s


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _prepare_plan(case, gen):
    """Pages in random order; the sequences in another order for every seed, so
    that the chunks lie anywhere; `short` fewer free pages than are wanted."""
    B, ps, mp = case["batch"], case["page"], _max_pages(case)
    order = torch.randperm(B, generator=gen, device=DEVICE)
    new, lens = _i32(_new_tokens(case))[order], _i32(_lens(case))[order]
    old = lens - new
    wanted = sum(_pages_needed(case))
    in_use = sum(_lens(case)) // ps + B
    pages = torch.randperm(in_use + wanted + 64, generator=gen, device=DEVICE).to(torch.int32)
    held = (old.long() + ps - 1) // ps
    first = torch.cumsum(held, 0) - held
    at = torch.arange(mp, device=DEVICE)
    table = torch.where(at < held[:, None], pages[(first[:, None] + at).clamp(max=in_use - 1)], -1)
    free = pages[in_use:].clone()
    rows = _plan_rows(case)
    return {"seq_lens": old, "new_tokens": new, "block_table": table.contiguous(), "free_pages": free,
            "free_count": _i32([max(1, wanted - case["short"]) if case["short"] else len(free)]),
            "num_pages": len(pages), "rows": rows,
            "new_lens": torch.empty_like(old), "token_starts": _i32([0] * (B + 1)),
            "positions": _i32([0]).expand(rows).contiguous(),
            "slots": _i32([0]).expand(rows).contiguous(), "free_left": _i32([0])}


def _normal(gen, shape, dtype, scale=1.0):
    x = torch.empty(shape, dtype=dtype, device=DEVICE).normal_(generator=gen)
    return x if scale == 1.0 else x.mul_(scale)


def _prepare_append(case, gen):
    """One projection's output a token: its queries, keys and values next to
    each other. Every token has a slot but each 50th, which is padding."""
    n, H, G, D, ps = (case[k] for k in ("rows", "heads", "kv_heads", "dim", "page"))
    x = _normal(gen, (n, (H + 2 * G) * D), _dtype(case["x"]))
    s = {"q": x[:, :H * D].view(n, H, D), "k": x[:, H * D:(H + G) * D].view(n, G, D),
         "v": x[:, (H + G) * D:].view(n, G, D)}
    pages = -(-n // ps) + 1
    slots = torch.randperm(pages * ps, generator=gen, device=DEVICE)[:n].to(torch.int32)
    slots[49::50] = -1
    s["slots"] = slots
    kv = _dtype(case["kv"])
    s["k_pool"] = torch.zeros((pages, G, ps, D), dtype=kv, device=DEVICE)
    s["v_pool"] = torch.zeros((pages, G, ps, D), dtype=kv, device=DEVICE)
    s["q_out"] = torch.empty((n, H, D), dtype=_dtype(case["q"]), device=DEVICE)
    s["positions"] = torch.randint(0, case["context"], (case["axes"], n), generator=gen,
                                   device=DEVICE, dtype=torch.int32)
    half = case["rot"] // 2
    s["freqs"] = s["pair_axis"] = s["q_weight"] = s["k_weight"] = None
    if half:
        e = torch.arange(half, dtype=torch.float64, device=DEVICE) / half
        s["freqs"] = 500000.0 ** -e
    if case["axes"] > 1:
        s["pair_axis"] = torch.randint(0, case["axes"], (half,), generator=gen, device=DEVICE,
                                       dtype=torch.int32).sort().values
    if case["norm"]:
        s["q_weight"] = 1.0 + _normal(gen, (D,), torch.float32, 0.2)
        s["k_weight"] = 1.0 + _normal(gen, (D,), torch.float32, 0.2)
    s["q_scale"] = 1.0 / math.sqrt(D)
    return s


def _prepare_chunk(case, gen):
    """Keys and values N(0, 1); queries N(0, (2.5 / sqrt(dim))^2): scores of a
    few units, pre-scaled as the library takes them; pages in random order."""
    B, H, G, D, ps = (case[k] for k in ("batch", "heads", "kv_heads", "dim", "page"))
    new, lens, mp = _new_tokens(case), _lens(case), _max_pages(case)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    pages = sum(-(-L // ps) for L in lens)
    order = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32)
    table, at = [], 0
    for L in lens:
        held = -(-L // ps)
        table.append(torch.nn.functional.pad(order[at:at + held], (0, mp - held), value=-1))
        at += held
    kv, q = _dtype(case["kv"]), _dtype(case["q"])
    return {"seq_lens": _i32(lens), "token_starts": _i32(starts), "block_table": torch.stack(table),
            "k_pool": _normal(gen, (pages, G, ps, D), kv),
            "v_pool": _normal(gen, (pages, G, ps, D), kv),
            "q": _normal(gen, (starts[-1], H, D), q, 2.5 / math.sqrt(D)),
            "out": torch.empty((starts[-1], H, D), dtype=q, device=DEVICE),
            "tau": torch.empty((starts[-1], H), device=DEVICE)}


# ---------------------------------------------------------------------------
# the operators


def _call(s):
    """The library's call on this state, its arguments marshalled once as a
    serving loop keeps it."""
    from sparse_long_context_page_amd import entmaxkv as E
    c = s["case"]
    if c["op"] == "plan":
        shape = E.make_shape(c["batch"], 1, 1, 64, c["page"], _max_pages(c), s["num_pages"], "bf16")
        return E.Prepared("plan_tokens", shape, s["seq_lens"], s["new_tokens"], s["free_pages"],
                          s["free_count"], s["block_table"], s["new_lens"], s["token_starts"],
                          s["positions"], s["slots"], s["free_left"])
    if c["op"] == "append":
        shape = E.make_shape(1, c["heads"], c["kv_heads"], c["dim"], c["page"], 1,
                             s["k_pool"].shape[0], c["kv"])
        return E.Prepared("append_kv", shape, s["q"], s["k"], s["v"], s["positions"], s["slots"],
                          s["q_out"], s["k_pool"], s["v_pool"], freqs=s["freqs"],
                          pair_axis=s["pair_axis"], interleaved=c["interleaved"],
                          q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6,
                          q_scale=s["q_scale"])
    shape = E.make_shape(c["batch"], c["heads"], c["kv_heads"], c["dim"], c["page"], _max_pages(c),
                         s["k_pool"].shape[0], c["kv"])
    return E.Prepared("entmax_chunk", shape, s["q"], s["token_starts"], s["k_pool"], s["v_pool"],
                      s["block_table"], s["seq_lens"], c["alpha"], s["out"], tau=s["tau"])


def run(state):
    op = state["case"]["op"]
    if own:
        state["call"]()
    else:
        {"plan": _plan, "append": _append, "chunk": _chunk}[op](state)
    return [state[k] for k in {"plan": ("block_table", "new_lens", "token_starts", "positions",
                                        "slots", "free_left"),
                               "append": ("q_out", "k_pool", "v_pool"),
                               "chunk": ("out", "tau")}[op]]


def _plan(s):
    c = s["case"]
    ps, N = c["page"], s["rows"]
    table, free, have = s["block_table"], s["free_pages"].long(), s["free_count"].long()
    L = s["seq_lens"].long()
    n = s["new_tokens"].long().clamp(min=0)
    end = torch.cumsum(n, 0)
    start = end - n
    fits = (L + n <= table.shape[1] * ps) & (end <= N)
    held = (L + ps - 1) // ps
    need = torch.where(fits, (L + n + ps - 1) // ps - held, 0)
    upto = torch.cumsum(need, 0)
    granted = fits & ((need == 0) | (upto <= have))
    s["new_lens"].copy_(torch.where(granted, L + n, L))
    s["token_starts"][1:] = end.clamp(max=N)
    s["free_left"].copy_(have - torch.where(granted, need, 0).sum())
    at = torch.arange(table.shape[1], device=DEVICE)
    i = at - held[:, None]
    mine = granted[:, None] & (i >= 0) & (i < need[:, None])
    pick = (have - 1 - (upto - need)[:, None] - i).clamp(0, len(free) - 1)
    table.copy_(torch.where(mine, free[pick], table.long()))
    r = torch.arange(N, device=DEVICE)
    b = torch.searchsorted(end, r, right=True)
    real = b < len(L)
    b = b.clamp(max=len(L) - 1)
    pos = torch.where(real, L[b] + r - start[b], 0)
    live = real & granted[b]
    page = table[b, torch.where(live, pos // ps, 0)].long()
    live &= (page >= 0) & (page < s["num_pages"])
    s["positions"].copy_(pos)
    s["slots"].copy_(torch.where(live, page * ps + pos % ps, -1))


def _normed(x, weight):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight


def _rotated(x, cos, sin, interleaved):
    half = cos.shape[-1]
    if half == 0:
        return x
    y = x.clone()
    a = x[..., 0:2 * half:2] if interleaved else x[..., :half]
    b = x[..., 1:2 * half:2] if interleaved else x[..., half:2 * half]
    pair = a * cos - b * sin, a * sin + b * cos
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = pair
    else:
        y[..., :half], y[..., half:2 * half] = pair
    return y


def _append(s):
    c = s["case"]
    G, ps = c["kv_heads"], c["page"]
    n, half = c["rows"], c["rot"] // 2
    pos = s["positions"].double()
    if half:
        axis = s["pair_axis"].long() if c["axes"] > 1 else torch.zeros(half, dtype=torch.long,
                                                                       device=DEVICE)
        angle = pos[axis].T * s["freqs"]  # 64 bits: float32 loses the angles of far positions
        cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    else:
        cos = sin = torch.empty((n, 1, 0), device=DEVICE)
    q = _rotated(_normed(s["q"], s["q_weight"]), cos, sin, c["interleaved"]) * s["q_scale"]
    k = _rotated(_normed(s["k"], s["k_weight"]), cos, sin, c["interleaved"])
    s["q_out"].copy_(q)
    live = s["slots"] >= 0
    slot = s["slots"][live].long()
    page, row, g = slot[:, None] // ps, slot[:, None] % ps, torch.arange(G, device=DEVICE)
    s["k_pool"][page, g, row] = k[live].to(s["k_pool"].dtype)
    s["v_pool"][page, g, row] = s["v"][live].to(s["v_pool"].dtype)


def _power(u, m):
    """u^m of u >= 0; the whole exponents by products."""
    if m == 1.0:
        return u
    if m == 2.0:
        return u * u
    if m == 4.0:
        return (u * u) * (u * u)
    return u.pow(m)


def _entmax(x, v):
    """x = (alpha - 1) z with hidden tokens at -inf, [..., T]; the threshold by
    Newton's steps on ||(x - tau)_+||_m = 1, a convex function of tau, from
    below; the weights' product with v."""
    def solve(m):
        top = x.amax(-1, keepdim=True)
        tau = top - 1.0
        for _ in range(10):
            u = (x - tau).clamp_min(0.0)
            p = _power(u, m)
            total = p.sum(-1, keepdim=True)
            slope = (u > 0).sum(-1, keepdim=True) if m == 1.0 else _power(u, m - 1.0).sum(
                -1, keepdim=True)
            tau = tau + (total - total.pow(1.0 - 1.0 / m)) / slope
            tau = torch.minimum(tau, top)
        p = _power((x - tau).clamp_min(0.0), m)
        return (p @ v) / p.sum(-1, keepdim=True), tau.squeeze(-1)
    return solve


def _chunk(s):
    c = s["case"]
    B, H, G, D, ps = (c[k] for k in ("batch", "heads", "kv_heads", "dim", "page"))
    a = c["alpha"]
    m = 1.0 / (a - 1.0)
    new, lens = _new_tokens(c), _lens(c)
    start = 0
    b = 0
    while b < B:
        n = new[b]
        if n > 1:
            k, v = (s[x][s["block_table"][b, :-(-lens[b] // ps)].long()].float().transpose(0, 1)
                    .reshape(G, -1, D)[:, :lens[b]] for x in ("k_pool", "v_pool"))
            k = k.transpose(1, 2).contiguous()
            step = max(1, (1 << 29) // (H * lens[b]))
            for i in range(0, n, step):
                w = min(step, n - i)
                rows = slice(start + i, start + i + w)
                T = lens[b] - n + i + w  # no query of these sees a later token
                q = s["q"][rows].float().view(w, G, H // G, D).transpose(0, 1).reshape(G, -1, D)
                x = (a - 1.0) * (q @ k[:, :, :T].contiguous()).view(G, w, H // G, T)
                pos = lens[b] - n + i + torch.arange(w, device=DEVICE)[:, None, None]
                x.masked_fill_(torch.arange(T, device=DEVICE) > pos, -torch.inf)
                o, tau = _entmax(x.view(G, -1, T), v[:, :T])(m)
                s["out"][rows] = (o.view(G, w, H // G, D).transpose(0, 1).reshape(w, H, D)
                                  .to(s["out"].dtype))
                s["tau"][rows] = tau.view(G, w, H // G).transpose(0, 1).reshape(w, H)
            start += n
            b += 1
            continue
        e = b
        most = max(1, (1 << 31) // (G * D * max(lens)))  # sequences of one token, as many at once
        while e < B and new[e] == 1 and e - b < most:
            e += 1
        T = max(lens[b:e])
        pages = s["block_table"][b:e, :-(-T // ps)].long().clamp(min=0)
        k, v = (s[x][pages].float().transpose(1, 2).reshape(e - b, G, -1, D)[:, :, :T]
                for x in ("k_pool", "v_pool"))
        rows = slice(start, start + e - b)
        q = s["q"][rows].float().view(e - b, G, H // G, D)
        x = (a - 1.0) * (q @ k.transpose(2, 3).contiguous())
        past = torch.arange(T, device=DEVICE) >= s["seq_lens"][b:e, None, None, None]
        x.masked_fill_(past, -torch.inf)
        o, tau = _entmax(x, v)(m)
        s["out"][rows] = o.reshape(e - b, H, D).to(s["out"].dtype)
        s["tau"][rows] = tau.reshape(e - b, H)
        start += e - b
        b = e


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _plan_exact, "append": _append64, "chunk": _chunk64}[case["op"]](s)


def _plan_exact(s):
    """Sequence by sequence, page by page."""
    c = s["case"]
    ps, N, cap = c["page"], s["rows"], _max_pages(c) * c["page"]
    table = s["block_table"].cpu().numpy().copy()
    free, have = s["free_pages"].tolist(), int(s["free_count"][0])
    lens, starts = [], [0]
    positions, slots = [0] * N, [-1] * N
    row = wanted = taken = 0
    for b, (L, n) in enumerate(zip(s["seq_lens"].tolist(), s["new_tokens"].tolist())):
        ok = L + n <= cap and row + n <= N
        pages = range(-(-L // ps), -(-(L + n) // ps)) if ok else range(0)
        wanted += len(pages)
        ok = ok and (not pages or wanted <= have)
        if ok:
            for i, j in enumerate(pages):
                table[b, j] = free[have - 1 - (wanted - len(pages) + i)]
            taken += len(pages)
        for i in range(n):
            if row + i < N:
                positions[row + i] = L + i
                if ok:
                    slots[row + i] = int(table[b, (L + i) // ps]) * ps + (L + i) % ps
        row += n
        starts.append(min(row, N))
        lens.append(L + n if ok else L)
    return [torch.tensor(x, dtype=torch.int32, device=DEVICE)
            for x in (table, lens, starts, positions, slots, [have - taken])]


def _append64(s):
    c = s["case"]
    n, D, half = c["rows"], c["dim"], c["rot"] // 2
    turn = torch.zeros((n, half), dtype=torch.complex128, device=DEVICE)
    for i in range(half):
        axis = 0 if s["pair_axis"] is None else int(s["pair_axis"][i])
        angle = s["positions"][axis].double() * s["freqs"][i]
        turn[:, i] = torch.polar(torch.ones_like(angle), angle)
    if c["interleaved"]:
        first = torch.arange(half, device=DEVICE) * 2
        second = first + 1
    else:
        first = torch.arange(half, device=DEVICE)
        second = first + half

    def finished(x, weight):
        y = x.double()
        if weight is not None:
            y = y / torch.sqrt(y.square().sum(2, keepdim=True) / D + 1e-6) * weight.double()
        if half:
            z = torch.complex(y[:, :, first], y[:, :, second]) * turn[:, None, :]
            y = y.index_copy(2, first, z.real).index_copy(2, second, z.imag)
        return y

    pools = []
    k = finished(s["k"], s["k_weight"])
    live = torch.nonzero(s["slots"] >= 0).flatten()
    for pool, rows in ((s["k_pool"], k), (s["v_pool"], s["v"].double())):
        by_slot = pool.double().transpose(1, 2).reshape(-1, c["kv_heads"], D)
        by_slot[s["slots"][live].long()] = rows[live]
        pools.append(by_slot.view(pool.shape[0], c["page"], c["kv_heads"], D).transpose(1, 2)
                     .contiguous())
    return [finished(s["q"], s["q_weight"]) * s["q_scale"], *pools]


def _chunk64(s):
    c = s["case"]
    G, R, m = c["kv_heads"], c["heads"] // c["kv_heads"], 1.0 / (c["alpha"] - 1.0)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    taus = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEVICE)
    starts, lens = s["token_starts"].tolist(), _lens(c)
    for b, L in enumerate(lens):
        pages = s["block_table"][b, :-(-L // c["page"])].long()
        for g in range(G):
            k = s["k_pool"][pages, g].reshape(-1, c["dim"])[:L].double()
            v = s["v_pool"][pages, g].reshape(-1, c["dim"])[:L].double()
            for lo in range(starts[b], starts[b + 1], 1024):
                hi = min(lo + 1024, starts[b + 1])
                last = L - starts[b + 1] + torch.arange(lo, hi, device=DEVICE)
                for h in range(g * R, (g + 1) * R):
                    z = s["q"][lo:hi, h].double() @ k.t().contiguous() * (c["alpha"] - 1.0)
                    z[torch.arange(L, device=DEVICE)[None] > last[:, None]] = -torch.inf
                    above = z.max(1, keepdim=True).values
                    below = above - 1.0
                    for _ in range(46):  # halves of a bracket of 1
                        mid = (above + below) / 2
                        small = torch.relu(z - mid).pow_(m).sum(1, keepdim=True) < 1.0
                        above = torch.where(small, mid, above)
                        below = torch.where(small, below, mid)
                    p = torch.relu(z - below) ** m
                    out[lo:hi, h] = (p @ v) / p.sum(1, keepdim=True)
                    taus[lo:hi, h] = below[:, 0]
    return [out, taus]
