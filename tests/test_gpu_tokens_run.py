"""The calls of a serving step together: plan, norm and rotation, append, page
boxes, prompt chunks and then single tokens by the chunk and the decode calls;
captured in a graph, on other streams, from two threads of work at once."""
import math

import numpy as np
import pytest
import torch

from oracle import tokens_oracle as T
from parity_util import announce

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def E():
    from sparse_long_context_page_amd import entmaxkv
    return entmaxkv


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


class Server:
    """A cache, its free pages and the state of a few sequences."""

    def __init__(self, batch=3, H=8, G=2, D=64, ps=16, mp=12, pages=40, rows=128, kv="bf16"):
        self.dims = batch, H, G, D, ps, mp, pages
        self.kv_t = BF if kv == "bf16" else F32
        self.shape = E().make_shape(batch, H, G, D, ps, mp, pages, kv)
        self.k, self.v = (torch.full((pages, G, ps, D), math.nan, dtype=self.kv_t, device="cuda")
                          for _ in range(2))
        self.meta = torch.zeros((pages, G, 2, D), dtype=self.kv_t, device="cuda")
        self.table = i32(np.full((batch, mp), -1))
        order = np.random.default_rng(0).permutation(pages)
        self.free, self.count = i32(order), [i32([pages]), i32([0])]
        self.lens = [i32([0] * batch), i32([0] * batch)]
        self.rows = rows
        self.starts, self.pos, self.slots = i32([0] * (batch + 1)), i32([0] * rows), i32([0] * rows)
        self.freqs = 10000.0 ** -(torch.arange(D // 2, dtype=torch.float64, device="cuda") / (D // 2))
        rng = np.random.default_rng(1)  # the same weights for every server
        self.qw, self.kw = (torch.from_numpy(rng.uniform(0.5, 1.5, D).astype(np.float32)).cuda()
                            for _ in range(2))
        self.x = torch.zeros((rows, (H + 2 * G) * D), dtype=BF, device="cuda")
        self.new = i32([0] * batch)
        self.q = torch.zeros((rows, H, D), device="cuda")
        self.out, self.tau = torch.zeros((rows, H, D), device="cuda"), torch.zeros(rows, H, device="cuda")
        self.ws = torch.empty(E().entmaxkv_entmax_chunk_ws(self.shape, rows, 1.5), dtype=torch.uint8,
                              device="cuda")
        self.turn = 0

    def parts(self):
        _, H, G, D, *_ = self.dims
        x = self.x
        return (x[:, :H * D].view(-1, H, D), x[:, H * D:(H + G) * D].view(-1, G, D),
                x[:, (H + G) * D:].view(-1, G, D))

    def step(self, stream=None):
        """One step of the tokens in self.new and self.x."""
        e, t = E(), self.turn
        kw = dict(stream=stream)
        e.entmaxkv_plan_tokens(self.shape, self.lens[t], self.new, self.free, self.count[t], self.table,
                               self.lens[1 - t], self.starts, self.pos, self.slots,
                               self.count[1 - t], **kw)
        q, k, v = self.parts()
        e.entmaxkv_append_kv(self.shape, q, k, v, self.pos, self.slots, self.q, self.k, self.v,
                             freqs=self.freqs, q_weight=self.qw, k_weight=self.kw, q_scale=0.3, **kw)
        e.entmaxkv_append_page_meta(self.shape, self.k, self.table, self.lens[t], self.lens[1 - t],
                                    self.rows, self.meta, **kw)
        e.entmaxkv_entmax_chunk(self.shape, self.q, self.starts, self.k, self.v, self.table,
                                self.lens[1 - t], 1.5, self.out, tau=self.tau, ws=self.ws, **kw)

    def feed(self, new, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.new.copy_(i32(new))
        self.x.normal_(generator=gen)

    def check(self):
        """The step just made against the oracle on the cache as it is."""
        B, H, G, D, ps, mp, pages = self.dims
        used = int(self.starts[-1])
        lens = self.lens[1 - self.turn].tolist()
        k, v = self.k.double().cpu().numpy(), self.v.double().cpu().numpy()
        table = self.table.cpu().numpy()
        q = self.q.double().cpu().numpy()
        starts = self.starts.tolist()
        # the appended keys: the oracle's norm and rotation, once rounded
        pos, slots = self.pos.cpu().numpy(), self.slots.cpu().numpy()
        xk = T.rotate(T.norm(self.parts()[1].double().cpu().numpy(), self.kw.cpu().numpy(), 1e-6),
                      pos[None], self.freqs.cpu().numpy())
        for r in range(used):
            if slots[r] >= 0:
                got = k[slots[r] // ps, :, slots[r] % ps]
                assert np.allclose(got, xk[r], rtol=2.0**-8, atol=1e-5)
                assert (v[slots[r] // ps, :, slots[r] % ps]
                        == self.parts()[2][r].double().cpu().numpy()).all()
        out, tau, _ = T.chunk(q[:used], starts, k, v, table, lens, 1.5)
        got = self.out.double().cpu().numpy()[:used]
        # (bf16 cache: the decode's tolerance)
        tol = 2e-3 * np.linalg.norm(out, axis=-1, keepdims=True) + 1e-6
        assert (np.abs(got - out) <= tol).all()
        # the boxes of the pages touched
        meta = torch.zeros_like(self.meta)
        E().entmaxkv_build_page_meta(self.shape, self.k, self.table, self.lens[1 - self.turn], meta)
        held = [table[b, :-(-L // ps)] for b, L in enumerate(lens)]
        idx = torch.from_numpy(np.concatenate(held).astype(np.int64)).cuda()
        assert torch.equal(meta[idx], self.meta[idx])
        return lens

    def advance(self):
        self.turn = 1 - self.turn


def test_a_serving_run():
    s = Server()
    free = s.dims[-1]
    want = [0, 0, 0]
    for i, new in enumerate([[50, 17, 0], [30, 1, 60], [1, 1, 1], [0, 40, 1], [1, 1, 1], [16, 0, 3]]):
        announce(f"serving step {i}: {new}")
        s.feed(new, i)
        s.step()
        torch.cuda.synchronize()
        lens = s.check()
        want = [a + b for a, b in zip(want, new)]
        assert lens == want
        free = s.dims[-1] - sum(-(-L // 16) for L in lens)
        assert int(s.count[1 - s.turn]) == free
        s.advance()
    # the last tokens once more by the decode calls
    s.feed([1, 1, 1], 99)
    s.step()
    lens = s.lens[1 - s.turn]
    B, H, G, D, ps, mp, pages = s.dims
    q = s.q[:3].contiguous()
    full = torch.empty((3, H, D), device="cuda")
    E().entmaxkv_decode_full(s.shape, q, s.k, s.v, s.table, lens, 1.5, full)
    sel = torch.empty((3, H, mp), dtype=I32, device="cuda")
    top = torch.empty_like(full)
    E().entmaxkv_decode_topk(s.shape, q, s.meta, s.k, s.v, s.table, lens, mp, 1.5, sel, top)
    tol = 2e-3 * full.norm(dim=-1, keepdim=True)
    assert ((s.out[:3] - full).abs() <= 2 * tol).all()
    assert ((top - full).abs() <= 2 * tol).all()  # every page selected: the full decode


def test_a_refused_sequence_waits_for_its_pages():
    s = Server(pages=6)
    s.feed([70, 40, 10], 1)  # 5 pages, then 3 too many, then 1 that the second may not lose
    s.step()
    torch.cuda.synchronize()
    assert s.lens[1].tolist() == [70, 0, 0] and int(s.count[1]) == 1
    assert (s.slots[70:120] == -1).all()
    # its rows attend to nothing: no token of theirs is in the cache
    assert (s.out[70:120] == 0).all() and s.tau[70:120].isnan().all()


def test_a_captured_step_replays():
    """Plan, append, boxes and attention in one graph, replayed with other lengths
    and values, eager work in between."""
    s, ref = Server(), Server()
    side = torch.cuda.Stream()
    for x in (s, ref):
        x.feed([20, 5, 33], 0)
        x.step()
        x.advance()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.step()
    keep = [x.clone() for x in (s.lens[1], s.count[1], s.table)]
    for i, new in enumerate([[1, 1, 1], [40, 0, 7], [0, 0, 0], [1, 30, 2]]):
        announce(f"replay {i}: {new}")
        for x in (s, ref):
            x.feed(new, 10 + i)
            x.lens[1].copy_(keep[0])
            x.count[1].copy_(keep[1])
            x.table.copy_(keep[2])
            x.out.zero_()
        graph.replay()
        ref.step()
        torch.cuda.synchronize()
        used = sum(new)
        assert torch.equal(s.table, ref.table) and torch.equal(s.slots, ref.slots)
        assert torch.equal(s.lens[0], ref.lens[0]) and torch.equal(s.out[:used], ref.out[:used])
        torch.randn(1 << 20, device="cuda").sum()


def test_two_streams_at_once():
    servers = [Server(), Server(kv="f32")]
    streams = [torch.cuda.Stream() for _ in servers]
    alone = []
    for i, s in enumerate(servers):
        s.feed([60, 3, 40], i)
        s.step()
        torch.cuda.synchronize()
        alone.append([x.clone() for x in (s.out, s.tau, s.slots, s.lens[1], s.k)])
    for _ in range(5):
        for s in servers:
            s.out.zero_()
            s.table.fill_(-1)
        torch.cuda.synchronize()
        for s, st in zip(servers, streams):
            s.step(stream=st)
        torch.cuda.synchronize()
        for s, want in zip(servers, alone):
            for x, y in zip((s.out, s.tau, s.slots, s.lens[1]), want):
                assert torch.equal(torch.nan_to_num(x.float(), 7.0), torch.nan_to_num(y.float(), 7.0))


def test_prepared_calls_equal_the_plain_ones():
    s = Server()
    s.feed([33, 1, 20], 4)
    s.step()
    torch.cuda.synchronize()
    want = [x.clone() for x in (s.out, s.slots, s.k)]
    s.table.fill_(-1)
    s.out.zero_()
    s.k.fill_(math.nan)
    q, k, v = s.parts()
    calls = [E().Prepared("plan_tokens", s.shape, s.lens[0], s.new, s.free, s.count[0], s.table,
                          s.lens[1], s.starts, s.pos, s.slots, s.count[1]),
             E().Prepared("append_kv", s.shape, q, k, v, s.pos, s.slots, s.q, s.k, s.v,
                          freqs=s.freqs, q_weight=s.qw, k_weight=s.kw, q_scale=0.3),
             E().Prepared("entmax_chunk", s.shape, s.q, s.starts, s.k, s.v, s.table, s.lens[1], 1.5,
                          s.out, tau=s.tau)]
    for c in calls:
        ev = E().HipEvents(2 * E().KERNELS[c.name.removeprefix("entmaxkv_")])
        c(events=list(ev))
        torch.cuda.synchronize()
        assert all(ev.elapsed_ms(2 * i, 2 * i + 1) >= 0 for i in range(len(ev) // 2))
    for x, y in zip((s.out, s.slots, s.k), want):
        assert torch.equal(torch.nan_to_num(x.float(), 7.0), torch.nan_to_num(y.float(), 7.0))


def test_workspace_allocated_by_the_call_on_another_stream():
    """Without ws the call allocates, and marks the memory as the stream's."""
    s = Server()
    s.feed([60, 3, 40], 5)
    s.step()
    torch.cuda.synchronize()
    want, st = s.out.clone(), torch.cuda.Stream()
    for _ in range(4):
        s.out.zero_()
        torch.cuda.synchronize()
        E().entmaxkv_entmax_chunk(s.shape, s.q, s.starts, s.k, s.v, s.table, s.lens[1], 1.5, s.out,
                                  stream=st)
        junk = [torch.full((1 << 20,), 3, dtype=torch.uint8, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        assert torch.equal(s.out, want)
        del junk
