"""Prepared calls: arguments by position or by name, and what a call costs
beside the library's own."""
import pytest
import torch

from test_abi import ek, shape  # noqa: F401


@pytest.fixture
def host(ek, monkeypatch):
    """Calls on host tensors that only note the library's arguments."""
    got = []

    def fn(*args):
        got.append([x if isinstance(x, (int, float)) else getattr(x, "value", None)
                    for x in args[1:]])
        return 0

    monkeypatch.setattr(ek, "_on_device", lambda **kw: None)
    monkeypatch.setattr(ek, "_stream", lambda stream, device: None)
    monkeypatch.setattr(ek.Prepared, "_makers", {
        name: (lambda make: lambda *a, **kw: (fn, *make(*a, **kw)[1:]))(make)
        for name, make in ek.Prepared._makers.items()})
    return got


def calls(ek):
    s = shape(ek, batch=2, num_q_heads=4, num_kv_heads=2, head_dim=64, page_size=16,
              max_pages_per_seq=3, num_phys_pages=9)
    bf, i32 = torch.bfloat16, torch.int32
    k, v = torch.zeros(9, 2, 16, 64, dtype=bf), torch.zeros(9, 2, 16, 64, dtype=bf)
    bt, lens = torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32)
    meta, q = torch.zeros(9, 2, 2, 64, dtype=bf), torch.zeros(2, 4, 64)
    out, lse, w = torch.zeros(2, 4, 64), torch.zeros(2, 4), torch.zeros(2, 2, 48)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    kept, nl = torch.zeros(2, 2, 20, dtype=i32), torch.zeros(2, dtype=i32)
    return {
        "build_page_meta": dict(shape=s, k_pool=k, block_table=bt, seq_lens=lens, meta=meta),
        "decode_full": dict(shape=s, q=q, k_pool=k, v_pool=v, block_table=bt, seq_lens=lens,
                            alpha=1.5, out=out, ws=ws),
        "softmax_window": dict(shape=s, q=q, k_pool=k, v_pool=v, block_table=bt, seq_lens=lens,
                               window=8, sinks=2, out=out, lse=lse, ws=ws),
        "accumulate_weights": dict(shape=s, q=q, k_pool=k, block_table=bt, seq_lens=lens,
                                   alpha=1.0, tau=lse, decay=0.5, weights_in=None, weights_out=w),
        "evict": dict(shape=s, k_pool=k, v_pool=v, block_table=bt, seq_lens=lens, weights=w,
                      keep=20, sinks=2, recent=3, new_table=bt, kept=kept, new_lens=nl),
    }


@pytest.mark.parametrize("name", ["build_page_meta", "decode_full", "softmax_window",
                                  "accumulate_weights", "evict"])
@pytest.mark.parametrize("gpus", [1, 2])
def test_arguments_by_name(ek, host, monkeypatch, name, gpus):
    monkeypatch.setattr(torch.cuda, "device_count", lambda: gpus)
    kw = calls(ek)[name]
    s, rest = kw["shape"], {x: y for x, y in kw.items() if x != "shape"}
    by_place = [y for x, y in rest.items() if x != "ws"]
    ws = {"ws": rest["ws"]} if "ws" in rest else {}
    ek.Prepared(name, s, *by_place, **ws)()
    ek.Prepared(name, s, **rest)()
    ek.Prepared(name, **kw)()
    assert len(host) == 3 and host[0] == host[1] == host[2]


def test_one_gpu_is_not_asked_for(ek, host, monkeypatch):
    """With one GPU there the current device is that one."""
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: pytest.fail("asked"))
    kw = calls(ek)["decode_full"]
    call = ek.Prepared("decode_full", **kw)
    assert call.device is None
    call()
    assert len(host) == 1
