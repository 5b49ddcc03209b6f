"""A workspace that a call allocates by itself belongs to the stream that its
kernels run on: memory that another stream has just given up, and may still be
reading, is not for it, and what is freed goes to work that follows on its own
stream."""
import pytest
import torch

from test_gpu_chunk import E

pytestmark = pytest.mark.gpu


def owner(t):
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not in a segment of the allocator")


@pytest.mark.parametrize("given", ["stream", "handle"])
def test_workspace_of_a_side_stream(given):
    q, st = torch.zeros(4, device="cuda"), torch.cuda.Stream()
    ptr, n, ws = E()._given_or_new(None, 12345, q, st if given == "stream" else st.cuda_stream)
    assert (ptr.value, n) == (ws.data_ptr(), 12345)
    assert owner(ws) == st.cuda_stream
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


def test_workspace_of_the_null_stream_from_another():
    q, st = torch.zeros(4, device="cuda"), torch.cuda.Stream()
    with torch.cuda.stream(st):
        assert owner(E()._given_or_new(None, 54321, q, 0)[2]) == 0
        assert owner(E()._given_or_new(None, 54321, q, None)[2]) == st.cuda_stream
        assert torch.cuda.current_stream() == st
