"""The default workspace's first use by a serving call on another stream, and inside a capture."""
import pytest
import torch

from test_serve8 import gen, i32, int8_operand, ss  # noqa: F401 (ss: the fixture)

pytestmark = pytest.mark.gpu


def append_with_a_bad_page(ss, **kw):  # noqa: F811
    cache = ss.kv_cache(4, 1, 64, page=16)
    x = torch.randn(3, 1, 64, generator=gen(1), device="cuda").bfloat16()
    args = (cache, x, x, i32([[99]]), i32([0, 3]), i32([3]))
    torch.cuda.synchronize()
    return lambda: ss.kv_append(*args, **kw)


def test_the_first_use_on_another_stream_is_ordered(ss, monkeypatch):  # noqa: F811
    """The current stream is busy: a clear of the new workspace that waited there would come after the call and erase
    what it recorded."""
    s = torch.cuda.Stream()
    append_with_a_bad_page(ss, ws=ss.Workspace())()  # the kernel is loaded
    call = append_with_a_bad_page(ss, stream=s)
    monkeypatch.setattr(ss, "_default_ws", {})
    # memory that was not zero before, if the allocator hands it out again
    n = ss.lib().ss24_workspace_bytes() + 256
    torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    call()
    s.synchronize()
    torch.cuda.synchronize()
    assert ss.default_workspace(torch.device("cuda", torch.cuda.current_device())).error() == 16


def test_the_first_use_inside_a_capture(ss, monkeypatch):  # noqa: F811
    """Its workspace is the graph's own: calls outside do not find one that only a replay clears."""
    a, b = int8_operand(5, 64, 1), int8_operand(40, 64, 2)
    call = append_with_a_bad_page(ss)
    ss.gemm_int8(a, b)
    torch.cuda.synchronize()
    monkeypatch.setattr(ss, "_default_ws", {})
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ss.gemm_int8(a, b)
    ws = ss.default_workspace(torch.device("cuda", torch.cuda.current_device()))
    assert ws.error() == 0
    call()
    assert ws.error() == 16
    graph.replay()
    torch.cuda.synchronize()
    assert ws.error() == 16
    assert torch.equal(y, ss.gemm_int8(a, b))
    del graph
