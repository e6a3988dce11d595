"""Memory that the package allocates for a call on an explicit stream comes from that stream's own."""
import contextlib

import pytest
import torch

import _kv
import weight_only_quantized_w4a16_amd as wq


def test_memory_is_allocated_on_the_launching_stream(monkeypatch):
    """(CPU) With another stream given, memory is allocated under it; what is returned is recorded on the current one."""
    seen = []

    class Stream:
        def __init__(self, handle):
            self.cuda_stream, self.device_index, self.device = handle, 0, torch.device("cuda", 0)

    class Tensor:
        def __init__(self):
            self.made_on, self.recorded = list(active), []

        def record_stream(self, s):
            self.recorded.append(s)

    active = []

    @contextlib.contextmanager
    def under(s):
        active.append(s)
        yield
        active.pop()

    class Like:
        device = torch.device("cuda", 0)

        def new_empty(self, shape, dtype):
            seen.append((shape, dtype))
            return Tensor()

    side, current = Stream(7), Stream(3)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: current.cuda_stream, raising=False)
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: current)
    for stream in (None, current):
        t = wq._empty(stream, Like(), (2, 3))
        assert t.made_on == [] and t.recorded == []
    t = wq._empty(side, Like(), (2, 3))
    assert t.made_on == [side] and t.recorded == [current]
    t = wq._empty(side, Like(), 64, torch.uint8, scratch=True)
    assert t.made_on == [side] and t.recorded == []
    assert seen == [((2, 3), None)] * 3 + [(64, torch.uint8)] and active == []


@pytest.fixture()
def busy():
    """The current stream with a while of work ahead of it."""
    wq.lib()
    a = torch.randn(4096, 4096, device="cuda").half()
    b = torch.empty_like(a)
    torch.cuda.synchronize()

    def start():
        for _ in range(40):
            torch.mm(a, a, out=b)
    return start


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.gpu
def test_attention_on_another_stream_beside_pending_work(busy):
    """Scratch and outputs released on the current stream with their work still ahead are not what a call on another
    stream writes to."""
    P = _kv.Problem([3000], [1], 2, 128, 128, 16, torch.float16, 3)
    cache = P.empty(wq)
    P.fill(wq, cache)
    args = (cache, P.table.cuda(), i32([3000]))
    q1, q2 = (torch.randn(1, 8, 128).half().cuda() for _ in range(2))
    assert wq.wq_kv_workspace_bytes(1, 1, False, 8, 2, 128, 128, args[1].shape[1] * 16) > 0
    want1, want2 = wq.wq_kv_attention(q1, *args).clone(), wq.wq_kv_attention(q2, *args).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept = torch.empty_like(want1)
    busy()
    out = wq.wq_kv_attention(q1, *args)      # its scratch is released here, its work is still to come
    kept.copy_(out)
    at = out.data_ptr()
    del out
    got = wq.wq_kv_attention(q2, *args, stream=side)
    assert got.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(kept, want1) and torch.equal(got, want2)
    # the other way round, into the caller's memory
    outs = [torch.empty_like(q1) for _ in range(2)]
    torch.cuda.synchronize()
    busy()
    for q, o, s in ((q1, outs[0], None), (q2, outs[1], side)):
        wq.wq_kv_attention(q, *args, out=o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want1) and torch.equal(outs[1], want2)


@pytest.mark.gpu
def test_rows_and_rotations_on_another_stream_beside_pending_work(busy):
    P = _kv.Problem([100], [1], 2, 64, 64, 16, torch.float16, 4)
    cache = P.empty(wq)
    P.fill(wq, cache)
    args = (cache, P.table.cuda(), i32([100]), 100)
    side = torch.cuda.Stream()
    x = torch.randn(64, 512).half().cuda()
    want = [t.clone() for t in wq.wq_kv_read(*args)] + [wq.wq_hadamard(x, 64).clone()]
    torch.cuda.synchronize()
    busy()
    held = [torch.full_like(t, 7) for t in want]
    at = {t.data_ptr() for t in held}
    del held
    got = list(wq.wq_kv_read(*args, stream=side)) + [wq.wq_hadamard(x, 64, stream=side)]
    assert not at & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.gpu
def test_products_on_another_stream_beside_pending_work(busy):
    """A product whose scratch (permuted activations, partial sums of a K split) was just released elsewhere."""
    import workloads as wl
    from _util import repack_layer
    L = wl.make_layer(2048, 256, 4, 128, wl.ZERO_F16, 5, act_order=True)
    layer = repack_layer(wq, L)
    M = 40
    assert wq.wq_workspace_bytes(M, 256, 2048, 4, True) > M * 2048 * 2
    x1, x2 = (torch.randn(M, 2048).half().cuda() for _ in range(2))
    want1, want2 = wq.linear(x1, layer).clone(), wq.linear(x2, layer).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept = torch.empty_like(want1)
    busy()
    out = wq.linear(x1, layer)
    kept.copy_(out)
    at = out.data_ptr()
    del out
    got = wq.linear(x2, layer, stream=side)
    w = wq.wq_dequant_debug(layer, torch.float16, stream=side)
    assert got.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(kept, want1) and torch.equal(got, want2)
    assert torch.equal(w, wq.wq_dequant_debug(layer, torch.float16))


@pytest.mark.gpu
def test_a_captured_branch_on_another_stream():
    """A graph whose capture forks to a second stream: outputs and scratch of the calls on it come from the graph's own
    memory, and every replay gives the eager results."""
    P = _kv.Problem([3000], [1], 2, 128, 128, 16, torch.float16, 3)
    cache = P.empty(wq)
    P.fill(wq, cache)
    args = (cache, P.table.cuda(), i32([3000]))
    q = torch.randn(1, 8, 128).half().cuda()
    x = torch.randn(64, 512).half().cuda()
    assert wq.wq_kv_workspace_bytes(1, 1, False, 8, 2, 128, 128, args[1].shape[1] * 16) > 0
    for _ in range(2):
        wq.wq_kv_attention(q, *args), wq.wq_hadamard(x, 64)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        a = wq.wq_kv_attention(q, *args, stream=side)
        k, v = wq.wq_kv_read(*args, 1, stream=side)
        b = wq.wq_kv_attention(q, *args)
        r = wq.wq_hadamard(x, 64, stream=side)
        main.wait_stream(side)
    for i in range(4):
        q.copy_(torch.randn(1, 8, 128, generator=torch.Generator().manual_seed(i)))
        x.mul_(0.5)
        want = wq.wq_kv_attention(q, *args)
        want_k, want_v = wq.wq_kv_read(*args, 1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want) and torch.equal(r, wq.wq_hadamard(x, 64)), i
        assert torch.equal(k, want_k) and torch.equal(v, want_v), i
