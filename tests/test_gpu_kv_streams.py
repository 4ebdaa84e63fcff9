"""The paged cache's calls on another stream than torch's current one, while work is queued on
that one: neither may use memory that the other still uses."""

import threading
import types

import numpy as np
import pytest
import torch

import test_gpu_kv as T
from test_gpu_kv import BF16, F8, _lib, make_batch, make_cache, randn  # noqa: F401

pytestmark = pytest.mark.gpu
BUSY = 100_000_000  # clocks that the current stream is kept busy: some 50 ms


def _setup(dtype, lens, rows):
    rng = np.random.default_rng(60)
    pages = sum(-(-n // 64) for n in lens)
    cache = make_cache(rng, pages, 64, 2, 128, BF16 if dtype == "bf16" else F8)
    batch, _, _ = make_batch(rng, pages, 64, lens, rows)
    return cache, batch, randn(rng, batch.num_rows, 8, 128)


def _dirt(*sizes):
    """Writes queued on the current stream to memory that is free for its next allocations."""
    x = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    for t in x:
        t.fill_(255)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,rows", [([9000, 300], None), ([1500, 40], [600, 1])])
def test_results_and_scratch_are_not_memory_of_queued_work(lens, rows, dtype):
    cache, batch, q = _setup(dtype, lens, rows)
    ws = T.F.Workspace()
    want = T.F.kv_attention(cache, batch, q, workspace=ws)
    need = ws.buf.numel() - 256
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(BUSY)
        _dirt(q.numel() * 2, want[1].numel() * 4, need)
        got = T.F.kv_attention(cache, batch, q, stream=side)
        side.synchronize()
        held = [x.clone() for x in got]  # queued behind the writes
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_append_results_are_not_memory_of_queued_work(dtype):
    cache, batch, q = _setup(dtype, [300, 70], [200, 3])
    rng = np.random.default_rng(61)
    k, v = (randn(rng, batch.num_rows, 2, 128) for _ in range(2))
    f = torch.full((64,), 0.01, device="cuda")
    want = T.F.kv_append(cache, batch, k, v, q=q, inv_freq=f)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    _dirt(q.numel() * 2)
    got = T.F.kv_append(cache, batch, k, v, q=q, inv_freq=f, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_arguments_dropped_at_once_outlive_the_call(dtype):
    """The side stream is the busy one: temporaries that the caller drops are handed out for
    later work of the current stream only when the call has read them."""
    cache, batch, q = _setup(dtype, [9000, 300], None)
    want = T.F.kv_attention(cache, batch, q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    mine = q.clone()
    torch.cuda.current_stream().synchronize()
    got = T.F.kv_attention(cache, batch, mine, stream=side)
    del mine
    _dirt(q.numel() * 2)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_a_workspace_that_grows_while_another_stream_uses_it(dtype):
    small, large = _setup(dtype, [9000, 300], None), _setup(dtype, [60000, 20000], [200, 1])
    want = [T.F.kv_attention(c, b, q) for c, b, q in (small, large)]
    torch.cuda.synchronize()
    ws, side = T.F.Workspace(), torch.cuda.Stream()
    T.F.kv_attention(*small, workspace=ws)
    old = ws.buf.numel()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    got = [T.F.kv_attention(*small, workspace=ws, stream=side)]
    got.append(T.F.kv_attention(*large, workspace=ws))  # drops the buffer that `side` will use
    assert ws.buf.numel() > old
    _dirt(old)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_a_workspace_knows_the_streams_it_was_used_on():
    ws, side = T.F.Workspace(), torch.cuda.Stream()
    a = ws.get(1000, side)
    assert ws._home == side.cuda_stream and a.data_ptr() % 256 == 0 and a.numel() == 1000
    assert ws.get(500).data_ptr() == a.data_ptr()
    with torch.cuda.stream(side):
        assert ws.get(1000).data_ptr() == a.data_ptr()
        ws.get(5000)
    assert ws._home == side.cuda_stream
    ws.get(9000)
    assert ws._home == torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_a_forked_stream_inside_a_capture(dtype):
    """Append on the captured stream, two attentions side by side on it and on a stream that
    forks from it; replays after other work has used the memory in between."""
    cache, batch, q = _setup(dtype, [9000, 1500, 300], [1, 200, 2])
    rng = np.random.default_rng(62)
    k, v = (randn(rng, batch.num_rows, 2, 128) for _ in range(2))
    f = torch.full((64,), 0.01, device="cuda")
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        qr = T.F.kv_append(cache, batch, k, v, q=q, inv_freq=f)
        side.wait_stream(here)
        full = T.F.kv_attention(cache, batch, qr, stream=side)
        win = T.F.kv_attention(cache, batch, qr, window=200, sinks=4)
        here.wait_stream(side)
        return (qr, *full, *win)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(3):
        for x in (k, v, q):
            x.copy_(randn(rng, *x.shape))
        _dirt(q.numel() * 2, 1 << 20)
        g.replay()
        torch.cuda.synchronize()
        held = [x.clone() for x in got]
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b)


def test_calls_from_several_threads():
    """Each thread with a stream of its own, calls of every kind at once."""
    jobs = [_setup(d, lens, rows) for d, lens, rows in (
        ("bf16", [9000, 300], None), ("e4m3", [9000, 300], None), ("bf16", [1500, 40], [600, 1]),
        ("e4m3", [1500, 40], [600, 1]))]
    want = [T.F.kv_attention(*j) for j in jobs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for n in range(20):
                    j = (i + n) % len(jobs)
                    with pytest.raises(T.F.FathomError, match="negative"):
                        T.F.kv_attention(*jobs[j], window=-1 - i)
                    got = T.F.kv_attention(*jobs[j])
                    torch.cuda.current_stream().synchronize()
                    if not (torch.equal(got[0], want[j][0]) and torch.equal(got[1], want[j][1])):
                        wrong.append((i, n))
        except BaseException as e:  # noqa: B902
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]


def test_a_stream_of_another_device_is_refused():
    """The default streams of two devices have one handle: the device decides."""
    cache, batch, q = _setup("bf16", [300], None)
    other = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(ValueError, match="the stream on cuda:1"):
        T.F.kv_attention(cache, batch, q, stream=other)
    with pytest.raises(ValueError, match="the stream on cuda:1"):
        T.F.kv_append(cache, batch, q[:, :2], q[:, :2], stream=other)
    T.F.kv_attention(cache, batch, q, stream=torch.cuda.default_stream())
