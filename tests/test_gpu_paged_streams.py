"""Streams: steps of a PagedWindow on ones given as torch streams and as numbers (cudaStream_t), as every
other call takes them, and captured calls side by side."""
import pytest
import torch

import paged_ref as ref
from block_causal_attention_b200 import PagedCache, _abi
from block_causal_attention_b200.streaming import PagedWindow
from test_gpu_paged import BF, gen, rand, widened

pytestmark = pytest.mark.gpu


def test_steps_on_streams_given_as_numbers():
    outs = []
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream, 0):
        g = gen(41)
        w = PagedWindow(4, 2, 24, 1, 10, 20, window=2, cache_chunks=2, kv_range=2, videos=3)
        a = w.open()
        x = [[rand((2 * 2 * 200, h, 24), BF, g) for h in (4, 2, 2)] for _ in range(3)]
        torch.cuda.synchronize()
        got = []
        for step in range(3):
            b = w.fork(a)                            # its pages are copied by the next begin
            s = w.begin([a, b], stream=stream)
            got.append(w.run(s, *x[step], stream=stream))
            w.close_video(b)
            w.compact(stream=stream)
            w.slide(a)
        assert w.cache.status(stream) == _abi.BCA_OK
        torch.cuda.synchronize()
        outs.append([o.clone() for o in got])
    assert all(torch.equal(o, p) for out in outs[1:] for o, p in zip(out, outs[0]))


def test_workspaces_on_streams_given_as_numbers():
    w = PagedWindow(4, 2, 24, 1, 10, 20, window=2, cache_chunks=2, kv_range=2, videos=1)
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream, 0):
        assert w.cache.alloc_workspace(50, 2, 300, stream=stream).numel() >= w.cache.workspace_bytes(50, 2, 300) > 0


def test_two_captured_calls_replayed_at_once():
    """Two graphs with a workspace each, side by side on two streams, again and again."""
    g = gen(42)
    kp, vp = ref.pools(80, 2, 48, BF, g)
    cache = PagedCache(16, 2, 48, 80, k_pages=kp, v_pages=vp)
    table = ref.table_of([40, 40], 80, g)
    runs = []
    for n in (1, 3, 20, 60, 300):                    # tiles of 16, 32, 128 and 384 rows, and clusters
        for wide in (False, True):
            t = widened(table) if wide else table
            q = rand((2 * n, 16, 48), BF, g)
            args = (q, t, ref.i32([0, n, 2 * n]), ref.i32([3, 0]), ref.i32([5001, 4700]))
            want = cache.attend(*args, causal=True)
            o, ws = torch.empty_like(q), cache.alloc_workspace(2 * n, 2, t.shape[1])
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                cache.attend(*args, causal=True, o=o, workspace=ws)
            runs.append((graph, o, want, args, ws))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(len(runs)):
        pair = (runs[i], runs[(i + 3) % len(runs)])
        for x in pair:
            x[1].zero_()
        torch.cuda.synchronize()
        for _ in range(10):
            for s, x in zip(streams, pair):
                with torch.cuda.stream(s):
                    x[0].replay()
        torch.cuda.synchronize()
        assert cache.status() == _abi.BCA_OK
        assert all(torch.equal(x[1], x[2]) for x in pair)
