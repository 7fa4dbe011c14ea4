"""Steps of a PagedWindow on streams given as torch streams and as numbers (cudaStream_t), as every
other call takes them."""
import pytest
import torch

from block_causal_attention_b200 import _abi
from block_causal_attention_b200.streaming import PagedWindow
from test_gpu_paged import BF, gen, rand

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
