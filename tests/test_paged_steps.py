"""Steps of a PagedWindow on the host: a step whose tables no longer say where its videos' pages are
is refused before anything is written."""
from types import SimpleNamespace

import pytest
import torch

from block_causal_attention_b200.streaming import PagedWindow

C = 200                                              # tokens of a chunk


def window(**kw):
    """A PagedWindow whose cache notes its calls in w.calls."""
    w = PagedWindow(2, 1, 24, 1, 10, 20, window=2, cache_chunks=2, kv_range=1, videos=4, host_only=True, **kw)
    w.calls = []

    def note(name):
        return lambda *a, **k: w.calls.append(name)
    w.cache = SimpleNamespace(device=torch.device("cpu"), write=note("write"), attend=note("attend"),
                              copy_pages=note("copy"))
    return w


def run(w, step):
    q = torch.zeros(step.rows, 2, 24)
    w.calls.clear()
    w.run(step, q, q[:, :1], q[:, :1])
    assert w.calls == ["write", "attend"]


def refused(w, step):
    q = torch.zeros(step.rows, 2, 24)
    w.calls.clear()
    with pytest.raises(ValueError, match="begin"):
        w.run(step, q, q[:, :1], q[:, :1])
    assert w.calls == []


def test_a_fork_after_begin():
    """The fork would find its parent's later keys in the pages that they share."""
    w = window()
    a, b = w.open(), w.open()
    one, both, other = w.begin([a]), w.begin([a, b]), w.begin([b])
    assert w.layout([a])[0].tolist() == one.table.tolist()
    c = w.fork(a)
    assert set(w.pool.row(c)) == set(one.table[0].tolist())
    refused(w, one)
    refused(w, both)
    run(w, other)
    run(w, w.begin([c]))
    run(w, w.begin([a, b, c]))


def test_a_slide_after_begin():
    """Pages behind the window go back to the pool and may be another video's."""
    w = window()
    a, b = w.open(), w.open()
    for _ in range(5):
        old, other = w.begin([a]), w.begin([b])
        run(w, old)
        run(w, old)                                  # layer after layer
        w.slide(a)
        refused(w, old)
        run(w, other)
        run(w, w.begin([a, b]))


def test_a_closed_video():
    w = window()
    a, b = w.open(), w.open()
    both, other = w.begin([b, a]), w.begin([b])
    w.close_video(a)
    refused(w, both)
    run(w, other)
    assert w.open() != a                             # a number is given once


def test_compaction_that_moves_pages():
    w = window()
    a, b = w.open(), w.open()
    w.begin([a])
    step = w.begin([b])
    assert w.compact() == 0
    run(w, step)                                     # nothing moved
    w.close_video(a)
    assert w.compact() > 0
    refused(w, step)
    run(w, w.begin([b]))


def test_a_second_begin_leaves_the_first_step_usable():
    w = window()
    a, b = w.open(), w.open()
    first = w.begin([a, b])
    again = w.begin([a, b])
    assert first.table.tolist() == again.table.tolist()
    w.add_transition(a, 9, [0])
    run(w, first)
    run(w, again)
