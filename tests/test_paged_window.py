"""Several videos' denoising windows over one paged cache (PagedWindow): the operators run
together as a server runs them, against the 64-bit plain forms and against the plan of the same
window over a contiguous cache."""
import math

import numpy as np
import pytest
import torch

import paged_ref as ref
from block_causal_attention_b200 import Plan, _abi
from block_causal_attention_b200.streaming import PagedWindow, PipelinedWindow

PAGE = 128


def test_layout_on_the_host():
    """Tables, starts and key ranges of a step against their definition in absolute tokens."""
    w = PagedWindow(4, 2, 24, 2, 7, 5, window=3, cache_chunks=4, kv_range=2, videos=3, host_only=True)
    C = w.chunk_tokens
    assert C == 70
    a, b = w.open(), w.open(5)
    w.add_transition(a, 1, [0, 1], 0)
    where = {}                                   # (video, token) -> (page, slot)
    for step in range(9):
        vids = [a, b] if step % 2 else [b, a]
        table, starts, seen = w.layout(vids)
        assert w.pending_copies == []
        assert (table < w.pool.pages).all()
        for i, v in enumerate(vids):
            f = w.first_chunk(v)
            base = f * C - starts[i]
            assert base % PAGE == 0 and base >= 0
            for t in range(3 * C):
                p = (starts[i] + t) // PAGE
                assert table[i, p] >= 0
                where[v, f * C + t] = (table[i, p], (starts[i] + t) % PAGE)
            for p in range(3):
                row, lo, hi = seen[3 * i + p]
                c = f + p
                r = 0 if (v == a and c == 1 and p in (0, 1)) else 2
                assert row == i and hi == (c + 1) * C - base
                oldest = {a: 0, b: 5}[v]
                assert lo == (c - min(r, c - oldest, 4 + p)) * C - base >= 0
                for t in range(lo + base, (c + 1) * C):   # tokens of earlier steps lie where they were
                    j = t - base
                    assert (table[i, j // PAGE], j % PAGE) == where[v, t]
        owned = [p for v in vids for p in w.pool.row(v) if p >= 0]
        assert len(set(owned)) == len(owned)     # nothing shared without a fork
        w.slide(a)
        if step % 3 == 0:
            w.slide(b)
    assert w.pool.free_pages > 0
    with pytest.raises(ValueError):
        w.layout([a, a])
    with pytest.raises(KeyError):
        w.layout([99])
    w.close_video(a)
    with pytest.raises(KeyError):
        w.slide(a)


def test_copies_outlive_a_step_that_finds_no_page():
    w = PagedWindow(2, 1, 24, 1, 10, 20, window=2, cache_chunks=1, kv_range=1, videos=2, pages=9, host_only=True)
    a = w.open()
    w.layout([a])                                # 400 tokens: 4 pages
    w.slide(a)
    w.layout([a])                                # tokens 200 .. 600: one page more, none released
    b, c = w.fork(a), w.fork(a)
    for v in (a, b, c):
        w.slide(v)                               # tokens 400 .. 800; page 1 holds the cached chunk's first tokens
    with pytest.raises(MemoryError):
        w.layout([a, b, c])                      # 3 copies and 2 new pages for a; not enough for b
    done = list(w.pending_copies)
    assert len(done) >= 1 and len({x for _, x in done}) == len(done)
    w.close_video(b)
    w.close_video(c)
    w.layout([a])
    assert w.pending_copies[:len(done)] == done


class History:
    """The last key and value written for each token of a video, in 64 bits."""

    def __init__(self, other=None):
        self.k, self.v = (dict(other.k), dict(other.v)) if other else ({}, {})


@pytest.mark.gpu
@pytest.mark.parametrize("d,hq,hkv,dtype", [(48, 16, 2, torch.bfloat16), (24, 6, 2, torch.float16), (32, 4, 4, torch.bfloat16)])
def test_windows_of_several_videos(d, hq, hkv, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    frames, height, width, window = 2, 7, 5, 3
    w = PagedWindow(hq, hkv, d, frames, height, width, window, cache_chunks=4, kv_range=2, videos=3, layers=2, dtype=dtype)
    C, kt = w.chunk_tokens, 2.0 ** -11
    w.cache.k_pages.fill_(math.nan)              # whatever a page held before must not matter
    w.cache.v_pages.fill_(math.nan)
    gain = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    a, b = w.open(), w.open(3)
    w.add_transition(a, 4, [2], 1)
    hist = {a: [History(), History()], b: [History(), History()]}
    videos = [a, b]
    for step in range(8):
        if step == 3:                            # a takes two ways from here
            c = w.fork(a)
            hist[c] = [History(h) for h in hist[a]]
            videos = [c, b, a]
        if step == 5:
            w.close_video(b)
            videos = [a, c]
        if step == 6:
            assert w.compact() > 0
        s = w.begin(videos)
        assert s.rows == len(videos) * window * C
        for layer in range(2):
            q = torch.empty((s.rows, hq, d), dtype=dtype, device="cuda").normal_(generator=g)
            k = torch.empty((s.rows, hkv, d), dtype=dtype, device="cuda").normal_(generator=g)
            v = torch.empty((s.rows, hkv, d), dtype=dtype, device="cuda").normal_(generator=g)
            lse = torch.empty((hq, s.rows), device="cuda")
            o = w.run(s, q, k, v, layer=layer, q_gain=gain, k_gain=gain, lse=lse)
            assert w.cache.status() == _abi.BCA_OK
            # attention against what the pages hold
            kp, vp = w.cache.k_pages[layer], w.cache.v_pages[layer]
            seq, kb, ke, off = (x.tolist() for x in (s.seq, s.k_begin, s.k_end, s.slice_off))
            rows = torch.arange(0, s.rows, 17).tolist()
            wo, wl, bo, bl = ref.attend_rows(q, kp, vp, s.table, off, seq, kb, ke, rows, s.pos, gain)
            for got, want, bound in ((o[rows].double(), wo, bo), (lse[:, rows].double(), wl, bl)):
                assert ((got - want).abs() <= bound).all()
            # and the pages against what was written, at the positions of the video
            kh = ref.prologue(k, s.pos, gain)
            for i, vid in enumerate(videos):
                first = w.first_chunk(vid)
                h = hist[vid][layer]
                for t in range(window * C):
                    h.k[first * C + t], h.v[first * C + t] = kh[i * window * C + t], v[i * window * C + t]
                base = first * C - s.start[i].item()
                lo = min(kb[i * window:(i + 1) * window])
                pk, pv = ref.unpage(kp, vp, s.table[i].tolist(), ke[(i + 1) * window - 1])
                for j in range(lo, ke[(i + 1) * window - 1]):
                    want = h.k[base + j]
                    assert ((pk[j] - want).abs() <= kt * want.abs() + 2.0 ** -20 * want.abs().amax() + 2.0 ** -25).all()
                    assert (pv[j] == h.v[base + j].double()).all()
            frame = s.pos[:, 0].view(len(videos), window, frames, height * width)
            for i, vid in enumerate(videos):
                want = torch.arange(window * frames, device="cuda").view(window, frames, 1) + w.first_chunk(vid) * frames
                assert (frame[i] == want).all()
        for vid in videos:
            w.slide(vid)
    w.close()


@pytest.mark.gpu
def test_a_window_over_pages_equals_the_plan_over_a_contiguous_cache():
    """The same step by Plan.fwd (keys of earlier chunks contiguous) and by PagedWindow: two
    kernels, each within its bound of the same 64-bit values."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    hq, hkv, d, frames, height, width, window, nc, r = 8, 2, 48, 2, 9, 8, 2, 3, 2
    w = PagedWindow(hq, hkv, d, frames, height, width, window, nc, r, videos=1)
    sched = PipelinedWindow(hq, hkv, d, frames, height, width, window, nc, r, host_only=True)
    C = w.chunk_tokens
    vid = w.open()
    bf = torch.bfloat16
    for step in range(6):
        first = w.first_chunk(vid)
        s = w.begin([vid])
        q, k, v = (torch.empty((window * C, h, d), dtype=bf, device="cuda").normal_(generator=g) for h in (hq, hkv, hkv))
        lse = torch.empty((hq, window * C), device="cuda")
        o = w.run(s, q, k, v, lse=lse)
        assert w.cache.status() == _abi.BCA_OK
        if first >= nc:
            pk, pv = ref.unpage(w.cache.k_pages[0], w.cache.v_pages[0], s.table[0].tolist(), (s.start[0].item()))
            kc, vc = pk[-nc * C:].half().contiguous(), pv[-nc * C:].to(bf).contiguous()
            plan = Plan(hq, hkv, d, sched.videos(first), nc * C, sched.slices(sched.ranges(first)), cache_k_fp16=True)
            o2, lse2 = plan.fwd(q, k, v, kc, vc)
            assert plan.status() == _abi.BCA_OK
            rows = list(range(window * C))
            wo, wl, bo, bl = ref.attend_rows(q, w.cache.k_pages[0], w.cache.v_pages[0], s.table, s.slice_off.tolist(),
                                             s.seq.tolist(), s.k_begin.tolist(), s.k_end.tolist(), rows, s.pos, None)
            assert ((o.double() - wo).abs() <= bo).all() and ((lse.double() - wl).abs() <= bl).all()
            # the plan rounds each new key to fp16 itself (half a step of its own: 2^-11 of a score) and
            # scales its queries before rounding them
            assert ((o2.double() - wo).abs() <= 2 * bo).all() and ((lse2.double() - wl).abs() <= 2 * bl).all()
        w.slide(vid)
