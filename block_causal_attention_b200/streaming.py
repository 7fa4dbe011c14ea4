"""The pipelined denoising window with a KV range per denoising stage.

MAGI-1 generates a video chunk by chunk: a window of consecutive chunks is denoised
together, the oldest chunk (least noise) at the front and the newest (most noise) at the
back, and each step the window slides by one chunk; fully denoised chunks leave the window
and their keys and values stay in a KV cache (MAGI-1 research notes, "Inference tricks >
KV Cache"; the pipelined denoising of the "Magi-1 开源&刷屏" article).  The KV range limits
how many earlier chunks a chunk attends to (a range of 8: each new chunk depends on the 8
chunks before it), and changing the range at chosen denoising stages gives controllable
transitions: a range of 1 at the high-noise stages changes the shot while keeping the
subject, a range of 1 at the low-noise stages keeps the layout and changes the details
(same page).

Readings taken here (the pages give the idea, not the indexing):
  * a window of W chunks; window position p = 0 .. W-1 from the least to the most noisy
    chunk, so a chunk's denoising stage is its window position and it moves to p - 1 each
    step;
  * KV range R: the chunk at absolute index c sees chunks [c - R, c] (fully), taken from the
    cache for chunks before the window and from the window itself (block-causal);
  * the cache holds the `cache_chunks` chunks just before the window, oldest first;
  * a transition at chunk X with stages S: while chunk X sits at a window position in S, its
    range is `transition_range` instead of the normal one.

The slice list of a step depends only on the ranges of the W window positions, so plans are
compiled once per distinct range tuple and reused: each step only moves the plan's start
frame (``Plan.update_positions``), which rewrites the RoPE tables and nothing else.

Two forms: ``PipelinedWindow`` drives plans over a contiguous cache of one video; ``PagedWindow``
drives any number of videos, each at its own chunk, over one paged cache, where keys and values
are written once and stay, and a video can be forked.
"""
from __future__ import annotations

import time
from dataclasses import dataclass
from typing import Any, Dict, Iterable, List, Optional, Sequence, Tuple

import numpy as np

from . import Plan


class PipelinedWindow:
    """Plans for the W-chunk denoising window of one video, one per distinct KV-range
    layout, moved to each step's frames on demand."""

    def __init__(self, hq: int, hkv: int, d: int, frames: int, height: int, width: int, window: int,
                 cache_chunks: int, kv_range: int, rope_base=(1e4, 1e4, 1e4), eps: float = 1e-6,
                 o_fp32: bool = False, host_only: bool = False):
        if window < 1 or cache_chunks < 0 or kv_range < 0:
            raise ValueError("window >= 1, cache_chunks >= 0 and kv_range >= 0 are required")
        self.hq, self.hkv, self.d = hq, hkv, d
        self.frames, self.height, self.width = frames, height, width
        self.window, self.cache_chunks, self.kv_range = window, cache_chunks, kv_range
        self.rope_base, self.eps, self.o_fp32, self.host_only = tuple(rope_base), eps, o_fp32, host_only
        self.chunk_tokens = frames * height * width
        self.transitions: Dict[int, Tuple[frozenset, int]] = {}
        self._plans: Dict[Tuple[int, ...], Plan] = {}
        self.compiles = 0                 # plans compiled so far (one per distinct layout)
        self.last_host_ms = 0.0           # host time of the last plan() call

    # ------------------------------------------------------------------ schedule
    def add_transition(self, chunk: int, stages: Iterable[int], kv_range: int = 1) -> None:
        """While `chunk` is at one of the window positions `stages`, it sees only the
        `kv_range` chunks before it."""
        self.transitions[int(chunk)] = (frozenset(int(s) for s in stages), int(kv_range))

    def ranges(self, first_chunk: int) -> Tuple[int, ...]:
        """KV range of each window position when the window starts at absolute chunk
        `first_chunk`, clipped to the chunks that exist (the cache and the window)."""
        out = []
        for p in range(self.window):
            c = first_chunk + p
            r = self.kv_range
            tr = self.transitions.get(c)
            if tr is not None and p in tr[0]:
                r = tr[1]
            out.append(min(r, self.cache_chunks + p, c))
        return tuple(out)

    def slices(self, ranges: Sequence[int]) -> np.ndarray:
        """One FULL slice per window chunk: position p sees keys of chunks
        [cache + p - R_p, cache + p] of the [cache | window] key space."""
        C, nc = self.chunk_tokens, self.cache_chunks
        out = [(p * C, (p + 1) * C, (nc + p - int(r)) * C, (nc + p + 1) * C, 0) for p, r in enumerate(ranges)]
        return np.asarray(out, np.int64)

    def videos(self, first_chunk: int) -> np.ndarray:
        return np.asarray([[self.window, self.frames, self.height, self.width, first_chunk * self.frames]], np.int32)

    # ------------------------------------------------------------------ plans
    def plan(self, first_chunk: int, stream=None) -> Plan:
        """The plan of the step whose window starts at absolute chunk `first_chunk`: the
        cached plan of its range layout, moved to the window's frames (compiled the first
        time the layout appears).  The cache given to the plan's fwd must hold the
        `cache_chunks` chunks before the window ([Nc, Hkv, D], Nc = cache_chunks * C)."""
        t = time.perf_counter()
        rg = self.ranges(first_chunk)
        vids = self.videos(first_chunk)
        p = self._plans.get(rg)
        if p is None:
            p = Plan(self.hq, self.hkv, self.d, vids, self.cache_chunks * self.chunk_tokens, self.slices(rg),
                     self.rope_base, self.eps, self.o_fp32, host_only=self.host_only)
            self._plans[rg] = p
            self.compiles += 1
        else:
            p.update_positions(vids, stream=stream)
        self.last_host_ms = (time.perf_counter() - t) * 1e3
        return p

    def close(self) -> None:
        for p in self._plans.values():
            p.close()
        self._plans.clear()


@dataclass
class PagedStep:
    """What the layers of one step of a ``PagedWindow`` share: which videos, where their tokens
    go and what they see (int32 tensors on the cache's device)."""
    videos: Tuple[int, ...]
    rows: int                # tokens of all windows
    table: Any               # [videos, width]
    row_off: Any             # [videos + 1] rows of each video
    start: Any               # [videos] first token of each window in its table row
    slice_off: Any           # [videos * window + 1] rows of each chunk
    seq: Any
    k_begin: Any
    k_end: Any
    pos: Any                 # [rows, 3]
    made: Tuple[int, ...]    # when the videos' pages last changed hands, as ``begin`` found it


class PagedWindow:
    """The denoising windows of several videos over one paged KV cache.

    Every video has the same geometry and its own window position (``open(first_chunk)``,
    ``slide``), KV-range transitions and pages.  A step: ``begin(videos)`` once, then ``run`` for
    each layer with the windows' tokens of all those videos, row after row.  The keys and values
    of a window chunk are written anew each step; the last ones, from the step before the chunk
    leaves the window, are what later chunks read.  ``fork`` continues a video in two ways: the
    pages are shared until one of the two writes to them.

    A step says where its videos' tokens lie as ``begin`` found it: once one of them has been forked,
    has slid or was closed, or ``compact`` has moved pages, ``run`` refuses it (ValueError), since the
    pages may be shared or another video's by then.  A step that was begun has to be run for all
    layers: pages of the window that were shared are replaced by ``begin``, and not copied where each
    of their tokens is about to be written.

    Pages change hands between videos, so the calls of one window belong on one stream, or on
    streams that the caller puts in the order of the calls."""

    def __init__(self, hq: int, hkv: int, d: int, frames: int, height: int, width: int, window: int,
                 cache_chunks: int, kv_range: int, videos: int, layers: int = 1, rope_base=(1e4, 1e4, 1e4),
                 eps: float = 1e-6, dtype=None, o_fp32: bool = False, pages: Optional[int] = None,
                 host_only: bool = False):
        """videos: how many are open at most; pages: the pool's size (default: enough for that
        many windows with their caches, nothing shared)."""
        from .paged import PAGE, PagedCache, PagePool
        self._page = PAGE
        self._schedule = lambda: PipelinedWindow(hq, hkv, d, frames, height, width, window, cache_chunks, kv_range,
                                                 rope_base, eps, o_fp32, host_only=True)
        geometry = self._schedule()
        self.frames, self.height, self.width, self.window = frames, height, width, window
        self.cache_chunks, self.chunk_tokens = cache_chunks, geometry.chunk_tokens
        span = (cache_chunks + window + 1) * self.chunk_tokens   # while a window slides, one chunk more
        pages = videos * (-(-span // PAGE) + 1) if pages is None else pages
        self.cache = PagedCache(hq, hkv, d, pages, layers=layers, dtype=dtype, rope_base=rope_base, eps=eps,
                                o_fp32=o_fp32, host_only=host_only)
        self.pool = PagePool(pages)
        self._videos: Dict[int, PipelinedWindow] = {}
        self._first: Dict[int, int] = {}
        self._oldest: Dict[int, int] = {}    # the first chunk that was ever in the window
        self._moved: Dict[int, int] = {}     # the event after which steps of the video are out of date
        self._events = 0
        self.pending_copies: List[Tuple[int, int]] = []   # that the tables count on already

    # ------------------------------------------------------------------ videos
    def open(self, first_chunk: int = 0) -> int:
        """A new video whose window starts at absolute chunk `first_chunk`.  Chunks before that
        one were never written: no range reaches them."""
        if first_chunk < 0:
            raise ValueError("first_chunk >= 0 is required")
        video = self.pool.open()
        self._videos[video], self._first[video] = self._schedule(), first_chunk
        self._oldest[video] = first_chunk
        self._out_of_date(video)
        return video

    def _out_of_date(self, *videos: int) -> None:
        """Steps of these videos begun so far no longer hold."""
        self._events += 1
        for v in videos:
            self._moved[v] = self._events

    def _get(self, video: int) -> PipelinedWindow:
        if video not in self._videos:
            raise KeyError(f"no open video {video}")
        return self._videos[video]

    def first_chunk(self, video: int) -> int:
        self._get(video)
        return self._first[video]

    def add_transition(self, video: int, chunk: int, stages: Iterable[int], kv_range: int = 1) -> None:
        self._get(video).add_transition(chunk, stages, kv_range)

    def slide(self, video: int) -> None:
        """The window moves on by one chunk; pages that no window chunk can see any more go back."""
        self._get(video)
        self._out_of_date(video)
        self._first[video] += 1
        self.pool.release_before(video, (self._first[video] - self.cache_chunks) * self.chunk_tokens)

    def fork(self, video: int) -> int:
        old = self._get(video)
        new = self.pool.fork(video)
        self._videos[new], self._first[new] = self._schedule(), self._first[video]
        self._oldest[new] = self._oldest[video]
        self._videos[new].transitions.update(old.transitions)
        self._out_of_date(video, new)
        return new

    def close_video(self, video: int) -> None:
        self._get(video)
        self.pool.close(video)
        del self._videos[video], self._first[video], self._oldest[video], self._moved[video]

    def compact(self, stream=None) -> int:
        """Move the pages in use to the front of the pool; returns how many moved.  If any did, steps
        begun before hold old tables: begin them again."""
        self._copy_pending(stream)
        self.pending_copies = self.pool.compact()
        if self.pending_copies:
            self._out_of_date(*self._videos)
        return self._copy_pending(stream)

    def _copy_pending(self, stream) -> int:
        n = len(self.pending_copies)
        if n:
            self.cache.copy_pages(self.pending_copies, stream=stream)
            self.pending_copies = []
        return n

    # ------------------------------------------------------------------ steps
    def layout(self, videos: Sequence[int]):
        """The host side of ``begin``: (table, first token of each window in its row, (table row,
        begin, end) of the keys of each window chunk).  Copies of shared pages that have to be made
        first are added to ``pending_copies`` (also when the pool runs out half way)."""
        if len(set(videos)) != len(videos):
            raise ValueError("a video can be in a step once")
        C, starts, seen, bases = self.chunk_tokens, [], [], []
        for v in videos:   # all checked before any page is taken
            self._get(v)
        for b, v in enumerate(videos):
            first = self._first[v]
            self.pending_copies += self.pool.grow(v, first * C, (first + self.window) * C)
            oldest = self._oldest[v]
            base = max(oldest, first - self.cache_chunks) * C // self._page * self._page   # the row's first page
            bases.append(base // self._page)
            starts.append(first * C - base)
            for p, r in enumerate(self._videos[v].ranges(first)):
                seen.append((b, (first + p - min(r, first + p - oldest)) * C - base, (first + p + 1) * C - base))
        rows = [self.pool.row(v, skip) for v, skip in zip(videos, bases)]
        table = np.full((len(rows), max((len(r) for r in rows), default=0)), -1, np.int32)
        for b, r in enumerate(rows):
            table[b, :len(r)] = r
        return table, starts, seen

    def begin(self, videos: Sequence[int], stream=None) -> PagedStep:
        """Pages for the windows of `videos` (copied first where they are shared) and the step's
        device data: new tensors each time, uploaded from pageable memory, so this waits for the
        stream and cannot be captured, and a graph captured over ``run`` goes on reading its own
        step's."""
        import torch

        from .paged import on_stream
        self._copy_pending(stream)   # of a step that found no page: before new ones can build on them
        table, starts, seen = self.layout(videos)
        with on_stream(stream, self.cache.device):
            self._copy_pending(stream)
            dev, C, per = self.cache.device, self.chunk_tokens, self.window * self.chunk_tokens
            n, i32 = len(videos) * per, torch.int32
            small = torch.tensor(starts + [x for row in seen for x in row], dtype=i32).to(dev)
            keys = small[len(starts):].view(-1, 3).t().contiguous()
            t = torch.arange(per, dtype=i32, device=dev)
            plane = self.height * self.width
            pos = torch.stack([t // plane, t % plane // self.width, t % self.width], 1).repeat(len(videos), 1)
            begun = torch.tensor([self._first[v] * self.frames for v in videos], dtype=i32).to(dev)
            pos[:, 0] += begun.repeat_interleave(per)
            return PagedStep(tuple(videos), n, torch.from_numpy(table).to(dev),
                             torch.arange(0, n + 1, per, dtype=i32, device=dev), small[:len(starts)],
                             torch.arange(0, n + 1, C, dtype=i32, device=dev), keys[0], keys[1], keys[2], pos,
                             tuple(self._moved[v] for v in videos))

    def run(self, step: PagedStep, q, k, v, *, layer: int = 0, q_gain=None, k_gain=None, o=None, lse=None,
            stream=None):
        """Write k, v [rows, Hkv, D] of the step's windows and attend q [rows, Hq, D]; returns o."""
        if step.made != tuple(self._moved.get(v) for v in step.videos):
            raise ValueError("the step is out of date: one of its videos was forked, slid or closed, or pages were "
                             "compacted; begin it again")
        if k.shape[0] != step.rows or q.shape[0] != step.rows:
            raise ValueError(f"expected {step.rows} rows of q, k and v")
        self.cache.write(k, v, step.table, step.row_off, step.start, pos=step.pos, k_gain=k_gain, layer=layer,
                         stream=stream)
        return self.cache.attend(q, step.table, step.slice_off, step.k_begin, step.k_end, seq=step.seq, pos=step.pos,
                                 q_gain=q_gain, layer=layer, o=o, lse=lse, stream=stream)

    def close(self) -> None:
        self.cache.close()
