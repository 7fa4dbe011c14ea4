"""The KV cache in pages: device operators (``PagedCache``) and page bookkeeping (``PagePool``).

A contiguous KV cache belongs to one video and is re-packed whenever its window slides.  In
pages of 128 tokens keys and values are written once and stay; several videos of any lengths
share one pool and one call; a fork shares its parent's pages until it writes (MAGI-1 research
notes, "Inference tricks > KV Cache": the cache of earlier chunks and its range).  The layouts
and the rules are in include/bca.h, "paged KV cache".
"""
from __future__ import annotations

import heapq
from typing import Dict, List, Optional, Sequence

import numpy as np

from . import _abi

PAGE = _abi.BCA_PAGE_TOKENS


def on_stream(stream, device):
    """The context of a stream given as a torch stream, as a number (cudaStream_t), or as None: the
    current one."""
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    return torch.cuda.stream(stream)


class PagedCache:
    """A pool of pages for `layers` layers and the operators on it: ``write`` new tokens,
    ``copy_pages`` and ``attend``.

    `dtype` (bf16 or fp16) is the type of q, k, v, o and the stored values; stored keys are
    fp16, post-prologue.  Calls run on `stream` (a torch stream, a number, or None: the current one)
    with the cache's device current; tensors of another stream have to stay alive, and their
    contents in place, until the call has run there.  `k_pages` / `v_pages` may be given (contiguous CUDA tensors of
    ``k_shape`` / ``v_shape``); otherwise they are allocated, uninitialised."""

    def __init__(self, hq: int, hkv: int, d: int, pages: int, *, layers: int = 1, dtype=None,
                 rope_base=(1e4, 1e4, 1e4), eps: float = 1e-6, o_fp32: bool = False, k_pages=None, v_pages=None,
                 host_only: bool = False, test_force_timeout: bool = False):
        import torch   # here and below: PagePool needs no PyTorch
        dtype = torch.bfloat16 if dtype is None else dtype
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"dtype: expected torch.bfloat16 or torch.float16, got {dtype}")
        desc = _abi.bca_paged_desc()
        desc.num_q_heads, desc.num_kv_heads, desc.head_dim = int(hq), int(hkv), int(d)
        desc.num_layers, desc.num_pages = int(layers), int(pages)
        desc.rope_base[:] = [float(x) for x in rope_base]
        desc.norm_eps = float(eps)
        desc.flags = (_abi.BCA_PAGED_FP16 if dtype == torch.float16 else 0) | (_abi.BCA_O_FP32 if o_fp32 else 0) | \
            (_abi.BCA_PLAN_HOST_ONLY if host_only else 0) | \
            (_abi.BCA_TEST_FORCE_TIMEOUT if test_force_timeout else 0)
        self._lib = _abi.lib()
        self._h = _abi.ctypes.c_void_p()
        _abi.check(self._lib.bca_paged_create(_abi.ctypes.byref(desc), _abi.ctypes.byref(self._h)),
                   "bca_paged_create")
        self.hq, self.hkv, self.d, self.pages, self.layers = int(hq), int(hkv), int(d), int(pages), int(layers)
        self.dtype, self.o_fp32, self.host_only = dtype, bool(o_fp32), bool(host_only)
        self.k_shape = (self.layers, self.pages, self.hkv, self.d // 8, PAGE, 8)
        self.v_shape = (self.layers, self.pages, self.hkv, PAGE // 8, self.d, 8)
        self.pool_bytes = int(self._lib.bca_paged_pool_bytes(self._h))
        self._pools: Dict[str, "torch.Tensor"] = {}
        self.device = None
        if self.host_only:
            return
        self.device = torch.device("cuda", torch.cuda.current_device())
        for name, t, dt, shape in (("k_pages", k_pages, torch.float16, self.k_shape),
                                   ("v_pages", v_pages, dtype, self.v_shape)):
            if t is None:
                t = torch.empty(shape, dtype=dt, device=self.device)
            elif t.dtype != dt or t.shape != shape or t.device != self.device or not t.is_contiguous():
                raise ValueError(f"{name}: expected a contiguous {dt} tensor of shape {shape} on {self.device}, got "
                                 f"{t.dtype} {tuple(t.shape)} on {t.device}")
            self._pools[name] = t
        self._calls = _abi.paged_binding()
        self._c = self._calls.cache(self._h.value, self.hq, self.hkv, self.d, self.layers, self.pool_bytes,
                                    self.k_pages.data_ptr(), self.v_pages.data_ptr(), int(dtype == torch.float16),
                                    int(self.o_fp32), self.device.index)

    @property
    def k_pages(self):
        """[layers][pages][Hkv][D/8][128][8] fp16 (None in a host-only cache)."""
        return self._pools.get("k_pages")

    @property
    def v_pages(self):
        """[layers][pages][Hkv][16][D][8], the cache's dtype."""
        return self._pools.get("v_pages")

    def _on_gpu(self):
        if self.host_only or not self._h.value:
            raise _abi.BcaError(_abi.BCA_ERR_HOST_ONLY_PLAN if self.host_only else _abi.BCA_ERR_INVALID_ARGUMENT,
                                "paged cache")
        return self._c

    @staticmethod
    def _stream(stream):
        """None: the current stream of the cache's device."""
        return stream if stream is None or isinstance(stream, int) else int(stream.cuda_stream)

    # ------------------------------------------------------------------ operators
    def write(self, k, v, table, off, start, *, pos=None, k_gain=None, layer: int = 0, stream=None) -> None:
        """Put rows off[b] .. off[b + 1] - 1 of k and v [n, Hkv, D] into the pages of table row
        b as its tokens start[b], start[b] + 1, ...  With pos (int32 [n, 3]) the keys pass
        through QK-Norm (k_gain, or ones) and RoPE; without, they are given post-prologue.
        table, off, start, pos: int32 tensors on the cache's device, read when the kernel runs.
        A token that has no page is dropped and reported by ``status``."""
        c = self._on_gpu()
        rc = self._calls.write(c, k, v, table, off, start, pos, k_gain, layer, self._stream(stream))
        if rc:
            _abi.check(rc, "bca_paged_write")

    def copy_pages(self, pairs, *, stream=None) -> None:
        """Make page pairs[i, 1] a copy of page pairs[i, 0], in every layer.  pairs: [n, 2] on
        the host (a CPU tensor, an array or a list), read before the call returns.  A page may
        be written once, and none that is written may be read."""
        import torch
        c = self._on_gpu()
        if not (isinstance(pairs, torch.Tensor) and pairs.dtype is torch.int32 and pairs.is_contiguous()):
            if isinstance(pairs, torch.Tensor) and pairs.is_cuda:
                raise ValueError("pairs: expected host data")
            pairs = np.asarray(pairs)
            if pairs.size == 0:
                pairs = np.zeros((0, 2), np.int32)
            if pairs.ndim != 2 or pairs.shape[1] != 2 or pairs.dtype.kind not in "iu":
                raise ValueError(f"pairs: expected whole numbers [n, 2], got {pairs.dtype} {pairs.shape}")
            if pairs.size and (pairs.min() < 0 or pairs.max() >= self.pages):
                raise _abi.BcaError(_abi.BCA_ERR_BAD_PAGE, "bca_paged_copy")
            pairs = torch.from_numpy(np.ascontiguousarray(pairs, dtype=np.int32))
        rc = self._calls.copy(c, pairs, self._stream(stream))
        if rc:
            _abi.check(rc, "bca_paged_copy")

    def attend(self, q, table, off, k_begin, k_end, *, seq=None, causal: bool = False, pos=None, q_gain=None,
               layer: int = 0, o=None, lse=None, workspace=None, stream=None):
        """Attention of q [nq, Hq, D] over the pages.  Rows off[i] .. off[i + 1] - 1 are slice i
        and see tokens k_begin[i] .. k_end[i] - 1 of table row seq[i] (seq=None: slice i reads
        row i), all of them, or with causal=True aligned at the last row and key.  pos (int32
        [nq, 3]) and q_gain as in ``write``.  off, seq, k_begin, k_end and table are int32
        tensors on the cache's device, read when the kernel runs.

        Returns o; rows that see no key are zero.  Rows outside every slice are left as they
        were in a given o (else uninitialised).  lse (fp32 [Hq, nq], optional) is filled in."""
        c = self._on_gpu()
        o = self._calls.attend(c, q, table, off, k_begin, k_end, seq, causal, pos, q_gain, layer, o, lse, workspace,
                               self._stream(stream))
        if isinstance(o, int):
            _abi.check(o, "bca_paged_attend")
        return o

    def workspace_bytes(self, nq: int, slices: int, width: int) -> int:
        """Bytes of workspace of an ``attend`` call: rows of q, slices, columns of the table.  A call
        of fewer rows or slices can need more."""
        return int(self._lib.bca_paged_workspace_bytes(self._h, nq, slices, width))

    def max_workspace_bytes(self) -> int:
        """What no ``attend`` call of this cache passes, whatever its sizes."""
        return int(self._lib.bca_paged_max_workspace_bytes(self._h))

    def alloc_workspace(self, nq: int, slices: int, width: int, stream=None):
        """Workspace of an ``attend`` call of these sizes, on its stream.  Calls that may overlap
        on the GPU (two streams, two captured graphs replayed side by side) need one each."""
        import torch
        n = max(16, self.workspace_bytes(nq, slices, width))
        with on_stream(stream, self.device):   # its next user is behind this call
            return torch.empty(n, dtype=torch.uint8, device=self.device)

    def status(self, stream=None) -> int:
        """Status of the cache's calls, those on `stream` waited for and those of other streams as
        far as they have run: BCA_OK, BCA_ERR_DEVICE_TIMEOUT, BCA_ERR_INVALID_ARGUMENT when
        overlapping calls shared a workspace and noticed it, or BCA_ERR_BAD_PAGE when a written
        token had no page.  Reading clears what is returned; another kind is left for the next call."""
        import torch
        if stream is None and not self.host_only:
            stream = torch.cuda.current_stream(self.device)
        return int(self._lib.bca_paged_status(self._h, self._stream(stream)))

    def close(self) -> None:
        """Free the handle (the pools are tensors of their own).  A captured graph holds neither:
        both have to outlive it."""
        if getattr(self, "_h", None) is not None and self._h.value:
            self._lib.bca_paged_destroy(self._h)
            self._h = _abi.ctypes.c_void_p()

    def __enter__(self) -> "PagedCache":
        return self

    def __exit__(self, *exc) -> None:
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PagePool:
    """Which page belongs to whom: sequences with page tables, shared pages counted, pages
    copied before a write when they are shared.  Host bookkeeping only; the copies it asks for
    (lists of (from, to)) go to ``PagedCache.copy_pages``.  A page given back may be another
    sequence's at once: work on both belongs on one stream, or on streams that the caller orders.

    Of a sequence it keeps the pages from the first one that is there on, so that calls cost what
    the pages in use cost, however far a window has slid (with an entry for every page there ever
    was, a slide and a layout of a 720p window took 42 ms at chunk 5,000; now 0.26 at any)."""

    def __init__(self, pages: int):
        if pages < 1:
            raise ValueError("pages >= 1 is required")
        self.pages = int(pages)
        self._free = list(range(self.pages))       # a heap: the lowest free page first
        self._users = np.zeros(self.pages, np.int64)
        self._rows: Dict[int, List[int]] = {}      # pages in order, -1: released; from page _base on
        self._base: Dict[int, int] = {}            # of each sequence: all pages before are absent
        self._next = 0

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def open(self) -> int:
        """A new, empty sequence."""
        self._next += 1
        self._rows[self._next], self._base[self._next] = [], 0
        return self._next

    def _row(self, seq: int) -> List[int]:
        if seq not in self._rows:
            raise KeyError(f"no open sequence {seq}")
        return self._rows[seq]

    def row(self, seq: int, first: int = 0) -> List[int]:
        """The sequence's pages in order (-1: released), from page `first` on."""
        if first < 0:
            raise ValueError(f"page {first}")
        row, base = self._row(seq), self._base[seq]
        return [-1] * (base - first) + row[max(0, first - base):]

    def _release(self, page: int) -> None:
        if page >= 0:
            self._users[page] -= 1
            if self._users[page] == 0:
                heapq.heappush(self._free, page)

    def _take(self) -> int:
        page = heapq.heappop(self._free)
        self._users[page] = 1
        return page

    def grow(self, seq: int, begin: int, end: int) -> List[tuple]:
        """Make tokens [begin, end) of the sequence writable: the pages that they touch exist
        (released ones come back, empty; pages skipped before `begin` stay absent) and are its
        own.  Returns the page copies to make before the write.  Raises MemoryError, with
        nothing changed, when the pool has too few free pages."""
        if begin < 0 or end < begin:
            raise ValueError(f"tokens [{begin}, {end})")
        row = self._row(seq)
        if begin == end:
            return []
        first, last, base = begin // PAGE, (end + PAGE - 1) // PAGE, self._base[seq]
        stop = base + len(row)                     # pages from here on are new
        touched = range(max(first, base), min(last, stop))
        need = last - first - len(touched) + sum(1 for i in touched if row[i - base] < 0 or
                                                 self._users[row[i - base]] > 1)
        if need > len(self._free):
            raise MemoryError(f"{need} pages needed, {len(self._free)} free")
        if not row and first > base:
            base = self._base[seq] = stop = first
        before = [self._take() for _ in range(first, min(last, base))]   # released: they come back
        moves = []
        for i in touched:
            old = row[i - base]
            if old < 0:
                row[i - base] = self._take()
            elif self._users[old] > 1:
                row[i - base] = self._take()
                self._users[old] -= 1
                if i * PAGE < begin or (i + 1) * PAGE > end:   # else every slot is written anew
                    moves.append((old, row[i - base]))
        if before:
            row[:0] = before + [-1] * (base - last)
            self._base[seq] = first
        row += [-1] * (first - stop)
        row += [self._take() for _ in range(max(first, stop), last)]
        return moves

    def fork(self, seq: int) -> int:
        """A new sequence with the same tokens, sharing every page."""
        row = list(self._row(seq))
        for p in row:
            if p >= 0:
                self._users[p] += 1
        new = self.open()
        self._rows[new], self._base[new] = row, self._base[seq]
        return new

    def release_before(self, seq: int, token: int) -> None:
        """Give back the pages that hold only tokens before `token` (behind a KV range)."""
        row, base = self._row(seq), self._base[seq]
        gone = min(token // PAGE - base, len(row))
        if gone > 0:
            for p in row[:gone]:
                self._release(p)
            while gone < len(row) and row[gone] < 0:
                gone += 1
            del row[:gone]
            self._base[seq] = base + gone

    def close(self, seq: int) -> None:
        """End a sequence and give its pages back."""
        for p in self._row(seq):
            self._release(p)
        del self._rows[seq], self._base[seq]

    def compact(self) -> List[tuple]:
        """Move the pages in use to the front of the pool.  Returns the copies to make; the
        tables already hold the new numbers."""
        used = int(np.count_nonzero(self._users))
        holes = [p for p in range(used) if self._users[p] == 0]
        high = [p for p in range(used, self.pages) if self._users[p] > 0]
        new = dict(zip(high, holes))
        for a, b in new.items():
            self._users[b], self._users[a] = self._users[a], 0
        for row in self._rows.values():
            row[:] = [new.get(p, p) for p in row]
        self._free = [p for p in range(self.pages) if self._users[p] == 0]
        heapq.heapify(self._free)
        return list(new.items())

    def table(self, seqs: Sequence[int], width: Optional[int] = None) -> np.ndarray:
        """int32 [len(seqs), width] (width: the longest row's, or given), absent pages -1."""
        rows = [(self._row(s), self._base[s]) for s in seqs]
        need = max((base + len(r) for r, base in rows), default=0)
        width = need if width is None else width
        if width < need:
            raise ValueError(f"width {width}: the longest row has {need} pages")
        out = np.full((len(rows), width), -1, np.int32)
        for i, (r, base) in enumerate(rows):
            out[i, base:base + len(r)] = r
        return out
