"""The paged cache without a GPU: refusals of the C ABI and of the binding, and the page
bookkeeping against a plain model of it."""
import ctypes

import numpy as np
import pytest
import torch

from block_causal_attention_b200 import BcaError, PagedCache, PagePool, _abi

PAGE = 128


def desc(**kw):
    d = _abi.bca_paged_desc()
    d.num_q_heads, d.num_kv_heads, d.head_dim, d.num_layers, d.num_pages = 16, 2, 48, 2, 10
    d.rope_base[:] = [1e4, 1e4, 1e4]
    d.norm_eps, d.flags = 1e-6, _abi.BCA_PLAN_HOST_ONLY
    for k, v in kw.items():
        if k == "rope_base":
            d.rope_base[:] = v
        else:
            setattr(d, k, v)
    return d


def create(d):
    h = ctypes.c_void_p()
    rc = _abi.lib().bca_paged_create(ctypes.byref(d), ctypes.byref(h))
    assert (rc == _abi.BCA_OK) == bool(h.value)
    _abi.lib().bca_paged_destroy(h)
    return rc


@pytest.mark.parametrize("kw,code", [
    ({}, _abi.BCA_OK), ({"head_dim": 24}, _abi.BCA_OK), ({"head_dim": 32}, _abi.BCA_OK),
    ({"head_dim": 64}, _abi.BCA_ERR_UNSUPPORTED), ({"head_dim": 0}, _abi.BCA_ERR_UNSUPPORTED),
    ({"num_q_heads": 15}, _abi.BCA_ERR_UNSUPPORTED), ({"num_q_heads": 0}, _abi.BCA_ERR_INVALID_ARGUMENT),
    ({"num_kv_heads": -1}, _abi.BCA_ERR_INVALID_ARGUMENT), ({"num_layers": 0}, _abi.BCA_ERR_INVALID_ARGUMENT),
    ({"num_pages": 0}, _abi.BCA_ERR_INVALID_ARGUMENT), ({"num_pages": 1 << 31}, _abi.BCA_ERR_INVALID_ARGUMENT),
    ({"norm_eps": -1.0}, _abi.BCA_ERR_INVALID_ARGUMENT), ({"norm_eps": float("nan")}, _abi.BCA_ERR_INVALID_ARGUMENT),
    ({"rope_base": [1e4, 0.0, 1e4]}, _abi.BCA_ERR_INVALID_ARGUMENT),
    ({"rope_base": [1e4, float("inf"), 1e4]}, _abi.BCA_ERR_INVALID_ARGUMENT),
    ({"flags": _abi.BCA_PLAN_HOST_ONLY | _abi.BCA_NO_PROLOGUE}, _abi.BCA_ERR_INVALID_ARGUMENT),
])
def test_create(kw, code):
    assert create(desc(**kw)) == code


def test_null_arguments_and_a_host_only_cache():
    L = _abi.lib()
    assert L.bca_paged_create(None, None) == _abi.BCA_ERR_INVALID_ARGUMENT
    h = ctypes.c_void_p(5)
    assert L.bca_paged_create(None, ctypes.byref(h)) == _abi.BCA_ERR_INVALID_ARGUMENT and not h.value
    L.bca_paged_destroy(None)
    assert L.bca_paged_pool_bytes(None) == 0 and L.bca_paged_workspace_bytes(None, 5, 5, 5) == 0
    assert L.bca_paged_status(None, None) == _abi.BCA_ERR_INVALID_ARGUMENT
    c = PagedCache(16, 2, 48, 10, layers=2, host_only=True)
    assert c.pool_bytes == 10 * 2 * PAGE * 48 * 2
    assert c.workspace_bytes(0, 5, 9) == 0 and c.workspace_bytes(5, 0, 9) == 0 and c.workspace_bytes(5, 1, -1) == 0
    assert c.workspace_bytes(1, 1, 9) == 0 and c.workspace_bytes(1, 1, 9999) > 0 and c.workspace_bytes(500, 1, 9) > 0
    assert c.status() == _abi.BCA_ERR_HOST_ONLY_PLAN
    z = [None] * 3
    assert L.bca_paged_write(c._h, None, None, 0, *z, 0, 0, *[None] * 5) == _abi.BCA_ERR_HOST_ONLY_PLAN
    assert L.bca_paged_write(c._h, None, None, -1, *z, 0, 0, *[None] * 5) == _abi.BCA_ERR_INVALID_ARGUMENT
    assert L.bca_paged_attend(c._h, None, 0, *[None] * 5, 0, 0, *[None] * 4, 0, 0, *[None] * 4) == \
        _abi.BCA_ERR_HOST_ONLY_PLAN
    for bad in ({"nq": -1}, {"nq": 1 << 31}, {"seqs": -1}, {"width": -1}, {"width": 1 << 24}, {"slices": -1}):
        a = {"nq": 1, "seqs": 1, "width": 1, "slices": 1, **bad}
        rc = L.bca_paged_attend(c._h, None, a["nq"], *[None] * 5, a["seqs"], a["width"], *[None] * 4, a["slices"], 0,
                                *[None] * 4)
        assert rc == _abi.BCA_ERR_INVALID_ARGUMENT, bad
    for call in (lambda: c.copy_pages([[0, 1]]), lambda: c.write(*[None] * 5), lambda: c.attend(*[None] * 5)):
        with pytest.raises(BcaError) as e:
            call()
        assert e.value.code == _abi.BCA_ERR_HOST_ONLY_PLAN
    with pytest.raises(BcaError) as e:
        c.copy_pages([[0, 1]])
    assert e.value.code == _abi.BCA_ERR_HOST_ONLY_PLAN
    with pytest.raises(ValueError):
        PagedCache(16, 2, 48, 10, dtype=torch.float32, host_only=True)


@pytest.mark.parametrize("pairs,code", [
    ([], _abi.BCA_ERR_HOST_ONLY_PLAN), ([(0, 1), (0, 2), (5, 9)], _abi.BCA_ERR_HOST_ONLY_PLAN),
    ([(0, 10)], _abi.BCA_ERR_BAD_PAGE), ([(-1, 3)], _abi.BCA_ERR_BAD_PAGE), ([(0, 1), (2, 1)], _abi.BCA_ERR_BAD_PAGE),
    ([(0, 1), (1, 2)], _abi.BCA_ERR_BAD_PAGE), ([(3, 3)], _abi.BCA_ERR_BAD_PAGE),
    ([(0, 1)] * 11, _abi.BCA_ERR_BAD_PAGE), ([(1, 2), (2, 1)], _abi.BCA_ERR_BAD_PAGE)])
def test_page_moves_are_checked_before_anything_else(pairs, code):
    a = np.asarray(pairs, np.int32).reshape(-1, 2)
    for pages in (10, 10_000_000):               # a bit a page, and a sorted list
        c = PagedCache(16, 2, 48, pages, host_only=True)
        b = np.where(a == 10, pages, a).astype(np.int32)
        assert _abi.lib().bca_paged_copy(c._h, b.ctypes.data, len(b), None, None, None) == code
    assert "page" in _abi.error_string(_abi.BCA_ERR_BAD_PAGE)


# ---------------------------------------------------------------------------------- PagePool

class Model:
    """Tokens of sequences as plain lists; pages as what their slots hold."""

    def __init__(self, pages):
        self.pool = PagePool(pages)
        self.slots = np.full((pages, PAGE), -1, np.int64)
        self.seqs = {}
        self.stamp = 0

    def move(self, pairs):
        src = self.slots[[a for a, _ in pairs]].copy()
        assert len({b for _, b in pairs}) == len(pairs) and not {a for a, _ in pairs} & {b for _, b in pairs}
        for (_, b), x in zip(pairs, src):
            self.slots[b] = x

    def write(self, s, at, n):
        self.move(self.pool.grow(s, at, at + n))
        row, want = self.pool.row(s), self.seqs[s]
        want.extend([None] * (at + n - len(want)))
        for i in range(at, at + n):
            self.stamp += 1
            self.slots[row[i // PAGE], i % PAGE] = want[i] = self.stamp

    def check(self):
        used = set()
        for s, want in self.seqs.items():
            row = self.pool.row(s)
            for i, x in enumerate(want):
                if x is not None:
                    assert self.slots[row[i // PAGE], i % PAGE] == x
            used |= {p for p in row if p >= 0}
        assert self.pool.free_pages == self.pool.pages - len(used)


def test_page_pool_against_a_model():
    rng = np.random.default_rng(5)
    m = Model(40)
    for _ in range(600):
        op = rng.integers(0, 6)
        s = rng.choice(list(m.seqs)) if m.seqs else None
        try:
            if s is None or op == 0:
                m.seqs[m.pool.open()] = []
            elif op in (1, 2):
                n = len(m.seqs[s])
                m.write(s, int(rng.integers(max(0, n - 200), n + 1)), int(rng.integers(0, 300)))
            elif op == 3:
                f = m.pool.fork(s)
                m.seqs[f] = list(m.seqs[s])
            elif op == 4:
                t = int(rng.integers(0, len(m.seqs[s]) + 1))
                m.pool.release_before(s, t)
                for i in range(t // PAGE * PAGE):
                    m.seqs[s][i] = None
            elif rng.random() < 0.5:
                m.pool.close(s)
                del m.seqs[s]
            else:
                m.move(m.pool.compact())
                top = max((p for q in m.seqs for p in m.pool.row(q)), default=-1)
                assert top + 1 == m.pool.pages - m.pool.free_pages
        except MemoryError:
            m.pool.close(s)
            del m.seqs[s]
        m.check()


def test_page_pool_tables_and_refusals():
    p = PagePool(4)
    a = p.open()
    assert p.grow(a, 0, 300) == [] and p.row(a) == [0, 1, 2]
    b = p.fork(a)
    assert p.free_pages == 1
    assert p.grow(b, 300, 301) == [(2, 3)]           # a partly written page is copied
    with pytest.raises(MemoryError):
        p.grow(a, 0, 1)
    assert p.row(a) == [0, 1, 2]
    p.release_before(a, 256)
    assert p.row(a) == [-1, -1, 2] and p.free_pages == 0
    assert p.table([a, b], 4).tolist() == [[-1, -1, 2, -1], [0, 1, 3, -1]]
    assert p.table([]).shape == (0, 0)
    with pytest.raises(ValueError):
        p.table([a], 2)
    with pytest.raises(ValueError):
        p.grow(a, 5, 4)
    p.close(a)
    with pytest.raises(KeyError):
        p.row(a)
    with pytest.raises(ValueError):
        PagePool(0)
    assert p.grow(b, 256, 384) == [] and p.free_pages == 1


def test_pages_skipped_before_the_first_token_stay_absent():
    p = PagePool(3)
    a = p.open()
    assert p.grow(a, 5 * PAGE + 100, 7 * PAGE) == [] and p.row(a) == [-1] * 5 + [0, 1] and p.free_pages == 1
    assert p.grow(a, 3 * PAGE, 3 * PAGE + 1) == [] and p.row(a) == [-1] * 3 + [2, -1, 0, 1]
    with pytest.raises(MemoryError):
        p.grow(a, 9 * PAGE, 9 * PAGE + 1)
    assert len(p.row(a)) == 7
    p.close(a)
    assert p.free_pages == 3
