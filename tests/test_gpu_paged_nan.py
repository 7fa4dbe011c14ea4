"""Attention over pages where scores are NaN: softmax over a NaN score is NaN, so a row that sees
one gets NaN in O and in its LSE, and only a row that sees no key gets O = 0 and LSE = -inf.
References and bounds from tests/paged_ref.py; NaN has to stand where the reference has it."""
import math

import pytest
import torch

import paged_ref as ref
from block_causal_attention_b200 import PagedCache, _abi
from test_gpu_paged import BF, HF, gen, no_worse, positions, rand, widened

pytestmark = pytest.mark.gpu
PAGE = 128


@pytest.mark.parametrize("d", [24, 48])
@pytest.mark.parametrize("dtype,prologue", [(BF, True), (BF, False), (HF, True), (HF, False)])
@pytest.mark.parametrize("rows", [1, 4, 20, 50, 150])       # tiles of 16, 32, 128 and 384 rows
def test_a_query_that_is_nan(rows, dtype, prologue, d):
    """One NaN channel of one head of one row: that head's row is NaN, all others are as ever, and a
    slice without keys stays zero beside it, its NaN queries included."""
    g = gen(rows + d)
    hq, hkv, ctx = 8, 2, 300
    kp, vp = ref.pools(8, hkv, d, dtype, g)
    table = ref.table_of([4, 4], 8, g)
    cache = PagedCache(hq, hkv, d, 8, dtype=dtype, k_pages=kp, v_pages=vp)
    q = rand((2 * rows, hq, d), dtype, g)
    q[rows // 2, 5, 3] = math.nan
    q[rows:, 2] = math.nan
    pos = positions(2 * rows, g) if prologue else None
    off, kb, ke = [0, rows, 2 * rows], [7, 50], [ctx + rows, 50]
    for causal in (False, True):
        wo, wl, bo, bl = ref.attend(q, kp[0], vp[0], table, off, [0, 1], kb, ke, causal, pos)
        assert wo[rows // 2, 5].isnan().all() and wl[5, rows // 2].isnan() and (wo[rows:] == 0).all()
        for tab in (table, widened(table)):      # by clusters or by shares
            o, lse = torch.full_like(q, 7.0), torch.full((hq, 2 * rows), 7.0, device="cuda")
            cache.attend(q, tab, ref.i32(off), ref.i32(kb), ref.i32(ke), causal=causal, pos=pos, o=o, lse=lse)
            assert cache.status() == _abi.BCA_OK
            no_worse(o, wo, bo, "o")
            no_worse(lse, wl, bl, "lse")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows", [1, 4, 20, 50, 150])
def test_the_only_key_is_nan(rows, dtype):
    g = gen(rows)
    hq, hkv, d, key = 8, 2, 32, 200
    kp, vp = ref.pools(2, hkv, d, dtype, g)
    kp[0, 1, 1, 2, key % PAGE, 5] = math.nan                  # of KV head 1
    table = ref.i32([[0, 1]])
    cache = PagedCache(hq, hkv, d, 2, dtype=dtype, k_pages=kp, v_pages=vp)
    q = rand((rows, hq, d), dtype, g)
    wo, wl, bo, bl = ref.attend(q, kp[0], vp[0], table, [0, rows], [0], [key], [key + 1], False)
    assert wo[:, 4:].isnan().all() and wl[4:].isnan().all() and wo[:, :4].isfinite().all()
    for tab in (table, widened(table)):
        o, lse = torch.full_like(q, 7.0), torch.full((hq, rows), 7.0, device="cuda")
        cache.attend(q, tab, ref.i32([0, rows]), ref.i32([key]), ref.i32([key + 1]), o=o, lse=lse)
        assert cache.status() == _abi.BCA_OK
        no_worse(o, wo, bo, "o")
        no_worse(lse, wl, bl, "lse")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hq,hkv,rows,pages", [
    (8, 2, 1, 60),          # 16-row tiles: by clusters where the table is narrow, else two items in 148 shares
    (12, 2, 4, 60),         # 32-row tiles, more than four pieces each
    (64, 64, 32, 12),       # 32-row tiles, up to four pieces each
    (16, 2, 20, 40),        # 128-row tiles, more than four pieces
    (96, 96, 100, 12),      # 128-row tiles, up to four pieces
    (16, 2, 100, 40),       # 384-row tiles, more than four pieces
    (60, 2, 700, 12)])      # 384-row tiles, up to four pieces
@pytest.mark.parametrize("first,last", [(0, 0.5), (0.5, 1), (0.25, 0.6)])
def test_pages_of_nan_keys(hq, hkv, rows, pages, first, last, dtype):
    """A stretch of pages whose keys are all NaN, for KV head 0: whatever piece of the work they make,
    its rows are NaN; the other heads see finite keys only."""
    g = gen(hq * rows)
    d = 24
    kp, vp = ref.pools(pages, hkv, d, dtype, g)
    table = ref.table_of([pages], pages, g)
    bad = table[0, int(first * pages):int(last * pages)].long()
    kp[0, bad, 0] = math.nan
    cache = PagedCache(hq, hkv, d, pages, dtype=dtype, k_pages=kp, v_pages=vp)
    q = rand((rows, hq, d), dtype, g)
    some = list(range(0, rows, max(1, rows // 6)))
    wo, wl, bo, bl = ref.attend_rows(q, kp[0], vp[0], table, [0, rows], [0], [0], [pages * PAGE], some)
    grp = hq // hkv
    assert wo[:, :grp].isnan().all() and wo[:, grp:].isfinite().all()
    for tab in (table, widened(table)):
        o, lse = torch.full_like(q, 7.0), torch.full((hq, rows), 7.0, device="cuda")
        cache.attend(q, tab, ref.i32([0, rows]), ref.i32([0]), ref.i32([pages * PAGE]), o=o, lse=lse)
        assert cache.status() == _abi.BCA_OK
        assert o[:, :grp].isnan().all() and lse[:grp].isnan().all()
        no_worse(o[some], wo, bo, "o")
        no_worse(lse[:, some], wl, bl, "lse")
