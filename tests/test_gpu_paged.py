"""The paged KV cache on the GPU against the 64-bit plain forms of tests/paged_ref.py."""
import math

import pytest
import torch

import paged_ref as ref
from block_causal_attention_b200 import BcaError, PagedCache, _abi

pytestmark = pytest.mark.gpu
PAGE = 128
BF, HF = torch.bfloat16, torch.float16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(shape, dtype, g):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def positions(n, g, far=100):
    return torch.randint(0, far, (n, 3), generator=g, device="cuda", dtype=torch.int32)


def no_worse(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    same = (got.double() == want) | (got.double().isnan() & want.isnan())
    bad &= ~same
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {err[bad].max().item():.3e}, " \
                          f"first at {bad.nonzero()[0].tolist()}"


def widened(table):
    """The same table with absent pages behind it, to 200 columns."""
    wide = torch.full((table.shape[0], max(200, table.shape[1])), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    return wide


def check_attend(hq, hkv, d, dtype, new, ctx, causal, prologue, seed, block=0, kv_range=0, o_fp32=False, far=100):
    g = gen(seed)
    need = [-(-(n + c) // PAGE) for n, c in zip(new, ctx)]
    pages = sum(need) + 2
    kp, vp = ref.pools(pages, hkv, d, dtype, g)
    table = ref.table_of(need, pages, g)
    cache = PagedCache(hq, hkv, d, pages, dtype=dtype, k_pages=kp, v_pages=vp, o_fp32=o_fp32)
    sl = []
    for b, (n, c) in enumerate(zip(new, ctx)):
        step = block or max(n, 1)
        for r in range(0, max(n, 1), step):
            m = min(step, n - r)
            sl.append((b, m, max(0, c + r - kv_range * step) if kv_range else 0, c + r + m))
    off = ref.offsets([x[1] for x in sl])
    nq = off[-1]
    q = rand((nq, hq, d), dtype, g)
    pos = positions(nq, g, far) if prologue else None
    gain = 1 + 0.1 * torch.randn(d, generator=g, device="cuda") if prologue else None
    o = torch.full((nq, hq, d), math.nan, dtype=torch.float32 if o_fp32 else dtype, device="cuda")
    lse = torch.full((hq, nq), math.nan, device="cuda")
    seq, kb, ke = [x[0] for x in sl], [x[2] for x in sl], [x[3] for x in sl]
    wo, wl, bo, bl = ref.attend(q, kp[0], vp[0], table, off, seq, kb, ke, causal, pos, gain)
    for tab in (table, widened(table)):          # few items go by clusters, or by shares where tables are wide
        o.fill_(math.nan)
        lse.fill_(math.nan)
        cache.attend(q, tab, ref.i32(off), ref.i32(kb), ref.i32(ke), seq=ref.i32(seq), causal=causal, pos=pos,
                     q_gain=gain, o=o, lse=lse)
        assert cache.status() == _abi.BCA_OK
        no_worse(o, wo, bo, "o")
        no_worse(lse, wl, bl, "lse")


# ---------------------------------------------------------------------------------- write

@pytest.mark.parametrize("d", [24, 32, 48])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("prologue", [True, False])
@pytest.mark.parametrize("new,at", [([1], [0]), ([1, 1, 1], [0, 127, 128]), ([0, 5, 0, 130], [7, 120, 0, 3]),
                                    ([128], [128]), ([257, 1, 31], [1, 255, 97])])
def test_write(d, dtype, prologue, new, at):
    g = gen(17)
    hkv = 3 if d == 32 else 2
    need = [-(-(n + a) // PAGE) for n, a in zip(new, at)]
    pages = sum(need) + 1
    kp, vp = ref.pools(pages, hkv, d, dtype, g, layers=2)
    kp[0], vp[0, 0] = math.nan, math.inf
    table = ref.table_of(need, pages, g)
    off = ref.offsets(new)
    n = off[-1]
    k, v = rand((n, hkv, d), dtype, g), rand((n, hkv, d), dtype, g)
    pos = positions(n, g, 1 << 20) if prologue else None
    gain = 1 + 0.1 * torch.randn(d, generator=g, device="cuda") if prologue else None
    cache = PagedCache(hkv, hkv, d, pages, layers=2, dtype=dtype, k_pages=kp, v_pages=vp)
    want_k, want_v = kp.clone(), vp.clone()
    cache.write(k, v, table, ref.i32(off), ref.i32(at), pos=pos, k_gain=gain, layer=1)
    assert cache.status() == _abi.BCA_OK
    kh = ref.prologue(k, pos, gain)
    wrote = torch.zeros_like(kp, dtype=torch.bool)
    exact = kp.double()
    tab = table.tolist()
    for b, m in enumerate(new):
        for i in range(m):
            p, s = tab[b][(at[b] + i) // PAGE], (at[b] + i) % PAGE
            exact[1, p, :, :, s] = kh[off[b] + i].view(hkv, d // 8, 8)
            wrote[1, p, :, :, s] = True
            want_v[1, p, :, s // 8, :, s % 8] = v[off[b] + i]
    assert torch.equal(vp.view(torch.int16), want_v.view(torch.int16))
    assert torch.equal(kp.view(torch.int16)[~wrote], want_k.view(torch.int16)[~wrote])
    # half a step of fp16 (2^-25 below its normal range), and 2^-20 of the row's largest value
    # for the norm, the angle (2 pi 2^-25 of a turn) and the rotation in fp32
    row = exact[1].abs().amax((1, 2, 4), keepdim=True).expand_as(exact[1])
    bound = 2.0 ** -11 * exact[1].abs() + 2.0 ** -25 + (2.0 ** -20 * row if prologue else 0)
    no_worse(kp[1][wrote[1]], exact[1][wrote[1]], bound[wrote[1]], "k_pages")


def test_write_drops_what_has_no_page_and_reports_it():
    g = gen(3)
    kp, vp = ref.pools(3, 2, 24, BF, g)
    cache = PagedCache(2, 2, 24, 3, k_pages=kp, v_pages=vp)
    k, v = rand((40, 2, 24), BF, g), rand((40, 2, 24), BF, g)
    before_k, before_v = kp.clone(), vp.clone()
    # an absent page, a page outside the pool, tokens behind the table, tokens before 0
    cache.write(k, v, ref.i32([[-1, 1], [3, 0], [0, 1], [2, 1]]), ref.i32([0, 10, 20, 30, 40]), ref.i32([0, 0, 256, -10]))
    assert cache.status() == _abi.BCA_ERR_BAD_PAGE
    assert cache.status() == _abi.BCA_OK
    assert torch.equal(kp, before_k) and torch.equal(vp, before_v)
    # the tokens of such a call that do have a page are written
    cache.write(k, v, ref.i32([[-1, 1]]), ref.i32([0, 40]), ref.i32([120]))
    assert cache.status() == _abi.BCA_ERR_BAD_PAGE
    assert torch.equal(kp[0, 1, :, :, :32].permute(2, 0, 1, 3).reshape(32, 2, 24), k[8:].half())
    assert torch.equal(kp[0, 0], before_k[0, 0]) and torch.equal(kp[0, 1, :, :, 32:], before_k[0, 1, :, :, 32:])


# ---------------------------------------------------------------------------------- copy

@pytest.mark.parametrize("d,hkv,layers,dtype", [(24, 1, 1, BF), (32, 3, 2, HF), (48, 8, 3, BF)])
@pytest.mark.parametrize("moves", [1, 7, 481])
def test_copy_pages(d, hkv, layers, dtype, moves):
    g = gen(moves)
    pages = 2 * moves + 1
    kp, vp = ref.pools(pages, hkv, d, dtype, g, layers=layers)
    cache = PagedCache(hkv, hkv, d, pages, layers=layers, dtype=dtype, k_pages=kp, v_pages=vp)
    order = torch.randperm(pages, generator=g, device="cuda")
    src, dst = order[:moves], order[moves:2 * moves]
    src = src[torch.randint(0, moves, (moves,), generator=g, device="cuda")]   # a page may be read often
    wk, wv = kp.clone(), vp.clone()
    wk[:, dst], wv[:, dst] = kp[:, src], vp[:, src]
    cache.copy_pages(torch.stack([src, dst], 1).cpu())
    torch.cuda.synchronize()
    assert torch.equal(kp, wk) and torch.equal(vp, wv)


# ---------------------------------------------------------------------------------- attend

@pytest.mark.parametrize("d", [24, 32, 48])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (16, 1), (12, 4), (10, 2), (128, 8)])
def test_attend_single_tokens(d, dtype, hq, hkv):
    check_attend(hq, hkv, d, dtype, [1, 1, 0, 1, 1], [0, 127, 300, 128, 1000], False, True, 1)


@pytest.mark.parametrize("d", [24, 32, 48])
@pytest.mark.parametrize("dtype,prologue", [(BF, True), (BF, False), (HF, True), (HF, False)])
@pytest.mark.parametrize("new,ctx", [([3, 1, 5], [0, 200, 127]), ([17, 40], [0, 333]), ([1, 129], [511, 5])])
def test_attend_causal(d, dtype, prologue, new, ctx):
    for hq, hkv in ((2, 2), (6, 2), (16, 1)):
        check_attend(hq, hkv, d, dtype, new, ctx, True, prologue, 2)


@pytest.mark.parametrize("d", [24, 32, 48])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (16, 1), (3, 1)])
def test_attend_blocks_with_a_key_range(d, hq, hkv):
    check_attend(hq, hkv, d, BF, [150, 90], [200, 0], False, True, 3, block=60, kv_range=2)
    check_attend(hq, hkv, d, HF, [150, 90], [200, 77], False, True, 3, block=37, kv_range=1, o_fp32=True)


def test_attend_long_and_far():
    check_attend(16, 2, 48, BF, [1, 1], [40000, 3], False, True, 4, far=1 << 22)
    check_attend(8, 8, 24, HF, [2], [20001], True, True, 5)
    check_attend(4, 1, 32, BF, [300], [5000], True, False, 6)


def test_attend_many_slices():
    """More slices than a block has threads, most of them without rows."""
    new = [1 if b % 7 == 3 else 0 for b in range(900)]
    ctx = [(b * 37) % 300 for b in range(900)]
    check_attend(4, 2, 24, BF, new, ctx, False, True, 7)


def test_attend_scores_that_grow_and_shrink():
    """Scores that rise by hundreds along the keys, then fall: the reference moves often."""
    g = gen(8)
    d, keys = 32, 1500
    for dtype in (BF, HF):
        kp, vp = ref.pools(12, 1, d, dtype, g)
        table = ref.table_of([12], 12, g)
        scale = torch.linspace(0.1, 40, 12, device="cuda")
        for i, p in enumerate(table[0].tolist()):
            kp[0, p] *= scale[i] if i < 8 else scale[11 - i]
        cache = PagedCache(8, 1, d, 12, dtype=dtype, k_pages=kp, v_pages=vp)
        q = rand((3, 8, d), dtype, g)
        o, lse = torch.empty_like(q), torch.empty((8, 3), device="cuda")
        cache.attend(q, table, ref.i32([0, 3]), ref.i32([0]), ref.i32([keys]), causal=True, o=o, lse=lse)
        assert cache.status() == _abi.BCA_OK
        wo, wl, bo, bl = ref.attend(q, kp[0], vp[0], table, [0, 3], [0], [0], [keys], True)
        no_worse(o, wo, bo, "o")
        no_worse(lse, wl, bl, "lse")


@pytest.mark.parametrize("d", [24, 32, 48])
@pytest.mark.parametrize("rows", [1, 20, 100, 400])
def test_attend_fp16_queries_keep_their_rounding(d, rows):
    """Over a single key the LSE is the score, so it shows the queries' precision alone.  Per element,
    relative to its RoPE pair's length: sine and cosine 2^-21.2 and 2^-21.4 (CUDA's bounds for the fast
    ones) with 2^-22 each for the angle in fp32, together below 2^-19.6; RMS norm, gain and RoPE's
    products and sum, six roundings, 2^-21.4; the second fp16 tile 2^-22; the sum of d <= 48 products in
    fp32, 2^-18.4; scale and LSE 2^-22.  Below 2^-17 in all; an fp16 rounding alone is 2^-11."""
    g = gen(d + rows)
    hq, hkv, key = 4, 2, 5
    kp, vp = ref.pools(2, hkv, d, HF, g)
    table = ref.table_of([1], 2, g)
    cache = PagedCache(hq, hkv, d, 2, dtype=HF, k_pages=kp, v_pages=vp)
    q, pos = rand((rows, hq, d), HF, g), positions(rows, g)
    gain = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    lse = torch.full((hq, rows), math.nan, device="cuda")
    cache.attend(q, table, ref.i32([0, rows]), ref.i32([key]), ref.i32([key + 1]), pos=pos, q_gain=gain, lse=lse)
    assert cache.status() == _abi.BCA_OK
    keys, _ = ref.unpage(kp[0], vp[0], table[0].tolist(), PAGE)
    k = keys[key].double().repeat_interleave(hq // hkv, 0)
    qh = ref.prologue(q, pos, gain)
    pair = qh.unflatten(-1, (d // 2, 2)).norm(dim=-1, keepdim=True).expand(-1, -1, -1, 2).flatten(-2)
    no_worse(lse, (qh * k).sum(-1).T / math.sqrt(d), 2.0 ** -17 * (pair * k.abs()).sum(-1).T / math.sqrt(d), "lse")


@pytest.mark.parametrize("rows", [1, 5, 40, 150])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_attend_empty_slices_and_rows_left_alone(rows, dtype):
    g = gen(9)
    kp, vp = ref.pools(6, 2, 48, dtype, g)
    table = ref.i32([[0, 1, 2], [3, -1, 9], [-1, -1, -1]])
    cache = PagedCache(4, 2, 48, 6, dtype=dtype, k_pages=kp, v_pages=vp)
    #      all keys, no keys, begin > end, no such row, an absent page inside, only absent pages, keys behind the table
    seq = [0, 0, 0, 7, 1, 2, 0, -1]
    kb = [0, 50, 60, 0, 10, 0, 384, 0]
    ke = [384, 50, 20, 300, 300, 384, 1000, 100]
    off = ref.offsets([rows] * len(seq))
    off = [x + 3 for x in off]                       # three rows before the first slice
    nq = off[-1] + 4                                 # four behind the last
    q = rand((nq, 4, 48), dtype, g)
    o = torch.full((nq, 4, 48), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((4, nq), 7.0, device="cuda")
    for causal, wide in ((False, False), (True, False), (False, True), (True, True)):
        if wide:
            ke[6] = 30000                        # keys behind the wider table too
            table = widened(table)
        cache.attend(q, table, ref.i32(off), ref.i32(kb), ref.i32(ke), seq=ref.i32(seq), causal=causal, o=o, lse=lse)
        assert cache.status() == _abi.BCA_OK
        wo, wl, bo, bl = ref.attend(q, kp[0], vp[0], table, off, seq, kb, ke, causal)
        for a, b in ((0, 3), (off[-1], nq)):
            wo[a:b], wl[:, a:b] = 7.0, 7.0
        no_worse(o, wo, bo, "o")
        no_worse(lse, wl, bl, "lse")


@pytest.mark.parametrize("rows", [1, 4, 30, 140])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [24, 48])
def test_attend_what_a_row_does_not_see_does_not_reach_it(rows, dtype, d):
    """NaN and infinities in free slots, behind the last key, before the first and, with the
    causal rule, at later tokens; a row that does see one gets what the formula gives."""
    g = gen(10)
    hq, hkv, ctx = 6, 2, 200
    kp, vp = ref.pools(5, hkv, d, dtype, g)
    kp[0, 4], vp[0, 4] = math.nan, math.inf
    table = ref.i32([[0, 1, 2, 3]])
    end = ctx + rows
    kb = 130
    for p in range(4):
        for s in range(PAGE):
            j = p * PAGE + s
            if j < kb or j >= end:
                kp[0, p, :, :, s] = math.nan if s % 2 else math.inf
                vp[0, p, :, s // 8, :, s % 8] = math.inf if s % 3 else math.nan
    for poison in (math.nan, math.inf, -math.inf):
        at = end - 1 - rows // 2                     # a new token in the middle
        vp[0, at // PAGE, 1, at % PAGE // 8, 3, at % 8] = poison
        cache = PagedCache(hq, hkv, d, 5, dtype=dtype, k_pages=kp, v_pages=vp)
        q = rand((rows, hq, d), dtype, g)
        o, lse = torch.empty_like(q), torch.empty((hq, rows), device="cuda")
        for causal, tab in ((True, table), (False, table), (True, widened(table)), (False, widened(table))):
            cache.attend(q, tab, ref.i32([0, rows]), ref.i32([kb]), ref.i32([end]), causal=causal, o=o, lse=lse)
            assert cache.status() == _abi.BCA_OK
            wo, wl, bo, bl = ref.attend(q, kp[0], vp[0], table, [0, rows], [0], [kb], [end], causal)
            assert wo.isnan().any() or wo.isinf().any()
            assert not causal or rows < 2 or wo[0].isfinite().all()
            no_worse(o, wo, bo, "o")
            no_worse(lse, wl, bl, "lse")
    kp[0, 1, 0, 0, (end - 1) % PAGE, 0] = math.nan   # the last key of KV head 0
    if (end - 1) // PAGE == 1:
        cache.attend(q, table, ref.i32([0, rows]), ref.i32([kb]), ref.i32([end]), causal=True, o=o, lse=lse)
        assert o[-1, :3].isnan().all() and lse[:3, -1].isnan().all()
        assert rows < 2 or o[0].isfinite().all()


def test_attend_any_offsets_stay_inside():
    """Tables, offsets, ranges and sequences are device data: nonsense in them must not lead a
    kernel outside its arrays (guard bands around the outputs)."""
    g = gen(11)
    cache = PagedCache(8, 2, 32, 4)
    cache.k_pages.zero_()
    cache.v_pages.zero_()
    big = 2 ** 31 - 1
    for rows in (5, 50, 400):
        raw = torch.full((rows + 64, 8, 32), 3.0, dtype=BF, device="cuda")
        q, o = rand((rows, 8, 32), BF, g), raw[32:32 + rows]
        for off, seq, kb, ke in (([5, 0, 9], [0, 1], [0, 0], [200, 200]), ([-4, 2, big], [0, 1], [-5, 3], [big, 60]),
                                 ([0, big, -big], [big, -big], [0, 0], [big, big]),
                                 ([-big, big, big], [0, 1], [-big, big], [big, -big])):
            for causal in (False, True):
                for tab in (ref.i32([[0, big, 1], [-big, 2, 4]]), widened(ref.i32([[0, big, 1], [-big, 2, 4]]))):
                    cache.attend(q, tab, ref.i32(off), ref.i32(kb), ref.i32(ke), seq=ref.i32(seq), causal=causal, o=o)
                    assert cache.status() == _abi.BCA_OK
        assert (raw[:32] == 3).all() and (raw[32 + rows:] == 3).all()
        kv = rand((rows, 2, 32), BF, g)
        for off, at in (([5, 0, 9], [0, 0]), ([-4, 2, big], [big, -big]), ([-big, big, big], [0, 5])):
            cache.write(kv, kv, ref.i32([[0, big, 1], [-big, 2, 4]]), ref.i32(off), ref.i32(at))
            assert cache.status() in (_abi.BCA_OK, _abi.BCA_ERR_BAD_PAGE)


def test_attend_same_bits_again_and_on_another_stream():
    g = gen(12)
    kp, vp = ref.pools(60, 2, 48, BF, g)
    table = ref.table_of([50, 9], 60, g)
    cache = PagedCache(16, 2, 48, 60, k_pages=kp, v_pages=vp)
    for n in (1, 3, 20, 300):
        q = rand((2 * n, 16, 48), BF, g)
        args = (q, table if n != 3 else widened(table), ref.i32([0, n, 2 * n]), ref.i32([0, 5]), ref.i32([6001, 1100]))
        first = cache.attend(*args, causal=True)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        o = torch.empty_like(q)
        torch.cuda.synchronize()
        for _ in range(5):
            assert torch.equal(cache.attend(*args, causal=True), first)
            cache.attend(*args, causal=True, o=o, stream=s)
            s.synchronize()
            assert torch.equal(o, first)


@pytest.mark.parametrize("most", [1, 4, 40, 200])
def test_captured_step_replays_for_other_lengths(most):
    """Write and attend in one graph; lengths, tables and positions change between replays."""
    g = gen(13)
    hq, hkv, d, pages = 12, 4, 32, 24
    kp, vp = ref.pools(pages, hkv, d, HF, g)
    cache = PagedCache(hq, hkv, d, pages, dtype=HF, k_pages=kp, v_pages=vp)
    nq = 3 * most
    q, k, v = rand((nq, hq, d), HF, g), rand((nq, hkv, d), HF, g), rand((nq, hkv, d), HF, g)
    table, off = ref.i32([[0] * 8] * 3), ref.i32([0] * 4)
    kb, ke, start, pos = ref.i32([0] * 3), ref.i32([0] * 3), ref.i32([0] * 3), positions(nq, g)
    o = torch.zeros_like(q)
    ws = cache.alloc_workspace(nq, 3, 8)

    def step():
        cache.write(k, v, table, off, start, pos=pos)
        cache.attend(q, table, off, kb, ke, causal=True, pos=pos, o=o, workspace=ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for new, ctx in (([1, 0, most], [300, 5, 700]), ([most, most, most], [0, 127, 511]), ([0, 0, 0], [1, 1, 1])):
        lens = ref.offsets(new)
        table.copy_(ref.table_of([8, 8, 8], pages, g))
        off.copy_(ref.i32(lens))
        start.copy_(ref.i32(ctx))
        ke.copy_(ref.i32([n + c for n, c in zip(new, ctx)]))
        pos.copy_(positions(nq, g))
        q.normal_(generator=g)
        graph.replay()
        assert cache.status() == _abi.BCA_OK
        wo, _, bo, _ = ref.attend(q, kp[0], vp[0], table, lens, [0, 1, 2], [0] * 3, ke.tolist(), True, pos)
        no_worse(o[:lens[-1]], wo[:lens[-1]], bo[:lens[-1]], "o")


def test_workspace_and_outputs_are_not_overrun():
    g = gen(14)
    for n, hq, hkv, d in ((1, 16, 1, 24), (2, 12, 1, 48), (3, 16, 1, 32), (10, 16, 1, 24), (100, 8, 2, 48)):
        kp, vp = ref.pools(30, hkv, d, BF, g)
        cache = PagedCache(hq, hkv, d, 30, k_pages=kp, v_pages=vp)
        table = widened(ref.table_of([30], 30, g))
        raw = []

        def guarded(shape, dtype):
            bytes_ = math.prod(shape) * dtype.itemsize
            r = torch.full((bytes_ + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
            raw.append((r, bytes_))
            return r[4096:4096 + bytes_].view(dtype).view(shape)
        o, lse = guarded((n, hq, d), BF), guarded((hq, n), torch.float32)
        ws = guarded((cache.workspace_bytes(n, 1, 200),), torch.uint8)
        cache.attend(rand((n, hq, d), BF, g), table, ref.i32([0, n]), ref.i32([0]), ref.i32([30 * PAGE]), causal=True,
                     o=o, lse=lse, workspace=ws)
        assert cache.status() == _abi.BCA_OK
        for r, b in raw:
            assert (r[:4096] == 0xA5).all() and (r[4096 + b:] == 0xA5).all()


@pytest.mark.parametrize("rows,wide", [(1, False), (1, True), (12, False), (200, False)])
def test_forced_timeout_is_reported_and_the_context_stays_usable(rows, wide):
    g = gen(15)
    kp, vp = ref.pools(4, 2, 48, BF, g)
    table = ref.table_of([4], 4, g)
    table = widened(table) if wide else table
    q = rand((rows, 16, 48), BF, g)
    args = (q, table, ref.i32([0, rows]), ref.i32([0]), ref.i32([512]))
    bad = PagedCache(16, 2, 48, 4, k_pages=kp, v_pages=vp, test_force_timeout=True)
    bad.attend(*args)
    assert bad.status() == _abi.BCA_ERR_DEVICE_TIMEOUT
    assert bad.status() == _abi.BCA_OK
    good = PagedCache(16, 2, 48, 4, k_pages=kp, v_pages=vp)
    o = good.attend(*args)
    assert good.status() == _abi.BCA_OK
    wo, _, bo, _ = ref.attend(q, kp[0], vp[0], table, [0, rows], [0], [0], [512], False)
    no_worse(o, wo, bo, "o")


def test_refusals_of_the_binding():
    g = gen(16)
    cache = PagedCache(4, 2, 48, 6, layers=2)
    k = rand((5, 2, 48), BF, g)
    q = rand((5, 4, 48), BF, g)
    table, off, one, pos = ref.i32([[0, 1]]), ref.i32([0, 5]), ref.i32([5]), positions(5, g)
    gain = torch.ones(48, device="cuda")
    good = dict(k=k, v=k, table=table, off=off, start=ref.i32([0]), pos=pos, k_gain=gain)
    cache.write(**good)
    for bad in (dict(k=k.half()), dict(v=k[:4]), dict(k=k.cpu()), dict(table=table[0]), dict(table=table.long()),
                dict(off=off[:1]), dict(off=off.cpu()), dict(start=off), dict(pos=pos[:, :2]), dict(pos=None),
                dict(k_gain=gain.half()), dict(k_gain=gain[:47]), dict(layer=2), dict(layer=-1),
                dict(k=rand((2, 5, 48), BF, g).transpose(0, 1))):
        with pytest.raises(ValueError):
            cache.write(**{**good, **bad})
    with pytest.raises(TypeError):
        cache.write(**{**good, "k": None})
    good = dict(q=q, table=table, off=off, k_begin=ref.i32([0]), k_end=one, seq=ref.i32([0]), pos=pos, q_gain=gain)
    o = cache.attend(**good)
    assert o.dtype is BF and o.shape == (5, 4, 48)
    small = torch.empty(cache.workspace_bytes(5, 1, 200) - 1, dtype=torch.uint8, device="cuda")
    wide = torch.full((1, 200), -1, dtype=torch.int32, device="cuda")
    for bad in (dict(q=q.half()), dict(q=q[:, :3]), dict(q=q[:4]), dict(table=table.cpu()), dict(off=off.long()),
                dict(k_begin=off), dict(k_end=one.cpu()), dict(seq=off), dict(pos=None), dict(q_gain=gain.double()),
                dict(o=o.float()), dict(o=o[:3]), dict(lse=torch.empty(4, 4, device="cuda")), dict(table=wide, workspace=small),
                dict(table=wide, workspace=small.cpu()), dict(layer=2), dict(off=off[:0]),
                dict(table=ref.i32([[0, 1], [2, 3]]), seq=None)):
        with pytest.raises(ValueError):
            cache.attend(**{**good, **bad})
    for bad in ([[0, 6]], [[-1, 0]], [[0, 1], [2, 1]], [[0, 1], [1, 2]], torch.tensor([[0, 1], [1, 2]])):
        with pytest.raises(BcaError) as e:
            cache.copy_pages(bad)
        assert e.value.code == _abi.BCA_ERR_BAD_PAGE
    for bad in (torch.zeros((1, 2), dtype=torch.int32, device="cuda"), [[0, 1, 2]], [0, 1], [[0.0, 1.0]]):
        with pytest.raises(ValueError):
            cache.copy_pages(bad)
    cache.copy_pages([])
    with pytest.raises(ValueError):
        PagedCache(4, 2, 48, 6, k_pages=cache.k_pages)       # of a cache with another shape
    # nothing to do is no error
    assert cache.attend(q[:0], table, ref.i32([0, 0]), ref.i32([0]), one).shape == (0, 4, 48)
    assert cache.attend(q[:0], table, ref.i32([0, 0]), ref.i32([0]), one, pos=pos[:0], q_gain=gain).shape == (0, 4, 48)
    cache.write(k[:0], k[:0], table, ref.i32([0, 0]), ref.i32([0]))
    cache.write(k[:0], k[:0], table, ref.i32([0, 0]), ref.i32([0]), pos=pos[:0], k_gain=gain)
    cache.close()
    for call in (lambda: cache.attend(**good), lambda: cache.copy_pages([])):
        with pytest.raises(BcaError):
            call()


def test_allocations_of_a_call_on_another_stream_belong_to_it():
    """Calls on a side stream while the current one keeps reusing freed memory."""
    g = gen(17)
    kp, vp = ref.pools(40, 1, 48, BF, g)
    cache = PagedCache(16, 1, 48, 40, k_pages=kp, v_pages=vp)
    table = torch.full((1, 200), -1, dtype=torch.int32, device="cuda")   # wide: with a workspace
    table[:, :40] = ref.table_of([40], 40, g)
    q = rand((2, 16, 48), BF, g)
    args = (q, table, ref.i32([0, 2]), ref.i32([0]), ref.i32([5001]))
    want = cache.attend(*args, causal=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(20):
        got.append(cache.attend(*args, causal=True, stream=side))
        for _ in range(3):
            torch.full((cache.workspace_bytes(2, 1, 200),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)


@pytest.mark.parametrize("hq,hkv,new", [(400, 1, [1, 3]), (130, 2, [1, 1, 2]), (9, 9, [40, 3]), (20, 20, [1] * 9)])
def test_attend_odd_groups_and_head_counts(hq, hkv, new):
    check_attend(hq, hkv, 24, BF, new, [300 + 7 * i for i in range(len(new))], True, True, 18)


@pytest.mark.parametrize("d", [24, 32, 48])
def test_any_positions_and_bases(d):
    """Negative and far positions, bases below, at and above 1: the angle is that of the 64-bit
    product (off by at most 2^31 * 2^-53 of its own turns in the reference, 2 pi 2^-22 rad)."""
    g = gen(19)
    # the ABI takes bases in fp32, so the reference has to start from fp32's 0.7 too: at 2^31 their
    # difference, 1.2e-8, is a hundred thousand turns
    base = tuple(torch.tensor(x, dtype=torch.float32).item() for x in (0.7, 1.0, 3e5))
    edge = torch.tensor([0, 1, -1, 12345678, -87654321, 2 ** 31 - 1, -2 ** 31], device="cuda", dtype=torch.int32)
    pos = edge[torch.randint(0, 7, (60, 3), generator=g, device="cuda")].contiguous()
    kp, vp = ref.pools(2, 2, d, BF, g)
    cache = PagedCache(4, 2, d, 2, rope_base=base, k_pages=kp, v_pages=vp)
    k, v, q = rand((60, 2, d), BF, g), rand((60, 2, d), BF, g), rand((60, 4, d), BF, g)
    table = ref.i32([[1]])
    cache.write(k, v, table, ref.i32([0, 60]), ref.i32([30]), pos=pos)
    got, _ = ref.unpage(kp[0], vp[0], [1], 90)
    want = ref.prologue(k, pos, None, base)
    # base 0.7: angles grow with the pair, up to 2^31 * 0.7^(-7/8) turns / 2 pi
    bound = 2.0 ** -11 * want.abs() + 2.0 ** -25 + 2.0 ** -18 * want.abs().amax(2, keepdim=True)
    no_worse(got[30:], want, bound, "k")
    o = cache.attend(q, table, ref.i32([0, 60]), ref.i32([30]), ref.i32([90]), pos=pos)
    assert cache.status() == _abi.BCA_OK
    wo, _, bo, _ = ref.attend(q, kp[0], vp[0], table, [0, 60], [0], [30], [90], False, pos, None, base)
    # the queries' angles: 2^-20 of a value more (cos and sin to 2^-20.5 each), in every product of a score
    no_worse(o, wo, bo + 2.0 ** -16, "o")


def test_large_values_survive_a_moving_reference():
    """Values near 2^90 while the scores rise by a hundred: no sum may overflow on the way."""
    g = gen(20)
    d = 32
    kp, vp = ref.pools(12, 1, d, BF, g)
    vp *= 2.0 ** 90
    table = ref.table_of([12], 12, g)
    for i, p in enumerate(table[0].tolist()):
        kp[0, p] *= 0.5 + 2 * i
    cache = PagedCache(8, 1, d, 12, k_pages=kp, v_pages=vp)
    for n in (1, 5, 20, 60):
        q = rand((n, 8, d), BF, g)
        o = cache.attend(q, table, ref.i32([0, n]), ref.i32([0]), ref.i32([1500]), causal=True)
        assert cache.status() == _abi.BCA_OK
        wo, _, bo, _ = ref.attend(q, kp[0], vp[0], table, [0, n], [0], [0], [1500], True)
        assert wo.isfinite().all()
        no_worse(o, wo, bo, "o")


def test_tables_without_rows_or_columns():
    g = gen(21)
    cache = PagedCache(4, 2, 48, 3)
    for shape in ((0, 5), (2, 0), (0, 0)):
        table = torch.zeros(shape, dtype=torch.int32, device="cuda")
        for n in (1, 40, 300):
            q, k = rand((2 * n, 4, 48), BF, g), rand((2 * n, 2, 48), BF, g)
            lse = torch.zeros((4, 2 * n), device="cuda")
            o = cache.attend(q, table, ref.i32([0, n, 2 * n]), ref.i32([0, 0]), ref.i32([10, 0]), seq=ref.i32([0, 1]), lse=lse)
            assert (o == 0).all() and (lse == -math.inf).all()
            cache.write(k, k, table, ref.i32([0, n, 2 * n][:shape[0] + 1]), ref.i32([0] * shape[0]))
            assert cache.status() == (_abi.BCA_ERR_BAD_PAGE if shape[0] else _abi.BCA_OK)
    assert cache.attend(rand((3, 4, 48), BF, g), table, ref.i32([0]), ref.i32([]), ref.i32([]), seq=ref.i32([])).shape[0] == 3


def test_pools_beyond_32_bits():
    """Page numbers whose bytes and elements pass 2^32: the last pages of a pool of 10 GB."""
    g = gen(22)
    hkv, d, pages, layers = 8, 48, 26000, 2
    cache = PagedCache(16, hkv, d, pages, layers=layers)
    assert cache.pool_bytes * layers > 2 ** 32
    row = [pages - 1, pages - 3, 5]
    table, n = ref.i32([row]), 300
    k, v, q = rand((n, hkv, d), BF, g), rand((n, hkv, d), BF, g), rand((2, 16, d), BF, g)
    cache.write(k, v, table, ref.i32([0, n]), ref.i32([0]), layer=1)
    got_k, got_v = ref.unpage(cache.k_pages[1], cache.v_pages[1], row, n)
    assert torch.equal(got_k, k.half().double()) and torch.equal(got_v, v.double())
    cache.copy_pages([[pages - 1, 7], [pages - 3, pages - 2]])
    moved = [7, pages - 2, 5]
    for r in (row, moved):
        o = cache.attend(q, ref.i32([r]), ref.i32([0, 2]), ref.i32([0]), ref.i32([n]), causal=True, layer=1)
        assert cache.status() == _abi.BCA_OK
        wo, _, bo, _ = ref.attend(q, cache.k_pages[1], cache.v_pages[1], ref.i32([r]), [0, 2], [0], [0], [n], True)
        no_worse(o, wo, bo, "o")


def test_copies_of_thousands_of_pages_and_in_a_graph():
    g = gen(23)
    moves = 4500
    kp, vp = ref.pools(2 * moves, 1, 24, BF, g)
    cache = PagedCache(1, 1, 24, 2 * moves, k_pages=kp, v_pages=vp)
    order = torch.randperm(2 * moves, generator=g, device="cuda")
    src, dst = order[:moves], order[moves:]
    wk, wv = kp.clone(), vp.clone()
    wk[:, dst], wv[:, dst] = kp[:, src], vp[:, src]
    pairs = torch.stack([src, dst], 1).cpu()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.copy_pages(pairs)
    pairs.zero_()                                # read before the call returned
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kp, wk) and torch.equal(vp, wv)


def test_calls_on_two_streams_at_once():
    g = gen(24)
    kp, vp = ref.pools(80, 2, 48, BF, g)
    cache = PagedCache(16, 2, 48, 80, k_pages=kp, v_pages=vp)
    table = widened(ref.table_of([40, 40], 80, g))
    calls = []
    for n in (1, 4, 20, 500):
        q = rand((2 * n, 16, 48), BF, g)
        calls.append((q, table, ref.i32([0, n, 2 * n]), ref.i32([3, 0]), ref.i32([5001, 4700])))
    want = [cache.attend(*c, causal=True) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[cache.attend(*c, causal=True, stream=s) for c, s in zip(calls, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    assert cache.status() == _abi.BCA_OK
    assert all(torch.equal(x, w) for r in got for x, w in zip(r, want))
