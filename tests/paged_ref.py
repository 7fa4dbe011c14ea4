"""The paged cache's operators in 64 bits, written out from their definitions, and inputs for
them.  Attention also returns what bounds the kernel's error, element by element."""
import math

import torch

PAGE = 128
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half a step


def prologue(x, pos, gain, base=(1e4, 1e4, 1e4), eps=1e-6):
    x = x.double()
    if pos is None:
        return x
    d = x.shape[2]
    x = x / torch.sqrt(x.square().mean(2, keepdim=True) + eps)
    if gain is not None:
        x = x * gain.double()
    p = d // 2 // 3
    y = x.clone()
    for axis in range(3):
        for i in range(p):
            ang = (pos[:, axis].double() * base[axis] ** (-i / p))[:, None]
            c = 2 * (axis * p + i)
            y[..., c] = x[..., c] * ang.cos() - x[..., c + 1] * ang.sin()
            y[..., c + 1] = x[..., c] * ang.sin() + x[..., c + 1] * ang.cos()
    return y


def unpage(k_pages, v_pages, row, tokens):
    """Keys and values [tokens, Hkv, D] of a list of pages (absent ones NaN)."""
    hkv, d = k_pages.shape[1], v_pages.shape[3]
    k = torch.full((len(row) * PAGE, hkv, d), math.nan, dtype=torch.float64, device=k_pages.device)
    v = k.clone()
    for i, p in enumerate(row):
        if 0 <= p < k_pages.shape[0]:
            k[i * PAGE:(i + 1) * PAGE] = k_pages[p].permute(2, 0, 1, 3).reshape(PAGE, hkv, d).double()
            v[i * PAGE:(i + 1) * PAGE] = v_pages[p].permute(1, 3, 0, 2).reshape(PAGE, hkv, d).double()
    return k[:tokens], v[:tokens]


def attend(q, k_pages, v_pages, table, off, seq, k_begin, k_end, causal, pos=None, gain=None,
           base=(1e4, 1e4, 1e4)):
    """(O, LSE [Hq, nq], error bound of O, error bound of LSE), row by row over the keys that
    are there.  The bounds count, to first order with a tenth on top: q_hat rounded to fp16
    (2^-11 of each product of a score), P rounded to the values' type, O rounded once, and
    2^-18 for the fp32 steps (a dozen of 2^-24, ex2 2^-22, products of up to 48 terms)."""
    t = q.dtype
    qh = prologue(q, pos, gain, base)
    nq, hq, d = q.shape
    hkv = k_pages.shape[1]
    grp = hq // hkv
    o = torch.zeros((nq, hq, d), dtype=torch.float64, device=q.device)
    bo = torch.zeros_like(o)
    lse = torch.full((hq, nq), -math.inf, dtype=torch.float64, device=q.device)
    bl = torch.zeros_like(lse)
    width = table.shape[1]
    tab = table.tolist()
    for i in range(len(k_begin)):
        b, lo, end = seq[i], max(k_begin[i], 0), min(k_end[i], width * PAGE)
        if not 0 <= b < len(tab) or end <= lo or off[i + 1] <= off[i]:
            continue
        kk, vv = unpage(k_pages, v_pages, tab[b], end)
        here = torch.tensor([0 <= tab[b][j // PAGE] < k_pages.shape[0] for j in range(lo, end)], device=q.device)
        for r in range(off[i], off[i + 1]):
            last = min(end, k_end[i] - (off[i + 1] - 1 - r)) if causal else end
            see = here[:max(last - lo, 0)]
            if last <= lo or not see.any():
                continue
            kr = kk[lo:last][see].repeat_interleave(grp, 1)
            vr = vv[lo:last][see].repeat_interleave(grp, 1)
            s = (qh[r] * kr).sum(2) / math.sqrt(d)
            ds = ((qh[r] * kr).abs().sum(2) / math.sqrt(d)).amax(0) * (2.0 ** -11 + 2.0 ** -18) + 2.0 ** -18
            l = torch.logsumexp(s, 0)
            p = torch.exp(s - l)[:, :, None]
            o[r] = (p * vr).sum(0)
            lse[:, r] = l
            a = (p * vr.abs()).sum(0)
            bo[r] = 1.1 * a * (2 * ds[:, None] + U[t]) + 1.1 * U[t] * o[r].abs() + 1e-7
            bl[:, r] = 1.1 * ds + 2.0 ** -20 * l.abs()
    return o, lse, bo, bl


def attend_rows(q, k_pages, v_pages, table, off, seq, k_begin, k_end, rows, pos=None, gain=None):
    """``attend`` of some rows of full slices: (O [rows], LSE [Hq, rows], and their bounds)."""
    which = [max(i for i in range(len(seq)) if off[i] <= r) for r in rows]
    return attend(q[rows], k_pages, v_pages, table, list(range(len(rows) + 1)), [seq[i] for i in which],
                  [k_begin[i] for i in which], [k_end[i] for i in which], False,
                  None if pos is None else pos[rows], gain)


def pools(pages, hkv, d, dtype, gen, layers=1):
    k = torch.empty((layers, pages, hkv, d // 8, PAGE, 8), dtype=torch.float16, device="cuda").normal_(generator=gen)
    v = torch.empty((layers, pages, hkv, PAGE // 8, d, 8), dtype=dtype, device="cuda").normal_(generator=gen)
    return k, v


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets(lengths):
    off = [0]
    for n in lengths:
        off.append(off[-1] + n)
    return off


def table_of(need, pages, gen, absent=-1):
    """Rows of distinct pages in random order, `absent` behind each row's own."""
    assert sum(need) <= pages
    order = torch.randperm(pages, generator=gen, device="cuda").tolist()
    width = max(max(need, default=0), 1)
    rows, at = [], 0
    for n in need:
        rows.append(order[at:at + n] + [absent] * (width - n))
        at += n
    return i32(rows)
