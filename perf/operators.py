"""The paged KV cache's operators as measured work: writing new tokens into pages (QK-Norm and 3D RoPE
of the keys on the way), copying pages (fork, compaction), and attention of new tokens over the pages.

Page layout (128 tokens a page; `layers` pools side by side):
  k_pages [layers][pages][Hkv][D/8][128][8] fp16      element (token s, channel c) at [..][c/8][s][c%8]
  v_pages [layers][pages][Hkv][16][D][8] io type      element (token s, channel c) at [..][s/8][c][s%8]
A table row lists a sequence's pages in order, so its token p lies in page table[p / 128], slot p % 128.

With `own` false, run() computes the plain form; with `own` true it calls the framework's kernels.
"""
import math

import torch

own = False

PAGE = 128
BASE = (10000.0, 10000.0, 10000.0)
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # One step of 64 token-by-token streams: each appends a single key and value at its own position.
        dict(name="write_tokens", op="write", seqs=64, new_min=1, new_max=1, at_min=0, at_max=4001, hkv=8, d=48,
             dtype="bf16", prologue=True, gh=45, gw=80),
        # The 4-chunk denoising window of the 4.5B shape (6 x 16 x 16 tokens a chunk) written behind 8 chunks.
        dict(name="write_window_b45", op="write", seqs=1, new_min=6144, new_max=6144, at_min=12288, at_max=12288,
             hkv=8, d=24, dtype="bf16", prologue=True, gh=16, gw=16),
        # Two 720p streams, one chunk each (6 x 45 x 80 tokens), behind a chunk that ends inside a page.
        dict(name="write_chunk_720p", op="write", seqs=2, new_min=21600, new_max=21600, at_min=21600, at_max=43200,
             hkv=8, d=48, dtype="bf16", prologue=True, gh=45, gw=80),
        # Forked streams that write again: the half-full tail page of each is copied before its first write.
        dict(name="copy_fork_tails", op="copy", moves=48, layers=1, hkv=8, d=48, dtype="bf16"),
        # Compaction of a fragmented pool over two layers.
        dict(name="copy_compact", op="copy", moves=1024, layers=2, hkv=8, d=48, dtype="bf16"),
        # The smallest call: one token of one stream over one chunk of the 4.5B shape.
        dict(name="attend_token", op="attend", seqs=1, new_min=1, new_max=1, ctx_min=1535, ctx_max=1535, block=0,
             kv_range=0, hq=128, hkv=8, d=24, dtype="bf16", prologue=True, gh=16, gw=16),
        # A serving batch of single tokens, contexts from one token to one and a half 720p chunks.
        dict(name="attend_batch", op="attend", seqs=32, new_min=1, new_max=1, ctx_min=0, ctx_max=32400, block=0,
             kv_range=0, hq=128, hkv=8, d=48, dtype="bf16", prologue=True, gh=45, gw=80),
        # One token over the eight clean chunks that a 720p window keeps in its cache.
        dict(name="attend_long", op="attend", seqs=1, new_min=1, new_max=1, ctx_min=172800, ctx_max=172800, block=0,
             kv_range=0, hq=128, hkv=8, d=48, dtype="bf16", prologue=True, gh=45, gw=80),
        # A few proposed tokens a stream, checked together (token-causal); three query heads a KV head, fp16.
        dict(name="attend_proposed", op="attend", seqs=24, new_min=2, new_max=5, ctx_min=100, ctx_max=9001, block=0,
             kv_range=0, hq=12, hkv=4, d=32, dtype="fp16", prologue=False, gh=16, gw=16),
        # Ragged token-causal chunks of several streams, fp16, odd lengths.
        dict(name="attend_ragged", op="attend", seqs=6, new_min=201, new_max=2001, ctx_min=0, ctx_max=5001, block=0,
             kv_range=0, hq=24, hkv=8, d=32, dtype="fp16", prologue=False, gh=16, gw=16),
        # The 4.5B window, one head shard of four: 4 chunks, each over the 8 chunks before it and its own.
        dict(name="attend_window_b45", op="attend", seqs=1, new_min=6144, new_max=6144, ctx_min=12288, ctx_max=12288,
             block=1536, kv_range=8, hq=32, hkv=2, d=24, dtype="bf16", prologue=True, gh=16, gw=16),
        # Half a 720p chunk over the chunk before it and itself, one head shard of eight: the largest work.
        dict(name="attend_chunk_720p", op="attend", seqs=1, new_min=10800, new_max=10800, ctx_min=21600,
             ctx_max=21600, block=10800, kv_range=0, hq=16, hkv=1, d=48, dtype="bf16", prologue=True, gh=45, gw=80),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "copy", "attend", "attend", "attend"])
    d = rng.choice([24, 32, 48])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    gh, gw = rng.choice([(16, 16), (32, 32), (45, 80)])
    if op == "write":
        seqs = _log(rng, 1, 64)
        most = _log(rng, 1, max(1, 43200 // seqs))
        at = _log(rng, 1, 30000)
        return dict(op=op, seqs=seqs, new_min=rng.choice([0, 1, most]) if most > 1 else 1, new_max=most,
                    at_min=rng.randrange(at), at_max=at, hkv=rng.choice([1, 2, 4, 8]), d=d, dtype=dtype,
                    prologue=rng.random() < 0.7, gh=gh, gw=gw)
    if op == "copy":
        return dict(op=op, moves=_log(rng, 1, 1024), layers=rng.choice([1, 2]), hkv=rng.choice([1, 2, 4, 8]), d=d,
                    dtype=dtype)
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 8, 16])
    form = rng.choice(["token", "proposed", "causal", "block"])
    seqs = _log(rng, 1, 48 if form in ("token", "proposed") else 6)
    new = {"token": 1, "proposed": rng.randint(2, 8), "causal": _log(rng, 9, 2001), "block": _log(rng, 9, 6144)}[form]
    ctx = _log(rng, 1, 60000)
    # at most half the score values of the largest listed case, at most the keys of the longest
    while hkv * group * seqs * new * (ctx + new) > 2_800_000_000 or seqs * hkv * (ctx + new) > 4_100_000:
        if seqs > 1:
            seqs = seqs // 2
        elif ctx > 4 * new:
            ctx = ctx // 2
        else:
            new = new // 2
    few = 1 if form in ("token", "proposed") else rng.choice([1, new])
    return dict(op=op, seqs=seqs, new_min=few, new_max=new, ctx_min=rng.choice([0, ctx // 7, ctx]), ctx_max=ctx,
                block=max(1, new // rng.choice([1, 2, 4])) if form == "block" else 0, kv_range=rng.choice([0, 0, 1, 3]),
                hq=hkv * group, hkv=hkv, d=d, dtype=dtype, prologue=rng.random() < 0.7, gh=gh, gw=gw)


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, the first hi and the last lo, the others spread between them."""
    golden = 0.6180339887498949
    return [hi if i == 0 else lo if i == n - 1 else lo + int((hi - lo + 1) * ((i * golden) % 1.0)) for i in range(n)]


def _write_lengths(c):
    return _spread(c["new_min"], c["new_max"], c["seqs"]), _spread(c["at_min"], c["at_max"], c["seqs"])


def _segments(c):
    """Rows of the queries that see one range of keys: (table row, rows, first key, end of keys) each."""
    out = []
    for b, (n, ctx) in enumerate(zip(_spread(c["new_min"], c["new_max"], c["seqs"]),
                                     _spread(c["ctx_min"], c["ctx_max"], c["seqs"]))):
        step = c["block"] or max(n, 1)
        for r in range(0, n, step):
            rows = min(step, n - r)
            first = max(0, ctx + r - c["kv_range"] * step) if c["kv_range"] and c["block"] else 0
            out.append((b, rows, first, ctx + r + rows))
    return out


def _pages_of(tokens):
    return -(-tokens // PAGE)


def work(case):
    c = case
    if c["op"] == "write":
        n = sum(_write_lengths(c)[0])
        values = 2 * n * c["hkv"] * c["d"]
        flops = n * c["hkv"] * c["d"] * 8 if c["prologue"] else 0
        return {"bytes": 2 * 2 * values + (12 * n if c["prologue"] else 0), "flops": flops}
    if c["op"] == "copy":
        return {"bytes": 2 * c["moves"] * c["layers"] * c["hkv"] * c["d"] * PAGE * 4, "flops": 0}
    seg = _segments(c)
    rows = sum(n for _, n, _, _ in seg)
    if c["block"]:
        pairs = sum(n * (end - first) for _, n, first, end in seg)
    else:
        pairs = sum(n * (end - first) - n * (n - 1) // 2 for _, n, first, end in seg)
    seen = {}
    for b, _, first, end in seg:
        lo, hi = seen.get(b, (first, end))
        seen[b] = (min(lo, first), max(hi, end))
    keys = sum(hi - lo for lo, hi in seen.values())
    return {"bytes": keys * c["hkv"] * c["d"] * 4 + rows * c["hq"] * c["d"] * 4, "flops": 4 * c["d"] * c["hq"] * pairs}


# ------------------------------------------------------------------------------------------ the inputs

def _offsets(lengths, device="cuda"):
    off = [0]
    for n in lengths:
        off.append(off[-1] + n)
    return torch.tensor(off, dtype=torch.int32, device=device)


def _positions(lengths, starts, gh, gw, device="cuda"):
    """(t, h, w) of each new token, raster order over frames of gh x gw tokens."""
    if not sum(lengths):
        return torch.zeros((0, 3), dtype=torch.int32, device=device)
    p = torch.cat([torch.arange(s, s + n, device=device) for n, s in zip(lengths, starts)])
    return torch.stack([p // (gh * gw), p % (gh * gw) // gw, p % gw], 1).to(torch.int32)


def _pool(c, pages, layers, gen):
    """Pages with what earlier tokens left in them: keys as an RMS norm leaves them, values about one."""
    t = TYPES[c["dtype"]]
    k = torch.empty((layers, pages, c["hkv"], c["d"] // 8, PAGE, 8), dtype=torch.float16, device="cuda")
    v = torch.empty((layers, pages, c["hkv"], PAGE // 8, c["d"], 8), dtype=t, device="cuda")
    return k.normal_(generator=gen), v.normal_(generator=gen)


def _table(need, gen, spare):
    """A table row for each sequence, its pages anywhere in the pool, and the pool's size."""
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((len(need), max(max(need), 1)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    t = TYPES[c["dtype"]]
    s = {"op": c["op"]}
    hq = c.get("hq", c["hkv"])
    if c["op"] == "copy":
        pages, layers = 2 * c["moves"] + 3, c["layers"]
        order = torch.randperm(pages, generator=gen, device="cuda")
        s["src"], s["dst"] = order[:c["moves"]], order[c["moves"]:2 * c["moves"]]
        s["pairs"] = torch.stack([s["src"], s["dst"]], 1).to(torch.int32).cpu()  # the page tables live on the host
    else:
        layers = 1
        if c["op"] == "write":
            lengths, starts = _write_lengths(c)
            need = [_pages_of(n + a) for n, a in zip(lengths, starts)]
            s["off"] = _offsets(lengths)
            s["start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
            rows = sum(lengths)
            s["k"] = torch.empty((rows, c["hkv"], c["d"]), dtype=t, device="cuda").normal_(generator=gen)
            s["v"] = torch.empty((rows, c["hkv"], c["d"]), dtype=t, device="cuda").normal_(generator=gen)
        else:
            seg = _segments(c)
            lengths = _spread(c["new_min"], c["new_max"], c["seqs"])
            starts = _spread(c["ctx_min"], c["ctx_max"], c["seqs"])
            need = [_pages_of(n + a) for n, a in zip(lengths, starts)]
            s["off"] = _offsets([x[1] for x in seg])
            for name, i in (("seq", 0), ("k_begin", 2), ("k_end", 3)):
                s[name] = torch.tensor([x[i] for x in seg], dtype=torch.int32, device="cuda")
            s["causal"] = not c["block"]
            s["most_new"] = max(lengths)
            rows = sum(lengths)
            s["q"] = torch.empty((rows, hq, c["d"]), dtype=t, device="cuda").normal_(generator=gen)
        s["pos"] = _positions(lengths, starts, c["gh"], c["gw"]) if c["prologue"] else None
        s["gain"] = 1 + 0.1 * torch.randn(c["d"], generator=gen, device="cuda") if c["prologue"] else None
        s["table"], pages = _table(need, gen, spare=2)
    s["k_pages"], s["v_pages"] = _pool(c, pages, layers, gen)
    if own:
        from block_causal_attention_b200 import PagedCache
        s["cache"] = PagedCache(hq, c["hkv"], c["d"], pages, layers=layers, dtype=t, rope_base=BASE, eps=EPS,
                                k_pages=s["k_pages"], v_pages=s["v_pages"])
    return s


# ------------------------------------------------------------------------------------------ one pass

def run(state):
    s = state
    if own:
        if s["op"] == "write":
            s["cache"].write(s["k"], s["v"], s["table"], s["off"], s["start"], pos=s["pos"], k_gain=s["gain"])
            return s["k_pages"], s["v_pages"]
        if s["op"] == "copy":
            s["cache"].copy_pages(s["pairs"])
            return s["k_pages"], s["v_pages"]
        return s["cache"].attend(s["q"], s["table"], s["off"], s["k_begin"], s["k_end"], seq=s["seq"],
                                 causal=s["causal"], pos=s["pos"], q_gain=s["gain"])
    return {"write": _plain_write, "copy": _plain_copy, "attend": _plain_attend}[s["op"]](s)


def _rotated(x, pos, gain):
    """QK-Norm with gain and 3D RoPE of the rows x [N, H, D], in 32 bits (the angles in 64)."""
    d = x.shape[2]
    x = x.float()
    if pos is None:
        return x
    x = x * torch.rsqrt(x.square().mean(2, keepdim=True) + EPS) * gain
    p = d // 2 // 3
    base = torch.tensor(BASE, dtype=torch.float64, device=x.device)
    freq = base[:, None] ** (-torch.arange(p, dtype=torch.float64, device=x.device) / p)
    angle = (pos.double()[:, :, None] * freq).reshape(len(pos), 1, 3 * p)
    cos, sin = angle.cos().float(), angle.sin().float()
    a, b = x[:, :, 0:6 * p:2], x[:, :, 1:6 * p:2]
    turned = torch.stack([a * cos - b * sin, a * sin + b * cos], 3).flatten(2)
    return torch.cat([turned, x[:, :, 6 * p:]], 2)


def _plain_write(s):
    k, v, table, off = s["k"], s["v"], s["table"].long(), s["off"].long()
    n, hkv, d = k.shape
    row = torch.arange(n, device=k.device)
    b = torch.searchsorted(off[1:], row, right=True)
    at = s["start"].long()[b] + row - off[b]
    page, slot = table[b, at // PAGE], at % PAGE
    k_pages, v_pages = s["k_pages"][0], s["v_pages"][0]
    k_pages[page, :, :, slot] = _rotated(k, s["pos"], s["gain"]).to(k_pages.dtype).view(n, hkv, d // 8, 8)
    v_pages[page, :, slot // 8, :, slot % 8] = v
    return s["k_pages"], s["v_pages"]


def _plain_copy(s):
    s["k_pages"][:, s["dst"]] = s["k_pages"][:, s["src"]]
    s["v_pages"][:, s["dst"]] = s["v_pages"][:, s["src"]]
    return s["k_pages"], s["v_pages"]


def _plain_attend(s):
    q, table, off, seq = s["q"], s["table"].long(), s["off"].long(), s["seq"].long()
    n, hq, d = q.shape
    k_pages, v_pages = s["k_pages"][0], s["v_pages"][0]
    hkv, seqs, width = k_pages.shape[1], table.shape[0], table.shape[1]
    keys = k_pages[table].permute(0, 2, 1, 4, 3, 5).reshape(seqs, hkv, 1, width * PAGE, d).float()
    values = v_pages[table].permute(0, 2, 1, 3, 5, 4).reshape(seqs, hkv, 1, width * PAGE, d).float()
    # each row's slice, its sequence, its place among the sequence's rows, and the keys it sees
    row = torch.arange(n, device=q.device)
    g = torch.searchsorted(off[1:], row, right=True)
    b = seq[g]
    place = row - off[torch.searchsorted(seq, b)]
    lo, hi = s["k_begin"].long()[g], s["k_end"].long()[g]
    if s["causal"]:
        hi = hi - (off[g + 1] - 1 - row)
    grid = torch.zeros((seqs, s["most_new"], hq, d), device=q.device)
    grid[b, place] = _rotated(q, s["pos"], s["gain"]) / math.sqrt(d)
    first = torch.zeros((seqs, s["most_new"]), dtype=torch.long, device=q.device)
    end = torch.zeros_like(first)
    first[b, place], end[b, place] = lo, hi
    at = torch.arange(width * PAGE, device=q.device)
    hidden = (at < first[:, :, None]) | (at >= end[:, :, None])
    grid = grid.view(seqs, -1, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    score = grid @ keys.transpose(3, 4)
    score.masked_fill_(hidden[:, None, None], -math.inf)
    top = score.amax(4, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    score.sub_(top).exp_()
    total = score.sum(4, keepdim=True)
    out = (score @ values) / torch.where(total > 0, total, 1)
    out = out.permute(0, 3, 1, 2, 4).reshape(seqs, -1, hq, d)
    return out[b, place].to(q.dtype)


# ------------------------------------------------------------------------------------------ in 64 bits

def _turn64(x, where, gain):
    """RMS norm and rotation of rows x [N, H, D] at positions `where` [N, 3], pair by pair, in 64 bits."""
    x = x.double()
    if where is None:
        return x
    d = x.shape[-1]
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS) * gain.double()
    out = y.clone()
    pairs = (d // 2) // 3
    for axis in range(3):
        for i in range(pairs):
            c = 2 * (axis * pairs + i)
            angle = where[:, axis].double()[:, None] * BASE[axis] ** (-i / pairs)
            z = torch.complex(y[..., c], y[..., c + 1]) * torch.polar(torch.ones_like(angle), angle)
            out[..., c], out[..., c + 1] = z.real, z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
    if s["op"] == "copy":
        for a, b in s["pairs"].tolist():
            k_pages[:, b].copy_(k_pages[:, a])
            v_pages[:, b].copy_(v_pages[:, a])
        return k_pages, v_pages
    off, table = s["off"].tolist(), s["table"].tolist()
    if s["op"] == "write":
        turned = _turn64(s["k"], s["pos"], s["gain"])
        for b, start in enumerate(s["start"].tolist()):
            r = off[b]
            while r < off[b + 1]:
                p = start + r - off[b]
                page, slot = table[b][p // PAGE], p % PAGE
                m = min(PAGE - slot, off[b + 1] - r)
                kk = turned[r:r + m].unflatten(2, (-1, 8)).permute(1, 2, 0, 3)     # [Hkv, D/8, m, 8]
                k_pages[0, page, :, :, slot:slot + m] = kk
                flat = v_pages[0, page].transpose(2, 3).flatten(1, 2).clone()      # [Hkv, 128, D]
                flat[:, slot:slot + m] = s["v"][r:r + m].double().transpose(0, 1)
                v_pages[0, page] = flat.unflatten(1, (-1, 8)).transpose(2, 3)
                r += m
        return k_pages, v_pages
    q = _turn64(s["q"], s["pos"], s["gain"])
    hq, hkv, d = q.shape[1], k_pages.shape[2], q.shape[2]
    out = torch.zeros_like(q)
    for g, (b, lo, hi) in enumerate(zip(s["seq"].tolist(), s["k_begin"].tolist(), s["k_end"].tolist())):
        if hi <= lo:
            continue
        ids = torch.tensor(table[b][lo // PAGE:_pages_of(hi)], device=q.device)
        cut = slice(lo - lo // PAGE * PAGE, hi - lo // PAGE * PAGE)
        for h in range(hkv):
            keys = k_pages[0, ids, h].transpose(1, 2).flatten(2).flatten(0, 1)[cut]          # [keys, D]
            values = v_pages[0, ids, h].transpose(2, 3).flatten(0, 2)[cut]
            for h2 in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                for r in range(off[g], off[g + 1], 4096):
                    end = min(r + 4096, off[g + 1])
                    score = q[r:end, h2] @ keys.T / math.sqrt(d)
                    if s["causal"]:
                        last = hi - off[g + 1] + torch.arange(r, end, device=q.device)
                        score[torch.arange(lo, hi, device=q.device) > last[:, None]] = -math.inf
                    out[r:end, h2] = torch.softmax(score, 1) @ values
    return out
