"""What the paged mixed-head cache's operators are measured on: decode over pages, packed prompts, page upkeep.

Retrieval KV heads keep every token in pages of `page` rows that a page table lists per sequence (one table for all
layers), streaming KV heads a window of `sink` + `recent` rows per sequence (sink position p in row p, any other p in
row sink + (p - sink) mod recent). A query at position p sees {0 .. p} or {j <= p : j < sink or p - j < recent}.

  decode   one layer's step for a batch of sequences: the new token's rows go into the cache, then attention over it
  prefill  one layer's whole prompts, packed one behind the other: causal attention, and their rows into the cache
  fork     sequences forked into beams (pages shared), one token more each (the shared last page copied), beams freed
           before the next pass
  compact  sequences copied, the originals freed, the pages that are left moved to the lowest numbers
"""
import math
import random

import torch

own = False

DEV = "cuda"
SINK, RECENT = 64, 256  # the window of the repository's benchmark layers


def _decode(name, batch, lo, hi, q_heads, kv_heads, retrieval, dim=128, sink=SINK, recent=RECENT, page=64, e4m3=False, ragged=0):
    c = dict(op="decode", batch=batch, lo=lo, hi=hi, q_heads=q_heads, kv_heads=kv_heads, retrieval=retrieval, dim=dim, sink=sink,
             recent=recent, page=page, e4m3=e4m3, ragged=ragged)
    return dict(c, name=name) if name else c


def _prefill(name, batch, lo, hi, q_heads, kv_heads, retrieval, dim=128, sink=SINK, recent=RECENT, page=64, ragged=0):
    c = dict(op="prefill", batch=batch, lo=lo, hi=hi, q_heads=q_heads, kv_heads=kv_heads, retrieval=retrieval, dim=dim, sink=sink,
             recent=recent, page=page, e4m3=False, ragged=ragged)
    return dict(c, name=name) if name else c


def _pages(name, op, batch, beams, lo, hi, layers, kv_heads, retrieval, dim=128, sink=SINK, recent=RECENT, page=64, e4m3=False, ragged=0):
    c = dict(op=op, batch=batch, beams=beams, lo=lo, hi=hi, layers=layers, kv_heads=kv_heads, retrieval=retrieval, dim=dim, sink=sink,
             recent=recent, page=page, e4m3=e4m3, ragged=ragged)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user of the repository's smallest layer, some 500 tokens in: latency alone
        _decode("decode 1 x 529 mha d64", 1, 529, 529, 4, 4, 2, dim=64, sink=4, recent=64, page=16),
        # the headline layer's decode step behind its 32K prompt, one sequence
        _decode("decode 1 x 32769 mha", 1, 32769, 32769, 32, 32, 8),
        # the grouped-heads layer at 128K, four sequences: the cache's bytes alone
        _decode("decode 4 x 131072 gqa", 4, 131072, 131072, 32, 8, 4),
        # a server's batch in flight: lengths from one token to thousands, quantized pages
        _decode("decode 48 ragged gqa e4m3", 48, 1, 9000, 32, 8, 4, page=32, e4m3=True, ragged=1),
        # many short conversations, wide groups, small pages
        _decode("decode 200 ragged g8", 200, 1, 1500, 32, 4, 2, page=16, ragged=2),
        # one short prompt of the smallest layer
        _prefill("prefill 1 x 37 mha d64", 1, 37, 37, 4, 4, 2, dim=64, sink=4, recent=64, page=16),
        # a server's prompts of one step, packed
        _prefill("prefill 12 ragged gqa", 12, 40, 2500, 32, 8, 4, ragged=3),
        # many short prompts
        _prefill("prefill 160 short g2 d64", 160, 1, 150, 16, 8, 4, dim=64, page=32, ragged=4),
        # the headline layer's whole 32K prompt
        _prefill("prefill 1 x 32768 mha", 1, 32768, 32768, 32, 32, 8),
        # one sequence into four beams, one small layer: latency alone
        _pages("fork 1 into 4 d64", "fork", 1, 4, 300, 300, 1, 4, 2, dim=64, sink=4, recent=64, page=16),
        # sixteen sequences into four beams each in the 32-layer grouped-heads stack
        _pages("fork 16 into 64 stack", "fork", 16, 4, 100, 4000, 32, 8, 4, ragged=5),
        # a scattered pool of the same stack put in order
        _pages("compact 12 ragged stack", "compact", 12, 1, 200, 4500, 32, 8, 4, ragged=6),
    ]


def _size(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "fork", "compact"])
    dim, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    sink, recent = rng.choice([0, 4, rng.randint(1, 100), SINK]), rng.choice([64, rng.randint(2, 700), RECENT])
    kv = rng.choice([1, 2, 4, 8])
    retrieval = rng.randint(0, kv)
    seed = rng.randrange(1 << 20)
    if op == "decode":
        group = rng.choice([1, 2, 4, 8])
        batch = _size(rng, 1, 200)
        hi = _size(rng, 2, min(131072, 400000 // (batch * max(1, retrieval) // 2 + 1)))
        return _decode(None, batch, rng.choice([1, max(1, hi // 2), hi]), hi, kv * group, kv, retrieval, dim, sink, recent, page, rng.random() < 0.4, seed)
    if op == "prefill":
        group = rng.choice([1, 2, 4])
        batch = _size(rng, 1, 160)
        hi = _size(rng, 1, max(2, 10000 // batch))
        return _prefill(None, batch, rng.choice([1, hi]), hi, kv * group, kv, retrieval, dim, sink, recent, page, seed)
    layers = _size(rng, 1, 16)
    batch = _size(rng, 1, 24)
    hi = _size(rng, 2, 4000)
    lo = rng.choice([1, max(1, hi // 2)])
    return _pages(None, op, batch, rng.randint(1, 4) if op == "fork" else 1, lo, hi, layers, kv, retrieval, dim, sink, recent, page, rng.random() < 0.3, seed)


# ---------------------------------------------------------------------------- shapes


def _lens(c):
    r = random.Random(c["ragged"])
    return [c["hi"] if c["lo"] == c["hi"] else _size(r, c["lo"], c["hi"]) for _ in range(c["batch"])]


def _cdiv(a, b):
    return -(-a // b)


def _elem(c):
    return 1 if c["e4m3"] else 2


def _row_counts(c, lens):
    return sum(lens), sum(min(n, c["sink"] + c["recent"]) for n in lens)


def _pairs(c, n):
    """Query and key pairs of a causal prompt of n tokens: of a retrieval head, and of a streaming one."""
    s, r = c["sink"], c["recent"]
    full = n * (n + 1) // 2
    w = s + r
    return full, full if n <= w else w * (w + 1) // 2 + (n - w) * w


def work(c):
    lens = _lens(c)
    dim, kv, retr = c["dim"], c["kv_heads"], c["retrieval"]
    strm = kv - retr
    if c["op"] == "decode":
        all_rows, win_rows = _row_counts(c, lens)
        rows = c["batch"] * (2 * c["q_heads"] + 2 * kv) * dim * 2  # q, out, the new rows
        cache = 2 * dim * (all_rows * retr * _elem(c) + win_rows * strm * 2)
        return {"bytes": rows + cache, "flops": 4 * dim * (c["q_heads"] // kv) * (all_rows * retr + win_rows * strm)}
    if c["op"] == "prefill":
        pairs = [_pairs(c, n) for n in lens]
        total, win_rows = _row_counts(c, lens)
        rows = total * (2 * c["q_heads"] + 2 * kv) * dim * 2
        cache = 2 * dim * 2 * (total * retr + win_rows * strm)
        g = c["q_heads"] // kv
        return {"bytes": rows + cache, "flops": 4 * dim * g * (retr * sum(p[0] for p in pairs) + strm * sum(p[1] for p in pairs))}
    page_bytes = 2 * c["layers"] * retr * c["page"] * dim * _elem(c)
    win_bytes = 2 * c["layers"] * strm * (c["sink"] + c["recent"]) * dim * 2
    pages = [_cdiv(n, c["page"]) for n in lens]
    if c["op"] == "fork":  # a shared last page that is not full is copied for each beam; the windows always are
        copies = sum(c["beams"] for n in lens if n % c["page"])
        words = 4 * c["beams"] * sum(pages)
        return {"bytes": 2 * copies * page_bytes + 2 * c["beams"] * c["batch"] * win_bytes + 2 * words, "flops": 0}
    return {"bytes": 4 * sum(pages) * page_bytes + 4 * c["batch"] * win_bytes + 16 * sum(pages), "flops": 0}


# ---------------------------------------------------------------------------- inputs


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 7919 + 11)
    dim, kv, retr, page, batch = c["dim"], c["kv_heads"], c["retrieval"], c["page"], c["batch"]
    layers = c.get("layers", 1)
    lens = _lens(c)
    pages = [_cdiv(n, page) for n in lens]
    beams = c.get("beams", 1)
    if c["op"] in ("decode", "prefill"):
        max_seqs, max_pages, num_pages = batch + 3, max(pages) + 2, sum(pages) + 5
    else:
        max_seqs, max_pages = batch * (1 + beams), max(pages) + 1
        num_pages = 2 * sum(pages) + 3 if c["op"] == "compact" else sum(pages) + 2 * batch * beams + 3
    # which KV heads are retrieval heads: drawn from the seed, as many in every layer
    heads = [sorted(torch.randperm(kv, generator=torch.Generator().manual_seed(seed + l)).tolist()[:retr]) for l in range(layers)]
    mask = [1 if h in heads[l] else 0 for l in range(layers) for h in range(kv)]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)

    def pool():
        x = normal(num_pages, layers * retr, page, dim)
        return x.to(torch.float8_e4m3fn) if c["e4m3"] else x

    # sequences in places of their own, their pages scattered over the pool; no page or table entry else means anything
    at = torch.randperm(max_seqs, generator=g, device=DEV)[:batch].to(torch.int32)
    order = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(max_seqs, max_pages, dtype=torch.int32, device=DEV)
    count = torch.tensor(pages, device=DEV)
    live = torch.arange(max_pages, device=DEV)[None] < count[:, None]
    mine = torch.zeros(batch, max_pages, dtype=torch.int32, device=DEV)
    mine[live] = order[: sum(pages)]
    table[at.long()] = mine
    seq_len = torch.zeros(max_seqs, dtype=torch.int32, device=DEV)
    seq_len[at.long()] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ref = torch.zeros(num_pages, dtype=torch.int32, device=DEV)
    ref[order[: sum(pages)].long()] = 1
    t = dict(k_pages=pool(), v_pages=pool(), k_window=normal(max_seqs, layers * (kv - retr), c["sink"] + c["recent"], dim),
             v_window=normal(max_seqs, layers * (kv - retr), c["sink"] + c["recent"], dim), page_table=table, seq_len=seq_len, page_ref=ref)
    q_heads = c.get("q_heads", kv)
    st = dict(case=c, t=t, seqs=at, retr=torch.tensor(heads[0], dtype=torch.long, device=DEV),
              strm=torch.tensor([h for h in range(kv) if h not in heads[0]], dtype=torch.long, device=DEV))
    if c["op"] == "decode":
        st.update(q=normal(batch, q_heads, dim), k=normal(batch, kv, dim), v=normal(batch, kv, dim), out=torch.zeros(batch, q_heads, dim, dtype=torch.bfloat16, device=DEV),
                  scales=[[0.25 + 0.5 * ((h * 5 + j) % 4) for h in range(kv)] for j in (0, 1)])
        st["scale_k"], st["scale_v"] = (torch.tensor(x, dtype=torch.float32, device=DEV) for x in st["scales"])
    elif c["op"] == "prefill":
        total = sum(lens) + 3  # rows behind the last prompt stay as they are
        st.update(q=normal(total, q_heads, dim), k=normal(total, kv, dim), v=normal(total, kv, dim), out=torch.zeros(total, q_heads, dim, dtype=torch.bfloat16, device=DEV),
                  row_start=torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32))
    else:
        free = torch.ones(max_seqs, dtype=torch.bool, device=DEV)
        free[at.long()] = False
        st.update(dst=free.nonzero()[:, 0].to(torch.int32)[: batch * beams], src=at.repeat_interleave(beams))
    if own:
        import mixed_head_kv_b200 as duo

        st["cache"] = duo.PagedCache(layers, max_seqs, q_heads, kv, dim, c["sink"], c["recent"], page, num_pages, max_pages, mask,
                                     kv_format=duo.DUO_KV_E4M3 if c["e4m3"] else duo.DUO_KV_BF16, tensors=t)
        if c["op"] == "decode" and c["e4m3"]:
            st["cache"].set_kv_scales(0, *st["scales"])
    return st


# ---------------------------------------------------------------------------- the plain forms


def _bits(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _codes(x, scale):
    """bf16 rows [..., heads, dim] as E4M3 codes under a scale per head."""
    y = x.float() * (1.0 / scale)[:, None]
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _store_rows(st, seq, pos, seq_end, k, v):
    """Rows k, v [n, kv, dim] of position pos[n] of sequences seq[n], which then hold seq_end[n] tokens, into pages and windows."""
    c, t = st["case"], st["t"]
    page, sink, recent = c["page"], c["sink"], c["recent"]
    number = t["page_table"][seq, pos // page].long()
    for x, rows, scale in ((t["k_pages"], k, st.get("scale_k")), (t["v_pages"], v, st.get("scale_v"))):
        r = rows[:, st["retr"]]
        r = _codes(r, scale[st["retr"]]) if c["e4m3"] else r
        _bits(x)[number, :, pos % page] = _bits(r)
    kept = (pos < sink) | (pos >= seq_end - recent)
    slot = torch.where(pos < sink, pos, sink + (pos - sink) % recent)[kept]
    for x, rows in ((t["k_window"], k), (t["v_window"], v)):
        x[seq[kept], :, slot] = rows[kept][:, st["strm"]]


def _attend(q, k, v, seen, scale):
    """q [..., g, d], k and v [..., n, d], seen [..., 1 or g, n] in 32 bits."""
    s = (q @ k.transpose(-1, -2)) * scale
    s = s.masked_fill(~seen, -torch.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return (p @ v) / p.sum(-1, keepdim=True)


def _run_decode(st):
    c, t = st["case"], st["t"]
    b, kv, dim, page = c["batch"], c["kv_heads"], c["dim"], c["page"]
    g = c["q_heads"] // kv
    seq = st["seqs"].long()
    n = t["seq_len"][seq].long()
    _store_rows(st, seq, n - 1, n, st["k"], st["v"])
    q = st["q"].view(b, kv, g, dim).float()
    out = st["out"].view(b, kv, g, dim)
    scale = 1.0 / math.sqrt(dim)
    j = torch.arange(max(_lens(c)), device=DEV)
    rows = t["page_table"][seq[:, None], j // page].long()
    seen = j[None] < n[:, None]
    rows = torch.where(seen, rows, 0)
    pick = lambda x: x[rows, :, j % page].permute(0, 2, 1, 3)  # noqa: E731
    k, v = (pick(_bits(t[x])) for x in ("k_pages", "v_pages"))
    if c["e4m3"]:
        k, v = (x.contiguous().view(torch.float8_e4m3fn).float() * s[st["retr"]][:, None, None] for x, s in ((k, st["scale_k"]), (v, st["scale_v"])))
    out[:, st["retr"]] = _attend(q[:, st["retr"]], k.float(), v.float(), seen[:, None, None], scale).to(out.dtype)
    w = torch.arange(c["sink"] + c["recent"], device=DEV)
    out[:, st["strm"]] = _attend(q[:, st["strm"]], t["k_window"][seq].float(), t["v_window"][seq].float(), (w[None] < n[:, None])[:, None, None], scale).to(out.dtype)
    return _cache_outputs(st)


def _cache_outputs(st):
    return dict({x: st["t"][x] for x in ("k_pages", "v_pages", "k_window", "v_window")}, out=st["out"])


def _run_prefill(st):
    c = st["case"]
    kv, dim, h = c["kv_heads"], c["dim"], c["q_heads"]
    g = h // kv
    start = st["row_start"].long()
    total = int(sum(_lens(c)))
    row = torch.arange(total, device=DEV)
    i = torch.searchsorted(start, row, right=True) - 1
    pos = row - start[i]
    n = start[i + 1] - start[i]
    k, v = (st[x][:total].permute(1, 0, 2).float().repeat_interleave(g, 0) for x in ("k", "v"))
    retr = torch.zeros(kv, dtype=torch.bool, device=DEV)
    retr[st["retr"]] = True
    retr = retr.repeat_interleave(g)[:, None, None]
    near = 2048  # rows of queries at a time: the scores of all of them would not fit
    for a in range(0, total, near):
        z = min(total, a + near)
        first = int(start[i[a]])  # no query of these rows sees a key of an earlier prompt
        back = pos[a:z, None] - pos[None, first:z]
        causal = (i[a:z, None] == i[None, first:z]) & (back >= 0)
        seen = causal[None] & (retr | (pos[None, first:z] < c["sink"])[None] | (back < c["recent"])[None])
        o = _attend(st["q"][a:z].permute(1, 0, 2).float(), k[:, first:z], v[:, first:z], seen, 1.0 / math.sqrt(dim))
        st["out"][a:z] = o.permute(1, 0, 2).to(st["out"].dtype)
    _store_rows(st, st["seqs"].long()[i], pos, n, st["k"][:total], st["v"][:total])
    return _cache_outputs(st)


def _free_pages(t):
    return (t["page_ref"] == 0).nonzero()[:, 0]


def _live(t, seq, page):
    count = (t["seq_len"][seq] + page - 1) // page
    return torch.arange(t["page_table"].shape[1], device=DEV)[None] < count[:, None]


def _release(st, seq):
    t, page = st["t"], st["case"]["page"]
    held = t["page_table"][seq][_live(t, seq, page)].long()
    t["page_ref"].scatter_add_(0, held, torch.full_like(held, -1, dtype=torch.int32))
    t["seq_len"][seq] = 0


def _share(st, src, dst):
    t, page = st["t"], st["case"]["page"]
    live = _live(t, src, page)
    held = t["page_table"][src]
    t["page_table"][dst] = torch.where(live, held, t["page_table"][dst])
    held = held[live].long()
    t["page_ref"].scatter_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    t["seq_len"][dst] = t["seq_len"][src]
    _copy_windows(t, src, dst)


def _copy_windows(t, src, dst):
    for x in ("k_window", "v_window"):
        t[x][dst] = t[x][src]


def _copy_pages(t, src, dst):
    for x in ("k_pages", "v_pages"):
        _bits(t[x])[dst] = _bits(t[x])[src]


def _extend_one(st, seq):
    """One token more for each sequence: a new page where the last is full, a copy of it where it is shared by others too."""
    t, page = st["t"], st["case"]["page"]
    n = t["seq_len"][seq].long()
    last = (n + page - 1) // page - 1
    tail = t["page_table"][seq, last.clamp(min=0)].long()
    partial = n % page != 0
    same = (tail[:, None] == tail[None]) & partial[:, None] & partial[None]
    before = torch.tril(same, -1).sum(1)  # sequences named earlier that leave the page
    cow = partial & (t["page_ref"][tail] - before > 1)
    take = cow | ~partial
    at = take.long().cumsum(0) - 1
    new = _free_pages(t)[at.clamp(min=0)]
    _copy_pages(t, tail[cow], new[cow])
    t["page_ref"].scatter_add_(0, tail[cow], torch.full_like(tail[cow], -1, dtype=torch.int32))
    t["page_ref"][new[take]] = 1
    t["page_table"][seq[take], (n // page)[take]] = new[take].to(torch.int32)
    t["seq_len"][seq] = (n + 1).to(torch.int32)


def _duplicate(st, src, dst):
    """dst with pages of its own: the lowest free ones, in order."""
    t, page = st["t"], st["case"]["page"]
    live = _live(t, src, page)
    old = t["page_table"][src][live].long()
    new = _free_pages(t)[: old.numel()]
    mine = t["page_table"][dst]
    mine[live] = new.to(torch.int32)
    t["page_table"][dst] = mine
    t["page_ref"][new] = 1
    t["seq_len"][dst] = t["seq_len"][src]
    _copy_pages(t, old, new)
    _copy_windows(t, src, dst)


def _compact(st):
    t, page = st["t"], st["case"]["page"]
    used = t["page_ref"] > 0
    n = used.sum()
    number = torch.arange(used.numel(), device=DEV)
    to, src = (number[~used & (number < n)], number[used & (number >= n)])
    _copy_pages(t, src, to)
    t["page_ref"][to] = t["page_ref"][src]
    t["page_ref"][src] = 0
    new = number.clone()
    new[src] = to
    every = torch.arange(t["seq_len"].numel(), device=DEV)
    t["page_table"].copy_(torch.where(_live(t, every, page), new[t["page_table"].long()].to(torch.int32), t["page_table"]))


def _run_fork(st):
    src, dst = st["src"].long(), st["dst"].long()
    _release(st, dst)
    _share(st, src, dst)
    _extend_one(st, dst)
    return st["t"]


def _run_compact(st):
    a, b = st["src"].long(), st["dst"].long()
    _duplicate(st, a, b)
    _release(st, a)
    _compact(st)
    _share(st, b, a)
    _release(st, b)
    return st["t"]


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"decode": _run_decode, "prefill": _run_prefill, "fork": _run_fork, "compact": _run_compact}[op](st)
    cache = st["cache"]
    if op == "decode":
        cache.decode(0, st["seqs"], st["q"], st["k"], st["v"], st["out"])
        return _cache_outputs(st)
    if op == "prefill":
        cache.prefill(0, st["row_start"], st["q"], st["k"], st["v"], st["out"])
        cache.append(0, st["seqs"], st["row_start"], st["k"], st["v"])
        return _cache_outputs(st)
    if op == "fork":
        cache.release(st["dst"])
        cache.fork(st["src"], st["dst"])
        cache.extend(st["dst"])
        return st["t"]
    cache.copy(st["src"], st["dst"])
    cache.release(st["src"])
    cache.compact()
    cache.fork(st["dst"], st["src"])
    cache.release(st["dst"])
    return st["t"]


# ---------------------------------------------------------------------------- the definition in 64 bits


def exact(c, seed):
    """The attention outputs by their definition, sequence by sequence and head by head; the cache's rows are copies, which have no other value."""
    if c["op"] in ("fork", "compact"):
        return None
    st = prepare(c, seed)
    t = st["t"]
    lens, dim, kv, page = _lens(c), c["dim"], c["kv_heads"], c["page"]
    g = c["q_heads"] // kv
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    retr = st["retr"].tolist()
    first = 0
    for i, n in enumerate(lens):
        s = int(st["seqs"][i])
        numbers = t["page_table"][s, : _cdiv(n, page)].long()
        at = torch.arange(n, device=DEV)
        for h in range(kv):
            if c["op"] == "prefill":
                rows = slice(first, first + n)
                q, k, v = (x.double() for x in (st["q"][rows, h * g : h * g + g], st["k"][rows, h], st["v"][rows, h]))
                seen = at[:, None] >= at
                if h not in retr:
                    seen &= (at < c["sink"]) | (at[:, None] - at < c["recent"])
                for e in range(g):
                    w = torch.softmax((q[:, e] @ k.T / dim**0.5).masked_fill_(~seen, -torch.inf), -1)
                    out[rows, h * g + e] = w @ v
                continue
            new_k, new_v = st["k"][i, h].double(), st["v"][i, h].double()
            if h in retr:
                r = retr.index(h)
                k, v = (t[x][numbers, r].double().reshape(-1, dim)[:n].clone() if not c["e4m3"] else t[x].view(torch.uint8)[numbers, r].view(torch.float8_e4m3fn).double().reshape(-1, dim)[:n].clone() for x in ("k_pages", "v_pages"))
                if c["e4m3"]:
                    sk, sv = st["scale_k"][h].double(), st["scale_v"][h].double()
                    # the code is the rounding of the product with the scale's reciprocal, both in 32 bits: that is the format's definition
                    k[n - 1], v[n - 1] = ((x.float() * (1 / y.float())).clamp(-448, 448).to(torch.float8_e4m3fn).double() for x, y in ((new_k, sk), (new_v, sv)))
                    k, v = k * sk, v * sv
                else:
                    k[n - 1], v[n - 1] = new_k, new_v
            else:
                r = [x for x in range(kv) if x not in retr].index(h)
                held = [p for p in range(n - 1) if p < c["sink"] or n - 1 - p < c["recent"]]
                slots = [p if p < c["sink"] else c["sink"] + (p - c["sink"]) % c["recent"] for p in held]
                k, v = (torch.cat([t[x][s, r][slots].double(), y[None]]) for x, y in (("k_window", new_k), ("v_window", new_v)))
            w = torch.softmax(st["q"][i, h * g : h * g + g].double() @ k.T / dim**0.5, -1)
            out[i, h * g : h * g + g] = w @ v
        first += n
    return dict(out=out, k_pages=None, v_pages=None, k_window=None, v_window=None)
