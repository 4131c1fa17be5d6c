"""Plain 64-bit forms of the paged cache's operators, for the tests: attention by
its definition, a cache that is a list of rows per sequence, and the page rules
(lowest free page first, entry by entry) written out one page at a time."""
from __future__ import annotations

import torch

DEV = "cuda"


def attend(q, k, v, positions, sink, recent, retrieval, scale):
    """q [m, G, D] at `positions` over rows k, v [n, D] of positions 0 .. n-1. Returns the output [m, G, D] and
    sum_j p_j |v_j|, the quantity that a rounding of the weights is relative to; both in 64 bits."""
    n = k.shape[0]
    q, k, v = q.double(), k.double(), v.double()
    j = torch.arange(n, device=q.device)
    i = torch.as_tensor(positions, device=q.device)[:, None]
    seen = j <= i
    if not retrieval:
        seen = seen & ((j < sink) | (i - j < recent))
    s = torch.einsum("mgd,nd->mgn", q, k) * scale
    s = s.masked_fill(~seen[:, None], -torch.inf)
    p = torch.softmax(s, -1)
    return torch.einsum("mgn,nd->mgd", p, v), torch.einsum("mgn,nd->mgd", p, v.abs())


def check_out(got, ref, weight, what="", half_p=2.0 ** -8):
    """|got - ref| is at most: the weights' rounding to bf16 (half a step, 2^-8; f16 2^-11) on sum p |v|, the
    output's rounding to bf16 (2^-8 of the value), and the 32-bit errors of scores, exponentials and sums. A score is a
    sum of 128 products of N(0,1) values times 0.09 or 0.13: its error is below 128 x 2^-24 x 20 = 1.6e-4, which
    counts once in the weight and once in their sum."""
    err = (got.double() - ref).abs()
    tol = (half_p + 4e-4) * weight + 2.0 ** -8 * ref.abs() + 1e-6
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol)[bad].nan_to_num(9e9).max()):.3g} x the bound"


def e4m3(x, scale):
    """bf16 rows as the values of their E4M3 codes under `scale` (the product with its 32-bit reciprocal, in 32 bits)."""
    inv = torch.tensor(1.0, dtype=torch.float32) / torch.tensor(scale, dtype=torch.float32)
    return (x.float() * inv.to(x.device)).clamp(-448, 448).to(torch.float8_e4m3fn)


class Model:
    """A paged cache as plain data: per sequence its page list and, per layer, its rows; the pool as reference counts."""

    def __init__(self, num_pages, page, max_pages, max_seqs):
        self.P, self.max_pages, self.num_pages = page, max_pages, num_pages
        self.ref = [0] * num_pages
        self.pages = {s: [] for s in range(max_seqs)}
        self.len = {s: 0 for s in range(max_seqs)}

    def free(self):
        return [i for i, r in enumerate(self.ref) if r == 0]

    def extend(self, seqs, n_tok):
        """True if it was done; else nothing changed."""
        import copy
        saved = copy.deepcopy((self.ref, self.pages, self.len))
        order = self.free()  # pages freed by this call are not taken by it
        take = iter(order)
        ok = len(set(seqs)) == len(seqs)
        try:
            for s, a in zip(seqs, n_tok):
                if a < 0:
                    ok = False
                    break
                if a == 0:
                    continue
                n = self.len[s]
                if n % self.P and self.ref[self.pages[s][-1]] > 1:
                    self.ref[self.pages[s][-1]] -= 1
                    self.pages[s][-1] = next(take)
                    self.ref[self.pages[s][-1]] = 1
                while len(self.pages[s]) * self.P < n + a:
                    self.pages[s].append(next(take))
                    self.ref[self.pages[s][-1]] = 1
                ok = ok and len(self.pages[s]) <= self.max_pages
                self.len[s] = n + a
        except StopIteration:
            ok = False
        if not ok:
            self.ref, self.pages, self.len = saved
        return ok

    def fork(self, src, dst):
        for s, d in zip(src, dst):
            self.pages[d] = list(self.pages[s])
            self.len[d] = self.len[s]
            for p in self.pages[d]:
                self.ref[p] += 1

    def copy(self, src, dst):
        take = iter(self.free())
        for s, d in zip(src, dst):
            self.pages[d] = [next(take) for _ in self.pages[s]]
            self.len[d] = self.len[s]
            for p in self.pages[d]:
                self.ref[p] = 1

    def release(self, seqs):
        for s in seqs:
            for p in self.pages[s]:
                self.ref[p] -= 1
            self.pages[s], self.len[s] = [], 0

    def compact(self):
        used = sum(r > 0 for r in self.ref)
        holes = [i for i in range(used) if self.ref[i] == 0]
        movers = [i for i in range(used, self.num_pages) if self.ref[i] > 0]
        to = dict(zip(movers, holes))
        for a, b in to.items():
            self.ref[b], self.ref[a] = self.ref[a], 0
        for s in self.pages:
            self.pages[s] = [to.get(p, p) for p in self.pages[s]]

    def check(self, cache):
        assert cache.page_ref.tolist() == self.ref
        lens, table = cache.seq_len.tolist(), cache.page_table.tolist()
        for s, pages in self.pages.items():
            assert lens[s] == self.len[s], f"length of {s}"
            assert table[s][:len(pages)] == pages, f"pages of {s}"


class Rows:
    """The rows every sequence should hold: rows[s] = (k, v) [layers, tokens, heads, D] bf16."""

    def __init__(self, cache):
        L = cache.layout
        self.c, self.L = cache, L
        empty = torch.zeros((L.num_layers, 0, L.num_kv_heads, L.head_dim), dtype=torch.bfloat16, device=cache.device)
        self.rows = {s: (empty, empty) for s in range(L.max_seqs)}
        m = cache.is_retrieval
        self.index, counts = [], [0, 0]
        for x in m:  # (is retrieval, index in its pool)
            self.index.append((x, counts[x]))
            counts[x] += 1

    def add(self, s, k, v):
        a, b = self.rows[s]
        self.rows[s] = (torch.cat([a, k], 1), torch.cat([b, v], 1))

    def stored(self, layer, head, x, which, scales):
        if self.L.kv_format and self.c.is_retrieval[layer * self.L.num_kv_heads + head]:
            sc = scales[which][head]
            return e4m3(x, sc).double() * sc
        return x.double()

    def check(self, model, scales=None):
        """The cache's pages and windows hold exactly these rows where a sequence has tokens."""
        L, c = self.L, self.c
        P, W = L.page_size, L.sink + L.recent
        for s, (k, v) in self.rows.items():
            n = model.len[s]
            assert k.shape[1] == n
            if n == 0:
                continue
            pages = torch.tensor(model.pages[s], device=c.device)
            pos = torch.arange(n, device=c.device)
            kept = (pos < L.sink) | (pos >= n - L.recent)
            slot = torch.where(pos < L.sink, pos, L.sink + (pos - L.sink) % L.recent)[kept]
            for which, (pool, win, x) in enumerate(((c.k_pages, c.k_window, k), (c.v_pages, c.v_window, v))):
                for i, (r, at) in enumerate(self.index):
                    layer, h = divmod(i, L.num_kv_heads)
                    want = x[layer, :, h]
                    if r:
                        raw = pool.view(torch.uint8) if L.kv_format else pool.view(torch.int16)
                        got = raw[pages, at].reshape(-1, L.head_dim)[:n]
                        exp = e4m3(want, scales[which][h]).view(torch.uint8) if L.kv_format else want.contiguous().view(torch.int16)
                    else:
                        got = win.view(torch.int16)[s, at][slot]
                        exp = want[kept].contiguous().view(torch.int16)
                    assert torch.equal(got, exp), f"rows of sequence {s}, layer {layer}, head {h}"

    def attention(self, layer, s, q, positions, scale, scales=None):
        """q [m, Hq, D] at `positions` of sequence s: (output, weight), [m, Hq, D]."""
        L = self.L
        g = L.num_q_heads // L.num_kv_heads
        k, v = self.rows[s]
        outs = []
        for h in range(L.num_kv_heads):
            r = self.c.is_retrieval[layer * L.num_kv_heads + h]
            outs.append(attend(q[:, h * g:h * g + g], self.stored(layer, h, k[layer, :, h], 0, scales),
                               self.stored(layer, h, v[layer, :, h], 1, scales), positions, L.sink, L.recent, r, scale))
        return torch.cat([o[0] for o in outs], 1), torch.cat([o[1] for o in outs], 1)


def ints(x, device=DEV):
    return torch.tensor(x, dtype=torch.int32, device=device)


def normal(*shape, seed=0, device=DEV):
    g = torch.Generator(device=device).manual_seed(seed)
    return torch.randn(shape, generator=g, device=device, dtype=torch.float32).to(torch.bfloat16)


def poison(cache):
    """Fills everything that no sequence owns yet with NaN: nothing of it may ever be seen."""
    for t in (cache.k_window, cache.v_window):
        t.fill_(float("nan"))
    for t in (cache.k_pages, cache.v_pages):
        if cache.layout.kv_format:
            t.view(torch.uint8).fill_(0x7F)
        else:
            t.fill_(float("nan"))
    cache.page_table.fill_(-7)
