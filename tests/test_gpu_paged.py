"""The paged mixed-head cache on the GPU, against plain 64-bit forms (paged_harness.py): decode over pages, packed
prompts, append, page upkeep, a run of them together, captured steps."""
import math
import random

import pytest
import torch

from paged_harness import Model, Rows, check_out, ints, normal, poison

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def duo():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    import mixed_head_kv_b200
    return mixed_head_kv_b200


def make(duo, Hkv=2, G=2, D=64, S=4, R=16, P=16, num_pages=64, max_pages=32, max_seqs=8, mask=None, layers=1, fp8=False):
    mask = mask if mask is not None else [(i + 1) % 2 for i in range(Hkv)] * layers
    c = duo.PagedCache(layers, max_seqs, Hkv * G, Hkv, D, S, R, P, num_pages, max_pages, mask,
                       kv_format=duo.DUO_KV_E4M3 if fp8 else duo.DUO_KV_BF16)
    poison(c)
    return c


def scales_for(c):
    H = c.layout.num_kv_heads
    return [[0.5 + 0.375 * h for h in range(H)], [0.25 + 0.5 * h for h in range(H)]]


def fill(c, model, rows, lens, seed):
    """Prompts of lens[s] tokens for sequences s = 0 .. by extend + append, all layers."""
    L = c.layout
    seqs = list(range(len(lens)))
    assert model.extend(seqs, lens)
    c.extend(ints(seqs), ints(lens))
    start = [0]
    for n in lens:
        start.append(start[-1] + n)
    for layer in range(L.num_layers):
        k, v = (normal(start[-1], L.num_kv_heads, L.head_dim, seed=seed * 100 + layer * 2 + i) for i in (0, 1))
        c.append(layer, ints(seqs), ints(start), k, v)
        for s in seqs:
            if layer == 0:
                rows.rows[s] = (torch.empty((0, lens[s], L.num_kv_heads, L.head_dim), dtype=torch.bfloat16, device="cuda"),) * 2
            part = slice(start[s], start[s + 1])
            rows.rows[s] = tuple(torch.cat([a, x[None, part]]) for a, x in zip(rows.rows[s], (k, v)))


def step(c, model, rows, seqs, seed, scales=None, half_p=2.0 ** -8, extend=True):
    """One token more for `seqs`, every layer decoded and checked."""
    L = c.layout
    n = len(seqs)
    if extend:
        assert model.extend(seqs, [1] * n)
        c.extend(ints(seqs))
    new = [tuple(normal(n, L.num_kv_heads, L.head_dim, seed=seed * 1000 + 10 * l + i) for i in (1, 2)) for l in range(L.num_layers)]
    for i, s in enumerate(seqs):
        rows.add(s, *(torch.stack([new[l][x][i] for l in range(L.num_layers)])[:, None] for x in (0, 1)))
    for l in range(L.num_layers):
        q = normal(n, L.num_q_heads, L.head_dim, seed=seed * 1000 + 10 * l)
        out = torch.full_like(q, float("nan"))
        c.decode(l, ints(seqs), q, *new[l], out)
        for i, s in enumerate(seqs):
            ref, w = rows.attention(l, s, q[i:i + 1], [model.len[s] - 1], 1 / math.sqrt(L.head_dim), scales)
            check_out(out[i:i + 1], ref, w, f"layer {l} sequence {s} of {model.len[s]}", half_p)


# ------------------------------------------------------------------------------ append


@pytest.mark.parametrize("D,P,fp8", [(64, 16, False), (128, 64, False), (128, 32, True), (64, 128, True)])
def test_append_fills_pages_and_windows(duo, D, P, fp8):
    c = make(duo, Hkv=3, G=1, D=D, P=P, S=4, R=16, num_pages=80, max_pages=40, layers=2, mask=[1, 0, 1, 0, 0, 1], fp8=fp8)
    sc = scales_for(c) if fp8 else None
    if fp8:
        for l in range(2):
            c.set_kv_scales(l, *sc)
    model, rows = Model(80, P, 40, 8), Rows(c)
    fill(c, model, rows, [1, 0, P, P + 1, 3 * P - 1, 19, 20], seed=1)
    model.check(c)
    rows.check(model, sc)
    assert c.error_flags() == 0


def test_append_in_pieces_strided_and_padded(duo):
    """The second half of a prompt, out of a fused projection's rows, with padding entries between."""
    c = make(duo, Hkv=2, G=1, D=64, P=16, S=2, R=5, mask=[1, 0])
    model, rows = Model(64, 16, 32, 8), Rows(c)
    for piece, lens in enumerate([(7, 30), (12, 1), (0, 5), (1, 40)]):
        assert model.extend([3, 5], lens)
        c.extend(ints([3, -1, 5, 8]), ints([lens[0], 9, lens[1], 9]))
        n = sum(lens)
        qkv = normal(n + 6, 6, 64, seed=piece)  # q, k, v of two heads each; rows 0 .. 3 and the last two belong to nobody
        qkv[:4] = float("nan")
        qkv[-2:] = float("nan")
        k, v = qkv[:, 2:4], qkv[:, 4:6]
        a, b = 4, 4 + lens[0]
        c.append(0, ints([3, -1, 5, 8]), ints([a, b, b, b + lens[1], b + lens[1]]), k, v)
        rows.add(3, k[None, a:b], v[None, a:b])
        rows.add(5, k[None, b:b + lens[1]], v[None, b:b + lens[1]])
    model.check(c)
    rows.check(model)
    assert c.error_flags() == 0


# ------------------------------------------------------------------------------ decode


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_groups(duo, G, D):
    c = make(duo, Hkv=2, G=G, D=D, P=32, S=4, R=60, num_pages=64, max_pages=40)
    model, rows = Model(64, 32, 40, 8), Rows(c)
    fill(c, model, rows, [1, 63, 64, 130, 700], seed=G)
    for t in range(3):
        step(c, model, rows, [4, 0, 2, 1, 3], seed=G * 10 + t)
    model.check(c)
    rows.check(model)
    assert c.error_flags() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_decode_page_sizes_and_edges(duo, P, D, fp8):
    """Lengths around page, tile and window edges, the first token of a sequence among them; pages scattered."""
    c = make(duo, Hkv=2, G=4, D=D, P=P, S=3, R=50, num_pages=300, max_pages=140, max_seqs=20, layers=2, mask=[1, 0, 0, 1], fp8=fp8)
    sc = scales_for(c) if fp8 else None
    if fp8:
        for l in range(2):
            c.set_kv_scales(l, *sc)
    model, rows = Model(300, P, 140, 20), Rows(c)
    lens = [0, 1, 14, 15, 16, 31, 49, 52, 53, 63, 64, 126, 127, 128, 191, 192, 255, 256, 500]
    order = list(range(len(lens)))
    random.Random(P).shuffle(order)
    for s in order:  # one by one, so that numbers interleave
        assert model.extend([s], [lens[s] // 2])
        c.extend(ints([s]), ints([lens[s] // 2]))
    rest = [lens[s] - lens[s] // 2 for s in order]
    assert model.extend(order, rest)
    c.extend(ints(order), ints(rest))
    for s in order:
        kv = [normal(2, lens[s], 2, D, seed=s * 2 + i) for i in (0, 1)]
        for l in range(2):
            c.append(l, ints([s]), ints([0, lens[s]]), kv[0][l], kv[1][l])
        rows.rows[s] = tuple(kv)
    for t in range(2):
        step(c, model, rows, order, seed=t + 5, scales=sc, half_p=2.0 ** -8)
    model.check(c)
    rows.check(model, sc)
    assert c.error_flags() == 0


@pytest.mark.parametrize("mask", [[1, 1], [0, 0]])
@pytest.mark.parametrize("S,R", [(0, 1), (0, 70), (100, 1), (64, 256)])
def test_decode_windows_and_uniform_heads(duo, mask, S, R):
    c = make(duo, Hkv=2, G=2, D=128, P=16, S=S, R=R, num_pages=120, max_pages=40, mask=mask)
    model, rows = Model(120, 16, 40, 8), Rows(c)
    fill(c, model, rows, [0, 1, 63, 99, 100, 101, 319, 330], seed=S + R)
    for t in range(2):
        step(c, model, rows, list(range(8)), seed=t)
    rows.check(model)
    assert c.error_flags() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_long_sequences_are_split_and_joined(duo, fp8):
    """One long sequence over all CTAs, one beside short ones, sink-like keys; the same call twice gives the same bits."""
    c = make(duo, Hkv=1, G=8, D=128, P=64, S=4, R=60, num_pages=700, max_pages=500, mask=[1], fp8=fp8)
    sc = [[0.5], [0.25]]
    if fp8:
        c.set_kv_scales(0, *sc)
    model, rows = Model(700, 64, 500, 8), Rows(c)
    lens = [20000, 17, 0, 3333]
    assert model.extend([0, 1, 2, 3], lens)
    c.extend(ints([0, 1, 2, 3]), ints(lens))
    for s, n in enumerate(lens):
        k, v = normal(n, 1, 128, seed=s), normal(n, 1, 128, seed=s + 50)
        k[:2] *= 8
        c.append(0, ints([s]), ints([0, n]), k, v)
        rows.rows[s] = (k[None], v[None])
    step(c, model, rows, [0], seed=1, scales=sc)
    step(c, model, rows, [1, 3, 0, 2], seed=2, scales=sc)
    q, k, v = (normal(4, h, 128, seed=9 + h) for h in (8, 1, 1))
    outs = []
    for _ in range(3):
        out = torch.empty_like(q)
        c.decode(0, ints([3, 1, 0, 2]), q, k, v, out)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert c.error_flags() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,G,Hkv", [(512, 1, 8), (300, 8, 2), (33, 4, 16)])
def test_decode_many_entries(duo, n, G, Hkv, fp8):
    """Every CTA works through several pairs: the largest batch, short and empty sequences among them."""
    c = make(duo, Hkv=Hkv, G=G, D=64, P=16, S=4, R=60, num_pages=n * 12, max_pages=40, max_seqs=n + 5, fp8=fp8)
    sc = scales_for(c) if fp8 else None
    if fp8:
        c.set_kv_scales(0, *sc)
    rng = random.Random(n)
    model, rows = Model(n * 12, 16, 40, n + 5), Rows(c)
    fill(c, model, rows, [rng.choice([0, 1, 15, 16, 40, 64, 130, 300]) for _ in range(n)], seed=2)
    order = list(range(n))
    rng.shuffle(order)
    assert model.extend(order, [1] * n)
    c.extend(ints(order))
    q, k, v = (normal(n, h, 64, seed=h) for h in (Hkv * G, Hkv, Hkv))
    out = torch.full_like(q, float("nan"))
    t0 = torch.cuda.Event(enable_timing=True)
    t1 = torch.cuda.Event(enable_timing=True)
    c.decode(0, ints(order), q, k, v, out)
    t0.record()
    c.decode(0, ints(order), q, k, v, out)
    t1.record()
    for i, s in enumerate(order):
        rows.add(s, k[None, i:i + 1], v[None, i:i + 1])
        if i % 7 == 0:
            ref, w = rows.attention(0, s, q[i:i + 1], [model.len[s] - 1], 1 / 8, sc)
            check_out(out[i:i + 1], ref, w, f"entry {i}")
    assert torch.isfinite(out).all() and c.error_flags() == 0
    assert t0.elapsed_time(t1) < 200  # no bounded wait (1 s) ran out


def test_decode_offsets_past_32_bits(duo):
    """A pool of more than 2^32 bytes in one tensor: the last pages are read and written where they are."""
    num_pages = 20000
    c = make(duo, Hkv=16, G=1, D=128, P=64, S=4, R=12, num_pages=num_pages, max_pages=16, mask=[1] * 16)
    assert c.k_pages.numel() * 2 > 2 ** 32
    c.page_ref[:num_pages - 12] = 1  # somebody else's
    model, rows = Model(num_pages, 64, 16, 8), Rows(c)
    model.ref[:num_pages - 12] = [1] * (num_pages - 12)
    fill(c, model, rows, [300, 200], seed=3)
    step(c, model, rows, [1, 0], seed=4)
    rows.check(model)
    assert model.pages[0][0] == num_pages - 12 and c.error_flags() == 0


def test_decode_padding_empty_strided(duo):
    """Padding entries' rows stay as they are, an empty sequence's row is zero, rows come out of wider tensors."""
    c = make(duo, Hkv=2, G=2, D=64)
    model, rows = Model(64, 16, 32, 8), Rows(c)
    fill(c, model, rows, [40, 33], seed=1)
    assert model.extend([0, 1], [1, 1])
    c.extend(ints([0, 1]))
    seqs = ints([8, 1, -1, 0, 5, 1 << 30])
    qkv = normal(6, 12, 64, seed=2)  # 4 q heads, 2 k, 2 v, 4 spare
    qkv[0] = qkv[2] = qkv[4] = qkv[5] = float("nan")
    wide = torch.full((6, 6, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    q, k, v, out = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:8], wide[:, 1:5]
    c.decode(0, seqs, q, k, v, out)
    for i, s in ((1, 1), (3, 0)):
        rows.add(s, k[None, i:i + 1], v[None, i:i + 1])
        ref, w = rows.attention(0, s, q[i:i + 1], [model.len[s] - 1], 1 / 8)
        check_out(out[i:i + 1], ref, w)
    assert (out[4] == 0).all()
    for i in (0, 2, 5):
        assert (out[i] == 7).all()
    assert (wide[:, 0] == 7).all() and (wide[:, 5] == 7).all()
    rows.check(model)
    assert c.error_flags() == 0


def test_decode_refuses_duplicates_bad_pages_and_shared_pages(duo):
    c = make(duo, Hkv=2, G=2, D=64)
    model, rows = Model(64, 16, 32, 8), Rows(c)
    fill(c, model, rows, [40, 33, 20, 18], seed=1)
    q, k, v = (normal(3, h, 64, seed=h) for h in (4, 2, 2))
    out = torch.full_like(q, 7.0)
    before = [t.clone() for t in (c.k_pages, c.v_pages, c.k_window, c.v_window)]
    c.decode(0, ints([1, 2, 1]), q, k, v, out)  # the two rows of sequence 1 are left out
    assert c.error_flags() == duo.DUO_ERR_BIT_PAGED_ARGUMENT
    assert (out[0] == 7).all() and (out[2] == 7).all() and not (out[1] == 7).any()
    for t, b in zip((c.k_pages, c.v_pages), before):  # and so are its pages
        assert torch.equal(t[model.pages[1]].view(torch.int16), b[model.pages[1]].view(torch.int16))
    # a page number outside the pool is reported, not used
    c.page_table[0, 1] = 64
    c.page_table[3, 1] = -3
    out = torch.full_like(q, 7.0)
    c.decode(0, ints([0, 3, 2]), q, k, v, out)
    assert c.error_flags() == duo.DUO_ERR_BIT_PAGED_ARGUMENT
    # a length that the table cannot hold
    c.seq_len[0] = 1 << 29
    c.decode(0, ints([0, 7, 2]), q, k, v, out)
    assert c.error_flags() == duo.DUO_ERR_BIT_PAGED_ARGUMENT
    # a shared last page is not written, the row's own output is still right
    c.fork(ints([2]), ints([6]))
    page = model.pages[2][-1]
    held = c.k_pages[page].clone()
    out = torch.full_like(q, float("nan"))
    c.decode(0, ints([-1, -1, 2]), q, k, v, out)
    assert c.error_flags() == duo.DUO_ERR_BIT_PAGED_SHARED
    assert torch.equal(c.k_pages[page].view(torch.int16), held.view(torch.int16)) and torch.isfinite(out[2]).all()
    c.append(0, ints([2]), ints([0, 1]), k, v)
    assert c.error_flags() == duo.DUO_ERR_BIT_PAGED_SHARED
    assert torch.equal(c.k_pages[page].view(torch.int16), held.view(torch.int16))


def test_decode_non_finite_values_follow_the_definition(duo):
    """An infinite or NaN row that is seen reaches the output of its head and no other."""
    c = make(duo, Hkv=2, G=2, D=64, mask=[1, 1])
    model, rows = Model(64, 16, 32, 8), Rows(c)
    fill(c, model, rows, [100], seed=1)
    page, at = model.pages[0][3], 5
    c.v_pages[page, 0, at, 7] = float("inf")
    assert model.extend([0], [1])
    c.extend(ints([0]))
    q, k, v = (normal(1, h, 64, seed=h) for h in (4, 2, 2))
    out = torch.empty_like(q)
    c.decode(0, ints([0]), q, k, v, out)
    assert torch.isposinf(out[0, :2, 7]).all()
    keep = torch.ones(64, dtype=torch.bool)
    keep[7] = False
    assert torch.isfinite(out[0, :2][:, keep]).all() and torch.isfinite(out[0, 2:]).all()
    c.k_pages[page, 1, at, 0] = float("nan")
    c.decode(0, ints([0]), q, k, v, out)
    assert torch.isnan(out[0, 2:]).all() and torch.isfinite(out[0, :2][:, keep]).all()


# ------------------------------------------------------------------------------ packed prompts


def packed(lens, Hq, Hkv, D, seed, lead=0, tail=0):
    start = [lead]
    for n in lens:
        start.append(start[-1] + n)
    total = start[-1] + tail
    return start, tuple(normal(total, h, D, seed=seed * 10 + i) for i, h in enumerate((Hq, Hkv, Hkv)))


def check_prompts(c, layer, start, q, k, v, out):
    L = c.layout
    g = L.num_q_heads // L.num_kv_heads
    for a, b in zip(start, start[1:]):
        for h in range(L.num_kv_heads):
            r = c.is_retrieval[layer * L.num_kv_heads + h]
            from paged_harness import attend
            ref, w = attend(q[a:b, h * g:h * g + g], k[a:b, h], v[a:b, h], list(range(b - a)), L.sink, L.recent, r, 1 / math.sqrt(L.head_dim))
            check_out(out[a:b, h * g:h * g + g], ref, w, f"prompt of {b - a} at {a}, head {h}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 7, 8])
def test_prefill_ragged_prompts(duo, G, D):
    """Lengths around the tile edges, empty prompts, NaN before, between and behind the prompts."""
    c = make(duo, Hkv=2, G=G, D=D, S=4, R=100)
    lens = [1, 127, 0, 128, 129, 255, 256, 0, 257, 2, 500, 640]
    start, (q, k, v) = packed(lens, 2 * G, 2, D, seed=G, lead=3, tail=5)
    for x in (q, k, v):
        x[:3] = float("nan")
        x[-5:] = float("nan")
    out = torch.full_like(q, 7.0)
    c.prefill(0, ints(start), q, k, v, out)
    assert c.error_flags() == 0
    assert (out[:3] == 7).all() and (out[-5:] == 7).all()
    check_prompts(c, 0, start, q, k, v, out)


@pytest.mark.parametrize("mask", [[1, 1], [0, 0]])
@pytest.mark.parametrize("S,R", [(0, 1), (0, 129), (300, 1), (64, 256), (127, 128), (128, 300), (1000, 5)])
def test_prefill_windows(duo, mask, S, R):
    for G in (1, 2):
        c = make(duo, Hkv=2, G=G, D=128, S=S, R=R, mask=mask)
        start, (q, k, v) = packed([700, 33, 1200], 2 * G, 2, 128, seed=S + R)
        out = torch.full_like(q, float("nan"))
        c.prefill(0, ints(start), q, k, v, out)
        check_prompts(c, 0, start, q, k, v, out)
        assert c.error_flags() == 0


def test_prefill_poisoned_neighbour_and_large_scores(duo):
    """A prompt of NaN and infinities changes nothing in the prompts around it; sink-like keys move the maxima."""
    c = make(duo, Hkv=2, G=2, D=128, S=4, R=60)
    start, (q, k, v) = packed([200, 90, 300], 4, 2, 128, seed=5)
    k[:3] *= 8
    k[start[2] + 150:start[2] + 160] *= 16
    q[start[2] + 100:] *= 4
    clean = torch.full_like(q, float("nan"))
    c.prefill(0, ints(start), q, k, v, clean)
    for x, bad in ((q, float("nan")), (k, float("inf")), (v, float("-inf"))):
        x[start[1]:start[2]] = bad
    out = torch.full_like(q, float("nan"))
    c.prefill(0, ints(start), q, k, v, out)
    assert torch.equal(out[:start[1]], clean[:start[1]]) and torch.equal(out[start[2]:], clean[start[2]:])
    v64 = v.clone()
    v64[start[1]:start[2]] = 0
    check_prompts(c, 0, [0, start[1]], q, k, v64, out)


@pytest.mark.parametrize("G,D", [(1, 128), (2, 128), (2, 64)])
def test_prefill_maxima_that_move_late(duo, G, D):
    """Scores whose maximum moves in the middle of a prompt, in either half of a key tile, by a little, by 2^30 and by
    more than 32 bits hold, up and down, for some rows of a tile and not for others. Keys are constant rows of few
    bits, so every score is exact up to the scale's rounding, whatever its size."""
    c = make(duo, Hkv=2, G=G, D=D, S=70, R=900, mask=[1, 0])
    n = 1300
    start, (q, k, v) = packed([n], 2 * G, 2, D, seed=40 + G)
    level = torch.zeros(n)
    for at, to in ((300, 0.25), (330, 0.5), (460, 2.5), (500, 2.0), (650, 4.5), (718, 5.0), (719, 15.0), (730, 6.0), (1100, 1.0),
                   (1170, 15.5)):
        level[at:] = to
    level += torch.randint(0, 6, (n,), generator=torch.Generator().manual_seed(3)) / 16
    k[:] = level.to(k).view(n, 1, 1)
    sign = torch.tensor([1.0, -1.0, 0.5, 1.0, 0.0])[torch.arange(n) % 5]
    q[:] = sign.to(q).view(n, 1, 1)
    out = torch.full_like(q, float("nan"))
    c.prefill(0, ints(start), q, k, v, out)
    check_prompts(c, 0, start, q, k, v, out)
    assert c.error_flags() == 0


@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("S,R", [(4, 40), (130, 300)])
def test_prefill_non_finite_values_reach_their_readers_only(duo, G, S, R):
    """Infinite and NaN value rows: exactly the queries that see such a row get them, in its columns alone."""
    lens = [500, 20, 3, 60, 0, 9, 700]  # the short ones share tiles
    c = make(duo, Hkv=2, G=G, D=128, S=S, R=R)
    start, (q, k, v) = packed(lens, 2 * G, 2, 128, seed=S)
    inf, nan = float("inf"), float("nan")
    odd = torch.zeros(v.shape, dtype=torch.float64, device="cuda")
    for row, col, x in ((5, 3, inf), (120, 7, -inf), (130, 3, nan), (400, 64, inf), (499, 1, nan), (505, 9, inf), (521, 100, -inf),
                        (540, 11, nan), (585, 127, inf), (592, 0, nan), (600, 5, -inf), (900, 5, inf), (1291, 8, nan)):
        odd[row, :, col] = x
    bad = ~torch.isfinite(odd)
    clean = v.clone()
    clean[bad] = 0
    v[bad] = odd[bad].to(v.dtype)
    out = torch.full_like(q, 7.0)
    c.prefill(0, ints(start), q, k, v, out)
    from paged_harness import attend
    for a, b in zip(start, start[1:]):
        i = torch.arange(b - a, device="cuda")
        for h in range(2):
            ref, w = attend(q[a:b, h * G:h * G + G], k[a:b, h], clean[a:b, h], i, S, R, h == 0, 1 / math.sqrt(128))
            seen = i[None] <= i[:, None]
            if h == 1:
                seen &= (i[None] < S) | (i[:, None] - i[None] < R)
            extra = torch.zeros((b - a, 128), dtype=torch.float64, device="cuda")
            for j in range(b - a):
                if bad[a + j, h].any():
                    extra = extra + torch.where(seen[:, j, None] & bad[a + j, h], odd[a + j, h], 0.0)
            got, special = out[a:b, h * G:h * G + G].double(), ~torch.isfinite(extra)
            special = special[:, None].expand(-1, G, -1)
            want = extra[:, None].expand(-1, G, -1)
            assert torch.equal(torch.isnan(got), torch.isnan(want)), (a, h)
            assert torch.equal(torch.isinf(got), torch.isinf(want)) and torch.equal(got[torch.isinf(got)], want[torch.isinf(want)])
            keep = ~special
            check_out(got[keep], ref[keep], w[keep], f"prompt at {a}, head {h}")
    assert c.error_flags() == 0


@pytest.mark.parametrize("S,R", [(4, 5), (0, 300), (40, 16)])
@pytest.mark.parametrize("G", [1, 4])
def test_prefill_prompts_that_share_tiles(duo, G, S, R):
    """Runs of short prompts between long ones, an unusable range among them: every row of every prompt."""
    c = make(duo, Hkv=2, G=G, D=64, S=S, R=R)
    lens = [30, 1, 96, 1, 128, 127, 2, 200, 0, 0, 64, 64, 64, 1, 1, 1, 1, 300, 5]
    start, (q, k, v) = packed(lens, 2 * G, 2, 64, seed=R, tail=40)
    out = torch.full_like(q, 7.0)
    rs = start + [start[-1] - 3, start[-1] + 20, start[-1] + 37]  # backwards; then two prompts over the last rows
    c.prefill(0, ints(rs), q, k, v, out)
    assert c.error_flags() == duo.DUO_ERR_BIT_PAGED_ARGUMENT
    check_prompts(c, 0, start[:-1], q, k, v, out)  # (the last prompt's final rows are the next but one's too)
    check_prompts(c, 0, [start[-1] + 20, start[-1] + 37], q, k, v, out)
    assert (out[start[-1] + 37:] == 7).all()


def test_prefill_many_prompts_strided(duo):
    """More prompts than SMs, out of a fused projection, into a wider tensor."""
    c = make(duo, Hkv=2, G=2, D=64, S=4, R=16)
    rng = random.Random(3)
    lens = [rng.randint(0, 90) for _ in range(512)]
    start = [0]
    for n in lens:
        start.append(start[-1] + n)
    qkv = normal(start[-1], 8, 64, seed=1)
    wide = torch.full((start[-1], 6, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    q, k, v, out = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], wide[:, 2:]
    c.prefill(0, ints(start), q, k, v, out)
    assert (wide[:, :2] == 7).all() and c.error_flags() == 0
    some = [i for i in range(0, 512, 7)]
    for i in some:
        check_prompts(c, 0, start[i:i + 2], q, k, v, out)


def test_prefill_bad_ranges_are_skipped(duo):
    c = make(duo, Hkv=2, G=2, D=64)
    q, k, v = (normal(100, h, 64, seed=h) for h in (4, 2, 2))
    out = torch.full_like(q, 7.0)
    c.prefill(0, ints([0, 40, 30, 101, -5, 10]), q, k, v, out)  # good; backwards; too long; ends before; starts below 0
    assert c.error_flags() == duo.DUO_ERR_BIT_PAGED_ARGUMENT
    check_prompts(c, 0, [0, 40], q, k, v, out)
    assert (out[40:] == 7).all()
    model = Model(64, 16, 32, 8)
    c.extend(ints([0, 1]), ints([5, 50]))
    held = c.k_pages.clone()
    c.append(0, ints([0, 1]), ints([0, 6, 101]), k, v)  # longer than the sequence; outside the rows
    assert c.error_flags() == duo.DUO_ERR_BIT_PAGED_ARGUMENT
    assert torch.equal(held.view(torch.int16), c.k_pages.view(torch.int16))


def test_prefill_long_prompt_rows(duo):
    """A 6000-token prompt beside a short one, grouped heads: sampled rows."""
    c = make(duo, Hkv=2, G=4, D=128, S=64, R=256)
    start, (q, k, v) = packed([6000, 100], 8, 2, 128, seed=8)
    out = torch.full_like(q, float("nan"))
    c.prefill(0, ints(start), q, k, v, out)
    from paged_harness import attend
    at = [0, 1, 127, 128, 3000, 4095, 4096, 5887, 5888, 5999]
    for h in range(2):
        ref, w = attend(q[at, h * 4:h * 4 + 4], k[:6000, h], v[:6000, h], at, 64, 256, h == 0, 1 / math.sqrt(128))
        check_out(out[at, h * 4:h * 4 + 4], ref, w)
    assert torch.isfinite(out).all() and c.error_flags() == 0


# ------------------------------------------------------------------------------ page upkeep


def test_pages_random_run_against_model(duo):
    """Hundreds of calls in a random order, some of which cannot be done: table, counts and lengths as in the model."""
    rng = random.Random(11)
    c = make(duo, Hkv=2, G=1, D=64, P=16, num_pages=90, max_pages=12, max_seqs=24, layers=2, mask=[1, 0, 0, 1])
    model = Model(90, 16, 12, 24)
    for turn in range(250):
        live = [s for s in model.len if model.len[s] > 0]
        empty = [s for s in model.len if model.len[s] == 0]
        op = rng.choice(["extend", "extend", "extend", "fork", "copy", "release", "compact"])
        want = 0
        if op == "extend":
            seqs = rng.sample(range(24), rng.randint(1, 10))
            n_tok = [rng.choice([0, 1, 1, 1, 5, 16, 33]) for _ in seqs]
            if all(x == 1 for x in n_tok):
                c.extend(ints(seqs))
            else:
                c.extend(ints(seqs), ints(n_tok))
            want = 0 if model.extend(seqs, n_tok) else duo.DUO_ERR_BIT_PAGED_CAPACITY
        elif op in ("fork", "copy") and live and empty:
            n = rng.randint(1, min(4, len(empty)))
            src, dst = [rng.choice(live) for _ in range(n)], rng.sample(empty, n)
            getattr(c, op)(ints(src), ints(dst))
            if op == "copy" and sum(len(model.pages[s]) for s in src) > len(model.free()):
                want = duo.DUO_ERR_BIT_PAGED_CAPACITY
            else:
                getattr(model, op)(src, dst)
        elif op == "release" and live:
            seqs = rng.sample(live, rng.randint(1, max(1, len(live) // 2)))
            c.release(ints(seqs))
            model.release(seqs)
        elif op == "compact":
            c.compact()
            model.compact()
        assert c.error_flags() == want, (turn, op)
        model.check(c)


def test_pages_refusals(duo):
    c = make(duo, Hkv=2, G=1, D=64, P=16, num_pages=20, max_pages=6, max_seqs=8)
    model = Model(20, 16, 6, 8)
    A, CAP = duo.DUO_ERR_BIT_PAGED_ARGUMENT, duo.DUO_ERR_BIT_PAGED_CAPACITY
    assert model.extend([0, 1, 2], [20, 33, 1])
    c.extend(ints([0, -1, 1, 2, 99]), ints([20, 7, 33, 1, 7]))  # padding entries are skipped
    model.check(c)
    for call, flag in ((lambda: c.extend(ints([3, 4, 3])), A), (lambda: c.extend(ints([3, 4]), ints([1, -1])), A),
                       (lambda: c.extend(ints([3, 4]), ints([1, 97])), CAP), (lambda: c.extend(ints([3, 4, 5]), ints([90, 90, 90])), CAP),
                       (lambda: c.fork(ints([0, 1]), ints([3, 3])), A), (lambda: c.fork(ints([0, 0]), ints([0, 1])), A),
                       (lambda: c.copy(ints([0, 1]), ints([3, 3])), A), (lambda: c.release(ints([1, 1])), A)):
        assert c.error_flags() == 0
        call()
        assert c.error_flags() == flag
        model.check(c)
    c.fork(ints([0, 3, 1]), ints([4, 5, 3]))  # 3 is a destination and a source: the entry that fills it is left out
    model.fork([0], [4])
    assert c.error_flags() == A
    model.check(c)
    c.seq_len[6] = -5
    c.release(ints([6]))
    assert c.error_flags() == A
    c.extend(ints([6]))
    assert c.error_flags() == A
    c.seq_len[6] = 0
    c.page_table[4, 1] = 4096  # a page number outside the pool
    c.extend(ints([4]))
    assert c.error_flags() == A
    c.release(ints([4]))
    assert c.error_flags() == A


@pytest.mark.parametrize("S,R,n", [(44, 256, 6), (0, 2, 40), (300, 700, 1)])
def test_fork_windows_of_many_chunks(duo, S, R, n):
    """Windows larger than one CTA's piece, and smaller: every fork has its source's, bit for bit, a second call gives
    what the first gave, and entries that are refused leave their sequence as it was."""
    c = make(duo, Hkv=4, G=1, D=128, S=S, R=R, max_seqs=64, mask=[0, 1, 0, 0, 1, 1, 0, 0, 0, 0, 0, 0], layers=3)
    for w in (c.k_window, c.v_window):
        w.copy_(torch.randint(-100, 100, w.shape, generator=torch.Generator().manual_seed(S + R)).to(w))
    c.extend(ints([0, 1, 2]), ints([37, 16, 5]))
    before = [w.clone() for w in (c.k_window, c.v_window)]
    for dst in (list(range(10, 10 + n)), list(range(63, 63 - min(n, 10), -1))):
        src = [(i * i) % 3 for i in range(len(dst))]
        # refused: a dst twice, a dst that is not empty, a dst that is a source; padding
        c.fork(ints(src + [0, 1, 0, 2, -1, 0]), ints(dst + [5, 5, 1, 2, 9, 64]))
        for w, b in zip((c.k_window, c.v_window), before):
            for i, d in zip(src, dst):
                b[d] = b[i]
            assert torch.equal(w, b)
        for i, d in zip(src, dst):
            pages = -(-int(c.seq_len[i]) // 16)
            assert c.seq_len[d] == c.seq_len[i] and torch.equal(c.page_table[d, :pages], c.page_table[i, :pages])
        assert c.seq_len[5] == 0 and c.seq_len[9] == 0
        assert c.error_flags() == duo.DUO_ERR_BIT_PAGED_ARGUMENT


def test_pages_requests_beyond_any_pool(duo):
    """Needs whose sum passes 32 bits are refused like any other that the pool cannot meet."""
    c = make(duo, Hkv=1, G=1, D=64, P=16, num_pages=9, max_pages=1 << 23, max_seqs=512, mask=[0])
    seqs = ints(range(512))
    c.extend(seqs, ints([1 << 27] * 512))
    assert c.error_flags() == duo.DUO_ERR_BIT_PAGED_CAPACITY
    assert int(c.seq_len.abs().sum()) == 0 and int(c.page_ref.abs().sum()) == 0
    c.extend(seqs, ints([(1 << 27) + 1] * 512))
    assert c.error_flags() == duo.DUO_ERR_BIT_PAGED_CAPACITY
    c.extend(ints([7]), ints([9 * 16]))
    assert c.error_flags() == 0 and int(c.seq_len[7]) == 144


@pytest.mark.parametrize("num_pages", [1, 3, 1023, 1025, 4097, 70001])
def test_pages_pool_sizes(duo, num_pages):
    """The last page of a pool of any size is found, and no page behind it."""
    c = make(duo, Hkv=1, G=1, D=64, P=16, num_pages=num_pages, max_pages=8, max_seqs=8, mask=[0])
    c.page_ref.fill_(1)
    c.page_ref[num_pages - 1] = 0
    c.extend(ints([2]), ints([16]))
    assert c.error_flags() == 0 and int(c.page_table[2, 0]) == num_pages - 1
    c.extend(ints([2]))
    assert c.error_flags() == duo.DUO_ERR_BIT_PAGED_CAPACITY and int(c.seq_len[2]) == 16
    if num_pages > 3:
        c.page_ref[5:] = 0
        c.page_ref[num_pages - 1] = 1
        c.page_ref[7] = 1
        c.compact()
        assert int(c.page_table[2, 0]) == 6 and int(c.page_ref.sum()) == 7 and int(c.page_ref[:7].sum()) == 7


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("G,D,P", [(2, 64, 16), (4, 128, 64)])
def test_run_of_all_operators(duo, G, D, P, fp8):
    """Prompts, beams, steps, beams dropped, a copy, a compaction and more steps, three layers: every output and every
    cached row on the way."""
    Hkv, layers = 2, 3
    c = make(duo, Hkv=Hkv, G=G, D=D, P=P, S=4, R=40, num_pages=160, max_pages=20, max_seqs=12, layers=layers, mask=[1, 0, 0, 1, 1, 1], fp8=fp8)
    sc = scales_for(c) if fp8 else None
    if fp8:
        for l in range(layers):
            c.set_kv_scales(l, *sc)
    model, rows = Model(160, P, 20, 12), Rows(c)
    lens = [37, 2 * P, 120]
    assert model.extend([0, 1, 2], lens)
    c.extend(ints([0, 1, 2]), ints(lens))
    start, _ = packed(lens, 1, 1, D, seed=0)
    kv = []
    for l in range(layers):
        _, (q, k, v) = packed(lens, Hkv * G, Hkv, D, seed=l)
        out = torch.full_like(q, float("nan"))
        c.prefill(l, ints(start), q, k, v, out)
        c.append(l, ints([0, 1, 2]), ints(start), k, v)
        check_prompts(c, l, start, q, k, v, out)
        kv.append((k, v))
    for s in range(3):
        rows.rows[s] = tuple(torch.stack([kv[l][x][start[s]:start[s + 1]] for l in range(layers)]) for x in (0, 1))
    step(c, model, rows, [0, 1, 2], 1, sc)
    c.fork(ints([0, 0, 2]), ints([3, 4, 5]))
    model.fork([0, 0, 2], [3, 4, 5])
    for a, b in ((0, 3), (0, 4), (2, 5)):
        rows.rows[b] = rows.rows[a]
    rows.check(model, sc)
    step(c, model, rows, [3, 0, 5, 4, 1, 2], 2, sc)
    step(c, model, rows, [4, 3, 1], 3, sc)
    model.check(c)
    rows.check(model, sc)
    c.release(ints([0, 5]))
    model.release([0, 5])
    for s in (0, 5):
        rows.rows[s] = tuple(x[:, :0] for x in rows.rows[s])
    c.copy(ints([4, 1]), ints([9, 5]))
    model.copy([4, 1], [9, 5])
    rows.rows[9], rows.rows[5] = rows.rows[4], rows.rows[1]
    c.release(ints([3]))
    model.release([3])
    rows.rows[3] = tuple(x[:, :0] for x in rows.rows[3])
    c.compact()
    model.compact()
    model.check(c)
    rows.check(model, sc)
    for t in range(3):
        step(c, model, rows, [9, 5, 4, 2], 4 + t, sc)
    model.check(c)
    rows.check(model, sc)
    assert c.error_flags() == 0


# ------------------------------------------------------------------------------ streams, graphs


def test_captured_step_serves_many_tokens(duo):
    """One captured step (extend, two layers of decode), replayed: each replay appends and attends at the next position."""
    c = make(duo, Hkv=2, G=2, D=64, P=16, S=4, R=16, layers=2, mask=[1, 0, 0, 1])
    model, rows = Model(64, 16, 32, 8), Rows(c)
    fill(c, model, rows, [30, 90], seed=1)
    seqs = ints([1, 0])
    q, k, v = (normal(2, 2, h, 64, seed=h) for h in (4, 2, 2))
    out = torch.empty_like(q)

    def one():
        c.extend(seqs)
        for l in range(2):
            c.decode(l, seqs, q[l], k[l], v[l], out[l])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            one()
    torch.cuda.current_stream().wait_stream(side)
    for t in range(40):
        for x, h in ((q, 4), (k, 2), (v, 2)):
            x.copy_(normal(2, 2, h, 64, seed=1000 + 10 * t + h))
        graph.replay()
        assert model.extend([1, 0], [1, 1])
        for i, s in enumerate([1, 0]):
            rows.add(s, k[:, i:i + 1].clone(), v[:, i:i + 1].clone())
            for l in range(2):
                ref, w = rows.attention(l, s, q[l, i:i + 1], [model.len[s] - 1], 1 / 8)
                check_out(out[l, i:i + 1], ref, w, f"replay {t}")
    model.check(c)
    rows.check(model)
    assert c.error_flags() == 0


def test_captured_prompts(duo):
    c = make(duo, Hkv=2, G=2, D=64, S=4, R=16)
    start, (q, k, v) = packed([100, 50], 4, 2, 64, seed=1, tail=60)
    rs = ints(start)
    out = torch.full_like(q, 7.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            c.prefill(0, rs, q, k, v, out)
    torch.cuda.current_stream().wait_stream(side)
    for start in ([0, 100, 150], [5, 200, 210], [0, 0, 129]):  # the prompts are what row_start says at the replay
        rs.copy_(ints(start))
        out.fill_(7.0)
        graph.replay()
        check_prompts(c, 0, start, q, k, v, out)
        assert (out[:start[0]] == 7).all() and (out[start[-1]:] == 7).all()
    assert c.error_flags() == 0


def test_other_stream_and_two_caches(duo):
    """Two caches on two streams at once do not meet; a stream argument is used."""
    made = []
    for i in range(2):
        c = make(duo, Hkv=2, G=4, D=128, P=32, num_pages=200, max_pages=100, S=4, R=60)
        model, rows = Model(200, 32, 100, 8), Rows(c)
        fill(c, model, rows, [2500, 300], seed=i)
        made.append((c, model, rows))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    args, seqs = [], ints([0, 1])
    for i, (c, model, rows) in enumerate(made):
        args.append([normal(2, h, 128, seed=i * 5 + h) for h in (8, 2, 2)])
        args[-1].append(torch.full_like(args[-1][0], float("nan")))
    torch.cuda.synchronize()
    for i, (c, model, rows) in enumerate(made):
        c.extend(seqs, stream=streams[i])
    for _ in range(20):
        for i, (c, model, rows) in enumerate(made):
            c.decode(0, seqs, *args[i], stream=streams[i].cuda_stream)
    torch.cuda.synchronize()
    for i, (c, model, rows) in enumerate(made):
        assert model.extend([0, 1], [1, 1])
        q, k, v, out = args[i]
        for s in range(2):
            rows.add(s, k[None, s:s + 1], v[None, s:s + 1])
            ref, w = rows.attention(0, s, q[s:s + 1], [model.len[s] - 1], 1 / math.sqrt(128))
            check_out(out[s:s + 1], ref, w)
        rows.check(model)
        assert c.error_flags() == 0
