"""Appending batches whose entries are of very different length, or share rows, to a paged cache: bits and time."""
import pytest
import torch

from paged_harness import Model, Rows, ints, normal, poison

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def duo():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    import mixed_head_kv_b200
    return mixed_head_kv_b200


def device_us(f, repeats=10):
    f()
    best = float("inf")
    for _ in range(repeats):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1000)
    return best


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,n", [(64, 512), (128, 301)])
def test_one_long_entry_among_many_short_ones(duo, D, n, fp8):
    """A prompt among hundreds of one-token entries, first, last and in the middle, empty entries and padding between."""
    c = duo.PagedCache(1, n, 2, 2, D, 4, 60, 32, 300 + n, 140, [1, 0], kv_format=duo.DUO_KV_E4M3 if fp8 else duo.DUO_KV_BF16)
    scales = [[0.5, 1.0], [0.25, 1.0]]
    if fp8:
        c.set_kv_scales(0, *scales)
    poison(c)
    model, rows = Model(300 + n, 32, 140, n), Rows(c)
    used = 0
    for long_at, length in ((0, 1500), (n - 1, 777), (n // 2, 1201)):
        lens = [1 if i % 3 else 0 for i in range(n)]
        lens[long_at] = length
        seqs = [i if i % 11 != 5 or i == long_at else -1 for i in range(n)]
        live = [i for i in range(n) if seqs[i] >= 0]
        assert model.extend(live, [lens[i] for i in live])
        c.extend(ints(seqs), ints(lens))
        start = [7]
        for x in lens:
            start.append(start[-1] + x)
        k, v = normal(start[-1] + 3, 2, D, seed=used), normal(start[-1] + 3, 2, D, seed=used + 1)
        used += 2
        c.append(0, ints(seqs), ints(start), k, v)
        for i in live:
            rows.add(i, k[None, start[i]:start[i + 1]], v[None, start[i]:start[i + 1]])
    model.check(c)
    rows.check(model, scales)
    assert c.error_flags() == 0


def test_a_long_entry_takes_no_longer_for_the_company(duo):
    """32768 tokens among 511 entries of one: not far from the two on their own (where every entry had as many CTAs, 1090 us
    instead of 23 and 6)."""
    c = duo.PagedCache(1, 512, 16, 8, 128, 64, 256, 64, 1100, 520, [1, 0] * 4)
    c.extend(ints(range(512)), ints([32768] + [1] * 511))
    k, v = normal(33279, 8, 128, seed=1), normal(33279, 8, 128, seed=2)
    seqs, start = ints(range(512)), ints([0] + [32768 + i for i in range(512)])
    one, first = ints([0]), ints([0, 32768])
    alone = device_us(lambda: c.append(0, one, first, k, v))
    both = device_us(lambda: c.append(0, seqs, start, k, v))
    assert c.error_flags() == 0
    assert both < 3 * alone + 20, f"{both:.1f} us against {alone:.1f}"


def test_rows_of_two_entries(duo):
    """Ranges may overlap behind one that runs backwards: both sequences get the rows."""
    c = duo.PagedCache(1, 4, 1, 1, 64, 2, 5, 16, 20, 8, [1])
    poison(c)
    model, rows = Model(20, 16, 8, 4), Rows(c)
    assert model.extend([0, 1, 2], [40, 3, 40])
    c.extend(ints([0, 1, 2]), ints([40, 3, 40]))
    k, v = normal(60, 1, 64, seed=1), normal(60, 1, 64, seed=2)
    c.append(0, ints([0, 1, 2]), ints([0, 40, 10, 50]), k, v)
    assert c.error_flags() == duo.DUO_ERR_BIT_PAGED_ARGUMENT
    for s, a in ((0, 0), (2, 10)):
        rows.rows[s] = (k[None, a:a + 40], v[None, a:a + 40])
    model.len[1] = 0
    rows.check(model)


def test_more_tokens_than_32_bits_hold_are_refused(duo):
    """Only overlapping ranges have so many: nothing is appended for any entry."""
    n = 1 << 26
    c = duo.PagedCache(1, 64, 1, 1, 64, 2, 5, 64, 4, 1 << 21, [0])
    c.k_window.fill_(3.0)
    c.v_window.fill_(3.0)
    c.seq_len.fill_(n)
    rows = torch.empty(n, 1, 64, dtype=torch.bfloat16, device="cuda")
    c.append(0, ints(range(64)), ints([0, n] * 32 + [0]), rows, rows)
    assert c.error_flags() == duo.DUO_ERR_BIT_PAGED_ARGUMENT
    assert (c.k_window == 3).all() and (c.v_window == 3).all()


def test_captured_append_follows_its_entries(duo):
    """One captured extend and append, replayed with other sequences, counts and rows."""
    c = duo.PagedCache(1, 8, 2, 2, 64, 4, 20, 16, 60, 20, [1, 0])
    poison(c)
    model, rows = Model(60, 16, 20, 8), Rows(c)
    seqs, n_tok, start = ints([0] * 4), ints([0] * 4), ints([0] * 5)
    k, v = normal(200, 2, 64, seed=1), normal(200, 2, 64, seed=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            c.extend(seqs, n_tok)
            c.append(0, seqs, start, k, v)
    torch.cuda.current_stream().wait_stream(side)
    for turn, (s, n) in enumerate((([3, 1, 7, -1], [150, 1, 0, 9]), ([0, 3, 9, 1], [1, 1, 5, 190]), ([5, -1, -1, 3], [17, 1, 1, 16]))):
        live = [(a, b) for a, b in zip(s, n) if 0 <= a < 8]
        assert model.extend([a for a, _ in live], [b for _, b in live])
        at = [0]
        for b in n:
            at.append(at[-1] + b)
        for t, x in ((seqs, s), (n_tok, n), (start, at)):
            t.copy_(ints(x))
        k.copy_(normal(200, 2, 64, seed=10 + turn))
        v.copy_(normal(200, 2, 64, seed=20 + turn))
        graph.replay()
        for i, a in enumerate(s):
            if 0 <= a < 8:
                rows.add(a, k[None, at[i]:at[i + 1]].clone(), v[None, at[i]:at[i + 1]].clone())
    model.check(c)
    rows.check(model)
    assert c.error_flags() == 0
