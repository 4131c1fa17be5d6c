"""The paged cache's attention where its arithmetic could give way, against the plain 64-bit forms (paged_harness.py)."""
import math

import pytest
import torch

from paged_harness import attend, check_out, ints, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def duo():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    import mixed_head_kv_b200
    return mixed_head_kv_b200


def device_ms(f, repeats=8):
    """Shortest of some calls, after a warm one."""
    f()
    best = float("inf")
    for _ in range(repeats):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


# ------------------------------------------------------------------------------ packed prompts


@pytest.mark.parametrize("above", [4.5, 6.5, 7.5])
def test_prefill_scores_a_little_above_the_first_tiles_cost_what_others_do(duo, above):
    """All scores behind the first 128 keys lie 2^above over theirs: too little to move the maximum by the 2^8 rule,
    enough for a half's 64 weights to add up to more than 2^10. The maximum has to move once and the rest of the prompt be taken in
    one pass; a prompt that stays in two passes takes 1.68 times as long."""
    n, heads = 16384, 4
    c = duo.PagedCache(1, 2, 2 * heads, heads, 128, 64, 256, 64, 4, 2, [1] * heads)
    q = torch.ones(n, 2 * heads, 128, dtype=torch.bfloat16, device="cuda")
    v = normal(n, heads, 128, seed=1)
    k = torch.full((n, heads, 128), above / (math.sqrt(128) * math.log2(math.e)), dtype=torch.bfloat16, device="cuda")
    flat = k.clone()
    k[:128] = 0
    start, out = ints([0, n]), torch.full_like(q, float("nan"))
    slow = device_ms(lambda: c.prefill(0, start, q, k, v, out))
    at = [0, 127, 128, 300, 8000, n - 1]
    ref, w = attend(q[at, :2], k[:, 0], v[:, 0], at, 64, 256, True, 1 / math.sqrt(128))
    check_out(out[at, :2], ref, w)
    fast = device_ms(lambda: c.prefill(0, start, q, flat, v, out))
    assert c.error_flags() == 0
    assert slow < 1.25 * fast, f"{slow:.3f} ms against {fast:.3f}"


@pytest.mark.parametrize("G,D", [(1, 128), (2, 64)])
@pytest.mark.parametrize("size", [22, 23, 24, 30, 31, 32, 33, 36, 45])
def test_prefill_scores_of_any_size(duo, G, D, size):
    """Scores of about 2^size, above and below zero: what a product with the scale loses to rounding is then 2^(size - 24)
    and more, all of which the weights must not see. Keys and queries are constant rows of few bits: every score is exact
    before the scale. Scores differ by at least 2^(size - 5) or not at all, so the weights are 0 or equal."""
    c = duo.PagedCache(1, 2, 2 * G, 2, D, 70, 400, 16, 4, 2, [1, 0])
    n = 900
    gen = torch.Generator().manual_seed(size)
    level = 1.0 + torch.randint(0, 8, (n,), generator=gen) / 8
    level[:130] = 1.0  # (a first tile of equal scores)
    level[500:] *= 1.5
    sign = torch.tensor([1.0, -1.0, 0.0, 1.0])[torch.arange(n) % 4]
    to = (size - math.log2(math.sqrt(D) * math.log2(math.e))) / 2  # D x 2^to x 2^to x the scale, in the exp2 domain
    q = (sign * 2.0 ** round(to)).to(torch.bfloat16).view(n, 1, 1).expand(n, 2 * G, D).contiguous().cuda()
    k = (level * 2.0 ** (size - math.floor(math.log2(math.sqrt(D) * math.log2(math.e))) - round(to))).to(torch.bfloat16).view(n, 1, 1)
    k = k.expand(n, 2, D).contiguous().cuda()
    v = normal(n, 2, D, seed=size)
    out = torch.full_like(q, float("nan"))
    c.prefill(0, ints([0, n]), q, k, v, out)
    assert c.error_flags() == 0
    for h in range(2):
        ref, w = attend(q[:, h * G:h * G + G], k[:, h], v[:, h], list(range(n)), 70, 400, h == 0, 1 / math.sqrt(D))
        check_out(out[:, h * G:h * G + G], ref, w, f"head {h}")


@pytest.mark.parametrize("G", [5, 6])
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_other_groups(duo, G, D):
    """Groups that no other test has: an odd one and an even one above four."""
    c = duo.PagedCache(1, 2, 2 * G, 2, D, 4, 100, 16, 4, 2, [1, 0])
    start = [0, 1, 130, 130, 387, 400, 1000]
    q, k, v = (normal(1000, h, D, seed=G + h) for h in (2 * G, 2, 2))
    out = torch.full_like(q, float("nan"))
    c.prefill(0, ints(start), q, k, v, out)
    assert c.error_flags() == 0
    for a, b in zip(start, start[1:]):
        for h in range(2):
            ref, w = attend(q[a:b, h * G:h * G + G], k[a:b, h], v[a:b, h], list(range(b - a)), 4, 100, h == 0, 1 / math.sqrt(D))
            check_out(out[a:b, h * G:h * G + G], ref, w, f"prompt at {a}, head {h}")


# ------------------------------------------------------------------------------ decode


@pytest.mark.parametrize("D,G", [(64, 1), (128, 4), (128, 8)])
def test_decode_e4m3_many_small_weights_beside_a_large_one(duo, D, G):
    """One key 2^25.5 above thousands of others: half of what f16 holds at its smallest. Its value row is zero, theirs are
    one, so the output is what they weigh together, and what a warp drops shows. As many sequences as make every pair
    lie in one share, where one warp has the large key and a quarter of the others."""
    n, seqs, P = 6000, 150, 128
    pages = -(-n // P)
    c = duo.PagedCache(1, seqs, 2 * G, 2, D, 4, 16, P, pages + seqs + 1, pages + 1, [1, 1], kv_format=duo.DUO_KV_E4M3)
    # q = 1: a key row of x in 13 columns scores 13 x scale x log2(e) above one of zeros (0 in the exp2 domain)
    x, cols = 16.0, round(25.5 * math.sqrt(D) / (16.0 * math.log2(math.e)))
    k, v = torch.zeros(n, 2, D, dtype=torch.bfloat16, device="cuda"), torch.ones(n, 2, D, dtype=torch.bfloat16, device="cuda")
    k[40, :, :cols] = x
    v[40] = 0
    c.extend(ints([0]), ints([n]))
    c.append(0, ints([0]), ints([0, n]), k, v)
    c.fork(ints([0] * (seqs - 1)), ints(range(1, seqs)))
    order = ints(range(seqs))
    c.extend(order)
    new_k, new_v = torch.zeros(seqs, 2, D, dtype=torch.bfloat16, device="cuda"), torch.ones(seqs, 2, D, dtype=torch.bfloat16, device="cuda")
    q = torch.ones(seqs, 2 * G, D, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, float("nan"))
    c.decode(0, order, q, new_k, new_v, out)
    assert c.error_flags() == 0
    one = torch.cat([k[:, 0], new_k[:1, 0]]), torch.cat([v[:, 0], new_v[:1, 0]])
    ref, w = attend(q[:1, :1], *one, [n], 4, 16, True, 1 / math.sqrt(D))
    assert 1e-5 < float(ref[0, 0, 0]) < 1e-3  # the others' part
    # Weights rounded to f16 (2^-11), their 32-bit errors (scores below 32: exp2 of one is off by 32 x 2^-24 and its own
    # 2^-22; sums of 6000 positive terms, 1500 in a row, by 1500 x 2^-24 at most), the output's rounding to bf16 (2^-8).
    # In the warp with the large key the others' weights times 2^7 are f16 numbers without leading bit, in steps of
    # 2^-24: half a step is 2^-32 of the large weight, for each of a quarter of the rows and one tile's share more.
    tol = float(ref[0, 0, 0]) * (2.0 ** -11 + 3e-6 + 1.1e-4 + 2.0 ** -8) + (n / 4 + 128) * 2.0 ** -32
    worst = float((out.double() - ref[0, 0, 0]).abs().max())
    assert worst <= tol, f"{worst:.3g} of {float(ref[0, 0, 0]):.3g}"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("G,D", [(1, 128), (8, 64)])
@pytest.mark.parametrize("size", [0, 20, 24, 25, 26, 27, 30, 32, 40])
def test_decode_scores_of_any_size(duo, G, D, size, fp8):
    """Scores of about 2^size that differ by 2^(size - 5) or not at all (weights 0 or equal), then value rows of ones with
    scores that differ by as little as 32 bits show: whatever the weights are, they divide by their sum."""
    n = 3000
    c = duo.PagedCache(1, 2, 2 * G, 2, D, 4, 60, 32, 100, 96, [1, 0], kv_format=duo.DUO_KV_E4M3 if fp8 else duo.DUO_KV_BF16)
    from paged_harness import Rows
    rows, gen = Rows(c), torch.Generator().manual_seed(size)
    level = 1.0 + torch.randint(0, 8, (n,), generator=gen) / 8
    level[:500] = 1.0
    level[n // 2:] *= 2
    k = level.to(torch.bfloat16).view(n, 1, 1).expand(n, 2, D).contiguous().cuda()
    v = normal(n, 2, D, seed=size)
    scales = [[1.0, 1.0], [1.0, 1.0]]
    c.extend(ints([0]), ints([n]))
    c.append(0, ints([0]), ints([0, n]), k, v)
    rows.rows[0] = (k[None], v[None])
    factor = 2.0 ** (size - round(math.log2(math.sqrt(D) * math.log2(math.e))))
    out = torch.empty(1, 2 * G, D, dtype=torch.bfloat16, device="cuda")
    if size > 9:
        for sign in (1.0, -1.0):
            q = torch.full((1, 2 * G, D), sign * factor, dtype=torch.bfloat16, device="cuda")
            c.decode(0, ints([0]), q, k[n - 1:], v[n - 1:], out)
            ref, w = rows.attention(0, 0, q, [n - 1], 1 / math.sqrt(D), scales)
            check_out(out, ref, w, f"sign {sign}")
    # Half of the columns give all rows the same large score, one column up to 15 units of 2^-23 of it more: a difference of
    # 2^8 between weights, the most that the maximum does not follow, is one or two such units from size 25 on.
    k = torch.ones(n, 2, D, dtype=torch.bfloat16, device="cuda")
    k[:, :, -1] = (torch.randint(0, 16, (n, 1), generator=gen)).to(k)
    k[:64, :, -1] = 0
    k[64:2000, :, -1].clamp_(max=1)
    c.append(0, ints([0]), ints([0, n]), k, torch.ones_like(k))
    q = torch.zeros(1, 2 * G, D, dtype=torch.bfloat16, device="cuda")
    q[:, :, :D // 2] = factor
    q[:, :, -1] = factor * D * 2.0 ** -24
    c.decode(0, ints([0]), q, k[n - 1:], torch.ones_like(k[:1]), out)
    assert float((out.double() - 1).abs().max()) <= 2.0 ** -8 + 4e-4 + 2.0 ** -8
    assert c.error_flags() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("G,D", [(1, 128), (2, 64), (2, 128), (3, 128), (4, 64), (4, 128)])
def test_decode_small_groups_keep_their_weights(duo, G, D, fp8):
    """Groups of up to four: bf16 weights are held in two parts, which lose 2^-16 at most (two roundings of half a step
    each), so that only the 32-bit errors and the output's rounding are left, cut pairs and whole ones alike. Weights of
    codes are f16: 2^-11."""
    P, Hkv = 32, 2
    lens = [1, 2, 5, 40, 700, 9000]
    c = duo.PagedCache(1, 8, Hkv * G, Hkv, D, 4, 60, P, 400, 300, [1, 0], kv_format=duo.DUO_KV_E4M3 if fp8 else duo.DUO_KV_BF16)
    scales = [[0.5, 1.0], [0.25, 1.0]]
    if fp8:
        c.set_kv_scales(0, *scales)
    from paged_harness import Rows
    rows = Rows(c)
    for s, n in enumerate(lens):
        k, v = normal(n, Hkv, D, seed=10 * s + G), normal(n, Hkv, D, seed=10 * s + G + 5)
        c.extend(ints([s]), ints([n]))
        if n > 1:
            c.append(0, ints([s]), ints([0, n]), k, v)
        rows.rows[s] = (k[None, :n - 1], v[None, :n - 1])
        q = normal(1, Hkv * G, D, seed=s)
        out = torch.full_like(q, float("nan"))
        c.decode(0, ints([s]), q, k[n - 1:], v[n - 1:], out)
        rows.add(s, k[None, n - 1:], v[None, n - 1:])
        ref, w = rows.attention(0, s, q, [n - 1], 1 / math.sqrt(D), scales)
        check_out(out, ref, w, f"{n} tokens", half_p=2.0 ** -11 if fp8 else 2.0 ** -16)
    assert c.error_flags() == 0


@pytest.mark.parametrize("G", [5, 6, 8])
def test_decode_e4m3_weights_lose_no_more_than_f16_does(duo, G):
    """Retrieval heads of codes: f16 weights, half a step of 2^-11."""
    c = duo.PagedCache(1, 8, 2 * G, 2, 128, 4, 60, 64, 400, 300, [1, 1], kv_format=duo.DUO_KV_E4M3)
    scales = [[0.5, 2.0], [0.25, 1.0]]
    c.set_kv_scales(0, *scales)
    from paged_harness import Rows
    rows = Rows(c)
    lens = [3, 130, 5000]
    for s, n in enumerate(lens):
        k, v = normal(n, 2, 128, seed=10 * s + G), normal(n, 2, 128, seed=10 * s + G + 5)
        c.extend(ints([s]), ints([n]))
        c.append(0, ints([s]), ints([0, n]), k, v)
        rows.rows[s] = (k[None], v[None])
    q = normal(3, 2 * G, 128, seed=G)
    out = torch.full_like(q, float("nan"))
    last = [torch.stack([rows.rows[s][i][0, -1] for s in range(3)]) for i in (0, 1)]
    c.decode(0, ints([0, 1, 2]), q, *last, out)
    assert c.error_flags() == 0
    for s, n in enumerate(lens):
        ref, w = rows.attention(0, s, q[s:s + 1], [n - 1], 1 / math.sqrt(128), scales)
        check_out(out[s:s + 1], ref, w, f"{n} tokens", half_p=2.0 ** -11)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_reads_every_tile(duo, fp8):
    """Eight heads ask for one row each out of 20000, another every call: a tile that is read twice, skipped or joined
    wrongly takes a whole output with it."""
    n, D = 20000, 128
    c = duo.PagedCache(1, 4, 8, 1, D, 4, 60, 64, 400, 320, [1], kv_format=duo.DUO_KV_E4M3 if fp8 else duo.DUO_KV_BF16)
    k = torch.where(normal(n, 1, D, seed=1) > 0, 1.0, -1.0).to(torch.bfloat16)
    v = (normal(n, 1, D, seed=2).float().clamp(-3, 3) * 4).round().div(4).to(torch.bfloat16)  # values that E4M3 holds
    c.extend(ints([0]), ints([n]))
    c.append(0, ints([0]), ints([0, n]), k, v)
    out = torch.empty(1, 8, D, dtype=torch.bfloat16, device="cuda")
    tile = 128 if fp8 else 64
    tiles = -(-n // tile)
    for first in range(0, tiles, 8):
        at = [min(min(first + h, tiles - 1) * tile + (first * 5 + h * 11) % tile, n - 1) for h in range(8)]
        q = (4 * k[at, 0]).view(1, 8, D).contiguous()
        c.decode(0, ints([0]), q, k[n - 1:], v[n - 1:], out)
        ref, w = attend(q, k[:, 0], v[:, 0], [n - 1], 4, 60, True, 1 / math.sqrt(D))
        # The asked row scores 4 x 128 / 11.3 = 45, a row by chance 4 standard deviations of 4: it has all the weight.
        assert float((ref[0] - v[at, 0].double()).abs().max()) < 1e-6
        check_out(out, ref, w, f"rows {at}")
    assert c.error_flags() == 0


@pytest.mark.parametrize("scale", [0.01, 0.4])
def test_a_softmax_scale_of_the_callers(duo, scale):
    """Prompts and steps with another scale than 1 / sqrt(head_dim)."""
    c = duo.PagedCache(1, 4, 6, 2, 64, 4, 60, 16, 40, 20, [1, 0], softmax_scale=scale)
    n = 200
    q, k, v = (normal(n + 1, h, 64, seed=h) for h in (6, 2, 2))
    out = torch.full_like(q, float("nan"))
    c.extend(ints([2]), ints([n]))
    c.prefill(0, ints([0, n]), q[:n], k[:n], v[:n], out[:n])
    c.append(0, ints([2]), ints([0, n]), k, v)
    c.extend(ints([2]))
    c.decode(0, ints([2]), q[n:], k[n:], v[n:], out[n:])
    for h in range(2):
        ref, w = attend(q[:, h * 3:h * 3 + 3], k[:, h], v[:, h], list(range(n + 1)), 4, 60, h == 0, scale)
        check_out(out[:, h * 3:h * 3 + 3], ref, w, f"head {h}")
    assert c.error_flags() == 0
