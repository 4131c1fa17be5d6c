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
