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
