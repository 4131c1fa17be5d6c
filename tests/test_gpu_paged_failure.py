"""The paged kernels' bounded waits, run out without any fault: duo_paged_test_wait_timeout makes one CTA of the next launch
load no K and V tiles. Nothing is left in flight, the waits give up after their second, the launch ends, the error word says
so, everybody else's outputs are right, and a new cache over the same tensors carries on."""
import math
import time

import pytest
import torch

from paged_harness import Model, Rows, attend, check_out, ints, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def duo():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    import mixed_head_kv_b200
    return mixed_head_kv_b200


def flags_within(c, seconds):
    t0 = time.perf_counter()
    f = c.error_flags()
    assert time.perf_counter() - t0 < seconds
    return f


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,G", [(64, 2), (128, 8)])
def test_decode_wait_runs_out(duo, D, G, fp8):
    n, args = 40, (1, 48, 2 * G, 2, D, 4, 60, 32, 600, 20, [1, 0])
    fmt = dict(kv_format=duo.DUO_KV_E4M3 if fp8 else duo.DUO_KV_BF16)
    scales = [[0.5, 1.0], [0.25, 1.0]]
    c = duo.PagedCache(*args, **fmt)
    if fp8:
        c.set_kv_scales(0, *scales)
    model, rows = Model(600, 32, 20, 48), Rows(c)
    lens = [300 + i for i in range(n)]
    assert model.extend(range(n), lens)
    c.extend(ints(range(n)), ints(lens))
    start = [0]
    for x in lens:
        start.append(start[-1] + x)
    k, v = normal(start[-1], 2, D, seed=1), normal(start[-1], 2, D, seed=2)
    c.append(0, ints(range(n)), ints(start), k, v)
    for s in range(n):
        rows.rows[s] = tuple(x[None, start[s]:start[s + 1]] for x in (k, v))
    q, k1, v1 = (normal(n, h, D, seed=3 + h) for h in (2 * G, 2, 2))
    newest = [torch.stack([rows.rows[s][i][0, -1] for s in range(n)]) for i in (0, 1)]  # (the tokens that are there already)
    assert c.error_flags() == 0
    assert duo.duo_paged_test_wait_timeout(c.handle, duo.DUO_TEST_WAIT_DECODE) == duo.DUO_OK
    out = torch.full_like(q, 7.0)
    c.decode(0, ints(range(n)), q, *newest, out)
    assert flags_within(c, 8) == duo.DUO_ERR_BIT_PAGED_WAIT
    assert c.error_flags() == 0

    def check(cache, out, first):
        for s in range(first, n):
            ref, w = rows.attention(0, s, q[s:s + 1], [model.len[s] - 1], 1 / math.sqrt(D), scales)
            check_out(out[s:s + 1], ref, w, f"sequence {s}")

    check(c, out, 3)  # the first CTA's share is within the first sequences
    tensors = {name: getattr(c, name) for name in c._NAMES}
    c.close()
    c = duo.PagedCache(*args, tensors=tensors, **fmt)
    if fp8:
        c.set_kv_scales(0, *scales)
    out = torch.full_like(q, float("nan"))
    c.decode(0, ints(range(n)), q, *newest, out)  # the step once more, then another
    check(c, out, 0)
    assert model.extend(range(n), [1] * n)
    c.extend(ints(range(n)))
    c.decode(0, ints(range(n)), q, k1, v1, out)
    for s in range(n):
        rows.add(s, k1[None, s:s + 1], v1[None, s:s + 1])
    check(c, out, 0)
    rows.check(model, scales)
    assert c.error_flags() == 0


def test_a_shared_page_is_not_written_after_a_wait_ran_out(duo):
    """The CTA that gives up before its first tile still has the new row to store: not into a page that is shared."""
    c = duo.PagedCache(1, 4, 4, 2, 64, 4, 60, 32, 8, 4, [1, 0])
    c.extend(ints([0]), ints([20]))
    k, v = normal(20, 2, 64, seed=1), normal(20, 2, 64, seed=2)
    c.append(0, ints([0]), ints([0, 20]), k, v)
    c.fork(ints([0]), ints([1]))
    held = [t.clone() for t in (c.k_pages, c.v_pages)]
    q, k1, v1 = (normal(1, h, 64, seed=3 + h) for h in (4, 2, 2))
    assert c.error_flags() == 0
    duo.duo_paged_test_wait_timeout(c.handle, duo.DUO_TEST_WAIT_DECODE)
    c.decode(0, ints([0]), q, k1, v1, torch.empty_like(q))
    assert flags_within(c, 8) == duo.DUO_ERR_BIT_PAGED_WAIT | duo.DUO_ERR_BIT_PAGED_SHARED
    for t, h in zip((c.k_pages, c.v_pages), held):
        assert torch.equal(t.view(torch.int16), h.view(torch.int16))


@pytest.mark.parametrize("D,G", [(64, 1), (128, 2)])
def test_prefill_wait_runs_out(duo, D, G):
    c = duo.PagedCache(1, 4, 2 * G, 2, D, 4, 100, 16, 4, 2, [1, 0])
    start = [0, 100, 1100, 1500]
    q, k, v = (normal(1500, h, D, seed=h) for h in (2 * G, 2, 2))
    assert duo.duo_paged_test_wait_timeout(c.handle, duo.DUO_TEST_WAIT_PREFILL) == duo.DUO_OK
    for armed in (True, False):
        out = torch.full_like(q, 7.0)
        c.prefill(0, ints(start), q, k, v, out)
        assert flags_within(c, 8) == (duo.DUO_ERR_BIT_PAGED_WAIT if armed else 0)
        lost = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
        if armed:  # the first item: the longest prompt's last tiles, the retrieval head's queries
            tile = 128 if G == 2 else 256
            lost[100 + 1000 // tile * tile:1100, :G] = True
            assert (out[lost] == 7).all()
        for a, b in zip(start, start[1:]):
            for h in range(2):
                ref, w = attend(q[a:b, h * G:h * G + G], k[a:b, h], v[a:b, h], list(range(b - a)), 4, 100, h == 0, 1 / math.sqrt(D))
                keep = ~lost[a:b, h * G:h * G + G]
                check_out(out[a:b, h * G:h * G + G][keep], ref[keep], w[keep], f"prompt at {a}, head {h}")


def test_hook_arguments(duo):
    c = duo.PagedCache(1, 4, 2, 2, 64, 4, 16, 16, 4, 2, [1, 0])
    assert duo.duo_paged_test_wait_timeout(c.handle, 4) == duo.DUO_ERR_INVALID_ARG
    assert duo.duo_paged_test_wait_timeout(None, 1) == duo.DUO_ERR_INVALID_ARG
    assert duo.duo_paged_test_wait_timeout(c.handle, 3) == duo.DUO_OK
    assert duo.duo_paged_test_wait_timeout(c.handle, 0) == duo.DUO_OK  # disarmed
    q, k, v = (normal(5, h, 64, seed=h) for h in (2, 2, 2))
    c.prefill(0, ints([0, 5]), q, k, v, torch.empty_like(q))
    assert c.error_flags() == 0
