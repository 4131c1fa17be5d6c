"""Host-only checks of the paged cache's calls (no GPU): buffer sizes, refused layouts and arguments, the plain page
rules that the GPU tests hold the kernels to."""
import ctypes

import pytest
import torch

import __graft_entry__

__graft_entry__.build()
import mixed_head_kv_b200 as duo  # noqa: E402
from paged_harness import Model  # noqa: E402


def layout(**kw):
    base = dict(num_layers=2, max_seqs=10, num_q_heads=12, num_kv_heads=4, head_dim=128, sink=4, recent=60, page_size=64,
                num_pages=100, max_pages=20)
    base.update(kw)
    return duo.make_paged_layout(**base)


MASK = [1, 0, 0, 1, 0, 0, 0, 1]


def test_sizes():
    st, s = duo.duo_paged_size(layout(), MASK)
    assert st == duo.DUO_OK
    assert s.pages == 100 * 3 * 64 * 128 * 2 and s.windows == 10 * 5 * 64 * 128 * 2
    assert s.page_table == 10 * 20 * 4 and s.seq_len == 40 and s.page_ref == 400
    assert 0 < s.workspace < 8 << 20
    st, s = duo.duo_paged_size(layout(kv_format=duo.DUO_KV_E4M3), MASK)
    assert st == duo.DUO_OK and s.pages == 100 * 3 * 64 * 128


@pytest.mark.parametrize("bad", [
    dict(num_layers=0), dict(max_seqs=0), dict(max_seqs=4097), dict(num_kv_heads=0), dict(num_q_heads=13),
    dict(num_q_heads=36), dict(head_dim=96), dict(sink=-1), dict(recent=0), dict(page_size=8), dict(page_size=48),
    dict(page_size=256), dict(num_pages=0), dict(num_pages=(1 << 20) + 1), dict(max_pages=0), dict(max_pages=1 << 25),
    dict(softmax_scale=-1.0), dict(softmax_scale=float("nan")), dict(kv_format=2)])
def test_bad_layouts(bad):
    L = layout(**bad)
    mask = [0, 1] * (max(L.num_layers, 1) * max(L.num_kv_heads, 1))
    assert duo.duo_paged_size(L, mask)[0] == duo.DUO_ERR_INVALID_ARG


def test_coordinates_that_do_not_fit_are_refused():
    L = layout(num_layers=80, num_kv_heads=128, num_q_heads=128, num_pages=1 << 20)
    assert duo.duo_paged_size(L, [1] * (80 * 128))[0] == duo.DUO_ERR_INVALID_ARG
    assert duo.duo_paged_size(L, [0] * (80 * 128))[0] == duo.DUO_OK
    assert duo.duo_paged_size(layout(), [1, 2] + [0] * 6)[0] == duo.DUO_ERR_INVALID_ARG


def test_alloc_checks_buffers_before_the_device():
    b = duo.duo_paged_buffers()
    assert duo.duo_paged_alloc(layout(), MASK, b, stream=0)[0] == duo.DUO_ERR_INVALID_ARG
    for name, _ in b._fields_:
        setattr(b, name, 0x10000)
    b.page_ref = 0x10010
    assert duo.duo_paged_alloc(layout(), MASK, b, stream=0)[0] == duo.DUO_ERR_ALIGNMENT
    b.page_ref, b.k_pages = 0x10000, None
    assert duo.duo_paged_alloc(layout(), MASK, b, stream=0)[0] == duo.DUO_ERR_INVALID_ARG
    lib = duo._lib
    assert lib.duo_paged_alloc(ctypes.byref(layout()), None, None, None, None) == duo.DUO_ERR_INVALID_ARG
    assert lib.duo_paged_size(ctypes.byref(layout()), ctypes.cast(duo._mask_buf(MASK), ctypes.c_void_p), None) == duo.DUO_ERR_INVALID_ARG


def test_null_cache():
    P = 0x1000
    assert duo.duo_paged_free(None) == duo.DUO_OK
    for st in (duo.duo_paged_extend(None, 1, P, None, stream=0), duo.duo_paged_append(None, 0, 1, P, P, P, P, 4, stream=0),
               duo.duo_paged_prefill(None, 0, 1, P, P, P, P, P, 4, stream=0),
               duo.duo_paged_decode(None, 0, 1, P, P, P, P, P, stream=0), duo.duo_paged_fork(None, 1, P, P, stream=0),
               duo.duo_paged_copy(None, 1, P, P, stream=0), duo.duo_paged_release(None, 1, P, stream=0),
               duo.duo_paged_compact(None, stream=0), duo.duo_paged_error(None, stream=0)[0],
               duo.duo_paged_set_kv_scales(None, 0, [1.0], [1.0], stream=0)):
        assert st == duo.DUO_ERR_INVALID_ARG


def test_class_refuses_before_the_device():
    with pytest.raises(ValueError):
        duo.PagedCache(1, 2, 4, 2, 64, 4, 16, 16, 8, 4, [1], device="cpu")
    with pytest.raises(ValueError):  # a paged cache lives on a CUDA device
        duo.PagedCache(1, 2, 4, 2, 64, 4, 16, 16, 8, 4, [1, 0], device="cpu")
    t = dict(k_pages=torch.zeros(8, 1, 16, 64), v_pages=torch.zeros(8, 1, 16, 64), k_window=torch.zeros(2, 1, 20, 64),
             v_window=torch.zeros(2, 1, 20, 64), page_table=torch.zeros(2, 4), seq_len=torch.zeros(2), page_ref=torch.zeros(8))
    with pytest.raises(ValueError):
        duo.PagedCache(1, 2, 4, 2, 64, 4, 16, 16, 8, 4, [1, 0], tensors=t)
    with pytest.raises(duo.DuoError):
        duo.PagedCache(1, 2, 4, 2, 64, 4, 16, 17, 8, 4, [1, 0], device="cpu")


class _Fake(duo.PagedCache):
    """The class's own argument checks, without a library handle."""

    def __init__(self):
        self.layout = layout()
        self.device = torch.device("cpu")
        self.handle = None
        self._constants()


def test_tensor_checks():
    c = _Fake()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    rows = lambda n, h, d=128, t=torch.bfloat16: torch.zeros(n, h, d, dtype=t)  # noqa: E731
    for bad in (torch.tensor([1]), i32(1, 2)[::2].expand(2), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            c.extend(bad)
    q, k, out = rows(2, 12), rows(2, 4), rows(2, 12)
    for args in ((i32(0), q, k, k, out), (i32(0, 1), rows(2, 11), k, k, out), (i32(0, 1), q, rows(2, 4, 64), k, out),
                 (i32(0, 1), q.float(), k, k, out), (i32(0, 1), q, k, rows(2, 8)[:, ::2], out),
                 (i32(0, 1), q, k, rows(2, 8)[:, :4], out), (i32(0, 1), q, k, k, out[:1]),
                 (i32(0, 1), q.transpose(0, 1).contiguous().transpose(0, 1), k, k, out),
                 (i32(0, 1), q[:1].expand(2, 12, 128), k, k, out), (i32(0, 1), q, k[:1].expand(2, 4, 128), k, out)):
        with pytest.raises(ValueError):
            c.decode(0, *args)
    with pytest.raises(ValueError):
        c.append(0, i32(0, 1), i32(0, 1), k, k)
    with pytest.raises(ValueError):
        c.prefill(0, i32(), q, k, k, out)
    with pytest.raises(ValueError):
        c.prefill(0, i32(0, 2), q, rows(3, 4), rows(3, 4), out)
    with pytest.raises(ValueError):
        c.fork(i32(0), i32(1, 2))
    with pytest.raises(ValueError):
        c.set_kv_scales(0, [1.0], [1.0])


def test_plain_page_rules():
    m = Model(num_pages=6, page=4, max_pages=4, max_seqs=4)
    assert m.extend([0, 1], [5, 4]) and m.pages == {0: [0, 1], 1: [2], 2: [], 3: []}
    m.fork([0], [2])
    assert m.ref == [2, 2, 1, 0, 0, 0]
    assert m.extend([0, 2], [1, 1])  # the first leaves the shared page, the second keeps it
    assert m.pages[0] == [0, 3] and m.pages[2] == [0, 1] and m.ref == [2, 1, 1, 1, 0, 0]
    assert not m.extend([1, 0], [9, 3]) and m.ref == [2, 1, 1, 1, 0, 0] and m.len[1] == 4
    m.release([1])
    m.copy([2], [1])
    assert m.pages[1] == [2, 4]
    m.release([0])
    assert m.ref == [1, 1, 1, 0, 1, 0]
    m.compact()
    assert m.pages[1] == [2, 3] and m.pages[2] == [0, 1] and m.ref == [1, 1, 1, 1, 0, 0]
