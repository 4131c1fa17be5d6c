"""A head mask shorter than the layout's heads is refused before the library reads behind it."""
import __graft_entry__

__graft_entry__.build()
import mixed_head_kv_b200 as duo  # noqa: E402


def test_short_masks_are_refused():
    L = duo.make_paged_layout(2, 4, 8, 4, 64, 4, 16, 16, 10, 4)
    assert duo.duo_paged_size(L, [1] * 8)[0] == duo.DUO_OK
    b = duo.duo_paged_buffers()
    for name, _ in b._fields_:
        setattr(b, name, 0x10010)  # refused for its alignment, if the mask is not
    for mask in ([], [1], [1, 0, 0] * 2, [1] * 7):
        assert duo.duo_paged_size(L, mask)[0] == duo.DUO_ERR_INVALID_ARG
        assert duo.duo_paged_alloc(L, mask, b, stream=0) == (duo.DUO_ERR_INVALID_ARG, None)
    assert duo.duo_paged_alloc(L, [1] * 8, b, stream=0)[0] == duo.DUO_ERR_ALIGNMENT
