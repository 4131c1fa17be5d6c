"""A paged cache that is set up on another stream than the current one."""
import pytest
import torch

from paged_harness import ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def duo():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    import mixed_head_kv_b200
    return mixed_head_kv_b200


@pytest.mark.parametrize("raw", [False, True])
def test_set_up_behind_the_current_stream(duo, raw):
    """The tensors' zeros are still to come on a busy current stream; the cache's stream waits for them."""
    side = torch.cuda.Stream()
    seqs = ints([0, 3])
    torch.cuda.synchronize()
    stream = side.cuda_stream if raw else side
    torch.cuda._sleep(200_000_000)  # some 0.1 s
    c = duo.PagedCache(1, 8, 2, 2, 64, 4, 16, 16, 32, 8, [1, 0], stream=stream)
    c.extend(seqs, stream=stream)
    c.extend(seqs, ints([20, 0]), stream=stream)
    assert c.error_flags(stream) == 0
    torch.cuda.synchronize()
    assert c.seq_len.tolist() == [21, 0, 0, 1, 0, 0, 0, 0] and int(c.page_ref.sum()) == 3
    assert c.error_flags() == 0


def test_set_up_on_the_default_stream_from_another(duo):
    side = torch.cuda.Stream()
    seqs = ints([1])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        c = duo.PagedCache(1, 8, 2, 2, 64, 4, 16, 16, 32, 8, [1, 0], stream=torch.cuda.default_stream())
    c.extend(seqs)
    torch.cuda.synchronize()
    assert int(c.seq_len[1]) == 1 and c.error_flags() == 0
