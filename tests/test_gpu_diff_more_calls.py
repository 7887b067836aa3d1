"""More ways of calling differential attention: member lists shorter than their ranges say."""
import pytest
import torch

from test_gpu_diff import D, Job, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_17_gb300 as m

    return m


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_range_past_the_member_list(pkv, e4m3):
    """A range of members within the batch but past the list's end is flagged and read no further than the list; the others
    are served.  (The list is the front of a longer tensor, whose rest names other sequences.)"""
    prefixes, tails = [64, 32], [5, 9, 300, 17, 0, 40]
    j = Job(6, prefixes + tails, 8, 2, e4m3, 3)
    front, own, c = j.tables[:2].contiguous(), j.tables[2:].contiguous(), ints(tails)
    longer = ints([4, 0, 5, 2, 1, 3])

    def call(ip, of, n):
        out = torch.full((6, 4, 2 * D), 7.0, dtype=torch.float32, device="cuda")
        pkv.cascade_diff_decode_attention(j.q, j.k, j.v, front, ints(prefixes), ints(ip), longer[:n], ints(of), own, c, 0.125,
                                          j.lam, out, max_members=3, **j.keys())
        return out, pkv.check_device_status()

    of = [0, -1, 1, -1, 0, 1]
    want, flags = call([0, 2, 4], of, 4)
    assert flags == 0
    got, flags = call([0, 2, 4], of, 3)
    assert flags == pkv.DEVFLAG_BAD_INDPTR
    assert torch.equal(got[[0, 1, 3, 4]], want[[0, 1, 3, 4]])
    got, flags = call([0, 2, 5], of, 4)
    assert flags == pkv.DEVFLAG_BAD_INDPTR
    assert torch.equal(got[[0, 1, 3, 4]], want[[0, 1, 3, 4]])
    again, flags = call([0, 2, 4], of, 4)
    assert flags == 0 and torch.equal(again, want)
