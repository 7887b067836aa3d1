"""Corners of the prompt side's calls that the tests by operator leave out."""
import pytest
import torch

from gpu_helpers import split_tokens
from prompt_helpers import make_pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_17_gb300 as m

    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def good_ranges(ip, rows):
    return [(b, ip[b], ip[b + 1]) for b in range(len(ip) - 1) if 0 <= ip[b] <= ip[b + 1] <= rows]


def test_workspace_without_memory_of_its_own(pkv):
    """The elements of an expanded or strided workspace are not the bytes behind it."""
    n, c, hq, hkv, d = 3, 900, 8, 2, 128
    k, v, _, tables = make_pool([c], hkv, d, False, 7)
    q = torch.randn((n, hq, d), device="cuda").to(torch.bfloat16)
    args = (q, ints([0, n]), k, v, tables, ints([c]), 0.1)
    with split_tokens(128):
        need = pkv.prefill_workspace_size(1, n, hq, hkv, d, tables.shape[1] * 16)
        assert need > 0
        want = pkv.paged_prefill_attention(*args)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        assert torch.equal(pkv.paged_prefill_attention(*args, workspace=ws), want)
        for bad in (ws[:1].expand(need), ws[:256].expand(need // 256 + 1, 256), torch.cat((ws, ws))[::2]):
            with pytest.raises(ValueError, match="contiguous"):
                pkv.paged_prefill_attention(*args, workspace=bad)
        ws.fill_(0xFF)
        assert torch.equal(pkv.paged_prefill_attention(*args, workspace=ws), want)
