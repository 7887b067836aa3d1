"""Chunk attention with every count of rows in a warp: the rows of a tile that do not exist part from the others
around the tensor-memory accesses, which are for whole warps.  One row a token (no query group), so that n tokens
are n rows; each form and each way of writing a row."""
import pytest
import torch

from gpu_helpers import split_tokens
from prompt_helpers import attention_64, attention_bounds, make_pool, offsets

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
@pytest.mark.parametrize("split", [None, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("base", [0, 128, 160])  # few rows; the second tile's first warp; its second
def test_every_count_of_rows(pkv, base, d, split, e4m3):
    counts = range(1, 33)
    lens = [base + n for n in counts]
    ctx = [n + 40 + 7 * i for i, n in enumerate(lens)]
    k, v, scales, tables = make_pool(ctx, 2, d, e4m3, d + base)
    g = torch.Generator().manual_seed(base + d)
    q = torch.randn((sum(lens), 2, d), generator=g).to(torch.bfloat16).cuda()
    ip, c = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (offsets(lens), ctx))
    lse = torch.empty(q.shape[:2], device="cuda")
    with split_tokens(split):
        out = pkv.paged_prefill_attention(q, ip, k, v, tables, c, d ** -0.5, lse=lse, scales=scales, max_context_len=max(ctx))
    assert pkv.check_device_status() == 0
    ref, ref_lse, mag, size = attention_64(q, lens, k, v, scales, tables, ctx, d ** -0.5, True)
    bound, lse_bound = attention_bounds(ref, mag, size, q, e4m3, d)
    assert float(((out.double() - ref).abs() - bound).max()) <= 0
    assert float(((lse.double() - ref_lse).abs() - ref_lse.abs() * 2.0 ** -22).max()) <= lse_bound


@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_of_part_of_a_warp_over_a_long_context(pkv, e4m3):
    """131 rows over 65,536 + 300 keys, so that a record is kept between the runs of an accumulator."""
    lens, d, n = [131], 64, 65536 + 300
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn((64, 16, 1, d), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    scales = None
    if e4m3:
        k, v, scales = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn), torch.ones(2, 1, device="cuda")
    q = torch.randn((131, 1, d), generator=g).to(torch.bfloat16).cuda()
    tables = (torch.arange((n + 15) // 16, dtype=torch.int32, device="cuda") % 64).view(1, -1)
    ip, c = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 131], [n]))
    with split_tokens(1 << 22):
        out = pkv.paged_prefill_attention(q, ip, k, v, tables, c, 0.125, causal=False, scales=scales)
    assert pkv.check_device_status() == 0
    ref, _, mag, size = attention_64(q, lens, k, v, scales, tables, [n], 0.125, False)
    bound, _ = attention_bounds(ref, mag, size, q, e4m3, d)
    # the sums of 65,836 weights: 2^-11 of truncation in one accumulator, of the weighted sizes
    assert float(((out.double() - ref).abs() - bound - 2.0 ** -11 * mag).max()) <= 0
