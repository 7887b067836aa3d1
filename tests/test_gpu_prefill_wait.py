"""Chunk attention whose waits run out: the call returns, the status word says so, and the next call is right.

Two test-only knobs: PKV_TEST_PREFILL_WAIT_TRIES shortens the waits for work and for scores, and
PKV_TEST_PREFILL_POST_DELAY_CYCLES lets the loading warp hold every work back.  With a delay far above the wait
every CTA gives up; with one near it some warps of a CTA see the work and others have given up, and they
have to leave together wherever they meet at a barrier."""
import pytest
import torch

from prompt_helpers import make_pool, offsets
from test_gpu_wait_timeout import env

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_17_gb300 as m

    return m


def job(pkv, lens, ctx, e4m3):
    hq, hkv, d = 8, 2, 64
    k, v, scales, tables = make_pool(ctx, hkv, d, e4m3, 3)
    g = torch.Generator().manual_seed(1)
    q = torch.randn((sum(lens), hq, d), generator=g).to(torch.bfloat16).cuda()
    ip, c = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (offsets(lens), ctx))
    out = torch.empty_like(q)

    def call():
        pkv.paged_prefill_attention(q, ip, k, v, tables, c, 0.125, out, scales=scales, max_context_len=max(ctx))

    pkv.check_device_status()
    call()
    assert pkv.check_device_status() == 0
    return call, out, out.clone()


# a few works a CTA: one tile each (few rows), two tiles each
CASES = [([1] * 400, [150 + i % 300 for i in range(400)]), ([70] * 330, [70 + i % 200 for i in range(330)])]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,ctx", CASES, ids=["narrow", "wide"])
def test_waits_run_out_and_the_next_call_is_right(pkv, lens, ctx, e4m3):
    call, out, want = job(pkv, lens, ctx, e4m3)
    with env(PKV_TEST_PREFILL_WAIT_TRIES=2, PKV_TEST_PREFILL_POST_DELAY_CYCLES=40000000):
        call()
        assert pkv.check_device_status() == pkv.DEVFLAG_WAIT_TIMEOUT
    out.fill_(7.0)
    call()
    assert pkv.check_device_status() == 0
    assert torch.equal(out, want)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,ctx", CASES, ids=["narrow", "wide"])
def test_waits_that_run_out_for_some_warps(pkv, lens, ctx, e4m3):
    call, out, want = job(pkv, lens, ctx, e4m3)
    for tries in (1, 3):
        for delay in (100, 1000, 3000, 10000, 20000, 40000, 100000, 1000000, 4000000):
            out.fill_(7.0)
            with env(PKV_TEST_PREFILL_WAIT_TRIES=tries, PKV_TEST_PREFILL_POST_DELAY_CYCLES=delay):
                call()
            flags = pkv.check_device_status()
            assert flags in (0, pkv.DEVFLAG_WAIT_TIMEOUT)
            if flags == 0:
                assert torch.equal(out, want)
    call()
    assert pkv.check_device_status() == 0
    assert torch.equal(out, want)
