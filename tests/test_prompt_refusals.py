"""Outputs that overlap inputs, refused before any CUDA call."""
import pytest

from test_prompt_abi import desc, gather, last, prefill


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_17_gb300 as m

    return m


def test_prefill_output_over_queries(pkv):
    bad, d, row = pkv.PKV_ERR_INVALID_ARG, desc(pkv), 8 * 64 * 2
    q = 0x600000
    for stride, out in ((512, q + row), (512, q - row), (512, q + 16), (512, q + 9 * row), (1024, q), (1024, q + 18 * row),
                        (1024, q + row)):
        assert prefill(pkv, d, q=q, stride=stride, out=out) == bad and "overlaps" in last(pkv), (stride, out)
    # in place, behind the last row, before the first: past this check, refused for something else
    for stride, out in ((512, q), (512, q + 10 * row), (512, q - 10 * row), (1024, q + 19 * row)):
        assert prefill(pkv, d, q=q, stride=stride, out=out, scale=float("nan")) == bad and "softmax_scale" in last(pkv)
    assert prefill(pkv, d, q=q, stride=1024, out=q, T=1, scale=float("nan")) == bad and "softmax_scale" in last(pkv)


def test_gather_outputs_over_each_other(pkv):
    d, row = desc(pkv), 2 * 64 * 2
    for dt, size in ((0, row), (1, 2 * row)):
        for off in (0, 16, size, 9 * size, -16, -9 * size):
            assert gather(pkv, d, k=0x600000, v=0x600000 + off, dt=dt) == pkv.PKV_ERR_INVALID_ARG
            assert "overlaps" in last(pkv)
