"""Refusals of differential attention's C entries that came later, without a GPU."""
from test_diff_abi import cascade, last, pkv  # noqa: F401  (a fixture)
from test_prompt_abi import desc


def test_refusals_of_member_lists(pkv):  # noqa: F811
    d = desc(pkv)
    assert cascade(pkv, d, num_member_seqs=-1) == pkv.PKV_ERR_INVALID_ARG and "num_member_seqs" in last(pkv)
