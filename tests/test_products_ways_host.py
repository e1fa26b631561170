"""How the library runs the products: the sizes of ``products_ways`` still take the kernels
that they are there for, and together take all of them. No GPU."""

import pytest

import products_ways as W
from chunk_schedule_execution_amd import capi


@pytest.mark.parametrize("case", W.CASES, ids=lambda c: "-".join(str(v) for v in c[:5]))
def test_case_takes_its_kernels(case):
    assert W.info(*case[:5]) == case[5:]


def test_the_cases_take_every_kernel():
    covered = set().union(*(W.ways(c[0], c[2], c[4], c[5:]) for c in W.CASES))
    assert not W.every_way() - covered


def test_info_refuses_what_the_calls_refuse():
    for bad in (dict(dtype=9), dict(rows=-1), dict(in_features=0), dict(experts=-1), dict(flags=2)):
        d = capi.ccl_linear_desc(**dict(dict(dtype=capi.CCL_F32, rows=8, in_features=8, out_features=8), **bad))
        for backward in (False, True):
            with pytest.raises(capi.CCLError):
                capi.ccl_linear_info(d, False, backward)
    d = capi.ccl_linear_desc(capi.CCL_F32, 0, 8, 8, 8)
    assert capi.lib().ccl_linear_info(d, 0, 0, None) == capi.CCL_ERR_INVALID_ARGUMENT
    assert capi.lib().ccl_linear_info(None, 0, 0, None) == capi.CCL_ERR_INVALID_ARGUMENT


def test_info_follows_the_alignment():
    """Off the 16-byte grid, by a base pointer or a stride, tiles need copies and the kernel
    for few rows reads the matrices as they are."""
    for rows, copies in ((8, 0), (300, 2)):
        for off in (dict(flags=capi.CCL_LINEAR_UNALIGNED), dict(ld_x=1025, ld_w=1025)):
            d = capi.ccl_linear_desc(dtype=capi.CCL_BF16, rows=rows, in_features=1024, out_features=512, **off)
            assert capi.ccl_linear_info(d, False, False)[0].copies == copies
        d = capi.ccl_linear_desc(dtype=capi.CCL_BF16, rows=rows, in_features=1024, out_features=512)
        assert capi.ccl_linear_info(d, False, False)[0].copies == 0
