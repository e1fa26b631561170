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


def few_row_workgroups(rows, n, experts, columns):
    return ((rows + 15) // 16 + experts) * ((n + columns - 1) // columns)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_few_row_kernel_has_a_grid_that_holds_it(dtype):
    """A workgroup of 256 threads per tile of 16 rows, one more per group, and per 16 or 32
    columns; a grid's dimension holds fewer than 2^32 threads. Beyond it tiles are taken."""
    few = many = 0
    for experts in (0, 2, 64, 512, 2048, 4096):
        for rows in (1, 16, 8 * max(1, experts)):
            for n in (1, 4096, 65536, 1 << 18, (1 << 20) - 1, 1 << 20):
                d = capi.ccl_linear_desc(W.TYPES[dtype], capi.CCL_ACT_RELU, rows, 8, n, experts, 0)
                i = capi.ccl_linear_info(d, experts > 0, False)[0]
                if i.tile_rows == 16:
                    few += 1
                    assert few_row_workgroups(rows, n, experts, i.tile_columns) * 256 < 1 << 32
                elif experts and few_row_workgroups(rows, n, experts, 32) * 256 >= 1 << 32:
                    many += 1
    assert few and many
