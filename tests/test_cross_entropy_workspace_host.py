"""The workspace of one gradient of the cross entropy alone: what only the other takes is not in
it, and it is what the call asks for. No GPU, nothing launched."""

import pytest

from chunk_schedule_execution_amd import capi

P = 1 << 20
BOTH, DX, DW = capi.CCL_GRADIENTS, capi.CCL_GRADIENT_DX, capi.CCL_GRADIENT_DW


def desc(dtype, rows, k, vocabulary, **kw):
    return capi.ccl_cross_entropy_desc(dtype=dtype, rows=rows, in_features=k, vocabulary=vocabulary, first=-1, **kw)


def query(d, gradients):
    return capi.ccl_linear_cross_entropy_workspace(d, gradients)


@pytest.mark.parametrize("dtype,size", [(capi.CCL_F32, 4), (capi.CCL_BF16, 2)])
@pytest.mark.parametrize("rows,k,vocabulary", [(16, 64, 100), (1000, 4096, 8192), (65536, 4096, 131072)])
def test_dx_alone_takes_no_copy_of_x(rows, k, vocabulary, dtype, size):
    d = desc(dtype, rows, k, vocabulary)
    copy = rows * k * size
    # dw's product may need splits' sums as well, which dx alone does not
    assert query(d, DX) <= query(d, BOTH) - copy
    off = desc(dtype, rows, k, vocabulary, flags=capi.CCL_LINEAR_UNALIGNED)
    assert query(off, DX) >= query(d, DX) + copy + vocabulary * k * size  # copied onto the grid


@pytest.mark.parametrize("dtype,size", [(capi.CCL_F32, 4), (capi.CCL_BF16, 2)])
def test_dw_alone_takes_no_sums_of_dx(dtype, size):
    d = desc(dtype, 65536, 4096, 131072)  # several pieces of the vocabulary
    assert query(d, DW) <= query(d, BOTH) - 65536 * 4096 * 4


@pytest.mark.parametrize("dtype", [capi.CCL_F32, capi.CCL_BF16])
def test_each_gradient_asks_for_its_own(dtype):
    for rows, k, vocabulary in ((3, 33, 50), (300, 264, 1031), (2048, 64, 140000), (32768, 64, 16500)):
        d = desc(dtype, rows, k, vocabulary)
        for gradients, dx, dw in ((BOTH, P, P), (DX, P, 0), (DW, 0, P)):
            need = query(d, gradients)
            assert 0 < need <= query(d, BOTH)
            with pytest.raises(capi.CCLError) as e:
                capi.ccl_linear_cross_entropy_backward(d, P, P, P, P, P, dx, dw, P, need - 1)
            assert e.value.status == capi.CCL_ERR_INVALID_ARGUMENT
            assert f"workspace: {need} bytes needed" in capi.ccl_last_error_detail()
