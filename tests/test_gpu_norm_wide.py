"""Layer norm and its gradients of rows that take the most registers, several to a workgroup."""

import pytest
import torch

from chunk_schedule_execution_amd import ops
from products_util import TYPES, normal
from test_gpu_norm import backward, forward, parameters, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width,pad", [(1030, 8200, 0), (1100, 16383, 0), (1061, 16384, 8), (1033, 12001, 3)])
def test_norm_of_many_wide_rows(rows, width, pad, dtype):
    x, r = rows_of(1, rows, width, dtype, pad), rows_of(3, rows, width, dtype, pad)
    w, b = parameters(width, dtype)
    forward(x, w, b, None)
    out, total, mean, rstd = forward(x, w, b, r)
    backward(total, w, r, normal(7, rows, width, dtype=TYPES[dtype]), mean, rstd)
    got = ops.layer_norm(x, weight=w, bias=b, residual=r, save_stats=True, out=x, total=r)
    assert got[0] is x and got[1] is r
    assert all(torch.equal(p, q) for p, q in zip(got, (out, total, mean, rstd)))
