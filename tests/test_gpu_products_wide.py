"""Very many experts with very wide outputs: more tiles of 16 rows than a grid holds."""

import pytest
import torch

from chunk_schedule_execution_amd import ops
from oracle import products as O
from products_util import forward_bounds, normal, within

pytestmark = pytest.mark.gpu


def test_grouped_linear_beyond_the_few_row_grid():
    experts, rows, k, n = 512, 4096, 8, 1 << 20
    torch.cuda.empty_cache()
    x = normal(1, rows, k, dtype=torch.bfloat16)
    w = torch.empty(experts, n, k, dtype=torch.bfloat16, device="cuda:0")
    for e in range(experts):
        w[e] = normal(2 + e, n, k, dtype=torch.bfloat16)
    offsets = torch.arange(experts + 1, dtype=torch.int32, device="cuda:0") * 8
    out = ops.grouped_linear(x, w, offsets)
    for row in (0, 7, 8, 2047, 4095):
        want, z, big = O.linear(x[row:row + 1], w[row // 8])
        within(out[row:row + 1], want, forward_bounds(want, z, big, k, torch.bfloat16)[0], f"row {row}")
    del x, w, out
    torch.cuda.empty_cache()
