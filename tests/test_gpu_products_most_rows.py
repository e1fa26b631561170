"""The products at the most rows a call takes, 2^31 - 1: row and step counts that end past
31 bits when rounded up to tiles and steps."""

import pytest
import torch

from chunk_schedule_execution_amd import ops
from oracle import products as O
from products_util import TYPES, backward_bounds, forward_bounds, normal, within

pytestmark = pytest.mark.gpu

ROWS = 2**31 - 1
#: rows with values, all others are zeros: both ends, the last tile and step of every size,
#: and those before them
PICK = [0, 1, 100, 1 << 30, ROWS - 300, ROWS - 256, ROWS - 129, ROWS - 127, ROWS - 65, ROWS - 64, ROWS - 63, ROWS - 33,
        ROWS - 31, ROWS - 12, ROWS - 2, ROWS - 1]


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()  # 34 GB per matrix go back


def matrix(seed, width, t):
    x = torch.zeros(ROWS, width, dtype=t, device="cuda:0")
    x[PICK] = normal(seed, len(PICK), width, dtype=t)
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_and_gradients(dtype):
    t = TYPES[dtype]
    width = 8 if dtype == "bf16" else 4
    x, w, b = matrix(1, width, t), normal(2, width, width, dtype=t), normal(3, width, dtype=t)
    out = ops.linear(x, w, bias=b)
    want, z, big = O.linear(x[PICK], w, bias=b)
    within(out[PICK], want, forward_bounds(want, z, big, width, t)[0], "out")
    assert bool((out[2:100] == b).all()) and bool((out[ROWS - 11:ROWS - 2] == b).all())
    del out
    dout = matrix(4, width, t)
    dx, dw, db = ops.linear_backward(dout, x, w, bias=True)
    grads, bigs = O.linear_backward(dout[PICK], x[PICK], w)
    # every other row adds zeros, which are exact
    bx, bw, bb = backward_bounds(grads, bigs, (width, len(PICK), len(PICK)), t, False)
    within(dx[PICK], grads[0], bx, "dx")
    within(dw, grads[1], bw, "dw")
    within(db, grads[2], bb, "dbias")
    assert not bool(dx[2:100].any()) and not bool(dx[ROWS - 11:ROWS - 2].any())


def test_groups_that_start_inside_the_last_tile():
    t, offsets = torch.bfloat16, [0, 101, ROWS - 40, ROWS - 12, ROWS - 1]  # the last row belongs to no group
    o = torch.tensor(offsets, dtype=torch.int32, device="cuda:0")
    x, w = matrix(1, 8, t), normal(2, 4, 8, 8, dtype=t)
    held = [sum(p < e for p in PICK) for e in offsets]  # the groups of the picked rows
    out = ops.grouped_linear(x, w, o)
    want, z, big = O.linear(x[PICK], w, held)
    within(out[PICK], want, forward_bounds(want, z, big, 8, t)[0], "out")
    assert not bool(out[2:100].any()) and not bool(out[ROWS - 11:ROWS - 2].any()) and not bool(out[ROWS - 1].any())
    del out
    dout = matrix(3, 8, t)
    (dx,) = ops.grouped_linear_backward(dout, x, w, o, need_dw=False)
    grads, bigs = O.linear_backward(dout[PICK], x[PICK], w, held)
    within(dx[PICK], grads[0], backward_bounds(grads, bigs, (8, 1, 1), t, False)[0], "dx")
    assert not bool(dx[2:100].any()) and not bool(dx[ROWS - 11:ROWS - 2].any()) and not bool(dx[ROWS - 1].any())
