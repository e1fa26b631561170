"""Layer norm's inputs and outputs as rows side by side in one buffer, and what is refused there."""

import pytest
import torch

from chunk_schedule_execution_amd import capi, ops
from products_util import TYPES, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width", [(5, 72), (700, 1001), (3, 20001)])
def test_norm_of_rows_side_by_side(rows, width, dtype):
    """x, residual, out and total are columns of one buffer: the same bits as apart."""
    t = TYPES[dtype]
    buffer = normal(1, rows, 4 * width + 3, dtype=t)
    x, r, out, total = (buffer[:, i * width:(i + 1) * width] for i in (2, 0, 3, 1))
    want = ops.layer_norm(x.clone(), residual=r.clone(), save_stats=True)
    behind = buffer[:, 4 * width:].clone()
    got = ops.layer_norm(x, residual=r, out=out, total=total, save_stats=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(buffer[:, 4 * width:], behind)
    # every other row of the buffer, and the rows between
    x, out = buffer[0::2, :width], buffer[1::2, :width]
    n = min(len(x), len(out))
    want = ops.layer_norm(x[:n].clone())
    assert torch.equal(ops.layer_norm(x[:n], out=out[:n]), want)


def test_norm_refuses_outputs_in_other_rows_of_its_inputs():
    buffer = normal(2, 9, 40)
    x, r = buffer[:8], normal(3, 8, 40)
    before = buffer.clone(), r.clone()
    other = torch.empty_like(r)
    for kw in (dict(out=buffer[1:]), dict(residual=r, total=buffer[1:]), dict(residual=r, out=r, total=r),
               dict(residual=r, out=other, total=other), dict(out=buffer.view(-1)[8:328].view(8, 40)),
               dict(residual=r, out=torch.as_strided(buffer, (8, 40), (42, 1)))):
        with pytest.raises(capi.CCLError, match="memory"):
            ops.layer_norm(x, **kw)
    torch.cuda.synchronize()
    assert torch.equal(buffer, before[0]) and torch.equal(r, before[1])
