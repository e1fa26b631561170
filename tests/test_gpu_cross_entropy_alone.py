"""One gradient of the cross entropy alone, in no more workspace than it asks for."""

import pytest
import torch

from chunk_schedule_execution_amd import capi, ops
from products_util import TYPES, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,vocabulary,pad", [(3, 64, 50, 0), (9, 33, 700, 1), (300, 264, 1031, 0),
                                                   (300, 260, 1031, 8), (16400, 64, 17000, 0)])
def test_each_gradient_in_its_workspace(rows, k, vocabulary, pad, dtype):
    """The same bits as both together, rows of NaN left out, and nothing behind the workspace is
    written. The last size takes several pieces of the vocabulary."""
    t = TYPES[dtype]
    x = normal(1, rows, k + pad, dtype=t)[:, :k]
    w = normal(2, vocabulary, k + pad, dtype=t, scale=0.2)[:, pad:]
    targets = torch.randint(0, vocabulary, (rows,), generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()
    targets[1::5] = -1
    dloss = normal(4, rows)
    _, lse = ops.linear_cross_entropy(x, w, targets)
    want = ops.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    x[1::5] = float("nan")
    d = capi.ccl_cross_entropy_desc(ops.DTYPES[t], 0, rows, k, vocabulary, -1, x.stride(0), w.stride(0))
    if (x.data_ptr() | w.data_ptr()) % 16:
        d.flags = capi.CCL_LINEAR_UNALIGNED
    stream = torch.cuda.current_stream().cuda_stream
    for gradients, with_dx, with_dw in ((capi.CCL_GRADIENTS, True, True), (capi.CCL_GRADIENT_DX, True, False),
                                        (capi.CCL_GRADIENT_DW, False, True)):
        need = capi.ccl_linear_cross_entropy_workspace(d, gradients)
        space = torch.full((need + 4096,), 0xa5, dtype=torch.uint8, device="cuda:0")
        dx, dw = (torch.full(s, 7.0, dtype=t, device="cuda:0") for s in ((rows, k), (vocabulary, k)))
        capi.ccl_linear_cross_entropy_backward(d, dloss.data_ptr(), x.data_ptr(), w.data_ptr(), targets.data_ptr(),
                                               lse.data_ptr(), dx.data_ptr() if with_dx else 0,
                                               dw.data_ptr() if with_dw else 0, space.data_ptr(), need, stream)
        assert torch.equal(dx, want[0]) if with_dx else bool((dx == 7.0).all())
        assert torch.equal(dw, want[1]) if with_dw else bool((dw == 7.0).all())
        assert bool((space[need:] == 0xa5).all())
