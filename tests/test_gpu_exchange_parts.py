"""The gradient of the expert combine, one output at a time through the C entry point."""

import pytest
import torch

from chunk_schedule_execution_amd import capi, ops
from products_util import TYPES, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,choices,width", [(37, 3, 264), (5, 70, 33), (300, 2, 8)])
def test_each_output_alone(tokens, choices, width, dtype):
    t = TYPES[dtype]
    ids = torch.randint(-1, 9, (tokens, choices), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    _, positions, slots = ops.expert_route(ids.to("cuda:0"), 8)
    h, dout = normal(1, tokens * choices, width, dtype=t), normal(2, tokens, width, dtype=t)
    gates = normal(3, tokens, choices)
    whole = ops.expert_combine_backward(dout, h, positions, slots, gates)
    dh, dgates = torch.full_like(h, 7), torch.full_like(gates, 7)

    def call(ph, pdh, pdg):
        capi.ccl_expert_combine_backward(ops.DTYPES[t], dout.data_ptr(), 0, ph, 0, positions.data_ptr(), slots.data_ptr(),
                                         gates.data_ptr(), tokens, choices, width, pdh, 0, pdg,
                                         torch.cuda.current_stream().cuda_stream)

    call(0, dh.data_ptr(), 0)  # h is not read then
    assert torch.equal(dh, whole[0]) and bool((dgates == 7).all())
    dh.fill_(7)
    call(h.data_ptr(), 0, dgates.data_ptr())
    assert torch.equal(dgates, whole[1]) and bool((dh == 7).all())
