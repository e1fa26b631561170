"""Numbers that a descriptor's fields do not hold are refused, not cut: no GPU, nothing launched."""

import pytest
import torch

from chunk_schedule_execution_amd import ops
from test_layers_host import fake, i32


@pytest.mark.skipif(torch.cuda.is_available(), reason="on tensors that only say they are on a GPU")
@pytest.mark.parametrize("kw", [dict(groups=(1 << 32) + 1), dict(groups=4, kept_groups=(1 << 32) + 2),
                                dict(groups=4, kept_groups=2, group_best=(1 << 32) + 2), dict(groups=0),
                                dict(groups=4, kept_groups=5), dict(groups=4, kept_groups=0),
                                dict(groups=4, kept_groups=2, group_best=3)])
def test_select_refuses_numbers_past_32_bits(kw):
    with pytest.raises(ValueError, match="groups"):
        ops.expert_select(fake(4, 8), 2, **kw)


@pytest.mark.skipif(torch.cuda.is_available(), reason="on tensors that only say they are on a GPU")
@pytest.mark.parametrize("shard", [1 << 31, 1 << 64, (1 << 64) - 1])
def test_cross_entropy_refuses_shards_past_31_bits(shard):
    with pytest.raises(ValueError, match="shard"):
        ops.linear_cross_entropy(fake(4, 8), fake(6, 8), i32(4), shard=shard)
    with pytest.raises(ValueError, match="shard"):
        ops.linear_cross_entropy_backward(fake(4), fake(4, 8), fake(6, 8), i32(4), fake(4), shard=shard)
