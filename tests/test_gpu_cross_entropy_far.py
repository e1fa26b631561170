"""Logits whose product with log2(e) is past fp32's range: sums and gradients stay the logits'."""

import pytest
import torch

from chunk_schedule_execution_amd import ops
from products_util import TYPES, normal

pytestmark = pytest.mark.gpu

# rows, in, vocabulary: tiles of 64, 128 and (bf16) 256, and logits that go through memory
SIZES = [(64, 64, 130), (700, 72, 3100), (2100, 512, 6200), (3, 40, 90)]


def far(rows, k, vocabulary, dtype, logits):
    """x and w whose logits are `logits` (vocabulary,) in every row, to the bit."""
    x = torch.zeros(rows, k, dtype=TYPES[dtype], device="cuda:0")
    w = normal(3, vocabulary, k, dtype=TYPES[dtype])
    x[:, 0] = 1.0
    w[:, 0] = logits.to(TYPES[dtype])
    return x, w


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,vocabulary", SIZES)
@pytest.mark.parametrize("kind", ["lowest", "highest", "highest at one", "lowest but one"])
def test_cross_entropy_of_far_logits(rows, k, vocabulary, kind, dtype):
    t = TYPES[dtype]
    lowest, highest = torch.finfo(t).min, torch.finfo(t).max
    logits = torch.full((vocabulary,), lowest if "lowest" in kind else highest, device="cuda:0")
    special = vocabulary - 3
    if kind == "highest at one":
        logits[:] = 1.0
        logits[special] = highest
    if kind == "lowest but one":
        logits[special] = 2.0
    x, w = far(rows, k, vocabulary, dtype, logits)
    targets = torch.full((rows,), special, dtype=torch.int32, device="cuda:0")
    targets[::3] = 1
    loss, lse = ops.linear_cross_entropy(x, w, targets)
    # the logarithm of how many are highest is far below half a step of such a sum
    want = torch.logsumexp(logits.double(), 0).float()
    assert bool((lse == want).all())
    at = logits.to(t).float()[targets.long()]
    assert torch.equal(loss, lse - at)
    # with lse as it is held, exp(z - lse) is 1 at the highest logits and 0 elsewhere
    p = torch.exp(logits.to(t).double() - lse[0].double())
    assert bool(((p == 0.0) | (p == 1.0)).all())
    dloss = torch.full((rows,), 0.5, device="cuda:0")
    (dw,) = ops.linear_cross_entropy_backward(dloss, x, w, targets, lse, need_dx=False)
    count = torch.bincount(targets.long(), minlength=vocabulary).double()
    assert torch.equal(dw[:, 0].double(), (0.5 * (rows * p - count)).to(t).double())
    assert not bool(dw[:, 1:].any())
