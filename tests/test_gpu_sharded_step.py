"""The operators of a training step together, with the collectives between them."""

import os
import sys

import pytest
import torch

from products_util import U32, half_step

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

SHAPES = [dict(), dict(ranks=2, tokens=33, width=40, experts=5, choices=3, vocabulary=130, score="softmax"),
          dict(ranks=8, tokens=300, width=136, experts=32, choices=4, vocabulary=4096)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_sharded_step(shape, dtype):
    """Twelve operators follow each other on the way to the last gradient. In fp32 each sums at
    most max(width, tokens, vocabulary) products, off by a step of each on the way, and is off
    by less than that many steps times the square root of it, by which the absolute products'
    sum may exceed the sum; in bf16 the roundings of what is stored between them come first: a
    half step of each of twelve tensors and, in the two norms' gradients and the gates', of the
    summands that cancel to a quarter of them."""
    from sharded_step import ShardedStep, tokens_of

    step = ShardedStep(dtype=dtype, **shape)
    n = max(step.width, step.tokens, step.share)
    bound = 12 * U32 * n ** 0.5 * 16 if dtype == "f32" else 12 ** 0.5 * 4 * half_step(torch.bfloat16)
    for seed in range(2):  # the second pass reuses plans and their slots
        x, targets = tokens_of(step, seed)
        loss, ids, grads = step.run(x, targets)
        want, want_grads = step.reference(x, targets, ids)
        assert not bool(loss[targets < 0].any())
        assert float((loss.double() - want).norm()) <= bound * float(want.norm())
        for name, g in want_grads.items():
            got, g = (torch.cat(v) if name == "shards" else v for v in (grads[name], g))
            assert got.shape == g.shape
            assert float((got.double() - g).norm()) <= bound * float(g.norm()), name
