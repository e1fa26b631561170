"""The expert-parallel example: products, row exchange and the collectives between them."""

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [dict(), dict(ranks=2, tokens=5, choices=3, experts=4, width=64, hidden=40),
                                   dict(ranks=8, tokens=33, choices=2, experts=32, width=128, hidden=96)])
def test_expert_layer(shape):
    """Seven roundings to bf16 follow each other (dispatch and the AllToAlls copy): the two
    products, the gated sum, the projection's partial products, and the ring's partial sums,
    one per rank. Each is off by half a step, 2^-8, relative to values of the result's size
    or, for the partial products and sums, sqrt(ranks) below it; independent roundings of
    uniform size add up to less than 2^-8 sqrt(7) of the result's norm."""
    from expert_layer import ExpertLayer

    layer = ExpertLayer(**shape)
    g = torch.Generator(device="cuda:0")
    g.manual_seed(2)
    for _ in range(2):  # the second pass reuses plans and their slots
        xs = [torch.randn(layer.tokens, layer.width, generator=g, device="cuda:0").to(torch.bfloat16)
              for _ in range(layer.ranks)]
        outs, routes = layer.forward(xs)
        want = layer.reference(xs, routes)
        for out in outs:
            assert torch.equal(out, outs[0])
            assert float((out.double() - want).norm()) <= 2.0 ** -8 * 7 ** 0.5 * float(want.norm())
