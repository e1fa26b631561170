"""Every way in which the products are run, against the definitions in 64 bits."""

import pytest
import torch

import products_ways as W
from test_gpu_products import backward_case, grouped_case, linear_case

pytestmark = pytest.mark.gpu


def ragged(rows, experts):
    """Offsets of uneven groups, the second one empty; the last rows belong to none."""
    g = torch.Generator().manual_seed(rows + experts)
    cuts = torch.randint(0, rows + 1, (experts,), generator=g).sort().values.tolist()
    cuts[0] = min(cuts[0], rows // 3)
    if experts > 1:
        cuts[1] = cuts[0]
    cuts[-1] = max(cuts[-1], rows - rows // 16)
    return [0] + cuts


@pytest.mark.parametrize("case", W.CASES, ids=lambda c: "-".join(str(v) for v in c[:5]))
def test_forward(case):
    dtype, rows, k, n, experts = case[:5]
    assert W.info(dtype, rows, k, n, experts)[0] == case[5]
    if experts:
        grouped_case(rows, k, n, ragged(rows, experts), dtype, "silu")
    else:
        linear_case(rows, k, n, dtype, "silu", bias=True, residual=True, save=True)


@pytest.mark.parametrize("case", W.CASES, ids=lambda c: "-".join(str(v) for v in c[:5]))
def test_backward(case):
    dtype, rows, k, n, experts = case[:5]
    assert W.info(dtype, rows, k, n, experts)[1:] == case[6:]
    if experts:
        backward_case(rows, k, n, dtype, "gelu_tanh", offsets=ragged(rows, experts), experts=experts)
    else:
        backward_case(rows, k, n, dtype, "gelu_tanh")
