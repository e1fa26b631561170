"""gelu and its slope against 64 bits, relative to the values themselves, far into the tail.

For z < 0 gelu is -|z| T and its slope T - |z| d with T = erfc(|z| / sqrt 2) / 2 and d =
exp(-z^2 / 2) / sqrt(2 pi). In steps u = 2^-24 of fp32, relative: exp's argument has two
roundings and a rounded constant, 3 u z^2 / 2 of exp's value, exp itself 2 u. T has that
error, 2 u of its own approximation, t = 1 / (1 + 0.305 s) off by 4 u, which t Q(t) makes
at most 2.6 times as large, 3 u of the polynomial's evaluation and 2 u of the product: (20 +
1.5 z^2) u in all. d has exp's and 3 u of its products. Then a product with z, a sum and one
rounding to the type. Values below the normal numbers of fp32 count as zero."""

import pytest
import torch

from chunk_schedule_execution_amd import ops
from products_util import TYPES, U32, half_step, within

pytestmark = pytest.mark.gpu

TINY = 64 * 2.0 ** -126


def arguments(dtype):
    z = torch.cat([torch.linspace(-13, 13, 80001), torch.logspace(-6, 1, 2000), -torch.logspace(-6, 1, 2000),
                   torch.zeros(1)])
    return z.to(TYPES[dtype]).to("cuda:0")


def parts(z):
    """T, d and the relative errors of both, in steps."""
    s = z.double().abs()
    tail = 0.5 * torch.special.erfc(s * 0.5 ** 0.5)
    density = torch.exp(-0.5 * s * s) / (2 * torch.pi) ** 0.5
    return s, tail, density, 20 + 1.5 * s * s, 5 + 1.5 * s * s


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gelu_relative_to_itself(dtype, few):
    """Products with 1 hand every argument over as it is, in both kernels."""
    z, one = arguments(dtype), torch.ones(1, 1, dtype=TYPES[dtype], device="cuda:0")
    out = (ops.linear(one, z[:, None], activation="gelu").t() if few else
           ops.linear(z[:, None], one, activation="gelu"))[:, 0]
    s, tail, _, steps, _ = parts(z)
    want = torch.where(z < 0, -s * tail, s - s * tail)
    off = (steps + 1) * U32 * s * tail + U32 * want.abs()
    within(out, want, off + half_step(out.dtype) * (want.abs() + off) + TINY, "gelu")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gelu_slope_relative_to_its_parts(dtype):
    """With weights and an output gradient of 1 the gradient of x is the slope."""
    z, one = arguments(dtype), torch.ones(1, 1, dtype=TYPES[dtype], device="cuda:0")
    (dx,) = ops.linear_backward(torch.ones_like(z)[:, None], z[:, None], one, preact=z[:, None], activation="gelu",
                                need_dw=False)
    s, tail, density, steps, more = parts(z)
    want = torch.where(z < 0, tail - s * density, 1 - tail + s * density)
    off = steps * U32 * tail + (more + 1) * U32 * s * density + 2 * U32 * (want.abs() + (z >= 0))
    within(dx[:, 0], want, off + half_step(dx.dtype) * (want.abs() + off) + TINY, "slope")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gelu_of_very_large_values(dtype):
    inf = float("inf")
    z = torch.tensor([20.0, 1e4, 1e30, inf, -20.0, -1e4, -1e30, -inf], dtype=TYPES[dtype], device="cuda:0")
    one = torch.ones(1, 1, dtype=TYPES[dtype], device="cuda:0")
    out = ops.linear(z[:, None], one, activation="gelu")[:, 0]
    assert torch.equal(out[:4], z[:4]) and bool((out[4:].abs() <= TINY).all())
    (dx,) = ops.linear_backward(torch.ones_like(z)[:, None], z[:, None], one, preact=z[:, None], activation="gelu",
                                need_dw=False)
    assert dx[:3, 0].tolist() == [1, 1, 1] and bool((dx[4:7, 0].abs() <= TINY).all())
