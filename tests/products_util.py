"""Inputs and error bounds of the product and exchange tests."""

import torch

from oracle import products as O

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
U32 = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def normal(seed, *shape, dtype=torch.float32, scale=1.0, device="cuda:0"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=device) * scale).to(dtype)


def within(got, want, bound, what):
    """|got - want| <= bound everywhere, and not-a-number nowhere."""
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    if bool(bad.any()):
        at = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at {at}: "
                             f"got {float(got[at])}, want {float(want[at])}, bound {float(bound[at])}")


def forward_bounds(out, z, big, k, dtype, residual=None):
    """Of out and preact: the fp32 sum of k products and the bias, the activation function
    (a few fp32 steps of its argument and of 1), the residual's addition, one rounding."""
    sums = (k + 2) * U32 * big
    pre = sums + half_step(dtype) * (z.abs() + sums) + 1e-38
    fn = O.STEEPEST * sums + 16 * U32 * z.abs()
    if residual is not None:
        fn = fn + U32 * (out.abs() + fn)
    return fn + half_step(dtype) * (out.abs() + fn) + 1e-38, pre


def backward_bounds(grads, bigs, lengths, dtype, rounded):
    """Of dx, dw, dbias: dz is off by 24 fp32 steps of |dout| at most times (the slope
    functions; |slope| may be far below its error, so relative to dout: covered by `bigs`
    computed from |dz| plus `slack`) and, for dx and dw, by one rounding to the type."""
    out = []
    for g, big, n, r in zip(grads, bigs, lengths, (rounded, rounded, False)):
        off = (n + 2) * U32 * big + (half_step(dtype) * big if r else 0)
        out.append(off + half_step(dtype) * (g.abs() + off) + 1e-38)
    return out
