"""Error bounds of the tests of the choice of experts, layer norm and the cross entropy."""

import torch

from products_util import U32, half_step


def select_bounds(gates, logits):
    """A gate is a score over a sum of scores: each exponential is off by the rounding of its
    argument (2^-24 of the logits' range) and two steps of the function, the sum by a step per
    addition (at most 16 in a lane and 6 over the lanes) and the quotient by a few."""
    x = logits.double()
    x = torch.where(x.isfinite(), x, torch.zeros_like(x))
    span = (x.amax(1, keepdim=True) - x.amin(1, keepdim=True)).clamp(max=110.0)
    return (40 + 2 * span) * U32 * gates.abs() + 1e-37


def select_backward_bounds(dx, big, logits, dtype, choices):
    x = logits.double()
    x = torch.where(x.isfinite(), x, torch.zeros_like(x))
    span = (x.amax(1, keepdim=True) - x.amin(1, keepdim=True)).clamp(max=110.0)
    off = (60 + choices + 4 * span) * U32 * big
    return off + half_step(dtype) * (dx.abs() + off) + 1e-37


def adds(n):
    """Additions that a value of a row's sum goes through at most: a thread's own, then the
    lanes' and waves'."""
    return 64 + n // 1024 + 24


def norm_bounds(out, h, mean, rstd, weight, bias, dtype):
    """Of out, total, mean and rstd, from the roundings in order: h, the mean (its sum's
    additions), the differences, their squares' sum, the root, the product with the weight."""
    n = h.shape[1]
    m, r = mean[:, None], rstd[:, None]
    off_h = U32 * h.abs()
    off_mean = (adds(n) * U32 * h.abs().mean(1) + 2 * U32 * mean.abs())[:, None]
    d = (h - m).abs()
    off_d = off_h + off_mean + U32 * d
    rel = (adds(n) + 4) * U32 * torch.ones_like(r) + (2 * (d * off_d).mean(1, keepdim=True)
                                                      + (off_d ** 2).mean(1, keepdim=True)) * r * r
    rel = rel + 6 * U32  # of rstd: half of it would do
    w = 1.0 if weight is None else weight.double().abs()
    off = w * r * (off_d + d * rel) + 4 * U32 * (w * r * d + (0.0 if bias is None else bias.double().abs()))
    return (off + half_step(dtype) * (out.abs() + off) + 1e-38, off_h + half_step(dtype) * (h.abs() + off_h) + 1e-38,
            off_mean[:, 0] + 1e-38, rel[:, 0] * rstd + 1e-38)


def norm_backward_bounds(grads, big, columns, rows, n, dtype):
    """dx: its summands, each off by the sums' additions; columns: a workgroup's rows one after
    another, then the workgroups in 16 runs."""
    dx, dw, db = grads
    off = (adds(n) + 12) * U32 * big + 4 * U32 * dx.abs()
    bounds = [off + half_step(dtype) * (dx.abs() + off) + 1e-38]
    for v, c in zip((dw, db), columns):
        off = (rows // 256 + 120) * U32 * c
        bounds.append(off + half_step(dtype) * (v.abs() + off) + 1e-38)
    return bounds


def logits_off(big, k):
    """A logit's error: an fp32 sum of k products."""
    return (k + 2) * U32 * big


def loss_bounds(lse, picked, big, span, k, vocabulary):
    """lse moves by at most the largest error of its row's logits, by its terms' roundings (of
    the exponentials' arguments, `span` wide at most, and of their sum) and its own."""
    off = logits_off(big, k)
    off_lse = off + (vocabulary // 512 + 300 + 3 * span) * U32 + 2 * U32 * lse.abs()
    return off_lse, off * (picked != 0) + 1e-38, off_lse + off + 2 * U32 * (lse - picked).abs()


def loss_backward_bounds(dz, p, d, x, w, lse, k, dtype):
    """dz's error (of its logit, of the exponential, of its rounding to the type), then the two
    products'."""
    x, w = x.double(), w.double()
    z_off = logits_off(torch.mm(x.abs(), w.abs().t()), k)
    rel = torch.expm1(z_off + U32 * (8 + 3 * torch.mm(x, w.t()).sub(lse.double()[:, None]).abs()))
    off = d[:, None] * (p * rel + 2 * U32 * (p + 1))
    off = off + half_step(dtype) * (dz.abs() + off)
    dx, dw = torch.mm(dz, w), torch.mm(dz.t(), x)
    out = []
    for v, a, b, c in ((dx, off, dz, w), (dw, off.t(), dz.t(), x)):
        o = torch.mm(a.contiguous(), c.abs()) + (b.shape[1] + 40) * U32 * torch.mm(b.abs().contiguous(), c.abs())
        out.append(o + half_step(dtype) * (v.abs() + o) + 1e-38)
    return (dx, dw), out
