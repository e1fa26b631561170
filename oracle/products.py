"""The products and the row exchange from their definitions, in 64 bits (torch, any device).

Every function also gives the absolute sums that error bounds are made of: with fp32
accumulation a sum of n products is off by at most (n + 1) 2^-24 times the sum of their
absolute values.
"""

from __future__ import annotations

import math

import torch

#: Largest slope of any activation (gelu's is 1.129).
STEEPEST = 1.13


def act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * torch.sigmoid(z)
    raise ValueError(name)


def slope(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    raise ValueError(name)


def groups(offsets, rows, experts):
    """(begin, end) of every group, read as the entry points read offsets."""
    if offsets is None:
        return [(0, rows)]
    o, out, last = [int(v) for v in offsets], [], 0
    for e in range(experts):
        hi = max(last, min(max(o[e + 1], 0), rows))
        out.append((last, hi))
        last = hi
    return out


def linear(x, w, offsets=None, bias=None, residual=None, activation="none"):
    """(out, preact, sum of absolute products of every preact value)."""
    x = x.double()
    w = w.double() if w.dim() == 3 else w.double()[None]
    b = None if bias is None else bias.double().reshape(w.shape[0], w.shape[1])
    z = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device=x.device)
    big, out = z.clone(), z.clone()
    for e, (lo, hi) in enumerate(groups(offsets, x.shape[0], w.shape[0])):
        z[lo:hi] = torch.mm(x[lo:hi], w[e].t())
        big[lo:hi] = torch.mm(x[lo:hi].abs(), w[e].abs().t())
        if b is not None:
            z[lo:hi] += b[e]
            big[lo:hi] += b[e].abs()
        out[lo:hi] = act(z[lo:hi], activation)
    if residual is not None:
        out = out + residual.double()
    return out, z, big


def linear_backward(dout, x, w, offsets=None, preact=None, activation="none"):
    """((dx, dw, dbias), the sums of absolute products of each)."""
    dout, x = dout.double(), x.double()
    flat = w.dim() == 2
    w = w.double()[None] if flat else w.double()
    dz = dout if activation == "none" else dout * slope(preact.double(), activation)
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    db = torch.zeros(w.shape[:2], dtype=torch.float64, device=x.device)
    bx, bw, bb = dx.clone(), dw.clone(), db.clone()
    for e, (lo, hi) in enumerate(groups(offsets, x.shape[0], w.shape[0])):
        d = dz[lo:hi]
        dx[lo:hi], bx[lo:hi] = torch.mm(d, w[e]), torch.mm(d.abs(), w[e].abs())
        dw[e], bw[e] = torch.mm(d.t(), x[lo:hi]), torch.mm(d.abs().t(), x[lo:hi].abs())
        db[e], bb[e] = d.sum(0), d.abs().sum(0)
    if flat:
        dw, db, bw, bb = dw[0], db[0], bw[0], bb[0]
    return (dx, dw, db), (bx, bw, bb)


def route(ids, experts):
    """(offsets, positions, slots) of a list of lists of ids, as Python lists."""
    flat = [int(v) for row in ids for v in row]
    order = [s for e in range(experts) for s, v in enumerate(flat) if v == e]
    offsets = [0]
    for e in range(experts):
        offsets.append(offsets[-1] + flat.count(e))
    positions = [-1] * len(flat)
    for i, s in enumerate(order):
        positions[s] = i
    return offsets, positions, order + [-1] * (len(flat) - len(order))


def dispatch(x, slots, choices):
    out = torch.zeros(slots.numel(), x.shape[1], dtype=x.dtype, device=x.device)
    used = (slots >= 0) & (slots < slots.numel())
    out[used] = x[slots[used].long() // choices]
    return out


def combine(h, positions, gates=None):
    """(out, the sums of absolute values)."""
    h = h.double()
    out = torch.zeros(positions.shape[0], h.shape[1], dtype=torch.float64, device=h.device)
    big = out.clone()
    for j in range(positions.shape[1]):
        here = (positions[:, j] >= 0) & (positions[:, j] < h.shape[0])
        row = h[positions[here, j].long()]
        if gates is not None:
            row = row * gates[here, j].double()[:, None]
        out[here] += row
        big[here] += row.abs()
    return out, big


def combine_backward(dout, h, positions, slots, gates=None):
    """((dh, dgates), the sums of absolute products of dgates)."""
    dout, h = dout.double(), h.double()
    tokens, choices = positions.shape
    dh = torch.zeros_like(h)
    dg = torch.zeros(tokens * choices, dtype=torch.float64, device=h.device)
    big = dg.clone()
    used = (slots >= 0) & (slots < slots.numel())
    s = slots[used].long()
    g = torch.ones_like(dg) if gates is None else gates.double().reshape(-1)
    dh[used] = dout[s // choices] * g[s][:, None]
    dg[s] = (dout[s // choices] * h[used]).sum(1)
    big[s] = (dout[s // choices] * h[used]).abs().sum(1)
    return (dh, dg.view(tokens, choices)), big.view(tokens, choices)
