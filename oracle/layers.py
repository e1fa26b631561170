"""The choice of experts, layer norm and the vocabulary's cross entropy from their
definitions, in 64 bits (torch, any device), with the sums of absolute values that error
bounds are made of."""

from __future__ import annotations

import math

import torch

INF = math.inf


# ---- the choice of experts ----------------------------------------------------------
def scores(x, score):
    """Softmax of the rows (zeros for a row of -inf) or sigmoids."""
    if score == "sigmoid":
        return torch.sigmoid(x)
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(top == -INF, torch.zeros_like(top), top))
    return e / e.sum(1, keepdim=True).clamp(min=1.0)  # the largest term is 1, unless there is none


def select(logits, choices, score="softmax", bias=None, groups=1, kept_groups=None, group_best=1, renormalise=False,
           scale=1.0):
    """(ids, gates), token by token as the words say it."""
    x = logits.double()
    p = scores(x, score).tolist()
    raw = x.tolist()
    b = None if bias is None else bias.double().tolist()
    experts = x.shape[1]
    per = experts // groups
    all_ids, all_gates = [], []
    for row, prob in zip(raw, p):
        closed = [v == -INF or (b is not None and b[e] == -INF) for e, v in enumerate(row)]

        def rank(v):
            return INF if math.isnan(v) else v

        value = [rank(prob[e] + (b[e] if b else 0.0)) for e in range(experts)]
        order = value if b else [rank(v) for v in row]
        open_ = [e for e in range(experts) if not closed[e]]
        if kept_groups is not None and kept_groups < groups:
            total = []
            for g in range(groups):
                best = sorted((value[e] for e in open_ if e // per == g), reverse=True)[:group_best]
                total.append(sum(best) if best else -INF)
            kept = sorted(range(groups), key=lambda g: (-total[g], g))[:kept_groups]
            open_ = [e for e in open_ if e // per in kept]
        ids = sorted(open_, key=lambda e: (-order[e], e))[:choices]
        gates = [prob[e] for e in ids]
        if renormalise and ids:
            # ratios of scores; sigmoids of far negative logits in logarithms
            logs = torch.nn.functional.logsigmoid if score == "sigmoid" else (lambda v: v)
            gates = torch.softmax(logs(torch.tensor([row[e] for e in ids], dtype=torch.float64)), 0).tolist()
        pad = choices - len(ids)
        all_ids.append(ids + [-1] * pad)
        all_gates.append([scale * g for g in gates] + [0.0] * pad)
    return (torch.tensor(all_ids, dtype=torch.int32, device=x.device).view(x.shape[0], choices),
            torch.tensor(all_gates, dtype=torch.float64, device=x.device).view(x.shape[0], choices))


def gates_of(x, ids, score="softmax", renormalise=False, scale=1.0):
    """The gates of given ids as a differentiable function of 64-bit logits."""
    used = (ids >= 0) & (ids < x.shape[1])
    at = torch.where(used, ids, torch.zeros_like(ids)).long()
    none = torch.full_like(x[:, :1], -INF)
    if renormalise:
        logs = torch.nn.functional.logsigmoid(x) if score == "sigmoid" else x
        picked = torch.where(used, logs.gather(1, at), none)
        top = picked.detach().amax(1, keepdim=True)
        e = torch.where(used, torch.exp(picked - torch.where(top == -INF, torch.zeros_like(top), top)), 0.0)
        return scale * e / e.sum(1, keepdim=True).clamp(min=0.5)
    p = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)
    return scale * torch.where(used, p.gather(1, at), torch.zeros_like(none))


def select_backward(dgates, logits, ids, score="softmax", renormalise=False, scale=1.0):
    """(dlogits, the absolute sums that make them up), from the formulas."""
    x = logits.double()
    used = (ids >= 0) & (ids < x.shape[1])
    at = torch.where(used, ids, torch.zeros_like(ids)).long()
    d = torch.where(used, dgates.double(), 0.0) * scale
    zero = torch.zeros_like(x)

    def spread(v):
        return zero.scatter_add(1, at, torch.where(used, v, 0.0))

    if renormalise:
        g = gates_of(x, ids, score, True, 1.0)
        flow = (g * d).sum(1, keepdim=True)
        big = (g * d.abs()).sum(1, keepdim=True)
        tail = torch.sigmoid(-x).gather(1, at) if score == "sigmoid" else 1.0
        return spread(g * (d - flow) * tail), spread(g * (d.abs() + big) * tail)
    p = scores(x, score)
    if score == "sigmoid":
        slope = p * torch.sigmoid(-x)
        return spread(d) * slope, spread(d.abs()) * slope
    ds, da = spread(d), spread(d.abs())
    return p * (ds - (p * ds).sum(1, keepdim=True)), p * (da + (p * da).sum(1, keepdim=True))


# ---- layer norm ---------------------------------------------------------------------------
def layer_norm(x, weight=None, bias=None, residual=None, eps=1e-5):
    """(out, total, mean, rstd)."""
    h = x.double() + (0.0 if residual is None else residual.double())
    mean = h.mean(1)
    rstd = 1.0 / torch.sqrt(((h - mean[:, None]) ** 2).mean(1) + eps)
    out = (h - mean[:, None]) * rstd[:, None]
    out = out * (1.0 if weight is None else weight.double()) + (0.0 if bias is None else bias.double())
    return out, h, mean, rstd


def layer_norm_backward(dout, x, mean, rstd, weight=None, dtotal=None):
    """((dx, dweight, dbias), dx's absolute summands, the columns' absolute sums)."""
    d, r = dout.double(), rstd.double()[:, None]
    y = (x.double() - mean.double()[:, None]) * r
    g = d * (1.0 if weight is None else weight.double())
    a, c = g.mean(1, keepdim=True), (g * y).mean(1, keepdim=True)
    dx = r * (g - a - y * c) + (0.0 if dtotal is None else dtotal.double())
    big = r * (g.abs() + g.abs().mean(1, keepdim=True) + y.abs() * (g * y).abs().mean(1, keepdim=True))
    return (dx, (d * y).sum(0), d.sum(0)), big, ((d * y).abs().sum(0), d.abs().sum(0))


# ---- cross entropy -------------------------------------------------------------------------
def column(targets, first, vocabulary):
    """(column of the target, whether it is one of w's rows)."""
    at = targets.long() - first
    here = (targets >= 0) & (at >= 0) & (at < vocabulary)
    return torch.where(here, at, torch.zeros_like(at)), here


def left_out(targets, shard, vocabulary):
    return (targets < 0) | ((targets >= vocabulary) if shard is None else torch.zeros_like(targets, dtype=torch.bool))


def cross_entropy(x, w, targets, shard=None):
    """(loss, lse, picked, the largest absolute sum of a row's logits)."""
    x, w = x.double(), w.double()
    z = torch.mm(x, w.t())
    lse = torch.logsumexp(z, 1)
    at, here = column(targets, shard or 0, w.shape[0])
    picked = torch.where(here, z.gather(1, at[:, None])[:, 0], torch.zeros_like(lse))
    loss = torch.where(left_out(targets, shard, w.shape[0]), torch.zeros_like(lse), lse - picked)
    return loss, lse, picked, torch.mm(x.abs(), w.abs().t()).amax(1)


def logits_gradient(dloss, x, w, targets, lse, shard=None):
    """(dz, p, |dloss| of the rows that are not left out)."""
    z = torch.mm(x.double(), w.double().t())
    at, here = column(targets, shard or 0, w.shape[0])
    d = torch.where(left_out(targets, shard, w.shape[0]), torch.zeros_like(dloss), dloss).double()
    p = torch.exp(z - lse.double()[:, None])
    hot = torch.zeros_like(z).scatter_(1, at[:, None], here[:, None].double())
    return d[:, None] * (p - hot), p, d.abs()
