"""What is measured of the layer's operators around the products: cases, inputs, plain forms.

Three operators of a step of a model whose weights, experts and vocabulary are spread over
ranks, each with its gradients:

* the choice of experts (what comes before the row exchange and the grouped products):
  softmax or sigmoid scores, a bias that balances the experts' load, groups, top-k, gates;
* layer norm with the residual's addition (what comes between an AllReduce and the next
  product), with the reduction of the weight's and bias's gradients;
* the cross entropy of a product with the vocabulary's matrix, or with a rank's shard of
  it, without keeping the logits.

``own`` False computes the plain forms in elementary torch operations, ``own`` True calls
the package's entry points. ``exact`` computes the definitions in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -------------------------------------------------------------------------
def select_case(op, dtype, tokens, experts, choices, score, bias=False, groups=1, kept=1, best=1, renorm=False,
                scale=1.0, closed=0.0):
    """``kept`` of ``groups`` groups stay, ranked by the sum of their ``best`` highest values;
    ``closed``: share of a token's experts that may not be chosen (logit -inf)."""
    return {"op": op, "dtype": dtype, "tokens": tokens, "experts": experts, "choices": choices, "score": score,
            "bias": bias, "groups": groups, "kept": kept, "best": best, "renorm": renorm, "scale": scale,
            "closed": closed}


def norm_case(op, dtype, rows, width, residual=False, stats=False, weight=True, bias=True, pad=0):
    """``residual``: forward, a second summand, whose sum with x is an output too; backward,
    the gradient that reaches that sum from elsewhere. ``pad``: rows of the inputs lie that
    many elements further apart than their length."""
    return {"op": op, "dtype": dtype, "rows": rows, "width": width, "residual": residual, "stats": stats,
            "weight": weight, "bias": bias, "pad": pad}


def loss_case(op, dtype, rows, k, vocabulary, shards=1, ignored=0.05, pad=0):
    """``vocabulary``: rows of w, one of ``shards`` shards; ``ignored``: share of the rows
    without a target (prompts, padding)."""
    return {"op": op, "dtype": dtype, "rows": rows, "k": k, "vocabulary": vocabulary, "shards": shards,
            "ignored": ignored, "pad": pad}


def listed():
    return [
        # a decoding step of 32 sequences over 64 experts: the smallest call
        dict(select_case("select", "bf16", 32, 64, 4, "softmax", renorm=True), name="select_decode"),
        # a training batch over 256 experts with a balancing bias and groups of experts
        dict(select_case("select", "f32", 16384, 256, 8, "sigmoid", bias=True, groups=8, kept=4, best=2, renorm=True,
                         scale=2.5), name="select_groups"),
        # an odd number of experts, a tenth of them closed to a token
        dict(select_case("select", "bf16", 5003, 61, 3, "softmax", bias=True, closed=0.1), name="select_odd"),
        # the gradient of a training batch's gates: every logit gets one
        dict(select_case("select_backward", "f32", 16384, 256, 8, "softmax"), name="select_backward"),
        # four sequences' next token: latency
        dict(norm_case("norm", "bf16", 4, 4096, residual=True), name="norm_token"),
        # a training batch between two blocks, with the statistics for the backward pass
        dict(norm_case("norm", "bf16", 16384, 4096, residual=True, stats=True), name="norm_large"),
        # its gradients, with the gradient that flows past the norm
        dict(norm_case("norm_backward", "bf16", 16384, 4096, residual=True), name="norm_backward"),
        # 32 bits, no size a multiple of a vector, rows in a wider buffer
        dict(norm_case("norm_backward", "f32", 1111, 1537, pad=3), name="norm_odd_f32"),
        # scoring a few rows over a whole vocabulary: weights bound it
        dict(loss_case("loss", "bf16", 64, 4096, 32768), name="loss_few_rows"),
        # a training batch over a rank's shard of the vocabulary: the largest forward product
        dict(loss_case("loss", "bf16", 8192, 4096, 65536, shards=2), name="loss_large"),
        # both gradients over a whole vocabulary
        dict(loss_case("loss_backward", "bf16", 4096, 4096, 65536), name="loss_backward"),
        # odd sizes, 32 bits, a shard of the vocabulary
        dict(loss_case("loss_backward", "f32", 515, 333, 10007, shards=4, pad=3), name="loss_odd_f32"),
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))

    def width(lo, hi):  # half of the widths are multiples of 64, as layers have them, half are any number
        v = spread(lo, hi)
        return max(64, v // 64 * 64) if rng.random() < 0.5 else v

    op = rng.choice(["select", "select", "select_backward", "norm", "norm_backward", "loss", "loss_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("select"):
        experts = rng.choice([8, 16, 32, 64, 128, 256, spread(2, 512), spread(2, 512)])
        groups = rng.choice([1, 1] + [g for g in range(2, 17) if experts % g == 0])
        kept = rng.randint(1, groups)
        choices = rng.randint(1, min(8, experts // groups * kept))
        return select_case(op, dtype, spread(1, 32768), experts, choices, rng.choice(["softmax", "sigmoid"]),
                           bias=rng.random() < 0.5, groups=groups, kept=kept, best=rng.choice([1, 2]),
                           renorm=choices > 1 and rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                           closed=rng.choice([0.0, 0.0, 0.1, 0.6]))
    if op.startswith("norm"):
        w = width(64, 16384)
        return norm_case(op, dtype, min(spread(1, 16384), (1 << 26) // w), w, residual=rng.random() < 0.5,
                         stats=op == "norm" and rng.random() < 0.5, weight=rng.random() < 0.8,
                         bias=rng.random() < 0.7, pad=rng.choice([0, 0, 8, 5]))
    k, v = width(64, 2048), width(100, 65536 if dtype == "bf16" else 16384)
    rows = min(spread(1, 8192), (1 << (37 if dtype == "bf16" else 33)) // (k * v) + 1)
    return loss_case(op, dtype, rows, k, v, shards=rng.choice([1, 1, 2, 8]), ignored=rng.choice([0.0, 0.05, 0.5]),
                     pad=rng.choice([0, 0, 8, 5]))


# ---- inputs ------------------------------------------------------------------------
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, kind=dtype):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(kind)

    s = dict(case)
    if case["op"].startswith("select"):
        t, e, c = case["tokens"], case["experts"], case["choices"]
        # a token's preferences and the experts' popularity
        logits = (normal(t, e, scale=1.5, kind=torch.float32) + normal(e, scale=0.5, kind=torch.float32)).to(dtype)
        logits[torch.rand(t, e, generator=g, device=dev) < case["closed"]] = -math.inf
        s["logits"] = logits
        s["b"] = normal(e, scale=0.05, kind=torch.float32) if case["bias"] else None
        if case["op"] == "select_backward":
            s["ids"], _ = plain_select(s)  # kept from the forward pass
            s["dgates"] = normal(t, c, kind=torch.float32)
        return s
    if case["op"].startswith("norm"):
        rows, n, pad = case["rows"], case["width"], case["pad"]
        # a stream of rows whose sizes and means differ
        x = (normal(rows, n + pad, kind=torch.float32) * (0.5 + torch.rand(rows, 1, generator=g, device=dev))
             + normal(rows, 1, scale=0.3, kind=torch.float32))
        s["x"] = x.to(dtype)[:, :n]
        s["w"] = (1 + normal(n, scale=0.2, kind=torch.float32)).to(dtype) if case["weight"] else None
        s["b"] = normal(n, scale=0.2) if case["bias"] else None
        s["eps"] = 1e-5
        # the second summand, or the gradient that flows past the norm
        s["r"] = normal(rows, n + pad, scale=0.5)[:, :n] if case["residual"] else None
        if case["op"] == "norm_backward":
            s["dout"] = normal(rows, n + pad)[:, :n]
            s["mean"], s["rstd"] = plain_stats(s["x"].float(), s["eps"])  # kept from the forward pass
        return s
    rows, k, v = case["rows"], case["k"], case["vocabulary"]
    s["x"] = normal(rows, k + case["pad"])[:, :k]
    s["w"] = normal(v, k, scale=2.0 * k ** -0.5)
    total = v * case["shards"]
    s["shard"] = None if case["shards"] == 1 else seed % case["shards"] * v  # of the vocabulary, w's first row
    targets = torch.randint(0, total, (rows,), generator=g, device=dev)
    targets[torch.rand(rows, generator=g, device=dev) < case["ignored"]] = -100
    s["targets"] = targets.to(torch.int32)
    if case["op"] == "loss_backward":
        s["dloss"] = torch.rand(rows, generator=g, device=dev) / rows
        # of the whole vocabulary, kept from the forward pass: shards of similar sums
        s["lse"] = plain_logsumexp(s)[0] + math.log(case["shards"])
    return s


# ---- one pass ----------------------------------------------------------------------
def run(s):
    if own:
        return run_own(s)
    return {"select": plain_select, "select_backward": plain_select_backward, "norm": plain_norm,
            "norm_backward": plain_norm_backward, "loss": plain_loss, "loss_backward": plain_loss_backward}[s["op"]](s)


def run_own(s):
    from chunk_schedule_execution_amd import ops

    op = s["op"]
    if op == "select":
        return ops.expert_select(s["logits"], s["choices"], score=s["score"], bias=s["b"], groups=s["groups"],
                                 kept_groups=s["kept"], group_best=s["best"], renormalise=s["renorm"],
                                 scale=s["scale"])
    if op == "select_backward":
        return ops.expert_select_backward(s["dgates"], s["logits"], s["ids"], score=s["score"],
                                          renormalise=s["renorm"], scale=s["scale"])
    if op == "norm":
        outs = ops.layer_norm(s["x"], weight=s["w"], bias=s["b"], residual=s["r"], eps=s["eps"],
                              save_stats=s["stats"])
        return outs if isinstance(outs, tuple) else [outs]  # out alone: neither a residual nor statistics
    if op == "norm_backward":
        return ops.layer_norm_backward(s["dout"], s["x"], s["mean"], s["rstd"], weight=s["w"], dtotal=s["r"],
                                       bias=s["b"] is not None)
    if op == "loss":
        return ops.linear_cross_entropy(s["x"], s["w"], s["targets"], shard=s["shard"])
    return ops.linear_cross_entropy_backward(s["dloss"], s["x"], s["w"], s["targets"], s["lse"], shard=s["shard"])


# ---- plain forms -------------------------------------------------------------------
def plain_scores(logits, score):
    """In 64 bits: the choice compares them. A logit of -inf scores 0."""
    x = logits.double()
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.max(1, keepdim=True).values
    e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def plain_select(s):
    """ids: the experts of highest value, -1 where none is left; gates: their scores."""
    logits, e = s["logits"], s["experts"]
    t = logits.shape[0]
    none = torch.full((), -math.inf, dtype=torch.float64, device=logits.device)
    scores = plain_scores(logits, s["score"])
    value = scores if s["b"] is None else scores + s["b"].double()
    value = torch.where(logits == -math.inf, none, value)
    if s["groups"] > 1 and s["kept"] < s["groups"]:
        inner = value.view(t, s["groups"], -1)
        best = inner.max(2, keepdim=True).values
        total = best[:, :, 0]
        if s["best"] == 2 and inner.shape[2] > 1:
            at = torch.arange(inner.shape[2], device=logits.device)
            first = torch.where(inner == best, at, at.numel()).min(2, keepdim=True).values
            second = torch.where(at == first, none, inner).max(2).values
            total = total + torch.where(second == -math.inf, torch.zeros_like(second), second)
        kept = torch.zeros_like(total, dtype=torch.bool)
        at = torch.arange(s["groups"], device=logits.device)
        for _ in range(s["kept"]):
            left = torch.where(kept, none, total)
            top = left.max(1, keepdim=True).values
            first = torch.where((left == top) & ~kept, at, at.numel()).min(1, keepdim=True).values
            kept |= at == first
        value = torch.where(kept[:, :, None], inner, none).view(t, e)
    if s["b"] is None:  # the same order, whatever the scores' rounding
        value = torch.where(value == -math.inf, none, logits.double())
    at = torch.arange(e, device=logits.device)
    ids = []
    for _ in range(s["choices"]):
        top = value.max(1, keepdim=True).values
        first = torch.where(value == top, at, e).min(1, keepdim=True).values
        ids.append(torch.where(top == -math.inf, torch.full_like(first, -1), first))
        value = torch.where(at == first, none, value)
    ids = torch.cat(ids, 1)
    gates = torch.where(ids >= 0, scores.gather(1, ids.clamp(min=0)), torch.zeros_like(none))
    if s["renorm"]:
        total = gates.sum(1, keepdim=True)
        gates = gates / torch.where(total == 0, torch.ones_like(total), total)
    return ids.to(torch.int32), (gates * s["scale"]).float()


def plain_select_backward(s):
    logits, ids = s["logits"].float(), s["ids"].long()
    p = plain_scores(s["logits"], s["score"]).float()
    dg = torch.where(ids >= 0, s["dgates"], torch.zeros_like(s["dgates"])) * s["scale"]
    at = ids.clamp(min=0)
    if s["renorm"]:  # gate = score / total of the chosen scores
        chosen = torch.where(ids >= 0, p.gather(1, at), torch.zeros_like(dg))
        total = chosen.sum(1, keepdim=True)
        total = torch.where(total == 0, torch.full_like(total, math.inf), total)
        dg = (dg - (dg * chosen / total).sum(1, keepdim=True)) / total
        dg = torch.where(ids >= 0, dg, torch.zeros_like(dg))
    ds = torch.zeros_like(logits).scatter_add_(1, at, dg)
    if s["score"] == "sigmoid":
        dx = ds * p * (1.0 - p)
    else:
        dx = p * (ds - (p * ds).sum(1, keepdim=True))
    return dx.to(s["logits"].dtype)


def plain_stats(h, eps):
    mean = h.sum(1) / h.shape[1]
    d = h - mean[:, None]
    return mean, 1.0 / torch.sqrt((d * d).sum(1) / h.shape[1] + eps)


def plain_norm(s):
    dtype = s["x"].dtype
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    mean, rstd = plain_stats(h, s["eps"])
    out = (h - mean[:, None]) * rstd[:, None]
    if s["w"] is not None:
        out = out * s["w"].float()
    if s["b"] is not None:
        out = out + s["b"].float()
    outs = [out.to(dtype)]
    if s["r"] is not None:
        outs.append(h.to(dtype))
    if s["stats"]:
        outs += [mean, rstd]
    return outs


def plain_norm_backward(s):
    dtype = s["x"].dtype
    dout, rstd = s["dout"].float(), s["rstd"][:, None]
    xhat = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dout if s["w"] is None else dout * s["w"].float()
    n = xhat.shape[1]
    dx = rstd * (g - g.sum(1, keepdim=True) / n - xhat * ((g * xhat).sum(1, keepdim=True) / n))
    if s["r"] is not None:
        dx = dx + s["r"].float()
    outs = [dx.to(dtype)]
    if s["w"] is not None:
        outs.append((dout * xhat).sum(0).to(dtype))
    if s["b"] is not None:
        outs.append(dout.sum(0).to(dtype))
    return outs


def plain_logsumexp(s):
    """(lse, the logits in 32 bits)."""
    z = s["x"].float() @ s["w"].float().t()
    top = z.max(1, keepdim=True).values
    return (top + torch.log(torch.exp(z - top).sum(1, keepdim=True)))[:, 0], z


def plain_target(s):
    """Column of a row's target in w, and whether it is one."""
    t = s["targets"].long() - (s["shard"] or 0)
    here = (s["targets"] >= 0) & (t >= 0) & (t < s["vocabulary"])
    return torch.where(here, t, torch.zeros_like(t)), here


def plain_loss(s):
    lse, z = plain_logsumexp(s)
    at, here = plain_target(s)
    picked = torch.where(here, z.gather(1, at[:, None])[:, 0], torch.zeros_like(lse))
    if s["shard"] is not None:
        return lse, picked
    return torch.where(here, lse - picked, torch.zeros_like(lse)), lse


def plain_loss_backward(s):
    dtype = s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    at, here = plain_target(s)
    d = torch.where(s["targets"] >= 0, s["dloss"], torch.zeros_like(s["dloss"]))
    dz = torch.exp(x @ w.t() - s["lse"][:, None]) * d[:, None]
    dz.scatter_add_(1, at[:, None], torch.where(here, -d, torch.zeros_like(d))[:, None])
    return [(dz @ w).to(dtype), (dz.t() @ x).to(dtype)]


# ---- what a pass cannot do without ---------------------------------------------------
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("select"):
        t, e, c = case["tokens"], case["experts"], case["choices"]
        logits = size * t * e * (2 if op == "select_backward" else 1)
        return {"bytes": logits + 8 * t * c + (4 * e if case["bias"] and op == "select" else 0), "flops": 4 * t * e}
    if op.startswith("norm"):
        rows, n = case["rows"], case["width"]
        params = int(case["weight"]) + int(case["bias"])
        if op == "norm":  # x and the residual in, out and their sum out
            return {"bytes": size * (rows * n * (4 if case["residual"] else 2) + params * n)
                    + (8 * rows if case["stats"] else 0), "flops": 8 * rows * n}
        # dout, x and the gradient from elsewhere in, dx out; weight in, its and the bias's gradients out
        return {"bytes": size * (rows * n * (4 if case["residual"] else 3) + (params + int(case["weight"])) * n)
                + 8 * rows, "flops": 12 * rows * n}
    rows, k, v = case["rows"], case["k"], case["vocabulary"]
    if op == "loss":
        return {"bytes": size * (rows + v) * k + 12 * rows, "flops": 2 * rows * k * v}
    # the logits are no input: their product is needed again beside the two of the gradients
    return {"bytes": 2 * size * (rows + v) * k + 12 * rows, "flops": 6 * rows * k * v}


# ---- the definitions, in 64 bits ------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"select": exact_select, "select_backward": exact_select_backward, "norm": exact_norm,
            "norm_backward": exact_norm_backward, "loss": exact_loss, "loss_backward": exact_loss_backward}[case["op"]](s)


def exact_score(x, score):
    if score == "sigmoid":
        return torch.sigmoid(x)
    return torch.softmax(x, 1).nan_to_num(0.0)  # a row of -inf: no scores


def exact_select(s):
    x = s["logits"].double()
    t, e = x.shape
    p = exact_score(x, s["score"])
    open_ = ~torch.isneginf(x)
    rank = p + (0.0 if s["b"] is None else s["b"].double())
    rank = rank.masked_fill(~open_, -math.inf)
    per = e // s["groups"]
    if s["kept"] < s["groups"]:
        ordered = rank.view(t, s["groups"], per).sort(2, descending=True).values[:, :, :s["best"]]
        # a group's value: its best open experts'; no open expert, no value
        value = ordered.masked_fill(torch.isneginf(ordered), 0.0).sum(2).masked_fill(torch.isneginf(ordered[:, :, 0]),
                                                                                    -math.inf)
        kept = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :s["kept"]]
        stays = torch.zeros(t, s["groups"], dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        open_ = open_ & stays.repeat_interleave(per, 1)
    order = (x if s["b"] is None else rank).masked_fill(~open_, -math.inf)
    values, ids = torch.sort(order, dim=1, descending=True, stable=True)
    values, ids = values[:, :s["choices"]], ids[:, :s["choices"]]
    gone = torch.isneginf(values)
    gates = p.gather(1, ids).masked_fill(gone, 0.0)
    if s["renorm"]:
        gates = (gates / gates.sum(1, keepdim=True)).nan_to_num(0.0)
    return ids.masked_fill(gone, -1).to(torch.int32), gates * s["scale"]


def exact_select_backward(s):
    """By differentiating the gates."""
    x = s["logits"].double().masked_fill(torch.isneginf(s["logits"]), -1e4).requires_grad_(True)
    p = torch.sigmoid(x) if s["score"] == "sigmoid" else torch.softmax(x, 1)
    used = s["ids"] >= 0
    gates = p.gather(1, s["ids"].long().clamp(min=0)) * used
    if s["renorm"]:
        gates = gates / gates.sum(1, keepdim=True).clamp(min=1e-300)
    (dx,) = torch.autograd.grad((gates * s["scale"] * s["dgates"].double()).sum(), x)
    return dx


def exact_norm(s):
    h = s["x"].double() + (0.0 if s["r"] is None else s["r"].double())
    mean = h.mean(1)
    rstd = (h.var(1, unbiased=False) + s["eps"]) ** -0.5
    out = (h - mean[:, None]) * rstd[:, None]
    out = out * (1.0 if s["w"] is None else s["w"].double()) + (0.0 if s["b"] is None else s["b"].double())
    return [out] + ([h] if s["r"] is not None else []) + ([mean, rstd] if s["stats"] else [])


def exact_norm_backward(s):
    d = s["dout"].double()
    rstd = s["rstd"].double()[:, None]
    xhat = (s["x"].double() - s["mean"].double()[:, None]) * rstd
    g = d * (1.0 if s["w"] is None else s["w"].double())
    dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * rstd
    dx = dx + (0.0 if s["r"] is None else s["r"].double())
    return [dx] + ([(d * xhat).sum(0)] if s["w"] is not None else []) + ([d.sum(0)] if s["b"] is not None else [])


PIECE = 8192  # columns of the vocabulary at a time


def exact_loss(s):
    x, rows = s["x"].double(), s["rows"]
    first = s["shard"] or 0
    lse = torch.full((rows,), -math.inf, dtype=torch.float64, device=x.device)
    picked = torch.zeros_like(lse)
    for lo in range(0, s["vocabulary"], PIECE):
        z = torch.mm(x, s["w"][lo:lo + PIECE].double().t())
        lse = torch.logaddexp(lse, torch.logsumexp(z, 1))
        row = ((s["targets"] >= first + lo) & (s["targets"] < first + lo + z.shape[1])).nonzero()[:, 0]
        picked[row] = z[row, s["targets"][row].long() - first - lo]
    if s["shard"] is not None:
        return lse, picked
    left_out = (s["targets"] < 0) | (s["targets"] >= s["vocabulary"])
    return (lse - picked).masked_fill(left_out, 0.0), lse


def exact_loss_backward(s):
    x = s["x"].double()
    first = s["shard"] or 0
    d = s["dloss"].double().masked_fill(s["targets"] < 0, 0.0)[:, None]
    dx, dw = torch.zeros_like(x), []
    for lo in range(0, s["vocabulary"], PIECE):
        w = s["w"][lo:lo + PIECE].double()
        dz = torch.exp(torch.mm(x, w.t()) - s["lse"].double()[:, None])
        row = ((s["targets"] >= first + lo) & (s["targets"] < first + lo + w.shape[0])).nonzero()[:, 0]
        dz[row, s["targets"][row].long() - first - lo] -= 1.0
        dz *= d
        dx += torch.mm(dz, w)
        dw.append(torch.mm(dz.t(), x))
    return [dx, torch.cat(dw)]
