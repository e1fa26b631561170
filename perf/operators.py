"""What is measured of the products beside the collectives: cases, inputs, plain forms.

Three operators of a layer whose weights or experts are spread over ranks:

* the product with bias, activation and residual in its epilogue (the shard of a tensor-
  parallel layer, between an AllGather and an AllReduce), forward and backward;
* products grouped by expert with ragged sizes (what an expert-parallel rank computes
  between its two AllToAlls), forward and backward;
* the expert exchange: rows brought into the experts' order and summed back with their
  gates (what packs and unpacks an AllToAll), forward and backward.

``own`` False computes the plain forms in elementary torch operations, ``own`` True calls
the package's entry points. ``exact`` computes the definitions in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ---- cases -------------------------------------------------------------------------
def linear_case(op, dtype, rows, k, n, act, bias=False, residual=False, save=False, pad=0):
    """out = act(x w^T + bias) + residual; ``save``: the pre-activation is an output too;
    ``pad``: x's rows lie that many elements further apart than their length."""
    return {"op": op, "dtype": dtype, "rows": rows, "k": k, "n": n, "act": act, "bias": bias, "residual": residual,
            "save": save, "pad": pad}


def grouped_case(op, dtype, rows, experts, k, n, act, bias=False, save=False, skew=0.0):
    """``skew``: spread of the experts' popularity (standard deviation of their logits)."""
    return {"op": op, "dtype": dtype, "rows": rows, "experts": experts, "k": k, "n": n, "act": act, "bias": bias,
            "save": save, "skew": skew}


def exchange_case(op, dtype, tokens, choices, experts, width, away=0.0):
    """``away``: share of the choices that another rank's experts serve (id -1 here)."""
    return {"op": op, "dtype": dtype, "tokens": tokens, "choices": choices, "experts": experts, "width": width,
            "away": away}


def listed():
    return [
        # four sequences' next token through a small output projection: the smallest call
        dict(linear_case("linear", "bf16", 4, 1024, 1024, "none", bias=True, residual=True), name="linear_token"),
        # a serving batch of 32 single tokens through one rank's widening layer: weights bound it
        dict(linear_case("linear", "bf16", 32, 4096, 16384, "gelu_tanh", bias=True), name="linear_decode"),
        # no size a multiple of a vector or a tile, rows in a wider buffer
        dict(linear_case("linear", "bf16", 1111, 1001, 1537, "silu", bias=True, residual=True, pad=3),
             name="linear_odd"),
        # the widening layer over a long batch: the largest product
        dict(linear_case("linear", "bf16", 16384, 4096, 16384, "gelu", bias=True, save=True), name="linear_large"),
        # 32-bit training of a small layer
        dict(linear_case("linear", "f32", 2048, 1024, 4096, "relu", bias=True), name="linear_f32"),
        # both gradients of a square layer
        dict(linear_case("linear_backward", "bf16", 8192, 4096, 4096, "gelu", bias=True), name="linear_backward"),
        # a decoding step over 64 experts: most get a row or none
        dict(grouped_case("grouped", "bf16", 64, 64, 2048, 1024, "silu", skew=0.5), name="grouped_decode"),
        # a training batch over 32 experts of uneven popularity
        dict(grouped_case("grouped", "bf16", 16384, 32, 2048, 4096, "silu", save=True, skew=0.3),
             name="grouped_ragged"),
        # its gradients over 16 experts
        dict(grouped_case("grouped_backward", "bf16", 8192, 16, 2048, 2048, "gelu", bias=True, skew=0.3),
             name="grouped_backward"),
        # odd sizes, 32 bits, few experts of very uneven popularity
        dict(grouped_case("grouped_backward", "f32", 1500, 7, 333, 515, "relu", bias=True, skew=1.0),
             name="grouped_odd_f32"),
        # a decoding step's rows to the experts and back, a quarter of them served elsewhere
        dict(exchange_case("exchange", "bf16", 48, 4, 64, 2048, away=0.25), name="exchange_decode"),
        # the gradients of a training batch's exchange
        dict(exchange_case("exchange_backward", "bf16", 16384, 4, 64, 4096), name="exchange_backward"),
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))

    def width(lo, hi):  # half of the widths are multiples of 64, as layers have them, half are any number
        v = spread(lo, hi)
        return max(64, v // 64 * 64) if rng.random() < 0.5 else v

    op = rng.choice(["linear", "linear", "linear_backward", "grouped", "grouped", "grouped_backward", "exchange",
                     "exchange_backward"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op.startswith("exchange"):
        experts = spread(2, 128)
        choices = rng.randint(1, min(8, experts))
        return exchange_case(op, dtype, spread(1, 16384), choices, experts, width(64, 2048 if dtype == "f32" else 4096),
                             away=rng.choice([0.0, 0.0, 0.25, 0.75]))
    backward = op.endswith("backward")
    bias = rng.random() < 0.5
    act = rng.choice(ACTIVATIONS)
    if op.startswith("linear"):
        return linear_case(op, dtype, spread(1, 8192), width(64, 4096), width(64, 4096 if backward else 8192), act,
                           bias=bias, residual=not backward and rng.random() < 0.5,
                           save=not backward and rng.random() < 0.3, pad=rng.choice([0, 0, 8, 5]))
    return grouped_case(op, dtype, spread(1, 8192), spread(1, 64), width(64, 2048), width(64, 2048), act, bias=bias,
                        save=not backward and rng.random() < 0.3, skew=rng.choice([0.0, 0.3, 1.0]))


# ---- inputs ------------------------------------------------------------------------
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, kind=dtype):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(kind)

    s = dict(case)
    if case["op"].startswith("exchange"):
        t, c, e, w = case["tokens"], case["choices"], case["experts"], case["width"]
        # each token's `choices` different experts, in the order of their scores
        ids = torch.rand(t, e, generator=g, device=dev).topk(c, dim=1).indices.to(torch.int32)
        ids[torch.rand(t, c, generator=g, device=dev) < case["away"]] = -1
        s["gates"] = torch.softmax(torch.randn(t, c, generator=g, device=dev), dim=1)
        s["h"] = normal(t * c, w)  # the experts' products, in the experts' order
        if case["op"] == "exchange":
            s["ids"], s["x"] = ids, normal(t, w)
        else:
            s["offsets"], s["positions"], s["slots"] = plain_route(ids, e)  # kept from the forward pass
            s["dout"], s["drows"] = normal(t, w), normal(t * c, w)
        return s
    rows, k, n = case["rows"], case["k"], case["n"]
    backward = case["op"].endswith("backward")
    if case["op"].startswith("grouped"):
        e = case["experts"]
        odds = torch.softmax(torch.randn(e, generator=g, device=dev) * case["skew"], dim=0)
        counts = torch.bincount(torch.multinomial(odds, rows, replacement=True, generator=g), minlength=e)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["most"] = int(counts.max())  # the longest group, for the plain form's padding
        s["x"] = normal(rows, k)
        s["w"] = normal(e, n, k, scale=k ** -0.5)
        s["b"] = normal(e, n, scale=0.1) if case["bias"] else None
    else:
        s["x"] = normal(rows, k + case["pad"])[:, :k]
        s["w"] = normal(n, k, scale=k ** -0.5)
        s["b"] = normal(n, scale=0.1) if case["bias"] else None
        s["residual"] = normal(rows, n) if case["residual"] else None
    if backward:
        s["preact"] = normal(rows, n)
        s["dout"] = normal(rows, n)
    return s


# ---- one pass ----------------------------------------------------------------------
def run(s):
    if own:
        return run_own(s)
    return {"linear": plain_linear, "linear_backward": plain_linear_backward, "grouped": plain_grouped,
            "grouped_backward": plain_grouped_backward, "exchange": plain_exchange,
            "exchange_backward": plain_exchange_backward}[s["op"]](s)


def run_own(s):
    from chunk_schedule_execution_amd import ops

    op = s["op"]
    if op == "linear":
        return ops.linear(s["x"], s["w"], bias=s["b"], residual=s["residual"], activation=s["act"],
                          save_preact=s["save"])
    if op == "linear_backward":
        return ops.linear_backward(s["dout"], s["x"], s["w"], preact=s["preact"], activation=s["act"],
                                   bias=s["bias"])
    if op == "grouped":
        return ops.grouped_linear(s["x"], s["w"], s["offsets"], bias=s["b"], activation=s["act"],
                                  save_preact=s["save"])
    if op == "grouped_backward":
        return ops.grouped_linear_backward(s["dout"], s["x"], s["w"], s["offsets"], preact=s["preact"],
                                           activation=s["act"], bias=s["bias"])
    if op == "exchange":
        offsets, positions, slots = ops.expert_route(s["ids"], s["experts"])
        rows = ops.expert_dispatch(s["x"], slots, s["choices"])
        return offsets, positions, slots, rows, ops.expert_combine(s["h"], positions, s["gates"])
    dh, dgates = ops.expert_combine_backward(s["dout"], s["h"], s["positions"], s["slots"], s["gates"])
    return dh, dgates, ops.expert_combine(s["drows"], s["positions"])


# ---- plain forms, in 32 bits -------------------------------------------------------
def plain_act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return z * 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return z * 0.5 * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    return z / (1.0 + torch.exp(-z))


def plain_slope(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (0.5 / math.pi) ** 0.5
    if act == "gelu_tanh":
        c = (2.0 / math.pi) ** 0.5
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    p = 1.0 / (1.0 + torch.exp(-z))
    return p * (1.0 + z * (1.0 - p))


def plain_linear(s):
    dtype = s["x"].dtype
    z = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        z = z + s["b"].float()
    out = plain_act(z, s["act"])
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return (out.to(dtype), z.to(dtype)) if s["save"] else out.to(dtype)


def plain_linear_backward(s):
    dtype = s["x"].dtype
    dz = s["dout"].float() * plain_slope(s["preact"].float(), s["act"])
    dx = dz @ s["w"].float()
    dw = dz.t() @ s["x"].float()
    db = dz.sum(0).to(dtype) if s["bias"] else None
    return [t for t in (dx.to(dtype), dw.to(dtype), db) if t is not None]


def padded(s, rows):
    """(experts, longest group) row indices of the groups, and which of them are real."""
    begin, end = s["offsets"][:-1].long(), s["offsets"][1:].long()
    at = begin[:, None] + torch.arange(max(1, s["most"]), device=begin.device)
    real = at < end[:, None]
    return at.clamp(max=rows - 1), real


def plain_grouped(s):
    x, dtype = s["x"], s["x"].dtype
    at, real = padded(s, x.shape[0])
    z = torch.bmm(x.float()[at], s["w"].float().transpose(1, 2))
    if s["b"] is not None:
        z = z + s["b"].float()[:, None, :]
    z = z[real]  # back to the rows in order: the groups follow each other
    out = plain_act(z, s["act"])
    return (out.to(dtype), z.to(dtype)) if s["save"] else out.to(dtype)


def plain_grouped_backward(s):
    x, dtype = s["x"], s["x"].dtype
    at, real = padded(s, x.shape[0])
    dz = s["dout"].float() * plain_slope(s["preact"].float(), s["act"])
    dzp = dz[at] * real[:, :, None]
    dx = torch.bmm(dzp, s["w"].float())[real]
    dw = torch.bmm(dzp.transpose(1, 2), x.float()[at])
    db = dzp.sum(1).to(dtype) if s["bias"] else None
    return [t for t in (dx.to(dtype), dw.to(dtype), db) if t is not None]


def plain_route(ids, experts):
    """Stable counting sort of the choices by expert: (offsets, positions, slots)."""
    flat = ids.reshape(-1).long()
    hot = flat[:, None] == torch.arange(experts, device=ids.device)
    before = hot.int().cumsum(0) - 1  # place within its expert
    counts = hot.int().sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    here = hot.any(1)
    own_expert = torch.where(here, flat, torch.zeros_like(flat))
    pos = offsets[own_expert] + before.gather(1, own_expert[:, None])[:, 0]
    pos = torch.where(here, pos, torch.full_like(pos, -1))
    # every row's slot: those served elsewhere all write a place past the end, cut off again
    slots = torch.full((flat.numel() + 1,), -1, dtype=torch.int64, device=ids.device)
    slots[torch.where(here, pos, torch.full_like(pos, flat.numel()))] = torch.arange(flat.numel(), device=ids.device)
    return offsets.to(torch.int32), pos.view(ids.shape).to(torch.int32), slots[:-1].to(torch.int32)


def plain_combine(h, positions, gates):
    here = (positions >= 0)[:, :, None]
    rows = torch.where(here, h.float()[positions.clamp(min=0).long()], torch.zeros((), device=h.device))
    if gates is not None:
        rows = rows * gates[:, :, None]
    return rows.sum(1).to(h.dtype)


def plain_exchange(s):
    offsets, positions, slots = plain_route(s["ids"], s["experts"])
    token = slots.clamp(min=0).long() // s["choices"]
    rows = torch.where((slots >= 0)[:, None], s["x"][token], torch.zeros((), dtype=s["x"].dtype, device=token.device))
    return offsets, positions, slots, rows, plain_combine(s["h"], positions, s["gates"])


def plain_exchange_backward(s):
    dout, h, positions, slots, gates = s["dout"].float(), s["h"], s["positions"], s["slots"], s["gates"]
    at = slots.clamp(min=0).long()
    dh = torch.where((slots >= 0)[:, None], dout[at // s["choices"]] * gates.reshape(-1)[at][:, None],
                     torch.zeros((), device=dout.device))
    prod = (h.float()[positions.clamp(min=0).long()] * dout[:, None, :]).sum(2)
    dgates = torch.where(positions >= 0, prod, torch.zeros_like(prod))
    return dh.to(h.dtype), dgates, plain_combine(s["drows"], positions, None)


# ---- what a pass cannot do without ---------------------------------------------------
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("exchange"):
        t, c, w = case["tokens"], case["choices"], case["width"]
        slots = t * c
        used = slots * (1.0 - case["away"])  # rows that this rank's experts serve
        if op == "exchange":
            # ids and gates in; positions and slots out; x in, rows out; h's used rows in, out out
            return {"bytes": round(16 * slots + size * w * (t + slots + used + t)), "flops": round(2 * used * w)}
        # dout, h, drows (used rows) and plan in; dh, dgates and dx out
        return {"bytes": round(16 * slots + size * w * (t + used + used + slots + t)), "flops": round(4 * used * w)}
    rows, k, n = case["rows"], case["k"], case["n"]
    e = case.get("experts", 1)
    if op == "grouped":  # experts that got no row need not be read; at least this many did, evenly spread
        e = min(e, max(1, round(e * (1.0 - (1.0 - 1.0 / e) ** rows))))
    bias = e * n if case["bias"] else 0
    if op in ("linear", "grouped"):
        extra = rows * n * (int(case.get("residual", False)) + int(case["save"]))
        return {"bytes": size * (rows * k + e * n * k + bias + rows * n + extra), "flops": 2 * rows * k * n}
    acts = rows * n * (1 if case["act"] == "none" else 2)  # dout, and the pre-activation where it matters
    return {"bytes": size * (acts + 2 * rows * k + 2 * e * n * k + bias), "flops": 4 * rows * k * n}


# ---- the definitions, in 64 bits ------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("exchange"):
        return exact_exchange(s) if op == "exchange" else exact_exchange_backward(s)
    if op.startswith("linear"):
        bounds = [(0, case["rows"])]
        weights = [s["w"]]
        biases = [s["b"]]
    else:
        o = s["offsets"].tolist()
        bounds = list(zip(o[:-1], o[1:]))
        weights = list(s["w"])
        biases = [None] * len(weights) if s["b"] is None else list(s["b"])
    if op in ("linear", "grouped"):
        zs = []
        for (lo, hi), w, b in zip(bounds, weights, biases):
            z = torch.mm(s["x"][lo:hi].double(), w.double().t())
            zs.append(z if b is None else z + b.double())
        z = torch.cat(zs)
        out = exact_act(z, case["act"])
        if s.get("residual") is not None:
            out = out + s["residual"].double()
        return (out, z) if case["save"] else out
    z = s["preact"].double().requires_grad_(True)
    (slope,) = torch.autograd.grad(exact_act(z, case["act"]).sum(), z)
    dz = s["dout"].double() * slope
    dx, dw, db = [], [], []
    for (lo, hi), w in zip(bounds, weights):
        dx.append(torch.mm(dz[lo:hi], w.double()))
        dw.append(torch.mm(dz[lo:hi].t(), s["x"][lo:hi].double()))
        db.append(dz[lo:hi].sum(0))
    if op == "linear_backward":
        dw, db = dw[0], db[0]
    else:
        dw, db = torch.stack(dw), torch.stack(db)
    return [torch.cat(dx), dw] + ([db] if case["bias"] else [])


def exact_act(z, act):
    """The activation from its definition; relu has slope 0 at 0."""
    if act == "none":
        return z * 1.0
    if act == "relu":
        return z.clamp(min=0.0) * (z > 0)
    if act == "gelu":  # z times the normal distribution function
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        u = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)
        return 0.5 * z * (1.0 + torch.tanh(u))
    return z * torch.sigmoid(z)


def exact_plan(ids, experts):
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    key, order = torch.sort(key, stable=True)
    used = int((key < experts).sum())
    offsets = torch.searchsorted(key, torch.arange(experts + 1, device=key.device))
    slots = torch.where(torch.arange(flat.numel(), device=key.device) < used, order, torch.full_like(order, -1))
    positions = torch.full_like(flat, -1)
    positions[order[:used]] = torch.arange(used, device=key.device)
    return offsets.to(torch.int32), positions.view(ids.shape).to(torch.int32), slots.to(torch.int32)


def exact_sum(h, positions, gates):
    out = torch.zeros(positions.shape[0], h.shape[1], dtype=torch.float64, device=h.device)
    for j in range(positions.shape[1]):
        here = positions[:, j] >= 0
        row = h[positions[here, j].long()].double()
        out[here] += row if gates is None else row * gates[here, j, None].double()
    return out


def exact_exchange(s):
    offsets, positions, slots = exact_plan(s["ids"], s["experts"])
    rows = torch.zeros(slots.numel(), s["x"].shape[1], dtype=torch.float64, device=slots.device)
    used = slots >= 0
    rows[used] = s["x"].double()[slots[used].long() // s["choices"]]
    return offsets, positions, slots, rows, exact_sum(s["h"], positions, s["gates"])


def exact_exchange_backward(s):
    positions, slots, c = s["positions"], s["slots"], s["choices"]
    dout, gates = s["dout"].double(), s["gates"].double()
    dh = torch.zeros(s["h"].shape, dtype=torch.float64, device=dout.device)
    used = slots >= 0
    at = slots[used].long()
    dh[used] = dout[at // c] * gates[at // c, at % c, None]
    dgates = torch.zeros(positions.shape, dtype=torch.float64, device=dout.device)
    for j in range(c):
        here = positions[:, j] >= 0
        dgates[here, j] = (dout[here] * s["h"][positions[here, j].long()].double()).sum(1)
    return dh, dgates, exact_sum(s["drows"], positions, None)
