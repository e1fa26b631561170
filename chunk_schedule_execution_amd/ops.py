"""Products, row exchange and the layer's operators around them, beside the collectives, over
torch tensors.

Thin wrappers of the ``ccl_linear*``, ``ccl_grouped_linear*``, ``ccl_expert_*``,
``ccl_layer_norm*`` and ``ccl_*cross_entropy*`` entry points: they read shapes, strides and
types off the tensors, allocate outputs and workspace from torch on the call's stream and launch
there (torch's current stream of the tensors' device unless ``stream``, a torch stream or a raw
handle, is given). A call on another stream orders nothing by itself, as with ``Plan.execute``:
the caller lets that stream wait for the inputs and keeps them (and an ``out`` of its own) until
it has passed the call. What the call allocates is that stream's, so nothing that torch's
current stream still works on is written; outputs may be dropped as soon as the current stream's
own work on them is enqueued. Everything else is in ``libccl.so``. Gradients are explicit calls;
nothing registers with torch's autograd.

Floating tensors of a call share one type, float32 or bfloat16 (gates, the bias that experts are
ranked with, a norm's statistics and losses are float32). Matrices may have rows further apart
than their length; their rows must be contiguous.
"""

from __future__ import annotations

import torch

from . import capi

DTYPES = {torch.float32: capi.CCL_F32, torch.bfloat16: capi.CCL_BF16}
ACTIVATIONS = {"none": capi.CCL_ACT_NONE, "relu": capi.CCL_ACT_RELU, "gelu": capi.CCL_ACT_GELU,
               "gelu_tanh": capi.CCL_ACT_GELU_TANH, "silu": capi.CCL_ACT_SILU}
SCORES = {"softmax": capi.CCL_SCORE_SOFTMAX, "sigmoid": capi.CCL_SCORE_SIGMOID}


# ---- arguments ----------------------------------------------------------------------
# These run on every call, in front of kernels that take a few microseconds: one look at
# each property, and messages are made only for what is refused.
def _refuse(what: str):
    raise ValueError(what)


def _first(t, name: str) -> int:
    """The device index of the matrix that the other arguments have to match."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        _refuse(f"{name}: a matrix wanted")
    if t.dtype not in DTYPES:
        _refuse(f"{name}: float32 or bfloat16 wanted, not {t.dtype}")
    if not t.is_cuda:
        _refuse(f"{name}: on {t.device}; GPU memory wanted")
    return t.get_device()


def _like(t, name: str, shape, dtype, device: int) -> None:
    if not isinstance(t, torch.Tensor):
        _refuse(f"{name}: a tensor wanted")
    if t.dtype is not dtype:
        _refuse(f"{name}: {dtype} wanted, not {t.dtype}")
    if t.shape != shape:
        _refuse(f"{name}: shape {tuple(shape)} wanted, not {tuple(t.shape)}")
    if not t.is_cuda or t.get_device() != device:
        _refuse(f"{name}: on {t.device}; memory of GPU {device} wanted")


def _packed(t, name: str, shape, dtype, device: int) -> int:
    """Address of a contiguous tensor."""
    _like(t, name, shape, dtype, device)
    if not t.is_contiguous():
        _refuse(f"{name}: contiguous wanted")
    return t.data_ptr()


def _ld(t, name: str) -> int:
    """Distance between the rows of a matrix, or of matrices that follow each other (0:
    there is one row, or none)."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 2:
        rows, width = shape
        if rows <= 1 or width == 0:
            if width > 1 and rows and stride[1] != 1:
                _refuse(f"{name}: rows must be contiguous")
            return 0
        ld = stride[0]
    else:
        experts, rows, width = shape
        if experts * rows <= 1 or width == 0:
            ld = 0
        elif rows == 1:
            ld = stride[0]
        else:
            ld = stride[1]
            if experts > 1 and stride[0] != rows * ld:
                _refuse(f"{name}: the experts' matrices must follow each other")
        if ld == 0 and experts * rows > 1:
            _refuse(f"{name}: rows must not overlap")
    if width > 1 and stride[-1] != 1:
        _refuse(f"{name}: rows must be contiguous")
    if 0 <= ld < width and (ld or len(shape) == 2):
        _refuse(f"{name}: rows must not overlap")
    return ld


# the handle alone, without a Stream object around it (0.1 us instead of 1.9)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


class _on:
    """The device and the stream of a call, made torch's current ones for its length where
    they are not, so that memory comes from the pool of the stream that uses it: a block of
    another stream's pool may still be in use there after its tensor is gone."""

    __slots__ = ("device", "before", "stream", "handle", "outer", "switch")

    def __init__(self, device: int, stream):
        self.device, self.stream, self.switch = device, stream, None
        if stream is not None:
            if getattr(stream, "device", None) is not None and stream.device.index != device:
                _refuse(f"stream: of {stream.device}; one of GPU {device} wanted")
            self.handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)

    def __enter__(self) -> int:
        """The handle to launch on."""
        self.before = torch.cuda.current_device()
        if self.before != self.device:
            torch.cuda.set_device(self.device)
        current = _raw_stream(self.device)
        if self.stream is None:
            return current
        if self.handle != current:
            self.outer = torch.cuda.current_stream()
            self.switch = torch.cuda.stream(
                self.stream if isinstance(self.stream, torch.cuda.Stream) else
                torch.cuda.ExternalStream(self.handle) if self.handle else torch.cuda.default_stream())
            self.switch.__enter__()
        return self.handle

    def give(self, *tensors) -> None:
        """Tells torch's allocator that outputs made here go to the stream that was current:
        freed, they are not handed out again before it has passed its work on them."""
        if self.switch is not None:
            for t in tensors:
                if t is not None and t.numel():
                    t.record_stream(self.outer)

    def __exit__(self, *a):
        if self.switch is not None:
            self.switch.__exit__(*a)
        if self.before != self.device:
            torch.cuda.set_device(self.before)


def _workspace(nbytes: int, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


# ---- products -----------------------------------------------------------------------
def linear(x, w, bias=None, residual=None, activation="none", save_preact=False, out=None, preact=None, stream=None):
    """act(x w^T + bias) + residual: x (rows, in), w (out, in), bias (out,), residual
    (rows, out). With ``save_preact`` (or a ``preact`` tensor to fill) returns (out,
    preact), preact being the activation's argument, which ``linear_backward`` takes.
    Autograd does not see the call: outputs require no gradient, whatever the inputs do."""
    return _forward(x, w, None, bias, residual, activation, save_preact, out, preact, stream)


def grouped_linear(x, w, offsets, bias=None, activation="none", save_preact=False, out=None, preact=None,
                   stream=None):
    """The same by groups of rows: rows offsets[e] .. offsets[e + 1] - 1 of x (rows, in) are
    multiplied by expert e's matrix of w (experts, out, in) and get row e of bias (experts,
    out). offsets: (experts + 1) int32 on the GPU, ascending from 0; rows from its last
    value on belong to no group and give zeros. Autograd does not see the call."""
    return _forward(x, w, offsets, bias, None, activation, save_preact, out, preact, stream)


def _weights(w, x, grouped: bool):
    """(experts, out_features) of w, which has to match x (rows, in)."""
    if not isinstance(w, torch.Tensor) or w.dim() != (3 if grouped else 2):
        _refuse("w: (experts, out, in) wanted" if grouped else "w: (out, in) wanted")
    return (w.shape[0] if grouped else 0), w.shape[-2]


def _forward(x, w, offsets, bias, residual, activation, save_preact, out, preact, stream):
    device, grouped = _first(x, "x"), offsets is not None
    experts, n = _weights(w, x, grouped)
    rows, k = x.shape
    dtype = x.dtype
    _like(w, "w", (experts, n, k) if grouped else (n, k), dtype, device)
    if activation not in ACTIVATIONS:
        _refuse(f"unknown activation {activation!r}")
    px, pw = x.data_ptr(), w.data_ptr()
    po = _packed(offsets, "offsets", (experts + 1,), torch.int32, device) if grouped else 0
    pb = 0 if bias is None else _packed(bias, "bias", (experts, n) if grouped else (n,), dtype, device)
    pr = ldr = pp = ldp = ldo = 0
    if residual is not None:
        _like(residual, "residual", (rows, n), dtype, device)
        pr, ldr = residual.data_ptr(), _ld(residual, "residual")
    on = _on(device, stream)
    with on as handle:
        made_out = out is None
        if made_out:
            out = torch.empty(rows, n, dtype=dtype, device=x.device)
        else:
            _like(out, "out", (rows, n), dtype, device)
            ldo = _ld(out, "out")
        pout = out.data_ptr()
        made_preact = preact is None and save_preact
        if made_preact:
            preact = torch.empty(rows, n, dtype=dtype, device=x.device)
        elif preact is not None:
            _like(preact, "preact", (rows, n), dtype, device)
            ldp = _ld(preact, "preact")
        if preact is not None:
            pp = preact.data_ptr()
        d = capi.ccl_linear_desc(DTYPES[dtype], ACTIVATIONS[activation], rows, k, n, experts,
                                 capi.CCL_LINEAR_UNALIGNED if (px | pw | pb | pr | pout | pp) % 16 else 0,
                                 _ld(x, "x"), _ld(w, "w"), ldo, ldr, ldp)
        nbytes = capi.ccl_linear_workspace(d, grouped, False)
        ws = _workspace(nbytes, x.device)
        pws = ws.data_ptr() if nbytes else 0
        if grouped:
            capi.ccl_grouped_linear(d, po, px, pw, pb, pout, pp, pws, nbytes, handle)
        else:
            capi.ccl_linear(d, px, pw, pb, pr, pout, pp, pws, nbytes, handle)
        on.give(out if made_out else None, preact if made_preact else None)
    return out if preact is None else (out, preact)


def linear_backward(dout, x, w, preact=None, activation="none", bias=False, need_dx=True, need_dw=True, stream=None):
    """Gradients of ``linear``: [dx, dw] and, with ``bias``, dbias; a gradient that is not
    needed is left out of the list. The residual's gradient is dout itself. preact: what the
    forward pass saved (not used for activation "none"). Between the activation and the
    products the gradient is rounded to the tensors' type, as one that is stored there is:
    in bfloat16 dx and dw are off by sqrt 2 of what their own rounding takes (0.0023 of
    them for 0.0017). Float32 tensors keep it whole."""
    return _backward(dout, x, w, None, preact, activation, bias, need_dx, need_dw, stream)


def grouped_linear_backward(dout, x, w, offsets, preact=None, activation="none", bias=False, need_dx=True,
                            need_dw=True, stream=None):
    """Gradients of ``grouped_linear``: dx (zeros for rows of no group), dw (experts, out,
    in) and dbias (experts, out), zeros for an empty group. Rounded as ``linear_backward``'s."""
    return _backward(dout, x, w, offsets, preact, activation, bias, need_dx, need_dw, stream)


def _backward(dout, x, w, offsets, preact, activation, bias, need_dx, need_dw, stream):
    device, grouped = _first(x, "x"), offsets is not None
    experts, n = _weights(w, x, grouped)
    rows, k = x.shape
    dtype = x.dtype
    _like(w, "w", (experts, n, k) if grouped else (n, k), dtype, device)
    _like(dout, "dout", (rows, n), dtype, device)
    if activation not in ACTIVATIONS:
        _refuse(f"unknown activation {activation!r}")
    px, pw, pd = x.data_ptr(), w.data_ptr(), dout.data_ptr()
    po = _packed(offsets, "offsets", (experts + 1,), torch.int32, device) if grouped else 0
    pp = ldp = 0
    if activation != "none":
        if preact is None:
            _refuse("the activation's gradient needs preact")
        _like(preact, "preact", (rows, n), dtype, device)
        pp, ldp = preact.data_ptr(), _ld(preact, "preact")
    on = _on(device, stream)
    with on as handle:
        dx = torch.empty(rows, k, dtype=dtype, device=x.device) if need_dx else None
        dw = torch.empty(w.shape, dtype=dtype, device=x.device) if need_dw else None
        db = torch.empty(w.shape[:-1], dtype=dtype, device=x.device) if bias else None
        d = capi.ccl_linear_desc(DTYPES[dtype], ACTIVATIONS[activation], rows, k, n, experts,
                                 capi.CCL_LINEAR_UNALIGNED if (px | pw | pd | pp) % 16 else 0,
                                 _ld(x, "x"), _ld(w, "w"), _ld(dout, "dout"), 0, ldp)
        nbytes = capi.ccl_linear_workspace(d, grouped, True)
        ws = _workspace(nbytes, x.device)
        tail = (pd, px, pw, pp, dx.data_ptr() if need_dx else 0, dw.data_ptr() if need_dw else 0,
                db.data_ptr() if bias else 0, ws.data_ptr() if nbytes else 0, nbytes, handle)
        if grouped:
            capi.ccl_grouped_linear_backward(d, po, *tail)
        else:
            capi.ccl_linear_backward(d, *tail)
        on.give(dx, dw, db)
    return [t for t in (dx, dw, db) if t is not None]


# ---- row exchange ---------------------------------------------------------------------
def expert_route(ids, experts, stream=None):
    """ids (tokens, choices) int32 -> (offsets (experts + 1), positions (tokens, choices),
    slots (tokens * choices)), int32: rows ordered by expert and, within an expert, by slot
    (the index of a choice in ids). positions: a choice's row, -1 where its id is not in
    [0, experts); slots: a row's choice, -1 for the rows from offsets[experts] on."""
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        _refuse("ids: (tokens, choices) wanted")
    device = ids.get_device()
    pi = _packed(ids, "ids", ids.shape, torch.int32, device)
    tokens, choices = ids.shape
    nbytes = capi.ccl_expert_route_workspace(tokens, choices, experts)
    on = _on(device, stream)
    with on as handle:
        offsets = torch.empty(experts + 1, dtype=torch.int32, device=ids.device)
        positions = torch.empty_like(ids)
        slots = torch.empty(tokens * choices, dtype=torch.int32, device=ids.device)
        ws = _workspace(nbytes, ids.device)
        capi.ccl_expert_route(pi, tokens, choices, experts, offsets.data_ptr(), positions.data_ptr(),
                              slots.data_ptr(), ws.data_ptr() if nbytes else 0, nbytes, handle)
        on.give(offsets, positions, slots)
    return offsets, positions, slots


def _gates(gates, positions, device: int) -> int:
    return 0 if gates is None else _packed(gates, "gates", positions.shape, torch.float32, device)


def expert_dispatch(x, slots, choices, out=None, stream=None):
    """rows[i] = x[slots[i] // choices], zeros where slots[i] is -1: x (tokens, width), rows
    (tokens * choices, width). Autograd does not see the call."""
    device = _first(x, "x")
    tokens, width = x.shape
    ps = _packed(slots, "slots", (tokens * choices,), torch.int32, device)
    on = _on(device, stream)
    with on as handle:
        made, ldo = out is None, 0
        if made:
            out = torch.empty(tokens * choices, width, dtype=x.dtype, device=x.device)
        else:
            _like(out, "out", (tokens * choices, width), x.dtype, device)
            ldo = _ld(out, "out")
        capi.ccl_expert_dispatch(DTYPES[x.dtype], x.data_ptr(), _ld(x, "x"), ps, tokens, choices, width,
                                 out.data_ptr(), ldo, handle)
        if made:
            on.give(out)
    return out


def expert_combine(h, positions, gates=None, out=None, stream=None):
    """out[t] = sum over j of gates[t, j] h[positions[t, j]]: h (tokens * choices, width),
    gates (tokens, choices) float32 or None for ones. Without gates it is also the gradient
    of ``expert_dispatch``'s x from its rows' gradients. Autograd does not see the call."""
    device = _first(h, "h")
    if not isinstance(positions, torch.Tensor) or positions.dim() != 2:
        _refuse("positions: (tokens, choices) wanted")
    tokens, choices = positions.shape
    width = h.shape[1]
    _like(h, "h", (tokens * choices, width), h.dtype, device)
    pp = _packed(positions, "positions", positions.shape, torch.int32, device)
    pg = _gates(gates, positions, device)
    on = _on(device, stream)
    with on as handle:
        made, ldo = out is None, 0
        if made:
            out = torch.empty(tokens, width, dtype=h.dtype, device=h.device)
        else:
            _like(out, "out", (tokens, width), h.dtype, device)
            ldo = _ld(out, "out")
        capi.ccl_expert_combine(DTYPES[h.dtype], h.data_ptr(), _ld(h, "h"), pp, pg, tokens, choices, width,
                                out.data_ptr(), ldo, handle)
        if made:
            on.give(out)
    return out


def expert_combine_backward(dout, h, positions, slots, gates=None, stream=None):
    """Gradients of ``expert_combine``: dh (tokens * choices, width) and dgates (tokens,
    choices) float32; positions and slots are the route's."""
    device = _first(dout, "dout")
    if not isinstance(positions, torch.Tensor) or positions.dim() != 2:
        _refuse("positions: (tokens, choices) wanted")
    tokens, choices = positions.shape
    width = dout.shape[1]
    _like(dout, "dout", (tokens, width), dout.dtype, device)
    _like(h, "h", (tokens * choices, width), dout.dtype, device)
    pp = _packed(positions, "positions", positions.shape, torch.int32, device)
    ps = _packed(slots, "slots", (tokens * choices,), torch.int32, device)
    pg = _gates(gates, positions, device)
    on = _on(device, stream)
    with on as handle:
        dh = torch.empty(tokens * choices, width, dtype=h.dtype, device=h.device)
        dgates = torch.empty(tokens, choices, dtype=torch.float32, device=h.device)
        capi.ccl_expert_combine_backward(DTYPES[h.dtype], dout.data_ptr(), _ld(dout, "dout"), h.data_ptr(),
                                         _ld(h, "h"), pp, ps, pg, tokens, choices, width, dh.data_ptr(), 0,
                                         dgates.data_ptr(), handle)
        on.give(dh, dgates)
    return dh, dgates


# ---- choice of experts ------------------------------------------------------------------
def _select_desc(logits, choices, score, groups, kept_groups, group_best, renormalise, scale):
    if score not in SCORES:
        _refuse(f"unknown score {score!r}")
    tokens, experts = logits.shape
    kept = groups if kept_groups is None else kept_groups
    # a descriptor's fields hold 32 bits and would take the rest of a number for the whole
    if not (1 <= kept <= groups <= 64 and 1 <= group_best <= 2):
        _refuse(f"groups: 1 .. 64 wanted, of which 1 to all stay by their 1 or 2 best, not {groups}, {kept}, {group_best}")
    return capi.ccl_select_desc(DTYPES[logits.dtype], SCORES[score], tokens, experts, choices, groups, kept, group_best,
                                int(bool(renormalise)), scale, _ld(logits, "logits"))


def expert_select(logits, choices, score="softmax", bias=None, groups=1, kept_groups=None, group_best=1,
                  renormalise=False, scale=1.0, stream=None):
    """The experts of every token: logits (tokens, experts) -> (ids (tokens, choices) int32,
    gates (tokens, choices) float32), which ``expert_route`` and ``expert_combine`` take.

    p is the softmax of a token's logits or their sigmoids (``score``). Experts are ranked by
    p + bias (bias (experts,) float32 or None, compared in 64 bits; ties go to the lower
    index); with ``kept_groups`` < ``groups`` only within the groups of neighbouring experts
    whose ``group_best`` (1 or 2) highest values sum up highest. gates: scale p of the chosen
    experts, divided by the sum of their p with ``renormalise``. An expert whose logit or bias
    is -inf is never chosen; a token with fewer open ones than ``choices`` gets ids -1 and
    gates 0 behind them. Autograd does not see the call."""
    device = _first(logits, "logits")
    tokens, experts = logits.shape
    d = _select_desc(logits, choices, score, groups, kept_groups, group_best, renormalise, scale)
    pb = 0 if bias is None else _packed(bias, "bias", (experts,), torch.float32, device)
    if not 1 <= choices <= experts:
        _refuse(f"choices: 1 .. {experts} wanted, not {choices}")
    on = _on(device, stream)
    with on as handle:
        ids = torch.empty(tokens, choices, dtype=torch.int32, device=logits.device)
        gates = torch.empty(tokens, choices, dtype=torch.float32, device=logits.device)
        capi.ccl_expert_select(d, logits.data_ptr(), pb, ids.data_ptr(), gates.data_ptr(), handle)
        on.give(ids, gates)
    return ids, gates


def expert_select_backward(dgates, logits, ids, score="softmax", renormalise=False, scale=1.0, stream=None):
    """Gradient of ``expert_select``'s gates by the logits, (tokens, experts) of their type:
    what was chosen counts as fixed, and so do bias and groups."""
    device = _first(logits, "logits")
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        _refuse("ids: (tokens, choices) wanted")
    tokens, experts = logits.shape
    pi = _packed(ids, "ids", (tokens, ids.shape[1]), torch.int32, device)
    pd = _packed(dgates, "dgates", ids.shape, torch.float32, device)
    d = _select_desc(logits, ids.shape[1], score, 1, 1, 1, renormalise, scale)
    on = _on(device, stream)
    with on as handle:
        dlogits = torch.empty(tokens, experts, dtype=logits.dtype, device=logits.device)
        capi.ccl_expert_select_backward(d, pd, logits.data_ptr(), pi, dlogits.data_ptr(), handle)
        on.give(dlogits)
    return dlogits


# ---- layer norm ---------------------------------------------------------------------------
def layer_norm(x, weight=None, bias=None, residual=None, eps=1e-5, save_stats=False, out=None, total=None,
               stream=None):
    """(h - mean) rstd weight + bias with h = x + residual: x and residual (rows, width),
    weight and bias (width,). Returns out; with a residual also total, h rounded to the type
    (the norm sees it unrounded); with ``save_stats`` also mean and rstd, (rows,) float32:
    (out[, total][, mean, rstd]). ``layer_norm_backward`` takes total (x without a residual)
    and the statistics. ``out`` and ``total`` may be given, also as x or residual themselves (not
    both as the same one, nor as other rows of their memory). Autograd does not see the call."""
    device = _first(x, "x")
    rows, width = x.shape
    dtype = x.dtype
    pw = 0 if weight is None else _packed(weight, "weight", (width,), dtype, device)
    pb = 0 if bias is None else _packed(bias, "bias", (width,), dtype, device)
    pr = ldr = ldo = pt = ldt = 0
    if residual is not None:
        _like(residual, "residual", (rows, width), dtype, device)
        pr, ldr = residual.data_ptr(), _ld(residual, "residual")
    elif total is not None:
        _refuse("total: without a residual it is x")
    ldx = _ld(x, "x")
    if out is not None:
        _like(out, "out", (rows, width), dtype, device)
        ldo = _ld(out, "out")
    if total is not None:
        _like(total, "total", (rows, width), dtype, device)
        ldt = _ld(total, "total")
    on = _on(device, stream)
    with on as handle:
        made_out, made_total = out is None, total is None and residual is not None
        if made_out:
            out = torch.empty(rows, width, dtype=dtype, device=x.device)
        if made_total:
            total = torch.empty(rows, width, dtype=dtype, device=x.device)
        if total is not None:
            pt = total.data_ptr()
        mean = torch.empty(rows, dtype=torch.float32, device=x.device) if save_stats else None
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device) if save_stats else None
        d = capi.ccl_norm_desc(DTYPES[dtype], eps, rows, width, ldx, ldr, ldo, ldt)
        capi.ccl_layer_norm(d, x.data_ptr(), pr, pw, pb, out.data_ptr(), pt, mean.data_ptr() if save_stats else 0,
                            rstd.data_ptr() if save_stats else 0, handle)
        on.give(out if made_out else None, total if made_total else None, mean, rstd)
    if total is None and not save_stats:
        return out
    return (out,) + ((total,) if total is not None else ()) + ((mean, rstd) if save_stats else ())


def layer_norm_backward(dout, x, mean, rstd, weight=None, dtotal=None, bias=False, need_dx=True, need_dweight=True,
                        stream=None):
    """Gradients of ``layer_norm``: [dx, dweight, dbias], without those that are not needed
    (dweight belongs to a call with a weight, dbias to ``bias``). x is what was normalised:
    the forward call's total where it had a residual, whose gradient is dx too. dtotal (rows,
    width): the gradient that reaches total from elsewhere, added to dx."""
    device = _first(x, "x")
    rows, width = x.shape
    dtype = x.dtype
    _like(dout, "dout", (rows, width), dtype, device)
    pm, ps = _packed(mean, "mean", (rows,), torch.float32, device), _packed(rstd, "rstd", (rows,), torch.float32, device)
    pw = 0 if weight is None else _packed(weight, "weight", (width,), dtype, device)
    pt = ldt = 0
    if dtotal is not None:
        _like(dtotal, "dtotal", (rows, width), dtype, device)
        pt, ldt = dtotal.data_ptr(), _ld(dtotal, "dtotal")
    need_dweight = need_dweight and weight is not None
    d = capi.ccl_norm_desc(DTYPES[dtype], 0.0, rows, width, _ld(x, "x"), 0, _ld(dout, "dout"), 0, ldt)
    on = _on(device, stream)
    with on as handle:
        dx = torch.empty(rows, width, dtype=dtype, device=x.device) if need_dx else None
        dw = torch.empty(width, dtype=dtype, device=x.device) if need_dweight else None
        db = torch.empty(width, dtype=dtype, device=x.device) if bias else None
        nbytes = capi.ccl_layer_norm_backward_workspace(d) if need_dweight or bias else 0
        ws = _workspace(nbytes, x.device)
        capi.ccl_layer_norm_backward(d, dout.data_ptr(), x.data_ptr(), pm, ps, pw, pt, dx.data_ptr() if need_dx else 0,
                                     dw.data_ptr() if need_dweight else 0, db.data_ptr() if bias else 0,
                                     ws.data_ptr() if nbytes else 0, nbytes, handle)
        on.give(dx, dw, db)
    return [t for t in (dx, dw, db) if t is not None]


# ---- cross entropy over a vocabulary --------------------------------------------------------
def _loss_desc(x, w, targets, shard, device):
    """(descriptor, targets' address)."""
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        _refuse("w: (vocabulary, in) wanted")
    rows, k = x.shape
    _like(w, "w", (w.shape[0], k), x.dtype, device)
    if shard is not None and not 0 <= shard < 1 << 31:
        _refuse("shard: the vocabulary's index of w's first row wanted")
    pt = _packed(targets, "targets", (rows,), torch.int32, device)
    d = capi.ccl_cross_entropy_desc(DTYPES[x.dtype], 0, rows, k, w.shape[0], -1 if shard is None else shard,
                                    _ld(x, "x"), _ld(w, "w"))
    if (x.data_ptr() | w.data_ptr()) % 16:
        d.flags = capi.CCL_LINEAR_UNALIGNED
    return d, pt


def linear_cross_entropy(x, w, targets, shard=None, stream=None):
    """Cross entropy of the logits z = x w^T, which are not kept: x (rows, in), w (vocabulary,
    in), targets (rows,) int32 -> (loss, lse), (rows,) float32, with lse = log sum exp z and
    loss = lse - z at the target. A row whose target is negative or, without ``shard``, past the
    vocabulary is left out: loss 0, no gradient.

    With ``shard``, w holds the rows of the vocabulary from that index on (one rank's share),
    and the call returns (lse, picked): lse over them, picked the target's logit, 0 where the
    target is another shard's. ``cross_entropy_join`` makes loss and lse of all shards' pairs,
    gathered. No shard knows where the vocabulary ends: there only a negative target leaves its
    row out, one past the vocabulary counts as a row with loss = lse. Autograd does not see the
    call."""
    device = _first(x, "x")
    d, pt = _loss_desc(x, w, targets, shard, device)
    on = _on(device, stream)
    with on as handle:
        first = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
        second = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
        nbytes = capi.ccl_linear_cross_entropy_workspace(d, False)
        ws = _workspace(nbytes, x.device)
        p1, p2 = first.data_ptr(), second.data_ptr()
        loss, lse, picked = (p1, p2, 0) if shard is None else (0, p1, p2)
        capi.ccl_linear_cross_entropy(d, x.data_ptr(), w.data_ptr(), pt, loss, lse, picked,
                                      ws.data_ptr() if nbytes else 0, nbytes, handle)
        on.give(first, second)
    return first, second


def cross_entropy_join(lse, picked, targets, stream=None):
    """(loss, lse) over a whole vocabulary from its shards' lse and picked, (shards, rows)
    float32 each: what an AllGather of ``linear_cross_entropy``'s results gives. A row whose
    target is negative has loss 0; the vocabulary's end is not known here, either."""
    if not isinstance(lse, torch.Tensor) or lse.dim() != 2:
        _refuse("lse: (shards, rows) wanted")
    shards, rows = lse.shape
    device = lse.get_device()
    pl, pp = (_packed(t, name, (shards, rows), torch.float32, device) for t, name in ((lse, "lse"), (picked, "picked")))
    pt = _packed(targets, "targets", (rows,), torch.int32, device)
    on = _on(device, stream)
    with on as handle:
        loss = torch.empty(rows, dtype=torch.float32, device=lse.device)
        total = torch.empty(rows, dtype=torch.float32, device=lse.device)
        capi.ccl_cross_entropy_join(shards, rows, pl, pp, pt, loss.data_ptr(), total.data_ptr(), handle)
        on.give(loss, total)
    return loss, total


def linear_cross_entropy_backward(dloss, x, w, targets, lse, shard=None, need_dx=True, need_dw=True, stream=None):
    """Gradients of the loss: [dx, dw], without those that are not needed. dloss (rows,)
    float32; lse is the whole vocabulary's. The logits are computed again, in pieces of the
    vocabulary. With ``shard`` dx is this shard's summand (an AllReduce adds them up), dw its
    own. dz is rounded to the tensors' type for the two products, as ``linear_backward``'s is.
    Rows left out have no part, whatever their x, dloss and lse hold."""
    device = _first(x, "x")
    d, pt = _loss_desc(x, w, targets, shard, device)
    rows = x.shape[0]
    pd, pl = _packed(dloss, "dloss", (rows,), torch.float32, device), _packed(lse, "lse", (rows,), torch.float32, device)
    on = _on(device, stream)
    with on as handle:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if need_dx else None
        dw = torch.empty(w.shape, dtype=x.dtype, device=x.device) if need_dw else None
        nbytes = capi.ccl_linear_cross_entropy_workspace(
            d, capi.CCL_GRADIENTS if need_dx and need_dw else capi.CCL_GRADIENT_DX if need_dx else capi.CCL_GRADIENT_DW)
        ws = _workspace(nbytes, x.device)
        capi.ccl_linear_cross_entropy_backward(d, pd, x.data_ptr(), w.data_ptr(), pt, pl, dx.data_ptr() if need_dx else 0,
                                               dw.data_ptr() if need_dw else 0, ws.data_ptr() if nbytes else 0, nbytes,
                                               handle)
        on.give(dx, dw)
    return [t for t in (dx, dw) if t is not None]
