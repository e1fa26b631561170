"""Products and row exchange beside the collectives, over torch tensors.

Thin wrappers of the ``ccl_linear*``, ``ccl_grouped_linear*`` and ``ccl_expert_*`` entry
points: they read shapes, strides and types off the tensors, allocate outputs and
workspace from torch on the call's stream and launch there (torch's current stream of the
tensors' device unless ``stream`` is given; a call on another stream orders nothing by
itself, as with ``Plan.execute``). Everything else is in ``libccl.so``. Gradients are
explicit calls; nothing registers with torch's autograd.

Floating tensors of a call share one type, float32 or bfloat16 (gates are float32).
Matrices may have rows further apart than their length; their rows must be contiguous.
"""

from __future__ import annotations

import torch

from . import capi

DTYPES = {torch.float32: capi.CCL_F32, torch.bfloat16: capi.CCL_BF16}
ACTIVATIONS = {"none": capi.CCL_ACT_NONE, "relu": capi.CCL_ACT_RELU, "gelu": capi.CCL_ACT_GELU,
               "gelu_tanh": capi.CCL_ACT_GELU_TANH, "silu": capi.CCL_ACT_SILU}


# ---- arguments ----------------------------------------------------------------------
def _check(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _float(t: torch.Tensor, name: str, shape, like: torch.Tensor | None = None) -> torch.Tensor:
    _check(isinstance(t, torch.Tensor), f"{name}: a tensor wanted")
    _check(t.dtype in DTYPES, f"{name}: float32 or bfloat16 wanted, not {t.dtype}")
    _check(tuple(t.shape) == tuple(shape), f"{name}: shape {tuple(shape)} wanted, not {tuple(t.shape)}")
    if like is not None:
        _check(t.dtype == like.dtype, f"{name}: {like.dtype} wanted, not {t.dtype}")
        _check(t.device == like.device, f"{name}: on {t.device}, not {like.device}")
    _check(t.device.type == "cuda", f"{name}: on {t.device}; GPU memory wanted")
    return t


def _index(t: torch.Tensor, name: str, shape, like: torch.Tensor) -> torch.Tensor:
    _check(isinstance(t, torch.Tensor) and t.dtype == torch.int32, f"{name}: an int32 tensor wanted")
    _check(tuple(t.shape) == tuple(shape), f"{name}: shape {tuple(shape)} wanted, not {tuple(t.shape)}")
    _check(t.device == like.device and t.device.type == "cuda", f"{name}: on {t.device}, not {like.device}")
    _check(t.is_contiguous(), f"{name}: contiguous wanted")
    return t


def _ld(t: torch.Tensor | None, name: str) -> int:
    """Distance between the rows of a matrix (0: packed, or a single row)."""
    if t is None or t.numel() == 0:
        return 0
    _check(t.shape[-1] == 1 or t.stride(-1) == 1, f"{name}: rows must be contiguous")
    if t.dim() == 3 and t.shape[1] == 1:
        ld = t.stride(0) if t.shape[0] > 1 else 0
    else:
        ld = t.stride(-2) if t.shape[-2] > 1 else 0
        if t.dim() == 3 and t.shape[0] > 1:
            _check(t.stride(0) == t.shape[1] * ld, f"{name}: the experts' matrices must follow each other")
    several = t.shape[-2] > 1 or (t.dim() == 3 and t.shape[0] > 1)
    _check(not several or ld >= t.shape[-1], f"{name}: rows must not overlap")
    return ld


def _ptr(t: torch.Tensor | None) -> int:
    return 0 if t is None else t.data_ptr()


def _stream(stream, device) -> int:
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _own(stream, *tensors) -> None:
    """Tells torch's allocator that memory allocated on its current stream is in use on
    ``stream``, so it is not handed out again before that stream passes the call."""
    if stream is None:
        return
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    for t in tensors:
        if t is not None and t.numel():
            t.record_stream(stream)


def _workspace(nbytes: int, device) -> torch.Tensor | None:
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _desc(x_shape, out_features, dtype, activation, experts, tensors, **ld) -> capi.ccl_linear_desc:
    _check(activation in ACTIVATIONS, f"unknown activation {activation!r}")
    flags = 0
    if any(t is not None and t.data_ptr() % 16 for t in tensors):
        flags |= capi.CCL_LINEAR_UNALIGNED
    d = capi.ccl_linear_desc(dtype=DTYPES[dtype], activation=ACTIVATIONS[activation], rows=x_shape[0],
                             in_features=x_shape[1], out_features=out_features, experts=experts, flags=flags)
    for name, value in ld.items():
        setattr(d, name, value)
    return d


# ---- products -----------------------------------------------------------------------
def linear(x, w, bias=None, residual=None, activation="none", save_preact=False, out=None, preact=None, stream=None):
    """act(x w^T + bias) + residual: x (rows, in), w (out, in), bias (out,), residual
    (rows, out). With ``save_preact`` (or a ``preact`` tensor to fill) returns (out,
    preact), preact being the activation's argument, which ``linear_backward`` takes."""
    return _forward(x, w, None, bias, residual, activation, save_preact, out, preact, stream)


def grouped_linear(x, w, offsets, bias=None, activation="none", save_preact=False, out=None, preact=None,
                   stream=None):
    """The same by groups of rows: rows offsets[e] .. offsets[e + 1] - 1 of x (rows, in) are
    multiplied by expert e's matrix of w (experts, out, in) and get row e of bias (experts,
    out). offsets: (experts + 1) int32 on the GPU, ascending from 0; rows from its last
    value on belong to no group and give zeros."""
    return _forward(x, w, offsets, bias, None, activation, save_preact, out, preact, stream)


def _forward(x, w, offsets, bias, residual, activation, save_preact, out, preact, stream):
    grouped = offsets is not None
    _check(isinstance(x, torch.Tensor) and x.dim() == 2, "x: a matrix wanted")
    _check(isinstance(w, torch.Tensor) and w.dim() == (3 if grouped else 2),
           "w: (experts, out, in) wanted" if grouped else "w: (out, in) wanted")
    rows, k = x.shape
    n = w.shape[-2]
    experts = w.shape[0] if grouped else 1
    _float(x, "x", x.shape)
    _float(w, "w", (experts, n, k) if grouped else (n, k), x)
    if grouped:
        _index(offsets, "offsets", (experts + 1,), x)
    if bias is not None:
        _float(bias, "bias", (experts, n) if grouped else (n,), x)
        _check(bias.is_contiguous(), "bias: contiguous wanted")
    if residual is not None:
        _float(residual, "residual", (rows, n), x)
    made = []
    if out is None:
        out = torch.empty(rows, n, dtype=x.dtype, device=x.device)
        made.append(out)
    _float(out, "out", (rows, n), x)
    if preact is None and save_preact:
        preact = torch.empty(rows, n, dtype=x.dtype, device=x.device)
        made.append(preact)
    if preact is not None:
        _float(preact, "preact", (rows, n), x)
    d = _desc(x.shape, n, x.dtype, activation, experts if grouped else 0, (x, w, bias, residual, out, preact),
              ld_x=_ld(x, "x"), ld_w=_ld(w, "w"), ld_out=_ld(out, "out"), ld_residual=_ld(residual, "residual"),
              ld_preact=_ld(preact, "preact"))
    nbytes = capi.ccl_linear_workspace(d, grouped, False)
    with torch.cuda.device(x.device):
        ws = _workspace(nbytes, x.device)
        s = _stream(stream, x.device)
        if grouped:
            capi.ccl_grouped_linear(d, _ptr(offsets), _ptr(x), _ptr(w), _ptr(bias), _ptr(out), _ptr(preact), _ptr(ws),
                                    nbytes, s)
        else:
            capi.ccl_linear(d, _ptr(x), _ptr(w), _ptr(bias), _ptr(residual), _ptr(out), _ptr(preact), _ptr(ws),
                            nbytes, s)
        _own(stream, ws, *made)
    return out if preact is None else (out, preact)


def linear_backward(dout, x, w, preact=None, activation="none", bias=False, need_dx=True, need_dw=True, stream=None):
    """Gradients of ``linear``: [dx, dw] and, with ``bias``, dbias; a gradient that is not
    needed is left out of the list. The residual's gradient is dout itself. preact: what the
    forward pass saved (not used for activation "none")."""
    return _backward(dout, x, w, None, preact, activation, bias, need_dx, need_dw, stream)


def grouped_linear_backward(dout, x, w, offsets, preact=None, activation="none", bias=False, need_dx=True,
                            need_dw=True, stream=None):
    """Gradients of ``grouped_linear``: dx (zeros for rows of no group), dw (experts, out,
    in) and dbias (experts, out), zeros for an empty group."""
    return _backward(dout, x, w, offsets, preact, activation, bias, need_dx, need_dw, stream)


def _backward(dout, x, w, offsets, preact, activation, bias, need_dx, need_dw, stream):
    grouped = offsets is not None
    _check(isinstance(x, torch.Tensor) and x.dim() == 2, "x: a matrix wanted")
    _check(isinstance(w, torch.Tensor) and w.dim() == (3 if grouped else 2),
           "w: (experts, out, in) wanted" if grouped else "w: (out, in) wanted")
    rows, k = x.shape
    n = w.shape[-2]
    experts = w.shape[0] if grouped else 1
    _float(x, "x", x.shape)
    _float(w, "w", (experts, n, k) if grouped else (n, k), x)
    _float(dout, "dout", (rows, n), x)
    if grouped:
        _index(offsets, "offsets", (experts + 1,), x)
    _check(activation == "none" or preact is not None, "the activation's gradient needs preact")
    if activation == "none":
        preact = None
    if preact is not None:
        _float(preact, "preact", (rows, n), x)
    dx = torch.empty(rows, k, dtype=x.dtype, device=x.device) if need_dx else None
    dw = torch.empty(w.shape, dtype=x.dtype, device=x.device) if need_dw else None
    db = torch.empty(w.shape[:-1], dtype=x.dtype, device=x.device) if bias else None
    d = _desc(x.shape, n, x.dtype, activation, experts if grouped else 0, (dout, x, w, preact, dx, dw, db),
              ld_x=_ld(x, "x"), ld_w=_ld(w, "w"), ld_out=_ld(dout, "dout"), ld_preact=_ld(preact, "preact"))
    nbytes = capi.ccl_linear_workspace(d, grouped, True)
    with torch.cuda.device(x.device):
        ws = _workspace(nbytes, x.device)
        s = _stream(stream, x.device)
        tail = (_ptr(dout), _ptr(x), _ptr(w), _ptr(preact), _ptr(dx), _ptr(dw), _ptr(db), _ptr(ws), nbytes, s)
        if grouped:
            capi.ccl_grouped_linear_backward(d, _ptr(offsets), *tail)
        else:
            capi.ccl_linear_backward(d, *tail)
        _own(stream, ws, dx, dw, db)
    return [t for t in (dx, dw, db) if t is not None]


# ---- row exchange ---------------------------------------------------------------------
def expert_route(ids, experts, stream=None):
    """ids (tokens, choices) int32 -> (offsets (experts + 1), positions (tokens, choices),
    slots (tokens * choices)), int32: rows ordered by expert and, within an expert, by slot
    (the index of a choice in ids). positions: a choice's row, -1 where its id is not in
    [0, experts); slots: a row's choice, -1 for the rows from offsets[experts] on."""
    _check(isinstance(ids, torch.Tensor) and ids.dim() == 2, "ids: (tokens, choices) wanted")
    _index(ids, "ids", ids.shape, ids)
    tokens, choices = ids.shape
    nbytes = capi.ccl_expert_route_workspace(tokens, choices, experts)
    with torch.cuda.device(ids.device):
        offsets = torch.empty(experts + 1, dtype=torch.int32, device=ids.device)
        positions = torch.empty_like(ids)
        slots = torch.empty(tokens * choices, dtype=torch.int32, device=ids.device)
        ws = _workspace(nbytes, ids.device)
        capi.ccl_expert_route(_ptr(ids), tokens, choices, experts, _ptr(offsets), _ptr(positions), _ptr(slots),
                              _ptr(ws), nbytes, _stream(stream, ids.device))
        _own(stream, ws, offsets, positions, slots)
    return offsets, positions, slots


def expert_dispatch(x, slots, choices, out=None, stream=None):
    """rows[i] = x[slots[i] // choices], zeros where slots[i] is -1: x (tokens, width), rows
    (tokens * choices, width)."""
    _check(isinstance(x, torch.Tensor) and x.dim() == 2, "x: a matrix wanted")
    tokens, width = x.shape
    _float(x, "x", x.shape)
    _index(slots, "slots", (tokens * choices,), x)
    with torch.cuda.device(x.device):
        made = out is None
        if made:
            out = torch.empty(tokens * choices, width, dtype=x.dtype, device=x.device)
        _float(out, "out", (tokens * choices, width), x)
        capi.ccl_expert_dispatch(DTYPES[x.dtype], _ptr(x), _ld(x, "x"), _ptr(slots), tokens, choices, width, _ptr(out),
                                 _ld(out, "out"), _stream(stream, x.device))
        _own(stream, out if made else None)
    return out


def expert_combine(h, positions, gates=None, out=None, stream=None):
    """out[t] = sum over j of gates[t, j] h[positions[t, j]]: h (tokens * choices, width),
    gates (tokens, choices) float32 or None for ones. Without gates it is also the gradient
    of ``expert_dispatch``'s x from its rows' gradients."""
    _check(isinstance(h, torch.Tensor) and h.dim() == 2, "h: a matrix wanted")
    _check(isinstance(positions, torch.Tensor) and positions.dim() == 2, "positions: (tokens, choices) wanted")
    tokens, choices = positions.shape
    width = h.shape[1]
    _float(h, "h", (tokens * choices, width))
    _index(positions, "positions", positions.shape, h)
    if gates is not None:
        _float(gates, "gates", positions.shape)
        _check(gates.dtype == torch.float32 and gates.is_contiguous() and gates.device == h.device,
               "gates: contiguous float32 on h's device wanted")
    with torch.cuda.device(h.device):
        made = out is None
        if made:
            out = torch.empty(tokens, width, dtype=h.dtype, device=h.device)
        _float(out, "out", (tokens, width), h)
        capi.ccl_expert_combine(DTYPES[h.dtype], _ptr(h), _ld(h, "h"), _ptr(positions), _ptr(gates), tokens, choices,
                                width, _ptr(out), _ld(out, "out"), _stream(stream, h.device))
        _own(stream, out if made else None)
    return out


def expert_combine_backward(dout, h, positions, slots, gates=None, stream=None):
    """Gradients of ``expert_combine``: dh (tokens * choices, width) and dgates (tokens,
    choices) float32; positions and slots are the route's."""
    _check(isinstance(dout, torch.Tensor) and dout.dim() == 2, "dout: a matrix wanted")
    _check(isinstance(positions, torch.Tensor) and positions.dim() == 2, "positions: (tokens, choices) wanted")
    tokens, choices = positions.shape
    width = dout.shape[1]
    _float(dout, "dout", (tokens, width))
    _float(h, "h", (tokens * choices, width), dout)
    _index(positions, "positions", positions.shape, dout)
    _index(slots, "slots", (tokens * choices,), dout)
    if gates is not None:
        _float(gates, "gates", positions.shape)
        _check(gates.dtype == torch.float32 and gates.is_contiguous() and gates.device == h.device,
               "gates: contiguous float32 on h's device wanted")
    with torch.cuda.device(h.device):
        dh = torch.empty(tokens * choices, width, dtype=h.dtype, device=h.device)
        dgates = torch.empty(tokens, choices, dtype=torch.float32, device=h.device)
        capi.ccl_expert_combine_backward(DTYPES[h.dtype], _ptr(dout), _ld(dout, "dout"), _ptr(h), _ld(h, "h"),
                                         _ptr(positions), _ptr(slots), _ptr(gates), tokens, choices, width, _ptr(dh),
                                         0, _ptr(dgates), _stream(stream, h.device))
        _own(stream, dh, dgates)
    return dh, dgates
