"""Refusals, workspace queries and streams of the choice of experts, layer norm and the cross
entropy: no GPU, nothing launched. Every refused call names an error before any device work."""

import types

import pytest
import torch

from chunk_schedule_execution_amd import capi, ops
from oracle import layers as L

P = 1 << 20  # an aligned address that no refused call looks at
BAD, NOT = capi.CCL_ERR_INVALID_ARGUMENT, capi.CCL_ERR_UNSUPPORTED
BIG = 1 << 60


def refused(status, f, *args, text=""):
    with pytest.raises(capi.CCLError) as e:
        f(*args)
    assert e.value.status == status and text in capi.ccl_last_error_detail() != ""


# ---- the choice of experts ------------------------------------------------------------------
def select_desc(**kw):
    d = dict(dtype=capi.CCL_BF16, score=capi.CCL_SCORE_SOFTMAX, tokens=8, experts=24, choices=4, groups=4,
             kept_groups=2, group_best=2, renormalise=1, scale=1.0)
    d.update(kw)
    return capi.ccl_select_desc(**d)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=capi.CCL_I32), NOT), (dict(score=2), NOT), (dict(score=-1), NOT), (dict(tokens=-1), BAD),
    (dict(tokens=1 << 31), BAD), (dict(experts=0), BAD), (dict(experts=1025, groups=1, kept_groups=1), BAD),
    (dict(choices=0), BAD), (dict(choices=25), BAD), (dict(experts=128, choices=65), BAD), (dict(groups=0), BAD),
    (dict(groups=5), BAD), (dict(experts=130, groups=65), BAD), (dict(kept_groups=0), BAD), (dict(kept_groups=5), BAD),
    (dict(group_best=0), BAD), (dict(group_best=3), BAD), (dict(renormalise=2), BAD), (dict(scale=float("nan")), BAD),
    (dict(scale=float("inf")), BAD), (dict(ld_logits=23), BAD), (dict(ld_logits=(1 << 22) + 1), BAD),
    (dict(ld_dlogits=-1), BAD)])
def test_select_refuses_bad_descriptors(bad, status):
    d = select_desc(**bad)
    refused(status, capi.ccl_expert_select, d, P, P, P, P)
    refused(status, capi.ccl_expert_select_backward, d, P, P, P, P)


def test_select_refuses_bad_pointers():
    names = ("logits", "bias", "ids", "gates")
    for i, name in enumerate(names):
        for bad in (0, P + 1):
            if name == "bias" and not bad:
                continue
            p = [P] * 4
            p[i] = bad
            refused(BAD, capi.ccl_expert_select, select_desc(), *p, text=name)
    for i, name in enumerate(("dgates", "logits", "ids", "dlogits")):
        for bad in (0, P + 1):
            p = [P] * 4
            p[i] = bad
            refused(BAD, capi.ccl_expert_select_backward, select_desc(), *p, text=name)


def test_null_descriptors():
    lib = capi.lib()
    assert lib.ccl_expert_select(None, P, P, P, P, 0) == BAD
    assert lib.ccl_expert_select_backward(None, P, P, P, P, 0) == BAD
    assert lib.ccl_layer_norm(None, P, P, P, P, P, P, P, P, 0) == BAD
    assert lib.ccl_layer_norm_backward_workspace(None) == BAD
    assert lib.ccl_layer_norm_backward(None, P, P, P, P, P, P, P, P, P, P, BIG, 0) == BAD
    assert lib.ccl_linear_cross_entropy_workspace(None, 0) == BAD
    assert lib.ccl_linear_cross_entropy(None, P, P, P, P, P, P, P, BIG, 0) == BAD
    assert lib.ccl_linear_cross_entropy_backward(None, P, P, P, P, P, P, P, P, BIG, 0) == BAD


# ---- layer norm -------------------------------------------------------------------------------
def norm_desc(**kw):
    d = dict(dtype=capi.CCL_BF16, eps=1e-5, rows=8, width=40)
    d.update(kw)
    return capi.ccl_norm_desc(**d)


NORM = ["x", "residual", "weight", "bias", "out", "total", "mean", "rstd"]
NORM_BACKWARD = ["dout", "x", "mean", "rstd", "weight", "dtotal", "dx", "dweight", "dbias"]


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=capi.CCL_I32), NOT), (dict(eps=-1e-6), BAD), (dict(eps=float("nan")), BAD),
    (dict(eps=float("inf")), BAD), (dict(rows=-1), BAD), (dict(rows=1 << 31), BAD), (dict(width=0), BAD),
    (dict(width=(1 << 20) + 1), BAD)] + [({f"ld_{n}": v}, BAD) for n in ("x", "residual", "out", "total", "dtotal", "dx")
                                         for v in (39, -40, (1 << 22) + 1)])
def test_norm_refuses_bad_descriptors(bad, status):
    d = norm_desc(**bad)
    refused(status, capi.ccl_layer_norm, d, *[P] * 8)
    refused(status, capi.ccl_layer_norm_backward_workspace, d)
    refused(status, capi.ccl_layer_norm_backward, d, *[P] * 9, P, BIG)


@pytest.mark.parametrize("name", NORM)
def test_norm_refuses_bad_pointers(name):
    a = dict.fromkeys(NORM, P)
    a[name] = P + 1
    refused(BAD, capi.ccl_layer_norm, norm_desc(), *a.values(), text=name)
    if name in ("x", "out", "mean", "rstd"):  # mean and rstd: both or neither
        a[name] = 0
        refused(BAD, capi.ccl_layer_norm, norm_desc(), *a.values(), text=name)
    if name == "residual":  # total is wanted
        a[name] = 0
        refused(BAD, capi.ccl_layer_norm, norm_desc(), *a.values(), text="total")


@pytest.mark.parametrize("name", NORM_BACKWARD)
def test_norm_backward_refuses_bad_pointers(name):
    a = dict.fromkeys(NORM_BACKWARD, P)
    a[name] = P + 1
    refused(BAD, capi.ccl_layer_norm_backward, norm_desc(), *a.values(), P, BIG, text=name)
    if name in ("dout", "x", "mean", "rstd"):
        a[name] = 0
        refused(BAD, capi.ccl_layer_norm_backward, norm_desc(), *a.values(), P, BIG, text=name)


def test_norm_workspace_is_checked():
    d = norm_desc()
    need = capi.ccl_layer_norm_backward_workspace(d)
    assert need > 0
    for ws, have in ((0, need), (P, need - 1), (P + 8, need)):
        refused(BAD, capi.ccl_layer_norm_backward, d, *[P] * 9, ws, have, text="workspace")
    for rows in (0, 1, 511, 100000, 2**31 - 1):
        for width in (1, 4096, 1 << 20):
            need = capi.ccl_layer_norm_backward_workspace(norm_desc(rows=rows, width=width))
            assert 0 < need <= 1024 * 2 * 4 * width + 16


# ---- cross entropy ------------------------------------------------------------------------------
def loss_desc(**kw):
    d = dict(dtype=capi.CCL_BF16, rows=8, in_features=40, vocabulary=100, first=-1)
    d.update(kw)
    return capi.ccl_cross_entropy_desc(**d)


LOSS = ["x", "w", "targets", "loss", "lse", "picked"]
LOSS_BACKWARD = ["dloss", "x", "w", "targets", "lse", "dx", "dw"]


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=capi.CCL_I32), NOT), (dict(flags=2), BAD), (dict(rows=-1), BAD), (dict(rows=1 << 31), BAD),
    (dict(in_features=0), BAD), (dict(in_features=(1 << 20) + 1), BAD), (dict(vocabulary=0), BAD),
    (dict(vocabulary=(1 << 20) + 1), BAD), (dict(first=-2), BAD), (dict(first=2**31 - 100), BAD)] +
    [({f"ld_{n}": v}, BAD) for n in ("x", "w", "dx", "dw") for v in (39, -1, (1 << 22) + 1)])
def test_cross_entropy_refuses_bad_descriptors(bad, status):
    d = loss_desc(**bad)
    for backward in (False, True):
        refused(status, capi.ccl_linear_cross_entropy_workspace, d, backward)
    refused(status, capi.ccl_linear_cross_entropy, d, *[P] * 6, P, BIG)
    refused(status, capi.ccl_linear_cross_entropy_backward, d, *[P] * 7, P, BIG)


@pytest.mark.parametrize("name", LOSS)
def test_cross_entropy_refuses_bad_pointers(name):
    a = dict.fromkeys(LOSS, P)
    for bad in (P + 1, P + 2) if name in ("x", "w") else (P + 2,):
        a[name] = bad
        refused(BAD, capi.ccl_linear_cross_entropy, loss_desc(), *a.values(), P, BIG, text=name)
    if name in ("x", "w", "targets", "lse"):
        a[name] = 0
        refused(BAD, capi.ccl_linear_cross_entropy, loss_desc(), *a.values(), P, BIG)


@pytest.mark.parametrize("name", LOSS_BACKWARD)
def test_cross_entropy_backward_refuses_bad_pointers(name):
    a = dict.fromkeys(LOSS_BACKWARD, P)
    a[name] = P + 2
    refused(BAD, capi.ccl_linear_cross_entropy_backward, loss_desc(), *a.values(), P, BIG, text=name)
    if name not in ("dx", "dw"):
        a[name] = 0
        refused(BAD, capi.ccl_linear_cross_entropy_backward, loss_desc(), *a.values(), P, BIG)


def test_cross_entropy_of_a_shard_gives_no_loss():
    refused(BAD, capi.ccl_linear_cross_entropy, loss_desc(first=0), *[P] * 6, P, BIG, text="loss")


def test_cross_entropy_workspace_is_checked():
    for d in (loss_desc(), loss_desc(in_features=41), loss_desc(flags=capi.CCL_LINEAR_UNALIGNED)):
        for backward, call in ((False, lambda *ws: capi.ccl_linear_cross_entropy(d, *[P] * 6, *ws)),
                               (True, lambda *ws: capi.ccl_linear_cross_entropy_backward(d, *[P] * 7, *ws))):
            need = capi.ccl_linear_cross_entropy_workspace(d, backward)
            assert need > 0
            for ws in ((0, need), (P, need - 1), (P + 8, need)):
                refused(BAD, call, *ws, text="workspace")


@pytest.mark.parametrize("dtype", [capi.CCL_F32, capi.CCL_BF16])
@pytest.mark.parametrize("rows", [0, 1, 17, 1000, 65536, 2**31 - 1])
def test_cross_entropy_workspace_of_every_size(rows, dtype):
    """Far below what the logits would take where those are large."""
    size = 4 if dtype == capi.CCL_F32 else 2
    for k, v in ((1, 1), (8, 8), (33, 1 << 20), (1 << 20, 33), (4096, 131072)):
        d = loss_desc(dtype=dtype, rows=rows, in_features=k, vocabulary=v)
        forward, backward = (capi.ccl_linear_cross_entropy_workspace(d, b) for b in (False, True))
        assert forward >= 0 and backward >= 0
        if k % 8 == 0:
            # a pair for 32 logits; small products' sums go through memory
            assert forward <= max(rows * ((v + 31) // 32 * 8 + 8) + 64, 256 << 20)
            dz = rows * max(8192 + 256, (512 << 20) // max(1, rows * size) + 256) * size
            assert backward <= dz + 17 * (rows + v) * (k + 16) * 4 + (256 << 20)


def test_join_refuses_bad_arguments():
    for shards, rows in ((0, 8), (65537, 8), (2, -1), (2, 1 << 31)):
        refused(BAD, capi.ccl_cross_entropy_join, shards, rows, P, P, P, P, P)
    for i, name in enumerate(("lse_parts", "picked_parts", "targets", "loss", "lse")):
        for bad in (0, P + 2):
            p = [P] * 5
            p[i] = bad
            refused(BAD, capi.ccl_cross_entropy_join, 2, 8, *p, text=name)


def test_calls_of_no_rows_are_done_at_once():
    capi.ccl_expert_select(select_desc(tokens=0), 0, 0, 0, 0)
    capi.ccl_expert_select_backward(select_desc(tokens=0), 0, 0, 0, 0)
    capi.ccl_layer_norm(norm_desc(rows=0), 0, 0, 0, 0, 0, 0, 0, 0)
    capi.ccl_linear_cross_entropy(loss_desc(rows=0), 0, 0, 0, 0, 0, 0, 0, 0)
    capi.ccl_cross_entropy_join(1, 0, 0, 0, 0, 0, 0)
    capi.ccl_layer_norm_backward(norm_desc(), P, P, P, P, 0, 0, 0, 0, 0, 0, 0)  # no gradient wanted
    capi.ccl_linear_cross_entropy_backward(loss_desc(), P, P, P, P, P, 0, 0, 0, 0)


# ---- the wrappers ---------------------------------------------------------------------------------
class Fake(torch.Tensor):
    """A host tensor that says it lies on GPU 0: for checks that come before any device work."""

    is_cuda = True

    def get_device(self):
        return 0


def fake(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Fake)


def i32(*shape):
    return fake(*shape, dtype=torch.int32)


WRONG = {
    "select: a vector": lambda: ops.expert_select(fake(8), 2),
    "select: half": lambda: ops.expert_select(fake(4, 8, dtype=torch.float16), 2),
    "select: unknown score": lambda: ops.expert_select(fake(4, 8), 2, score="relu"),
    "select: bias of another type": lambda: ops.expert_select(fake(4, 8), 2, bias=fake(8, dtype=torch.bfloat16)),
    "select: bias of another length": lambda: ops.expert_select(fake(4, 8), 2, bias=fake(7)),
    "select: more choices than experts": lambda: ops.expert_select(fake(4, 8), 9),
    "select: no choices": lambda: ops.expert_select(fake(4, 8), 0),
    "select: columns apart": lambda: ops.expert_select(fake(8, 4).t(), 2),
    "select backward: ids of other tokens": lambda: ops.expert_select_backward(fake(3, 2), fake(4, 8), i32(3, 2)),
    "select backward: 64-bit ids": lambda: ops.expert_select_backward(fake(4, 2), fake(4, 8),
                                                                      fake(4, 2, dtype=torch.int64)),
    "select backward: gates of another shape": lambda: ops.expert_select_backward(fake(4, 3), fake(4, 8), i32(4, 2)),
    "norm: residual of another shape": lambda: ops.layer_norm(fake(4, 8), residual=fake(4, 9)),
    "norm: weight of another type": lambda: ops.layer_norm(fake(4, 8), weight=fake(8, dtype=torch.bfloat16)),
    "norm: total without a residual": lambda: ops.layer_norm(fake(4, 8), total=fake(4, 8)),
    "norm: overlapping rows": lambda: ops.layer_norm(fake(1, 8).expand(4, 8)),
    "norm: out of another shape": lambda: ops.layer_norm(fake(4, 8), out=fake(5, 8)),
    "norm backward: statistics of other rows": lambda: ops.layer_norm_backward(fake(4, 8), fake(4, 8), fake(3), fake(4)),
    "norm backward: dout of another type": lambda: ops.layer_norm_backward(fake(4, 8, dtype=torch.bfloat16), fake(4, 8),
                                                                           fake(4), fake(4)),
    "norm backward: dtotal of another shape": lambda: ops.layer_norm_backward(fake(4, 8), fake(4, 8), fake(4), fake(4),
                                                                              dtotal=fake(4, 7)),
    "loss: w of another length": lambda: ops.linear_cross_entropy(fake(4, 8), fake(6, 9), i32(4)),
    "loss: w of another type": lambda: ops.linear_cross_entropy(fake(4, 8), fake(6, 8, dtype=torch.bfloat16), i32(4)),
    "loss: 64-bit targets": lambda: ops.linear_cross_entropy(fake(4, 8), fake(6, 8), fake(4, dtype=torch.int64)),
    "loss: a shard below 0": lambda: ops.linear_cross_entropy(fake(4, 8), fake(6, 8), i32(4), shard=-1),
    "loss backward: dloss of other rows": lambda: ops.linear_cross_entropy_backward(fake(5), fake(4, 8), fake(6, 8),
                                                                                    i32(4), fake(4)),
    "loss backward: lse of another type": lambda: ops.linear_cross_entropy_backward(
        fake(4), fake(4, 8), fake(6, 8), i32(4), fake(4, dtype=torch.bfloat16)),
    "join: a vector": lambda: ops.cross_entropy_join(fake(4), fake(4), i32(4)),
    "join: other rows": lambda: ops.cross_entropy_join(fake(2, 4), fake(2, 5), i32(4)),
}


@pytest.mark.parametrize("name", list(WRONG))
def test_wrappers_refuse(name):
    with pytest.raises(ValueError):
        WRONG[name]()


def test_wrappers_refuse_host_tensors():
    x = torch.zeros(4, 8)
    for f in (lambda: ops.expert_select(x, 2), lambda: ops.layer_norm(x),
              lambda: ops.linear_cross_entropy(x, x, torch.zeros(4, dtype=torch.int32)),
              lambda: ops.cross_entropy_join(x, x, torch.zeros(8, dtype=torch.int32))):
        with pytest.raises(ValueError, match="GPU"):
            f()


# ---- streams: the wrappers over host tensors, torch's stream state replaced by a recorder -----------
class Stream:
    def __init__(self, cuda_stream):
        self.cuda_stream = cuda_stream


class Recorder:
    def __init__(self, monkeypatch):
        self.current, self.made, self.launched, self.recorded = Stream(7), [], [], []
        recorder = self

        class switch:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                self.outer, recorder.current = recorder.current, self.stream

            def __exit__(self, *a):
                recorder.current = self.outer

        def empty(*a, **kw):
            t = torch.empty(*a, **kw)
            self.made.append((t, self.current.cuda_stream))
            return t

        cuda = types.SimpleNamespace(
            Stream=Stream, ExternalStream=Stream, stream=switch, current_device=lambda: -1,
            set_device=lambda d: None, current_stream=lambda *a: self.current, default_stream=lambda *a: Stream(0))
        fake_torch = types.SimpleNamespace(
            **{n: getattr(torch, n) for n in ("Tensor", "float32", "bfloat16", "int32", "uint8")}, cuda=cuda, empty=empty)
        monkeypatch.setattr(ops, "torch", fake_torch)
        monkeypatch.setattr(ops, "_raw_stream", lambda device: self.current.cuda_stream)
        monkeypatch.setattr(ops, "_first", lambda t, name: -1)
        monkeypatch.setattr(ops, "_like", lambda *a: None)
        monkeypatch.setattr(torch.Tensor, "record_stream",
                            lambda t, s: self.recorded.append((t.data_ptr(), s.cuda_stream)), raising=False)
        for n in ("ccl_expert_select", "ccl_expert_select_backward", "ccl_layer_norm", "ccl_layer_norm_backward",
                  "ccl_linear_cross_entropy", "ccl_linear_cross_entropy_backward", "ccl_cross_entropy_join"):
            monkeypatch.setattr(ops.capi, n, lambda *a: self.launched.append(a[-1]))


def calls():
    x, w, row = torch.zeros(40, 33), torch.zeros(24, 33), torch.zeros(40)
    ids, targets = torch.zeros(40, 2, dtype=torch.int32), torch.zeros(40, dtype=torch.int32)
    parts = torch.zeros(3, 40)
    return {
        "expert_select": lambda s: ops.expert_select(x, 2, stream=s),
        "expert_select_backward": lambda s: ops.expert_select_backward(torch.zeros(40, 2), x, ids, stream=s),
        "layer_norm": lambda s: ops.layer_norm(x, residual=x, save_stats=True, stream=s),
        "layer_norm_backward": lambda s: ops.layer_norm_backward(x, x, row, row, weight=x[0], bias=True, stream=s),
        "linear_cross_entropy": lambda s: ops.linear_cross_entropy(x, w, targets, stream=s),
        "linear_cross_entropy_backward": lambda s: ops.linear_cross_entropy_backward(row, x, w, targets, row, stream=s),
        "cross_entropy_join": lambda s: ops.cross_entropy_join(parts, parts, targets, stream=s),
    }


@pytest.mark.parametrize("stream,handle", [(Stream(99), 99), (99, 99), (0, 0)])
@pytest.mark.parametrize("name", list(calls()))
def test_memory_comes_from_the_calls_stream(monkeypatch, name, stream, handle):
    r = Recorder(monkeypatch)
    out = calls()[name](stream)
    out = list(out) if isinstance(out, (tuple, list)) else [out]
    assert r.launched == [handle]
    assert len(r.made) >= len(out) and all(s == handle for _, s in r.made)
    # the outputs go to the stream that was current, which is current again
    assert sorted(r.recorded) == sorted((t.data_ptr(), 7) for t in out)
    assert r.current.cuda_stream == 7


@pytest.mark.parametrize("stream", [None, Stream(7), 7])
@pytest.mark.parametrize("name", list(calls()))
def test_the_current_stream_needs_nothing(monkeypatch, name, stream):
    r = Recorder(monkeypatch)
    calls()[name](stream)
    assert r.launched == [7] and all(s == 7 for _, s in r.made) and not r.recorded


@pytest.mark.parametrize("name", list(calls()))
def test_a_stream_of_another_device_is_refused(monkeypatch, name):
    r = Recorder(monkeypatch)
    other = Stream(99)
    other.device = types.SimpleNamespace(index=3)
    with pytest.raises(ValueError, match="stream"):
        calls()[name](other)
    assert not r.launched and not r.made


# ---- the oracle ------------------------------------------------------------------------------------
def test_oracle_select_by_hand():
    x = torch.tensor([[1.0, 3.0, 2.0, 3.0], [0.0, -float("inf"), 5.0, 1.0]])
    ids, gates = L.select(x, 2, renormalise=True)
    assert ids.tolist() == [[1, 3], [2, 3]] and gates[0].tolist() == [0.5, 0.5]
    # two groups of two: the first row's are worth 4 and 5, by the best value alone 3 and 3
    assert L.select(x, 1, groups=2, kept_groups=1, group_best=2)[0][0].tolist() == [3]
    assert L.select(x, 1, groups=2, kept_groups=1, group_best=1)[0][0].tolist() == [1]
    assert L.select(x[1:], 3, groups=2, kept_groups=1)[0].tolist() == [[2, 3, -1]]
    assert L.select(x, 1, bias=torch.tensor([0.0, -0.9, 0.0, -0.9]))[0].tolist() == [[2], [2]]


@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_oracle_select_gradient(score, renormalise):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(6, 9, generator=g, dtype=torch.float64).requires_grad_(True)
    ids = torch.randint(0, 9, (6, 3), generator=g, dtype=torch.int32)
    ids[2, 1], ids[3] = -1, 4
    dgates = torch.randn(6, 3, generator=g, dtype=torch.float64)
    (want,) = torch.autograd.grad((L.gates_of(x, ids, score, renormalise, 1.5) * dgates).sum(), x)
    got, big = L.select_backward(dgates, x.detach(), ids, score, renormalise, 1.5)
    assert float((got - want).abs().max()) < 1e-14 and bool((got.abs() <= big + 1e-300).all())


def test_oracle_gradients_of_norm_and_loss():
    g = torch.Generator().manual_seed(2)
    x, w, b, d = (torch.randn(*s, generator=g, dtype=torch.float64).requires_grad_(True) for s in ((5, 7), (7,), (7,), (5, 7)))
    out, _, mean, rstd = L.layer_norm(x, w, b)
    want = torch.autograd.grad((out * d.detach()).sum(), (x, w, b))
    got = L.layer_norm_backward(d.detach(), x.detach(), mean.detach(), rstd.detach(), w.detach())[0]
    assert all(float((a - c).abs().max()) < 1e-13 for a, c in zip(got, want))
    v = torch.randn(11, 7, generator=g, dtype=torch.float64).requires_grad_(True)
    targets = torch.tensor([0, 10, -1, 11, 3], dtype=torch.int32)
    dloss = torch.randn(5, generator=g, dtype=torch.float64)
    loss, lse, _, _ = L.cross_entropy(x, v, targets)
    want = torch.autograd.grad((loss * dloss).sum(), (x, v))
    dz, _, _ = L.logits_gradient(dloss, x.detach(), v.detach(), targets, lse.detach())
    assert float((dz @ v.detach() - want[0]).abs().max()) < 1e-13
    assert float((dz.t() @ x.detach() - want[1]).abs().max()) < 1e-13
