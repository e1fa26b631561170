"""The products beside the collectives against their definitions in 64 bits."""

import pytest
import torch

from chunk_schedule_execution_amd import ops
from oracle import products as O
from products_util import TYPES, U32, backward_bounds, forward_bounds, normal, within

pytestmark = pytest.mark.gpu

# rows, in, out: single values and rows, sizes around tiles and vectors, long ones
SHAPES = [(1, 1, 1), (1, 8, 16), (1, 64, 40), (2, 7, 5), (3, 4096, 24), (4, 1024, 1024), (15, 33, 130), (16, 64, 64),
          (17, 100, 33), (31, 520, 72), (33, 256, 264), (63, 257, 65), (64, 128, 128), (65, 65, 257), (100, 1000, 48),
          (128, 512, 256), (130, 72, 300), (255, 192, 513), (256, 64, 256), (257, 320, 512), (300, 1001, 77),
          (512, 2048, 128), (520, 136, 1032), (1000, 40, 8), (1111, 333, 259), (48, 16384, 16), (2, 16392, 9)]


def linear_case(rows, k, n, dtype, act, bias, residual, save, pad=0, seed=0, wide_out=0):
    t = TYPES[dtype]
    x = normal(seed + 1, rows, k + pad, dtype=t)[:, :k]
    w = normal(seed + 2, n, k + pad, dtype=t, scale=k ** -0.5)[:, :k]
    b = normal(seed + 3, n, dtype=t) if bias else None
    r = normal(seed + 4, rows, n + pad, dtype=t)[:, :n] if residual else None
    out = pre = None
    if wide_out:
        out = torch.full((rows, n + wide_out), 7.0, dtype=t, device="cuda:0")
        pre = torch.full((rows, n + wide_out), 7.0, dtype=t, device="cuda:0")
    got = ops.linear(x, w, bias=b, residual=r, activation=act, save_preact=save,
                     out=None if out is None else out[:, :n], preact=None if pre is None else pre[:, :n])
    want, z, big = O.linear(x, w, bias=b, residual=r, activation=act)
    bo, bz = forward_bounds(want, z, big, k, t, r)
    if save or wide_out:
        within(got[0], want, bo, "out")
        within(got[1], z, bz, "preact")
    else:
        within(got, want, bo, "out")
    if wide_out:  # nothing beside the rows was written
        assert bool((out[:, n:] == 7.0).all()) and bool((pre[:, n:] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,n", SHAPES)
def test_linear(rows, k, n, dtype):
    linear_case(rows, k, n, dtype, "silu", bias=True, residual=True, save=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("rows,k,n", [(5, 96, 72), (200, 96, 136)])
def test_linear_activations(rows, k, n, act, dtype):
    linear_case(rows, k, n, dtype, act, bias=False, residual=False, save=True)
    linear_case(rows, k, n, dtype, act, bias=True, residual=False, save=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [1, 3, 8, 64])
@pytest.mark.parametrize("rows,k,n", [(3, 136, 40), (70, 136, 72), (300, 264, 264)])
def test_linear_strides(rows, k, n, pad, dtype):
    linear_case(rows, k, n, dtype, "gelu", bias=True, residual=True, save=True, pad=pad)
    linear_case(rows, k, n, dtype, "none", bias=False, residual=False, save=False, pad=pad, wide_out=pad)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [2, 40, 300])
def test_linear_from_an_unaligned_base(rows, dtype):
    t = TYPES[dtype]
    k, n = 128, 96
    x = normal(1, rows * k + 1, dtype=t)[1:].view(rows, k)
    w = normal(2, n * k + 3, dtype=t, scale=k ** -0.5)[3:].view(n, k)
    got = ops.linear(x, w)
    want, z, big = O.linear(x, w)
    within(got, want, forward_bounds(want, z, big, k, t)[0], "out")
    dout = normal(3, rows * n + 1, dtype=t)[1:].view(rows, n)
    grads, bigs = O.linear_backward(dout, x, w)
    for g, v, b, name in zip(ops.linear_backward(dout, x, w, bias=True), grads,
                             backward_bounds(grads, bigs, (n, rows, rows), t, False), ("dx", "dw", "dbias")):
        within(g, v, b, name)


def test_linear_of_no_rows():
    x, w = normal(1, 0, 24, dtype=torch.bfloat16), normal(2, 16, 24, dtype=torch.bfloat16)
    assert ops.linear(x, w).shape == (0, 16)
    dx, dw, db = ops.linear_backward(normal(3, 0, 16, dtype=torch.bfloat16), x, w, bias=True)
    assert dx.shape == (0, 24) and not bool(dw.any()) and not bool(db.any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_special_values(dtype):
    """Infinities and NaN reach the outputs that their rows and columns feed, and no others."""
    t = TYPES[dtype]
    for rows in (3, 40, 300):
        x, w = normal(1, rows, 160, dtype=t), normal(2, 200, 160, dtype=t)
        x[1, 5], w[3, 7], w[100, 9] = float("inf"), float("nan"), float("-inf")
        got = ops.linear(x, w, activation="relu")
        want = O.act(torch.mm(x.double(), w.double().t()), "relu")
        zs = torch.mm(x.double(), w.double().t())
        want = torch.where(zs.isnan(), zs, want)
        fine = want.isfinite()
        assert bool((got.isnan() == want.isnan()).all())
        assert bool((got[want.isinf()].double() == want[want.isinf()]).all())
        big = torch.mm(x.double().abs(), w.double().abs().t())
        bound = forward_bounds(want, zs, big, 160, t)[0]
        within(torch.where(fine, got.double(), 0.0), torch.where(fine, want, 0.0), torch.where(fine, bound, 1.0), "out")


def slope_slack(act, dout, preact):
    """dz's error from the slope function in fp32: a few steps of 1 (and of z exp(-z^2 / 2),
    below 1) times dout."""
    return 0.0 if act in ("none", "relu") else 16 * U32 * dout.double().abs()


def backward_case(rows, k, n, dtype, act, pad=0, offsets=None, experts=0):
    t = TYPES[dtype]
    x = normal(1, rows, k + pad, dtype=t)[:, :k]
    shape = (experts, n, k) if experts else (n, k)
    w = normal(2, *shape, dtype=t, scale=k ** -0.5)
    pre = normal(3, rows, n + pad, dtype=t)[:, :n]
    dout = normal(4, rows, n + pad, dtype=t)[:, :n]
    grads, bigs = O.linear_backward(dout, x, w, offsets, pre, act)
    slack = slope_slack(act, dout, pre)
    if act not in ("none", "relu"):  # the same sums over the slope's error
        _, more = O.linear_backward(slack, x, w, offsets, None, "none")
    if experts:
        o = torch.tensor(offsets, dtype=torch.int32, device="cuda:0")
        got = ops.grouped_linear_backward(dout, x, w, o, preact=pre, activation=act, bias=True)
    else:
        got = ops.linear_backward(dout, x, w, preact=pre, activation=act, bias=True)
    bounds = backward_bounds(grads, bigs, (n, rows, rows), t, act not in ("none",))
    for i, (g, v, b, name) in enumerate(zip(got, grads, bounds, ("dx", "dw", "dbias"))):
        if act not in ("none", "relu"):
            b = b + 1.01 * more[i]
        within(g, v, b, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,n", SHAPES)
def test_linear_backward(rows, k, n, dtype):
    backward_case(rows, k, n, dtype, "gelu")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("pad", [0, 5, 8])
def test_linear_backward_activations(act, dtype, pad):
    backward_case(150, 136, 72, dtype, act, pad)


@pytest.mark.parametrize("need", [(True, False, False), (False, True, False), (False, False, True)])
def test_linear_backward_in_parts(need):
    x, w = normal(1, 70, 48, dtype=torch.bfloat16), normal(2, 56, 48, dtype=torch.bfloat16)
    pre, dout = normal(3, 70, 56, dtype=torch.bfloat16), normal(4, 70, 56, dtype=torch.bfloat16)
    whole = ops.linear_backward(dout, x, w, preact=pre, activation="silu", bias=True)
    part = ops.linear_backward(dout, x, w, preact=pre, activation="silu", need_dx=need[0], need_dw=need[1],
                               bias=need[2])
    assert len(part) == 1 and torch.equal(part[0], whole[need.index(True)])


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_gradients_against_differences(act):
    """<gradient, direction> against central differences of the definition in 64 bits: the
    differences' own error is of the order step^2 = 1e-8 (times third derivatives below 4
    and sums below 1e3), the fp32 gradients' is 1e-6 of the sums."""
    rows, k, n, step = 37, 24, 29, 1e-4
    x, w, b = normal(1, rows, k), normal(2, n, k, scale=k ** -0.5), normal(3, n)
    dout = normal(4, rows, n)
    _, preact = ops.linear(x, w, bias=b, activation=act, save_preact=True)
    got = ops.linear_backward(dout, x, w, preact=preact, activation=act, bias=True)
    at = [x.double(), w.double(), b.double()]
    for i, g in enumerate(got):
        d = normal(10 + i, *at[i].shape).double()
        side = []
        for sign in (1, -1):
            p = list(at)
            p[i] = p[i] + sign * step * d
            side.append((O.linear(p[0], p[1], bias=p[2], activation=act)[0] * dout.double()).sum())
        want = float((side[0] - side[1]) / (2 * step))
        assert abs(float((g.double() * d).sum()) - want) <= 1e-5 * float((g.double() * d).abs().sum()) + 4e-5


# ---- grouped ------------------------------------------------------------------------------
GROUPS = {
    "even": [0, 40, 80, 120, 160],
    "ragged": [0, 1, 66, 66, 150, 160],
    "empty ends": [0, 0, 0, 97, 160, 160],
    "rest": [0, 30, 31, 100],          # rows 100 .. 159 belong to no group
    "none": [0, 0, 0, 0],
    "one": [0, 160],
    "tiny": [0, 1, 2, 3, 3, 4, 160],
    "disordered": [5, 50, 20, 300, 40, 160],  # read as 0, 50, 50, 160, 160, 160
    "negative": [0, -7, 60, 160],
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("k,n", [(64, 72), (33, 130)])
def test_grouped_linear(name, k, n, dtype):
    grouped_case(160, k, n, GROUPS[name], dtype, "silu")


def grouped_case(rows, k, n, offsets, dtype, act, bias=True):
    t, e = TYPES[dtype], len(offsets) - 1
    x, w = normal(1, rows, k, dtype=t), normal(2, e, n, k, dtype=t, scale=k ** -0.5)
    b = normal(3, e, n, dtype=t) if bias else None
    o = torch.tensor(offsets, dtype=torch.int32, device="cuda:0")
    out, pre = ops.grouped_linear(x, w, o, bias=b, activation=act, save_preact=True)
    want, z, big = O.linear(x, w, offsets, bias=b, activation=act)
    bo, bz = forward_bounds(want, z, big, k, t)
    within(out, want, bo, "out")
    within(pre, z, bz, "preact")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,experts,k,n", [(1, 8, 64, 64), (8, 200, 72, 40), (64, 64, 256, 128), (600, 3, 264, 520),
                                              (1500, 7, 333, 515), (2000, 130, 64, 96)])
def test_grouped_linear_sizes(rows, experts, k, n, dtype):
    cuts = torch.randint(0, rows + 1, (experts - 1,), generator=torch.Generator().manual_seed(5)).sort().values
    offsets = [0] + cuts.tolist() + [rows]
    grouped_case(rows, k, n, offsets, dtype, "gelu_tanh")
    backward_case(rows, k, n, dtype, "gelu_tanh", offsets=offsets, experts=experts)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_grouped_linear_backward(name, act, dtype):
    o = GROUPS[name]
    backward_case(160, 72, 136, dtype, act, offsets=o, experts=len(o) - 1)
    backward_case(160, 35, 43, dtype, act, offsets=o, experts=len(o) - 1)


def test_grouped_rows_of_no_group_are_zero():
    x, w = normal(1, 100, 64, dtype=torch.bfloat16), normal(2, 3, 64, 64, dtype=torch.bfloat16)
    x[60:] = float("nan")
    b = normal(3, 3, 64, dtype=torch.bfloat16)
    o = torch.tensor([0, 10, 30, 60], dtype=torch.int32, device="cuda:0")
    out, pre = ops.grouped_linear(x, w, o, bias=b, activation="silu", save_preact=True)
    assert not bool(out[60:].any()) and not bool(pre[60:].any()) and bool(out[:60].isfinite().all())
    dout = normal(4, 100, 64, dtype=torch.bfloat16)
    dout[60:] = float("nan")
    dx, dw, db = ops.grouped_linear_backward(dout, x, w, o, preact=pre, activation="silu", bias=True)
    assert not bool(dx[60:].any())
    assert bool(dx.isfinite().all()) and bool(dw.isfinite().all()) and bool(db.isfinite().all())


def test_grouped_nan_stays_in_its_group():
    x, w = normal(1, 90, 72, dtype=torch.bfloat16), normal(2, 3, 40, 72, dtype=torch.bfloat16)
    o = torch.tensor([0, 31, 62, 90], dtype=torch.int32, device="cuda:0")
    dout = normal(4, 90, 40, dtype=torch.bfloat16)
    clean = [t.clone() for t in ops.grouped_linear_backward(dout, x, w, o)]
    first = ops.grouped_linear(x, w, o)
    x[31:62], w[1] = float("nan"), float("inf")
    got = ops.grouped_linear(x, w, o)
    assert torch.equal(got[:31], first[:31]) and torch.equal(got[62:], first[62:])
    dx, dw = ops.grouped_linear_backward(dout, x, w, o)
    assert torch.equal(dx[:31], clean[0][:31]) and torch.equal(dx[62:], clean[0][62:])
    assert torch.equal(dw[0], clean[1][0]) and torch.equal(dw[2], clean[1][2])


# ---- the largest tiles, several of them per workgroup ---------------------------------------
@pytest.mark.parametrize("rows,k,n,act,residual,save,pad", [
    (4000, 1000, 4088, "gelu", True, True, 8), (8100, 1000, 4088, "none", False, False, 0),
    (4001, 1001, 4085, "silu", True, True, 3)])
def test_linear_of_many_large_tiles(rows, k, n, act, residual, save, pad):
    linear_case(rows, k, n, "bf16", act, bias=True, residual=residual, save=save, pad=pad)


@pytest.mark.parametrize("pad", [0, 5])
def test_linear_backward_of_many_large_tiles(pad):
    backward_case(4000, 4088, 4096, "bf16", "gelu", pad)


def test_grouped_linear_of_many_large_tiles():
    offsets = [0, 1, 2700, 2700, 6111, 7950]  # the last 50 rows belong to no group
    grouped_case(8000, 2000, 4088, offsets, "bf16", "gelu_tanh")
    backward_case(8000, 2000, 4088, "bf16", "silu", offsets=offsets, experts=5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,n", [(40, 16384, 300), (130, 8200, 130), (500, 4104, 72), (33, 16400, 1)])
def test_linear_of_split_sums(rows, k, n, dtype):
    linear_case(rows, k, n, dtype, "silu", bias=True, residual=True, save=True)
    backward_case(n, rows, k, dtype, "gelu")
    backward_case(k, rows, n, dtype, "none")


# ---- as a user has them ---------------------------------------------------------------------
def test_same_bits_again_and_on_another_stream():
    x, w = normal(1, 700, 520, dtype=torch.bfloat16), normal(2, 264, 520, dtype=torch.bfloat16)
    pre, dout = normal(3, 700, 264, dtype=torch.bfloat16), normal(4, 700, 264, dtype=torch.bfloat16)

    def run(stream=None):
        return [ops.linear(x, w, activation="gelu", stream=stream)] + ops.linear_backward(
            dout, x, w, preact=pre, activation="gelu", bias=True, stream=stream)

    first = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for again in (run(), run(side), run(side.cuda_stream)):
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    with torch.cuda.stream(side):
        again = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("rows", [3, 300])
def test_graph_replays(rows):
    """Captured once, replayed with new inputs, eager work and synchronizations between."""
    x, w = normal(1, rows, 264, dtype=torch.bfloat16), normal(2, 4, 136, 264, dtype=torch.bfloat16)
    o = torch.tensor([0, rows // 3, rows // 3, rows - 1, rows], dtype=torch.int32, device="cuda:0")
    dout = normal(4, rows, 136, dtype=torch.bfloat16)

    def run():
        out, pre = ops.grouped_linear(x, w, o, activation="silu", save_preact=True)
        return [out, ops.linear(x, w[0])] + ops.grouped_linear_backward(
            dout, x, w, o, preact=pre, activation="silu", bias=True)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for i in range(4):
        x.copy_(normal(20 + i, rows, 264, dtype=torch.bfloat16))
        dout.copy_(normal(30 + i, rows, 136, dtype=torch.bfloat16))
        o.copy_(torch.tensor([0, i % rows, i % rows, rows - 1, rows], dtype=torch.int32))
        want = run()
        torch.cuda.synchronize()
        for t in held:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), i


def test_rows_beyond_four_gigabytes():
    """Element offsets past 32 bits in x, out and the weight gradient's summed rows."""
    rows, k, n = (1 << 31) // 4096 + 513, 4096 + 8, 32
    x = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda:0")
    pick = [0, 1, rows // 2, rows - 514, rows - 2, rows - 1]
    x[pick] = normal(1, len(pick), k, dtype=torch.bfloat16)
    w = normal(2, n, k, dtype=torch.bfloat16, scale=k ** -0.5)
    got = ops.linear(x, w)
    want, z, big = O.linear(x[pick], w)
    within(got[pick], want, forward_bounds(want, z, big, k, torch.bfloat16)[0], "out")
    dout = normal(3, rows, n, dtype=torch.bfloat16)
    dx, dw = ops.linear_backward(dout, x, w)
    grads, bigs = O.linear_backward(dout[pick], x[pick], w)
    bx, bw, _ = backward_bounds(grads, bigs, (n, rows, rows), torch.bfloat16, False)
    within(dx[pick], grads[0], bx, "dx")
    within(dw, grads[1], bw, "dw")
