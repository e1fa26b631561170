"""Layer norm and its gradients against their definitions in 64 bits."""

import pytest
import torch

from chunk_schedule_execution_amd import ops
from layers_util import norm_backward_bounds, norm_bounds
from oracle import layers as L
from products_util import TYPES, normal, within

pytestmark = pytest.mark.gpu

# rows, width: single values, each number of packs in registers (a wave or a workgroup a row),
# odd widths, rows that registers do not hold
SHAPES = [(1, 1), (1, 8), (2, 7), (3, 64), (1, 4096), (4, 4096), (5, 1000), (17, 1001), (33, 2048), (9, 4104), (6, 8192),
          (3, 16384), (2, 16392), (3, 20001), (2, 40000), (1024, 8), (1025, 520), (1500, 1024), (1100, 2056), (1030, 4096),
          (1026, 333), (2050, 72), (1029, 4099)]


def rows_of(seed, rows, width, dtype, pad=0, offset=0.0):
    x = normal(seed, rows, width + pad) * (0.5 + normal(seed + 1, rows, 1).abs()) + offset
    return x.to(TYPES[dtype])[:, :width]


def parameters(width, dtype):
    t = TYPES[dtype]
    return (1 + normal(91, width, scale=0.3)).to(t), normal(92, width, dtype=t)


def forward(x, w, b, r, eps=1e-5):
    got = ops.layer_norm(x, weight=w, bias=b, residual=r, eps=eps, save_stats=True)
    want, h, mean, rstd = L.layer_norm(x, w, b, r, eps)
    bo, bh, bm, br = norm_bounds(want, h, mean, rstd, w, b, x.dtype)
    within(got[0], want, bo, "out")
    if r is not None:
        within(got[1], h, bh, "total")
    within(got[-2], mean, bm, "mean")
    within(got[-1], rstd, br, "rstd")
    # the same without the statistics
    plain = ops.layer_norm(x, weight=w, bias=b, residual=r, eps=eps)
    assert torch.equal(plain if r is None else plain[0], got[0])
    return got


def backward(x, w, dtotal, dout, mean, rstd):
    got = ops.layer_norm_backward(dout, x, mean, rstd, weight=w, dtotal=dtotal, bias=True)
    grads, big, columns = L.layer_norm_backward(dout, x, mean, rstd, w, dtotal)
    bounds = norm_backward_bounds(grads, big, columns, x.shape[0], x.shape[1], x.dtype)
    names = ("dx", "dweight", "dbias") if w is not None else ("dx", "dbias")
    keep = [i for i in range(3) if w is not None or i != 1]
    assert len(got) == len(names)
    for g, i, name in zip(got, keep, names):
        within(g, grads[i], bounds[i], name)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width", SHAPES)
def test_norm(rows, width, dtype):
    x, r = rows_of(1, rows, width, dtype), rows_of(3, rows, width, dtype)
    w, b = parameters(width, dtype)
    forward(x, w, b, None)
    out, total, mean, rstd = forward(x, w, b, r)
    dout = normal(7, rows, width, dtype=TYPES[dtype])
    backward(total, w, None, dout, mean, rstd)
    backward(total, w, r, dout, mean, rstd)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width", [(6, 72), (1030, 1000)])
def test_norm_with_and_without_each_argument(rows, width, dtype):
    x, r = rows_of(1, rows, width, dtype), rows_of(3, rows, width, dtype)
    dout = normal(7, rows, width, dtype=TYPES[dtype])
    for w in (None, parameters(width, dtype)[0]):
        for b in (None, parameters(width, dtype)[1]):
            _, mean, rstd = forward(x, w, b, None)
        all_three = backward(x, w, r, dout, mean, rstd)
        # each gradient alone gives the same bits
        for keep, kw in ((0, dict(need_dweight=False)), (len(all_three) - 1, dict(need_dx=False, need_dweight=False, bias=True)),
                         (1, dict(need_dx=False))):
            if keep == 1 and w is None:
                continue
            got = ops.layer_norm_backward(dout, x, mean, rstd, weight=w, dtotal=r, **kw)
            assert len(got) == 1 and torch.equal(got[0], all_three[keep])
    assert ops.layer_norm_backward(dout, x, mean, rstd, need_dx=False) == []


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("rows,width", [(5, 264), (1028, 264), (3, 20000)])
def test_norm_strides(rows, width, pad, dtype):
    """Rows in wider buffers, from bases off the 16-byte grid; nothing beside the rows is
    written."""
    t = TYPES[dtype]
    x, r = rows_of(1, rows, width, dtype, pad), normal(3, rows, width + pad, dtype=t)[:, pad:]
    w = normal(4, width + pad, dtype=t)[pad:]
    b = normal(5, width + pad, dtype=t)[pad:]
    out = torch.full((rows, width + pad), 7.0, dtype=t, device="cuda:0")
    total = torch.full((rows, width + pad), 7.0, dtype=t, device="cuda:0")
    got = ops.layer_norm(x, weight=w, bias=b, residual=r, out=out[:, pad:], total=total[:, :width], save_stats=True)
    want, h, mean, rstd = L.layer_norm(x, w, b, r)
    bo, bh, _, _ = norm_bounds(want, h, mean, rstd, w, b, t)
    within(got[0], want, bo, "out")
    within(got[1], h, bh, "total")
    assert bool((out[:, :pad] == 7.0).all()) and bool((total[:, width:] == 7.0).all())
    backward(got[1], w, r, normal(8, rows, width + pad, dtype=t)[:, pad:], got[2], got[3])


@pytest.mark.parametrize("width", [40, 4096, 17000])
def test_norm_of_rows_far_from_zero(width):
    """A mean 1000 times the spread: the variance comes from differences."""
    x = rows_of(1, 20, width, "f32", offset=1000.0)
    forward(x, None, None, None)
    x[3] = 5.0  # no spread at all: rstd is eps^-1/2
    out, mean, rstd = ops.layer_norm(x, save_stats=True, eps=1e-4)
    assert not bool(out[3].any()) and mean[3] == 5.0 and abs(float(rstd[3]) - 100.0) < 1e-3


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_of_rows_of_zeros(dtype):
    """Padding: such rows give the bias and, with no gradient of their own, add nothing."""
    x = rows_of(1, 1100, 200, dtype)
    w, b = parameters(200, dtype)
    dout = normal(2, 1100, 200, dtype=TYPES[dtype])
    x[600:], dout[600:] = 0.0, 0.0
    out, mean, rstd = forward(x, w, b, None)
    assert torch.equal(out[600:], b.expand(500, 200))
    dx, _, _ = backward(x, w, None, dout, mean, rstd)
    assert not bool(dx[600:].any())


def test_norm_special_values():
    """Infinities and NaN stay in their row; gradients of columns take them up."""
    for rows, width in ((6, 300), (1030, 4096), (4, 20000)):
        x = normal(1, rows, width, dtype=torch.bfloat16)
        plain, mean0, rstd0 = ops.layer_norm(x, save_stats=True)
        x[1, 5], x[3, 7] = float("inf"), float("nan")
        out, mean, rstd = ops.layer_norm(x, save_stats=True)
        fine = [i for i in range(rows) if i not in (1, 3)]
        assert torch.equal(out[fine], plain[fine]) and bool(out[3].isnan().all()) and bool(out[1].isnan().any())
        dx, dw, db = ops.layer_norm_backward(x.clone(), normal(1, rows, width, dtype=torch.bfloat16), mean0, rstd0,
                                             weight=torch.ones_like(x[0]), bias=True)
        assert bool(dx[fine].isfinite().all()) and bool(dx[3].isnan().all())
        assert bool(db[7].isnan()) and bool(db[5].isinf()) and bool(db[8:].isfinite().all())


def test_norm_of_no_rows():
    x = normal(1, 0, 48, dtype=torch.bfloat16)
    out, mean, rstd = ops.layer_norm(x, save_stats=True)
    assert out.shape == (0, 48) and mean.shape == rstd.shape == (0,)
    dx, dw, db = ops.layer_norm_backward(x, x, mean, rstd, weight=torch.ones(48, dtype=x.dtype, device="cuda:0"), bias=True)
    assert dx.shape == (0, 48) and not bool(dw.any()) and not bool(db.any())


def test_norm_rows_past_31_bits():
    ld, rows, width = 1 << 21, 1100, 136
    store = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda:0")
    x = store.view(rows, ld)[:, :width]
    x.copy_(rows_of(1, rows, width, "bf16"))
    got, want = ops.layer_norm(x, save_stats=True), ops.layer_norm(x.contiguous(), save_stats=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dout = normal(2, rows, width, dtype=torch.bfloat16)
    got = ops.layer_norm_backward(dout, x, *want[1:], bias=True)
    assert all(torch.equal(a, b) for a, b in zip(got, ops.layer_norm_backward(dout, x.contiguous(), *want[1:], bias=True)))


@pytest.mark.parametrize("rows", [5000, 70000])
def test_norm_many_rows(rows):
    """More rows than workgroups, several to each; bands of rows of the columns' sums."""
    for width in (64, 4100 if rows < 10000 else 100):
        x = rows_of(1, rows, width, "f32")
        w, b = parameters(width, "f32")
        _, mean, rstd = forward(x, w, b, None)
        backward(x, w, None, normal(2, rows, width), mean, rstd)


def test_norm_gradient_against_differences():
    """Central differences in 64 bits; their own error, h^2 times third derivatives, is below
    1e-8 here."""
    x, w, b = rows_of(1, 30, 50, "f32"), *parameters(50, "f32")
    dout = normal(2, 30, 50)
    _, mean, rstd = ops.layer_norm(x, weight=w, bias=b, save_stats=True)
    grads = ops.layer_norm_backward(dout, x, mean, rstd, weight=w, bias=True)
    _, big, columns = L.layer_norm_backward(dout, x, mean, rstd, w)
    bounds = norm_backward_bounds([g.double() for g in grads], big, columns, 30, 50, torch.float32)
    args = [x.double(), w.double(), b.double()]
    for i, grad in enumerate(grads):
        step = normal(10 + i, *grad.shape).double()
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-5 * step, args[i] - 1e-5 * step
        want = float(((L.layer_norm(*up)[0] - L.layer_norm(*down)[0]) * dout.double()).sum()) / 2e-5
        # the statistics that the call takes are themselves fp32: a few steps of every summand
        off = float((bounds[i] * step.abs()).sum()) + 100 * 2.0 ** -24 * float((grad.double() * step).abs().sum()) + 1e-6
        assert abs(float((grad.double() * step).sum()) - want) <= off


def test_norm_graph_replays_and_streams():
    x, r = rows_of(1, 1200, 520, "bf16"), rows_of(3, 1200, 520, "bf16")
    w, b = parameters(520, "bf16")
    dout = normal(7, 1200, 520, dtype=torch.bfloat16)

    def run(stream=None):
        out, total, mean, rstd = ops.layer_norm(x, weight=w, bias=b, residual=r, save_stats=True, stream=stream)
        return [out, total, mean, rstd, *ops.layer_norm_backward(dout, total, mean, rstd, weight=w, dtotal=r, bias=True,
                                                                 stream=stream)]

    first = run()
    torch.cuda.synchronize()
    again = run(torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for i in range(4):
        x.copy_(rows_of(60 + i, 1200, 520, "bf16"))
        want = run()
        torch.cuda.synchronize()
        for t in held:
            t.fill_(99)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width,pad", [(3, 72, 0), (1030, 1000, 3), (3, 20001, 1), (1100, 17000, 0)])
def test_norm_in_place(rows, width, pad, dtype):
    """total onto the residual (or x) and out onto the other: the same bits as apart."""
    w, b = parameters(width, dtype)

    def inputs():
        return rows_of(1, rows, width, dtype, pad), rows_of(3, rows, width, dtype, pad)

    x, r = inputs()
    want = ops.layer_norm(x, weight=w, bias=b, residual=r, save_stats=True)
    alone = ops.layer_norm(x, weight=w, bias=b)
    for total_onto_x in (False, True):
        x, r = inputs()
        out, total = (r, x) if total_onto_x else (x, r)
        got = ops.layer_norm(x, weight=w, bias=b, residual=r, save_stats=True, out=out, total=total)
        assert got[0] is out and got[1] is total and all(torch.equal(p, q) for p, q in zip(got, want))
    x, _ = inputs()
    assert torch.equal(ops.layer_norm(x, weight=w, bias=b, out=x), alone)
