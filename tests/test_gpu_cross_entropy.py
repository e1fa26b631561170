"""The vocabulary's cross entropy and its gradients against their definitions in 64 bits."""

import pytest
import torch

from chunk_schedule_execution_amd import ops
from layers_util import loss_backward_bounds, loss_bounds
from oracle import layers as L
from products_util import TYPES, U32, half_step, normal, within

pytestmark = pytest.mark.gpu

# rows, in, vocabulary: single values and rows, sizes around tiles and vectors, copies onto the
# 16-byte grid, each tile
SHAPES = [(1, 1, 1), (1, 8, 2), (2, 7, 5), (3, 64, 40), (1, 512, 1000), (16, 33, 130), (17, 100, 33), (63, 257, 65),
          (64, 128, 128), (65, 72, 257), (100, 1000, 48), (130, 72, 300), (255, 192, 513), (300, 264, 1031),
          (520, 136, 2050), (257, 320, 4096), (3, 1190, 11136), (15, 810, 683), (16, 2048, 5003), (40, 4096, 77),
          (64, 831, 7552), (300, 4096, 1000), (500, 2050, 9), (1000, 40, 3001), (2100, 64, 2600), (40, 128, 20000), (2048, 512, 6144)]


def inputs(seed, rows, k, vocabulary, dtype, shard=None, pad=0, total=None):
    t = TYPES[dtype]
    x = normal(seed, rows, k + pad, dtype=t)[:, :k]
    w = normal(seed + 1, vocabulary, k + pad, dtype=t, scale=2.0 * k ** -0.5)[:, pad:]
    g = torch.Generator().manual_seed(seed)
    targets = torch.randint(0, total or vocabulary, (rows,), generator=g)
    targets[torch.rand(rows, generator=g) < 0.1] = -100
    return x, w, targets.to(torch.int32).to("cuda:0")


def forward(x, w, targets, shard=None):
    got = ops.linear_cross_entropy(x, w, targets, shard=shard)
    loss, lse, picked, big = L.cross_entropy(x, w, targets, shard)
    z = torch.mm(x.double(), w.double().t())
    bl, bp, bo = loss_bounds(lse, picked, big, z.amax(1) - z.amin(1), x.shape[1], w.shape[0])
    if shard is None:
        within(got[0], loss, bo, "loss")
        within(got[1], lse, bl, "lse")
        assert not bool(got[0][L.left_out(targets, None, w.shape[0])].any())
    else:
        within(got[0], lse, bl, "lse")
        within(got[1], picked, bp, "picked")
    return got


def backward(x, w, targets, lse, shard=None, dloss=None):
    dloss = normal(50, x.shape[0]) if dloss is None else dloss
    got = ops.linear_cross_entropy_backward(dloss, x, w, targets, lse, shard=shard)
    want, bounds = loss_backward_bounds(*L.logits_gradient(dloss, x, w, targets, lse, shard), x, w, lse, x.shape[1], x.dtype)
    for g, v, b, name in zip(got, want, bounds, ("dx", "dw")):
        within(g, v, b, name)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,vocabulary", SHAPES)
def test_cross_entropy(rows, k, vocabulary, dtype):
    x, w, targets = inputs(1, rows, k, vocabulary, dtype)
    _, lse = forward(x, w, targets)
    backward(x, w, targets, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [1, 8])
@pytest.mark.parametrize("rows,k,vocabulary", [(5, 64, 100), (200, 136, 333), (300, 65, 1000)])
def test_cross_entropy_strides(rows, k, vocabulary, pad, dtype):
    x, w, targets = inputs(3, rows, k, vocabulary, dtype, pad=pad)
    _, lse = forward(x, w, targets)
    dloss = normal(50, rows)
    both = backward(x, w, targets, lse, dloss=dloss)
    # each gradient alone gives the same bits
    (dx,) = ops.linear_cross_entropy_backward(dloss, x, w, targets, lse, need_dw=False)
    (dw,) = ops.linear_cross_entropy_backward(dloss, x, w, targets, lse, need_dx=False)
    assert torch.equal(dx, both[0]) and torch.equal(dw, both[1])
    assert ops.linear_cross_entropy_backward(dloss, x, w, targets, lse, need_dx=False, need_dw=False) == []


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,vocabulary,shards", [(50, 64, 96, 2), (130, 72, 1001, 7), (33, 40, 64, 1)])
def test_cross_entropy_shards(rows, k, vocabulary, shards, dtype):
    """Shards of any sizes join to the whole, and so do their gradients."""
    x, w, targets = inputs(5, rows, k, vocabulary, dtype)
    bounds = [i * vocabulary // shards for i in range(shards + 1)]
    parts = [forward(x, w[a:b], targets, shard=a) for a, b in zip(bounds, bounds[1:])]
    lse_parts, picked_parts = (torch.stack([p[i] for p in parts]) for i in (0, 1))
    loss, lse = ops.cross_entropy_join(lse_parts, picked_parts, targets)
    whole, whole_lse, picked, big = L.cross_entropy(x, w, targets)
    z = torch.mm(x.double(), w.double().t())
    bl, _, bo = loss_bounds(whole_lse, picked, big, z.amax(1) - z.amin(1), k, vocabulary)
    within(lse, whole_lse, bl + 8 * U32 * (1 + whole_lse.abs()), "lse")
    within(loss, whole, bo + 8 * U32 * (1 + whole_lse.abs()), "loss")
    dloss = normal(50, rows)
    for a, b in zip(bounds, bounds[1:]):
        backward(x, w[a:b], targets, lse, shard=a, dloss=dloss)


def test_cross_entropy_join_of_many_shards_and_of_nothing():
    lse, picked = normal(1, 200, 77, scale=30.0), normal(2, 200, 77)
    lse[5] = float("-inf")  # a shard whose logits are all -inf
    lse[:, 3] = float("-inf")
    targets = torch.zeros(77, dtype=torch.int32, device="cuda:0")
    targets[10] = -1
    loss, total = ops.cross_entropy_join(lse, picked, targets)
    want = torch.logsumexp(lse.double(), 0)
    fine = want.isfinite()
    within(total[fine], want[fine], (40 * U32 * (1 + lse.abs().amax(0, keepdim=False).double())[fine]).nan_to_num(1e-3, posinf=1e-3), "lse")
    assert total[3] == float("-inf") and loss[10] == 0
    off = 200 * U32 * (picked.double().abs().sum(0) + 200)
    keep = fine.clone()
    keep[10] = False
    within(loss[keep], (want - picked.double().sum(0))[keep], off[keep], "loss")
    empty = ops.cross_entropy_join(lse[:, :0], picked[:, :0], targets[:0])
    assert empty[0].shape == empty[1].shape == (0,)


def test_cross_entropy_targets_outside():
    """Targets below 0 or past the vocabulary leave a row out; past a shard they are another's."""
    x, w, _ = inputs(7, 70, 64, 200, "bf16")
    targets = torch.randint(0, 200, (70,), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    targets[:6] = torch.tensor([-1, -2**31, 200, 2**31 - 1, 199, 0], dtype=torch.int32)
    targets = targets.to("cuda:0")
    loss, lse = forward(x, w, targets)
    assert not bool(loss[:4].any()) and bool((loss[4:] > 0).all())
    dx, _ = backward(x, w, targets, lse)
    assert not bool(dx[:4].any())
    for first in (0, 150, 2**31 - 201):
        lse, picked = forward(x, w, targets, shard=first)
        backward(x, w, targets, lse, shard=first)


def test_cross_entropy_of_left_out_rows_ignores_their_values():
    x, w, targets = inputs(9, 40, 64, 300, "bf16")
    targets[3] = -1
    _, lse = ops.linear_cross_entropy(x, w, targets)
    dloss = normal(50, 40)
    want = ops.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    lse[3], dloss[3] = float("nan"), float("inf")
    got = ops.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_cross_entropy_special_values():
    x, w, targets = inputs(11, 80, 64, 500, "f32")
    targets.clamp_(min=0)
    plain, plain_lse = ops.linear_cross_entropy(x, w, targets)
    x[2, 4] = float("nan")
    loss, lse = ops.linear_cross_entropy(x, w, targets)
    keep = [i for i in range(80) if i != 2]
    assert bool(loss[2].isnan()) and torch.equal(loss[keep], plain[keep]) and torch.equal(lse[keep], plain_lse[keep])
    # -inf logits are no part of the sum
    x, w, targets = inputs(12, 20, 8, 100, "f32")
    x[:, 0], w[:, 0] = 1.0, 0.0
    masked = w.clone()
    masked[30:, 0] = float("-inf")
    targets = targets.clamp(0, 29)
    loss, lse = ops.linear_cross_entropy(x, masked, targets)
    want, want_lse = ops.linear_cross_entropy(x, w[:30].contiguous(), targets)
    assert torch.allclose(loss, want, rtol=0, atol=1e-5) and torch.allclose(lse, want_lse, rtol=0, atol=1e-5)
    all_masked = masked.clone()
    all_masked[:, 0] = float("-inf")
    assert bool((ops.linear_cross_entropy(x, all_masked, targets)[1] == float("-inf")).all())


@pytest.mark.parametrize("scale", [0.0, 30.0])
def test_cross_entropy_of_equal_and_of_far_logits(scale):
    x, w, targets = inputs(13, 100, 64, 700, "bf16")
    x = (x.float() * scale).to(torch.bfloat16)
    _, lse = forward(x, w, targets)
    backward(x, w, targets, lse)


def test_cross_entropy_of_no_rows():
    x, w, targets = inputs(1, 0, 24, 50, "bf16")
    loss, lse = ops.linear_cross_entropy(x, w, targets)
    assert loss.shape == lse.shape == (0,)
    dx, dw = ops.linear_cross_entropy_backward(loss, x, w, targets, lse)
    assert dx.shape == (0, 24) and dw.shape == (50, 24) and not bool(dw.any())


@pytest.mark.parametrize("dtype,rows,k,vocabulary", [("bf16", 32768, 64, 16500), ("f32", 16384, 72, 17001)])
def test_cross_entropy_in_pieces(dtype, rows, k, vocabulary):
    """More than one piece of the vocabulary, the last one shorter: dx is summed over them."""
    x, w, targets = inputs(15, rows, k, vocabulary, dtype)
    loss, lse = ops.linear_cross_entropy(x, w, targets)
    keep = slice(0, 600)
    want, want_lse, picked, big = L.cross_entropy(x[keep], w, targets[keep])
    z = torch.mm(x[keep].double(), w.double().t())
    bl, _, bo = loss_bounds(want_lse, picked, big, z.amax(1) - z.amin(1), k, vocabulary)
    within(loss[keep], want, bo, "loss")
    within(lse[keep], want_lse, bl, "lse")
    dloss = normal(50, rows)
    # dw of 32768 rows by hand: rows beyond the first 600 and last 600 get no gradient
    targets[600:-600] = -1
    dx, dw = ops.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    assert not bool(dx[600:-600].any())
    pick = torch.cat([torch.arange(600), torch.arange(rows - 600, rows)]).to("cuda:0")
    xs, ts, ls, ds = x[pick], targets[pick], lse[pick], dloss[pick]
    (wx, ww), (bx, bw) = loss_backward_bounds(*L.logits_gradient(ds, xs, w, ts, ls), xs, w, ls, k, x.dtype)
    within(dx[pick], wx, bx + 64 * U32 * wx.abs(), "dx")
    within(dw, ww, bw, "dw")


def test_cross_entropy_in_pieces_and_splits():
    """Two pieces of the vocabulary whose dx is a few tiles of a long sum, so that each piece's
    is split and the splits are added up over the pieces."""
    rows, k, vocabulary = 2048, 64, 140000
    x, w, targets = inputs(21, rows, k, vocabulary, "bf16")
    _, lse = ops.linear_cross_entropy(x, w, targets)
    targets[100:-100] = -1
    dloss = normal(50, rows)
    dx, dw = ops.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    assert not bool(dx[100:-100].any())
    pick = torch.cat([torch.arange(100), torch.arange(rows - 100, rows)]).to("cuda:0")
    xs, ts, ls, ds = x[pick], targets[pick], lse[pick], dloss[pick]
    (wx, ww), (bx, bw) = loss_backward_bounds(*L.logits_gradient(ds, xs, w, ts, ls), xs, w, ls, k, x.dtype)
    within(dx[pick], wx, bx + 64 * U32 * wx.abs(), "dx")
    within(dw, ww, bw, "dw")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,vocabulary", [(3, 33, 50), (200, 128, 700)])
def test_cross_entropy_of_rows_that_are_all_left_out(rows, k, vocabulary, dtype):
    x, w, targets = inputs(23, rows, k, vocabulary, dtype)
    targets.fill_(-1)
    loss, lse = forward(x, w, targets)
    assert not bool(loss.any())
    for shard in (None, 0, 7):
        dx, dw = ops.linear_cross_entropy_backward(normal(50, rows), x, w, targets, lse, shard=shard)
        assert not bool(dx.any()) and not bool(dw.any())


def test_cross_entropy_of_one_target_for_all_rows():
    """Every row's gradient meets in one row of dw."""
    x, w, targets = inputs(24, 300, 72, 500, "bf16")
    targets.fill_(411)
    _, lse = forward(x, w, targets)
    backward(x, w, targets, lse)


def test_cross_entropy_of_weights_past_31_bits():
    """A vocabulary whose matrix has more than 2^31 elements: its last rows count."""
    rows, k, vocabulary = 3, 4096, 530000
    w = torch.zeros(vocabulary, k, dtype=torch.bfloat16, device="cuda:0")
    x = normal(1, rows, k, dtype=torch.bfloat16)
    tail = normal(2, 100, k, dtype=torch.bfloat16, scale=0.1)
    w[-100:] = tail
    targets = torch.tensor([vocabulary - 1, 5, vocabulary - 50], dtype=torch.int32, device="cuda:0")
    loss, lse = ops.linear_cross_entropy(x, w, targets)
    z = torch.mm(x.double(), tail.double().t())
    want = torch.logsumexp(torch.cat([z, torch.full((rows, 1), float(torch.tensor(vocabulary - 100.0).double().log()),
                                                    dtype=torch.float64, device="cuda:0")], 1), 1)
    big = torch.mm(x.double().abs(), tail.double().abs().t()).amax(1)
    off = (k + 2) * U32 * big + (vocabulary // 512 + 400) * U32 + 4 * U32 * want
    within(lse, want, off, "lse")
    at = torch.stack([z[0, 99], torch.zeros_like(z[0, 0]), z[2, 50]])
    within(loss, want - at, 2 * off, "loss")
    dloss = torch.ones(rows, device="cuda:0")
    dx, dw = ops.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    p = torch.exp(z - lse.double()[:, None])
    hot = torch.zeros_like(p)
    hot[0, 99] = hot[2, 50] = 1.0
    wdx, wdw = torch.mm(p - hot, tail.double()), torch.mm((p - hot).t(), x.double())
    slack = 4 * half_step(torch.bfloat16)
    within(dx, wdx, slack * torch.mm((p + hot), tail.double().abs()) + 1e-6, "dx")
    within(dw[-100:], wdw, slack * torch.mm((p + hot).t(), x.double().abs()) + 1e-6, "dw")


def test_cross_entropy_gradient_against_differences():
    """Central differences in 64 bits; their own error is below 1e-8 here."""
    x, w, targets = inputs(17, 30, 20, 50, "f32")
    loss, lse = ops.linear_cross_entropy(x, w, targets)
    dloss = normal(50, 30)
    grads = ops.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    _, bounds = loss_backward_bounds(*L.logits_gradient(dloss, x, w, targets, lse), x, w, lse, 20, torch.float32)
    args = [x.double(), w.double()]
    for i, (grad, bound) in enumerate(zip(grads, bounds)):
        step = normal(60 + i, *grad.shape).double()
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-5 * step, args[i] - 1e-5 * step
        want = float(((L.cross_entropy(*up, targets)[0] - L.cross_entropy(*down, targets)[0]) * dloss.double()).sum()) / 2e-5
        # lse is fp32: p is off by a few steps of it
        off = float((bound * step.abs()).sum()) + 200 * U32 * float((grad.double() * step).abs().sum()) + 1e-5
        assert abs(float((grad.double() * step).sum()) - want) <= off


def test_cross_entropy_graph_replays_and_streams():
    x, w, targets = inputs(19, 300, 136, 1100, "bf16")
    dloss = normal(50, 300)

    def run(stream=None):
        loss, lse = ops.linear_cross_entropy(x, w, targets, stream=stream)
        part = ops.linear_cross_entropy(x, w, targets, shard=500, stream=stream)
        joined = ops.cross_entropy_join(torch.stack([part[0], part[0]]) if stream is None else pair(part[0]),
                                        torch.stack([part[1], part[1]]) if stream is None else pair(part[1]), targets,
                                        stream=stream)
        return [loss, lse, *part, *joined, *ops.linear_cross_entropy_backward(dloss, x, w, targets, lse, stream=stream)]

    def pair(t):
        with torch.cuda.stream(side):
            return torch.stack([t, t])

    side = torch.cuda.Stream()
    first = run()
    torch.cuda.synchronize()
    again = run(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for i in range(4):
        nx, _, nt = inputs(70 + i, 300, 136, 1100, "bf16")
        x.copy_(nx)
        targets.copy_(nt)
        want = run()
        torch.cuda.synchronize()
        for t in held:
            t.fill_(99)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,vocabulary,pad", [(3, 64, 50, 0), (9, 33, 700, 1), (200, 128, 700, 0), (300, 65, 1000, 1),
                                                   (1100, 264, 2500, 8)])
def test_cross_entropy_of_left_out_rows_of_nan(rows, k, vocabulary, pad, dtype):
    """What padding holds reaches neither another row's loss nor a gradient, to the bit."""
    x, w, targets = inputs(31, rows, k, vocabulary, dtype, pad=pad)
    targets[1] = -1
    out = targets < 0
    dloss = normal(50, rows)
    for shard in (None, 7):
        clean = ops.linear_cross_entropy(x, w, targets, shard=shard)
        lse = clean[1] if shard is None else clean[0]
        want = ops.linear_cross_entropy_backward(dloss, x, w, targets, lse, shard=shard)
        for value in (float("nan"), float("inf"), -3e38):
            y = x.clone()
            y[out] = value
            got = ops.linear_cross_entropy(y, w, targets, shard=shard)
            assert all(torch.equal(a[~out], b[~out]) for a, b in zip(got, clean))
            if shard is None:
                assert not bool(got[0][out].any())
            got = ops.linear_cross_entropy_backward(dloss, y, w, targets, got[1] if shard is None else got[0], shard=shard)
            assert all(torch.equal(a, b) for a, b in zip(got, want)) and not bool(got[0][out].any())
            # one gradient alone as well
            for only in (dict(need_dx=False), dict(need_dw=False)):
                alone = ops.linear_cross_entropy_backward(dloss, y, w, targets, lse, shard=shard, **only)
                assert torch.equal(alone[0], want[1 if "need_dx" in only else 0])
