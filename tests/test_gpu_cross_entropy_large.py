"""The cross entropy in tiles of 256: rows and columns that end inside a tile, shards, several
pieces of the vocabulary whose dx is summed up over them, split or not."""

import pytest
import torch

from chunk_schedule_execution_amd import capi, ops
from layers_util import loss_backward_bounds
from oracle import layers as L
from products_util import U32, normal, within
from test_gpu_cross_entropy import backward, forward, inputs

pytestmark = pytest.mark.gpu


def tiles(rows, k, columns):
    """(tile rows, splits) of the products of a call: the logits, dx and dw."""
    d = capi.ccl_linear_desc(dtype=capi.CCL_BF16, rows=rows, in_features=k, out_features=columns)
    return [(i.tile_rows, i.splits) for i in (*capi.ccl_linear_info(d, False, False), *capi.ccl_linear_info(d, False, True))]


@pytest.mark.parametrize("rows,k,vocabulary", [(2047, 2056, 6151), (2047, 2051, 6151), (4099, 2056, 6145)])
def test_cross_entropy_ends_inside_tiles(rows, k, vocabulary):
    assert [t for t, _ in tiles(rows, k, vocabulary)] == [256, 256, 256]
    assert rows % 256 and vocabulary % 256 and k % 256
    x, w, targets = inputs(41, rows, k, vocabulary, "bf16", total=vocabulary + 1)
    targets[-1], targets[-2], targets[0] = vocabulary - 1, 0, vocabulary
    _, lse = forward(x, w, targets)
    backward(x, w, targets, lse)


@pytest.mark.parametrize("rows,k,vocabulary", [(2047, 2056, 6151)])
def test_cross_entropy_of_a_shard_ends_inside_tiles(rows, k, vocabulary):
    """Targets before, inside and behind the shard, and at its first and last row."""
    x, w, targets = inputs(43, rows, k, vocabulary, "bf16", total=3 * vocabulary)
    first = vocabulary
    targets[-4:] = torch.tensor([first - 1, first, 2 * first - 1, 2 * first], dtype=torch.int32)
    lse, picked = forward(x, w, targets, shard=first)
    assert [bool(v) for v in picked[-4:]] == [False, True, True, False]
    backward(x, w, targets, lse + 1.0, shard=first)  # the other shards make up the rest


@pytest.mark.parametrize("rows,k,vocabulary,pieces,splits", [(33000, 1032, 16500, [5632, 5632, 5236], 1),
                                                             (4099, 1032, 140500, [46848, 46848, 46804], 3)])
def test_cross_entropy_in_pieces_of_large_tiles(rows, k, vocabulary, pieces, splits):
    for columns in (pieces[0], pieces[-1]):
        of_logits, of_dx, _ = tiles(rows, k, columns)
        assert of_logits[0] == 256 and of_dx == (256, splits)
    x, w, targets = inputs(45, rows, k, vocabulary, "bf16")
    loss, lse = ops.linear_cross_entropy(x, w, targets)
    g = torch.Generator().manual_seed(46)
    # of 64 bits' logits only so many: the other rows are left out of the gradients
    pick = torch.cat([torch.randperm(rows - 140, generator=g)[:160], torch.arange(rows - 140, rows)]).to("cuda:0")
    xs, ts, ls = x[pick], targets[pick].clone(), lse[pick]
    forward(xs, w, ts)
    want, want_lse, _, big = L.cross_entropy(xs, w, ts)
    # a logit's error, and as many roundings as sums of a row go through
    off = (k + 2) * U32 * big + (vocabulary // 512 + 400 + 2 * want_lse.abs()) * U32
    within(ls, want_lse, off, "lse")
    within(loss[pick], want, 3 * off + 2 * U32 * want.abs(), "loss")
    targets.fill_(-1)
    targets[pick] = ts
    dloss = normal(50, rows)
    dx, dw = ops.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    (wx, ww), (bx, bw) = loss_backward_bounds(*L.logits_gradient(dloss[pick], xs, w, ts, ls), xs, w, ls, k, x.dtype)
    within(dx[pick], wx, bx + 64 * U32 * wx.abs(), "dx")
    within(dw, ww, bw, "dw")
    dx[pick] = 0.0
    assert not bool(dx.any())
    alone = ops.linear_cross_entropy_backward(dloss, x, w, targets, lse, need_dw=False)[0]
    dx, _ = ops.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    assert torch.equal(alone, dx)


def test_targets_past_the_vocabulary_of_shards():
    """The whole vocabulary leaves such rows out. Shards do not know its end: the rows count, with
    loss = lse and a gradient without a target; negative targets leave them out of both."""
    rows, k, vocabulary = 90, 64, 200
    x, w, targets = inputs(47, rows, k, vocabulary, "bf16")
    targets[:10] = torch.tensor([vocabulary, vocabulary + 1, 2**31 - 1, -1, -2**31] * 2, dtype=torch.int32)
    past = targets >= vocabulary
    whole, whole_lse = ops.linear_cross_entropy(x, w, targets)
    assert not bool(whole[past].any())
    parts = [ops.linear_cross_entropy(x, w[a:a + 100], targets, shard=a) for a in (0, 100)]
    loss, lse = ops.cross_entropy_join(*(torch.stack([p[i] for p in parts]) for i in (0, 1)), targets)
    assert torch.equal(loss[past], lse[past]) and not bool(loss[targets < 0].any())
    dloss = normal(50, rows)
    for a in (0, 100):
        dx, _ = backward(x, w[a:a + 100], targets, lse, shard=a, dloss=dloss)
        assert bool(dx[past].any(1).all()) and not bool(dx[targets < 0].any())
    negative = torch.where(past, torch.full_like(targets, -1), targets)
    loss, _ = ops.cross_entropy_join(*(torch.stack([p[i] for p in parts]) for i in (0, 1)), negative)
    assert not bool(loss[past].any())
