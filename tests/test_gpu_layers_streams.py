"""The choice of experts, layer norm and the cross entropy on a stream of their own, beside
work on torch's current stream, and several of their graphs at once."""

import pytest
import torch

from chunk_schedule_execution_amd import ops
from products_util import normal

pytestmark = pytest.mark.gpu


def layer(seed):
    """Odd sizes, so that every call that can use a workspace does."""
    t = torch.bfloat16
    targets = torch.randint(-40, 1500, (900,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    return {"logits": normal(seed, 3000, 60, dtype=t), "bias": normal(seed + 1, 60, scale=0.1),
            "dgates": normal(seed + 2, 3000, 4), "x": normal(seed + 3, 900, 333, dtype=t),
            "r": normal(seed + 4, 900, 333, dtype=t), "w": normal(seed + 5, 333, dtype=t),
            "v": normal(seed + 6, 1500, 333, dtype=t, scale=0.1), "targets": targets.to("cuda:0"),
            "dloss": normal(seed + 7, 900)}


def run(s, stream=None):
    ids, gates = ops.expert_select(s["logits"], 4, score="sigmoid", bias=s["bias"], groups=6, kept_groups=3, group_best=2,
                                   stream=stream)
    dlogits = ops.expert_select_backward(s["dgates"], s["logits"], ids, score="sigmoid", stream=stream)
    out, total, mean, rstd = ops.layer_norm(s["x"], weight=s["w"], residual=s["r"], save_stats=True, stream=stream)
    grads = ops.layer_norm_backward(out, total, mean, rstd, weight=s["w"], dtotal=s["r"], bias=True, stream=stream)
    loss, lse = ops.linear_cross_entropy(out, s["v"], s["targets"], stream=stream)
    part = ops.linear_cross_entropy(out, s["v"], s["targets"], shard=700, stream=stream)
    dx, dv = ops.linear_cross_entropy_backward(s["dloss"], out, s["v"], s["targets"], lse, stream=stream)
    return [ids, gates, dlogits, out, total, mean, rstd, *grads, loss, lse, *part, dx, dv]


@pytest.mark.parametrize("raw", [False, True])
def test_two_streams_of_different_inputs(raw):
    here, there = [layer(100 * i) for i in range(4)], [layer(100 * i + 50) for i in range(4)]
    want = [[t.clone() for t in run(s)] for s in here + there]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    handle = side.cuda_stream if raw else side
    got_here, got_there = [], []
    for a, b in zip(here, there):
        got_here.append(run(a))
        got_there.append(run(b, handle))
    torch.cuda.synchronize()
    for got, right in zip(got_here + got_there, want):
        assert all(torch.equal(g, r) for g, r in zip(got, right))


def test_graphs_of_one_pool_replayed_in_turn_and_a_side_stream_inside():
    a, b = layer(7), layer(8)
    side = torch.cuda.Stream()

    def both(s):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        there = run(s, side)
        first = run(s)
        here.wait_stream(side)
        return first + there

    both(a)
    torch.cuda.synchronize()
    graphs, held = [], []
    pool = torch.cuda.graph_pool_handle()
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            held.append(both(s))
        graphs.append(g)
    for i in range(4):
        for s, seed in ((a, 300 + 10 * i), (b, 500 + 10 * i)):
            for name, t in layer(seed).items():
                s[name].copy_(t)
        want = [run(a), run(b)]
        torch.cuda.synchronize()
        for ts in held:
            for t in ts:
                t.fill_(77)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for ts, w in zip(held, want):
            assert all(torch.equal(x, y) for x, y in zip(ts, w + w)), i
