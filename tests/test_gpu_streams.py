"""Calls of ``ops`` on a stream of their own, beside work on torch's current stream."""

import pytest
import torch

from chunk_schedule_execution_amd import ops
from products_util import normal

pytestmark = pytest.mark.gpu


def layer(seed, rows=1500, k=1000, n=1032):
    """Inputs of one layer and its expert exchange: odd sizes, so that copies and dz need a
    workspace."""
    t = torch.bfloat16
    ids = torch.randint(0, 9, (6000, 2), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    return {"x": normal(seed, rows, k + 1, dtype=t)[:, :k], "w": normal(seed + 1, n, k, dtype=t, scale=k ** -0.5),
            "dout": normal(seed + 2, rows, n, dtype=t), "tokens": normal(seed + 3, 6000, 72, dtype=t),
            "gates": normal(seed + 4, 6000, 2), "ids": ids.to("cuda:0")}


def run(s, stream=None):
    out, preact = ops.linear(s["x"], s["w"], activation="gelu", save_preact=True, stream=stream)
    grads = ops.linear_backward(s["dout"], s["x"], s["w"], preact=preact, activation="gelu", bias=True, stream=stream)
    offsets, positions, slots = ops.expert_route(s["ids"], 8, stream=stream)
    rows = ops.expert_dispatch(s["tokens"], slots, 2, stream=stream)
    mixed = ops.expert_combine(rows, positions, s["gates"], stream=stream)
    back = ops.expert_combine_backward(s["tokens"], rows, positions, slots, s["gates"], stream=stream)
    return [out, preact, *grads, offsets, positions, slots, rows, mixed, *back]


@pytest.mark.parametrize("raw", [False, True])
def test_two_streams_of_different_inputs(raw):
    """Nothing that one stream still works on is written by the other, in either direction:
    many calls of equal sizes and different values, without a synchronization between."""
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


def test_blocks_of_the_current_stream_stay_there(monkeypatch):
    """A block that the current stream has let go is not handed to a call on another one."""
    rows, k = 6000, 2048  # results of 24 MB: blocks that are not shared with other tensors
    x, w = normal(1, rows, k, dtype=torch.bfloat16), normal(2, k, k, dtype=torch.bfloat16)
    dout, preact = normal(3, rows, k, dtype=torch.bfloat16), normal(4, rows, k, dtype=torch.bfloat16)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    free = [torch.empty(rows, k, dtype=torch.bfloat16, device="cuda:0") for _ in range(4)]
    let_go = {t.data_ptr() for t in free}
    del free
    workspaces = []
    real = ops.capi.ccl_linear_backward

    def spy(*a):
        workspaces.append(a[-3])
        real(*a)

    monkeypatch.setattr(ops.capi, "ccl_linear_backward", spy)
    side = torch.cuda.Stream()
    out = ops.linear(x, w, stream=side)
    grads = ops.linear_backward(dout, x, w, preact=preact, activation="silu", stream=side)
    torch.cuda.synchronize()
    assert workspaces and workspaces[0] and not let_go & {t.data_ptr() for t in [out, *grads]} | let_go & set(workspaces)


def test_side_stream_inside_a_graph():
    s = layer(7)

    def both():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        there = run(s, side)
        first = run(s)
        here.wait_stream(side)
        return first + there

    side = torch.cuda.Stream()
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for i in range(4):
        for name, t in layer(300 + 10 * i).items():
            s[name].copy_(t)
        want = run(s)
        torch.cuda.synchronize()
        for t in held:
            t.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want + want)), i
