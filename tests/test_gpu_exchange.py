"""The row exchange around an expert-parallel layer's AllToAlls against its definitions."""

import pytest
import torch

from chunk_schedule_execution_amd import ops
from oracle import products as O
from products_util import TYPES, U32, half_step, normal, within

pytestmark = pytest.mark.gpu


def ids_of(seed, tokens, choices, experts, away=0.0, spread=None):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, spread or experts, (tokens, choices), generator=g, dtype=torch.int32)
    if away:
        out = torch.rand(tokens, choices, generator=g) < away
        ids[out] = torch.where(torch.rand(tokens, choices, generator=g) < 0.5, -1, experts + 3)[out].to(torch.int32)
    return ids


ROUTES = [(1, 1, 1, 0.0), (1, 1, 1, 1.0), (3, 2, 5, 0.0), (64, 1, 3, 0.2), (65, 4, 64, 0.25), (300, 8, 1024, 0.0),
          (700, 3, 7, 0.5), (2049, 2, 1000, 0.1), (5000, 4, 2, 0.0), (100, 5, 31, 1.0), (3, 400, 33, 0.1)]


@pytest.mark.parametrize("tokens,choices,experts,away", ROUTES)
def test_route(tokens, choices, experts, away):
    ids = ids_of(3, tokens, choices, experts, away)
    offsets, positions, slots = ops.expert_route(ids.to("cuda:0"), experts)
    want = O.route(ids.tolist(), experts)
    assert offsets.tolist() == want[0]
    assert positions.reshape(-1).tolist() == want[1]
    assert slots.tolist() == want[2]


@pytest.mark.parametrize("tokens,choices,experts", [(40000, 8, 64), (200000, 8, 128), (1 << 20, 2, 16)])
def test_route_long(tokens, choices, experts):
    ids = ids_of(5, tokens, choices, experts, 0.1).to("cuda:0")
    offsets, positions, slots = ops.expert_route(ids, experts)
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    key, order = torch.sort(key, stable=True)
    used = int((key < experts).sum())
    assert torch.equal(offsets.long(), torch.searchsorted(key, torch.arange(experts + 1, device="cuda:0")))
    assert torch.equal(slots[:used].long(), order[:used]) and bool((slots[used:] == -1).all())
    back = torch.full_like(flat, -1)
    back[order[:used]] = torch.arange(used, device="cuda:0")
    assert torch.equal(positions.reshape(-1).long(), back)


def test_route_of_one_expert_and_of_no_tokens():
    ids = torch.zeros(130, 3, dtype=torch.int32, device="cuda:0")
    offsets, positions, slots = ops.expert_route(ids, 4)
    assert offsets.tolist() == [0, 390, 390, 390, 390] and slots.tolist() == list(range(390))
    offsets, positions, slots = ops.expert_route(ids[:0], 4)
    assert offsets.tolist() == [0] * 5 and positions.shape == (0, 3) and slots.numel() == 0


EXCHANGES = [(1, 1, 2, 1, 0.0, 0), (1, 2, 4, 64, 0.0, 0), (5, 3, 4, 7, 0.3, 0), (48, 4, 64, 2048, 0.25, 0),
             (33, 2, 8, 1000, 0.0, 8), (129, 8, 16, 136, 0.1, 3), (257, 1, 3, 4104, 0.5, 0), (700, 2, 5, 33, 1.0, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,choices,experts,width,away,pad", EXCHANGES)
def test_exchange(tokens, choices, experts, width, away, pad, dtype):
    t = TYPES[dtype]
    ids = ids_of(7, tokens, choices, experts, away).to("cuda:0")
    _, positions, slots = ops.expert_route(ids, experts)
    x = normal(1, tokens, width + pad, dtype=t)[:, :width]
    rows = ops.expert_dispatch(x, slots, choices)
    assert torch.equal(rows, O.dispatch(x, slots, choices))
    h = normal(2, tokens * choices, width + pad, dtype=t)[:, :width]
    gates = normal(3, tokens, choices)
    for g in (gates, None):
        out = ops.expert_combine(h, positions, g)
        want, big = O.combine(h, positions, g)
        off = (choices + 1) * U32 * big
        within(out, want, off + half_step(t) * (want.abs() + off) + 1e-38, "combine")
        dout = normal(4, tokens, width + pad, dtype=t)[:, :width]
        dh, dg = ops.expert_combine_backward(dout, h, positions, slots, g)
        (wh, wg), bg = O.combine_backward(dout, h, positions, slots, g)
        within(dh, wh, (half_step(t) * 1.01 + U32) * wh.abs() + 1e-38, "dh")
        within(dg, wg, (width + 2) * U32 * bg + 1e-38, "dgates")


def test_exchange_ignores_rows_served_elsewhere():
    """Rows that no slot has may hold anything: nothing of them reaches an output."""
    ids = ids_of(9, 40, 3, 6, 0.4).to("cuda:0")
    offsets, positions, slots = ops.expert_route(ids, 6)
    h = normal(2, 120, 256, dtype=torch.bfloat16)
    h[int(offsets[-1]):] = float("nan")
    gates = normal(3, 40, 3)
    gates[positions < 0] = float("nan")
    assert bool(ops.expert_combine(h, positions, gates).isfinite().all())
    dh, dg = ops.expert_combine_backward(normal(4, 40, 256, dtype=torch.bfloat16), h, positions, slots, gates)
    assert bool(dh.isfinite().all()) and bool(dg.isfinite().all())
    assert not bool(dh[int(offsets[-1]):].any()) and not bool(dg[positions < 0].any())


def test_exchange_reads_indexes_outside_the_rows_as_none():
    x = normal(1, 10, 64)
    slots = torch.tensor([0, 20, -5, 2**31 - 1, 3, -2**31] + [1] * 14, dtype=torch.int32, device="cuda:0")
    rows = ops.expert_dispatch(x, slots, 2)
    assert torch.equal(rows, O.dispatch(x, slots, 2)) and not bool(rows[1:4].any())
    positions = slots.view(10, 2)
    h = normal(2, 20, 64)
    want, big = O.combine(h, positions)
    within(ops.expert_combine(h, positions), want, 4 * U32 * (want.abs() + big) + 1e-38, "combine")


def test_combine_gradient_against_differences():
    """The combine is linear in h and in the gates: differences are exact up to fp32."""
    ids = ids_of(11, 30, 3, 5, 0.2).to("cuda:0")
    _, positions, slots = ops.expert_route(ids, 5)
    h, gates, dout = normal(1, 90, 40), normal(2, 30, 3), normal(3, 30, 40)
    dh, dg = ops.expert_combine_backward(dout, h, positions, slots, gates)
    d, e = normal(4, 90, 40).double(), normal(5, 30, 3).double()
    for grad, a, b in ((dh.double() * d, (h.double() + d, gates), (h.double() - d, gates)),
                       (dg.double() * e, (h, gates.double() + e), (h, gates.double() - e))):
        want = ((O.combine(a[0], positions, a[1])[0] - O.combine(b[0], positions, b[1])[0]) * dout.double()).sum() / 2
        assert abs(float(grad.sum() - want)) <= 50 * U32 * float(grad.abs().sum()) + 1e-30


def test_dispatch_gradient_is_the_combine():
    """<rows gradient, dispatch(x)> = <x, combine(rows gradient)> for integers, exactly."""
    ids = ids_of(13, 50, 4, 9, 0.3).to("cuda:0")
    _, positions, slots = ops.expert_route(ids, 9)
    g = torch.Generator(device="cuda:0").manual_seed(1)
    x = torch.randint(-8, 9, (50, 24), generator=g, device="cuda:0").float()
    d = torch.randint(-8, 9, (200, 24), generator=g, device="cuda:0").float()
    left = (ops.expert_dispatch(x, slots, 4).double() * d.double()).sum()
    right = (x.double() * ops.expert_combine(d, positions).double()).sum()
    assert float(left) == float(right)


def test_exchange_graph_replays_and_streams():
    x, gates = normal(1, 96, 264, dtype=torch.bfloat16), normal(2, 96, 4)
    ids = ids_of(15, 96, 4, 16, 0.1).to("cuda:0")
    dout = normal(3, 96, 264, dtype=torch.bfloat16)

    def run(stream=None):
        o, p, s = ops.expert_route(ids, 16, stream=stream)
        rows = ops.expert_dispatch(x, s, 4, stream=stream)
        out = ops.expert_combine(rows, p, gates, stream=stream)
        return [o, p, s, rows, out, *ops.expert_combine_backward(dout, rows, p, s, gates, stream=stream)]

    first = run()
    torch.cuda.synchronize()
    again = run(torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for i in range(4):
        ids.copy_(ids_of(40 + i, 96, 4, 16, 0.2))
        x.copy_(normal(50 + i, 96, 264, dtype=torch.bfloat16))
        want = run()
        torch.cuda.synchronize()
        for t in held:
            t.fill_(99)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), i
