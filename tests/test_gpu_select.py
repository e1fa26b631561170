"""The choice of experts and its gradient against their definitions in 64 bits."""

import math

import pytest
import torch

from chunk_schedule_execution_amd import ops
from layers_util import select_backward_bounds, select_bounds
from oracle import layers as L
from products_util import TYPES, normal, within

pytestmark = pytest.mark.gpu

INF = math.inf

# tokens, experts, choices, groups, kept groups, best of a group: every number of lanes and
# values a lane, odd numbers, all experts chosen, groups of one
SHAPES = [(1, 1, 1, 1, 1, 1), (1, 2, 2, 1, 1, 1), (3, 7, 3, 1, 1, 1), (17, 16, 4, 4, 2, 1), (33, 32, 8, 8, 3, 2),
          (5, 33, 33, 3, 2, 2), (64, 64, 4, 1, 1, 1), (31, 61, 3, 61, 5, 1), (40, 96, 6, 4, 1, 2), (20, 128, 8, 16, 4, 1),
          (9, 200, 20, 8, 3, 2), (50, 256, 8, 8, 4, 2), (7, 257, 5, 1, 1, 1), (12, 320, 64, 5, 4, 1),
          (6, 512, 16, 64, 9, 2), (5, 513, 7, 27, 2, 2), (4, 1000, 10, 50, 30, 1), (3, 1024, 64, 64, 64, 1)]


def inputs(seed, tokens, experts, dtype, closed=0.0):
    logits = normal(seed, tokens, experts, scale=2.0, dtype=TYPES[dtype])
    if closed:
        g = torch.Generator(device="cuda:0").manual_seed(seed + 1)
        logits[torch.rand(tokens, experts, generator=g, device="cuda:0") < closed] = -INF
    return logits


def check(logits, choices, **kw):
    ids, gates = ops.expert_select(logits, choices, **kw)
    want, wg = L.select(logits, choices, **kw)
    assert ids.tolist() == want.tolist()
    within(gates, wg, select_bounds(wg, logits), "gates")
    return ids


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,choices,groups,kept,best", SHAPES)
def test_select(tokens, experts, choices, groups, kept, best, score, dtype):
    logits = inputs(1, tokens, experts, dtype)
    bias = normal(2, experts, scale=0.1)
    for b in (None, bias):
        for renormalise, scale in ((False, 1.0), (True, 2.5)):
            check(logits, choices, score=score, bias=b, groups=groups, kept_groups=kept, group_best=best,
                  renormalise=renormalise, scale=scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("closed", [0.3, 0.9, 1.0])
@pytest.mark.parametrize("experts,groups,kept", [(12, 3, 2), (64, 8, 2), (300, 6, 3)])
def test_select_closed_experts(experts, groups, kept, closed, score):
    """Rows with few open experts, or none: the rest of the ids are -1 and their gates 0."""
    logits = inputs(3, 40, experts, "f32", closed)
    logits[0] = -INF
    for bias in (None, normal(4, experts, scale=0.1)):
        for best in (1, 2):
            for renormalise in (False, True):
                ids = check(logits, 4, score=score, bias=bias, groups=groups, kept_groups=kept, group_best=best,
                            renormalise=renormalise)
                assert ids[0].tolist() == [-1] * 4
    bias = normal(4, experts, scale=0.1)
    bias[::2] = -INF
    assert not bool((check(logits, 3, score=score, bias=bias) % 2 == 0).any())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_select_ties_go_to_the_lower_index(score):
    logits = torch.zeros(20, 72, device="cuda:0")
    assert check(logits, 5, score=score)[0].tolist() == [0, 1, 2, 3, 4]
    assert check(logits, 3, score=score, groups=8, kept_groups=2, group_best=2)[0].tolist() == [0, 1, 2]
    # few values, many of each
    logits = normal(5, 200, 72).round()
    check(logits, 9, score=score)
    check(logits, 9, score=score, groups=12, kept_groups=5, group_best=2)
    check(logits, 9, score=score, bias=normal(6, 72).round() * 0.25, groups=12, kept_groups=5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_select_compares_in_64_bits(score):
    """Biases that make sums equal but for less than a step of fp32 of them."""
    x = normal(7, 300, 40)
    bias = torch.full((40,), 1.0, device="cuda:0")  # p + 1 in fp32 loses p's low bits
    check(x * 1e-4, 6, score=score, bias=bias)
    check(x * 1e-4, 6, score=score, bias=bias, groups=8, kept_groups=3, group_best=2)
    check(x * 1e-6, 6, score=score, groups=8, kept_groups=3, group_best=2)


def ids_in_order(logits, choices, score, bias, groups, kept, best):
    """Many tokens at once: stable sorts of the 64-bit values."""
    x = logits.double()
    t, e = x.shape
    value = L.scores(x, score) + (0.0 if bias is None else bias.double())
    value = value.masked_fill(x == -INF, -INF)
    order = value if bias is not None else x
    if kept < groups:
        top = value.view(t, groups, -1).sort(2, descending=True).values[:, :, :best]
        total = top.masked_fill(top == -INF, 0.0).sum(2).masked_fill(top[:, :, 0] == -INF, -INF)
        stay = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :kept]
        mask = torch.zeros(t, groups, dtype=torch.bool, device=x.device).scatter_(1, stay, True)
        order = order.masked_fill(~mask.repeat_interleave(e // groups, 1), -INF)
    values, ids = torch.sort(order, dim=1, descending=True, stable=True)
    return ids.masked_fill(values == -INF, -1)[:, :choices].to(torch.int32)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,choices,groups,kept,best", [
    (256, 8, 8, 4, 2), (256, 8, 1, 1, 1), (128, 12, 16, 3, 1), (64, 4, 4, 2, 2), (61, 3, 1, 1, 1), (250, 10, 25, 6, 2),
    (32, 2, 32, 20, 2), (192, 13, 6, 2, 2), (128, 4, 64, 5, 2)])
def test_select_many_tokens(experts, choices, groups, kept, best, score):
    """Enough tokens that some are close to a tie, in fp32 below what it resolves, and some have
    more experts near the border than are looked at in 64 bits one by one."""
    for dtype, rounded in (("f32", False), ("bf16", False), ("f32", True)):
        logits = inputs(17, 20000, experts, dtype, 0.05)
        if rounded:  # few different logits: ties everywhere
            logits = logits.mul(2).round().div(2)
        for bias in (None, normal(18, experts, scale=0.05), normal(19, experts).round() * 2.0 ** 20):
            got, _ = ops.expert_select(logits, choices, score=score, bias=bias, groups=groups, kept_groups=kept,
                                       group_best=best)
            want = ids_in_order(logits, choices, score, bias, groups, kept, best)
            assert torch.equal(got, want), (dtype, rounded, int((got != want).any(1).sum()))


@pytest.mark.parametrize("lowest", [-100.0, -700.0, float(torch.finfo(torch.bfloat16).min)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_select_of_masks_of_the_lowest_value(score, lowest):
    """Such experts are open: they come last, with gates that vanish beside others' and share
    what there is where all chosen ones are such."""
    logits = normal(8, 30, 24, dtype=torch.bfloat16)
    logits[:, 5:] = lowest
    logits[10:] = lowest
    for renormalise in (False, True):
        check(logits, 8, score=score, renormalise=renormalise)


def test_select_special_values():
    logits = normal(9, 8, 20)
    logits[1, 7] = float("nan")
    logits[2, 3] = INF
    logits[3] = float("nan")
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(20, device="cuda:0")):
            ids, gates = ops.expert_select(logits, 4, score=score, bias=bias)
            plain, _ = ops.expert_select(normal(9, 8, 20), 4, score=score, bias=bias)
            assert bool(((ids >= 0) & (ids < 20)).all())
            assert torch.equal(ids[[0, 4, 5, 6, 7]], plain[[0, 4, 5, 6, 7]])  # no other row notices
            assert bool(gates[[0, 4, 5, 6, 7]].isfinite().all())
            assert bool(gates[3].isnan().all()) and bool(gates[1].isnan().any())
            if score == "sigmoid":
                assert ids[1, 0] == 7 and ids[2, 0] == 3 and gates[2, 0] == 1.0
                assert bool(gates[1, 1:].isfinite().all())
    bias = torch.zeros(20, device="cuda:0")
    bias[11] = float("nan")
    ids, gates = ops.expert_select(logits[4:], 3, score="sigmoid", bias=bias)
    assert bool((ids[:, 0] == 11).all()) and bool(gates.isfinite().all())


@pytest.mark.parametrize("pad", [1, 8])
def test_select_strides_and_bases(pad):
    wide = normal(10, 70, 64 + pad, dtype=torch.bfloat16)
    check(wide[:, :64], 4)
    check(wide[:, pad:], 4, score="sigmoid", bias=normal(11, 64, scale=0.1))
    logits = wide[:, pad:]
    ids, _ = ops.expert_select(logits, 4)
    backward(logits, ids, score="softmax")


def test_select_of_no_tokens_and_of_many():
    ids, gates = ops.expert_select(torch.zeros(0, 8, device="cuda:0"), 2)
    assert ids.shape == gates.shape == (0, 2)
    assert ops.expert_select_backward(gates, torch.zeros(0, 8, device="cuda:0"), ids).shape == (0, 8)
    # tokens whose rows start past 2^31 elements
    ld = 1 << 21
    store = torch.empty(1100 * ld, dtype=torch.bfloat16, device="cuda:0")
    logits = store.view(1100, ld)[:, :40]
    logits.copy_(normal(12, 1100, 40, dtype=torch.bfloat16))
    ids = check(logits, 3)
    dgates = normal(13, 1100, 3)
    assert torch.equal(ops.expert_select_backward(dgates, logits, ids),
                       ops.expert_select_backward(dgates, logits.contiguous(), ids))


# ---- the gradient --------------------------------------------------------------------------
def backward(logits, ids, **kw):
    tokens, choices = ids.shape
    dgates = normal(20, tokens, choices)
    dgates[ids < 0] = float("nan")  # nothing reads them
    got = ops.expert_select_backward(dgates, logits, ids, **kw)
    dgates = torch.where(ids < 0, 0.0, dgates)
    want, big = L.select_backward(dgates, logits, ids, **kw)
    within(got, want, select_backward_bounds(want, big, logits, logits.dtype, choices), "dlogits")
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,choices", [s[:3] for s in SHAPES])
def test_select_backward(tokens, experts, choices, score, renormalise, dtype):
    logits = inputs(21, tokens, experts, dtype)
    ids, _ = ops.expert_select(logits, choices, score=score)
    backward(logits, ids, score=score, renormalise=renormalise, scale=1.5)


@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_select_backward_of_closed_and_far_experts(score, renormalise):
    logits = inputs(22, 60, 40, "f32", 0.85)
    logits[0] = -INF
    logits[1] = -90.0
    ids, _ = ops.expert_select(logits, 5, score=score)
    dx = backward(logits, ids, score=score, renormalise=renormalise)
    assert not bool(dx[0].any()) and not bool(dx[logits == -INF].any())


@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_select_backward_takes_any_ids(score, renormalise):
    """The same expert twice adds up; ids that are no expert's have no part."""
    logits = normal(23, 4, 300)
    ids = torch.tensor([[5, 5, 7, 5], [0, 299, 300, -7], [-1, -1, -1, -1], [2**31 - 1, 8, 8, -2**31]],
                       dtype=torch.int32, device="cuda:0")
    dgates = normal(24, 4, 4)
    got = ops.expert_select_backward(dgates, logits, ids, score=score, renormalise=renormalise)
    want, big = L.select_backward(dgates, logits, ids, score, renormalise)
    within(got, want, select_backward_bounds(want, big, logits, torch.float32, 4), "dlogits")
    assert not bool(got[2].any())


@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_select_gradient_against_differences(score, renormalise):
    """Central differences of the gates in 64 bits, off by h^2 = 1e-10 of them at most times
    their third derivatives, which are below 10."""
    logits = normal(25, 40, 30)
    ids, _ = ops.expert_select(logits, 4, score=score)
    dgates = normal(26, 40, 4)
    grad = ops.expert_select_backward(dgates, logits, ids, score=score, renormalise=renormalise, scale=2.0).double()
    _, big = L.select_backward(dgates, logits, ids, score, renormalise, 2.0)
    x, step = logits.double(), normal(27, 40, 30).double()
    up, down = (L.gates_of(x + s * step, ids, score, renormalise, 2.0) for s in (1e-5, -1e-5))
    want = ((up - down) * dgates.double()).sum(1) / 2e-5
    off = ((grad * step).sum(1) - want).abs()
    bound = (select_backward_bounds(grad, big, logits, torch.float32, 4) * step.abs()).sum(1)
    assert bool((off <= bound + 1e-7).all())


def test_select_graph_replays_and_streams():
    logits, dgates = inputs(30, 130, 64, "bf16", 0.1), normal(31, 130, 4)
    bias = normal(32, 64, scale=0.1)

    def run(stream=None):
        ids, gates = ops.expert_select(logits, 4, score="sigmoid", bias=bias, groups=8, kept_groups=3, group_best=2,
                                       renormalise=True, stream=stream)
        return [ids, gates, ops.expert_select_backward(dgates, logits, ids, score="sigmoid", renormalise=True,
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
        logits.copy_(inputs(40 + i, 130, 64, "bf16", 0.2))
        want = run()
        torch.cuda.synchronize()
        for t in held:
            t.fill_(99)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), i
