"""Groups are ranked by their scores in 64 bits, also where logits that differ have equal ones:
sigmoids that round to 1, softmax terms that round to 0 or are equal beside the largest."""

import math

import pytest
import torch

from chunk_schedule_execution_amd import ops
from oracle import layers as L
from products_util import TYPES, normal

pytestmark = pytest.mark.gpu

INF = math.inf

# experts, choices, groups, kept groups: 16 lanes a token by vectors and by single values, a group's
# experts in parts of lanes or not; a wave a token for many experts, choices or groups
SIZES = [(64, 4, 8, 3), (63, 3, 9, 2), (32, 2, 32, 5), (256, 8, 2, 1), (500, 5, 20, 7), (640, 6, 10, 4), (128, 4, 64, 9),
         (96, 14, 6, 3)]


def check(logits, choices, groups, kept, score):
    for best in (1, 2):
        kw = dict(score=score, groups=groups, kept_groups=kept, group_best=best)
        ids, _ = ops.expert_select(logits, choices, **kw)
        want, _ = L.select(logits, choices, **kw)
        wrong = [t for t in range(len(want)) if ids[t].tolist() != want[t].tolist()]
        assert not wrong, (best, wrong[:5], ids[wrong[0]].tolist(), want[wrong[0]].tolist())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("experts,choices,groups,kept", SIZES)
def test_groups_of_sigmoids_near_one(experts, choices, groups, kept, dtype):
    x = normal(1, 150, experts)
    far = x * 25.0  # some of a row above 37, where 1 + exp(-x) is 1
    far[50:100] = 45.0 + 4.0 * x[50:100]  # all of them
    far[100:110] = 40.0
    far[110:150] = (x[110:150] > 1.0) * 50.0 + x[110:150].round()  # ties of logits as well
    check(far.to(TYPES[dtype]), choices, groups, kept, "sigmoid")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("experts,choices,groups,kept", SIZES)
def test_groups_of_softmax_near_zero(experts, choices, groups, kept, dtype):
    x = normal(2, 120, experts)
    x[:60] = x[:60] * 20.0 - 900.0  # all terms but the first expert's are 0
    x[:60, 0] = 0.0
    x[60:90] = x[60:90] * 400.0  # some of them
    x[90:] = (x[90:] * 2).round()
    check(x.to(TYPES[dtype]), choices, groups, kept, "softmax")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,choices,groups,kept", SIZES)
def test_groups_of_logits_that_scores_cannot_tell(experts, choices, groups, kept, score):
    """Logits so small that all scores are the same in 64 bits: the first groups stay, and in
    them the largest logits are chosen."""
    check(normal(3, 60, experts) * 1e-25, choices, groups, kept, score)


@pytest.mark.parametrize("experts,choices,groups,kept", SIZES)
def test_groups_with_nan_and_infinities(experts, choices, groups, kept):
    x = normal(4, 40, experts)
    x[:10, experts - 1] = INF
    x[10:20, experts // 2] = float("nan")
    x[20:30, experts // 2], x[20:30, experts - 1] = INF, float("nan")
    x[30:, : experts - experts // groups] = -INF  # one group open
    for score in ("softmax", "sigmoid"):
        check(x, choices, groups, kept, score)
