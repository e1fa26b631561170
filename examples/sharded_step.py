"""A training step of a block of experts and a loss whose vocabulary is spread over ranks.

The tokens are on every virtual rank, each rank holds an equal share of the vocabulary's
matrix. Forward: layer norm, the choice of experts (``ops.expert_select``), their route and
product, the gated sum, layer norm of its sum with the residual stream, and per rank the
cross entropy's sums over its share (``ops.linear_cross_entropy``), which an AllGather
(``Plan``) brings together and ``ops.cross_entropy_join`` joins. Backward: every rank's share
of the gradients, an AllReduce of the tokens' one, and the operators' gradients in turn. Run
it on an MI355X:

    python examples/sharded_step.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from chunk_schedule_execution_amd import Plan, PlanConfig, ops, programs  # noqa: E402

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


class ShardedStep:
    """ranks virtual ranks with vocabulary / ranks rows of its matrix each; tokens of `width`
    values, `choices` of `experts` experts each."""

    def __init__(self, ranks=4, tokens=64, width=64, experts=8, choices=2, vocabulary=512, dtype="f32",
                 score="sigmoid", seed=0, device="cuda:0"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        kind = DTYPES[dtype]
        self.ranks, self.tokens, self.width, self.share = ranks, tokens, width, vocabulary // ranks
        self.experts, self.choices, self.score, self.device = experts, choices, score, device

        def normal(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g, device=device) * scale).to(kind)

        self.w = {"norm1": 1 + normal(width, scale=0.1), "bias1": normal(width, scale=0.1),
                  "router": normal(experts, width, scale=width ** -0.5),
                  "expert": normal(experts, width, width, scale=width ** -0.5),
                  "norm2": 1 + normal(width, scale=0.1), "bias2": normal(width, scale=0.1)}
        self.shards = [normal(self.share, width, scale=2 * width ** -0.5) for _ in range(ranks)]
        self.balance = torch.randn(experts, generator=g, device=device) * 0.05
        self.gather = Plan(programs.ring_allgather(ranks), 1, PlanConfig(dtype="f32", max_count=2 * tokens))
        self.sum = Plan(programs.ring_allreduce(ranks), 1, PlanConfig(dtype=dtype, max_count=tokens * width))

    def run(self, x, targets):
        """x (tokens, width), targets (tokens,) int32 -> loss by token, the chosen experts, and
        the gradients of the tokens' mean loss by x, every weight and every rank's shard."""
        w, choice = self.w, dict(score=self.score, renormalise=True)
        n1, mean1, rstd1 = ops.layer_norm(x, weight=w["norm1"], bias=w["bias1"], save_stats=True)
        logits = ops.linear(n1, w["router"])
        ids, gates = ops.expert_select(logits, self.choices, bias=self.balance, **choice)
        offsets, positions, slots = ops.expert_route(ids, self.experts)
        rows = ops.expert_dispatch(n1, slots, self.choices)
        inner, preact = ops.grouped_linear(rows, w["expert"], offsets, activation="silu", save_preact=True)
        mixed = ops.expert_combine(inner, positions, gates)
        n2, total, mean2, rstd2 = ops.layer_norm(mixed, weight=w["norm2"], bias=w["bias2"], residual=x, save_stats=True)
        # every rank's (lse, picked) to all ranks
        parts = [torch.cat(ops.linear_cross_entropy(n2, v, targets, shard=r * self.share))
                 for r, v in enumerate(self.shards)]
        gathered = [torch.empty(self.ranks * 2 * self.tokens, device=self.device) for _ in parts]
        self.gather.execute(parts, gathered, 2 * self.tokens)
        lse_parts, picked = gathered[0].view(self.ranks, 2, self.tokens).unbind(1)
        loss, lse = ops.cross_entropy_join(lse_parts.contiguous(), picked.contiguous(), targets)

        dloss = torch.full_like(loss, 1.0 / self.tokens)
        shares = [ops.linear_cross_entropy_backward(dloss, n2, v, targets, lse, shard=r * self.share)
                  for r, v in enumerate(self.shards)]
        summed = [torch.empty_like(n2) for _ in shares]
        self.sum.execute([dx for dx, _ in shares], summed, self.tokens * self.width)
        grads = {"shards": [dv for _, dv in shares]}
        dtotal, grads["norm2"], grads["bias2"] = ops.layer_norm_backward(summed[0], total, mean2, rstd2,
                                                                         weight=w["norm2"], bias=True)
        dinner, dgates = ops.expert_combine_backward(dtotal, inner, positions, slots, gates)
        drows, grads["expert"] = ops.grouped_linear_backward(dinner, rows, w["expert"], offsets, preact=preact,
                                                             activation="silu")
        dlogits = ops.expert_select_backward(dgates, logits, ids, **choice)
        dn1, grads["router"] = ops.linear_backward(dlogits, n1, w["router"])
        dn1 = dn1 + ops.expert_combine(drows, positions)
        grads["x"], grads["norm1"], grads["bias1"] = ops.layer_norm_backward(dn1, x, mean1, rstd1, weight=w["norm1"],
                                                                             dtotal=dtotal, bias=True)
        for plan in (self.gather, self.sum):
            plan.status()
        return loss, ids, grads

    def reference(self, x, targets, ids):
        """The same from the definitions in 64 bits by automatic differentiation, for the
        experts chosen."""
        leaves = {name: t.double().requires_grad_(True) for name, t in dict(self.w, x=x).items()}
        shards = [v.double().requires_grad_(True) for v in self.shards]

        def norm(h, n):
            d = h - h.mean(1, keepdim=True)
            return d / (d.square().mean(1, keepdim=True) + 1e-5).sqrt() * leaves[f"norm{n}"] + leaves[f"bias{n}"]

        n1 = norm(leaves["x"], 1)
        z = n1 @ leaves["router"].t()
        p = torch.sigmoid(z) if self.score == "sigmoid" else torch.softmax(z, 1)
        gates = p.gather(1, ids.long())
        gates = gates / gates.sum(1, keepdim=True)
        mixed = torch.zeros_like(n1)
        for e in range(self.experts):
            y = torch.nn.functional.silu(n1 @ leaves["expert"][e].t())
            mixed = mixed + y * (gates * (ids == e)).sum(1, keepdim=True)
        z = norm(leaves["x"] + mixed, 2) @ torch.cat(shards).t()
        loss = torch.nn.functional.cross_entropy(z, targets.long(), ignore_index=-100, reduction="none")
        names = list(leaves)
        grads = torch.autograd.grad(loss.mean(), [leaves[n] for n in names] + shards)
        return loss.detach(), dict(zip(names, grads), shards=list(grads[len(names):]))


def tokens_of(step, seed, ignored=0.1):
    g = torch.Generator(device=step.device)
    g.manual_seed(seed)
    x = torch.randn(step.tokens, step.width, generator=g, device=step.device).to(step.shards[0].dtype)
    targets = torch.randint(0, step.ranks * step.share, (step.tokens,), generator=g, device=step.device)
    targets[torch.rand(step.tokens, generator=g, device=step.device) < ignored] = -100
    return x, targets.to(torch.int32)


def main():
    step = ShardedStep()
    x, targets = tokens_of(step, 1)
    loss, ids, grads = step.run(x, targets)
    want, want_grads = step.reference(x, targets, ids)
    print(f"loss {float(loss.mean()):.4f}, in 64 bits {float(want.mean()):.4f}")
    for name, g in want_grads.items():
        got, g = (torch.cat(v) if name == "shards" else v for v in (grads[name], g))
        print(f"gradient of {name}: error {float((got.double() - g).norm() / g.norm()):.2e}")


if __name__ == "__main__":
    main()
