"""An expert-parallel layer on virtual ranks: the collectives and the products together.

Every rank holds its own tokens and a share of the experts. Per rank: router logits
(``ops.linear``), the choice of experts (``ops.expert_select``), a route of the tokens'
choices by expert (``ops.expert_route``, ``ops.expert_dispatch``), an AllToAll that takes
rows to their experts' ranks (``Plan``), the experts' two products (``ops.grouped_linear``),
an AllToAll back, the gated sum (``ops.expert_combine``) and a tensor-parallel output
projection whose partial products an AllReduce sums. Run it on an MI355X:

    python examples/expert_layer.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from chunk_schedule_execution_amd import Plan, PlanConfig, ops, programs  # noqa: E402


class ExpertLayer:
    """ranks virtual ranks with experts / ranks experts each; tokens per rank, choices
    experts per token, width in and out, hidden inside an expert."""

    def __init__(self, ranks=4, tokens=96, choices=2, experts=8, width=256, hidden=512, seed=0, device="cuda:0"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.ranks, self.tokens, self.choices, self.experts = ranks, tokens, choices, experts
        self.width, self.hidden, self.device = width, hidden, device
        self.local = experts // ranks

        def weights(*shape):
            return (torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5).to(torch.bfloat16)

        self.router = weights(experts, width)
        self.up = [weights(self.local, hidden, width) for _ in range(ranks)]
        self.up_bias = [weights(self.local, hidden) for _ in range(ranks)]
        self.down = [weights(self.local, width, hidden) for _ in range(ranks)]
        self.project = weights(width, width)  # rank r multiplies columns r width / ranks .. of its input
        # a rank may send all its rows to one other rank: every block holds that many
        self.block = tokens * choices
        n = ranks * self.block * width
        self.rows_plan = Plan(programs.direct_alltoall(ranks), 1, PlanConfig(dtype="bf16", max_count=n))
        self.counts_plan = Plan(programs.direct_alltoall(ranks), 1, PlanConfig(dtype="i32", max_count=experts))
        self.sum_plan = Plan(programs.ring_allreduce(ranks), 1,
                             PlanConfig(dtype="bf16", max_count=ranks * tokens * width))

    def exchange(self, sent, plan, count):
        got = [torch.empty_like(t) for t in sent]
        plan.execute(sent, got, count)
        return got

    def forward(self, xs):
        """xs: per rank (tokens, width) bf16. Returns the layer's outputs per rank, all tokens
        of all ranks (the AllReduce's result), and the routes."""
        P, C, W, L = self.ranks, self.block, self.width, self.local
        routes, sent, counts = [], [], []
        for x in xs:
            ids, gates = ops.expert_select(ops.linear(x, self.router), self.choices, renormalise=True)
            offsets, positions, slots = ops.expert_route(ids, self.experts)
            rows = ops.expert_dispatch(x, slots, self.choices)
            # rank d's rows follow each other; row i goes to place i - begin of block d
            begin = offsets[:-1:L].long()
            row = torch.arange(C, device=self.device)
            dest = torch.searchsorted(offsets[L::L].contiguous(), row.to(torch.int32), right=True)
            place = dest * C + row - begin[dest]
            packed = torch.zeros(P * C, W, dtype=x.dtype, device=self.device)
            packed[place] = rows
            sent.append(packed)
            counts.append((offsets[1:] - offsets[:-1]).contiguous())
            routes.append((positions, gates, place, ids))
        there = self.exchange(sent, self.rows_plan, P * C * W)
        there_counts = self.exchange(counts, self.counts_plan, self.experts)

        outs = []
        for r in range(P):
            # block s holds rank s's rows for this rank, by local expert; padding gets id -1
            ends = there_counts[r].view(P, L).cumsum(1)
            at = torch.arange(C, device=self.device).expand(P, C).contiguous()
            ids = torch.searchsorted(ends.long(), at, right=True)
            ids = torch.where(ids < L, ids, -1).to(torch.int32).view(P * C, 1)
            offsets, positions, slots = ops.expert_route(ids, L)
            rows = ops.expert_dispatch(there[r], slots, 1)
            inner = ops.grouped_linear(rows, self.up[r], offsets, bias=self.up_bias[r], activation="gelu")
            result = ops.grouped_linear(inner, self.down[r], offsets)
            outs.append(ops.expert_combine(result, positions))  # back in the blocks' order
        back = self.exchange(outs, self.rows_plan, P * C * W)

        mixed = []
        for r in range(P):
            positions, gates, place, _ = routes[r]
            mixed.append(ops.expert_combine(back[r][place], positions, gates))
        # the output projection's weights are split by input columns: every rank multiplies its
        # share of all tokens' columns and the AllReduce sums the partial products
        everything = torch.cat(mixed)
        share = W // P
        partial = [ops.linear(everything[:, r * share:(r + 1) * share], self.project[:, r * share:(r + 1) * share])
                   for r in range(P)]
        summed = [torch.empty_like(t) for t in partial]
        self.sum_plan.execute(partial, summed, P * self.tokens * W)
        for plan in (self.rows_plan, self.counts_plan, self.sum_plan):
            plan.status()
        return summed, routes

    def reference(self, xs, routes):
        """The layer from its definition in 64 bits, for the routes taken."""
        mixed = []
        for x, (_, gates, _, ids) in zip(xs, routes):
            y = torch.zeros(self.tokens, self.width, dtype=torch.float64, device=self.device)
            for e in range(self.experts):
                r, i = divmod(e, self.local)
                z = x.double() @ self.up[r][i].double().t() + self.up_bias[r][i].double()
                h = z * torch.special.ndtr(z)
                y += (h @ self.down[r][i].double().t()) * (gates.double() * (ids == e)).sum(1, keepdim=True)
            mixed.append(y)
        return torch.cat(mixed) @ self.project.double().t()


def main():
    layer = ExpertLayer()
    g = torch.Generator(device="cuda:0")
    g.manual_seed(1)
    xs = [torch.randn(layer.tokens, layer.width, generator=g, device="cuda:0").to(torch.bfloat16)
          for _ in range(layer.ranks)]
    outs, routes = layer.forward(xs)
    want = layer.reference(xs, routes)
    for r, out in enumerate(outs):
        print(f"rank {r}: {tuple(out.shape)}, error {float((out.double() - want).norm() / want.norm()):.2e}")


if __name__ == "__main__":
    main()
