"""A small sequence model over looked-up behaviour sequences: the padded lookup,
a gated recurrence over it, a layer of experts behind that, and a step of
sparse Adagrad on the table and of AdamW (8-bit states) on the dense weights;
then the same model one event at a time, as a server runs it.

    python examples/sequence_tower.py [--steps 60]

The task is synthetic: a session walks through the items of one of several
hidden groups, and the model predicts the group from the events so far.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_lookup_gb300 as sl  # noqa: E402
from sparse_lookup_gb300.synth import ColumnSpec  # noqa: E402


class Recurrence(torch.autograd.Function):
    """GatedScan with its gradient, over sequences whose lengths are the
    lookup's own bag offsets."""

    @staticmethod
    def forward(ctx, scan, x, gate, offsets):
        y, _ = scan.forward(x, gate, offsets)
        ctx.scan, ctx.offsets = scan, offsets
        ctx.save_for_backward(x, gate, y)
        return y

    @staticmethod
    def backward(ctx, grad_y):
        x, gate, y = ctx.saved_tensors
        grad_x, grad_gate, _ = ctx.scan.backward(x, gate, y, grad_y.contiguous(), ctx.offsets)
        return None, grad_x, grad_gate, None


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, router, x, routing):
        ctx.router, ctx.routing = router, routing
        return router.dispatch(x, routing)

    @staticmethod
    def backward(ctx, grad_xs):
        return None, ctx.router.dispatch_backward(grad_xs.contiguous(), ctx.routing), None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, router, ys, weights, routing):
        ctx.router, ctx.routing = router, routing
        ctx.save_for_backward(ys, weights)
        return router.combine(ys, weights, routing)

    @staticmethod
    def backward(ctx, grad_y):
        ys, weights = ctx.saved_tensors
        grad_ys, grad_weights = ctx.router.combine_backward(grad_y.contiguous(), ys, weights, ctx.routing)
        return None, grad_ys, grad_weights, None


class SequenceTower:
    """items [num_items, dim] -> recurrence -> experts -> classes."""

    def __init__(self, num_items, dim, max_len, max_batch, n_experts, top_k, n_classes, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape, scale):
            return (torch.randn(*shape, generator=gen, device="cuda") * scale).requires_grad_()
        self.dim, self.max_len, self.top_k, self.n_experts = dim, max_len, top_k, n_experts
        self.table = torch.randn(num_items, dim, generator=gen, device="cuda") * 0.1
        self.acc = torch.zeros_like(self.table)
        column = ColumnSpec("identity", "padded", num_items, dim, 0, pad_len=max_len)
        self.plan = sl.Plan([column], [self.table], [self.acc], max_batch=max_batch, max_ids=max_batch * max_len,
                            training=True)
        self.scan = sl.GatedScan(dim, max_batch, max_len)
        self.router = sl.ExpertRouter(n_experts, top_k, max_batch * max_len, align=8)
        self.w_in = weight(dim, 2 * dim, scale=dim ** -0.5)              # the recurrence's input and gate
        self.w_route = weight(dim, n_experts, scale=dim ** -0.5)
        self.w_up = weight(n_experts, dim, 2 * dim, scale=dim ** -0.5)
        self.w_down = weight(n_experts, 2 * dim, dim, scale=(2 * dim) ** -0.5)
        self.w_out = weight(dim, n_classes, scale=dim ** -0.5)
        self.params = [self.w_in, self.w_route, self.w_up, self.w_down, self.w_out]
        for p in self.params:
            p.grad = torch.zeros_like(p)                                  # AdamW reads them where they are
        self.optimizer = sl.AdamW([p.detach() for p in self.params], [p.grad for p in self.params],
                                  weight_decay=0.01, state_bits=8, seed=seed)

    def experts(self, tokens):
        """tokens [n, dim] through top_k experts each."""
        logits, chosen = (tokens @ self.w_route).topk(self.top_k, dim=1)
        routing = self.router.route(chosen.int())
        xs = Dispatch.apply(self.router, tokens, routing)
        edges, out = routing.offsets.tolist(), []
        for e in range(self.n_experts):
            out.append(torch.relu(xs[edges[e]:edges[e + 1]] @ self.w_up[e]) @ self.w_down[e])
        out.append(torch.zeros_like(xs[edges[-1]:]))
        return tokens + Combine.apply(self.router, torch.cat(out), torch.softmax(logits, 1), routing)

    def classes(self, states):
        return self.experts(states) @ self.w_out

    def step(self, ids, offsets, targets, lr_sparse=0.05, lr_dense=3e-3):
        """One training step; returns the loss (a tensor)."""
        B, L, D = offsets.numel() - 1, self.max_len, self.dim
        _, seq = self.plan.forward(B, ids, offsets, None, None)
        seq = seq.view(B, L, D).requires_grad_()
        both = seq @ self.w_in
        h = Recurrence.apply(self.scan, both[..., :D], both[..., D:], offsets)
        live = (torch.arange(L, device="cuda")[None] < offsets.diff()[:, None]).reshape(-1)
        tokens = torch.nonzero(live)[:, 0]
        scores = self.classes(h.reshape(B * L, D)[tokens])
        loss = torch.nn.functional.cross_entropy(scores, targets.repeat_interleave(offsets.diff().long()))
        for p in self.params:
            p.grad.zero_()
        loss.backward()
        self.plan.backward_update(None, seq.grad.contiguous().view(-1), lr_sparse, 1e-10)
        self.optimizer.step(lr_dense)
        return loss.detach()

    def serve(self, items, rows, states):
        """One event for each of n sessions, their states rows of a pool
        (updated in place): scores [n, classes]."""
        with torch.no_grad():
            both = self.table[items] @ self.w_in
            return self.classes(self.scan.step(both[:, :self.dim], both[:, self.dim:], rows, states))


def sessions(gen, batch, max_len, num_items, n_classes):
    """ids, offsets and groups of a batch of sessions."""
    groups = torch.randint(0, n_classes, (batch,), generator=gen, device="cuda")
    lens = torch.randint(3, max_len + 1, (batch,), generator=gen, device="cuda")
    offsets = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).int()
    of = groups.repeat_interleave(lens)
    share = num_items // n_classes
    ids = of * share + torch.randint(0, share, of.shape, generator=gen, device="cuda")
    noise = torch.rand(of.shape, generator=gen, device="cuda") < 0.5
    return torch.where(noise, torch.randint(0, num_items, of.shape, generator=gen, device="cuda"), ids), offsets, groups


def main(steps=60, batch=64, max_len=40, num_items=2000, n_classes=8, dim=32, verbose=True):
    tower = SequenceTower(num_items, dim, max_len, batch, n_experts=8, top_k=2, n_classes=n_classes)
    gen = torch.Generator(device="cuda").manual_seed(1)
    losses = []
    for i in range(steps):
        losses.append(tower.step(*sessions(gen, batch, max_len, num_items, n_classes)))
        if verbose and (i % 10 == 0 or i == steps - 1):
            print("step %3d  loss %.4f" % (i, losses[-1].item()))
    for status in (tower.plan.device_status(), tower.scan.device_status()):
        assert status == 0, status
    # the same sessions, one event at a time
    ids, offsets, groups = sessions(gen, batch, max_len, num_items, n_classes)
    pool = torch.zeros(4 * batch, dim, device="cuda")
    mine = torch.randperm(4 * batch, generator=gen, device="cuda")[:batch]
    lens, right, scored = offsets.diff().long(), 0, 0
    for t in range(max_len):
        on = t < lens
        items = ids[(offsets[:-1].long() + t).clamp(max=ids.numel() - 1)]
        rows = torch.where(on, mine, -1)                                  # sessions that are over: dropped
        scores = tower.serve(items, rows, pool)
        if t >= 2:
            right += (scores.argmax(1) == groups)[on].sum().item()
            scored += on.sum().item()
    if verbose:
        print("served: %.1f %% of the events after the third give the session's group" % (100.0 * right / scored))
    return [x.item() for x in losses], right / scored, (tower, ids, offsets, pool[mine])


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    main(ap.parse_args().steps)
