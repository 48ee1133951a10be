"""A deeper sequence model over looked-up behaviour sequences: the padded lookup,
a layer norm and the gated delta rule over time, a second norm and a layer of
experts behind a gate with its balance and z losses, trained by sparse Adagrad on
the table and AdamW on the dense weights; then the same model one event at a time,
as a server runs it.

    python examples/delta_tower.py [--steps 40]

The task is that of sequence_tower.py: a session walks through the items of one of
several hidden groups, and the model predicts the group from the events so far.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from sequence_tower import Combine, Dispatch, sessions, sl  # noqa: E402
from sparse_lookup_gb300.synth import ColumnSpec  # noqa: E402


class Norm(torch.autograd.Function):
    """LayerNorm over padded sequences or rows."""

    @staticmethod
    def forward(ctx, norm, x, weight, bias, offsets):
        y, stats = norm.forward(x, weight, bias, offsets)
        ctx.norm, ctx.offsets = norm, offsets
        ctx.save_for_backward(x, weight, stats)
        return y

    @staticmethod
    def backward(ctx, grad_y):
        x, weight, stats = ctx.saved_tensors
        return (None, *ctx.norm.backward(x, grad_y.contiguous(), stats, weight, ctx.offsets), None)


class Delta(torch.autograd.Function):
    """DeltaScan with its gradients, over sequences whose lengths are the lookup's own bag offsets."""

    @staticmethod
    def forward(ctx, scan, q, k, v, decay, beta, offsets):
        y, _ = scan.forward(q, k, v, decay, beta, offsets)
        ctx.scan, ctx.offsets = scan, offsets
        ctx.save_for_backward(q, k, v, decay, beta)
        return y

    @staticmethod
    def backward(ctx, grad_y):
        return (None, *ctx.scan.backward(*ctx.saved_tensors, grad_y.contiguous(), ctx.offsets)[:5], None)


class Choose(torch.autograd.Function):
    """ExpertRouter.gate: the choices' weights and the two losses; the choices themselves by the gate."""

    @staticmethod
    def forward(ctx, router, logits, found):
        gate = router.gate(logits)
        found.append(gate)
        ctx.router, ctx.gate = router, gate
        ctx.save_for_backward(logits)
        return gate.weights, gate.losses

    @staticmethod
    def backward(ctx, grad_weights, grad_losses):
        logits, = ctx.saved_tensors
        return None, ctx.router.gate_backward(logits, ctx.gate, grad_weights.contiguous(), grad_losses.contiguous()), None


class DeltaTower:
    """items [num_items, dim] -> norm -> delta rule -> norm -> gated experts -> classes."""

    def __init__(self, num_items, dim, heads, max_len, max_batch, n_experts, top_k, n_classes, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape, scale):
            return (torch.randn(*shape, generator=gen, device="cuda") * scale).requires_grad_()

        def constant(value, n):
            return torch.full((n,), value, device="cuda").requires_grad_()
        self.dim, self.heads, self.max_len, self.n_experts = dim, heads, max_len, n_experts
        self.table = torch.randn(num_items, dim, generator=gen, device="cuda") * 0.1
        self.acc = torch.zeros_like(self.table)
        column = ColumnSpec("identity", "padded", num_items, dim, 0, pad_len=max_len)
        self.plan = sl.Plan([column], [self.table], [self.acc], max_batch=max_batch, max_ids=max_batch * max_len,
                            training=True)
        self.norm = sl.LayerNorm(dim)
        self.scan = sl.DeltaScan(dim // heads, dim // heads, heads, max_batch, max_len, training=True)
        self.router = sl.ExpertRouter(n_experts, top_k, max_batch * max_len, align=8)
        self.w_in = weight(dim, 3 * dim + 2 * heads, scale=dim ** -0.5)   # queries, keys, values; decay and beta
        self.w_mix = weight(dim, dim, scale=dim ** -0.5)
        self.norms = [constant(1.0, dim), constant(0.0, dim), constant(1.0, dim), constant(0.0, dim)]
        self.w_route = weight(dim, n_experts, scale=dim ** -0.5)
        self.w_up = weight(n_experts, dim, 2 * dim, scale=dim ** -0.5)
        self.w_down = weight(n_experts, 2 * dim, dim, scale=(2 * dim) ** -0.5)
        self.w_out = weight(dim, n_classes, scale=dim ** -0.5)
        self.params = [self.w_in, self.w_mix, *self.norms, self.w_route, self.w_up, self.w_down, self.w_out]
        for p in self.params:
            p.grad = torch.zeros_like(p)                                  # AdamW reads them where they are
        self.optimizer = sl.AdamW([p.detach() for p in self.params], [p.grad for p in self.params], weight_decay=0.01,
                                  seed=seed)

    def inputs(self, x):
        """q, k, v, decay and beta of normalised events [..., dim]."""
        D, H = self.dim, self.heads
        all_ = x @ self.w_in
        q, k, v = (all_[..., i * D:(i + 1) * D].unflatten(-1, (H, D // H)) for i in range(3))
        k = torch.nn.functional.normalize(k, dim=-1, eps=1e-6)
        decay = -torch.nn.functional.softplus(all_[..., 3 * D:3 * D + H] - 3.0)
        return q, k, v, decay, torch.sigmoid(all_[..., 3 * D + H:])

    def classes(self, events, mixed):
        """events [n, dim] and what the recurrence made of them: scores [n, classes], the gate's losses."""
        tokens = events + mixed.flatten(-2) @ self.w_mix
        normed = Norm.apply(self.norm, tokens, self.norms[2], self.norms[3], None)
        found = []
        weights, losses = Choose.apply(self.router, normed @ self.w_route, found)
        routing = self.router.route(found[0].experts)
        xs = Dispatch.apply(self.router, normed, routing)
        edges, out = routing.offsets.tolist(), []
        for e in range(self.n_experts):
            out.append(torch.relu(xs[edges[e]:edges[e + 1]] @ self.w_up[e]) @ self.w_down[e])
        out.append(torch.zeros_like(xs[edges[-1]:]))
        return (tokens + Combine.apply(self.router, torch.cat(out), weights, routing)) @ self.w_out, losses

    def loss(self, seq, offsets, targets):
        """seq [batch, time, dim], padded; the classes' cross entropy with the gate's losses."""
        B, L, D = seq.shape
        normed = Norm.apply(self.norm, seq, self.norms[0], self.norms[1], offsets)
        mixed = Delta.apply(self.scan, *self.inputs(normed), offsets)
        live = (torch.arange(L, device="cuda")[None] < offsets.diff()[:, None]).reshape(-1)
        events = torch.nonzero(live)[:, 0]
        scores, losses = self.classes(seq.reshape(B * L, D)[events], mixed.flatten(0, 1)[events])
        entropy = torch.nn.functional.cross_entropy(scores, targets.repeat_interleave(offsets.diff().long()))
        return entropy + (losses * torch.tensor([1e-2, 1e-3], device="cuda")).sum()

    def step(self, ids, offsets, targets, lr_sparse=0.05, lr_dense=3e-3):
        """One training step; returns the loss (a tensor)."""
        B, L, D = offsets.numel() - 1, self.max_len, self.dim
        _, seq = self.plan.forward(B, ids, offsets, None, None)
        seq = seq.view(B, L, D).requires_grad_()
        loss = self.loss(seq, offsets, targets)
        for p in self.params:
            p.grad.zero_()
        loss.backward()
        self.plan.backward_update(None, seq.grad.contiguous().view(-1), lr_sparse, 1e-10)
        self.optimizer.step(lr_dense)
        return loss.detach()

    def serve(self, items, rows, states):
        """One event for each of n sessions, their states rows of a pool [rows, heads, dim / heads, dim / heads]
        (updated in place): scores [n, classes]."""
        with torch.no_grad():
            x = self.table[items]
            normed, _ = self.norm.forward(x, self.norms[0], self.norms[1])
            mixed = self.scan.step(*(t.contiguous() for t in self.inputs(normed)), rows, states)
            return self.classes(x, mixed)[0]


def main(steps=40, batch=64, max_len=40, num_items=2000, n_classes=8, dim=32, heads=2, verbose=True):
    tower = DeltaTower(num_items, dim, heads, max_len, batch, n_experts=8, top_k=2, n_classes=n_classes)
    gen = torch.Generator(device="cuda").manual_seed(1)
    losses = []
    for i in range(steps):
        losses.append(tower.step(*sessions(gen, batch, max_len, num_items, n_classes)))
        if verbose and (i % 10 == 0 or i == steps - 1):
            print("step %3d  loss %.4f" % (i, losses[-1].item()))
    assert tower.plan.device_status() == 0
    # the same sessions, one event at a time
    ids, offsets, groups = sessions(gen, batch, max_len, num_items, n_classes)
    pool = torch.zeros(4 * batch, heads, dim // heads, dim // heads, device="cuda")
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
    return [x.item() for x in losses], (tower, ids, offsets, pool[mine])


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=40)
    main(ap.parse_args().steps)
