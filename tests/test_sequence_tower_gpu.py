"""The sequence model of examples/ runs the lookup, the recurrence, the experts
and both optimizers together: it learns its task, serving event by event
reaches the states of the whole sequences, and its gradients through the
library's operators are those of plain torch operations."""
import importlib.util
import os

import pytest

import sparse_lookup_gb300 as sl
from sparse_lookup_gb300 import build as slbuild

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    slbuild.build()
    sl.lib()
    spec = importlib.util.spec_from_file_location("sequence_tower", os.path.join(ROOT, "examples",
                                                                                "sequence_tower.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_it_learns_and_serves(example):
    """Half of the events name the session's group.  From ln 8 = 2.08 the loss
    falls below two thirds of it, and serving finds the group far more often
    than one time in eight.  The states that serving leaves are the ones after
    the whole sequences: both are fp32 sums of at most 40 terms of a convex
    combination, 40 * 20 u apart at the most."""
    import torch
    losses, right, (tower, ids, offsets, served) = example.main(verbose=False)
    assert 1.5 < losses[0] < 2.7 and sum(losses[-5:]) / 5 < 1.39, losses
    assert right > 0.5, right
    B, L, D = offsets.numel() - 1, tower.max_len, tower.dim
    _, seq = tower.plan.forward(B, ids, offsets, None, None)
    with torch.no_grad():
        both = seq.view(B, L, D).double() @ tower.w_in.double()
    x, gate = both[..., :D].float(), both[..., D:].float()
    _, last = tower.scan.forward(x, gate, offsets)
    # the projections themselves (fp32 products of 32 terms) differ by up to 1e-5 of the largest value
    assert (last - served).abs().max() <= 1e-4 * x.abs().max()


def test_gradients_match_plain_torch(example):
    """One batch through the operators and through elementary torch operations
    in 64 bits; every gradient within 1e-4 of its largest element (fp32
    products and sums of at most a few thousand terms)."""
    import torch
    tower = example.SequenceTower(200, 16, 12, 6, n_experts=4, top_k=2, n_classes=5, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(2)
    ids, offsets, groups = example.sessions(gen, 6, 12, 200, 5)
    B, L, D = 6, 12, 16
    lens = offsets.diff().long()
    table = tower.table.clone()
    params = [p.detach().double().requires_grad_() for p in tower.params]
    w_in, w_route, w_up, w_down, w_out = params
    seq = torch.zeros(B, L, D, dtype=torch.float64, device="cuda")
    for b in range(B):
        seq[b, :lens[b]] = table[ids[offsets[b]:offsets[b + 1]]].double()
    seq.requires_grad_()
    both = seq @ w_in
    h, hs = torch.zeros(B, D, dtype=torch.float64, device="cuda"), []
    for t in range(L):
        a = torch.sigmoid(both[:, t, D:])
        h = a * h + (1 - a) * both[:, t, :D]
        hs.append(h)
    live = (torch.arange(L, device="cuda")[None] < lens[:, None]).reshape(-1)
    tokens = torch.stack(hs, 1).reshape(B * L, D)[live]
    logits, chosen = (tokens @ w_route).topk(2, dim=1)
    weights, out = torch.softmax(logits, 1), tokens
    for k in range(2):
        up = torch.relu(torch.einsum("nd,ndf->nf", tokens, w_up[chosen[:, k]]))
        out = out + weights[:, k, None] * torch.einsum("nf,nfd->nd", up, w_down[chosen[:, k]])
    loss = torch.nn.functional.cross_entropy(out @ w_out, groups.repeat_interleave(lens))
    loss.backward()
    before, acc = tower.table.clone(), tower.acc.clone()
    got = tower.step(ids, offsets, groups, lr_sparse=0.05, lr_dense=0.0)
    assert abs(got.item() - loss.item()) <= 1e-5
    for p, q in zip(tower.params, params):
        assert (p.grad.double() - q.grad).abs().max() <= 1e-4 * q.grad.abs().max()
    # the table took one Adagrad step along the sequence gradient
    g = torch.zeros_like(before, dtype=torch.float64)
    rows = torch.cat([ids[offsets[b]:offsets[b + 1]] for b in range(B)])
    g.index_add_(0, rows, torch.cat([seq.grad[b, :lens[b]] for b in range(B)]))
    grown = (tower.acc - acc).double()
    assert (grown.sqrt() - g.abs()).abs().max() <= 1e-4 * g.abs().max()
