"""The model of examples/delta_tower.py runs the lookup, the norms, the delta rule,
the gate, the experts and both optimizers together: serving event by event
reaches the states of the whole sequences, and its gradients through the library's
operators are those of plain torch operations."""
import importlib.util
import os
import sys

import pytest

import sparse_lookup_gb300 as sl
from sparse_lookup_gb300 import build as slbuild

pytestmark = pytest.mark.gpu

EXAMPLES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


@pytest.fixture(scope="module")
def example():
    slbuild.build()
    sl.lib()
    sys.path.insert(0, EXAMPLES)
    try:
        spec = importlib.util.spec_from_file_location("delta_tower", os.path.join(EXAMPLES, "delta_tower.py"))
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
    finally:
        sys.path.remove(EXAMPLES)
    return mod


def test_it_trains_and_serves(example):
    """The states that serving leaves are the ones after the whole sequences: both are fp32 recurrences of at most 40
    steps whose inputs (products of 32 terms) differ by roundings, 1e-4 of the largest."""
    import math

    import torch
    losses, (tower, ids, offsets, served) = example.main(steps=6, verbose=False)
    assert len(losses) == 6 and all(math.isfinite(x) for x in losses)
    B, L, D = offsets.numel() - 1, tower.max_len, tower.dim
    _, seq = tower.plan.forward(B, ids, offsets, None, None)
    with torch.no_grad():
        normed, _ = tower.norm.forward(seq.view(B, L, D), tower.norms[0], tower.norms[1], offsets)
        _, last = tower.scan.forward(*tower.inputs(normed), offsets)
    assert (last - served).abs().max() <= 1e-4 * last.abs().max()


def test_gradients_match_plain_torch(example):
    """One batch through the operators and through elementary torch operations in 64 bits; every gradient within 1e-4
    of its largest element (fp32 products and sums of at most a few thousand terms)."""
    import torch
    H, D, E, K, C = 2, 16, 4, 2, 5
    tower = example.DeltaTower(200, D, H, 12, 6, n_experts=E, top_k=K, n_classes=C, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(2)
    ids, offsets, groups = example.sessions(gen, 6, 12, 200, C)
    B, L = 6, 12
    lens = offsets.diff().long()
    _, seq = tower.plan.forward(B, ids, offsets, None, None)
    seq = seq.view(B, L, D).clone().requires_grad_()
    for p in tower.params:
        p.grad.zero_()
    loss = tower.loss(seq, offsets, groups)
    loss.backward()
    # the same in 64 bits
    x = seq.detach().double().requires_grad_()
    params = [p.detach().double().requires_grad_() for p in tower.params]
    w_in, w_mix, n0w, n0b, n1w, n1b, w_route, w_up, w_down, w_out = params

    def norm(t, w, b):
        c = t - t.mean(-1, keepdim=True)
        return c / (c.square().mean(-1, keepdim=True) + tower.norm.eps).sqrt() * w + b
    live = torch.arange(L, device="cuda")[None] < lens[:, None]
    all_ = (norm(x, n0w, n0b) * live[..., None]) @ w_in
    q, k, v = (all_[..., i * D:(i + 1) * D].unflatten(-1, (H, D // H)) for i in range(3))
    k = torch.nn.functional.normalize(k, dim=-1, eps=1e-6)
    decay = torch.exp(-torch.nn.functional.softplus(all_[..., 3 * D:3 * D + H] - 3.0))
    beta = torch.sigmoid(all_[..., 3 * D + H:])
    S, ys = torch.zeros(B, H, D // H, D // H, dtype=torch.float64, device="cuda"), []
    for t in range(L):
        S1 = S * decay[:, t, :, None, None]
        e = v[:, t] - (S1 * k[:, t, :, :, None]).sum(2)
        S = S1 + k[:, t, :, :, None] * (beta[:, t, :, None] * e)[:, :, None]
        ys.append(tower.scan.scale * (S * q[:, t, :, :, None]).sum(2))
    tokens = (x + torch.stack(ys, 1).flatten(-2) @ w_mix)[live]
    normed = norm(tokens, n1w, n1b)
    logits = normed @ w_route
    top, chosen = logits.topk(K, 1)
    weights, p = torch.softmax(top, 1), torch.softmax(logits, 1)
    n = logits.shape[0]
    f = torch.bincount(chosen.reshape(-1), minlength=E).double() / (n * K)
    experts = 0
    for j in range(K):
        e = chosen[:, j]
        hidden = torch.relu(torch.einsum("nd,ndh->nh", normed, w_up[e]))
        experts = experts + weights[:, j, None] * torch.einsum("nh,nhd->nd", hidden, w_down[e])
    scores = (tokens + experts) @ w_out
    want = torch.nn.functional.cross_entropy(scores, groups.repeat_interleave(lens))
    want = want + 1e-2 * E * (f * p.mean(0)).sum() + 1e-3 * torch.logsumexp(logits, 1).square().mean()
    want.backward()
    assert abs(loss.item() - want.item()) <= 1e-5 * abs(want.item())
    for got, ref in [(seq.grad, x.grad)] + [(a.grad, b.grad) for a, b in zip(tower.params, params)]:
        assert (got.double() - ref).abs().max() <= 1e-4 * ref.abs().max()
