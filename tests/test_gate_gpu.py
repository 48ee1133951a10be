"""The router's gate and its gradient against the formulas in 64 bits.  Choices
and counts are exact.

Tolerances, u = 2^-24: expf is within 2 u; a row's sum of at most 2048
exponentials is added up in chains of at most 64 + 5, so probabilities and
weights are within 80 u + 2 u |logit - lse| of themselves.  Sums over n tokens:
n u sum|terms| in any order, and each term as above."""
import pytest

import sparse_lookup_gb300 as sl
from sparse_lookup_gb300 import build as slbuild

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
TINY = {"float32": 1e-37, "bfloat16": 1e-37, "float16": 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def built():
    slbuild.build()
    sl.lib()


def make(T, E, dtype, seed, steps=None):
    """Logits with a tilt; steps: rounded so that rows hold equal ones."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, E, generator=gen, device="cuda") + torch.randn(E, generator=gen, device="cuda")
    if steps:
        x = (x * steps).round() / steps
    return x.to(getattr(torch, dtype)), gen


def reference(logits, K, live, normalize, gw, gl):
    """Outputs and bounds, with loops over the choices."""
    import torch
    T, E = logits.shape
    x = logits.double()
    on = torch.ones(T, dtype=torch.bool, device="cuda") if live is None else live.clone()
    on &= ~(torch.where(on[:, None], x, 0.0) == -torch.inf).all(1)
    x = torch.where(on[:, None], x, 0.0)
    lse = torch.logsumexp(x, 1)
    p = torch.softmax(x, 1)     # not exp(x - lse), which loses the sum beside the types' lowest value
    left, ids = x.clone(), torch.full((T, K), -1, dtype=torch.int64, device="cuda")
    for k in range(K):
        best = left.amax(1, keepdim=True)
        at = torch.where(left == best, torch.arange(E, device="cuda"), E).amin(1)
        ids[:, k] = torch.where(on & (best[:, 0] > -torch.inf), at, -1)
        left.scatter_(1, at[:, None], -torch.inf)
    held = ids >= 0
    w = torch.where(held, p.gather(1, ids.clamp(min=0)), 0.0)
    if normalize:
        w = torch.where(held, w / w.sum(1, keepdim=True).clamp(min=1e-300), 0.0)
    counts = torch.bincount(ids[held], minlength=E)
    n = max(int(on.sum()), 1)
    f = counts.double() / (n * K)
    losses = torch.stack([E * (f * p[on].sum(0) / n).sum(), lse[on].square().sum() / n])
    far = (x - lse[:, None]).abs()
    far = torch.where(far < 200, far, 0.0).amax(1)
    rel = (80 + 4 * far) * U                      # of a probability
    c = gl[0].double() * E * f / n
    z = 2 * gl[1].double() * lse / n
    dp = c[None] + z[:, None]
    along = (p * c).sum(1)
    g = torch.where(held, gw.double(), 0.0)
    mean = (w * g).sum(1)
    grad = p * (dp - along[:, None] - (0 if normalize else mean[:, None]))
    extra = w * (g - (mean[:, None] if normalize else 0))
    grad.scatter_add_(1, ids.clamp(min=0), torch.where(held, extra, 0.0))
    grad = torch.where(on[:, None], grad, 0.0)
    size = p * (c.abs()[None] + (along.abs() + z.abs() + (w * g.abs()).sum(1))[:, None])
    size.scatter_add_(1, ids.clamp(min=0), w * (g.abs() + (w * g.abs()).sum(1, keepdim=True)))
    return dict(experts=ids.int(), weights=w, counts=counts.int(), losses=losses, grad=grad, rel=rel, size=size, n=n,
                lse=lse, on=on)


def check(logits, K, live=None, normalize=True, seed=0, router=None):
    import torch
    T, E = logits.shape
    dtype = str(logits.dtype).replace("torch.", "")
    gen = torch.Generator(device="cuda").manual_seed(seed)
    gw = torch.randn(T, K, generator=gen, device="cuda")
    gl = torch.tensor([0.3 * max(T, 1), 0.1 * max(T, 1)], device="cuda")
    router = router or sl.ExpertRouter(E, K, max(T, 1))
    g = router.gate(logits, live=live, normalize=normalize)
    r = reference(logits, K, live, normalize, gw, gl)
    assert torch.equal(g.experts, r["experts"])
    assert torch.equal(g.counts, r["counts"])
    assert int(g.live_count) == int(r["on"].sum())
    rel = r["rel"][:, None]
    assert ((g.weights.double() - r["weights"]).abs() <= 2 * rel * r["weights"] + 1e-37).all()
    assert torch.equal(g.stats[:, 0] == -torch.inf, ~r["on"])
    worst = r["rel"].max() if T else 0.0
    bound = (T * U + 2 * worst + 8 * U) * r["losses"].abs() + 1e-37
    z = r["lse"][r["on"]].abs()
    bound[1] += (2 * z * (80 * U + 2 * U * z)).sum() / r["n"]         # of lse itself: the sum's error and a rounding
    held = torch.isfinite(r["losses"].float())      # others are beyond fp32 and round to infinity
    assert ((g.losses.double() - r["losses"]).abs() <= bound)[held].all(), (g.losses, r["losses"])
    assert torch.equal(g.losses[~held], r["losses"].float()[~held])
    got = router.gate_backward(logits, g, gw, gl).double()
    tol = (4 * rel + 80 * U) * r["size"] + HALF[dtype] * r["grad"].abs() + TINY[dtype]
    assert ((got - r["grad"]).abs() <= tol).all(), ((got - r["grad"]).abs() - tol).max()
    return router, g, r


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 4, 2), (8, 16, 2), (7, 5, 3), (33, 32, 8), (100, 17, 1), (1000, 37, 3),
                                   (5003, 128, 4), (300, 130, 6), (64, 512, 8), (50, 513, 2), (3000, 1024, 8),
                                   (40, 2047, 5), (90, 2048, 64), (20, 40, 40), (70000, 64, 2), (0, 8, 2)])
def test_gate(T, E, K, dtype):
    logits, _ = make(T, E, dtype, T + E)
    check(logits, K)
    check(logits, K, normalize=False, seed=1)


@pytest.mark.parametrize("dtype", ["float32", "float16"])
@pytest.mark.parametrize("E", [8, 30, 256, 1000])
def test_equal_logits_go_to_the_lowest_experts(E, dtype):
    logits, _ = make(400, E, dtype, E, steps=2)
    logits[3] = 0.5
    logits[4, E // 2:] = logits[4].max() + 1
    router, g, _ = check(logits, min(6, E))
    assert g.experts[3].tolist() == list(range(min(6, E)))
    assert g.experts[4].tolist()[:4] == list(range(E // 2, E // 2 + 4))


@pytest.mark.parametrize("normalize", [True, False])
def test_tokens_that_are_not_live(normalize):
    """Their logits are NaN and infinite, and have no part in anything."""
    import torch
    logits, gen = make(2000, 48, "float32", 5)
    live = torch.rand(2000, generator=gen, device="cuda") < 0.6
    logits[~live] = float("nan")
    logits[torch.nonzero(~live)[::3, 0]] = float("inf")
    _, g, _ = check(logits, 3, live=live, normalize=normalize)
    assert (g.experts[~live] == -1).all() and not g.weights[~live].any()
    _, g, _ = check(logits, 3, live=torch.zeros_like(live), normalize=normalize)
    assert not g.losses.any() and not g.counts.any()


@pytest.mark.parametrize("normalize", [True, False])
def test_masked_experts_are_never_chosen(normalize):
    """-infinity, the types' lowest value, fewer experts than choices, none at all."""
    import torch
    logits, _ = make(300, 24, "float32", 6)
    logits[:, ::3] = -torch.inf
    logits[5] = -torch.inf                      # no expert: as a token that is not live
    logits[6], logits[6, 7] = -torch.inf, 1.0   # one expert for four choices
    logits[8, 1:] = torch.finfo(torch.float32).min
    _, g, _ = check(logits, 4, normalize=normalize)
    assert (g.experts[5] == -1).all() and g.experts[6].tolist() == [7, -1, -1, -1]
    assert g.weights[6].tolist() == [1.0, 0.0, 0.0, 0.0]
    masked = torch.isin(g.experts, torch.arange(0, 24, 3, device="cuda", dtype=torch.int32))
    assert masked[8].any() and not masked[:8].any() and not masked[9:].any()      # row 8 has no -infinity there
    low = torch.full((4, 12), -65504.0, device="cuda", dtype=torch.float16)
    low[1, 5] = 3.0
    check(low, 2, normalize=normalize)


def test_a_fault_shows():
    import torch
    logits, _ = make(50, 16, "float32", 7)
    for bad in (float("nan"), float("inf")):
        x = logits.clone()
        x[9, 4] = bad
        router = sl.ExpertRouter(16, 2, 50)
        g = router.gate(x)
        assert torch.isnan(g.losses).all() and torch.isnan(g.weights[9]).all() and torch.isnan(g.stats[9, 1])
        others = torch.arange(50, device="cuda") != 9
        assert torch.isfinite(g.weights[others]).all()
        assert ((g.experts >= -1) & (g.experts < 16)).all()
        assert torch.isnan(router.gate_backward(x, g, torch.ones(50, 2, device="cuda"))[9]).all()
    x[9] = float("nan")
    g = router.gate(x)
    assert torch.isnan(g.losses).all() and (g.experts[9] == -1).all()
    # the handle's next call is as ever
    check(logits, 2, router=router)


def test_wide_and_narrow_logits():
    import torch
    logits, _ = make(500, 64, "float32", 8)
    check(logits * 30, 4)
    check(logits * 1e-4, 4)
    check(logits + 1000, 4, normalize=False)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("first", [0, 8, 3])
def test_views(dtype, first):
    import torch
    both, _ = make(700, 200, dtype, 9)
    logits = both[:, first:first + 64]
    router, g, _ = check(logits, 4)
    wide = torch.full((700, 96), 5.0, device="cuda", dtype=both.dtype)
    gw = torch.ones(700, 4, device="cuda") * torch.arange(4, device="cuda")
    got = router.gate_backward(logits, g, gw, grad_logits=wide[:, 16:80])
    assert torch.equal(got, router.gate_backward(logits.contiguous(), router.gate(logits.contiguous()), gw))
    assert (wide[:, :16] == 5).all() and (wide[:, 80:] == 5).all()


def test_missing_gradients_are_zero():
    import torch
    logits, _ = make(100, 32, "float32", 10)
    router = sl.ExpertRouter(32, 2, 100)
    g = router.gate(logits)
    gw, gl = torch.randn(100, 2, device="cuda"), torch.tensor([3.0, 2.0], device="cuda")
    assert not router.gate_backward(logits, g).any()
    a, b = router.gate_backward(logits, g, gw), router.gate_backward(logits, g, grad_losses=gl)
    both = router.gate_backward(logits, g, gw, gl)
    assert (a + b - both).abs().max() <= 16 * U * (a.abs() + b.abs() + 1).max()
    assert torch.equal(router.gate_backward(logits, g, gw, torch.zeros_like(gl)), a)


def test_the_routing_counts_the_same_choices():
    import torch
    logits, gen = make(5000, 40, "bfloat16", 11)
    live = torch.rand(5000, generator=gen, device="cuda") < 0.9
    router = sl.ExpertRouter(40, 3, 5000, align=8)
    g = router.gate(logits, live=live)
    r = router.route(g.experts)
    assert torch.equal(r.counts, g.counts)


def test_results_repeat_and_replay():
    import torch
    logits, _ = make(30000, 96, "float32", 12)
    router = sl.ExpertRouter(96, 4, 30000)
    gw, gl = torch.randn(30000, 4, device="cuda"), torch.tensor([3.0, 2.0], device="cuda")
    g = router.gate(logits)
    grad = router.gate_backward(logits, g, gw, gl)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        h = router.gate(logits)
        out = router.gate_backward(logits, h, gw, gl)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in ((h.losses, g.losses), (h.weights, g.weights), (h.counts, g.counts), (out, grad)):
            assert torch.equal(a, b)


def test_gradients_are_differences():
    """A step along a direction, in 64 bits with the choices and counts held: the terms of third order of a step of 1e-3
    are below 1e-5 of the gradient's magnitudes."""
    import torch
    logits, _ = make(30, 12, "float32", 13)
    K, T, E = 3, 30, 12
    gw, gl = torch.randn(T, K, device="cuda"), torch.tensor([2.0, 0.5], device="cuda")
    for normalize in (True, False):
        router = sl.ExpertRouter(E, K, T)
        g = router.gate(logits, normalize=normalize)
        grad = router.gate_backward(logits, g, gw, gl).double()
        f = g.counts.double() / (T * K)

        def value(x):
            p, lse = torch.softmax(x, 1), torch.logsumexp(x, 1)
            w = p.gather(1, g.experts.long())
            w = w / w.sum(1, keepdim=True) if normalize else w
            return (w * gw.double()).sum() + gl[0].double() * E * (f * p.mean(0)).sum() + gl[1].double() * (lse ** 2).mean()
        d = torch.randn(T, E, device="cuda").double()
        diff = (value(logits.double() + 1e-3 * d) - value(logits.double() - 1e-3 * d)) / 2e-3
        assert (diff - (grad * d).sum()).abs() <= 1e-4 * (grad * d).abs().sum()


def test_refusals():
    import torch
    logits, _ = make(20, 16, "float32", 1)
    router = sl.ExpertRouter(16, 2, 20)
    g = router.gate(logits)
    gw = torch.zeros(20, 2, device="cuda")
    for f in (lambda: router.gate(logits[:, :8]), lambda: router.gate(logits.cpu()), lambda: router.gate(logits[0]),
              lambda: router.gate(logits.double()), lambda: router.gate(logits, live=torch.ones(20, device="cuda")),
              lambda: router.gate(logits, live=torch.ones(19, dtype=torch.bool, device="cuda")),
              lambda: router.gate(logits.t().contiguous().t()),
              lambda: router.gate_backward(logits[:10], g, gw), lambda: router.gate_backward(logits, g, gw[:, :1]),
              lambda: router.gate_backward(logits, g, gw, torch.zeros(3, device="cuda")),
              lambda: router.gate_backward(logits, g, gw, grad_logits=logits.half()),
              lambda: sl.ExpertRouter(16, 3, 20).gate_backward(logits, g, gw)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: router.gate(logits.repeat(2, 1)),
              lambda: router.gate_backward(logits, g, gw, grad_logits=logits[:1].clone().expand(20, 16))):
        with pytest.raises(sl.EmbError):
            f()
