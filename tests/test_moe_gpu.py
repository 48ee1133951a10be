"""Tokens sorted by expert and back, against loops over the choices in 64 bits.
Index results are exact.  Sums of n fp32 terms in any order are within
n u sum|terms| (u = 2^-24, n counting the products' own roundings); stores of
16 bits add half a unit."""
import gc

import numpy as np
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


def f64(t):
    return t.detach().double().cpu().numpy()


def order(experts, E, align, rows):
    flat = experts.reshape(-1)
    offsets, counts = np.zeros(E + 1, np.int64), np.zeros(E, np.int64)
    pos, src = np.full(flat.size, -1, np.int64), np.full(rows, -1, np.int64)
    for e in range(E):
        mine = np.flatnonzero(flat == e)
        counts[e] = mine.size
        pos[mine] = offsets[e] + np.arange(mine.size)
        src[pos[mine]] = mine
        offsets[e + 1] = offsets[e] + -(-mine.size // align) * align
    return offsets, counts, pos.reshape(experts.shape), src


def choices(T, K, E, seed, drop=0.0, skew=False):
    rng = np.random.default_rng(seed)
    if skew:
        e = np.minimum(rng.geometric(0.3, (T, K)) - 1, E - 1)
    else:
        e = rng.integers(0, E, (T, K))
    if drop:
        bad = rng.random((T, K)) < drop
        e = np.where(bad, rng.choice([-1, E, -7, 2 ** 31 - 1, -2 ** 31], (T, K)), e)
    return e.astype(np.int32)


def check_route(experts, E, align):
    import torch
    T, K = experts.shape
    plan = sl.ExpertRouter(E, K, max(T, 1), align)
    r = plan.route(torch.from_numpy(experts).cuda())
    offsets, counts, pos, src = order(experts, E, align, plan.rows(T))
    assert np.array_equal(r.counts.cpu().numpy(), counts)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.pos.cpu().numpy(), pos)
    assert np.array_equal(r.src.cpu().numpy(), src)
    return plan, r, pos, src


@pytest.mark.parametrize("T,K,E,align,drop", [
    (1, 1, 1, 1, 0), (1, 8, 16, 1, 0), (3, 2, 5, 4, 0.5), (100, 2, 8, 1, 0), (1000, 3, 37, 8, 0.1),
    (4096, 1, 64, 1, 0), (4097, 1, 64, 128, 0.02), (5003, 6, 300, 16, 0.05), (70001, 4, 128, 1, 0),
    (200000, 8, 256, 64, 0.01), (3000, 2, 2048, 1, 0), (20000, 2, 2047, 3, 0.3), (600, 64, 70, 1, 0)])
def test_route(T, K, E, align, drop):
    check_route(choices(T, K, E, T + E, drop), E, align)


def test_route_one_expert_takes_all_and_none_live():
    check_route(np.zeros((30000, 2), np.int32), 16, 8)
    check_route(np.full((30000, 2), 15, np.int32), 16, 1)
    check_route(np.full((5000, 2), -1, np.int32), 16, 8)
    check_route(choices(50000, 2, 64, 5, skew=True), 64, 32)


def close(got, ref, bound, dtype, what):
    got = f64(got)
    ok = np.abs(got - ref) <= bound + HALF[dtype] * (np.abs(ref) + bound) + TINY[dtype]
    assert ok.all(), "%s: %d of %d outside the bound" % (what, (~ok).sum(), ok.size)


def check_rows(T, K, E, D, align, drop, dtype, seed=0, x=None, weighted=True):
    import torch
    experts = choices(T, K, E, seed + T, drop)
    plan, r, pos, src = check_route(experts, E, align)
    R = plan.rows(T)
    gen = torch.Generator().manual_seed(seed)
    dt = getattr(torch, dtype)
    if x is None:
        x = torch.randn(T, D, generator=gen).to(dt).cuda()
    ys = torch.randn(R, D, generator=gen).to(dt).cuda()
    ys[r.src < 0] = float("nan")          # padding is never read
    w = torch.rand(T, K, generator=gen).cuda() if weighted else None
    gy = torch.randn(T, D, generator=gen).to(dt).cuda()
    xs = plan.dispatch(x, r)
    want = np.zeros((R, D))
    want[src >= 0] = f64(x)[src[src >= 0] // K]
    assert np.array_equal(f64(xs), want)
    y = plan.combine(ys, w, r)
    gys, gw = plan.combine_backward(gy, ys, w, r)
    Y, W, G = f64(ys), f64(w) if weighted else np.ones((T, K)), f64(gy)
    ry, by = np.zeros((T, D)), np.zeros((T, D))
    rw, bw = np.zeros((T, K)), np.zeros((T, K))
    rg = np.zeros((R, D))
    for k in range(K):
        t = np.flatnonzero(pos[:, k] >= 0)
        p = pos[t, k]
        ry[t] += W[t, k, None] * Y[p]
        by[t] += np.abs(W[t, k, None] * Y[p])
        rw[t, k] = (G[t] * Y[p]).sum(1)
        bw[t, k] = np.abs(G[t] * Y[p]).sum(1)
        rg[p] = W[t, k, None] * G[t]
    close(y, ry, (K + 1) * U * by, dtype, "y")
    close(gys, rg, U * np.abs(rg), dtype, "grad_ys")
    if weighted:
        close(gw, rw, (D + 1) * U * bw, "float32", "grad_weights")
    else:
        assert gw is None
    gx = plan.dispatch_backward(gys, r)
    rx, bx = np.zeros((T, D)), np.zeros((T, D))
    GY = f64(gys)
    for k in range(K):
        t = np.flatnonzero(pos[:, k] >= 0)
        rx[t] += GY[pos[t, k]]
        bx[t] += np.abs(GY[pos[t, k]])
    close(gx, rx, (K + 1) * U * bx, dtype, "grad_x")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("T,K,E,D,align,drop", [
    (1, 1, 1, 1, 1, 0), (1, 2, 4, 256, 1, 0), (9, 3, 5, 7, 4, 0.4), (333, 2, 16, 99, 8, 0.1), (200, 8, 64, 64, 1, 0),
    (500, 4, 32, 1030, 1, 0.05), (2000, 2, 8, 18, 1, 0), (4, 2, 3, 4097, 2, 0), (1500, 6, 12, 512, 128, 0),
    (37, 64, 100, 40, 1, 0.1), (3000, 1, 9, 36, 16, 0.2)])
def test_rows(T, K, E, D, align, drop, dtype):
    check_rows(T, K, E, D, align, drop, dtype)


def test_rows_without_weights():
    check_rows(700, 4, 16, 128, 1, 0.1, "bfloat16", weighted=False)


def test_strided_and_unaligned_rows():
    import torch
    for dtype in ("float32", "bfloat16"):
        dt = getattr(torch, dtype)
        base = torch.randn(300, 130).to(dt).cuda()
        check_rows(300, 2, 8, 64, 4, 0.1, dtype, x=base[:, :64])
        check_rows(300, 2, 8, 64, 4, 0.1, dtype, x=base[:, 3:67])
        check_rows(300, 2, 8, 64, 4, 0.1, dtype, x=base[:1, :64].expand(300, 64))
    plan = sl.ExpertRouter(8, 2, 300)
    r = plan.route(torch.from_numpy(choices(300, 2, 8, 1)).cuda())
    ys = torch.randn(600, 64, device="cuda")
    wide = torch.full((300, 67), 5.0, device="cuda")
    y = plan.combine(ys, None, r)
    plan.combine(ys, None, r, y=wide[:, 1:65])
    assert torch.equal(wide[:, 1:65], y) and (wide[:, 0] == 5).all() and (wide[:, 65:] == 5).all()


def test_gradients_against_differences():
    """Directional derivatives of sum(y g) in ys, weights and x (through the
    identity as expert) against central differences of the 64-bit sums, which
    are linear in each: exact up to 64-bit rounding; the fp32 results are
    within 1e-5 of the sum of magnitudes."""
    import torch
    T, K, E, D = 120, 3, 11, 20
    experts = choices(T, K, E, 9, 0.1)
    plan, r, pos, src = check_route(experts, E, 4)
    R = plan.rows(T)
    gen = torch.Generator().manual_seed(4)
    ys, w, gy = torch.randn(R, D, generator=gen).cuda(), torch.rand(T, K, generator=gen).cuda(), \
        torch.randn(T, D, generator=gen).cuda()
    gys, gw = plan.combine_backward(gy, ys, w, r)
    gx = plan.dispatch_backward(gys, r)
    rng = np.random.default_rng(0)

    def loss(yy, ww, xx):
        out = 0.0
        for t in range(T):
            for k in range(K):
                if pos[t, k] >= 0:
                    row = yy[pos[t, k]] if xx is None else xx[t]
                    out += (ww[t, k] * row * f64(gy)[t]).sum()
        return out
    Y, W, X = f64(ys), f64(w), rng.standard_normal((T, D))
    for grad, base, f in ((gys, Y, lambda v: loss(v, W, None)), (gw, W, lambda v: loss(Y, v, None)),
                          (gx, X, lambda v: loss(None, W, v))):
        d = rng.standard_normal(base.shape)
        num = (f(base + 1e-2 * d) - f(base - 1e-2 * d)) / 2e-2
        assert abs((f64(grad) * d).sum() - num) <= 1e-5 * np.abs(f64(grad) * d).sum()


def test_large_values_do_not_overflow_between():
    """fp16 rows whose weighted sum fits although a plain sum would not."""
    import torch
    plan = sl.ExpertRouter(2, 2, 4)
    r = plan.route(torch.tensor([[0, 1]] * 4, dtype=torch.int32, device="cuda"))
    ys = torch.full((8, 16), 60000.0, dtype=torch.float16, device="cuda")
    y = plan.combine(ys, torch.full((4, 2), 0.5, device="cuda"), r)
    assert (y == 60000).all()


def test_fewer_tokens_than_the_plan_and_none():
    import torch
    plan = sl.ExpertRouter(5, 2, 1000, align=4)
    r = plan.route(torch.zeros(0, 2, dtype=torch.int32, device="cuda"))
    assert (r.counts == 0).all() and (r.offsets == 0).all() and (r.src == -1).all()
    xs = plan.dispatch(torch.zeros(0, 8, device="cuda"), r)
    assert xs.shape == (16, 8) and (xs == 0).all()
    assert plan.combine(xs, None, r).shape == (0, 8)
    gys, gw = plan.combine_backward(torch.zeros(0, 8, device="cuda"), xs, torch.zeros(0, 2, device="cuda"), r)
    assert (gys == 0).all() and gw.shape == (0, 2)


def test_graph_replay_and_another_stream():
    import torch
    plan = sl.ExpertRouter(32, 4, 20000, align=16)
    ids = torch.from_numpy(choices(20000, 4, 32, 3, 0.05)).cuda()
    x, w = torch.randn(20000, 72, device="cuda"), torch.rand(20000, 4, device="cuda")

    def step(stream=None):
        r = plan.route(ids, stream)
        xs = plan.dispatch(x, r, stream=stream)
        y = plan.combine(xs, w, r, stream=stream)
        return (*r, xs, y) + plan.combine_backward(x, xs, w, r, stream=stream)
    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        got = step()
    for _ in range(3):
        for t in got:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(got, want):
            assert torch.equal(p, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    for p, q in zip(got, want):
        assert torch.equal(p, q)


def test_refusals():
    import torch
    plan = sl.ExpertRouter(4, 2, 10)
    ids = torch.zeros(10, 2, dtype=torch.int32, device="cuda")
    for bad in (ids.long(), ids[:, :1], ids.cpu(), ids.t()):
        with pytest.raises(ValueError):
            plan.route(bad)
    with pytest.raises(sl.EmbError) as e:
        plan.route(torch.zeros(11, 2, dtype=torch.int32, device="cuda"))
    assert e.value.status == 1
    r = plan.route(ids)
    with pytest.raises(ValueError):
        plan.dispatch(torch.zeros(9, 4, device="cuda"), r)
    with pytest.raises(ValueError):
        plan.combine(torch.zeros(19, 4, device="cuda"), None, r)
    with pytest.raises(ValueError):
        plan.combine(torch.zeros(20, 4, device="cuda"), torch.zeros(10, 2, device="cuda").half(), r)
    with pytest.raises(ValueError):
        plan.combine_backward(torch.zeros(10, 4, device="cuda"), torch.zeros(20, 4, device="cuda").half(), None, r)
    for args in ((0, 1, 1, 1), (4, 0, 1, 1), (4, 1, 0, 1), (4, 1, 1, 0)):
        with pytest.raises(sl.EmbError) as e:
            sl.ExpertRouter(*args)
        assert e.value.status == 1
    for args in ((2049, 1, 1, 1), (4, 65, 1, 1), (4, 8, 1 << 30, 1)):
        with pytest.raises(sl.EmbError) as e:
            sl.ExpertRouter(*args)
        assert e.value.status == 2


def test_allocation_failure():
    gc.collect()   # handles of earlier tests are freed now, not in the middle of the count
    base = sl.emb_debug_live_allocations()
    sl.emb_debug_fail_alloc(0)
    with pytest.raises(sl.EmbError) as e:
        sl.ExpertRouter(4, 2, 10)
    sl.emb_debug_fail_alloc(-1)
    assert e.value.status == 3 and sl.emb_debug_live_allocations() == base
