"""The gated recurrence against its formulas in 64 bits, with error bounds that
run along the recurrence, and its gradients against differences of the 64-bit
forward.

Bounds (u = 2^-24).  Each gate value carries a relative error of at most
(|gate| + 8) u (argument reduction of the exponential, its own 2 ulp, one
quotient), each step three roundings, so the error of h obeys
    e_t <= a_t e_{t-1} + (|gate_t| + 12) u (a_t |h_{t-1}| + (1 - a_t) |x_t|)
and the same recurrence, reversed, bounds what a position passes back.  The
scan may join stretches of a sequence in another order, which costs each
product of gates at most its own errors once more on either side: factor 3.
Stores of 16 bits add half a unit (2^-8 or 2^-11 of the value, and half the
smallest fp16), and the backward may read such a stored state."""
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


def sig(g):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))


def forward64(x, g, lens, h0):
    """(y, last, error bounds of both)."""
    B, T, D = x.shape
    a, na = sig(g)
    h, e = h0.copy(), np.zeros((B, D))
    y, ey = np.zeros_like(x), np.zeros_like(x)
    for t in range(T):
        on = (t < lens)[:, None]
        step = (np.abs(g[:, t]) + 12) * U * (a[:, t] * np.abs(h) + na[:, t] * np.abs(x[:, t]))
        e = np.where(on, a[:, t] * e + step, e)
        h = np.where(on, a[:, t] * h + na[:, t] * x[:, t], h)
        y[:, t] = np.where(on, h, 0)
        ey[:, t] = np.where(on, e, 0)
    return y, h, 3 * ey, 3 * e


def backward64(x, g, lens, h0, gy, gl, half):
    """Gradients of x, gate and the first state, and their error bounds."""
    B, T, D = x.shape
    a, na = sig(g)
    y, _, ey, _ = forward64(x, g, lens, h0)
    before = np.concatenate([h0[:, None], y[:, :-1]], 1)
    eb = np.concatenate([np.zeros((B, 1, D)), ey[:, :-1] + half * np.abs(y[:, :-1])], 1)
    c, e = gl.copy(), np.zeros((B, D))
    out = [np.zeros_like(x) for _ in range(4)]
    for t in range(T - 1, -1, -1):
        on = (t < lens)[:, None]
        k = (np.abs(g[:, t]) + 12) * U
        G = gy[:, t] + c
        eG = e + U * (np.abs(gy[:, t]) + np.abs(c))
        d = before[:, t] - x[:, t]
        ed = eb[:, t] + U * (np.abs(before[:, t]) + np.abs(x[:, t]))
        vals = (na[:, t] * G, na[:, t] * (3 * eG + k * np.abs(G)), a[:, t] * na[:, t] * d * G,
                a[:, t] * na[:, t] * (np.abs(d) * (3 * eG + 2 * k * np.abs(G)) + ed * (np.abs(G) + 3 * eG)))
        for o, v in zip(out, vals):
            o[:, t] = np.where(on, v, 0)
        e = np.where(on, a[:, t] * eG + k * a[:, t] * np.abs(G), e)
        c = np.where(on, a[:, t] * G, c)
    gx, ex, gg, eg = out
    return gx, gg, c, ex, eg, 3 * e


def close(got, ref, bound, dtype, what):
    got = f64(got)
    ok = np.abs(got - ref) <= bound + HALF[dtype] * (np.abs(ref) + bound) + TINY[dtype]
    assert ok.all(), "%s: %d of %d outside the bound, worst %g of it" % (
        what, (~ok).sum(), ok.size, np.max(np.abs(got - ref) / (bound + HALF[dtype] * np.abs(ref) + TINY[dtype])))


def make(B, T, D, dtype, seed, lens=None, spread=1.5):
    import torch
    gen = torch.Generator().manual_seed(seed)
    dt = getattr(torch, dtype)
    x = torch.randn(B, T, D, generator=gen).to(dt).cuda()
    g = (torch.randn(B, T, D, generator=gen) * spread + 1).to(dt).cuda()
    gy = torch.randn(B, T, D, generator=gen).to(dt).cuda()
    h0 = torch.randn(B, D, generator=gen).cuda()
    gl = torch.randn(B, D, generator=gen).cuda()
    if lens is None:
        lens = torch.randint(0, T + 1, (B,), generator=gen).numpy()
    lens = np.asarray(lens)
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()
    return x, g, gy, h0, gl, np.minimum(lens, T), off


def check(B, T, D, dtype, seed, lens=None, x=None, g=None, spread=1.5):
    x0, g0, gy, h0, gl, lens, off = make(B, T, D, dtype, seed, lens, spread)
    x, g = x0 if x is None else x, g0 if g is None else g
    plan = sl.GatedScan(D, max_batch=B, max_len=T)
    y, last = plan.forward(x, g, off, h0)
    gx, gg, gs = plan.backward(x, g, y, gy, off, h0, gl)
    again = plan.forward(x, g, off, h0) + plan.backward(x, g, y, gy, off, h0, gl)
    assert plan.device_status() == 0
    for p, q in zip((y, last, gx, gg, gs), again):
        assert (p == q).all(), "a second call gives other bits"
    ry, rl, ey, el = forward64(f64(x), f64(g), lens, f64(h0))
    close(y, ry, ey, dtype, "y")
    close(last, rl, el, "float32", "last")
    half = HALF[dtype] if dtype != "float32" else 0.0
    rx, rg, rs, ex, eg, es = backward64(f64(x), f64(g), lens, f64(h0), f64(gy), f64(gl), half)
    close(gx, rx, ex, dtype, "grad_x")
    close(gg, rg, eg, dtype, "grad_gate")
    close(gs, rs, es, "float32", "grad_state")
    plan.close()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (3, 1, 8), (2, 2, 3), (5, 37, 50), (2, 333, 64), (7, 130, 24),
                                   (1, 1025, 256), (130, 9, 16), (1, 2500, 36), (3, 515, 513)])
def test_matches_the_formulas(B, T, D, dtype):
    check(B, T, D, dtype, B * 1000 + T + D)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("B,T,D", [(1, 20000, 64), (2, 9001, 20), (600, 70, 128), (4000, 11, 32)])
def test_long_and_wide(B, T, D, dtype):
    check(B, T, D, dtype, T)


def test_lengths_zero_one_full_and_past_the_end():
    check(8, 45, 40, "float32", 3, lens=[0, 1, 45, 44, 100, 2, 0, 33])
    check(8, 300, 16, "bfloat16", 4, lens=[0, 1, 300, 299, 1000, 2, 256, 257])
    check(4, 64, 8, "float16", 5, lens=[0, 0, 0, 0])


def test_slow_gates_carry_far():
    """Gates near 1: a state reaches thousands of positions on."""
    import torch
    x, g, *_ = make(1, 6000, 32, "float32", 9)
    check(1, 6000, 32, "float32", 9, lens=[6000], g=(g - 1) * 0.2 + 8)
    check(2, 700, 32, "float32", 10, lens=[700, 650], spread=30.0)   # saturated both ways


def test_strides_and_unaligned_views():
    """x and gate as the halves of one projection, time-major arrays, rows that
    start off any 16-byte boundary."""
    import torch
    B, T, D = 3, 150, 32
    for dtype in ("float32", "bfloat16"):
        x0, g0, *_ = make(B, T, D, dtype, 21)
        both = torch.cat([x0, g0], 2)
        check(B, T, D, dtype, 21, x=both[..., :D], g=both[..., D:])
        check(B, T, D, dtype, 21, x=x0.transpose(0, 1).contiguous().transpose(0, 1))
        odd = torch.empty(B * T * D + 1, dtype=x0.dtype, device="cuda")[1:].view(B, T, D)
        odd.copy_(x0)
        check(B, T, D, dtype, 21, x=odd)
        one = x0[:1].expand(B, T, D)
        check(B, T, D, dtype, 21, x=one)


def test_outputs_into_views():
    import torch
    B, T, D = 2, 70, 24
    x, g, gy, h0, gl, lens, off = make(B, T, D, "float32", 5)
    plan = sl.GatedScan(D, B, T)
    y, last = plan.forward(x, g, off, h0)
    gx, gg, gs = plan.backward(x, g, y, gy, off, h0, gl)
    wide = torch.full((B, T, 2 * D + 1), 7.0, device="cuda")
    plan.backward(x, g, y, gy, off, h0, gl, grad_x=wide[..., :D], grad_gate=wide[..., D:2 * D])
    assert (wide[..., :D] == gx).all() and (wide[..., D:2 * D] == gg).all() and (wide[..., 2 * D:] == 7).all()
    tm = torch.full((T, B, D), 7.0, device="cuda")
    plan.forward(x, g, off, h0, y=tm.transpose(0, 1))
    assert (tm.transpose(0, 1) == y).all()


def test_nothing_past_the_end_is_read():
    """NaN and infinities in dead positions of x, gate and grad_y change
    nothing."""
    import torch
    B, T, D = 6, 200, 32
    for dtype in ("float32", "float16"):
        x, g, gy, h0, gl, lens, off = make(B, T, D, dtype, 8, lens=[0, 1, 199, 100, 64, 128])
        plan = sl.GatedScan(D, B, T)
        want = plan.forward(x, g, off, h0)
        want += plan.backward(x, g, want[0], gy, off, h0, gl)
        dead = torch.arange(T, device="cuda")[None, :] >= torch.from_numpy(lens).cuda()[:, None]
        for bad in (float("nan"), float("inf"), float("-inf")):
            for t in (x, g, gy):
                t[dead] = bad
            got = plan.forward(x, g, off, h0)
            got += plan.backward(x, g, got[0], gy, off, h0, gl)
            for p, q in zip(got, want):
                assert torch.equal(p, q)


def test_infinite_gates_keep_or_replace_the_state():
    import torch
    x = torch.tensor([[[1.0], [2.0], [3.0], [4.0]]], device="cuda")
    g = torch.tensor([[[float("-inf")], [float("inf")], [float("inf")], [float("-inf")]]], device="cuda")
    plan = sl.GatedScan(1, 1, 4)
    y, last = plan.forward(x, g)
    assert y.flatten().tolist() == [1.0, 1.0, 1.0, 4.0] and last.item() == 4.0


def test_a_nan_stays_in_its_channel_and_sequence():
    import torch
    x, g, gy, h0, gl, lens, off = make(3, 100, 16, "float32", 2, lens=[100, 100, 100])
    plan = sl.GatedScan(16, 3, 100)
    clean, _ = plan.forward(x, g, off, h0)
    x[1, 40, 5] = float("nan")
    y, _ = plan.forward(x, g, off, h0)
    assert torch.isnan(y[1, 40:, 5]).all()
    mask = torch.ones_like(y, dtype=torch.bool)
    mask[1, 40:, 5] = False
    assert torch.equal(y[mask], clean[mask])


def test_no_offsets_no_states():
    import torch
    x, g, gy, *_ = make(2, 80, 12, "float32", 6)
    plan = sl.GatedScan(12, 4, 100)
    y, last = plan.forward(x, g)
    lens, z = np.array([80, 80]), np.zeros((2, 12))
    ry, rl, ey, el = forward64(f64(x), f64(g), lens, z)
    close(y, ry, ey, "float32", "y")
    close(last, rl, el, "float32", "last")
    gx, gg, gs = plan.backward(x, g, y, gy)
    rx, rg, rs, ex, eg, es = backward64(f64(x), f64(g), lens, z, f64(gy), z, 0.0)
    close(gx, rx, ex, "float32", "grad_x")
    close(gg, rg, eg, "float32", "grad_gate")
    close(gs, rs, es, "float32", "grad_state")


def test_gradients_against_differences():
    """Directional derivatives of sum(y w) + sum(last v), from the kernel's
    gradients and from central differences of the 64-bit forward.  Step 1e-4:
    truncation below 1e-6 of the sum of magnitudes (third derivatives of order
    1), rounding 1e-12; the kernel's fp32 gradients below 1e-5 of it."""
    import torch
    B, T, D = 3, 60, 10
    x, g, gy, h0, gl, lens, off = make(B, T, D, "float32", 77)
    plan = sl.GatedScan(D, B, T)
    y, last = plan.forward(x, g, off, h0)
    grads = [f64(t) for t in plan.backward(x, g, y, gy, off, h0, gl)]
    ins = [f64(x), f64(g), f64(h0)]
    rng = np.random.default_rng(1)

    def loss(xx, gg, hh):
        yy, ll, _, _ = forward64(xx, gg, lens, hh)
        live = np.arange(T)[None, :, None] < lens[:, None, None]
        return (yy * f64(gy) * live).sum() + (ll * f64(gl)).sum()
    for which in range(3):
        for _ in range(4):
            d = rng.standard_normal(ins[which].shape)
            hi, lo = list(ins), list(ins)
            hi[which], lo[which] = ins[which] + 1e-4 * d, ins[which] - 1e-4 * d
            num = (loss(*hi) - loss(*lo)) / 2e-4
            assert abs((grads[which] * d).sum() - num) <= 1.1e-5 * np.abs(grads[which] * d).sum()


def test_pieces_of_a_sequence_join():
    """A sequence cut in two, the state handed on: the second piece continues
    the first."""
    x, g, gy, h0, *_ = make(2, 300, 48, "float32", 12)
    plan = sl.GatedScan(48, 2, 300)
    y, last = plan.forward(x, g, state=h0)
    y1, mid = plan.forward(x[:, :101], g[:, :101], state=h0)
    y2, end = plan.forward(x[:, 101:], g[:, 101:], state=mid)
    _, _, ey, el = forward64(f64(x), f64(g), np.array([300, 300]), f64(h0))
    assert np.all(np.abs(f64(y1) - f64(y)[:, :101]) <= 2 * ey[:, :101])
    assert np.all(np.abs(f64(y2) - f64(y)[:, 101:]) <= 2 * ey[:, 101:])
    assert np.all(np.abs(f64(end) - f64(last)) <= 2 * el)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("n,D", [(1, 1), (7, 33), (64, 256), (300, 50), (1, 1030), (5000, 64)])
def test_step(n, D, dtype):
    import torch
    gen = torch.Generator().manual_seed(n + D)
    dt = getattr(torch, dtype)
    R = n + 37
    x = torch.randn(n, D, generator=gen).to(dt).cuda()
    both = (torch.randn(n, 2 * D, generator=gen) * 2).to(dt).cuda()
    g = both[:, D:]
    states = torch.randn(R, D, generator=gen).cuda()
    rows = torch.randperm(R, generator=gen)[:n].cuda()
    if n > 4:
        rows[2], rows[3] = -1, R
    s0, xs, gs, r = f64(states), f64(x), f64(g), rows.cpu().numpy()
    live = (r >= 0) & (r < R)
    plan = sl.GatedScan(D, 1, 1)
    y = plan.step(x, g, rows, states)
    old = np.where(live[:, None], s0[np.where(live, r, 0)], 0)
    a, na = sig(gs)
    h = a * old + na * xs
    bound = (np.abs(gs) + 12) * U * (a * np.abs(old) + na * np.abs(xs))
    h, bound = np.where(live[:, None], h, 0), np.where(live[:, None], bound, 0)
    close(y, h, bound, dtype, "y")
    s0[r[live]] = h[live]
    tol = np.zeros_like(s0)
    tol[r[live]] = bound[live]
    got = f64(states)
    assert np.all(np.abs(got - s0) <= tol + U * np.abs(s0) * (tol > 0))


def test_steps_follow_the_sequence():
    """One position at a time gives what the whole sequence gives."""
    import torch
    x, g, _, h0, *_ = make(9, 25, 64, "float32", 31)
    plan = sl.GatedScan(64, 9, 25)
    y, last = plan.forward(x, g, state=h0)
    states = torch.zeros(20, 64, device="cuda")
    rows = torch.arange(9, device="cuda") * 2
    states[rows] = h0
    _, _, ey, el = forward64(f64(x), f64(g), np.full(9, 25), f64(h0))
    for t in range(25):
        yt = plan.step(x[:, t], g[:, t], rows, states)
        assert np.all(np.abs(f64(yt) - f64(y)[:, t]) <= 2 * ey[:, t])
    assert np.all(np.abs(f64(states)[::2][:9] - f64(last)) <= 2 * el)


def test_graph_replay_and_another_stream():
    import torch
    x, g, gy, h0, gl, lens, off = make(2, 3000, 64, "bfloat16", 14)
    plan = sl.GatedScan(64, 2, 3000)
    y, last = plan.forward(x, g, off, h0)
    want = (y, last) + plan.backward(x, g, y, gy, off, h0, gl)
    out = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        plan.forward(x, g, off, h0, y=out[0], last=out[1])
        plan.backward(x, g, out[0], gy, off, h0, gl, grad_x=out[2], grad_gate=out[3], grad_state=out[4])
    for _ in range(3):
        for t in out:
            t.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, want):
            assert torch.equal(p, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, last2 = plan.forward(x, g, off, h0, stream=side)
    side.synchronize()
    assert torch.equal(y2, want[0]) and torch.equal(last2, want[1])
    assert plan.device_status() == 0


def test_decreasing_offsets_are_reported():
    import torch
    x, g, gy, h0, *_ = make(3, 20, 8, "float32", 1)
    off = torch.tensor([0, 20, 5, 25], dtype=torch.int32, device="cuda")
    plan = sl.GatedScan(8, 3, 20)
    y, last = plan.forward(x, g, off, h0)
    assert plan.device_status() == 7 and plan.device_status() == 0
    assert (y[1] == 0).all() and torch.equal(last[1], h0[1])


def test_empty_calls():
    import torch
    plan = sl.GatedScan(8, 3, 20)
    e = torch.empty(0, 20, 8, device="cuda")
    y, last = plan.forward(e, e)
    assert y.shape == (0, 20, 8) and last.shape == (0, 8)
    z, h0 = torch.empty(3, 0, 8, device="cuda"), torch.randn(3, 8, device="cuda")
    y, last = plan.forward(z, z, state=h0)
    assert torch.equal(last, h0)
    gx, gg, gs = plan.backward(z, z, y, z, state=h0, grad_last=h0)
    assert torch.equal(gs, h0)
    plan.step(e[:, 0], e[:, 0], torch.empty(0, dtype=torch.int64, device="cuda"), torch.zeros(1, 8, device="cuda"))


def test_refusals():
    import torch
    plan = sl.GatedScan(8, 2, 16)
    x = torch.zeros(2, 16, 8, device="cuda")
    for bad in (x.double(), x[..., :7], x.cpu(), torch.zeros(2, 16, 16, device="cuda")[..., ::2]):
        with pytest.raises(ValueError):
            plan.forward(x, bad)
    with pytest.raises(ValueError):
        plan.forward(x, x, offsets=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        plan.forward(x, x, state=torch.zeros(2, 7, device="cuda"))
    for B, T in ((3, 16), (2, 17)):          # more than the plan was made for
        z = torch.zeros(B, T, 8, device="cuda")
        with pytest.raises(sl.EmbError) as e:
            plan.forward(z, z)
        assert e.value.status == 1
    with pytest.raises(sl.EmbError):         # an output with two elements at one place
        plan.forward(x, x, y=torch.zeros(1, 16, 8, device="cuda").expand(2, 16, 8))
    with pytest.raises(ValueError):
        plan.step(x[0], x[0], torch.zeros(16, dtype=torch.int32, device="cuda"), torch.zeros(4, 8, device="cuda"))


def test_allocation_failure():
    gc.collect()   # handles of earlier tests are freed now, not in the middle of the count
    base = sl.emb_debug_live_allocations()
    for k in range(20):
        sl.emb_debug_fail_alloc(k)
        try:
            plan = sl.GatedScan(64, 4, 4096)
        except sl.EmbError as e:
            assert e.status == 3 and sl.emb_debug_live_allocations() == base
            continue
        sl.emb_debug_fail_alloc(-1)
        plan.close()
        break
    assert k >= 1 and sl.emb_debug_live_allocations() == base


def test_wait_that_runs_out_is_reported():
    r = sl.scan_selftest_timeout()
    assert r["status"] == 0 and r["latched"] == 8 and r["latched_after"] == 0, r
    assert 0.0 < r["wait_ms"] < 60000.0, r


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("D", [32, 30, 33])
def test_every_short_length(D, dtype):
    """Lengths around every change of kernel, widths of each access."""
    for T in (1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 24, 25, 32, 33):
        check(7, T, D, dtype, T)


def test_even_and_odd_widths_in_long_sequences():
    check(1, 9000, 34, "float32", 1)
    check(2, 5000, 18, "float16", 2)
    check(1, 7001, 35, "bfloat16", 3)
    check(700, 130, 30, "bfloat16", 4)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("B,T,D", [(1, 30000, 16), (1, 20000, 30), (1, 20000, 15), (1, 12000, 96), (2, 9000, 256),
                                   (41, 600, 256)])
def test_chains_of_few_and_of_many_tiles_across(B, T, D, dtype):
    check(B, T, D, dtype, B + T + D)


def test_one_handle_for_chains_of_other_shapes():
    """The records of one call lie where another call's groups begin."""
    import torch
    plan = sl.GatedScan(32, max_batch=12, max_len=12000)
    for B, T in [(12, 12000), (1, 12000), (4, 5000), (1, 700), (12, 12000), (2, 11999)]:
        x, g, gy, h0, gl, lens, off = make(B, T, 32, "float32", B + T)
        y, last = plan.forward(x, g, off, h0)
        got = (y, last) + plan.backward(x, g, y, gy, off, h0, gl)
        other = sl.GatedScan(32, max_batch=B, max_len=T)
        y, last = other.forward(x, g, off, h0)
        want = (y, last) + other.backward(x, g, y, gy, off, h0, gl)
        for p, q in zip(got, want):
            assert torch.equal(p, q)
        other.close()
    assert plan.device_status() == 0
    plan.close()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("T,D", [(2, 24), (4, 32), (7, 24), (8, 30), (11, 24), (13, 30), (16, 33), (17, 24)])
def test_short_sequences_in_views_and_with_dead_positions(T, D, dtype):
    """Sequences held whole: the same bits from halves of one projection,
    time-major arrays, rows off the access boundaries and broadcast entries,
    whatever the dead positions hold."""
    import torch
    B = 19
    x, g, gy, h0, gl, lens, off = make(B, T, D, dtype, T * D)
    plan = sl.GatedScan(D, B, T)

    def run(x, g, gy):
        y, last = plan.forward(x, g, off, h0)
        return (y, last) + plan.backward(x, g, y, gy, off, h0, gl)

    def off_boundary(t):
        u = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        return u.copy_(t)

    want = run(x, g, gy)
    both = torch.cat([x, g], 2)
    for views in ((both[..., :D], both[..., D:], gy), (off_boundary(x), off_boundary(g), off_boundary(gy)),
                  tuple(t.transpose(0, 1).contiguous().transpose(0, 1) for t in (x, g, gy))):
        for p, q in zip(run(*views), want):
            assert torch.equal(p, q)
    dead = (torch.arange(T)[None, :] >= torch.from_numpy(lens)[:, None]).cuda()[..., None]
    for fill in (float("nan"), float("inf"), torch.finfo(x.dtype).min):
        for p, q in zip(run(*(torch.where(dead, fill, t) for t in (x, g, gy))), want):
            assert torch.equal(p, q)
    one = run(x[:1].expand(B, T, D), g, gy)
    for p, q in zip(one, run(x[:1].repeat(B, 1, 1), g, gy)):
        assert torch.equal(p, q)
    assert plan.device_status() == 0
    plan.close()
    check(B, T, D, dtype, T * D)
