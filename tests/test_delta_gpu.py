"""The gated delta rule and its gradients against the recurrence and its adjoint,
position by position in 64 bits.

Tolerances.  A result is a sum of parts that are rounded on their own, so its error
is measured against the root of its parts' sum of squares (`sizes` below: with them a
state is the sum of what each position wrote to it, e the difference of v and of what
the state says), which is near the result itself unless the parts cancel:
    norm(got - want) <= tol * norm(size) + half a rounding of a 16-bit result.
Operands carry 24 bits in three terms; a result passes a chain of up to 48 additions
that the matrix units may cut instead of rounding (2^-23 each), and through two or
three such products: 1e-5 in the forward.  The backward's products are up to five in
a chain, operands of fp16 and fp32 with more than 64 key channels carry 16 bits (off by
2^-17 at most, by a third of it as a root of squares): 2e-5.  The states of a bf16 call's
grad_q and grad_k are rounded to bf16: 2^-9 more."""
import pytest

import sparse_lookup_gb300 as sl
from sparse_lookup_gb300 import build as slbuild

pytestmark = pytest.mark.gpu

HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
NAMES = ("grad_q", "grad_k", "grad_v", "grad_decay", "grad_beta", "grad_state")


@pytest.fixture(scope="module", autouse=True)
def built():
    slbuild.build()
    sl.lib()


def make(B, T, H, J, N, V, dtype, seed, slow=False):
    """q, k, v, decay, beta, state, grad_y, grad_last"""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = getattr(torch, dtype)

    def r(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    def unit(x):
        return x / x.norm(dim=-1, keepdim=True).clamp(min=1e-6)
    k = unit(r(B, T, J, N))
    again = torch.rand(B, T, 1, 1, generator=gen, device="cuda") < 0.2
    k = torch.where(again, k.roll(1, 1), k)
    decay = -torch.exp(r(B, T, H) * 1.2 - (6.0 if slow else 2.5))
    return (unit(r(B, T, J, N)).to(dt), k.to(dt), r(B, T, H, V).to(dt), decay, torch.sigmoid(r(B, T, H)),
            r(B, H, N, V) * 0.3, r(B, T, H, V).to(dt), r(B, H, N, V) * 0.1)


def reference(q, k, v, decay, beta, state, gy, gl, scale, lens=None):
    """[y, last, *gradients (NAMES)] in 64 bits, and the sizes of each."""
    import torch
    B, T, H, V = v.shape
    J, N = q.shape[2:]
    live = torch.ones(B, T, dtype=torch.bool, device="cuda") if lens is None else (
        torch.arange(T, device="cuda")[None] < lens[:, None])
    on4, on3 = live[:, :, None, None], live[:, :, None]
    q, k, v, gy = (torch.where(on4, x, 0.0).double() for x in (q, k, v, gy))
    decay, beta = (torch.where(on3, x, 0.0).double() for x in (decay, beta))
    q, k = q.repeat_interleave(H // J, 2), k.repeat_interleave(H // J, 2)
    a = torch.exp(decay)[..., None, None]
    b = beta[..., None]
    nothing = torch.zeros(B, H, N, V, dtype=torch.float64, device="cuda")
    S = nothing if state is None else state.double()
    R = S.square()
    y, ys = torch.zeros_like(v), torch.zeros_like(v)
    steps = []

    def col(x, t):
        return x[:, t, :, :, None]

    def row(x, t):
        return x[:, t, :, None, :]
    for t in range(T):
        S1, R1 = S * a[:, t], R * a[:, t] ** 2
        e = v[:, t] - (S1 * col(k, t)).sum(2)
        es = v[:, t].square() + (R1 * col(k, t) ** 2).sum(2)
        steps.append((S1, R1, e, es))
        S = S1 + col(k, t) * (b[:, t] * e)[:, :, None]
        R = R1 + col(k, t) ** 2 * (b[:, t] ** 2 * es)[:, :, None]
        steps[-1] += (S, R)
        y[:, t] = scale * (S * col(q, t)).sum(2)
        ys[:, t] = scale ** 2 * (R * col(q, t) ** 2).sum(2)
    last, lasts = S, R
    dS = nothing if gl is None else gl.double()
    D = dS.square()
    g = [torch.zeros_like(x) for x in (q, k, v, decay, beta)]
    s = [torch.zeros_like(x) for x in (q, k, v, decay, beta)]
    for t in range(T - 1, -1, -1):
        S1, R1, e, es, S, R = steps[t]
        dS = dS + scale * col(q, t) * row(gy, t)
        D = D + (scale * col(q, t) * row(gy, t)) ** 2
        g[0][:, t] = scale * (S * row(gy, t)).sum(3)
        s[0][:, t] = scale ** 2 * (R * row(gy, t) ** 2).sum(3)
        along, alongs = (dS * col(k, t)).sum(2), (D * col(k, t) ** 2).sum(2)
        de, des = b[:, t] * along, b[:, t] ** 2 * alongs
        g[1][:, t] = (dS * (b[:, t] * e)[:, :, None]).sum(3) - (S1 * de[:, :, None]).sum(3)
        s[1][:, t] = (D * (b[:, t] ** 2 * e ** 2)[:, :, None] + dS ** 2 * (b[:, t] ** 2 * es)[:, :, None]
                      + R1 * de[:, :, None] ** 2 + S1 ** 2 * des[:, :, None]).sum(3)
        g[2][:, t], s[2][:, t] = de, des
        g[4][:, t], s[4][:, t] = (along * e).sum(-1), (alongs * e ** 2 + along ** 2 * es).sum(-1)
        # the decay's gradient is found by sums of <grad_y, y> - <grad_v, v> to where <dS, S> is known, 160 positions
        # ahead at most
        s[3][:, t] = (ys[:, t] * gy[:, t] ** 2 + des * v[:, t] ** 2).sum(-1)
        both = (D * S ** 2 + dS ** 2 * R).sum((-1, -2))
        dS = dS - col(k, t) * de[:, :, None]
        D = D + col(k, t) ** 2 * des[:, :, None]
        g[3][:, t] = (dS * S1).sum((-1, -2))
        s[3][:, t] += both / 160
        dS, D = dS * a[:, t], D * a[:, t] ** 2
    ahead = torch.cat([s[3], s[3].new_zeros(B, 160, H)], 1).flip(1).cumsum(1).flip(1)
    s[3] = ahead[:, :T] - ahead[:, 160:]

    def joined(x):
        return x.view(B, T, J, H // J, N).sum(3)
    g[0], g[1], s[0], s[1] = (joined(x) for x in (g[0], g[1], s[0], s[1]))
    for i in (0, 1, 2):
        g[i] = g[i] * on4
    for i in (3, 4):
        g[i] = g[i] * on3
    return [y * on4, last, *g, dS], [ys, lasts, *s, D]


def near(got, want, size, tol, dtype, what):
    import torch
    assert got.shape == want.shape, what
    if not got.numel():
        return
    assert torch.isfinite(got).all(), what
    off = (got.double() - want).norm().item()
    whole = max(want.norm().item(), size.clamp(min=0).sum().sqrt().item())
    # fp16's smallest step adds to its relative rounding
    tiny = 2.0 ** -25 * got.numel() ** 0.5 if dtype == "float16" else 0.0
    half = HALF[dtype] * want.norm().item() if dtype != "float32" else 0.0
    assert off <= tol * whole + half + tiny + 1e-30, (what, off / max(whole, 1e-30), off / max(want.norm().item(), 1e-30))


def compare(results, case, scale, lens=None):
    want, size = reference(*case, scale, lens)
    dtype = str(case[2].dtype).replace("torch.", "")
    for name, got, w, s in zip(("y", "last") + NAMES, results, want, size):
        kind = dtype if name in ("y", "grad_q", "grad_k", "grad_v") else "float32"
        tol = 1e-5 if name in ("y", "last") else 2e-5
        if dtype == "bfloat16" and name in ("grad_q", "grad_k"):
            tol += 2.0 ** -9
        near(got, w, s, tol, kind, name)


def check(case, offsets=None, lens=None, scale=None, state=True, last=True):
    q, k, v, decay, beta, s0, gy, gl = case
    B, T, H, V = v.shape
    J, N = q.shape[2:]
    plan = sl.DeltaScan(N, V, H, max_batch=max(B, 1), max_len=max(T, 1), key_heads=J, scale=scale, training=True)
    s0, gl = s0 if state else None, gl if last else None
    y, end = plan.forward(q, k, v, decay, beta, offsets=offsets, state=s0)
    got = plan.backward(q, k, v, decay, beta, gy, offsets=offsets, state=s0, grad_last=gl)
    compare((y, end) + got, (q, k, v, decay, beta, s0, gy, gl), plan.scale, lens)
    return plan, y, end, got


# lengths around the chunk of 32 and over several, widths on and off the tiles of 16, 32, 64 and 128
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("B,T,H,J,N,V", [
    (1, 1, 1, 1, 1, 1), (2, 5, 2, 2, 16, 16), (1, 31, 1, 1, 32, 32), (3, 32, 2, 1, 32, 16), (2, 33, 3, 3, 64, 48),
    (1, 64, 4, 2, 50, 42), (2, 100, 2, 2, 128, 128), (1, 97, 2, 1, 100, 7), (1, 70, 1, 1, 7, 100), (2, 200, 4, 4, 64, 64),
    (1, 300, 6, 2, 33, 128), (5, 40, 3, 1, 128, 33), (1, 259, 1, 1, 128, 112), (4, 65, 1, 1, 24, 80), (2, 70, 2, 2, 64, 128),
    (2, 0, 2, 1, 16, 16)])
def test_shapes(B, T, H, J, N, V, dtype):
    check(make(B, T, H, J, N, V, dtype, B + T + N))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_many_sequences_and_long_memory(dtype):
    check(make(200, 70, 2, 2, 32, 32, dtype, 1))
    check(make(1, 700, 2, 2, 64, 64, dtype, 2, slow=True))
    check(make(2, 400, 1, 1, 128, 128, dtype, 3, slow=True))


# more heads than an SM takes two of, values of six to eight tiles of 16: in one CTA and in two, with fewer chunks than
# a CTA may have producers
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("B,T,H,J,N,V", [(100, 3, 4, 2, 16, 83), (90, 40, 4, 4, 64, 128), (80, 33, 4, 1, 128, 112),
                                         (85, 70, 4, 2, 100, 96), (400, 1, 1, 1, 128, 128)])
def test_many_wide_heads(B, T, H, J, N, V, dtype):
    import torch
    case = make(B, T, H, J, N, V, dtype, B + T)
    lens = torch.arange(B, device="cuda") * 7 % (T + 1)
    offsets = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).int()
    _, y, end, got = check(case, offsets=offsets, lens=lens)
    dead = torch.arange(T, device="cuda")[None] >= lens[:, None]
    assert not y[dead].any() and not any(g[dead].any() for g in got[:5])


# sequences that are cut into segments: of lengths on and off theirs, entries that end in each, and none
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("T,H,J,N,V,slow", [(2048, 2, 1, 32, 32, True), (2100, 1, 1, 128, 128, False),
                                            (2305, 3, 3, 64, 40, True), (3000, 1, 1, 100, 120, True),
                                            (2500, 2, 2, 16, 128, False)])
def test_long_sequences(T, H, J, N, V, slow, dtype):
    check(make(1, T, H, J, N, V, dtype, T, slow=slow))


def test_long_sequences_of_many_lengths():
    import torch
    B, T = 6, 2200
    case = make(B, T, 1, 1, 32, 48, "bfloat16", 21, slow=True)
    lens = torch.tensor([0, 5, 256, 700, 2177, 2200], device="cuda")
    offsets = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).int()
    _, y, end, got = check(case, offsets=offsets, lens=lens)
    dead = torch.arange(T, device="cuda")[None] >= lens[:, None]
    assert not y[dead].any() and torch.equal(end[0], case[5][0])
    assert not any(g[dead].any() for g in got[:5]) and torch.equal(got[5][0], case[7][0])


@pytest.mark.parametrize("dtype", ["float32", "float16"])
def test_lengths(dtype):
    """Entries of no position, of some, of all and (by their offsets) of more than the time axis; NaN and infinities
    lie past the ends."""
    import torch
    B, T = 9, 90
    case = list(make(B, T, 2, 1, 24, 40, dtype, 4))
    lens = torch.tensor([0, 1, 31, 32, 33, 64, 89, 90, 120], device="cuda")
    offsets = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).int()
    dead = torch.arange(T, device="cuda")[None] >= lens[:, None]
    for i in (0, 1, 2, 3, 4, 6):
        case[i][dead] = float("nan") if i % 2 else float("inf")
    plan, y, end, got = check(case, offsets=offsets, lens=lens)
    assert not y[dead].any() and torch.equal(end[0], case[5][0])
    assert not any(g[dead].any() for g in got[:5]) and torch.equal(got[5][0], case[7][0])


def test_no_states_and_other_scales():
    case = make(2, 75, 2, 2, 32, 32, "float32", 5)
    check(case, state=False)
    check(case, last=False)
    check(case, state=False, last=False, scale=1.0)
    check(case, scale=-0.3)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_beta_of_zero_and_one_and_two(dtype):
    """beta 0 leaves the state alone (and has a gradient), 2 reflects it."""
    import torch
    case = list(make(2, 80, 2, 2, 32, 24, dtype, 6))
    for value in (0.0, 1.0, 2.0):
        case[4] = torch.full_like(case[4], value)
        check(case)
    case[4][:, ::3], case[4][:, 1::3] = 0.0, 1.0
    check(case)
    case[4] = torch.zeros_like(case[4])
    _, y, end, _ = check(case, state=False)
    assert not y.any() and not end.any()


def test_the_same_key_again_and_again():
    """Powers of M would cancel here; the substitution does not."""
    case = list(make(2, 130, 2, 2, 32, 32, "float32", 7, slow=True))
    case[1] = case[1][:, :1].expand_as(case[1]).contiguous()
    check(case)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_decays_of_all_sizes(dtype):
    """0, tiny, so large that exp underflows beside ones that matter, and -infinity, which forgets: a chunk's sums of
    them keep their digits."""
    import torch
    case = list(make(3, 150, 2, 2, 32, 32, dtype, 8))
    d = case[3]
    d[:, ::5], d[:, 1::7], d[:, 10::31], d[:, 17::29] = 0.0, -1e-9, -300.0, -90.0
    check(case)
    d[:, 45], d[:, 100:103], d[0, 64] = -torch.inf, -torch.inf, -1e30
    _, _, _, got = check(case)
    assert not got[3][:, 45].any()


def test_growing_states():
    """Decays above 0 are the formula's too."""
    case = list(make(1, 100, 1, 1, 16, 16, "float32", 9))
    case[3] = -case[3] * 0.2
    check(case)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_views(dtype):
    """q, k and v as parts of one projection, decay and beta as parts of another, outputs in the middle of others."""
    import torch
    B, T, H, N, V = 2, 77, 2, 32, 48
    q, k, v, decay, beta, s0, gy, gl = make(B, T, H, H, N, V, dtype, 10)
    plan = sl.DeltaScan(N, V, H, B, T, training=True)
    args = (q, k, v, decay, beta)
    want = plan.forward(*args, state=s0) + plan.backward(*args, gy, state=s0, grad_last=gl)
    for shift in (0, 8, 3):
        both = torch.full((B, T + 2, H, 3 * 64 + shift), 9.0, device="cuda", dtype=q.dtype)
        views = [both[:, 1:-1, :, shift + i * 64:shift + i * 64 + w] for i, w in enumerate((N, N, V))]
        for to, x in zip(views, (q, k, v)):
            to.copy_(x)
        out = torch.full((B, T, H, 64 + shift), 5.0, device="cuda", dtype=q.dtype)
        grads = torch.full_like(both, 5.0)
        gviews = [grads[:, 1:-1, :, shift + i * 64:shift + i * 64 + w] for i, w in enumerate((N, N, V))]
        nums = torch.cat([decay, beta], 2)
        gnums = torch.full_like(nums, 5.0)
        plan.forward(*views, nums[..., :H], nums[..., H:], state=s0, y=out[..., shift:shift + V])
        plan.backward(*views, nums[..., :H], nums[..., H:], gy, state=s0, grad_last=gl, grad_q=gviews[0],
                      grad_k=gviews[1], grad_v=gviews[2], grad_decay=gnums[..., :H], grad_beta=gnums[..., H:])
        assert torch.equal(out[..., shift:shift + V], want[0])
        for a, b in zip(gviews + [gnums[..., :H], gnums[..., H:]], want[2:7]):
            assert torch.equal(a, b)
        assert (out[..., shift + V:] == 5).all() and (out[..., :shift] == 5).all()
        assert (grads[:, 0] == 5).all() and (grads[:, -1] == 5).all() and (grads[..., shift + 32:shift + 64] == 5).all()
    # the same keys for every entry; decay and beta as neighbours of one tensor
    one = [x[:1].expand_as(x) for x in (q, k)]
    nums = torch.stack([decay, beta], -1)
    a = plan.forward(*one, v, nums[..., 0], nums[..., 1])
    b = plan.forward(*(x.contiguous() for x in one), v, decay, beta)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_results_repeat_and_replay():
    import torch
    case = make(4, 150, 4, 2, 64, 64, "bfloat16", 11)
    q, k, v, decay, beta, s0, gy, gl = case
    plan = sl.DeltaScan(64, 64, 4, 4, 150, key_heads=2, training=True)

    def both():
        return plan.forward(q, k, v, decay, beta, state=s0) + plan.backward(q, k, v, decay, beta, gy, state=s0,
                                                                            grad_last=gl)
    first = both()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, both()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = both()
    for t in case:
        t.copy_(t.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b.flip(0)) for a, b in zip(out, first))


def test_sequences_in_pieces_and_in_steps():
    """A sequence forward in two calls through the state, and one position at a time: all the same recurrence, fp32
    roundings apart."""
    import torch
    B, T, H, J, N, V = 3, 75, 4, 2, 32, 40
    case = make(B, T, H, J, N, V, "float32", 12)
    q, k, v, decay, beta, s0, gy, gl = case
    plan = sl.DeltaScan(N, V, H, B, T, key_heads=J)
    cut = 41
    y1, mid = plan.forward(q[:, :cut], k[:, :cut], v[:, :cut], decay[:, :cut], beta[:, :cut], state=s0)
    y2, end = plan.forward(q[:, cut:], k[:, cut:], v[:, cut:], decay[:, cut:], beta[:, cut:], state=mid)
    want, size = reference(*case, plan.scale)
    near(torch.cat([y1, y2], 1), want[0], size[0], 1e-5, "float32", "y in pieces")
    near(end, want[1], size[1], 1e-5, "float32", "last in pieces")
    pool = torch.randn(10, H, N, V, device="cuda")
    rows = torch.tensor([7, 0, 4], device="cuda")
    pool[rows] = s0
    before = pool.clone()
    ys = [plan.step(q[:, t], k[:, t], v[:, t], decay[:, t], beta[:, t], rows, pool) for t in range(T)]
    near(torch.stack(ys, 1), want[0], size[0], 1e-5, "float32", "y in steps")
    near(pool[rows], want[1], size[1], 1e-5, "float32", "states of steps")
    others = torch.tensor([1, 2, 3, 5, 6, 8, 9], device="cuda")
    assert torch.equal(pool[others], before[others])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("n,H,J,N,V", [(1, 1, 1, 1, 1), (7, 4, 2, 64, 64), (33, 2, 2, 128, 128), (5, 3, 1, 50, 42),
                                       (200, 1, 1, 16, 8), (9, 2, 1, 128, 127), (3, 2, 2, 100, 4), (0, 2, 2, 8, 8),
                                       (20, 2, 2, 33, 96), (6, 1, 1, 128, 17), (4, 2, 1, 30, 64)])
def test_step(n, H, J, N, V, dtype):
    """fp32 sums of at most 128 terms: 128 u in the worst case, 1e-6 as a norm over the parts."""
    import torch
    case = make(n, 1, H, J, N, V, dtype, n + V)
    q, k, v, decay, beta = (x[:, 0] for x in case[:5])
    pool = torch.randn(n + 5, H, N, V, device="cuda")
    rows = torch.randperm(n + 5, device="cuda")[:n].contiguous()
    if n > 4:
        rows[1], rows[3] = -1, n + 5
    if n > 6:
        decay[6] = -torch.inf
    plan = sl.DeltaScan(N, V, H, 1, 1, key_heads=J)
    before = pool.clone()
    y = plan.step(q, k, v, decay, beta, rows, pool)
    on = (rows >= 0) & (rows < n + 5)
    if on.any():
        part = [x[on] for x in case[:5]]
        want, size = reference(*part, before[rows[on]], case[6][on], None, plan.scale)
        near(y[on], want[0][:, 0], size[0], 1e-6, dtype, "y")
        near(pool[rows[on]], want[1], size[1], 1e-6, "float32", "states")
    others = torch.ones(n + 5, dtype=torch.bool, device="cuda")
    others[rows[on]] = False
    assert torch.equal(pool[others], before[others]) and not y[~on].any()


# accesses of two channels and of one, with few and many rows of the state to a thread
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("n,H,J,N,V", [(6, 2, 2, 100, 50), (6, 2, 1, 128, 126), (5, 1, 1, 60, 127), (50, 2, 2, 16, 6),
                                       (4, 1, 1, 128, 65), (4, 3, 3, 64, 62)])
def test_step_widths(n, H, J, N, V, dtype):
    test_step(n, H, J, N, V, dtype)


def test_gradients_are_differences():
    """A step of 1e-3 along a direction through the recurrence in 64 bits against the gradient: third order terms are
    below 1e-4 of the gradient's magnitudes."""
    import torch
    case = make(1, 50, 2, 1, 16, 16, "float32", 13)
    plan = sl.DeltaScan(16, 16, 2, 1, 50, key_heads=1, training=True)
    q, k, v, decay, beta, s0, gy, gl = case
    got = plan.backward(q, k, v, decay, beta, gy, state=s0, grad_last=gl)
    gen = torch.Generator(device="cuda").manual_seed(5)
    for i, g in enumerate(got):
        d = torch.randn(g.shape, generator=gen, device="cuda").double()
        ends = []
        for sign in (1, -1):
            at = [x.double() for x in (q, k, v, decay, beta, s0)]
            at[i] = at[i] + sign * 1e-3 * d
            y, end = reference(*at, gy, gl, plan.scale)[0][:2]
            ends.append((y * gy.double()).sum() + (end * gl.double()).sum())
        diff = (ends[0] - ends[1]) / 2e-3
        assert (diff - (g.double() * d).sum()).abs() <= 1e-3 * (g.double() * d).norm(), NAMES[i]


def test_refusals():
    import torch
    case = make(2, 20, 4, 2, 16, 24, "float32", 1)
    q, k, v, decay, beta, s0, gy, gl = case
    plan = sl.DeltaScan(16, 24, 4, 2, 20, key_heads=2, training=True)
    args = (q, k, v, decay, beta)
    y, _ = plan.forward(*args)

    def swap(i, x):
        a = list(args)
        a[i] = x
        return a
    i64 = torch.zeros(2, dtype=torch.int64, device="cuda")
    first = [x[:, 0] for x in args]
    for f in (lambda: plan.forward(*swap(0, q[:, :, :1])), lambda: plan.forward(*swap(1, k.half())),
              lambda: plan.forward(*swap(2, v[..., :16])), lambda: plan.forward(*swap(2, v.cpu())),
              lambda: plan.forward(*swap(3, decay[:, :10])), lambda: plan.forward(*swap(4, beta.double())),
              lambda: plan.forward(*swap(0, q.transpose(2, 3).contiguous().transpose(2, 3))),
              lambda: plan.forward(*args, state=s0[:1]), lambda: plan.forward(*args, y=y[..., :8]),
              lambda: plan.forward(*args, offsets=torch.zeros(2, dtype=torch.int32, device="cuda")),
              lambda: plan.backward(*args, gy[:, :5]), lambda: plan.backward(*args, gy, grad_last=gl.half()),
              lambda: plan.backward(*args, gy, grad_beta=beta[:1]), lambda: plan.step(*first, i64.int(), s0),
              lambda: plan.step(*first, i64, s0[:, :2]), lambda: plan.step(*first[:2], v, *first[3:], i64, s0)):
        with pytest.raises(ValueError):
            f()
    small = sl.DeltaScan(16, 24, 4, 1, 20, key_heads=2)
    for f in (lambda: small.forward(*args), lambda: small.backward(*(x[:1] for x in args), gy[:1]),
              lambda: plan.forward(*args, y=y[:, :1].expand_as(y)),
              lambda: plan.forward(*(torch.cat([x, x], 1) for x in args)),
              lambda: sl.DeltaScan(129, 16, 1, 1, 1), lambda: sl.DeltaScan(16, 129, 1, 1, 1),
              lambda: sl.DeltaScan(16, 16, 3, 1, 1, key_heads=2), lambda: sl.DeltaScan(16, 16, 1, 0, 1),
              lambda: sl.DeltaScan(16, 16, 1, 1, 1, scale=float("inf")).forward(*(x[:1, :1, :1, :16] if x.dim() == 4
                                                                                  else x[:1, :1, :1] for x in args))):
        with pytest.raises(sl.EmbError):
            f()
