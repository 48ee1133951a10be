"""Layer norm, forward and backward, against the formulas in 64 bits.

Tolerances, u = 2^-24: a lane adds at most 32 values and 9 partial sums of other
lanes, so a row's sums are within 64 u of the sum of magnitudes.  The mean is off
by at most 64 u max|x|, hence xh by 64 u (max|x| rstd + |xh|); sums of squares and
the root add 64 u |xh| more.  Sums over rows: n u sum|terms| in any order.  A
stored result of 16 bits adds half a unit."""
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


def make(shape, dtype, seed, spread=1.0, mean=0.5):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=gen, device="cuda")
    D, dt = shape[-1], getattr(torch, dtype)
    x = (r(*shape) * spread + mean).to(dt)
    return x, r(*shape).to(dt), 1 + 0.2 * r(D), 0.2 * r(D)


def reference(x, dy, w, b, eps, live=None):
    """y, grad_x, grad_weight, grad_bias in 64 bits, and the bounds of the module's comment."""
    import torch
    D = x.shape[-1]
    x, dy = x.double().reshape(-1, D), dy.double().reshape(-1, D)
    w = torch.ones(D, dtype=torch.float64, device="cuda") if w is None else w.double()
    b = torch.zeros(D, dtype=torch.float64, device="cuda") if b is None else b.double()
    if live is not None:
        on = live.reshape(-1, 1)
        x, dy = torch.where(on, x, 0.0), torch.where(on, dy, 0.0)
    mean = x.mean(1, keepdim=True)
    rstd = 1 / ((x - mean).square().mean(1, keepdim=True) + eps).sqrt()
    h = (x - mean) * rstd
    y = h * w + b
    g = dy * w
    gx = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    off = 64 * U * (x.abs().amax(1, keepdim=True) * rstd + 2 * h.abs() + 1)          # of xh
    G, X, S = g.abs().amax(1, keepdim=True), 1 + h.abs().amax(1, keepdim=True), 1 + x.abs().amax(1, keepdim=True) * rstd
    tol = [off * w.abs() + 4 * U * (y.abs() + b.abs()), 256 * U * rstd * G * X * X * S,
           (dy.abs() * (off + (x.shape[0] + 4) * U * h.abs())).sum(0), (x.shape[0] * U * dy.abs()).sum(0)]
    if live is not None:
        y, gx = y * on, gx * on
    return [y, gx, (dy * h).sum(0), dy.sum(0)], tol


def check(got, want, tol, dtype, what):
    import torch
    got = got.double().reshape(want.shape)
    if not got.numel():
        return
    assert torch.isfinite(got).all(), what
    slack = (got - want).abs() - (tol + HALF[dtype] * want.abs() + TINY[dtype])
    assert slack.max() <= 0, (what, slack.max().item(), (got - want).abs().max().item())


def run(x, dy, w, b, eps=1e-5, offsets=None, live=None):
    plan = sl.LayerNorm(x.shape[-1], eps=eps)
    y, stats = plan.forward(x, w, b, offsets=offsets)
    gx, gw, gb = plan.backward(x, dy, stats, w, offsets=offsets)
    dtype = str(x.dtype).replace("torch.", "")
    want, tol = reference(x, dy, w, b, eps, live)
    for name, got, ref, t, kind in zip(("y", "grad_x", "grad_weight", "grad_bias"), (y, gx, gw, gb), want, tol,
                                       (dtype, dtype, "float32", "float32")):
        check(got, ref, t, kind, name)
    return y, gx, gw, gb


# every variant: one access a lane, several, a row over a CTA, the most that a thread holds; accesses of 1, 2, 4, 8
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("rows,dim", [(1, 1), (1, 8), (3, 2), (700, 7), (1000, 15), (333, 24), (5003, 99), (65, 50),
                                      (2000, 64), (77, 256), (130, 257), (40, 512), (33, 1000), (300, 1024), (9, 1030),
                                      (21, 2049), (700, 4096), (3, 4098), (2, 5001), (4, 8192), (1, 8194), (2, 16383),
                                      (5, 16384), (700, 16384), (0, 64)])
def test_rows(rows, dim, dtype):
    run(*make((rows, dim), dtype, rows + dim))


# rows at the ends of what a warp holds, of each access, and rows enough that a CTA has several
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("rows,dim", [(3000, 56), (3000, 64), (900, 127), (3000, 258), (3000, 499), (20, 511), (3000, 513),
                                      (3000, 514), (3000, 516), (3000, 618), (20, 767), (3000, 768), (3000, 1020),
                                      (3000, 1022), (3000, 1023), (3000, 1025), (3000, 1028), (3000, 1536),
                                      (3000, 2046), (2000, 4553), (700, 8190), (700, 8193), (300, 16382)])
def test_widths(rows, dim, dtype):
    run(*make((rows, dim), dtype, rows + dim))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("dim", [64, 99, 1024, 2048])
def test_many_rows(dim, dtype):
    run(*make((40_000_000 // dim // 4, dim), dtype, dim))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_weights_of_the_rows_type_and_none(dtype):
    x, dy, w, b = make((50, 96), dtype, 3)
    run(x, dy, w.to(x.dtype), b.to(x.dtype))
    run(x, dy, None, None)
    run(x, dy, w, None)
    run(x, dy, None, b)


def test_a_large_mean_keeps_its_digits():
    """Deviations of 1 around a mean of 3000: two passes over the row lose 64 u max|x| of a deviation, as bounded."""
    run(*make((100, 300), "float32", 5, mean=3000.0))


def test_rows_without_deviation():
    import torch
    x, dy, w, b = make((6, 40), "float32", 6)
    x[1], x[3] = 0.0, 2.5
    y, gx, _, _ = run(x, dy, w, b)
    assert torch.equal(y[1], b) and torch.equal(y[3], b)


@pytest.mark.parametrize("dtype", ["float32", "float16"])
@pytest.mark.parametrize("batch,time,dim", [(5, 7, 19), (1, 9, 32), (70, 1, 64), (33, 100, 128), (3, 2, 3000)])
def test_padded_sequences(batch, time, dim, dtype):
    """Past the ends lie NaN and infinities; offsets may be longer than the time axis."""
    import torch
    x, dy, w, b = make((batch, time, dim), dtype, dim)
    lens = torch.arange(batch, device="cuda") * 7 % (time + 3)
    live = torch.arange(time, device="cuda")[None] < lens[:, None]
    x[~live], dy[~live] = float("nan"), float("inf")
    offsets = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).int()
    y, gx, _, _ = run(x, dy, w, b, offsets=offsets, live=live)
    assert not y[~live].any() and not gx[~live].any()


def test_nothing_live():
    import torch
    x, dy, w, b = make((4, 5, 16), "float32", 1)
    offsets = torch.zeros(5, dtype=torch.int32, device="cuda")
    x[:], dy[:] = float("nan"), float("nan")
    plan = sl.LayerNorm(16)
    y, stats = plan.forward(x, w, b, offsets=offsets)
    out = plan.backward(x, dy, stats, w, offsets=offsets)
    assert not y.any() and not stats.any() and not any(t.any() for t in out)
    empty = x[:, :0]
    y, stats = plan.forward(empty, w, b)
    gx, gw, gb = plan.backward(empty, empty, stats, w, grad_weight=torch.ones(16, device="cuda"))
    assert y.shape == (4, 0, 16) and not gw.any() and not gb.any()


def test_strided_views_and_given_outputs():
    import torch
    x, dy, w, b = make((6, 11, 64), "bfloat16", 9)
    wide = torch.randn(6, 11, 200, device="cuda", dtype=torch.bfloat16)
    for first in (0, 8, 3):             # aligned to 16 bytes, and to 2
        v = wide[:, 1:9, first:first + 64]
        out = torch.full((6, 8, 130), 7.0, device="cuda", dtype=torch.bfloat16)
        plan = sl.LayerNorm(64)
        # the accesses' width decides the order of a row's sums: against the formulas, not against each other
        got, stats = plan.forward(v, w, b, y=out[..., 1:65])
        want, tol = reference(v, dy[:, :8], w, b, plan.eps)
        grads = plan.backward(v, dy[:, :8], stats, w)
        for name, p, q, t, kind in zip(("y", "grad_x", "grad_weight", "grad_bias"), (got, *grads), want, tol,
                                       ("bfloat16", "bfloat16", "float32", "float32")):
            check(p, q, t, kind, name)
        assert (out[..., 65:] == 7).all() and (out[..., 0] == 7).all()
    rows = x[:, 4]                      # rows with a stride of their own
    want, _ = sl.LayerNorm(64).forward(rows.contiguous(), w, b)
    assert torch.equal(sl.LayerNorm(64).forward(rows, w, b)[0], want)
    one = x[0, :1].expand(9, 64)        # the same row again and again
    assert torch.equal(sl.LayerNorm(64).forward(one, w, b)[0], sl.LayerNorm(64).forward(one.contiguous(), w, b)[0])


def test_results_repeat_and_replay():
    import torch
    x, dy, w, b = make((3000, 192), "bfloat16", 2)
    plan = sl.LayerNorm(192)
    y, stats = plan.forward(x, w, b)
    first = plan.backward(x, dy, stats, w)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(first, plan.backward(x, dy, stats, w)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        y2, stats2 = plan.forward(x, w, b)
        out = plan.backward(x, dy, stats2, w)
    x.copy_(x.flip(0))
    dy.copy_(dy.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, y.flip(0)) and torch.equal(out[0], first[0].flip(0))


def test_gradients_are_differences():
    """A step along a direction against the gradient, in 64 bits around the fp32 result: second order terms of a
    step of 1e-3 times rows of unit deviation stay below 1e-5 of the sum's magnitudes."""
    import torch
    x, dy, w, b = make((40, 33), "float32", 12, mean=0.0)
    plan = sl.LayerNorm(33)
    _, stats = plan.forward(x, w, b)
    gx, gw, gb = plan.backward(x, dy, stats, w)
    gen = torch.Generator(device="cuda").manual_seed(4)
    for t, g in ((x, gx), (w, gw), (b, gb)):
        d = torch.randn(t.shape, generator=gen, device="cuda").double()
        ends = []
        for sign in (1, -1):
            at = [u.double() + (sign * 1e-3 * d if u is t else 0) for u in (x, w, b)]
            y = reference(at[0], dy, at[1], at[2], plan.eps)[0][0]
            ends.append((y * dy.double()).sum())
        diff = (ends[0] - ends[1]) / 2e-3
        assert (diff - (g.double() * d).sum()).abs() <= 1e-4 * (g.double() * d).abs().sum()


def test_refusals():
    import torch
    x, dy, w, b = make((4, 5, 16), "float32", 1)
    plan = sl.LayerNorm(16)
    y, stats = plan.forward(x, w, b)
    o = torch.zeros(5, dtype=torch.int32, device="cuda")
    for f in (lambda: plan.forward(x[..., :8], w, b), lambda: plan.forward(x.cpu(), w, b),
              lambda: plan.forward(x, w[:8], b), lambda: plan.forward(x, w, b.half()),
              lambda: plan.forward(x.double(), w, b), lambda: plan.forward(x, w, b, offsets=o[:4]),
              lambda: plan.forward(x, w, b, offsets=o.long()), lambda: plan.forward(x[0], w, b, offsets=o[:2]),
              lambda: plan.forward(x, w, b, y=y[:, :4]), lambda: plan.forward(x, w, b, stats=stats[:3]),
              lambda: plan.forward(x.transpose(1, 2).contiguous().transpose(1, 2), w, b),
              lambda: plan.backward(x, dy.half(), stats, w), lambda: plan.backward(x, dy, stats[:2], w),
              lambda: plan.backward(x, dy, stats, w, grad_weight=w.half())):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: plan.forward(x, w, b, y=y[:, :1].expand(4, 5, 16)),       # outputs on top of one another
              lambda: sl.LayerNorm(0), lambda: sl.LayerNorm(16385), lambda: sl.LayerNorm(16, eps=-1.0).forward(x)):
        with pytest.raises(sl.EmbError):
            f()
