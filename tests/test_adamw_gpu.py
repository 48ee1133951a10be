"""AdamW over many tensors.  The states are checked bit for bit against the
formulas' operations in numpy float32, rounded one by one; the 8-bit codes
against the grid's definition on those values.  The weights lie within the
bound of their own arithmetic: w' = w - lr d w - lr q, each product and
difference one rounding (3 u |w| and 2 u lr |q| in all, u = 2^-24), and q, from
an approximate root and quotient of a few ulp and four roundings, within 12 u;
16-bit weights add half a unit of their type."""
import gc

import numpy as np
import pytest

import sparse_lookup_gb300 as sl
from sparse_lookup_gb300 import build as slbuild

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"float32": 0.0, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
TINY = 2.0 ** -25      # half the smallest fp16: what rounding to it costs below its normal range
SIZES = [0, 1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 5000, 40000]
F = np.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    slbuild.build()
    sl.lib()


def splitmix64(x):
    with np.errstate(over="ignore"):
        z = np.asarray(x, np.uint64) + np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        return z ^ (z >> np.uint64(31))


def noise(start, n, seed, step):
    """The 16 random bits of elements start .. start + n of the padded order."""
    key = splitmix64((seed << 32) + step)
    i = np.arange(start, start + n, dtype=np.uint64)
    with np.errstate(over="ignore"):
        z = splitmix64(key + i // np.uint64(4))
    return (z >> (np.uint64(16) * (i % np.uint64(4))) & np.uint64(0xFFFF)).astype(np.int64)


def encode(x, nz, signed):
    levels = 127 if signed else 255
    bits = x.view(np.int32).astype(np.int64)
    mag = bits & 0x7FFFFFFF
    mag = np.where(mag < 0x7F800000, mag, 0)
    blocks = [mag[i:i + 256] for i in range(0, x.size, 256)]
    top = np.array([(int(b.max()) + 0xFFFFF) >> 20 for b in blocks], np.int64)
    base = np.repeat(np.maximum(top - levels, 0), 256)[:x.size]
    code = np.maximum(((mag + nz * 16) >> 20) - base, 0)
    assert code.max(initial=0) <= levels
    if signed:
        code = code | np.where(bits < 0, 128, 0)
    return code.astype(np.uint8), top.astype(np.int16)


def decode(code, top, signed):
    levels = 127 if signed else 255
    c = code.astype(np.int64)
    base = np.repeat(np.maximum(top.astype(np.int64) - levels, 0), 256)[:c.size]
    mag = np.where(c & levels, ((c & levels) + base) << 20, 0)
    if signed:
        mag = mag | ((c & 128) << 24)
    return mag.astype(np.uint32).view(np.float32)


class Model:
    """The same optimizer in numpy, tensor by tensor."""

    def __init__(self, w, bits, decay, b1, b2, eps, seed):
        self.w = [x.astype(np.float64) for x in w]
        self.bits, self.decay, self.b1, self.b2, self.eps, self.seed = bits, decay, b1, b2, eps, seed
        if bits == 8:
            self.m = [encode(np.zeros(x.size, F), 0, True) for x in w]
            self.v = [encode(np.zeros(x.size, F), 0, False) for x in w]
        else:
            self.m = [np.zeros(x.size, F) for x in w]
            self.v = [np.zeros(x.size, F) for x in w]
        self.t = 0

    def step(self, grads, lr, scale=None):
        """Updates the states; returns (weights from self.w, their bounds)."""
        self.t += 1
        out, start = [], 0
        for i, g in enumerate(grads):
            with np.errstate(all="ignore"):
                g = g.astype(F) * (F(scale) if scale is not None else F(1))
                m = decode(*self.m[i], True) if self.bits == 8 else self.m[i]
                v = decode(*self.v[i], False) if self.bits == 8 else self.v[i]
                m = m * F(self.b1) + g * F(1 - self.b1)
                v = v * F(self.b2) + (g * g) * F(1 - self.b2)
                q = (m.astype(np.float64) / (1 - self.b1 ** self.t)) / (
                    np.sqrt(v.astype(np.float64) / (1 - self.b2 ** self.t)) + self.eps)
                w = self.w[i]
                new = w - lr * float(F(self.decay[i])) * w - lr * q
                out.append((new, 3 * U * np.abs(w) + 2 * U * np.abs(new) + 14 * U * lr * np.abs(q) + 1e-38))
            nz = noise(start, g.size, self.seed, self.t)
            start += -(-g.size // 256) * 256
            if self.bits == 8:
                self.m[i], self.v[i] = encode(m, nz, True), encode(v, nz, False)
            else:
                self.m[i], self.v[i] = m, v
        return out


def make(sizes, dtype, grad_dtype, seed, offset=0):
    import torch
    gen = torch.Generator().manual_seed(seed)
    dt, gt = getattr(torch, dtype), getattr(torch, grad_dtype)

    def place(x):
        room = torch.zeros(x.numel() + offset, dtype=x.dtype, device="cuda")[offset:]
        return room.copy_(x)
    p = [place(torch.randn(n, generator=gen).to(dt)) for n in sizes]
    g = [place((torch.randn(n, generator=gen) * 10.0 ** (i % 5 - 3)).to(gt)) for i, n in enumerate(sizes)]
    return p, g


def host(ts):
    return [t.detach().float().cpu().numpy() for t in ts]


def check_states(opt, model):
    for i in range(len(opt.params)):
        if model.bits == 8:
            for name, ref in (("m", model.m[i]), ("v", model.v[i])):
                assert np.array_equal(getattr(opt, name)[i].cpu().numpy(), ref[0]), (name, i, "codes")
                assert np.array_equal(getattr(opt, name + "_top")[i].cpu().numpy(), ref[1]), (name, i, "tops")
        else:
            assert np.array_equal(opt.m[i].cpu().numpy().view(np.int32), model.m[i].view(np.int32)), ("m", i)
            assert np.array_equal(opt.v[i].cpu().numpy().view(np.int32), model.v[i].view(np.int32)), ("v", i)


@pytest.mark.parametrize("dtype,grad_dtype,master", [("float32", "float32", False), ("bfloat16", "bfloat16", False),
                                                     ("bfloat16", "float32", True), ("bfloat16", "bfloat16", True),
                                                     ("float16", "float16", True), ("float16", "float32", False)])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("offset", [0, 3])
def test_steps(dtype, grad_dtype, master, bits, offset):
    """Four steps with fresh gradients on sizes around every boundary; offset 3
    puts every tensor off the 16-byte boundaries."""
    import torch
    p, g = make(SIZES, dtype, grad_dtype, 5, offset)
    masters = [x.float() for x in p] if master else None
    decay = [0.1 * (i % 3) for i in range(len(p))]
    opt = sl.AdamW(p, g, masters=masters, weight_decay=decay, betas=(0.9, 0.99), eps=1e-6, state_bits=bits, seed=77)
    model = Model(host(p), bits, decay, 0.9, 0.99, 1e-6, 77)
    for step in range(4):
        scale = None if step % 2 else 0.37
        model.w = [x.astype(np.float64) for x in host(masters if master else p)]
        want = model.step(host(g), 0.01, scale)
        opt.step(0.01, None if scale is None else torch.tensor([scale], device="cuda"))
        check_states(opt, model)
        for i, (ref, bound) in enumerate(want):
            held = host(masters if master else p)[i]
            half = 0.0 if master else HALF[dtype]
            assert np.all(np.abs(held - ref) <= bound + half * (np.abs(ref) + bound) + TINY * (half == HALF["float16"])), (step, i)
            if master:
                assert torch.equal(p[i], masters[i].to(p[i].dtype)), (step, i)
        for i, x in enumerate(g):
            x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(step * 50 + i)) * 0.1)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_of_mixed_kinds(bits):
    """Several hundred tensors of three kinds in one call."""
    import torch
    rng = np.random.default_rng(3)
    p, g, masters = [], [], []
    for i in range(400):
        n = int(rng.integers(0, 3000))
        dt = (torch.float32, torch.bfloat16, torch.float16)[i % 3]
        p.append(torch.randn(n).to(dt).cuda())
        g.append(torch.randn(n).to(dt).cuda())
        masters.append(p[-1].float() if i % 3 and i % 2 else None)
    model = Model([host([x])[0] for x in p], bits, [0.01] * 400, 0.9, 0.999, 1e-8, 5)
    opt = sl.AdamW(p, g, masters=masters, state_bits=bits, seed=5)
    want = model.step(host(g), 1e-3)
    opt.step(1e-3)
    check_states(opt, model)
    for i, (ref, bound) in enumerate(want):
        half = 0.0 if masters[i] is not None else HALF[str(p[i].dtype)[6:]]
        got = host([p[i] if masters[i] is None else masters[i]])[0]
        assert np.all(np.abs(got - ref) <= bound + half * (np.abs(ref) + bound) + TINY * (half == HALF["float16"])), i


def test_states_of_very_different_sizes():
    """Magnitudes over more octaves than a code has, zeros, values below fp32's
    normal range and a block of zeros."""
    import torch
    n = 256 * 6
    x = torch.randn(n) * torch.exp2(torch.randint(-60, 20, (n,)).float())
    x[256:512] = 0
    x[512:768] *= 1e-30
    x[768:1024] = 1e-42
    p, g = [torch.zeros(n, device="cuda")], [x.cuda()]
    model = Model([np.zeros(n, F)], 8, [0.0], 0.9, 0.999, 1e-8, 1)
    opt = sl.AdamW(p, g, weight_decay=0.0, state_bits=8, seed=1)
    for _ in range(3):
        model.step(host(g), 1e-3)
        opt.step(1e-3)
        check_states(opt, model)
    m, v = opt.states()
    assert np.array_equal(m.float().cpu().numpy(), decode(*model.m[0], True))
    assert np.array_equal(v.float().cpu().numpy(), decode(*model.v[0], False))


def test_states_export_layout():
    import torch
    p, g = make(SIZES, "bfloat16", "bfloat16", 9)
    opt = sl.AdamW(p, g, state_bits=8)
    opt.step(1e-3)
    m, v = opt.states()
    at = 0
    for i, n in enumerate(SIZES):
        for got, name, signed in ((m, "m", True), (v, "v", False)):
            want = decode(getattr(opt, name)[i].cpu().numpy(), getattr(opt, name + "_top")[i].cpu().numpy(), signed)
            assert np.array_equal(got[at:at + n].float().cpu().numpy(), want), (name, i)
        room = -(-n // 256) * 256
        assert (m[at + n:at + room] == 0).all()
        at += room
    assert at == m.numel() == v.numel()


def test_rounding_keeps_small_changes():
    """v moves although each step changes it by far less than a place: after 400
    steps of a constant gradient its mean over 64 Ki elements is within five
    standard errors of 1 - beta2^400 times g^2 (each step's rounding has zero
    mean and at most half a place, 2^-4, of standard deviation; the errors of
    400 steps of one element add up to at most 2^-4 / sqrt(1 - beta2^2), and
    the elements' are independent)."""
    import torch
    n = 1 << 16
    p, g = [torch.zeros(n, device="cuda")], [torch.ones(n, device="cuda")]
    opt = sl.AdamW(p, g, weight_decay=0.0, betas=(0.9, 0.999), state_bits=8, seed=11)
    for _ in range(400):
        opt.step(0.0)
    want = 1 - 0.999 ** 400
    got = opt.states()[1].double().mean().item()
    assert abs(got - want) <= 5 * want * 2.0 ** -4 / np.sqrt(1 - 0.999 ** 2) / np.sqrt(n)


@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_that_are_not_finite_stay_in_their_elements(bits):
    import torch
    p, g = make([1000, 300], "float32", "float32", 3)
    clean_p, clean_g = [x.clone() for x in p], [x.clone() for x in g]
    bad = [5, 256, 999]
    for i, v in zip(bad, (float("nan"), float("inf"), float("-inf"))):
        g[0][i] = v
        clean_g[0][i] = 0
    a = sl.AdamW(p, g, state_bits=bits, seed=2)
    b = sl.AdamW(clean_p, clean_g, state_bits=bits, seed=2)
    a.step(1e-3)
    b.step(1e-3)
    keep = torch.ones(1000, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert torch.equal(p[0][keep], clean_p[0][keep]) and torch.equal(p[1], clean_p[1])
    assert not torch.isfinite(p[0][~keep]).any()
    if bits == 8:
        m, v = a.states()
        assert (m[:1000][~keep] == 0).all() and (v[:1000][~keep] == 0).all()
        assert torch.equal(a.m_top[0], b.m_top[0]) and torch.equal(a.v_top[0], b.v_top[0])
        assert torch.equal(a.m[0][keep], b.m[0][keep]) and torch.equal(a.v[0][keep], b.v[0][keep])


def test_bind_grads_streams_and_graphs():
    import torch
    p, g = make([5000, 33], "float32", "float32", 8)
    q = [x.clone() for x in p]
    other = [x * 2 for x in g]
    a, b = sl.AdamW(p, g), sl.AdamW(q, other)
    a.bind_grads(other)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a.step(1e-2, stream=side)
    side.synchronize()
    b.step(1e-2)
    assert all(torch.equal(x, y) for x, y in zip(p + a.m + a.v, q + b.m + b.v))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        a.step(1e-2)
    graph.replay()
    b.step(1e-2)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(p + a.m + a.v, q + b.m + b.v))


def test_refusals():
    import torch
    p = [torch.zeros(8, device="cuda")]
    g = [torch.zeros(8, device="cuda")]
    for args, kw in (((p, [g[0].half()]), {}), ((p, [g[0][:7]]), {}), ((p, g + g), {}), ((p, g), dict(state_bits=16)),
                     (([p[0].double()], [g[0].double()]), {}), ((p, [g[0].cpu()]), {}),
                     ((p, g), dict(m=[torch.zeros(8, dtype=torch.uint8, device="cuda")])),
                     (([torch.zeros(8, 8, device="cuda").t()], [torch.zeros(8, 8, device="cuda")]), {}),
                     ((p, g), dict(weight_decay=[0.1, 0.2]))):
        with pytest.raises(ValueError):
            sl.AdamW(*args, **kw)
    for kw in (dict(masters=[torch.zeros(8, device="cuda")]), dict(weight_decay=-1.0),
               dict(weight_decay=float("nan"))):
        with pytest.raises(sl.EmbError) as e:
            sl.AdamW(p, g, **kw)
        assert e.value.status == 1
    opt = sl.AdamW(p, g)
    for kw in (dict(lr=-1.0), dict(lr=float("nan")), dict(lr=float("inf"))):
        with pytest.raises(sl.EmbError):
            opt.step(**kw)
    assert opt.step_count == 0
    with pytest.raises(sl.EmbError) as e:
        opt.states()
    assert e.value.status == 2
    with pytest.raises(ValueError):
        opt.bind_grads([torch.zeros(7, device="cuda")])
    with pytest.raises(sl.EmbError):
        sl.AdamW(p, g, betas=(1.0, 0.9)).step(0.1)
    with pytest.raises(sl.EmbError):
        sl.AdamW([], [])


def test_allocation_failure():
    import torch
    p, g = [torch.zeros(8, device="cuda")], [torch.zeros(8, device="cuda")]
    gc.collect()   # handles of earlier tests are freed now, not in the middle of the count
    base = sl.emb_debug_live_allocations()
    for k in range(3):
        sl.emb_debug_fail_alloc(k)
        with pytest.raises(sl.EmbError) as e:
            sl.AdamW(p, g)
        sl.emb_debug_fail_alloc(-1)
        assert e.value.status == 3 and sl.emb_debug_live_allocations() == base
