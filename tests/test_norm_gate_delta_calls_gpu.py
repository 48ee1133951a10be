"""The norm, the gate and the delta rule called as programs call them: on other
streams, on several at once with a handle each, with offsets that pass 32 bits,
and when the device has no memory left for a handle.  Results are those of the same
call alone, bit for bit."""
import gc

import pytest

import sparse_lookup_gb300 as sl
from sparse_lookup_gb300 import build as slbuild

pytestmark = pytest.mark.gpu
FAR = 1 << 31
OOM = 3


@pytest.fixture(scope="module", autouse=True)
def built():
    slbuild.build()
    sl.lib()
    yield
    import torch
    torch.cuda.empty_cache()


def far(like, strides):
    """`like` as a view of these strides in a buffer of its own."""
    import torch
    last = sum((n - 1) * s for n, s in zip(like.shape, strides))
    t = torch.empty(last + 1, dtype=like.dtype, device="cuda").as_strided(like.shape, strides)
    return t.copy_(like)


class Work:
    """One handle of each kind and a call of each with inputs of a seed."""

    def __init__(self, seed):
        import torch
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def r(*s):
            return torch.randn(*s, generator=gen, device="cuda")
        self.norm, self.router = sl.LayerNorm(96), sl.ExpertRouter(24, 3, 4000)
        self.delta = sl.DeltaScan(32, 48, 4, 3, 170, key_heads=2, training=True)
        self.rows = (r(4000, 96), r(4000, 96), r(96), r(96))
        self.logits = (r(4000, 24), r(4000, 3), r(2))
        k = torch.nn.functional.normalize(r(3, 170, 2, 32), dim=-1)
        self.seq = (r(3, 170, 2, 32).bfloat16(), k.bfloat16(), r(3, 170, 4, 48).bfloat16(), -r(3, 170, 4).abs() * 0.1,
                    torch.sigmoid(r(3, 170, 4)))
        self.gy, self.states, self.at = r(3, 170, 4, 48).bfloat16(), r(9, 4, 32, 48), torch.tensor([4, 0, 8], device="cuda")

    def run(self, stream=None):
        x, dy, w, b = self.rows
        y, stats = self.norm.forward(x, w, b, stream=stream)
        out = [y, *self.norm.backward(x, dy, stats, w, stream=stream)]
        g = self.router.gate(self.logits[0], stream=stream)
        out += [g.experts, g.weights, g.counts, g.losses,
                self.router.gate_backward(self.logits[0], g, *self.logits[1:], stream=stream)]
        out += [*self.delta.forward(*self.seq, stream=stream), *self.delta.backward(*self.seq, self.gy, stream=stream)]
        states = self.states.clone() if stream is None else self.states
        out += [self.delta.step(*(t[:, 5] for t in self.seq), self.at, states, stream=stream), states]
        return out


def test_another_stream():
    import torch
    work = Work(1)
    want = work.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = work.run(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_handles_at_once():
    import torch
    works = [Work(s) for s in range(4)]
    want = [w.run() for w in works]
    streams = [torch.cuda.Stream() for _ in works]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = []
        for w, s in zip(works, streams):
            with torch.cuda.stream(s):
                got.append(w.run())
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("shape,strides", [((9, 64), (FAR // 8, 1)), ((2, 70, 33), (FAR, 33, 1))])
def test_norm_past_32_bits(shape, strides):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, dy = (torch.randn(shape, generator=gen, device="cuda").bfloat16() for _ in range(2))
    norm = sl.LayerNorm(shape[-1])
    y, stats = norm.forward(x)
    want = [y, *norm.backward(x, dy, stats)]
    y2, stats = norm.forward(far(x, strides), y=far(torch.zeros_like(x), strides))
    got = [y2, *norm.backward(far(x, strides), far(dy, strides), stats, grad_x=far(torch.zeros_like(x), strides))]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gate_past_32_bits():
    import torch
    gen = torch.Generator(device="cuda").manual_seed(4)
    logits = torch.randn(9, 40, generator=gen, device="cuda").bfloat16()
    router, gl = sl.ExpertRouter(40, 2, 9), torch.ones(2, device="cuda")
    want = router.gate(logits)
    grad = router.gate_backward(logits, want, want.weights, gl)
    wide = far(logits, (FAR // 8, 1))
    got = router.gate(wide)
    assert torch.equal(got.weights, want.weights) and torch.equal(got.experts, want.experts)
    assert torch.equal(router.gate_backward(wide, got, want.weights, gl, grad_logits=far(torch.zeros_like(logits),
                                                                                       (FAR // 8, 1))), grad)


@pytest.mark.parametrize("strides", [(FAR, 64, 32, 1), (64, FAR // 64, 32, 1), (2048, 32, FAR, 1)])
def test_delta_past_32_bits(strides):
    """Entries, positions and heads far apart; of outputs only the first two lie as they must."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(5)
    B, T, H, N = 2, 64, 2, 32
    if strides[1] > 1000:
        B = 1
    q, k, v, gy = (torch.randn(B, T, H, N, generator=gen, device="cuda").bfloat16() * 0.2 for _ in range(4))
    decay, beta = -torch.rand(B, T, H, generator=gen, device="cuda"), torch.rand(B, T, H, generator=gen, device="cuda")
    plan = sl.DeltaScan(N, N, H, B, T, training=True)
    want = [*plan.forward(q, k, v, decay, beta), *plan.backward(q, k, v, decay, beta, gy)]
    args = [far(t, strides) for t in (q, k, v)] + [decay, beta]
    outs = [torch.zeros_like(q) if strides[2] == FAR else far(torch.zeros_like(q), strides) for _ in range(4)]
    got = [*plan.forward(*args, y=outs[0]),
           *plan.backward(*args, far(gy, strides), grad_q=outs[1], grad_k=outs[2], grad_v=outs[3])]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_pool_past_32_bits():
    import torch
    H, N = 4, 128
    rows = FAR // (H * N * N) + 3
    states = torch.zeros(rows, H, N, N, device="cuda")
    at = torch.tensor([rows - 1, 0], device="cuda")
    k = torch.nn.functional.normalize(torch.randn(2, H, N, device="cuda"), dim=-1)
    v, plan = torch.randn(2, H, N, device="cuda"), sl.DeltaScan(N, N, H, 1, 1, scale=1.0)
    one = torch.ones(2, H, device="cuda")
    y = plan.step(k, k, v, 0 * one, one, at, states)        # written and read with the same key: v again
    assert (y - v).abs().max() <= 1e-5 * v.abs().max()
    small = torch.zeros(2, H, N, N, device="cuda")
    plan.step(k, k, v, 0 * one, one, torch.tensor([0, 1], device="cuda"), small)
    assert torch.equal(states[at], small)
    states[at] = 0
    assert not states[::1000].any()


@pytest.mark.parametrize("create", [lambda: sl.LayerNorm(64), lambda: sl.ExpertRouter(16, 2, 100),
                                    lambda: sl.DeltaScan(32, 32, 2, 2, 4096),
                                    lambda: sl.DeltaScan(32, 32, 2, 2, 4096, training=True)])
def test_no_memory_for_a_handle(create):
    """Every allocation fails in turn; nothing is leaked."""
    gc.collect()
    before = sl.emb_debug_live_allocations()
    try:
        for after in range(40):
            sl.emb_debug_fail_alloc(after)
            try:
                handle = create()
            except sl.EmbError as e:
                assert e.status == OOM
                assert sl.emb_debug_live_allocations() == before
            else:
                break
        else:
            raise AssertionError("no creation succeeded")
        assert after >= 1
    finally:
        sl.emb_debug_fail_alloc(-1)
    handle.close()
    assert sl.emb_debug_live_allocations() == before
