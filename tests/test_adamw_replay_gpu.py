"""AdamW under graph replay: every replay is a step of its own, the same bits as
that step taken one by one."""
import pytest

import sparse_lookup_gb300 as sl
from sparse_lookup_gb300 import build as slbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    slbuild.build()
    sl.lib()


class Twins:
    """Two optimizers of the same tensors, one replayed and one stepped."""

    def __init__(self, dtype, master, bits, step=0, sizes=(1, 257, 5000, 40000)):
        import torch
        self.torch, self.gen = torch, torch.Generator(device="cuda").manual_seed(len(dtype) + bits)
        dt = getattr(torch, dtype)
        self.g = [torch.zeros(n, dtype=dt, device="cuda") for n in sizes]
        w = [torch.randn(n, generator=self.gen, device="cuda") for n in sizes]
        self.opts = []
        for _ in range(2):
            masters = [x.clone() for x in w] if master else None
            self.opts.append(sl.AdamW([x.to(dt).clone() for x in w], self.g, masters=masters, betas=(0.8, 0.95),
                                      state_bits=bits, seed=9, step=step))
        self.fresh()

    def fresh(self):
        for i, x in enumerate(self.g):
            x.copy_(self.torch.randn(x.shape, generator=self.gen, device="cuda") * 10.0 ** (i - 2))

    def same(self):
        a, b = self.opts
        assert a.step_count == b.step_count
        for name in ("params", "masters", "m", "v", "m_top", "v_top"):
            for x, y in zip(getattr(a, name) or [], getattr(b, name) or []):
                if x is not None:
                    assert self.torch.equal(x, y), name


def capture(torch, f):
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        f()
    return graph


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,master", [("float32", False), ("bfloat16", True), ("float16", False)])
@pytest.mark.parametrize("step", [0, 41])
def test_replays_are_steps_of_their_own(dtype, master, bits, step):
    """Replays, steps outside the graph and replays again, with fresh gradients
    and a gradient scale that changes on the device."""
    import torch
    t = Twins(dtype, master, bits, step)
    a, b = t.opts
    a.step(1e-2), b.step(1e-2)
    scale = torch.tensor([1.0], device="cuda")
    graph = capture(torch, lambda: a.step(1e-2, scale))
    t.same()                                  # a capture is no step
    for i in range(5):
        scale.fill_(0.5 + i)
        t.fresh()
        graph.replay()
        b.step(1e-2, scale)
        t.same()
    for lr in (2e-2, 0.0):
        t.fresh()
        a.step(lr), b.step(lr)
        t.same()
    for _ in range(3):
        t.fresh()
        graph.replay()
        b.step(1e-2, scale)
        t.same()
    assert a.step_count == step + 11


def test_several_steps_in_one_graph_and_a_count_that_is_set():
    import torch
    t = Twins("float32", False, 8)
    a, b = t.opts

    def three():
        for _ in range(3):
            a.step(1e-2)
    graph = capture(torch, three)
    for count in (None, 1000, 7):
        if count is not None:
            a.step_count = count
            b.step_count = count
        for _ in range(2):
            graph.replay()
            for _ in range(3):
                b.step(1e-2)
        t.same()
    assert a.step_count == b.step_count == 13


def test_a_capture_that_names_its_step_is_refused():
    import torch
    t = Twins("float32", False, 32)
    h = t.opts[0].handle
    got = []

    def named():
        stream = torch.cuda.current_stream().cuda_stream
        got.append(sl.lib().adamw_step(h, 1, 1e-2, 0.9, 0.99, 1e-8, None, 0, stream))
        got.append(sl.lib().adamw_step(h, 0, 1e-2, 0.9, 0.99, 1e-8, None, 0, stream))
    capture(torch, named)
    assert got == [2, 0] and sl.adamw_get_step(h) == 0
    assert sl.lib().adamw_step(h, -1, 1e-2, 0.9, 0.99, 1e-8, None, 0, None) == 1
    with pytest.raises(sl.EmbError):
        sl.adamw_set_step(h, -1)


def test_nothing_to_step():
    import torch
    p, g = [torch.empty(0, device="cuda")], [torch.empty(0, device="cuda")]
    opt = sl.AdamW(p, g)
    opt.step(0.1)
    assert opt.step_count == 1 == sl.adamw_get_step(opt.handle)
    capture(torch, lambda: opt.step(0.1)).replay()
    assert opt.step_count == 2
