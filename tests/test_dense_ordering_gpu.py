"""What the dense operators' host calls leave on the device is there, and in
order, for the next call on any stream: torch's side streams do not wait for
the default stream."""

import threading
import time

import pytest

import sparse_lookup_gb300 as sl
from sparse_lookup_gb300 import build as slbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    slbuild.build()
    sl.lib()


def test_a_first_step_on_another_stream_finds_the_handle_complete():
    """Created while large copies to the device are under way, stepped at once
    on a side stream."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(4)
    p = [torch.randn(700 + i, generator=gen, device="cuda") for i in range(2000)]
    g = [torch.randn(700 + i, generator=gen, device="cuda") for i in range(2000)]
    want = [x.clone() for x in p]
    sl.AdamW(want, g).step(1e-2)
    copying, side = torch.cuda.Stream(), torch.cuda.Stream()
    host = torch.empty(64 << 20, dtype=torch.uint8).pin_memory()
    room = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    m, v = ([torch.zeros_like(x) for x in p] for _ in range(2))
    for _ in range(5):
        q = [x.clone() for x in p]
        for x in m + v:
            x.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(copying):
            for _ in range(4):
                room.copy_(host, non_blocking=True)
        opt = sl.AdamW(q, g, m=m, v=v)
        opt.step(1e-2, stream=side)
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(q, want))
        torch.cuda.synchronize()
        opt.close()


def test_reading_the_status_does_not_clear_a_later_error():
    """The status is read on a side stream while the default stream is busy: the
    clear belongs before the next call, whose error must stay."""
    import torch
    plan = sl.GatedScan(8, 2, 20)
    x = torch.randn(2, 20, 8, device="cuda")
    good, bad = (torch.tensor(o, dtype=torch.int32, device="cuda") for o in ([0, 20, 40], [0, 20, 5]))
    side = torch.cuda.Stream()
    y, last = plan.forward(x, x, good)
    torch.cuda.synchronize()
    ms = int(2e6)   # cycles, about a millisecond
    for _ in range(3):
        torch.cuda._sleep(60 * ms)                        # the default stream is busy ...
        busy = torch.cuda.Event()
        busy.record()
        more = threading.Thread(target=lambda: (time.sleep(0.02), torch.cuda._sleep(60 * ms)))
        more.start()                                      # ... and gets more while the status is read
        assert plan.device_status(stream=side) == 0
        assert not busy.query()                           # nothing of it went through the default stream
        plan.forward(x, x, bad, y=y, last=last, stream=side)
        more.join()
        torch.cuda.synchronize()
        assert plan.device_status(stream=side) == 7
    plan.close()


@pytest.mark.parametrize("n", [1, 3, 480, 481, 1500])
def test_bound_gradients_are_those_of_the_call(n):
    """The host's array of addresses is gone when the call returns; a captured
    call binds the same gradients in every replay."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(n)
    p = [torch.randn(5 + i % 7, generator=gen, device="cuda") for i in range(n)]
    sets = [[torch.randn(x.shape, generator=gen, device="cuda") for x in p] for _ in range(3)]
    q = [x.clone() for x in p]
    a, b = sl.AdamW(p, sets[0]), sl.AdamW(q, sets[0])

    def follow(grads):
        """b does what a did, with a handle's own first gradients."""
        for x, y in zip(sets[0], grads):
            x.copy_(y)
        b.step(1e-2)
        assert all(torch.equal(x, y) for x, y in zip(p + a.m + a.v, q + b.m + b.v))
    first = [x.clone() for x in sets[0]]
    a.bind_grads(sets[1])
    a.step(1e-2)
    follow(sets[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        a.bind_grads(sets[2])
    junk = [[k] * 2000 for k in range(200)]   # what was freed is used again
    for _ in range(3):
        a.bind_grads(sets[1])
        graph.replay()
        a.step(1e-2)
        follow(sets[2])
        a.bind_grads(sets[0])
        for x, y in zip(sets[0], first):
            x.copy_(y)
        a.step(1e-2)
        follow(first)
    assert len(junk) == 200
