"""What the dense operators' host calls leave on the device is there, and in
order, for the next call on any stream: torch's side streams do not wait for
the default stream."""

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
