"""What a recurrence's handle holds on the device is what the header says, and the
calls on both sides of the rule that it is sized by still fit it."""
import pytest

import sparse_lookup_gb300 as sl
from sparse_lookup_gb300 import build as slbuild

pytestmark = pytest.mark.gpu
MB = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def built():
    slbuild.build()
    sl.lib()


@pytest.mark.parametrize("dim,batch,length", [(512, 40, 1 << 18), (512, 1, 1 << 20), (33, 4, 1 << 20),
                                              (64, 1 << 20, 20000), (64, 1024, 1000)])
def test_memory_of_a_handle(dim, batch, length):
    """The header's formula, within the allocator's granularity of 2 MB for each
    of three allocations and what the first call of a kind may load."""
    import torch
    sl.GatedScan(dim, 1, 1).close()
    torch.cuda.synchronize()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    want = 16 * min(batch * dim, 77 * sms) * 9 / 8 * (length / (64 if dim % 2 else 128) + 1)
    before = torch.cuda.mem_get_info()[0]
    plan = sl.GatedScan(dim, batch, length)
    held = before - torch.cuda.mem_get_info()[0]
    plan.close()
    assert held <= want + 8 * MB, (held / MB, want / MB)


@pytest.mark.parametrize("dim,batch,length", [(32, b, 3000) for b in (181, 182, 183, 303, 304, 305, 363, 364, 365, 366)] +
                         [(33, 352, 1500), (30, 385, 1500)])
def test_calls_around_the_widest_chain(dim, batch, length):
    """Tiles across from under 3/5 of the places to over 6/5 (304 places on 152
    SMs): chained and walking calls agree with each entry alone."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(batch)
    x, g, gy = (torch.randn(batch, length, dim, generator=gen, device="cuda") for _ in range(3))
    plan, one = sl.GatedScan(dim, batch, length), sl.GatedScan(dim, 1, length)
    y, last = plan.forward(x, g)
    grads = plan.backward(x, g, y, gy)
    for b in (0, batch // 2, batch - 1):
        alone = [t[b:b + 1] for t in (x, g, gy)]
        yb, lb = one.forward(*alone[:2])
        for p, q in zip((y, last) + grads, (yb, lb) + one.backward(alone[0], alone[1], yb, alone[2])):
            assert torch.allclose(p[b], q[0], rtol=2e-5, atol=2e-5)
    assert plan.device_status() == 0
    plan.close()
    one.close()
