"""Weight decay at small lr * weight_decay: the rate that is taken off is the one
that was asked for, not one rounded to a place of 1."""
import numpy as np
import pytest

import sparse_lookup_gb300 as sl
from sparse_lookup_gb300 import build as slbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    slbuild.build()
    sl.lib()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("lr,decay", [(1e-5, 0.01), (1e-6, 0.01), (1e-6, 1.0), (1e-4, 0.1)])
def test_the_rate_of_decay(lr, decay, master, bits):
    """Two runs of the same gradients, with decay and without: their weights differ
    by n lr decay |w| on average.  Weights lie in [1, 2), so half a place is 2^-24
    for all.  A step rounds each weight by at most that, with a mean of zero where
    its update is spread over places, as all are but the first (which is lr up or
    down for every weight): 2 2^-24 for the two first steps, and for the rest of n
    steps of N weights five standard deviations of 2^-24 sqrt(2 n / N) at most.
    1e-3 of the shift covers lr decay in fp32 (1.2e-7), the decay's own effect on
    later decay (n lr decay / 2 <= 2e-4) and the weights' drift."""
    import torch
    n, N = 40, 1 << 20
    gen = torch.Generator(device="cuda").manual_seed(3)
    w = 1 + torch.rand(N, generator=gen, device="cuda") * 0.99
    dt = torch.bfloat16 if master else torch.float32
    g = torch.empty(N, dtype=dt, device="cuda")
    runs = []
    for d in (decay, 0.0):
        held = w.clone()
        p = held.to(dt) if master else held
        opt = sl.AdamW([p], [g], masters=[held] if master else None, weight_decay=d, state_bits=bits, seed=1)
        runs.append((opt, held))
    for _ in range(n):
        g.copy_(torch.randn(N, generator=gen, device="cuda"))
        for opt, _ in runs:
            opt.step(lr)
    shift = (runs[1][1].double() - runs[0][1].double()).mean().item()
    want = n * lr * decay * w.double().mean().item()
    assert abs(shift - want) <= 2.0 ** -24 * (2 + 5 * np.sqrt(2 * n / N)) + 1e-3 * want
