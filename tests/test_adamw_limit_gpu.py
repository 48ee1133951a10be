"""8-bit states beside one large element of their block, and the limit on updates
that bounds what they lose.  The case of emb.h: one gradient of +-1 among 255 of
1e-5, which then become 0."""
import numpy as np
import pytest

import sparse_lookup_gb300 as sl
from sparse_lookup_gb300 import build as slbuild
from test_adamw_gpu import SIZES, U, Model, check_states, host, make

pytestmark = pytest.mark.gpu
LIMIT = 0.1 / np.sqrt(0.001 * (1 - 0.81 / 0.999))   # 7.27


@pytest.fixture(scope="module", autouse=True)
def built():
    slbuild.build()
    sl.lib()


def moves(bits, limit):
    """The largest move of the small elements in units of lr: while their
    gradient is constant, and after it has become 0."""
    import torch
    p, g = [torch.zeros(256, device="cuda")], [torch.full((256,), 1e-5, device="cuda")]
    opt = sl.AdamW(p, g, weight_decay=0.0, state_bits=bits, seed=1, max_update=limit)
    most = [0.0, 0.0]
    for t in range(320):
        if t == 300:
            g[0].zero_()
        g[0][0] = 1.0 if t % 2 else -1.0
        p[0].zero_()
        opt.step(1.0)
        most[t >= 300] = max(most[t >= 300], p[0][1:].abs().max().item())
    return most


def test_the_documented_case():
    """32-bit states: |g| / (|g| + eps) = 1 / 1.001 of lr, and about 0.9 of it; the
    8-bit states' moves are the header's figures, whole numbers of a reproducible
    run, and the limit's with it."""
    a, b = moves(32, None)
    assert abs(a - 1 / 1.001) < 1e-4 and abs(b - 0.9) < 1e-2
    a, b = moves(8, None)
    assert round(a) in (16, 17) and 900 < b < 1000
    a, b = moves(8, LIMIT)
    assert a <= LIMIT * (1 + 4 * U) and b <= LIMIT * (1 + 4 * U)


@pytest.mark.parametrize("bits", [32, 8])
def test_the_limit_leaves_exact_updates_alone(bits):
    """Gradients of any sign and size: 32-bit moments never reach it, so the
    weights are the same bits; 8-bit ones follow the limited model."""
    import torch
    p, g = make(SIZES, "float32", "float32", 6)
    q = [x.clone() for x in p]
    a = sl.AdamW(p, g, state_bits=bits, seed=3, max_update=LIMIT)
    b = sl.AdamW(q, g, state_bits=bits, seed=3)
    for step in range(30):
        for i, x in enumerate(g):
            r = torch.randn(x.shape, generator=torch.Generator().manual_seed(step * 50 + i))
            x.copy_(r * torch.exp2((r * 1e4 % 20)) * (1 if step % 7 else 100))
        a.step(0.01), b.step(0.01)
        if bits == 32:
            assert all(torch.equal(x, y) for x, y in zip(p + a.m + a.v, q + b.m + b.v))
        else:
            assert all(torch.equal(x, y) for x, y in zip(a.m + a.v + a.m_top + a.v_top, b.m + b.v + b.m_top + b.v_top))


@pytest.mark.parametrize("dtype,master", [("float32", False), ("bfloat16", True)])
def test_updates_are_cut_at_the_limit(dtype, master):
    """A limit of 0.7 against the model's own updates: a sign step of 0.7 lr for
    the first, in which every update is 1 in magnitude; NaN stays; 0 and infinity
    take the limit away."""
    import torch
    p, g = make([1000, 300], dtype, dtype, 3)
    g = [torch.sign(x) * (x.abs() + 1) for x in g]
    g[0][5] = float("nan")
    masters = [x.float() for x in p] if master else None
    held = masters or p
    opt = sl.AdamW(p, g, masters=masters, weight_decay=0.0, max_update=0.7)
    for limit, want in ((None, 0.7), (0.0, 1.0), (0.25, 0.25), (float("inf"), 1.0)):
        if limit is not None:
            sl.adamw_set_max_update(opt.handle, limit)
        before = [x.double() for x in held]
        for x in opt.m + opt.v:
            x.zero_()
        opt.step_count = 0
        opt.step(0.5)
        for i, x in enumerate(held):
            moved = before[i] - x.double() - 0.5 * want * torch.sign(g[i].double())
            ok = moved.abs() <= 2 * U * before[i].abs() + 20 * U
            if i == 0:
                assert torch.isnan(x[5])
                ok[5] = True
                x[5] = 1.0
            assert ok.all()
    for bad in (-1.0, float("nan")):
        with pytest.raises(sl.EmbError):
            sl.AdamW([p[1]], [g[1]], max_update=bad)
