"""AdamW with eps below 1e-12, which takes the square root and quotient that do
not flush small numbers, and on both sides of that limit.  Bounds and model as
in tests/test_adamw_gpu.py; second moments stay in fp32's normal range or are
0, so that v / (1 - beta2^t) is a normal number in the kernel too."""
import numpy as np
import pytest

import sparse_lookup_gb300 as sl
from sparse_lookup_gb300 import build as slbuild
from test_adamw_gpu import SIZES, Model, check_states, host, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    slbuild.build()
    sl.lib()


@pytest.mark.parametrize("eps", [0.0, 1e-35, 1e-20, 9.9e-13, 1e-12, 1e-3])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("size", [1.0, 1e-12, 1e12])
def test_steps(eps, bits, size):
    """Gradients from the sizes' powers of ten times `size`, never 0; with
    eps > 0 also some whose squares are 0 in fp32."""
    import torch
    p, g = make(SIZES, "float32", "float32", 6)
    decay = [0.1 * (i % 3) for i in range(len(p))]
    opt = sl.AdamW(p, g, weight_decay=decay, betas=(0.9, 0.99), eps=eps, state_bits=bits, seed=77)
    model = Model(host(p), bits, decay, 0.9, 0.99, eps, 77)
    for step in range(3):
        for i, x in enumerate(g):
            r = torch.randn(x.shape, generator=torch.Generator().manual_seed(step * 50 + i))
            x.copy_(torch.sign(r) * (r.abs() + 0.1) * 10.0 ** (i % 5 - 3) * size)
            if eps > 0 and i % 2:
                x[::3] = 1e-28
        model.w = [x.astype(np.float64) for x in host(p)]
        want = model.step(host(g), 0.01)
        opt.step(0.01)
        check_states(opt, model)
        for i, (ref, bound) in enumerate(want):
            assert np.all(np.abs(host(p)[i] - ref) <= bound), (step, i)


def test_no_gradient_and_no_eps():
    """0 / 0 is what the formula says: such weights become NaN and the others are
    untouched by it; a state whose eps keeps the quotient finite stays."""
    import torch
    for eps, nan in ((0.0, True), (1e-30, False)):
        p, g = [torch.ones(600, device="cuda")], [torch.ones(600, device="cuda")]
        g[0][::7] = 0
        opt = sl.AdamW(p, g, weight_decay=0.0, eps=eps)
        opt.step(0.5)
        off = g[0] == 0
        assert torch.isnan(p[0][off]).all() if nan else (p[0][off] == 1).all()
        assert ((p[0][~off] - 0.5).abs() <= 2.0 ** -20).all()
