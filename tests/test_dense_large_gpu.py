"""Dense operators where element offsets pass 32 bits: the results are those of
the same rows close together."""
import pytest

import sparse_lookup_gb300 as sl

pytestmark = pytest.mark.gpu
FAR = 1 << 31


@pytest.fixture(scope="module", autouse=True)
def built():
    from sparse_lookup_gb300 import build
    build.build()
    yield
    import torch
    torch.cuda.empty_cache()


def far(shape, strides, like=None):
    """A bf16 view of these strides in a buffer of its own."""
    import torch
    last = sum((n - 1) * s for n, s in zip(shape, strides))
    t = torch.empty(last + 1, dtype=torch.bfloat16, device="cuda").as_strided(shape, strides)
    if like is not None:
        t.copy_(like)
    return t


@pytest.mark.parametrize("shape,strides", [((2, 700, 64), (FAR, 64, 1)), ((2, 700, 33), (FAR, 33, 1)),
                                           ((1, 9, 64), (64, FAR // 8, 1)), ((1, 5, 30), (30, FAR // 4, 1))])
def test_scan_views_past_32_bits(shape, strides):
    import torch
    gen = torch.Generator().manual_seed(shape[1])
    x, g, gy = (torch.randn(shape, generator=gen).to(torch.bfloat16).cuda() for _ in range(3))
    plan = sl.GatedScan(shape[2], max_batch=shape[0], max_len=shape[1])
    y, last = plan.forward(x, g)
    gx, gg, gs = plan.backward(x, g, y, gy)
    fx, fg, fgy, fy = far(shape, strides, x), far(shape, strides, g), far(shape, strides, gy), far(shape, strides)
    y2, last2 = plan.forward(fx, fg, y=fy)
    gx2, gg2, gs2 = plan.backward(fx, fg, fy, fgy, grad_x=far(shape, strides), grad_gate=far(shape, strides))
    for p, q in ((y, y2), (last, last2), (gx, gx2), (gg, gg2), (gs, gs2)):
        assert torch.equal(p, q)
    assert plan.device_status() == 0
    plan.close()


def test_rows_past_32_bits():
    import torch
    n, dim = FAR // 2048 + 777, 2048
    gen = torch.Generator("cuda").manual_seed(1)
    router = sl.ExpertRouter(5, 1, n)
    experts = torch.randint(0, 5, (n, 1), generator=gen, device="cuda", dtype=torch.int32)
    r = router.route(experts)
    line = torch.randn(dim, generator=gen, device="cuda")
    x = (line * (torch.arange(n, device="cuda") % 251)[:, None].to(torch.bfloat16)).to(torch.bfloat16)
    xs = router.dispatch(x, r)
    w = torch.rand(n, 1, generator=gen, device="cuda")
    y = router.combine(xs, w, r)
    gys, gw = router.combine_backward(x, xs, w, r)
    tokens = torch.cat([torch.arange(500), torch.arange(n - 500, n), r.src[-500:].cpu()]).cuda()
    rows = r.pos[tokens, 0].long()
    assert rows.max() * dim > FAR
    assert torch.equal(xs[rows], x[tokens])
    want = (x[tokens].float() * w[tokens]).to(torch.bfloat16)
    assert torch.equal(y[tokens], want) and torch.equal(gys[rows], want)
    square = x[tokens].double().square().sum(1)
    assert ((gw[tokens, 0].double() - square).abs() <= dim * 2.0 ** -24 * square).all()
    router.close()


def test_a_tensor_past_32_bits():
    import torch
    n, tail = FAR + 1000, 1000 + 256 * 3
    gen = torch.Generator("cuda").manual_seed(2)
    p, g = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    p[-tail:] = torch.randn(tail, generator=gen, device="cuda").to(torch.bfloat16)
    g[-tail:] = torch.randn(tail, generator=gen, device="cuda").to(torch.bfloat16)
    q, gq = p[-tail:].clone(), g[-tail:].clone()
    big, small = (sl.AdamW([t], [h], state_bits=8) for t, h in ((p, g), (q, gq)))
    big.step(1e-2)
    small.step(1e-2)
    assert torch.equal(p[-tail:], q)          # a step moves by the moments before they are rounded
    assert torch.equal(big.m_top[0][-7:], small.m_top[0]) and torch.equal(big.v_top[0][-7:], small.v_top[0])
    assert not p[:-tail].any()
    for a, b in zip(big.states(), small.states()):
        a, b = a[-7 * 256:].float(), b.float()
        assert ((a - b).abs() <= b.abs() * 2.0 ** -3 + (a.abs().max() * 2.0 ** -15)).all()   # a place apart at most
    big.close()
    small.close()
