"""The 16-bit backward of the recurrence takes the states before its positions
in fp32, whatever the length: x with a mean far from zero makes h_{t-1} - x_t
small beside h, so that a state rounded to 16 bits would show in the gate's
gradient.  The bounds are those of tests/test_scan_gpu.py without the term for
a stored state: fp32 throughout, and one rounding where a gradient is stored."""
import numpy as np
import pytest

import sparse_lookup_gb300 as sl
from sparse_lookup_gb300 import build as slbuild
from test_scan_gpu import backward64, close, f64, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    slbuild.build()
    sl.lib()


def run(B, T, D, dtype, lens=None, mean=16.0, views=None):
    import torch
    x, g, gy, h0, gl, lens, off = make(B, T, D, dtype, B + T + D, lens)
    x, h0 = x + mean, h0 + mean
    if views == "halves":
        both = torch.cat([x, g], 2)
        x, g = both[..., :D], both[..., D:]
    plan = sl.GatedScan(D, max_batch=B, max_len=T)
    y, _ = plan.forward(x, g, off, h0)
    out = {}
    if views == "halves":
        room = torch.full((B, T, 2 * D), float("nan"), dtype=x.dtype, device="cuda")
        out = dict(grad_x=room[..., :D], grad_gate=room[..., D:])
    gx, gg, gs = plan.backward(x, g, y, gy, off, h0, gl, **out)
    again = plan.backward(x, g, y, gy, off, h0, gl)
    for p, q in zip((gx, gg, gs), again):
        assert torch.equal(p, q)
    assert plan.device_status() == 0
    plan.close()
    rx, rg, rs, ex, eg, es = backward64(f64(x), f64(g), lens, f64(h0), f64(gy), f64(gl), 0.0)
    close(gx, rx, ex, dtype, "grad_x")
    close(gg, rg, eg, dtype, "grad_gate")
    close(gs, rs, es, "float32", "grad_state")


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("B,T,D", [(7, 8, 24), (7, 9, 24), (50, 16, 32), (40, 17, 24), (9, 128, 32), (9, 129, 32),
                                   (5, 130, 33), (700, 300, 32), (600, 257, 30), (700, 260, 15), (1, 9000, 64),
                                   (1, 5001, 30), (1, 5003, 33), (2, 700, 512)])
def test_states_are_fp32(B, T, D, dtype):
    run(B, T, D, dtype)


@pytest.mark.parametrize("D", [32, 30, 33])
def test_every_end_of_a_tile(D):
    """Lengths of one position more and less than whole tiles, walking and in
    a chain."""
    ends = [0, 1, 2, 15, 16, 17, 127, 128, 129, 159, 160, 161, 255, 256, 257, 319, 320, 321, 384, 385]
    run(len(ends), 385, D, "bfloat16", lens=ends)
    run(len(ends) * 30, 385, D, "bfloat16", lens=ends * 30)
    run(3, 2561, D, "bfloat16", lens=[2561, 2560, 0])


@pytest.mark.parametrize("B,T,D", [(3, 400, 32), (700, 300, 32), (1, 4000, 64), (2, 500, 33)])
def test_halves_of_one_projection(B, T, D):
    run(B, T, D, "bfloat16", views="halves")


def test_what_dead_positions_and_the_outputs_held_changes_nothing():
    import torch
    for B, T in ((8, 700), (500, 300)):
        x, g, gy, h0, gl, lens, off = make(B, T, 32, "bfloat16", T)
        plan = sl.GatedScan(32, B, T)
        y, _ = plan.forward(x, g, off, h0)
        want = plan.backward(x, g, y, gy, off, h0, gl)
        dead = torch.from_numpy(np.arange(T)[None, :] >= lens[:, None]).cuda()
        for fill in (float("nan"), float("inf")):
            for t in (x, g, gy):
                t[dead] = fill
            out = [torch.full_like(x, fill) for _ in range(2)]
            got = plan.backward(x, g, y, gy, off, h0, gl, grad_x=out[0], grad_gate=out[1])
            for p, q in zip(got, want):
                assert torch.equal(p, q)
        plan.close()


@pytest.mark.parametrize("B,T,D", [(1, 41000, 16), (1, 41120, 30), (1, 33000, 33), (2, 90000, 8), (1, 200000, 8),
                                   (1, 330000, 4)])
def test_more_tiles_than_one_cta_joins(B, T, D):
    """From 257 tiles on, clusters of two, four and eight CTAs, and more tiles than
    those read at once."""
    run(B, T, D, "bfloat16")


def test_a_walking_call_of_many_tiles():
    """Enough sequences to walk, long enough for a cluster; three of them against
    the formulas."""
    import torch
    B, T, D = 190, 33500, 32
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, g, gy = (torch.empty(B, T, D, device="cuda").normal_(m, s, generator=gen).to(torch.bfloat16)
                for m, s in ((16.0, 1.0), (1.0, 1.5), (0.0, 1.0)))
    h0, gl = (torch.randn(B, D, generator=gen, device="cuda") for _ in range(2))
    lens = torch.randint(0, T + 1, (B,), generator=gen, device="cuda")
    lens[0], lens[1] = T, 32769
    off = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).int()
    plan = sl.GatedScan(D, B, T)
    y, _ = plan.forward(x, g, off, h0)
    grads = plan.backward(x, g, y, gy, off, h0, gl)
    assert plan.device_status() == 0
    for b in (slice(0, 2), slice(B - 1, B)):
        rx, rg, rs, ex, eg, es = backward64(f64(x[b]), f64(g[b]), lens[b].cpu().numpy(), f64(h0[b]), f64(gy[b]),
                                            f64(gl[b]), 0.0)
        close(grads[0][b], rx, ex, "bfloat16", "grad_x")
        close(grads[1][b], rg, eg, "bfloat16", "grad_gate")
        close(grads[2][b], rs, es, "float32", "grad_state")
    plan.close()


def test_replayed_in_a_graph_and_on_another_stream():
    import torch
    B, T, D = 1, 41000, 32
    x, g, gy, h0, gl, lens, off = make(B, T, D, "bfloat16", 3)
    plan = sl.GatedScan(D, B, T)
    y, _ = plan.forward(x, g, off, h0)
    want = plan.backward(x, g, y, gy, off, h0, gl)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = plan.backward(x, g, y, gy, off, h0, gl, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    out = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        plan.backward(x, g, y, gy, off, h0, gl, grad_x=out[0], grad_gate=out[1], grad_state=out[2])
    for _ in range(3):
        for t in out:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want))
    assert plan.device_status() == 0
