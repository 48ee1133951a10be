"""CPU checks of the norm's, the gate's and the delta rule's entry points: bad
arguments are refused before any device work, and the tensor wrappers hand over
what belongs together.  No GPU compute."""
import ctypes

import pytest
import torch

import sparse_lookup_gb300 as sl
from sparse_lookup_gb300 import build as slbuild
from sparse_lookup_gb300 import dense
from test_dense_binding import Fake, refuse

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module", autouse=True)
def L():
    slbuild.build()
    return sl.lib()


def status(f, *args):
    with pytest.raises(sl.EmbError) as e:
        f(*args)
    return e.value.status


def test_norm_create(L):
    assert status(sl.norm_create, 0) == INVALID and status(sl.norm_create, 16385) == UNSUPPORTED
    assert L.norm_create(8, None) == INVALID and L.norm_destroy(None) == INVALID


@pytest.mark.parametrize("args,want", [((0, 1, 1, 1, 1, 1, 0), INVALID), ((1, 0, 1, 1, 1, 1, 0), INVALID),
                                       ((1, 1, 0, 1, 1, 1, 0), INVALID), ((1, 1, 1, 0, 1, 1, 0), INVALID),
                                       ((1, 1, 3, 2, 1, 1, 0), INVALID), ((1, 1, 1, 1, 0, 1, 0), INVALID),
                                       ((1, 1, 1, 1, 1, 0, 0), INVALID), ((129, 1, 1, 1, 1, 1, 0), UNSUPPORTED),
                                       ((1, 129, 1, 1, 1, 1, 0), UNSUPPORTED), ((1, 1, 65537, 1, 1, 1, 0), UNSUPPORTED),
                                       ((1, 1, 1, 1, 1, (1 << 30) + 1, 0), UNSUPPORTED),
                                       ((1, 1, 8, 1, 1 << 24, 1, 0), UNSUPPORTED),
                                       ((1, 1, 8, 1, 1 << 10, 1 << 23, 0), UNSUPPORTED)])
def test_delta_create(args, want):
    assert status(sl.delta_create, *args) == want


def test_null_handles(L):
    assert L.delta_create(1, 1, 1, 1, 1, 1, 0, None) == INVALID and L.delta_destroy(None) == INVALID
    assert L.delta_forward(None, 0, 0, 0, *[None] * 6, 1.0, *[None] * 4) == INVALID
    assert L.delta_backward(None, 0, 0, 0, *[None] * 6, 1.0, *[None] * 10) == INVALID
    assert L.norm_forward(None, 0, 0, 0, None, None, 0, None, None, 1e-5, None, None, None) == INVALID
    assert L.norm_backward(None, 0, 0, 0, None, None, 0, *[None] * 7) == INVALID
    assert L.moe_gate(None, 0, 0, None, 0, None, 0, *[None] * 7) == INVALID
    assert L.moe_gate_backward(None, 0, 0, None, 0, 0, *[None] * 8, 0, None) == INVALID


def test_delta_step_arguments(L):
    """Of plausible addresses (nothing is read) one argument at a time is bad."""
    def call(**kw):
        d = dict(n=2, N=8, V=16, H=4, J=2, dtype=0, q=(4096, 16, 0, 8), k=(8192, 16, 0, 8), v=(16384, 64, 0, 16),
                 decay=(32768, 4, 0, 1), beta=(65536, 4, 0, 1), scale=1.0, rows=4096, states=8192, num_rows=3,
                 y=(16384, 64, 0, 16))
        d.update(kw)
        views = [None if d[x] is None else ctypes.byref(sl.DeltaView(*d[x])) for x in ("q", "k", "v", "decay", "beta")]
        y = None if d["y"] is None else ctypes.byref(sl.DeltaView(*d["y"]))
        return L.delta_step(d["n"], d["N"], d["V"], d["H"], d["J"], d["dtype"], *views, d["scale"], d["rows"],
                            d["states"], d["num_rows"], y, None)
    for bad in (dict(n=-1), dict(N=0), dict(V=0), dict(H=0), dict(J=0), dict(J=3), dict(dtype=3), dict(q=None),
                dict(k=(8194, 16, 0, 8)), dict(v=(0, 64, 0, 16)), dict(decay=(32770, 4, 0, 1)), dict(beta=(65536, -1, 0, 1)),
                dict(scale=float("inf")), dict(scale=float("nan")), dict(rows=None), dict(rows=4100), dict(states=None),
                dict(states=8193), dict(num_rows=-1), dict(y=None), dict(y=(16384, 63, 0, 16)), dict(y=(16384, 64, 0, 15))):
        assert call(**bad) == INVALID, bad
    assert call(N=129) == UNSUPPORTED and call(V=129, v=(16384, 1024, 0, 129), y=(16384, 1024, 0, 129)) == UNSUPPORTED
    assert call(n=0, q=(0, 0, 0, 0), k=(0, 0, 0, 0), v=(0, 0, 0, 0), y=(0, 0, 0, 0), rows=None, states=None) == 0


@pytest.fixture
def fakes(monkeypatch):
    """Handles without a GPU: null, so that none is destroyed."""
    for name in ("delta_create", "moe_create", "norm_create"):
        monkeypatch.setattr(dense, name, lambda *a: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return monkeypatch


def elsewhere(f, args, **kw):
    """f with each of its tensors on another GPU in turn, and on none."""
    for at in list(range(len(args))) + list(kw):
        for device in (1, -1):
            given, named = [Fake(*a) for a in args], {k: Fake(*a) for k, a in kw.items()}
            (given if isinstance(at, int) else named)[at].__init__(*(args if isinstance(at, int) else kw)[at],
                                                                  device=device)
            with pytest.raises(ValueError):
                f(*given, **named, stream=7)


def test_every_tensor_of_a_call_lies_on_the_handles_device(fakes):
    f32, i32, i64 = torch.float32, torch.int32, torch.int64
    norm, scan, router = sl.LayerNorm(8), sl.DeltaScan(8, 16, 4, 2, 20, key_heads=2), sl.ExpertRouter(4, 2, 10)
    norm._fwd = norm._bwd = scan._fwd = scan._bwd = scan._step = router._gate = router._gate_backward = refuse
    seq, flat, two = ((2, 20, 8), f32), ((8,), f32), ((2, 20, 2), f32)
    elsewhere(norm.forward, [seq, flat, flat], offsets=((3,), i32), y=seq, stats=two)
    elsewhere(norm.backward, [seq, seq, two, flat], offsets=((3,), i32), grad_x=seq, grad_weight=flat, grad_bias=flat)
    key, value, each, end = ((2, 20, 2, 8), f32), ((2, 20, 4, 16), f32), ((2, 20, 4), f32), ((2, 4, 8, 16), f32)
    inputs = [key, key, value, each, each]
    elsewhere(scan.forward, inputs, offsets=((3,), i32), state=end, y=value, last=end)
    elsewhere(scan.backward, inputs + [value], offsets=((3,), i32), state=end, grad_last=end, grad_q=key, grad_k=key,
              grad_v=value, grad_decay=each, grad_beta=each, grad_state=end)
    elsewhere(scan.step, [((2, 2, 8), f32), ((2, 2, 8), f32), ((2, 4, 16), f32), ((2, 4), f32), ((2, 4), f32),
                          ((2,), i64), end], y=((2, 4, 16), f32))
    elsewhere(router.gate, [((5, 4), f32)], live=((5,), torch.bool))
    gate = dense.Gate(None, (0,) * 5, (5, 2, 4, 0), True)
    elsewhere(lambda x, gw, gl, to, stream: router.gate_backward(x, gate, gw, gl, to, stream),
              [((5, 4), f32), ((5, 2), f32), ((2,), f32), ((5, 4), f32)])
    with pytest.raises(ValueError):
        router.gate_backward(Fake((5, 4)), dense.Gate(None, (0,) * 5, (5, 2, 4, 1), True), stream=7)


def test_a_call_hands_over_views_and_sizes(fakes):
    scan, seen = sl.DeltaScan(8, 16, 4, 2, 20, key_heads=2, scale=0.5), []

    def entry(*a):
        views = [(ctypes.c_int64 * 4).from_address(x)[:] for x in (*a[4:9], a[12])]
        seen.append((a[1:4], views, a[9:12], a[13:]))
        return 0
    scan._fwd = entry
    key, value, each = (2, 20, 2, 8), (2, 20, 4, 16), (2, 20, 4)
    t = [Fake(s, at=4096 * (i + 1)) for i, s in enumerate((key, key, value, each, each, value))]
    scan.forward(*t[:5], y=t[5], last=Fake((2, 4, 8, 16), at=128), stream=7)
    steps = [[320, 16, 8]] * 2 + [[1280, 64, 16], [80, 4, 1], [80, 4, 1], [1280, 64, 16]]
    assert seen == [((2, 20, 0), [[4096 * (i + 1)] + x for i, x in enumerate(steps)], (None, 0.5, None), (128, 7))]
