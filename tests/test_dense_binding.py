"""CPU checks of the dense operators' tensor wrappers: what they hand to the C
entries and what they refuse, with stand-ins for tensors and entries.  No GPU
compute."""
import ctypes
import threading

import pytest
import torch

import sparse_lookup_gb300 as sl
from sparse_lookup_gb300 import build as slbuild
from sparse_lookup_gb300 import dense


class Fake:
    """What the wrappers ask of a tensor on a GPU; contiguous."""

    def __init__(self, shape, dtype=torch.float32, device=0, at=4096):
        self.shape, self.dtype, self.at = torch.Size(shape), dtype, at
        self.is_cuda, self.device = device >= 0, torch.device("cuda", device) if device >= 0 else torch.device("cpu")

    def get_device(self):
        return self.device.index if self.is_cuda else -1

    def is_contiguous(self):
        return True

    def stride(self, i=None):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s) if i is None else s[i]

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return self.at


@pytest.fixture
def fakes(monkeypatch):
    """Handles without a GPU: null, so that none is destroyed."""
    slbuild.build()
    for name in ("scan_create", "moe_create", "adamw_create"):
        monkeypatch.setattr(dense, name, lambda *a: None)
    monkeypatch.setattr(dense, "adamw_export_size", lambda h: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return monkeypatch


def views(*at):
    return [(ctypes.c_int64 * 3).from_address(a)[:] for a in at]


def test_a_call_hands_over_its_own_views(fakes):
    """Another thread's call on the same handle comes in between: the entries
    are called without the interpreter's lock."""
    plan = sl.GatedScan(8, 2, 20)
    seen = {}

    def call(base):
        t = [Fake((2, 20, 8), at=base + 512 * i) for i in range(6)]
        s = [Fake((2, 8), at=base + 8192 + 512 * i) for i in range(3)]
        plan.forward(t[0], t[1], y=t[2], last=s[0], stream=7)
        plan.backward(t[0], t[1], t[2], t[3], grad_x=t[4], grad_gate=t[5], grad_state=s[1], stream=7)

    def entry(which, places, last):
        def run(*args):
            if threading.current_thread() is threading.main_thread():
                other = threading.Thread(target=call, args=(1 << 20,))
                other.start()
                other.join()
            seen[which, args[last]] = views(*[args[i] for i in places])
            return 0
        return run
    plan._fwd = entry("forward", (4, 5, 8), 9)
    plan._bwd = entry("backward", (4, 5, 8, 9, 11, 12), 13)
    call(4096)
    for base in (4096, 1 << 20):
        want = [[base + 512 * i, 160, 8] for i in range(6)]
        assert seen["forward", base + 8192] == want[:3]
        assert seen["backward", base + 8192 + 512] == want


def refuse(*args):
    raise AssertionError("a launch on the wrong device")


def test_every_tensor_of_a_call_lies_on_the_handles_device(fakes):
    scan, router = sl.GatedScan(8, 2, 20), sl.ExpertRouter(4, 2, 10)
    scan._fwd = scan._bwd = scan._step = refuse
    router._route = router._dispatch = router._combine = router._combine_backward = refuse
    f32, i32, i64 = torch.float32, torch.int32, torch.int64
    seq, end = ((2, 20, 8), f32), ((2, 8), f32)

    def call(f, args, **kw):
        """f with each of its tensors on another GPU in turn, and on none."""
        for at in list(range(len(args))) + list(kw):
            for device in (1, -1):
                given = [Fake(*a) for a in args]
                named = {k: Fake(*a) for k, a in kw.items()}
                (given if isinstance(at, int) else named)[at].__init__(*(args if isinstance(at, int) else kw)[at],
                                                                      device=device)
                with pytest.raises(ValueError):
                    f(*given, **named, stream=7)
    call(scan.forward, [seq, seq], offsets=((3,), i32), state=end, y=seq, last=end)
    call(scan.backward, [seq, seq, seq, seq], offsets=((3,), i32), state=end, grad_last=end, grad_x=seq,
         grad_gate=seq, grad_state=end)
    call(scan.step, [end, end, ((2,), i64), ((9, 8), f32)], y=end)
    call(router.route, [((5, 2), i32)])
    R = router.rows(5)
    arrays = [((5,), i32), ((4,), i32), ((5, 2), i32), ((R,), i32)]
    routing = sl.Routing(*[Fake(*a) for a in arrays])
    call(lambda x, xs, stream: router.dispatch(x, routing, xs, stream), [((5, 16), f32)], xs=((R, 16), f32))
    call(lambda ys, w, y, stream: router.combine(ys, w, routing, y, stream), [((R, 16), f32), ((5, 2), f32)],
         y=((5, 16), f32))
    call(lambda gy, ys, w, a, b, stream: router.combine_backward(gy, ys, w, routing, a, b, stream),
         [((5, 16), f32), ((R, 16), f32), ((5, 2), f32)], a=((R, 16), f32), b=((5, 2), f32))
    for at in range(4):
        with pytest.raises(ValueError):
            sl.Routing(*[Fake(*a, device=1 if i == at else 0) for i, a in enumerate(arrays)])
    elsewhere = sl.Routing(*[Fake(*a, device=1) for a in arrays])
    with pytest.raises(ValueError):
        router.dispatch(Fake((5, 16)), elsewhere, Fake((R, 16)), stream=7)


def test_every_tensor_of_an_optimizer_lies_on_one_device(fakes):
    u8, i16, bf16 = torch.uint8, torch.int16, torch.bfloat16
    kinds = dict(params=((300,), bf16), grads=((300,), bf16), masters=((300,),), m=((300,), u8), v=((300,), u8),
                 m_top=((2,), i16), v_top=((2,), i16))
    for at in kinds:
        for device in (1, -1):
            with pytest.raises(ValueError):
                sl.AdamW(state_bits=8, **{k: [Fake(*a, device=device if k == at else 0)] for k, a in kinds.items()})
    opt = sl.AdamW(state_bits=8, **{k: [Fake(*a)] for k, a in kinds.items()})
    opt._step = refuse
    with pytest.raises(ValueError):
        opt.step(0.1, grad_scale=Fake((1,), device=1), stream=7)
    with pytest.raises(ValueError):
        opt.bind_grads([Fake((300,), bf16, device=1)], stream=7)


def test_the_current_device_and_the_stream_are_the_handles(fakes):
    plan = sl.GatedScan(8, 2, 20)
    plan._fwd = refuse
    t = [Fake((2, 20, 8)) for _ in range(3)]

    class Stream:
        device_index, cuda_stream = 1, 7
    with pytest.raises(ValueError):
        plan.forward(*t[:2], y=t[2], last=Fake((2, 8)), stream=Stream())
    plan._current = lambda: 1
    with pytest.raises(ValueError):
        plan.forward(*t[:2], y=t[2], last=Fake((2, 8)), stream=7)


def test_null_handles_of_the_count_and_the_limit():
    slbuild.build()
    L, n = sl.lib(), ctypes.c_int64()
    assert L.adamw_get_step(None, ctypes.byref(n), None) == 1
    assert L.adamw_set_step(None, 1, None) == 1
    assert L.adamw_set_max_update(None, 1.0) == 1
