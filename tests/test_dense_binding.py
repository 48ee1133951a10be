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
