"""CPU checks of the dense operators' C entry points: bad arguments are refused
before any device work, with the status the header states and nothing handed
out.  No GPU compute."""
import ctypes

import pytest

import sparse_lookup_gb300 as sl
from sparse_lookup_gb300 import build as slbuild
from sparse_lookup_gb300.dense import AdamwTensor

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module", autouse=True)
def L():
    slbuild.build()
    return sl.lib()


def status(f, *args):
    with pytest.raises(sl.EmbError) as e:
        f(*args)
    return e.value.status


@pytest.mark.parametrize("args,want", [((0, 1, 1), INVALID), ((4, 0, 1), INVALID), ((4, 1, 0), INVALID),
                                       ((65537, 1, 1), UNSUPPORTED), ((4, 1, (1 << 30) + 1), UNSUPPORTED)])
def test_scan_create(args, want):
    assert status(sl.scan_create, *args) == want


@pytest.mark.parametrize("args,want", [((0, 1, 1, 1), INVALID), ((1, 0, 1, 1), INVALID), ((1, 1, 0, 1), INVALID),
                                       ((1, 1, 1, 0), INVALID), ((2049, 1, 1, 1), UNSUPPORTED),
                                       ((1, 65, 1, 1), UNSUPPORTED), ((1, 1, 1, 65537), UNSUPPORTED),
                                       ((1, 1, 1 << 31, 1), UNSUPPORTED), ((2048, 1, (1 << 31) - 2048, 1), UNSUPPORTED)])
def test_moe_create(args, want):
    assert status(sl.moe_create, *args) == want


def tensor(**kw):
    """A tensor with plausible addresses (nothing is read)."""
    d = dict(param=4096, grad=8192, master=None, m=16384, v=32768, m_top=None, v_top=None, numel=10, weight_decay=0.0,
             dtype=0, grad_dtype=0, reserved=0)
    d.update(kw)
    return AdamwTensor(*[d[k] for k, _ in AdamwTensor._fields_])


@pytest.mark.parametrize("kw,flags", [
    (dict(param=None), 0), (dict(grad=None), 0), (dict(m=None), 0), (dict(v=None), 0), (dict(numel=-1), 0),
    (dict(param=4097), 0), (dict(grad=8194), 0), (dict(m=16386), 0), (dict(weight_decay=-1.0), 0),
    (dict(weight_decay=float("nan")), 0), (dict(weight_decay=float("inf")), 0), (dict(dtype=3), 0),
    (dict(dtype=7), 0), (dict(grad_dtype=1), 0), (dict(dtype=1, grad_dtype=2), 0), (dict(reserved=1), 0),
    (dict(master=1024), 0), (dict(), 2), (dict(), 1), (dict(m_top=64, v_top=None), 1), (dict(m_top=65, v_top=66), 1)])
def test_adamw_create(kw, flags):
    assert status(sl.adamw_create, [tensor(**kw)], flags) == INVALID


def test_adamw_create_counts():
    assert status(sl.adamw_create, [], 0) == INVALID
    assert status(sl.adamw_create, [tensor(numel=1 << 40)], 0) == UNSUPPORTED


def test_null_handles(L):
    z = ctypes.c_int64()
    for call in (lambda: L.scan_destroy(None), lambda: L.moe_destroy(None), lambda: L.adamw_destroy(None),
                 lambda: L.scan_get_device_status(None, None), lambda: L.adamw_export_size(None, ctypes.byref(z)),
                 lambda: L.adamw_step(None, 1, 0.1, 0.9, 0.999, 1e-8, None, 0, None),
                 lambda: L.adamw_bind_grads(None, None, None), lambda: L.adamw_export_states(None, None, None, None),
                 lambda: L.moe_route(None, 0, None, None, None, None, None, None),
                 lambda: L.moe_dispatch(None, 0, 1, 0, None, 0, None, None, None, None),
                 lambda: L.moe_combine(None, 0, 1, 0, None, None, None, None, 0, None),
                 lambda: L.moe_combine_backward(None, 0, 1, 0, None, 0, None, None, None, None, None, None, None),
                 lambda: L.scan_forward(None, 0, 0, 0, None, None, None, None, None, None, None),
                 lambda: L.scan_backward(None, 0, 0, 0, *[None] * 11),
                 lambda: L.scan_create(1, 1, 1, None), lambda: L.moe_create(1, 1, 1, 1, None),
                 lambda: L.adamw_create(None, 1, 0, None), lambda: L.scan_selftest_timeout(None, None, None)):
        assert call() == INVALID


def test_scan_step_arguments(L):
    ok = [1, 8, 0, 4096, 8, 8192, 8, 16384, 32768, 4, 65536, 8, None]
    for at, bad in ((0, -1), (1, 0), (2, 3), (3, None), (3, 4098), (4, -8), (5, None), (6, -1), (7, None), (7, 16388),
                    (8, None), (8, 32770), (9, -1), (10, None), (10, 65538)):
        args = list(ok)
        args[at] = bad
        assert L.scan_step(*args) == INVALID, at
    assert L.scan_step(*[2 if i == 0 else 7 if i == 11 else v for i, v in enumerate(ok)]) == INVALID   # rows overlap
    assert L.scan_step(*[65537 if i == 1 else v for i, v in enumerate(ok)]) == UNSUPPORTED
    assert L.scan_step(0, 8, 0, *[None if i in (0, 2, 4, 5, 7) else 8 for i in range(10)]) == 0        # nothing to do
