"""Operators of the dense layers behind the lookups (scan_*, delta_*, moe_*,
norm_* and adamw_* of include/emb.h): raw C names, then GatedScan, DeltaScan,
ExpertRouter, LayerNorm and AdamW over PyTorch tensors.  Marshalling only, like the rest of the binding; arguments
that the library cannot see (shapes, element types, devices) are checked here
and raise ValueError: every tensor of a call, its stream and the current device
are those of the handle, which is the device that was current when it was made.

An output that a call allocates belongs to the stream the call runs on.
Tensors that come from another stream are the caller's to order (an event, or
record_stream), as everywhere in this package.
"""
from __future__ import annotations

import ctypes
from ctypes import c_float, c_int32, c_int64, c_void_p

from . import TABLE_DTYPE, _check, lib, ptr

STATES_8BIT = 1
UNSUPPORTED = 2      # EMB_ERR_UNSUPPORTED
BLOCK = 256          # elements that share a top in an 8-bit state
_ELEMENT = {k: v for k, v in TABLE_DTYPE.items() if k != "int8"}
_dtype_codes = {}    # torch dtype -> emb_table_dtype


class ScanView(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("batch_stride", c_int64), ("time_stride", c_int64)]


class DeltaView(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("batch_stride", c_int64), ("time_stride", c_int64), ("head_stride", c_int64)]


_Views = c_int64 * 18   # a call's scan_views, one after the other: each call has its own


class AdamwTensor(ctypes.Structure):
    _fields_ = [("param", c_void_p), ("grad", c_void_p), ("master", c_void_p), ("m", c_void_p), ("v", c_void_p),
                ("m_top", c_void_p), ("v_top", c_void_p), ("numel", c_int64), ("weight_decay", c_float),
                ("dtype", c_int32), ("grad_dtype", c_int32), ("reserved", c_int32)]


# ---------------------------------------------------------------------------
# raw C names
# ---------------------------------------------------------------------------

_current_stream = None


def _stream(stream, device=None):
    """The raw handle of a stream; None: the current stream of the device (the
    short way to it: a call may be a few microseconds of work)."""
    global _current_stream
    if stream is None:
        if _current_stream is None:
            import torch
            _current_stream = torch._C._cuda_getCurrentRawStream
        if device is None:
            import torch
            device = torch.cuda.current_device()
        return _current_stream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _ref(view):
    return None if view is None else ctypes.byref(view)


def scan_create(dim, max_batch, max_len):
    h = c_void_p()
    _check(lib().scan_create(dim, max_batch, max_len, ctypes.byref(h)), "scan_create")
    return h.value


def scan_forward(h, batch, length, dtype, x, gate, offsets, state_in, y, state_out, stream=None):
    _check(lib().scan_forward(h, batch, length, dtype, _ref(x), _ref(gate), ptr(offsets), ptr(state_in), _ref(y),
                              ptr(state_out), _stream(stream)), "scan_forward")


def scan_backward(h, batch, length, dtype, x, gate, offsets, state_in, y, grad_y, grad_state_out, grad_x, grad_gate,
                  grad_state_in, stream=None):
    _check(lib().scan_backward(h, batch, length, dtype, _ref(x), _ref(gate), ptr(offsets), ptr(state_in), _ref(y),
                               _ref(grad_y), ptr(grad_state_out), _ref(grad_x), _ref(grad_gate), ptr(grad_state_in),
                               _stream(stream)), "scan_backward")


def scan_step(n, dim, dtype, x, x_stride, gate, gate_stride, rows, states, num_rows, y, y_stride, stream=None):
    _check(lib().scan_step(n, dim, dtype, ptr(x), x_stride, ptr(gate), gate_stride, ptr(rows), ptr(states), num_rows,
                           ptr(y), y_stride, _stream(stream)), "scan_step")


def scan_get_device_status(h, stream=None):
    return int(lib().scan_get_device_status(h, _stream(stream)))


def scan_selftest_timeout():
    """Runs the chain's bounded-wait self test; returns dict(status, latched,
    latched_after, wait_ms)."""
    latched, after, ms = ctypes.c_uint32(0), ctypes.c_uint32(0), c_float(0.0)
    st = lib().scan_selftest_timeout(ctypes.byref(latched), ctypes.byref(after), ctypes.byref(ms))
    return dict(status=int(st), latched=latched.value, latched_after=after.value, wait_ms=ms.value)


def scan_destroy(h):
    _check(lib().scan_destroy(h), "scan_destroy")


def moe_create(n_experts, top_k, max_tokens, align):
    h = c_void_p()
    _check(lib().moe_create(n_experts, top_k, max_tokens, align, ctypes.byref(h)), "moe_create")
    return h.value


def moe_route(h, n, experts, offsets, counts, pos, src, stream=None):
    _check(lib().moe_route(h, n, ptr(experts), ptr(offsets), ptr(counts), ptr(pos), ptr(src), _stream(stream)),
           "moe_route")


def moe_dispatch(h, n, dim, dtype, x, x_stride, pos, src, xs, stream=None):
    _check(lib().moe_dispatch(h, n, dim, dtype, ptr(x), x_stride, ptr(pos), ptr(src), ptr(xs), _stream(stream)),
           "moe_dispatch")


def moe_combine(h, n, dim, dtype, ys, weights, pos, y, y_stride, stream=None):
    _check(lib().moe_combine(h, n, dim, dtype, ptr(ys), ptr(weights), ptr(pos), ptr(y), y_stride, _stream(stream)),
           "moe_combine")


def moe_combine_backward(h, n, dim, dtype, grad_y, grad_y_stride, ys, weights, pos, src, grad_ys, grad_weights,
                         stream=None):
    _check(lib().moe_combine_backward(h, n, dim, dtype, ptr(grad_y), grad_y_stride, ptr(ys), ptr(weights), ptr(pos),
                                      ptr(src), ptr(grad_ys), ptr(grad_weights), _stream(stream)),
           "moe_combine_backward")


def moe_gate(h, n, dtype, logits, logits_stride, live, normalize, experts, weights, counts, losses, stats, live_count,
             stream=None):
    _check(lib().moe_gate(h, n, dtype, ptr(logits), logits_stride, ptr(live), normalize, ptr(experts), ptr(weights),
                          ptr(counts), ptr(losses), ptr(stats), ptr(live_count), _stream(stream)), "moe_gate")


def moe_gate_backward(h, n, dtype, logits, logits_stride, normalize, experts, weights, counts, stats, live_count,
                      grad_weights, grad_losses, grad_logits, grad_stride, stream=None):
    _check(lib().moe_gate_backward(h, n, dtype, ptr(logits), logits_stride, normalize, ptr(experts), ptr(weights),
                                   ptr(counts), ptr(stats), ptr(live_count), ptr(grad_weights), ptr(grad_losses),
                                   ptr(grad_logits), grad_stride, _stream(stream)), "moe_gate_backward")


def moe_destroy(h):
    _check(lib().moe_destroy(h), "moe_destroy")


def delta_create(key_dim, value_dim, heads, key_heads, max_batch, max_len, training):
    h = c_void_p()
    _check(lib().delta_create(key_dim, value_dim, heads, key_heads, max_batch, max_len, training, ctypes.byref(h)),
           "delta_create")
    return h.value


def delta_forward(h, batch, length, dtype, q, k, v, decay, beta, offsets, scale, state_in, y, state_out, stream=None):
    _check(lib().delta_forward(h, batch, length, dtype, _ref(q), _ref(k), _ref(v), _ref(decay), _ref(beta),
                               ptr(offsets), scale, ptr(state_in), _ref(y), ptr(state_out), _stream(stream)),
           "delta_forward")


def delta_backward(h, batch, length, dtype, q, k, v, decay, beta, offsets, scale, state_in, grad_y, grad_state_out,
                   grad_q, grad_k, grad_v, grad_decay, grad_beta, grad_state_in, stream=None):
    _check(lib().delta_backward(h, batch, length, dtype, _ref(q), _ref(k), _ref(v), _ref(decay), _ref(beta),
                                ptr(offsets), scale, ptr(state_in), _ref(grad_y), ptr(grad_state_out), _ref(grad_q),
                                _ref(grad_k), _ref(grad_v), _ref(grad_decay), _ref(grad_beta), ptr(grad_state_in),
                                _stream(stream)), "delta_backward")


def delta_step(n, key_dim, value_dim, heads, key_heads, dtype, q, k, v, decay, beta, scale, rows, states, num_rows, y,
               stream=None):
    _check(lib().delta_step(n, key_dim, value_dim, heads, key_heads, dtype, _ref(q), _ref(k), _ref(v), _ref(decay),
                            _ref(beta), scale, ptr(rows), ptr(states), num_rows, _ref(y), _stream(stream)),
           "delta_step")


def delta_destroy(h):
    _check(lib().delta_destroy(h), "delta_destroy")


def norm_create(dim):
    h = c_void_p()
    _check(lib().norm_create(dim, ctypes.byref(h)), "norm_create")
    return h.value


def norm_forward(h, batch, length, dtype, x, offsets, weight_dtype, weight, bias, eps, y, stats, stream=None):
    _check(lib().norm_forward(h, batch, length, dtype, _ref(x), ptr(offsets), weight_dtype, ptr(weight), ptr(bias),
                              eps, _ref(y), ptr(stats), _stream(stream)), "norm_forward")


def norm_backward(h, batch, length, dtype, x, offsets, weight_dtype, weight, grad_y, stats, grad_x, grad_weight,
                  grad_bias, stream=None):
    _check(lib().norm_backward(h, batch, length, dtype, _ref(x), ptr(offsets), weight_dtype, ptr(weight),
                               _ref(grad_y), ptr(stats), _ref(grad_x), ptr(grad_weight), ptr(grad_bias),
                               _stream(stream)), "norm_backward")


def norm_destroy(h):
    _check(lib().norm_destroy(h), "norm_destroy")


def adamw_create(tensors, flags):
    """tensors: AdamwTensor structures, or a numpy array of their type."""
    arr = tensors if hasattr(tensors, "ctypes") else (AdamwTensor * max(1, len(tensors)))(*tensors)
    h = c_void_p()
    at = ptr(arr) if hasattr(arr, "ctypes") else arr
    _check(lib().adamw_create(at, len(tensors), flags, ctypes.byref(h)), "adamw_create")
    return h.value


def adamw_bind_grads(h, grads, stream=None):
    arr = (c_void_p * max(1, len(grads)))(*[ptr(g) for g in grads])
    _check(lib().adamw_bind_grads(h, arr, _stream(stream)), "adamw_bind_grads")


def adamw_step(h, step, lr, beta1, beta2, eps, grad_scale, seed, stream=None):
    _check(lib().adamw_step(h, step, lr, beta1, beta2, eps, ptr(grad_scale), seed, _stream(stream)), "adamw_step")


def adamw_set_max_update(h, limit):
    _check(lib().adamw_set_max_update(h, limit), "adamw_set_max_update")


def adamw_get_step(h, stream=None):
    n = c_int64()
    _check(lib().adamw_get_step(h, ctypes.byref(n), _stream(stream)), "adamw_get_step")
    return n.value


def adamw_set_step(h, step, stream=None):
    _check(lib().adamw_set_step(h, step, _stream(stream)), "adamw_set_step")


def adamw_export_states(h, m_out, v_out, stream=None):
    _check(lib().adamw_export_states(h, ptr(m_out), ptr(v_out), _stream(stream)), "adamw_export_states")


def adamw_export_size(h):
    n = c_int64()
    _check(lib().adamw_export_size(h, ctypes.byref(n)), "adamw_export_size")
    return n.value


def adamw_destroy(h):
    _check(lib().adamw_destroy(h), "adamw_destroy")


# ---------------------------------------------------------------------------
# tensor-level wrappers
# ---------------------------------------------------------------------------

def _element(dtype):
    code = _dtype_codes.get(dtype)
    if code is None:
        code = _ELEMENT.get(str(dtype).replace("torch.", ""))
        if code is None:
            raise ValueError("element type %s: float32, bfloat16 or float16" % dtype)
        _dtype_codes[dtype] = code
    return code


def _want(t, name, shape, dtype, device, dense=True):
    """Checks one tensor argument -- on this GPU, of this shape and type, dense
    (or only its last axis contiguous) -- and returns its pointer."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        raise ValueError("%s: %s %s on cuda:%d expected, got %s %s on %s" % (
            name, tuple(shape), dtype, device, tuple(t.shape), t.dtype, t.device))
    if not t.is_contiguous():
        if dense:
            raise ValueError("%s: a contiguous tensor expected, got strides %s" % (name, t.stride()))
        if t.stride(-1) != 1 and t.shape[-1] > 1 and t.numel():
            raise ValueError("%s: a contiguous last axis expected, got strides %s" % (name, t.stride()))
    return t.data_ptr()


class _Handle:
    handle = None

    def __init__(self):
        import torch
        self._t, self._f32, self._i32, self._new = torch, torch.float32, torch.int32, torch.empty
        self._current = torch._C._cuda_getDevice

    def _made(self, handle):
        """The handle belongs to the device that is current now."""
        self.handle, self._device = handle, self._current()

    def _want(self, t, name, shape, dtype, dense=True):
        return _want(t, name, shape, dtype, self._device, dense)

    def _at(self, stream):
        """The raw stream of a call (None: the current one)."""
        device = self._device
        if self._current() != device:
            raise ValueError("a handle of cuda:%d, but cuda:%d is the current device" % (device, self._current()))
        if stream is None or isinstance(stream, int):
            return _stream(stream, device)
        if stream.device_index != device:
            raise ValueError("a handle of cuda:%d, but a stream of cuda:%d" % (device, stream.device_index))
        return stream.cuda_stream

    def close(self):
        if self.handle:
            h, self.handle = self.handle, None
            self._destroy(h)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _empty(self, shape, dtype, like, stream):
        """A tensor beside `like` that belongs to the stream the kernel will
        run on."""
        if stream is None:
            return self._new(shape, dtype=dtype, device=like.device)
        torch = self._t
        s = torch.cuda.ExternalStream(stream, device=like.device) if isinstance(stream, int) else stream
        with torch.cuda.stream(s):
            return torch.empty(shape, dtype=dtype, device=like.device)


class GatedScan(_Handle):
    """A gated linear recurrence over [batch, time, dim] sequences:

        a = sigmoid(gate);  h_t = a_t h_{t-1} + (1 - a_t) x_t

    forward and backward over whole sequences (float32, bfloat16 or float16,
    any strides with a contiguous last axis, states in float32), and one step
    for serving on state rows of a pool.  ``offsets`` is [batch + 1] int32, the
    bags' offsets as Plan.forward takes them: entry b has offsets[b+1] -
    offsets[b] live positions, at most time; past them y and the gradients
    are 0.  None: all positions are live."""

    _destroy = staticmethod(scan_destroy)

    def __init__(self, dim, max_batch, max_len):
        super().__init__()
        self.dim = dim
        self._made(scan_create(dim, max_batch, max_len))
        L = lib()
        self._fwd, self._bwd, self._step = L.scan_forward, L.scan_backward, L.scan_step

    def _view(self, t, name, shape, dtype):
        """(pointer, batch stride, time stride) of a [batch, time, dim] tensor."""
        p = self._want(t, name, shape, dtype, False)
        if t.is_contiguous():
            return p, shape[1] * shape[2], shape[2]
        sb, st, _ = t.stride()
        return p, sb, st

    def _common(self, x, gate, offsets, state):
        shape, dt = x.shape, x.dtype
        if len(shape) != 3 or shape[2] != self.dim:
            raise ValueError("x: [batch, time, %d] expected, got %s" % (self.dim, tuple(shape)))
        code = _dtype_codes.get(dt)
        if code is None:
            code = _element(dt)
        B = shape[0]
        return (code, dt, shape,
                None if offsets is None else self._want(offsets, "offsets", (B + 1,), self._i32),
                None if state is None else self._want(state, "state", (B, self.dim), self._f32),
                self._view(x, "x", shape, dt) + self._view(gate, "gate", shape, dt))

    def forward(self, x, gate, offsets=None, state=None, y=None, last=None, stream=None):
        """(y, last): h_t at every position, and the state [batch, dim]
        float32 after the last live one.  state: the one before the first
        (None = 0).  y and last may be given."""
        code, dt, shape, o, s, views = self._common(x, gate, offsets, state)
        ends = (shape[0], shape[2])
        if y is None:
            y = self._empty(shape, dt, x, stream)
        if last is None:
            last = self._empty(ends, self._f32, x, stream)
        held = _Views(*views, *self._view(y, "y", shape, dt))
        v = ctypes.addressof(held)
        st = self._fwd(self.handle, shape[0], shape[1], code, v, v + 24, o, s, v + 48,
                       self._want(last, "last", ends, self._f32), self._at(stream))
        if st:
            _check(st, "scan_forward")
        return y, last

    def backward(self, x, gate, y, grad_y, offsets=None, state=None, grad_last=None, grad_x=None, grad_gate=None,
                 grad_state=None, stream=None):
        """(grad_x, grad_gate, grad_state) from the gradients of y and (None =
        0) of last; x, gate, offsets and state as in forward, y as it gave
        it.  The results may be given."""
        code, dt, shape, o, s, views = self._common(x, gate, offsets, state)
        f32, ends = self._f32, (shape[0], shape[2])
        gl = None if grad_last is None else self._want(grad_last, "grad_last", ends, f32)
        if grad_x is None:
            grad_x = self._empty(shape, dt, x, stream)
        if grad_gate is None:
            grad_gate = self._empty(shape, dt, x, stream)
        if grad_state is None:
            grad_state = self._empty(ends, f32, x, stream)
        held = _Views(*views, *self._view(y, "y", shape, dt), *self._view(grad_y, "grad_y", shape, dt),
                      *self._view(grad_x, "grad_x", shape, dt), *self._view(grad_gate, "grad_gate", shape, dt))
        v = ctypes.addressof(held)
        st = self._bwd(self.handle, shape[0], shape[1], code, v, v + 24, o, s, v + 48, v + 72, gl, v + 96, v + 120,
                       self._want(grad_state, "grad_state", ends, f32), self._at(stream))
        if st:
            _check(st, "scan_backward")
        return grad_x, grad_gate, grad_state

    def step(self, x, gate, rows, states, y=None, stream=None):
        """One position for each of n sessions: x, gate [n, dim]; rows [n]
        int64, the session's row of states [num_rows, dim] float32 (outside:
        dropped, y = 0).  Updates states in place, returns y [n, dim].  Rows
        of one call must be distinct."""
        shape, dt, D = x.shape, x.dtype, self.dim
        if len(shape) != 2 or shape[1] != D or states.dim() != 2:
            raise ValueError("x: [n, %d] and states [num_rows, %d] expected" % (D, D))
        n, pool = shape[0], states.shape[0]
        if y is None:
            y = self._empty(shape, dt, x, stream)
        st = self._step(n, D, _element(dt), self._want(x, "x", shape, dt, False), x.stride(0),
                        self._want(gate, "gate", shape, dt, False), gate.stride(0),
                        self._want(rows, "rows", (n,), self._t.int64),
                        self._want(states, "states", (pool, D), self._f32), pool,
                        self._want(y, "y", shape, dt, False), y.stride(0), self._at(stream))
        if st:
            _check(st, "scan_step")
        return y

    def device_status(self, stream=None):
        return scan_get_device_status(self.handle, self._at(stream))


class DeltaScan(_Handle):
    """The gated delta rule over [batch, time, heads, dim] sequences, a recurrence
    whose state of a head is a matrix S [key_dim, value_dim]:

        S' = exp(decay_t) S_{t-1};  S_t = S' + beta_t k_t (v_t - S'^T k_t)^T;  y_t = scale S_t^T q_t

    forward and backward over whole sequences (float32, bfloat16 or float16, any
    strides with a contiguous last axis; decay, beta and states in float32), and one
    step for serving on state rows of a pool.  v, y, decay and beta have ``heads``
    heads, q and k ``key_heads`` (None: as many), each for heads / key_heads
    neighbouring ones.  decay is a logarithm (<= 0; -infinity forgets the state).
    scale: key_dim ** -0.5 if None.  ``offsets`` as GatedScan takes them: past an
    entry's end y and the gradients are 0.  training: room for backward."""

    _destroy = staticmethod(delta_destroy)

    def __init__(self, key_dim, value_dim, heads, max_batch, max_len, key_heads=None, scale=None, training=False):
        super().__init__()
        self.key_dim, self.value_dim, self.heads = key_dim, value_dim, heads
        self.key_heads = heads if key_heads is None else key_heads
        self.scale = (key_dim ** -0.5 if key_dim > 0 else 1.0) if scale is None else scale
        self.training = bool(training)
        self._made(delta_create(key_dim, value_dim, heads, self.key_heads, max_batch, max_len, self.training))
        L = lib()
        self._fwd, self._bwd, self._step = L.delta_forward, L.delta_backward, L.delta_step

    def _view(self, t, name, shape, dtype):
        """(pointer, batch, time and head stride) of a [batch, time, heads, dim] tensor."""
        p = self._want(t, name, shape, dtype, False)
        return (p, *t.stride()[:3])

    def _each(self, t, name, shape):
        """The same of a [batch, time, heads] float32 tensor of any strides."""
        if t.dtype is not self._f32 or t.shape != shape or t.get_device() != self._device:
            self._want(t, name, shape, self._f32)
        return (t.data_ptr(), *t.stride())

    def _common(self, q, k, v, decay, beta, offsets, state):
        shape, dt = v.shape, v.dtype
        if len(shape) != 4 or shape[2] != self.heads or shape[3] != self.value_dim:
            raise ValueError("v: [batch, time, %d, %d] expected, got %s" % (self.heads, self.value_dim, tuple(shape)))
        B, n = shape[0], shape[1]
        keys, each, ends = (B, n, self.key_heads, self.key_dim), (B, n, self.heads), self._ends(B)
        views = (*self._view(q, "q", keys, dt), *self._view(k, "k", keys, dt), *self._view(v, "v", shape, dt),
                 *self._each(decay, "decay", each), *self._each(beta, "beta", each))
        return (B, n, _element(dt), dt, shape, keys, each, ends,
                None if offsets is None else self._want(offsets, "offsets", (B + 1,), self._i32),
                None if state is None else self._want(state, "state", ends, self._f32), views)

    def _ends(self, n):
        return (n, self.heads, self.key_dim, self.value_dim)

    def forward(self, q, k, v, decay, beta, offsets=None, state=None, y=None, last=None, stream=None):
        """(y, last): [batch, time, heads, value_dim], and the state [batch, heads,
        key_dim, value_dim] float32 after the last live position.  state: the one
        before the first (None = 0).  y and last may be given."""
        B, n, code, dt, shape, _, _, ends, o, s, views = self._common(q, k, v, decay, beta, offsets, state)
        if y is None:
            y = self._empty(shape, dt, v, stream)
        if last is None:
            last = self._empty(ends, self._f32, v, stream)
        held = (c_int64 * 24)(*views, *self._view(y, "y", shape, dt))
        a = ctypes.addressof(held)
        st = self._fwd(self.handle, B, n, code, a, a + 32, a + 64, a + 96, a + 128, o, self.scale, s, a + 160,
                       self._want(last, "last", ends, self._f32), self._at(stream))
        if st:
            _check(st, "delta_forward")
        return y, last

    def backward(self, q, k, v, decay, beta, grad_y, offsets=None, state=None, grad_last=None, grad_q=None,
                 grad_k=None, grad_v=None, grad_decay=None, grad_beta=None, grad_state=None, stream=None):
        """(grad_q, grad_k, grad_v, grad_decay, grad_beta, grad_state) from the
        gradients of y and (None = 0) of last; the inputs as in forward.  The
        results may be given."""
        B, n, code, dt, shape, keys, each, ends, o, s, views = self._common(q, k, v, decay, beta, offsets, state)
        f32 = self._f32
        gl = None if grad_last is None else self._want(grad_last, "grad_last", ends, f32)
        if grad_q is None:
            grad_q = self._empty(keys, dt, v, stream)
        if grad_k is None:
            grad_k = self._empty(keys, dt, v, stream)
        if grad_v is None:
            grad_v = self._empty(shape, dt, v, stream)
        if grad_decay is None:
            grad_decay = self._empty(each, f32, v, stream)
        if grad_beta is None:
            grad_beta = self._empty(each, f32, v, stream)
        if grad_state is None:
            grad_state = self._empty(ends, f32, v, stream)
        held = (c_int64 * 44)(*views, *self._view(grad_y, "grad_y", shape, dt), *self._view(grad_q, "grad_q", keys, dt),
                              *self._view(grad_k, "grad_k", keys, dt), *self._view(grad_v, "grad_v", shape, dt),
                              *self._each(grad_decay, "grad_decay", each), *self._each(grad_beta, "grad_beta", each))
        a = ctypes.addressof(held)
        st = self._bwd(self.handle, B, n, code, a, a + 32, a + 64, a + 96, a + 128, o, self.scale, s, a + 160, gl,
                       a + 192, a + 224, a + 256, a + 288, a + 320, self._want(grad_state, "grad_state", ends, f32),
                       self._at(stream))
        if st:
            _check(st, "delta_backward")
        return grad_q, grad_k, grad_v, grad_decay, grad_beta, grad_state

    def step(self, q, k, v, decay, beta, rows, states, y=None, stream=None):
        """One position for each of n sessions: q, k [n, key_heads, key_dim], v [n,
        heads, value_dim], decay, beta [n, heads]; rows [n] int64, the session's row of
        states [num_rows, heads, key_dim, value_dim] float32 (outside: dropped, y = 0).
        Updates states in place, returns y [n, heads, value_dim].  Rows of one call
        must be distinct."""
        shape, dt, H = v.shape, v.dtype, self.heads
        if len(shape) != 3 or shape[1] != H or shape[2] != self.value_dim or states.dim() != 4:
            raise ValueError("v: [n, %d, %d] and states [num_rows, %d, %d, %d] expected" % (
                H, self.value_dim, H, self.key_dim, self.value_dim))
        n, pool = shape[0], states.shape[0]
        keys = (n, self.key_heads, self.key_dim)
        if y is None:
            y = self._empty(shape, dt, v, stream)
        held = []
        for t, name, want in ((q, "q", keys), (k, "k", keys), (v, "v", shape), (y, "y", shape)):
            p = self._want(t, name, want, dt, False)
            held += (p, t.stride(0), 0, t.stride(1))
        for t, name in ((decay, "decay"), (beta, "beta")):
            p = self._each(t, name, (n, H))
            held += (p[0], p[1], 0, p[2])
        held = (c_int64 * 24)(*held)
        a = ctypes.addressof(held)
        st = self._step(n, self.key_dim, self.value_dim, H, self.key_heads, _element(dt), a, a + 32, a + 64, a + 128,
                        a + 160, self.scale, self._want(rows, "rows", (n,), self._t.int64),
                        self._want(states, "states", self._ends(pool), self._f32), pool, a + 96, self._at(stream))
        if st:
            _check(st, "delta_step")
        return y


class Routing:
    """The order of a batch's choices by expert (moe_route of emb.h):
    offsets  [experts + 1] int32: first row of each expert's segment
    counts   [experts] int32: live rows of each segment
    pos      [tokens, top_k] int32: row of each choice, -1 where dropped
    src      [rows] int32: flat choice of each row, -1 for padding"""

    __slots__ = ("_arrays", "_at", "_shape")

    def __init__(self, offsets, counts, pos, src):
        import torch
        if not offsets.is_cuda or pos.dim() != 2:
            raise ValueError("a routing's arrays: on the GPU expected, and pos [tokens, top_k]")
        device = offsets.get_device()
        for t, name in ((offsets, "offsets"), (counts, "counts"), (pos, "pos"), (src, "src")):
            _want(t, name, t.shape, torch.int32, device)
        self._arrays = (offsets, counts, pos, src)
        self._at, self._shape = (pos.data_ptr(), src.data_ptr()), (*pos.shape, src.numel(), device)

    def __iter__(self):
        return iter(self._arrays)

    # not to be replaced: the calls use the addresses found when it was made
    offsets = property(lambda self: self._arrays[0])
    counts = property(lambda self: self._arrays[1])
    pos = property(lambda self: self._arrays[2])
    src = property(lambda self: self._arrays[3])

    @classmethod
    def _made(cls, offsets, counts, pos, src, at, shape):
        r = cls.__new__(cls)
        r._arrays, r._at, r._shape = (offsets, counts, pos, src), at, shape
        return r


class Gate:
    """What a batch's logits gave (moe_gate of emb.h):
    experts     [tokens, top_k] int32: choices, -1 where there is none
    weights     [tokens, top_k] float32
    counts      [experts] int32: choices of each expert
    losses      [2] float32: balance and z
    stats       [tokens, 2] float32: largest logit, -infinity for a token that is
                not live, and sum of the exponentials beside it
    live_count  [1] int32
    normalize   whether the weights are a softmax over the choices alone"""

    __slots__ = ("_arrays", "_at", "_shape", "normalize")

    def __init__(self, arrays, at, shape, normalize):
        self._arrays, self._at, self._shape, self.normalize = arrays, at, shape, normalize

    # not to be replaced: the calls use the addresses found when it was made
    experts = property(lambda self: self._arrays[0])
    weights = property(lambda self: self._arrays[1])
    counts = property(lambda self: self._arrays[2])
    losses = property(lambda self: self._arrays[3])
    stats = property(lambda self: self._arrays[4][:2 * self._shape[0]].view(-1, 2))
    live_count = property(lambda self: self._arrays[4][2 * self._shape[0]:].view(self._arrays[0].dtype))


class ExpertRouter(_Handle):
    """Tokens sorted by expert and back, and the gate that chooses their experts.
    Each of at most max_tokens tokens chooses top_k experts; every expert's rows
    start at a multiple of align."""

    _destroy = staticmethod(moe_destroy)

    def __init__(self, n_experts, top_k, max_tokens, align=1):
        super().__init__()
        self.n_experts, self.top_k, self.align = n_experts, top_k, align
        self._made(moe_create(n_experts, top_k, max_tokens, align))
        L = lib()
        self._route, self._dispatch, self._combine = L.moe_route, L.moe_dispatch, L.moe_combine
        self._combine_backward = L.moe_combine_backward
        self._gate, self._gate_backward = L.moe_gate, L.moe_gate_backward

    def rows(self, n_tokens):
        """Rows of the expert-ordered arrays for n_tokens tokens."""
        a = self.align
        return (n_tokens * self.top_k + self.n_experts * (a - 1) + a - 1) // a * a

    def gate(self, logits, live=None, normalize=True, stream=None):
        """Gate of logits [tokens, experts]: every live token's top_k choices
        (equal logits in the experts' order), their weights (normalize: a softmax
        over the choices, else over all), the experts' counts and the balance
        and z losses.  live: [tokens] bool, None = all."""
        shape, E, K, i32, f32 = logits.shape, self.n_experts, self.top_k, self._i32, self._f32
        if len(shape) != 2 or shape[1] != E:
            raise ValueError("logits: [tokens, %d] expected, got %s" % (E, tuple(shape)))
        n, dt = shape[0], logits.dtype
        x = self._want(logits, "logits", shape, dt, False)
        on = None if live is None else self._want(live, "live", (n,), self._t.bool)
        s = self._at(stream)
        experts, weights = self._empty((n, K), i32, logits, stream), self._empty((n, K), f32, logits, stream)
        counts, losses = self._empty((E,), i32, logits, stream), self._empty((2,), f32, logits, stream)
        stats = self._empty((2 * n + 1,), f32, logits, stream)      # and the live count
        p = stats.data_ptr()
        at = (experts.data_ptr(), weights.data_ptr(), counts.data_ptr(), p, p + 8 * n)
        st = self._gate(self.handle, n, _element(dt), x, logits.stride(0), on, normalize, at[0], at[1], at[2],
                        losses.data_ptr(), p, at[4], s)
        if st:
            _check(st, "moe_gate")
        return Gate((experts, weights, counts, losses, stats), at, (n, K, E, self._device), bool(normalize))

    def gate_backward(self, logits, gate, grad_weights=None, grad_losses=None, grad_logits=None, stream=None):
        """Gradient of gate()'s logits from those of its weights [tokens, top_k]
        and losses [2] (float32, None = 0)."""
        shape, dt, f32 = logits.shape, logits.dtype, self._f32
        n, K, E, device = gate._shape
        if K != self.top_k or E != self.n_experts or device != self._device:
            raise ValueError("gate: %d of %d experts on cuda:%d" % (K, E, device))
        at = self._want(logits, "logits", (n, E), dt, False)
        gw = None if grad_weights is None else self._want(grad_weights, "grad_weights", (n, K), f32)
        gl = None if grad_losses is None else self._want(grad_losses, "grad_losses", (2,), f32)
        if grad_logits is None:
            grad_logits = self._empty(shape, dt, logits, stream)
        to = self._want(grad_logits, "grad_logits", shape, dt, False)
        st = self._gate_backward(self.handle, n, _element(dt), at, logits.stride(0), gate.normalize, *gate._at, gw, gl,
                                 to, grad_logits.stride(0), self._at(stream))
        if st:
            _check(st, "moe_gate_backward")
        return grad_logits

    def route(self, experts, stream=None):
        """Routing of experts [tokens, top_k] int32 (a choice outside [0,
        n_experts) is dropped)."""
        shape, i32, E = experts.shape, self._i32, self.n_experts
        if len(shape) != 2:
            raise ValueError("experts: [tokens, %d] expected, got %s" % (self.top_k, tuple(shape)))
        n = shape[0]
        pos = (n, self.top_k)
        e = self._want(experts, "experts", pos, i32)
        rows = self.rows(n)
        offsets, counts = self._empty((E + 1,), i32, experts, stream), self._empty((E,), i32, experts, stream)
        pos, src = self._empty(pos, i32, experts, stream), self._empty((rows,), i32, experts, stream)
        at = (pos.data_ptr(), src.data_ptr())
        st = self._route(self.handle, n, e, offsets.data_ptr(), counts.data_ptr(), at[0], at[1],
                         self._at(stream))
        if st:
            _check(st, "moe_route")
        return Routing._made(offsets, counts, pos, src, at, (n, self.top_k, rows, self._device))

    def _routed(self, n, r):
        """(pointer of pos, pointer of src, rows) of a routing of n tokens."""
        m, k, rows, device = r._shape
        if m != n or k != self.top_k or rows != self.rows(n) or device != self._device:
            raise ValueError("routing: of %d tokens by %d and %d rows on cuda:%d, for %d tokens" % (
                m, k, rows, device, n))
        return r._at[0], r._at[1], rows

    def dispatch(self, x, routing, xs=None, stream=None):
        """xs [rows, dim]: the token of each row; padding rows are 0."""
        shape, dt = x.shape, x.dtype
        if len(shape) != 2:
            raise ValueError("x: [tokens, dim] expected, got %s" % (tuple(shape),))
        n, dim = shape
        pos, src, rows = self._routed(n, routing)
        if xs is None:
            xs = self._empty((rows, dim), dt, x, stream)
            to = xs.data_ptr()
        else:
            to = self._want(xs, "xs", (rows, dim), dt)
        st = self._dispatch(self.handle, n, dim, _element(dt), self._want(x, "x", shape, dt, False), x.stride(0),
                            pos, src, to, self._at(stream))
        if st:
            _check(st, "moe_dispatch")
        return xs

    def combine(self, ys, weights, routing, y=None, stream=None):
        """y [tokens, dim]: the sum of each token's rows of ys, each times its
        weight ([tokens, top_k] float32; None = 1)."""
        shape, dt = ys.shape, ys.dtype
        if len(shape) != 2:
            raise ValueError("ys: [rows, dim] expected, got %s" % (tuple(shape),))
        n, dim = routing._shape[0], shape[1]
        pos, _, rows = self._routed(n, routing)
        w = None if weights is None else self._want(weights, "weights", (n, self.top_k), self._f32)
        if y is None:
            y = self._empty((n, dim), dt, ys, stream)
            to, stride = y.data_ptr(), dim
        else:
            to, stride = self._want(y, "y", (n, dim), dt, False), y.stride(0)
        st = self._combine(self.handle, n, dim, _element(dt), self._want(ys, "ys", (rows, dim), dt), w, pos, to, stride,
                           self._at(stream))
        if st:
            _check(st, "moe_combine")
        return y

    def combine_backward(self, grad_y, ys, weights, routing, grad_ys=None, grad_weights=None, stream=None):
        """(grad_ys, grad_weights) of combine; weights None gives grad_weights
        None."""
        shape, dt, f32 = grad_y.shape, grad_y.dtype, self._f32
        if len(shape) != 2:
            raise ValueError("grad_y: [tokens, dim] expected, got %s" % (tuple(shape),))
        n, dim = shape
        pos, src, rows = self._routed(n, routing)
        wide, each = (rows, dim), (n, self.top_k)
        w = None if weights is None else self._want(weights, "weights", each, f32)
        if weights is not None and grad_weights is None:
            grad_weights = self._empty(each, f32, weights, stream)
        gw = None if grad_weights is None else self._want(grad_weights, "grad_weights", each, f32)
        if grad_ys is None:
            grad_ys = self._empty(wide, dt, grad_y, stream)
        st = self._combine_backward(self.handle, n, dim, _element(dt), self._want(grad_y, "grad_y", shape, dt, False),
                                    grad_y.stride(0), self._want(ys, "ys", wide, dt), w, pos, src,
                                    self._want(grad_ys, "grad_ys", wide, dt), gw, self._at(stream))
        if st:
            _check(st, "moe_combine_backward")
        return grad_ys, grad_weights

    def dispatch_backward(self, grad_xs, routing, grad_x=None, stream=None):
        """grad_x [tokens, dim] of dispatch: the sum of each token's rows."""
        return self.combine(grad_xs, None, routing, grad_x, stream)


class LayerNorm(_Handle):
    """Layer norm over the last axis of rows [rows, dim] or of padded sequences
    [batch, time, dim] (float32, bfloat16 or float16, any strides with a contiguous
    last axis), forward and backward with the gradients of weight and bias.  weight
    and bias are float32 or of the rows' type; None = 1 and 0.  ``offsets`` as
    GatedScan takes them: past an entry's end y and the gradient are 0, and nothing
    is added to the weight's."""

    _destroy = staticmethod(norm_destroy)

    def __init__(self, dim, eps=1e-5):
        super().__init__()
        self.dim, self.eps = dim, eps
        self._made(norm_create(dim))
        L = lib()
        self._fwd, self._bwd = L.norm_forward, L.norm_backward

    def _view(self, t, name, shape, dtype):
        """(pointer, batch stride, row stride) of rows or of padded sequences."""
        p = self._want(t, name, shape, dtype, False)
        s = t.stride()
        return (p, 0, s[0]) if len(s) == 2 else (p, s[0], s[1])

    def _common(self, x, weight, bias, offsets):
        shape, dt = x.shape, x.dtype
        if len(shape) not in (2, 3) or shape[-1] != self.dim:
            raise ValueError("x: [rows, %d] or [batch, time, %d] expected, got %s" % (self.dim, self.dim, tuple(shape)))
        B, n = (1, shape[0]) if len(shape) == 2 else (shape[0], shape[1])
        if offsets is not None and len(shape) == 2:
            raise ValueError("offsets: of [batch, time, dim] sequences only")
        code, wdt = _element(dt), self._f32
        given = weight if weight is not None else bias
        if given is not None and given.dtype is dt:
            wdt = dt
        flat = (self.dim,)
        return (B, n, code, dt, shape, None if offsets is None else self._want(offsets, "offsets", (B + 1,), self._i32),
                _element(wdt), None if weight is None else self._want(weight, "weight", flat, wdt),
                None if bias is None else self._want(bias, "bias", flat, wdt))

    def forward(self, x, weight=None, bias=None, offsets=None, y=None, stats=None, stream=None):
        """(y, stats): the normalised rows, and [..., 2] float32 with each row's
        mean and 1 / deviation, which backward takes.  Both may be given."""
        B, n, code, dt, shape, o, wc, w, b = self._common(x, weight, bias, offsets)
        if y is None:
            y = self._empty(shape, dt, x, stream)
        two = (*shape[:-1], 2)
        if stats is None:
            stats = self._empty(two, self._f32, x, stream)
        held = (c_int64 * 6)(*self._view(x, "x", shape, dt), *self._view(y, "y", shape, dt))
        v = ctypes.addressof(held)
        st = self._fwd(self.handle, B, n, code, v, o, wc, w, b, self.eps, v + 24,
                       self._want(stats, "stats", two, self._f32), self._at(stream))
        if st:
            _check(st, "norm_forward")
        return y, stats

    def backward(self, x, grad_y, stats, weight=None, offsets=None, grad_x=None, grad_weight=None, grad_bias=None,
                 stream=None):
        """(grad_x, grad_weight, grad_bias) from the gradient of y; x, weight and
        offsets as in forward, stats as it gave them.  The weight's and the bias'
        are [dim] float32.  The results may be given."""
        B, n, code, dt, shape, o, wc, w, _ = self._common(x, weight, None, offsets)
        f32, flat = self._f32, (self.dim,)
        if grad_x is None:
            grad_x = self._empty(shape, dt, x, stream)
        if grad_weight is None:
            grad_weight = self._empty(flat, f32, x, stream)
        if grad_bias is None:
            grad_bias = self._empty(flat, f32, x, stream)
        held = (c_int64 * 9)(*self._view(x, "x", shape, dt), *self._view(grad_y, "grad_y", shape, dt),
                             *self._view(grad_x, "grad_x", shape, dt))
        v = ctypes.addressof(held)
        st = self._bwd(self.handle, B, n, code, v, o, wc, w, v + 24, self._want(stats, "stats", (*shape[:-1], 2), f32),
                       v + 48, self._want(grad_weight, "grad_weight", flat, f32),
                       self._want(grad_bias, "grad_bias", flat, f32), self._at(stream))
        if st:
            _check(st, "norm_backward")
        return grad_x, grad_weight, grad_bias


class AdamW(_Handle):
    """AdamW over a list of parameter tensors, one call per step (adamw_* of
    emb.h).  params are float32, bfloat16 or float16; grads have the same type
    or float32 and are read at every step from the tensors given here (or to
    bind_grads); masters (float32, optional) hold the weights of 16-bit params.
    weight_decay is a number or one per tensor.  state_bits 32: m and v are
    float32 tensors shaped like the params; 8: uint8 codes of that shape and
    int16 tops, one per 256 elements (``m``, ``v``, ``m_top``, ``v_top``; created
    at zero, or given).  step: steps already taken.

    max_update: the largest magnitude of m / sqrt(v) that a step may use (None: no
    limit).  8-bit states can lose a small second moment beside a large one in its
    block and keep the first: such a weight would move by many lr (emb.h gives a
    case of 16, and of 940 when its gradient stops).  7.3 bounds that for betas
    (0.9, 0.999) and leaves every update of unrounded moments as it is.

    A step may be captured in a graph: each replay is a step of its own, counted
    on the device, with the lr and grad_scale tensor of the capture.  From then
    on every step of the handle is counted there (a launch more), and reading
    step_count waits for the current stream."""

    _destroy = staticmethod(adamw_destroy)

    def __init__(self, params, grads, masters=None, weight_decay=0.01, betas=(0.9, 0.999), eps=1e-8, state_bits=32,
                 m=None, v=None, m_top=None, v_top=None, seed=0, step=0, max_update=None):
        super().__init__()
        torch = self._t
        self.params, self.betas, self.eps, self.seed = list(params), betas, eps, seed
        self.grads = list(grads)
        self.masters = list(masters) if masters is not None else [None] * len(self.params)
        n = len(self.params)
        decay = [weight_decay] * n if isinstance(weight_decay, (int, float)) else list(weight_decay)
        if state_bits not in (8, 32):
            raise ValueError("state_bits: 8 or 32")
        if len(self.grads) != n or len(self.masters) != n or len(decay) != n:
            raise ValueError("one gradient, master and weight decay per parameter")
        self.state_bits = state_bits
        eight = state_bits == 8
        state = torch.uint8 if eight else torch.float32
        self._device = self._current()
        shapes = [p.shape for p in self.params]
        blocks = [_blocks(p) for p in self.params] if eight else None
        fields = {"param": [self._want(p, "params", k, p.dtype) for p, k in zip(self.params, shapes)],
                  "grad": [self._want(g, "grads", k, p.dtype if g.dtype is p.dtype else torch.float32)
                           for g, p, k in zip(self.grads, self.params, shapes)],
                  "master": [0 if w is None else self._want(w, "masters", k, torch.float32)
                             for w, k in zip(self.masters, shapes)]}
        for given, name, dtype, sizes in ((m, "m", state, shapes), (v, "v", state, shapes),
                                          (m_top, "m_top", torch.int16, blocks), (v_top, "v_top", torch.int16, blocks)):
            if sizes is None:
                if given is not None:
                    raise ValueError("%s: 8-bit states only" % name)
                setattr(self, name, None)
                continue
            held = ([torch.zeros(k, dtype=dtype, device=p.device) for p, k in zip(self.params, sizes)]
                    if given is None else list(given))
            if len(held) != n:
                raise ValueError("%s: one per parameter" % name)
            fields[name] = [self._want(t, name, k, dtype) for t, k in zip(held, sizes)]
            setattr(self, name, held)
        fields["numel"] = [p.numel() for p in self.params]
        fields["weight_decay"] = decay
        fields["dtype"] = [_element(p.dtype) for p in self.params]
        fields["grad_dtype"] = [_element(g.dtype) for g in self.grads]
        self._grad_dtypes = [g.dtype for g in self.grads]
        self._made(adamw_create(_tensors(fields, n), STATES_8BIT if eight else 0))
        self._step, self._size = lib().adamw_step, adamw_export_size(self.handle)
        self._taken, self._counted = 0, False   # steps, where the host counts them
        if step:
            self.step_count = step
        if max_update is not None:
            adamw_set_max_update(self.handle, max_update)

    @property
    def step_count(self):
        """Steps taken; may be set."""
        if self._counted:
            return adamw_get_step(self.handle, self._at(None))
        return self._taken

    @step_count.setter
    def step_count(self, step):
        adamw_set_step(self.handle, step, self._at(None))
        self._taken = step

    def bind_grads(self, grads, stream=None):
        """Read other gradient tensors (same shapes and types) from the next
        step on."""
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError("one gradient per parameter")
        for i, g in enumerate(grads):
            self._want(g, "grads", self.params[i].shape, self._grad_dtypes[i])
        adamw_bind_grads(self.handle, grads, self._at(stream))
        self.grads = grads

    def step(self, lr, grad_scale=None, stream=None):
        """One step on every parameter.  grad_scale: a float32 scalar tensor
        on the GPU that every gradient is multiplied by."""
        if grad_scale is not None:
            if (grad_scale.numel() != 1 or grad_scale.get_device() != self._device or
                    grad_scale.dtype != self._t.float32):
                raise ValueError("grad_scale: one float32 on cuda:%d" % self._device)
        args = (lr, self.betas[0], self.betas[1], self.eps, None if grad_scale is None else grad_scale.data_ptr(),
                self.seed, self._at(stream))
        if not self._counted:
            st = self._step(self.handle, self._taken + 1, *args)
            if not st:
                self._taken += 1
                return
            if st != UNSUPPORTED:
                _check(st, "adamw_step")
            self._counted = True   # the stream is being captured
        st = self._step(self.handle, 0, *args)
        if st:
            _check(st, "adamw_step")

    def states(self, stream=None):
        """What the 8-bit states stand for: (m, v), bfloat16 (exact), tensor
        after tensor, each from the next multiple of 256 elements on, zeros
        between them."""
        like, bf16 = self.params[0], self._t.bfloat16
        m, v = self._empty((self._size,), bf16, like, stream), self._empty((self._size,), bf16, like, stream)
        adamw_export_states(self.handle, m, v, self._at(stream))
        return m, v


def _blocks(p):
    return ((p.numel() + BLOCK - 1) // BLOCK,)


def _tensors(fields, n):
    """adamw_tensor structures from lists of their fields (fast for thousands
    of tensors)."""
    import numpy as np
    out = np.zeros(n, np.dtype(AdamwTensor))
    for name, values in fields.items():
        out[name] = values
    return out
