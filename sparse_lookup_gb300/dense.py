"""Operators of the dense layers behind the lookups (scan_*, moe_* and adamw_*
of include/emb.h): raw C names, then GatedScan, ExpertRouter and AdamW over
PyTorch tensors.  Marshalling only, like the rest of the binding; arguments
that the library cannot see (shapes, element types, devices) are checked here
and raise ValueError.

An output that a call allocates belongs to the stream the call runs on.
Tensors that come from another stream are the caller's to order (an event, or
record_stream), as everywhere in this package.
"""
from __future__ import annotations

import ctypes
from ctypes import c_float, c_int32, c_int64, c_void_p
from typing import NamedTuple

from . import TABLE_DTYPE, EmbError, _check, lib, ptr

STATES_8BIT = 1
BLOCK = 256          # elements that share a top in an 8-bit state
_ELEMENT = {k: v for k, v in TABLE_DTYPE.items() if k != "int8"}
_dtype_codes = {}    # torch dtype -> emb_table_dtype


class ScanView(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("batch_stride", c_int64), ("time_stride", c_int64)]


class AdamwTensor(ctypes.Structure):
    _fields_ = [("param", c_void_p), ("grad", c_void_p), ("master", c_void_p), ("m", c_void_p), ("v", c_void_p),
                ("m_top", c_void_p), ("v_top", c_void_p), ("numel", c_int64), ("weight_decay", c_float),
                ("dtype", c_int32), ("grad_dtype", c_int32), ("reserved", c_int32)]


# ---------------------------------------------------------------------------
# raw C names
# ---------------------------------------------------------------------------

def _stream(stream):
    """The raw handle of a stream; None: the current stream of the current
    device (the short way to it: a call may be a few microseconds of work)."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
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


def moe_destroy(h):
    _check(lib().moe_destroy(h), "moe_destroy")


def adamw_create(tensors, flags):
    arr = (AdamwTensor * max(1, len(tensors)))(*tensors)
    h = c_void_p()
    _check(lib().adamw_create(arr, len(tensors), flags, ctypes.byref(h)), "adamw_create")
    return h.value


def adamw_bind_grads(h, grads, stream=None):
    arr = (c_void_p * max(1, len(grads)))(*[ptr(g) for g in grads])
    _check(lib().adamw_bind_grads(h, arr, _stream(stream)), "adamw_bind_grads")


def adamw_step(h, step, lr, beta1, beta2, eps, grad_scale, seed, stream=None):
    _check(lib().adamw_step(h, step, lr, beta1, beta2, eps, ptr(grad_scale), seed, _stream(stream)), "adamw_step")


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


def _want(t, name, shape, dtype, dense=True):
    """Checks one tensor argument: on the GPU, of this shape and type, dense
    (or only its last axis contiguous)."""
    if not t.is_cuda or t.shape != shape or t.dtype != dtype:
        raise ValueError("%s: %s %s on the GPU expected, got %s %s on %s" % (
            name, tuple(shape), dtype, tuple(t.shape), t.dtype, t.device))
    if dense:
        if not t.is_contiguous():
            raise ValueError("%s: a contiguous tensor expected, got strides %s" % (name, t.stride()))
    elif t.stride(-1) != 1 and t.shape[-1] > 1 and t.numel():
        raise ValueError("%s: a contiguous last axis expected, got strides %s" % (name, t.stride()))
    return t


def _empty(shape, dtype, device, stream):
    """A tensor that belongs to the stream the kernel will run on."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    s = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
    with torch.cuda.stream(s):
        return torch.empty(shape, dtype=dtype, device=device)


class _Handle:
    handle = None

    def close(self):
        if self.handle:
            h, self.handle = self.handle, None
            self._destroy(h)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


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
        self.dim = dim
        self.handle = scan_create(dim, max_batch, max_len)

    def _view(self, t, name, shape, dtype):
        _want(t, name, shape, dtype, dense=False)
        sb, st, _ = t.stride()
        return ScanView(t.data_ptr(), sb, st)

    def _common(self, x, gate, offsets, state):
        import torch
        if x.dim() != 3 or x.shape[2] != self.dim:
            raise ValueError("x: [batch, time, %d] expected, got %s" % (self.dim, tuple(x.shape)))
        code, shape = _element(x.dtype), x.shape
        vx = self._view(x, "x", shape, x.dtype)
        vg = self._view(gate, "gate", shape, x.dtype)
        if offsets is not None:
            _want(offsets, "offsets", (shape[0] + 1,), torch.int32)
        if state is not None:
            _want(state, "state", (shape[0], self.dim), torch.float32)
        return code, shape, vx, vg

    def forward(self, x, gate, offsets=None, state=None, y=None, last=None, stream=None):
        """(y, last): h_t at every position, and the state [batch, dim]
        float32 after the last live one.  state: the one before the first
        (None = 0).  y and last may be given."""
        import torch
        code, shape, vx, vg = self._common(x, gate, offsets, state)
        if y is None:
            y = _empty(shape, x.dtype, x.device, stream)
        if last is None:
            last = _empty((shape[0], self.dim), torch.float32, x.device, stream)
        else:
            _want(last, "last", (shape[0], self.dim), torch.float32)
        scan_forward(self.handle, shape[0], shape[1], code, vx, vg, offsets, state,
                     self._view(y, "y", shape, x.dtype), last, stream)
        return y, last

    def backward(self, x, gate, y, grad_y, offsets=None, state=None, grad_last=None, grad_x=None, grad_gate=None,
                 grad_state=None, stream=None):
        """(grad_x, grad_gate, grad_state) from the gradients of y and (None =
        0) of last; x, gate, offsets and state as in forward, y as it gave
        it.  The results may be given."""
        import torch
        code, shape, vx, vg = self._common(x, gate, offsets, state)
        dt = x.dtype
        for t, name in ((grad_last, "grad_last"), (grad_state, "grad_state")):
            if t is not None:
                _want(t, name, (shape[0], self.dim), torch.float32)
        if grad_x is None:
            grad_x = _empty(shape, dt, x.device, stream)
        if grad_gate is None:
            grad_gate = _empty(shape, dt, x.device, stream)
        if grad_state is None:
            grad_state = _empty((shape[0], self.dim), torch.float32, x.device, stream)
        scan_backward(self.handle, shape[0], shape[1], code, vx, vg, offsets, state, self._view(y, "y", shape, dt),
                      self._view(grad_y, "grad_y", shape, dt), grad_last, self._view(grad_x, "grad_x", shape, dt),
                      self._view(grad_gate, "grad_gate", shape, dt), grad_state, stream)
        return grad_x, grad_gate, grad_state

    def step(self, x, gate, rows, states, y=None, stream=None):
        """One position for each of n sessions: x, gate [n, dim]; rows [n]
        int64, the session's row of states [num_rows, dim] float32 (outside:
        dropped, y = 0).  Updates states in place, returns y [n, dim].  Rows
        of one call must be distinct."""
        import torch
        if x.dim() != 2 or x.shape[1] != self.dim or states.dim() != 2:
            raise ValueError("x: [n, %d] and states [num_rows, %d] expected" % (self.dim, self.dim))
        shape, dt = x.shape, x.dtype
        code = _element(dt)
        _want(x, "x", shape, dt, dense=False)
        _want(gate, "gate", shape, dt, dense=False)
        _want(rows, "rows", shape[:1], torch.int64)
        _want(states, "states", (states.shape[0], self.dim), torch.float32)
        if y is None:
            y = _empty(shape, dt, x.device, stream)
        else:
            _want(y, "y", shape, dt, dense=False)
        scan_step(shape[0], self.dim, code, x, x.stride(0), gate, gate.stride(0), rows, states, states.shape[0], y,
                  y.stride(0), stream)
        return y

    def device_status(self, stream=None):
        return scan_get_device_status(self.handle, stream)


class Routing(NamedTuple):
    """The order of a batch's choices by expert (moe_route of emb.h)."""
    offsets: object      # [experts + 1] int32: first row of each expert's segment
    counts: object       # [experts] int32: live rows of each segment
    pos: object          # [tokens, top_k] int32: row of each choice, -1 where dropped
    src: object          # [rows] int32: flat choice of each row, -1 for padding


class ExpertRouter(_Handle):
    """Tokens sorted by expert and back.  Each of at most max_tokens tokens
    chooses top_k experts; every expert's rows start at a multiple of
    align."""

    _destroy = staticmethod(moe_destroy)

    def __init__(self, n_experts, top_k, max_tokens, align=1):
        self.n_experts, self.top_k, self.align = n_experts, top_k, align
        self.handle = moe_create(n_experts, top_k, max_tokens, align)

    def rows(self, n_tokens):
        """Rows of the expert-ordered arrays for n_tokens tokens."""
        a = self.align
        return (n_tokens * self.top_k + self.n_experts * (a - 1) + a - 1) // a * a

    def route(self, experts, stream=None):
        """Routing of experts [tokens, top_k] int32 (a choice outside [0,
        n_experts) is dropped)."""
        import torch
        if experts.dim() != 2:
            raise ValueError("experts: [tokens, %d] expected, got %s" % (self.top_k, tuple(experts.shape)))
        n, dev = experts.shape[0], experts.device
        _want(experts, "experts", (n, self.top_k), torch.int32)
        E, K, R = self.n_experts, self.top_k, self.rows(n)
        # one allocation, each part at a multiple of 32 bytes
        at, end = [], 0
        for k in (E + 1, E, n * K, R):
            at.append((end, k))
            end += (k + 7) // 8 * 8
        whole = _empty((end,), torch.int32, dev, stream)
        offsets, counts, pos, src = [whole[a:a + k] for a, k in at]
        moe_route(self.handle, n, experts, offsets, counts, pos, src, stream)
        return Routing(offsets, counts, pos.view(n, K), src)

    def _routed(self, n, r):
        import torch
        _want(r.pos, "pos", (n, self.top_k), torch.int32)
        _want(r.src, "src", (self.rows(n),), torch.int32)

    def _tokens(self, x, name):
        if x.dim() != 2:
            raise ValueError("%s: [tokens, dim] expected, got %s" % (name, tuple(x.shape)))
        _want(x, name, x.shape, x.dtype, dense=False)
        return x.shape[0], x.shape[1], _element(x.dtype)

    def dispatch(self, x, routing, xs=None, stream=None):
        """xs [rows, dim]: the token of each row; padding rows are 0."""
        n, dim, code = self._tokens(x, "x")
        self._routed(n, routing)
        if xs is None:
            xs = _empty((self.rows(n), dim), x.dtype, x.device, stream)
        else:
            _want(xs, "xs", (self.rows(n), dim), x.dtype)
        moe_dispatch(self.handle, n, dim, code, x, x.stride(0), routing.pos, routing.src, xs, stream)
        return xs

    def combine(self, ys, weights, routing, y=None, stream=None):
        """y [tokens, dim]: the sum of each token's rows of ys, each times its
        weight ([tokens, top_k] float32; None = 1)."""
        import torch
        n, dt = routing.pos.shape[0], ys.dtype
        self._routed(n, routing)
        if ys.dim() != 2:
            raise ValueError("ys: [rows, dim] expected, got %s" % (tuple(ys.shape),))
        dim, code = ys.shape[1], _element(dt)
        _want(ys, "ys", (self.rows(n), dim), dt)
        if weights is not None:
            _want(weights, "weights", (n, self.top_k), torch.float32)
        if y is None:
            y = _empty((n, dim), dt, ys.device, stream)
        else:
            _want(y, "y", (n, dim), dt, dense=False)
        moe_combine(self.handle, n, dim, code, ys, weights, routing.pos, y, y.stride(0), stream)
        return y

    def combine_backward(self, grad_y, ys, weights, routing, grad_ys=None, grad_weights=None, stream=None):
        """(grad_ys, grad_weights) of combine; weights None gives grad_weights
        None."""
        import torch
        n, dim, code = self._tokens(grad_y, "grad_y")
        self._routed(n, routing)
        dt, R = grad_y.dtype, self.rows(n)
        _want(ys, "ys", (R, dim), dt)
        if weights is not None:
            _want(weights, "weights", (n, self.top_k), torch.float32)
            if grad_weights is None:
                grad_weights = _empty((n, self.top_k), torch.float32, grad_y.device, stream)
        if grad_weights is not None:
            _want(grad_weights, "grad_weights", (n, self.top_k), torch.float32)
        if grad_ys is None:
            grad_ys = _empty((R, dim), dt, grad_y.device, stream)
        else:
            _want(grad_ys, "grad_ys", (R, dim), dt)
        moe_combine_backward(self.handle, n, dim, code, grad_y, grad_y.stride(0), ys, weights, routing.pos,
                             routing.src, grad_ys, grad_weights, stream)
        return grad_ys, grad_weights

    def dispatch_backward(self, grad_xs, routing, grad_x=None, stream=None):
        """grad_x [tokens, dim] of dispatch: the sum of each token's rows."""
        return self.combine(grad_xs, None, routing, grad_x, stream)


class AdamW(_Handle):
    """AdamW over a list of parameter tensors, one call per step (adamw_* of
    emb.h).  params are float32, bfloat16 or float16; grads have the same type
    or float32 and are read at every step from the tensors given here (or to
    bind_grads); masters (float32, optional) hold the weights of 16-bit params.
    weight_decay is a number or one per tensor.  state_bits 32: m and v are
    float32 tensors shaped like the params; 8: uint8 codes of that shape and
    int16 tops, one per 256 elements (``m``, ``v``, ``m_top``, ``v_top``; created
    at zero, or given).  step: steps already taken."""

    _destroy = staticmethod(adamw_destroy)

    def __init__(self, params, grads, masters=None, weight_decay=0.01, betas=(0.9, 0.999), eps=1e-8, state_bits=32,
                 m=None, v=None, m_top=None, v_top=None, seed=0, step=0):
        import torch
        self.params, self.betas, self.eps, self.seed, self.step_count = list(params), betas, eps, seed, step
        self.grads = list(grads)
        self.masters = list(masters) if masters is not None else [None] * len(self.params)
        n = len(self.params)
        decay = [weight_decay] * n if isinstance(weight_decay, (int, float)) else list(weight_decay)
        if state_bits not in (8, 32):
            raise ValueError("state_bits: 8 or 32")
        if len(self.grads) != n or len(self.masters) != n or len(decay) != n:
            raise ValueError("one gradient, master and weight decay per parameter")
        self.state_bits = state_bits
        state = torch.float32 if state_bits == 32 else torch.uint8

        def states(given, make, name, dtype, shape):
            out = [make(p) for p in self.params] if given is None else list(given)
            if len(out) != n:
                raise ValueError("%s: one per parameter" % name)
            for t, p in zip(out, self.params):
                _want(t, name, shape(p), dtype)
            return out
        for given, name, dtype, shape in ((m, "m", state, lambda p: p.shape), (v, "v", state, lambda p: p.shape),
                                          (m_top, "m_top", torch.int16, _blocks), (v_top, "v_top", torch.int16, _blocks)):
            if name.endswith("_top") and state_bits == 32:
                if given is not None:
                    raise ValueError("%s: 8-bit states only" % name)
                setattr(self, name, None)
                continue
            setattr(self, name, states(given, lambda p: torch.zeros(shape(p), dtype=dtype, device=p.device), name,
                                       dtype, shape))
        descs = []
        for i, p in enumerate(self.params):
            code = _element(p.dtype)
            _want(p, "params", p.shape, p.dtype)
            g = self._grad(i, self.grads[i])
            if self.masters[i] is not None:
                _want(self.masters[i], "masters", p.shape, torch.float32)
            eight = state_bits == 8
            descs.append(AdamwTensor(ptr(p), ptr(g), ptr(self.masters[i]), ptr(self.m[i]), ptr(self.v[i]),
                                     ptr(self.m_top[i]) if eight else None, ptr(self.v_top[i]) if eight else None,
                                     p.numel(), decay[i], code, _element(g.dtype), 0))
        self._grad_dtypes = [g.dtype for g in self.grads]
        self.handle = adamw_create(descs, STATES_8BIT if state_bits == 8 else 0)

    def _grad(self, i, g):
        import torch
        p = self.params[i]
        return _want(g, "grads", p.shape, p.dtype if g.dtype == p.dtype else torch.float32)

    def bind_grads(self, grads, stream=None):
        """Read other gradient tensors (same shapes and types) from the next
        step on."""
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError("one gradient per parameter")
        for i, g in enumerate(grads):
            _want(g, "grads", self.params[i].shape, self._grad_dtypes[i])
        adamw_bind_grads(self.handle, grads, stream)
        self.grads = grads

    def step(self, lr, grad_scale=None, stream=None):
        """One step on every parameter.  grad_scale: a float32 scalar tensor
        on the GPU that every gradient is multiplied by."""
        import torch
        if grad_scale is not None:
            if grad_scale.numel() != 1 or not grad_scale.is_cuda or grad_scale.dtype != torch.float32:
                raise ValueError("grad_scale: one float32 on the GPU")
        adamw_step(self.handle, self.step_count + 1, lr, self.betas[0], self.betas[1], self.eps, grad_scale, self.seed,
                   stream)
        self.step_count += 1

    def states(self, stream=None):
        """What the 8-bit states stand for: (m, v), bfloat16 (exact), tensor
        after tensor, each from the next multiple of 256 elements on, zeros
        between them."""
        import torch
        n = adamw_export_size(self.handle)
        dev = self.params[0].device
        m = _empty((n,), torch.bfloat16, dev, stream)
        v = _empty((n,), torch.bfloat16, dev, stream)
        adamw_export_states(self.handle, m, v, stream)
        return m, v


def _blocks(p):
    return ((p.numel() + BLOCK - 1) // BLOCK,)
