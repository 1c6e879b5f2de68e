"""The sequence and training operators (C ABI: ``include/fno_ops.h``).

``SandwichNorm``      norms before and after a block with its gate, residual
                      scale and residual sum, and their gradients
``pack_activation`` / ``PackedActivation``
                      activation checkpoints in 8 bits
``LinearGrad``        weight and bias gradient of a 1x1 linear from one
``LinearAttention``   linear attention with a decay for each head: prompts,
                      single tokens, gradients
``Rotary``            rotary positions of its queries and keys
``CausalConv``        short causal convolutions along time, and
``SelectiveScan``     the selective state space scan behind them: prompts, single
                      tokens, gradients

As in the rest of the package, the classes marshal arguments: a plan, a
workspace from torch, tensor pointers and the current stream.  A plan is of the
device that was current when it was made, and takes that device's tensors while it
is the current one.  A plan object holds one workspace, so calls on it have to be
ordered (one stream).  A call with ``stream=`` is launched there and allocates its
results on the current stream: that stream has to wait for the current one's work
before the call, and the current one for it before the results are used or dropped.
"""
from __future__ import annotations

import functools

import torch

from . import _require, _stream_handle, capi, check

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_CODES = {torch.float32: capi.FNO_F32, torch.float16: capi.FNO_F16,
          torch.bfloat16: capi.FNO_BF16}
GROUP = capi.FNO_ACT8_GROUP


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(device, stream):
    """The handle of ``stream``, or of the current stream of ``device`` (by the raw
    query where torch has it: the call is most of a small operator's cost).  That has
    to be the current device, where the launch goes."""
    if _current_device() != device:
        raise ValueError(f"the operands are on cuda:{device}, which is not the current device")
    if stream is None and _raw_stream is not None:
        return _raw_stream(device)
    return _stream_handle(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _field(device, t, dtype, shape, name):
    """t's pointer, once its type, shape, layout and device are those wanted."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.is_contiguous() and t.get_device() == device):
        _require(t, dtype, shape, name)
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    return t.data_ptr()


class PackedActivation:
    """An activation in 8 bits: int8 ``codes`` of the activation's shape and
    float32 ``scales``, one for each run of 128 elements along the last axis."""

    def __init__(self, codes, scales, dtype):
        if dtype not in _CODES:
            raise TypeError(f"dtype must be one of {list(_CODES)}, got {dtype}")
        if not isinstance(codes, torch.Tensor):
            raise TypeError("codes must be a CUDA tensor")
        if codes.dim() < 1 or codes.numel() < 1:
            raise ValueError("codes must have at least one element")
        if not codes.is_cuda:
            raise TypeError("codes must be a CUDA tensor")
        device = codes.get_device()
        _field(device, codes, torch.int8, codes.shape, "codes")
        _field(device, scales, torch.float32,
               codes.shape[:-1] + (-(-codes.shape[-1] // GROUP),), "scales")
        self.codes, self.scales, self.dtype = codes, scales, dtype
        self.shape = codes.shape

    def _rows(self):
        cols = self.shape[-1]
        return self.codes.numel() // cols, cols

    def values(self, out=None, stream=None):
        """The values that the codes stand for, in the storage type."""
        device = self.codes.get_device()
        if out is None:
            out = torch.empty(self.shape, dtype=self.dtype, device=self.codes.device)
        ptr = _field(device, out, self.dtype, self.shape, "out")
        rows, cols = self._rows()
        check(capi.fno_act8_unpack(rows, cols, _CODES[self.dtype], self.codes.data_ptr(),
                                   self.scales.data_ptr(), ptr, _stream(device, stream)),
              "fno_act8_unpack")
        return out

    def gelu_backward(self, dy, out=None, stream=None):
        """dy * GELU'(values); ``out`` may be dy."""
        device = self.codes.get_device()
        dyp = _field(device, dy, self.dtype, self.shape, "dy")
        if out is None:
            out = torch.empty_like(dy)
        ptr = _field(device, out, self.dtype, self.shape, "out")
        rows, cols = self._rows()
        check(capi.fno_act8_gelu_backward(rows, cols, _CODES[self.dtype], self.codes.data_ptr(),
                                          self.scales.data_ptr(), dyp, ptr,
                                          _stream(device, stream)), "fno_act8_gelu_backward")
        return out


def _empty_packed(shape, dtype, device):
    p = PackedActivation.__new__(PackedActivation)
    p.codes = torch.empty(shape, dtype=torch.int8, device=device)
    p.scales = torch.empty((*shape[:-1], -(-shape[-1] // GROUP)), dtype=torch.float32,
                           device=device)
    p.dtype, p.shape = dtype, p.codes.shape
    return p


def pack_activation(x, stream=None) -> PackedActivation:
    """x in 8 bits (x is left alone)."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _CODES:
        raise TypeError("x must be a float32, float16 or bfloat16 CUDA tensor")
    if x.dim() < 1 or x.numel() < 1:
        raise ValueError("x must have at least one element")
    if not x.is_cuda:
        raise TypeError("x must be a CUDA tensor")
    ptr = _field(x.get_device(), x, x.dtype, x.shape, "x")
    p = _empty_packed(x.shape, x.dtype, x.device)
    rows, cols = p._rows()
    check(capi.fno_act8_pack(rows, cols, _CODES[x.dtype], ptr, p.codes.data_ptr(),
                             p.scales.data_ptr(), _stream(x.get_device(), stream)),
          "fno_act8_pack")
    return p


class _Plan:
    """A plan handle with its workspace, of the device that was current when it was
    made: its calls take that device's tensors while it is the current one."""

    def _own(self, status, handle, name, workspace=True):
        check(status, f"fno_{name}_plan")
        self.handle, self._name = handle, name
        self.workspace, self.workspace_bytes = None, 0
        if workspace:
            st, self.workspace_bytes = getattr(capi, f"fno_{name}_workspace_size")(handle)
            check(st)
        self.device = torch.cuda.current_device()
        self._torch_device = torch.device("cuda", self.device)
        # (partials: methods in their place take about 1 us more of a call)
        self._at = functools.partial(_field, self.device)
        self._launch_stream = functools.partial(_stream, self.device)

    def _workspace(self):
        """Allocated at the first call that needs it, then kept."""
        if self.workspace is None and self.workspace_bytes:
            self.workspace = self._empty((self.workspace_bytes,), torch.uint8)
        return _ptr(self.workspace)

    def device_error(self, stream=None) -> int:
        return getattr(capi, f"fno_{self._name}_get_device_error")(self.handle,
                                                                   _stream_handle(stream))

    def _maybe_at(self, t, dtype, shape, name):
        return None if t is None else self._at(t, dtype, shape, name)

    def _empty(self, shape, dtype):
        return torch.empty(shape, dtype=dtype, device=self._torch_device)

    def _out(self, t, dtype, shape, name):
        if t is None:
            t = self._empty(shape, dtype)
            return t, t.data_ptr()
        return t, self._at(t, dtype, shape, name)

    def _packed(self, p, dtype, shape, name):
        """The pointers of a PackedActivation's codes and scales."""
        if tuple(p.shape) != tuple(shape) or p.dtype is not dtype:
            raise ValueError(f"{name} must hold {tuple(shape)} {dtype}, got {tuple(p.shape)} "
                             f"{p.dtype}")
        if p.codes.get_device() != self.device:
            raise ValueError(f"{name} must be on cuda:{self.device}, got {p.codes.device}")
        return p.codes.data_ptr(), p.scales.data_ptr()

    def close(self):
        if getattr(self, "handle", None):
            check(getattr(capi, f"fno_{self._name}_destroy")(self.handle))
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class SandwichNorm(_Plan):
    """Norms around a residual block (``fno_sandwich_*``):

        y = x + s * a * (n2(f) * w2 + b2),    u = n1(y) * w1 + b1

    ``layout`` "grid": fields (batch, channels, points); "tokens": (batch,
    points, channels).  ``params`` is a dict of float32 (channels,) tensors: s,
    w2, w1, and b2, b1 for norm="layer".  ``gate`` "channel" takes float32
    (batch, channels) of up to 65535 samples, "full" a field.
    """

    def __init__(self, channels, points, batch, layout="grid", norm="rms", gate="none",
                 gate_sigmoid=False, eps=1e-5, dtype="f32"):
        d = capi.fno_sandwich_desc_t()
        d.batch, d.points, d.channels = int(batch), int(points), int(channels)
        d.layout, d.norm = capi.LAYOUT_CODES[layout], capi.NORM_CODES[norm]
        d.gate, d.gate_sigmoid = capi.GATE_CODES[gate], int(bool(gate_sigmoid))
        d.eps, d.dtype = float(eps), capi.DTYPE_CODES[dtype]
        self._own(*capi.fno_sandwich_plan(d), "sandwich")
        self.layer, self.gate_kind = norm == "layer", gate
        self.channels = d.channels
        self.torch_dtype = _DTYPES[dtype]
        self.shape = ((d.batch, d.channels, d.points) if layout == "grid"
                      else (d.batch, d.points, d.channels))
        self.gate_shape, self.gate_dtype = (
            ((d.batch, d.channels), torch.float32) if gate == "channel"
            else (self.shape, self.torch_dtype))

    def device_error(self, stream=None) -> int:
        """The sandwich kernels have no device-side waits or checks to report."""
        return capi.FNO_OK

    def _vec(self, params, name, want=True):
        if not want:
            return None
        if name not in params:
            raise ValueError(f"params needs {name!r}")
        return self._at(params[name], torch.float32, (self.channels,), name)

    def _gate(self, gate):
        if self.gate_kind == "none":
            if gate is not None:
                raise ValueError("this plan has no gate")
            return None
        return self._at(gate, self.gate_dtype, self.gate_shape, "gate")

    def _new(self, t, name):
        return self._out(t, self.torch_dtype, self.shape, name)[0]

    def pre(self, x, params, u=None, stream=None):
        """u = n1(x) * w1 + b1: the norm in front of the first block."""
        xp = self._at(x, self.torch_dtype, self.shape, "x")
        u = self._new(u, "u")
        check(capi.fno_sandwich_forward(self.handle, xp, None, None, None, None, None,
                                        self._vec(params, "w1"),
                                        self._vec(params, "b1", self.layer), None, u.data_ptr(),
                                        None, None, self._launch_stream(stream)),
              "fno_sandwich_forward")
        return u

    def forward(self, x, f, params, gate=None, save8=False, want_u=True, y=None, u=None,
                stream=None):
        """(y, u, f8): the stream after the block, the next block's input (None
        unless ``want_u``) and the 8-bit checkpoint of f (None unless
        ``save8``).  ``y`` may be x."""
        dt, shape = self.torch_dtype, self.shape
        xp, fp = self._at(x, dt, shape, "x"), self._at(f, dt, shape, "f")
        gp = self._gate(gate)
        y = self._new(y, "y")
        u = self._new(u, "u") if want_u else None
        f8 = _empty_packed(shape, dt, x.device) if save8 else None
        layer = self.layer
        check(capi.fno_sandwich_forward(
            self.handle, xp, fp, gp, self._vec(params, "s"), self._vec(params, "w2"),
            self._vec(params, "b2", layer), self._vec(params, "w1", want_u),
            self._vec(params, "b1", layer and want_u), y.data_ptr(), _ptr(u),
            f8.codes.data_ptr() if save8 else None, f8.scales.data_ptr() if save8 else None,
            self._launch_stream(stream)), "fno_sandwich_forward")
        return y, u, f8

    __call__ = forward

    def backward(self, y, f, params, dy, du=None, gate=None, stream=None):
        """Gradients as a dict: dx, df, ds, dw2, (db2), (dgate), and with ``du``
        dw1, (db1).  ``f`` is the field, its PackedActivation, or None for the
        backward of ``pre`` (y is then its x).  ``dy`` may be None (zero)."""
        dt, shape, C = self.torch_dtype, self.shape, self.channels
        yp = self._at(y, dt, shape, "y")
        packed = isinstance(f, PackedActivation)
        codes, scales = self._packed(f, dt, shape, "f") if packed else (None, None)
        block = f is not None
        fp = self._at(f, dt, shape, "f") if block and not packed else None
        gp = self._gate(gate) if block else None
        dyp, dup = self._maybe_at(dy, dt, shape, "dy"), self._maybe_at(du, dt, shape, "du")
        layer = self.layer
        out = {"dx": torch.empty_like(y)}
        names = (["s", "w2"] + ["b2"] * layer if block else []) + \
                (["w1"] + ["b1"] * layer if du is not None else [])
        vecs = torch.empty((len(names), (C + 3) // 4 * 4), dtype=torch.float32, device=y.device)
        if block:
            out["df"] = torch.empty_like(y)
            if gp is not None:
                out["dgate"] = torch.empty(self.gate_shape, dtype=self.gate_dtype,
                                           device=y.device)
        for n, row in zip(names, vecs.narrow(1, 0, C).unbind(0)):      # (one view, not five)
            out["d" + n] = row
        ptr = {n: t.data_ptr() for n, t in out.items()}
        check(capi.fno_sandwich_backward(
            self.handle, yp, fp, codes, scales, gp, self._vec(params, "s", block),
            self._vec(params, "w2", block), self._vec(params, "b2", block and layer),
            self._vec(params, "w1", du is not None), dyp, dup, ptr["dx"], ptr.get("df"),
            ptr.get("dgate"), ptr.get("ds"), ptr.get("dw2"), ptr.get("db2"), ptr.get("dw1"),
            ptr.get("db1"), self._workspace(), self._launch_stream(stream)),
              "fno_sandwich_backward")
        return out


class LinearGrad(_Plan):
    """dw (cout, cin) and db (cout) of a 1x1 linear t = W x + b from dy (batch,
    cout, points) and the 8-bit checkpoint of x (batch, cin, points)."""

    def __init__(self, batch, cin, cout, points, dtype="f32"):
        self.torch_dtype = _DTYPES[dtype]
        self.x_shape = (int(batch), int(cin), int(points))
        self.dy_shape = (int(batch), int(cout), int(points))
        self._own(*capi.fno_linear_grad_plan(*self.x_shape[:2], int(cout), int(points),
                                             capi.DTYPE_CODES[dtype]), "linear_grad")

    def backward(self, dy, x8, stream=None):
        dyp = self._at(dy, self.torch_dtype, self.dy_shape, "dy")
        if not isinstance(x8, PackedActivation):
            raise TypeError("x8 must be a PackedActivation")
        codes, scales = self._packed(x8, x8.dtype, self.x_shape, "x8")
        cout, cin = self.dy_shape[1], self.x_shape[1]
        dw = torch.empty((cout, cin), dtype=torch.float32, device=dy.device)
        db = torch.empty((cout,), dtype=torch.float32, device=dy.device)
        check(capi.fno_linear_grad(self.handle, dyp, codes, scales, dw.data_ptr(), db.data_ptr(),
                                   self._workspace(), self._launch_stream(stream)),
              "fno_linear_grad")
        return dw, db

    __call__ = backward


class LinearAttention(_Plan):
    """S_t = e^{log_decay} S_{t-1} + k_t v_t^T, o_t = scale q_t S_t for each
    sequence and query head (``fno_linattn_*``); query heads share key/value
    heads in groups of heads // kv_heads.  States are float32 (batch, heads,
    dk, dv); ``scale`` defaults to dk ** -0.5.  ``backward=True`` prepares the
    workspace of ``backward``."""

    def __init__(self, batch, length, heads, kv_heads, dk, dv, dtype="f32", backward=False):
        b, t, h, g = int(batch), int(length), int(heads), int(kv_heads)
        self.batch, self.heads, self.kv_heads, self.dk, self.dv = b, h, g, int(dk), int(dv)
        self.torch_dtype = _DTYPES[dtype]
        self._own(*capi.fno_linattn_plan(b, t, h, g, int(dk), int(dv), capi.DTYPE_CODES[dtype],
                                         capi.FNO_LINATTN_BACKWARD if backward else 0),
                  "linattn")
        self.q_shape, self.k_shape = (b, t, h, self.dk), (b, t, g, self.dk)
        self.v_shape, self.o_shape = (b, t, g, self.dv), (b, t, h, self.dv)
        self.state_shape = (b, h, self.dk, self.dv)
        self._shapes = (self.q_shape, self.k_shape, self.v_shape)
        self._step_shapes = tuple(s[:1] + s[2:] for s in self._shapes)

    def _qkv(self, q, k, v, log_decay, shapes):
        dt = self.torch_dtype
        return (self._at(q, dt, shapes[0], "q"), self._at(k, dt, shapes[1], "k"),
                self._at(v, dt, shapes[2], "v"),
                self._at(log_decay, torch.float32, (self.heads,), "log_decay"))

    def _scale(self, scale):
        return self.dk ** -0.5 if scale is None else float(scale)

    def forward(self, q, k, v, log_decay, scale=None, lengths=None, state=None, want_state=False,
                out=None, stream=None):
        """(o, final state or None).  ``lengths`` int32 (batch,): tokens of each
        sequence; ``state``: the initial state (None: zero)."""
        ptrs = self._qkv(q, k, v, log_decay, self._shapes)
        lp = self._maybe_at(lengths, torch.int32, (self.batch,), "lengths")
        sp = self._maybe_at(state, torch.float32, self.state_shape, "state")
        out, op = self._out(out, self.torch_dtype, self.o_shape, "out")
        final = (torch.empty(self.state_shape, dtype=torch.float32, device=q.device)
                 if want_state else None)
        check(capi.fno_linattn_forward(self.handle, *ptrs, self._scale(scale), lp, sp,
                                       op, _ptr(final), self._workspace(),
                                       self._launch_stream(stream)), "fno_linattn_forward")
        return out, final

    __call__ = forward

    def backward(self, q, k, v, log_decay, do, scale=None, lengths=None, state=None, dstate=None,
                 stream=None):
        """(dq, dk, dv, gradient of the initial state or None).  ``dstate`` is
        the gradient of the final state (None: zero)."""
        ptrs = self._qkv(q, k, v, log_decay, self._shapes)
        lp = self._maybe_at(lengths, torch.int32, (self.batch,), "lengths")
        sp = self._maybe_at(state, torch.float32, self.state_shape, "state")
        dop = self._at(do, self.torch_dtype, self.o_shape, "do")
        dsp = self._maybe_at(dstate, torch.float32, self.state_shape, "dstate")
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        ds0 = torch.empty_like(state) if state is not None else None
        check(capi.fno_linattn_backward(self.handle, *ptrs, self._scale(scale), lp, sp, dop, dsp,
                                        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(ds0),
                                        self._workspace(), self._launch_stream(stream)),
              "fno_linattn_backward")
        return dq, dk, dv, ds0

    def step(self, q, k, v, log_decay, state, slots=None, new_state=None, scale=None, out=None,
             stream=None):
        """One token for each row: q (batch, heads, dk), k and v (batch,
        kv_heads, ...) -> o (batch, heads, dv).  ``state`` (slots, heads, dk,
        dv) is updated in place unless ``new_state`` is given; ``slots`` int32
        (batch,) says which state a row has (outside: the row is idle)."""
        ptrs = self._qkv(q, k, v, log_decay, self._step_shapes)
        n = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() else 0
        sp = self._at(state, torch.float32, (n,) + self.state_shape[1:], "state")
        tp = self._maybe_at(slots, torch.int32, (self.batch,), "slots")
        np_ = sp if new_state is None else self._at(new_state, torch.float32, state.shape,
                                                    "new_state")
        shape = (self.batch, self.heads, self.dv)
        out, op = self._out(out, self.torch_dtype, shape, "out")
        check(capi.fno_linattn_step(self.handle, *ptrs, self._scale(scale), tp, n, sp, np_,
                                    op, self._launch_stream(stream)), "fno_linattn_step")
        return out


def _int32(v, name):
    v = int(v)
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{name} must fit in 32 bits, got {v}")
    return v


def _code(codes, key, name):
    if key not in codes:
        raise ValueError(f"{name} must be one of {list(codes)}, got {key!r}")
    return codes[key]


class _TimePlan(_Plan):
    """A plan of an operator along time."""

    def device_error(self, stream=None) -> int:
        """These kernels have no device-side waits or checks to report."""
        return capi.FNO_OK

    def _slots(self, state, new_state, slots, dtype, rest):
        """(number of slots, pointers of slots, state and new state) of a step."""
        n = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() else 0
        sp = self._at(state, dtype, (n,) + rest, "state")
        if n < 1:
            raise ValueError("state must have at least one slot")
        if slots is None and n < self.batch:
            raise ValueError(f"state must have {self.batch} slots without slots=, got {n}")
        np_ = sp if new_state is None else self._at(new_state, dtype, (n,) + rest, "new_state")
        return n, self._maybe_at(slots, torch.int32, (self.batch,), "slots"), sp, np_


class Rotary(_TimePlan):
    """Rotary positions (``fno_rotary_*``): the pairs in the first ``rotary_dim``
    elements (default: all) of every head of q (batch, length, heads, dim) and k
    (batch, length, kv_heads, dim; none for kv_heads=0) turned by position times
    base ** (-2 i / rotary_dim).  ``layout`` "half" pairs elements i and i +
    rotary_dim / 2, "interleaved" 2 i and 2 i + 1.  ``scaling`` for contexts longer
    than those trained on: None, ("linear", factor), ("base", factor) or ("ramp",
    factor, original length, fast, slow)."""

    def __init__(self, batch, length, heads, kv_heads, dim, rotary_dim=None, layout="half",
                 base=10000.0, scaling=None, dtype="f32"):
        d = capi.fno_rotary_desc_t()
        d.batch, d.length = int(batch), int(length)
        d.heads, d.kv_heads = _int32(heads, "heads"), _int32(kv_heads, "kv_heads")
        d.dim = _int32(dim, "dim")
        d.rotary_dim = d.dim if rotary_dim is None else _int32(rotary_dim, "rotary_dim")
        d.layout = _code(capi.ROTARY_LAYOUT_CODES, layout, "layout")
        kind, *values = ("none",) if scaling is None else tuple(scaling)
        d.scaling = _code(capi.ROTARY_SCALING_CODES, kind, "scaling")
        names = {"none": (), "linear": ("factor",), "base": ("factor",),
                 "ramp": ("factor", "original", "fast", "slow")}[kind]
        if len(values) != len(names):
            raise ValueError(f"scaling {kind!r} takes {names}, got {tuple(values)}")
        for name, v in zip(names, values):
            setattr(d, name, float(v))
        d.base, d.dtype = float(base), _code(capi.DTYPE_CODES, dtype, "dtype")
        self._own(*capi.fno_rotary_plan(d), "rotary", workspace=False)
        self.torch_dtype = _DTYPES[dtype]
        self.batch, self.length = d.batch, d.length
        self.q_shape = (d.batch, d.length, d.heads, d.dim)
        self.k_shape = (d.batch, d.length, d.kv_heads, d.dim) if d.kv_heads else None

    def _apply(self, q, k, positions, offsets, q_out, k_out, transpose, stream):
        dt = self.torch_dtype
        qp = self._at(q, dt, self.q_shape, "q")
        q_out, qop = self._out(q_out, dt, self.q_shape, "q_out")
        kp = kop = None
        if self.k_shape is None:
            if k is not None or k_out is not None:
                raise ValueError("this plan has no k")
        else:
            kp = self._at(k, dt, self.k_shape, "k")
            k_out, kop = self._out(k_out, dt, self.k_shape, "k_out")
        if positions is not None and offsets is not None:
            raise ValueError("positions and offsets exclude each other")
        pp = self._maybe_at(positions, torch.int32, (self.batch, self.length), "positions")
        op = self._maybe_at(offsets, torch.int32, (self.batch,), "offsets")
        check(capi.fno_rotary_apply(self.handle, qp, kp, pp, op, transpose, qop, kop,
                                    self._launch_stream(stream)), "fno_rotary_apply")
        return q_out, k_out

    def forward(self, q, k=None, positions=None, offsets=None, q_out=None, k_out=None,
                stream=None):
        """(q, k) turned.  Token t of sequence b is at ``positions[b, t]`` (int32), at
        ``offsets[b]`` + t, or at t.  ``q_out`` and ``k_out`` may be q and k."""
        return self._apply(q, k, positions, offsets, q_out, k_out, 0, stream)

    __call__ = forward

    def backward(self, dq, dk=None, positions=None, offsets=None, q_out=None, k_out=None,
                 stream=None):
        """Gradients of q and k from those of ``forward``'s outputs."""
        return self._apply(dq, dk, positions, offsets, q_out, k_out, 1, stream)


class CausalConv(_TimePlan):
    """y_t = act(bias + sum_j w[:, j] x_{t - width + 1 + j}) for each channel of x
    (batch, length, channels) (``fno_causal_conv_*``).  w (channels, width) and bias
    (channels,) are float32; ``act`` is "silu" or "none"; states (batch, width - 1,
    channels) of the storage type hold the last inputs, oldest first.
    ``backward=True`` prepares the workspace of ``backward``."""

    def __init__(self, batch, length, channels, width, act="silu", dtype="f32", backward=False):
        self.batch, self.length = int(batch), int(length)
        self.channels, self.width = _int32(channels, "channels"), _int32(width, "width")
        self._own(*capi.fno_causal_conv_plan(
            self.batch, self.length, self.channels, self.width,
            _code(capi.ACT_CODES, act, "act"), _code(capi.DTYPE_CODES, dtype, "dtype"),
            capi.FNO_CAUSAL_CONV_BACKWARD if backward else 0), "causal_conv")
        self.torch_dtype = _DTYPES[dtype]
        self.x_shape = (self.batch, self.length, self.channels)
        self.state_shape = (self.batch, self.width - 1, self.channels)

    def _inputs(self, x, w, bias, lengths, state):
        return (self._at(x, self.torch_dtype, self.x_shape, "x"),
                self._at(w, torch.float32, (self.channels, self.width), "w"),
                self._maybe_at(bias, torch.float32, (self.channels,), "bias"),
                self._maybe_at(lengths, torch.int32, (self.batch,), "lengths"),
                self._maybe_at(state, self.torch_dtype, self.state_shape, "state"))

    def forward(self, x, w, bias=None, lengths=None, state=None, want_state=False, out=None,
                stream=None):
        """(y, final state or None).  ``lengths`` int32 (batch,): tokens of each
        sequence; ``state``: the inputs in front of the first token (None: zeros)."""
        ptrs = self._inputs(x, w, bias, lengths, state)
        out, op = self._out(out, self.torch_dtype, self.x_shape, "out")
        final = self._empty(self.state_shape, self.torch_dtype) if want_state else None
        check(capi.fno_causal_conv_forward(self.handle, *ptrs, op, _ptr(final),
                                           self._launch_stream(stream)),
              "fno_causal_conv_forward")
        return out, final

    __call__ = forward

    def backward(self, x, w, dy, bias=None, lengths=None, state=None, dstate=None, stream=None):
        """(dx, dw, dbias or None, gradient of the initial state or None).  ``dstate`` is
        the gradient of the final state (None: zero)."""
        ptrs = self._inputs(x, w, bias, lengths, state)
        dyp = self._at(dy, self.torch_dtype, self.x_shape, "dy")
        dsp = self._maybe_at(dstate, self.torch_dtype, self.state_shape, "dstate")
        dx = self._empty(self.x_shape, self.torch_dtype)
        dw = self._empty((self.channels, self.width), torch.float32)
        db = None if bias is None else self._empty((self.channels,), torch.float32)
        ds0 = None if state is None else self._empty(self.state_shape, self.torch_dtype)
        check(capi.fno_causal_conv_backward(
            self.handle, *ptrs, dyp, dsp, dx.data_ptr(), dw.data_ptr(), _ptr(db), _ptr(ds0),
            self._workspace(), self._launch_stream(stream)), "fno_causal_conv_backward")
        return dx, dw, db, ds0

    def step(self, x, w, state, bias=None, slots=None, new_state=None, out=None, stream=None):
        """One token for each row: x (batch, channels) -> y (batch, channels).  ``state``
        (slots, width - 1, channels) is updated in place unless ``new_state`` is given;
        ``slots`` int32 (batch,) says which state a row has (outside: the row is idle)."""
        shape = (self.batch, self.channels)
        xp = self._at(x, self.torch_dtype, shape, "x")
        wp = self._at(w, torch.float32, (self.channels, self.width), "w")
        bp = self._maybe_at(bias, torch.float32, (self.channels,), "bias")
        n, tp, sp, np_ = self._slots(state, new_state, slots, self.torch_dtype,
                                     self.state_shape[1:])
        out, op = self._out(out, self.torch_dtype, shape, "out")
        check(capi.fno_causal_conv_step(self.handle, xp, wp, bp, tp, n, sp, np_, op,
                                        self._launch_stream(stream)), "fno_causal_conv_step")
        return out


class SelectiveScan(_TimePlan):
    """The selective state space scan (``fno_scan_*``): with d = softplus(dt + dt_bias)
    (or the sum itself for softplus=False),

        h_t = e^{d_t A} h_{t-1} + d_t x_t B_t,   y_t = (C_t h_t + D x_t) silu(z_t)

    for each channel of x, dt, z (batch, length, channels), whose group shares B and C
    (batch, length, groups, states).  A (channels, states), D and dt_bias (channels,)
    are float32, states h (batch, channels, states) float32; D, z, dt_bias may be None.
    ``backward=True`` prepares the workspace of ``backward``."""

    def __init__(self, batch, length, channels, states, groups=1, softplus=True, dtype="f32",
                 backward=False):
        d = capi.fno_scan_desc_t()
        d.batch, d.length = int(batch), int(length)
        d.channels, d.states = _int32(channels, "channels"), _int32(states, "states")
        d.groups, d.softplus = _int32(groups, "groups"), int(bool(softplus))
        d.dtype = _code(capi.DTYPE_CODES, dtype, "dtype")
        d.flags = capi.FNO_SCAN_BACKWARD if backward else 0
        self._own(*capi.fno_scan_plan(d), "scan")
        self.torch_dtype = _DTYPES[dtype]
        self.batch, self.length, self.channels = d.batch, d.length, d.channels
        self.a_shape = (d.channels, d.states)
        self.x_shape = (d.batch, d.length, d.channels)
        self.b_shape = (d.batch, d.length, d.groups, d.states)
        self.state_shape = (d.batch, d.channels, d.states)

    def _inputs(self, x, dt, A, B, C, D, z, dt_bias, row, bc):
        at, maybe, t = self._at, self._maybe_at, self.torch_dtype
        f32, c = torch.float32, (self.channels,)
        return (at(x, t, row, "x"), at(dt, t, row, "dt"), at(A, f32, self.a_shape, "A"),
                at(B, t, bc, "B"), at(C, t, bc, "C"), maybe(D, f32, c, "D"),
                maybe(z, t, row, "z"), maybe(dt_bias, f32, c, "dt_bias"))

    def _sequence(self, x, dt, A, B, C, D, z, dt_bias, lengths, state):
        return (*self._inputs(x, dt, A, B, C, D, z, dt_bias, self.x_shape, self.b_shape),
                self._maybe_at(lengths, torch.int32, (self.batch,), "lengths"),
                self._maybe_at(state, torch.float32, self.state_shape, "state"))

    def forward(self, x, dt, A, B, C, D=None, z=None, dt_bias=None, lengths=None, state=None,
                want_state=False, out=None, stream=None):
        """(y, final state or None).  ``lengths`` int32 (batch,): tokens of each
        sequence; ``state``: the initial state (None: zero)."""
        ptrs = self._sequence(x, dt, A, B, C, D, z, dt_bias, lengths, state)
        out, op = self._out(out, self.torch_dtype, self.x_shape, "out")
        final = self._empty(self.state_shape, torch.float32) if want_state else None
        check(capi.fno_scan_forward(self.handle, *ptrs, op, _ptr(final), self._workspace(),
                                    self._launch_stream(stream)), "fno_scan_forward")
        return out, final

    __call__ = forward

    def backward(self, x, dt, A, B, C, dy, D=None, z=None, dt_bias=None, lengths=None, state=None,
                 dstate=None, stream=None):
        """Gradients as a dict: dx, ddt, dA, dB, dC, and where their input was given dD,
        dz, ddt_bias, dstate (of the initial state).  ``dstate=`` is the gradient of the
        final state (None: zero)."""
        ptrs = self._sequence(x, dt, A, B, C, D, z, dt_bias, lengths, state)
        dyp = self._at(dy, self.torch_dtype, self.x_shape, "dy")
        dsp = self._maybe_at(dstate, torch.float32, self.state_shape, "dstate")
        t, f32 = self.torch_dtype, torch.float32
        shapes = {"dx": (self.x_shape, t), "ddt": (self.x_shape, t), "dA": (self.a_shape, f32),
                  "dB": (self.b_shape, t), "dC": (self.b_shape, t)}
        if D is not None:
            shapes["dD"] = ((self.channels,), f32)
        if z is not None:
            shapes["dz"] = (self.x_shape, t)
        if dt_bias is not None:
            shapes["ddt_bias"] = ((self.channels,), f32)
        if state is not None:
            shapes["dstate"] = (self.state_shape, f32)
        out = {name: self._empty(*s) for name, s in shapes.items()}
        p = {name: v.data_ptr() for name, v in out.items()}
        check(capi.fno_scan_backward(
            self.handle, *ptrs, dyp, dsp, p["dx"], p["ddt"], p["dA"], p["dB"], p["dC"],
            p.get("dD"), p.get("dz"), p.get("ddt_bias"), p.get("dstate"), self._workspace(),
            self._launch_stream(stream)), "fno_scan_backward")
        return out

    def step(self, x, dt, A, B, C, state, D=None, z=None, dt_bias=None, slots=None,
             new_state=None, out=None, stream=None):
        """One token for each row: x, dt, z (batch, channels), B, C (batch, groups,
        states) -> y (batch, channels).  ``state`` (slots, channels, states) is updated in
        place unless ``new_state`` is given; ``slots`` int32 (batch,) says which state a
        row has (outside: the row is idle)."""
        shape = (self.batch, self.channels)
        ptrs = self._inputs(x, dt, A, B, C, D, z, dt_bias, shape,
                            (self.batch,) + self.b_shape[2:])
        n, tp, sp, np_ = self._slots(state, new_state, slots, torch.float32, self.a_shape)
        out, op = self._out(out, self.torch_dtype, shape, "out")
        check(capi.fno_scan_step(self.handle, *ptrs, tp, n, sp, np_, op,
                                 self._launch_stream(stream)), "fno_scan_step")
        return out
