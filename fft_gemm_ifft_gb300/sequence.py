"""The sequence and training operators (C ABI: ``include/fno_ops.h``).

``SandwichNorm``      norms before and after a block with its gate, residual
                      scale and residual sum, and their gradients
``pack_activation`` / ``PackedActivation``
                      activation checkpoints in 8 bits
``LinearGrad``        weight and bias gradient of a 1x1 linear from one
``LinearAttention``   linear attention with a decay for each head: prompts,
                      single tokens, gradients

As in the rest of the package, the classes marshal arguments: a plan, a
workspace from torch, tensor pointers and the current stream.  A plan object
holds one workspace, so calls on it have to be ordered (one stream).  A call with
``stream=`` is launched there and allocates its results on the current stream:
that stream has to wait for the current one's work before the call, and the
current one for it before the results are used or dropped.
"""
from __future__ import annotations

import torch

from . import _require, _stream_handle, capi, check

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_CODES = {torch.float32: capi.FNO_F32, torch.float16: capi.FNO_F16,
          torch.bfloat16: capi.FNO_BF16}
GROUP = capi.FNO_ACT8_GROUP


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, t):
    """The handle of ``stream``, or of the current stream of t's device (by the
    raw query where torch has it: the call is most of a small operator's cost)."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(t.device.index)
    return _stream_handle(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _field(t, dtype, shape, name):
    """t's pointer, once its type, shape and layout are those wanted."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.shape == shape
            and t.is_contiguous()):
        _require(t, dtype, shape, name)
    return t.data_ptr()


def _maybe(t, dtype, shape, name):
    return None if t is None else _field(t, dtype, shape, name)


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
        _field(codes, torch.int8, codes.shape, "codes")
        _field(scales, torch.float32, codes.shape[:-1] + (-(-codes.shape[-1] // GROUP),),
               "scales")
        self.codes, self.scales, self.dtype = codes, scales, dtype
        self.shape = codes.shape

    def _rows(self):
        cols = self.shape[-1]
        return self.codes.numel() // cols, cols

    def values(self, out=None, stream=None):
        """The values that the codes stand for, in the storage type."""
        if out is None:
            out = torch.empty(self.shape, dtype=self.dtype, device=self.codes.device)
        ptr = _field(out, self.dtype, self.shape, "out")
        rows, cols = self._rows()
        check(capi.fno_act8_unpack(rows, cols, _CODES[self.dtype], self.codes.data_ptr(),
                                   self.scales.data_ptr(), ptr, _stream(stream, out)),
              "fno_act8_unpack")
        return out

    def gelu_backward(self, dy, out=None, stream=None):
        """dy * GELU'(values); ``out`` may be dy."""
        dyp = _field(dy, self.dtype, self.shape, "dy")
        if out is None:
            out = torch.empty_like(dy)
        ptr = _field(out, self.dtype, self.shape, "out")
        rows, cols = self._rows()
        check(capi.fno_act8_gelu_backward(rows, cols, _CODES[self.dtype], self.codes.data_ptr(),
                                          self.scales.data_ptr(), dyp, ptr,
                                          _stream(stream, dy)), "fno_act8_gelu_backward")
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
    ptr = _field(x, x.dtype, x.shape, "x")
    p = _empty_packed(x.shape, x.dtype, x.device)
    rows, cols = p._rows()
    check(capi.fno_act8_pack(rows, cols, _CODES[x.dtype], ptr, p.codes.data_ptr(),
                             p.scales.data_ptr(), _stream(stream, x)), "fno_act8_pack")
    return p


class _Plan:
    """A plan handle with its workspace."""

    def _own(self, status, handle, name):
        check(status, f"fno_{name}_plan")
        self.handle, self._name = handle, name
        st, self.workspace_bytes = getattr(capi, f"fno_{name}_workspace_size")(handle)
        check(st)
        self.workspace = None

    def _workspace(self):
        """Allocated at the first call that needs it, then kept."""
        if self.workspace is None and self.workspace_bytes:
            self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device="cuda")
        return _ptr(self.workspace)

    def device_error(self, stream=None) -> int:
        return getattr(capi, f"fno_{self._name}_get_device_error")(self.handle,
                                                                   _stream_handle(stream))

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
        return _field(params[name], torch.float32, (self.channels,), name)

    def _gate(self, gate):
        if self.gate_kind == "none":
            if gate is not None:
                raise ValueError("this plan has no gate")
            return None
        return _field(gate, self.gate_dtype, self.gate_shape, "gate")

    def _new(self, t, name):
        if t is None:
            return torch.empty(self.shape, dtype=self.torch_dtype, device="cuda")
        _require(t, self.torch_dtype, self.shape, name)
        return t

    def pre(self, x, params, u=None, stream=None):
        """u = n1(x) * w1 + b1: the norm in front of the first block."""
        xp = _field(x, self.torch_dtype, self.shape, "x")
        u = self._new(u, "u")
        check(capi.fno_sandwich_forward(self.handle, xp, None, None, None, None, None,
                                        self._vec(params, "w1"),
                                        self._vec(params, "b1", self.layer), None, u.data_ptr(),
                                        None, None, _stream(stream, x)),
              "fno_sandwich_forward")
        return u

    def forward(self, x, f, params, gate=None, save8=False, want_u=True, y=None, u=None,
                stream=None):
        """(y, u, f8): the stream after the block, the next block's input (None
        unless ``want_u``) and the 8-bit checkpoint of f (None unless
        ``save8``).  ``y`` may be x."""
        dt, shape = self.torch_dtype, self.shape
        xp, fp = _field(x, dt, shape, "x"), _field(f, dt, shape, "f")
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
            _stream(stream, x)), "fno_sandwich_forward")
        return y, u, f8

    __call__ = forward

    def backward(self, y, f, params, dy, du=None, gate=None, stream=None):
        """Gradients as a dict: dx, df, ds, dw2, (db2), (dgate), and with ``du``
        dw1, (db1).  ``f`` is the field, its PackedActivation, or None for the
        backward of ``pre`` (y is then its x).  ``dy`` may be None (zero)."""
        dt, shape, C = self.torch_dtype, self.shape, self.channels
        yp = _field(y, dt, shape, "y")
        packed = isinstance(f, PackedActivation)
        if packed and (tuple(f.shape) != shape or f.dtype != dt):
            raise ValueError(f"f must hold {shape} {dt}, got {tuple(f.shape)} {f.dtype}")
        block = f is not None
        fp = _field(f, dt, shape, "f") if block and not packed else None
        gp = self._gate(gate) if block else None
        dyp, dup = _maybe(dy, dt, shape, "dy"), _maybe(du, dt, shape, "du")
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
            self.handle, yp, fp, f.codes.data_ptr() if packed else None,
            f.scales.data_ptr() if packed else None, gp, self._vec(params, "s", block),
            self._vec(params, "w2", block), self._vec(params, "b2", block and layer),
            self._vec(params, "w1", du is not None), dyp, dup, ptr["dx"], ptr.get("df"),
            ptr.get("dgate"), ptr.get("ds"), ptr.get("dw2"), ptr.get("db2"), ptr.get("dw1"),
            ptr.get("db1"), self._workspace(), _stream(stream, y)), "fno_sandwich_backward")
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
        dyp = _field(dy, self.torch_dtype, self.dy_shape, "dy")
        if not isinstance(x8, PackedActivation):
            raise TypeError("x8 must be a PackedActivation")
        if tuple(x8.shape) != self.x_shape:
            raise ValueError(f"x8 must have shape {self.x_shape}, got {tuple(x8.shape)}")
        cout, cin = self.dy_shape[1], self.x_shape[1]
        dw = torch.empty((cout, cin), dtype=torch.float32, device=dy.device)
        db = torch.empty((cout,), dtype=torch.float32, device=dy.device)
        check(capi.fno_linear_grad(self.handle, dyp, x8.codes.data_ptr(), x8.scales.data_ptr(),
                                   dw.data_ptr(), db.data_ptr(), self._workspace(),
                                   _stream(stream, dy)), "fno_linear_grad")
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
        return (_field(q, dt, shapes[0], "q"), _field(k, dt, shapes[1], "k"),
                _field(v, dt, shapes[2], "v"),
                _field(log_decay, torch.float32, (self.heads,), "log_decay"))

    def _scale(self, scale):
        return self.dk ** -0.5 if scale is None else float(scale)

    def forward(self, q, k, v, log_decay, scale=None, lengths=None, state=None, want_state=False,
                out=None, stream=None):
        """(o, final state or None).  ``lengths`` int32 (batch,): tokens of each
        sequence; ``state``: the initial state (None: zero)."""
        ptrs = self._qkv(q, k, v, log_decay, self._shapes)
        lp = _maybe(lengths, torch.int32, (self.batch,), "lengths")
        sp = _maybe(state, torch.float32, self.state_shape, "state")
        if out is None:
            out = torch.empty(self.o_shape, dtype=self.torch_dtype, device=q.device)
        op = _field(out, self.torch_dtype, self.o_shape, "out")
        final = (torch.empty(self.state_shape, dtype=torch.float32, device=q.device)
                 if want_state else None)
        check(capi.fno_linattn_forward(self.handle, *ptrs, self._scale(scale), lp, sp,
                                       op, _ptr(final), self._workspace(),
                                       _stream(stream, q)), "fno_linattn_forward")
        return out, final

    __call__ = forward

    def backward(self, q, k, v, log_decay, do, scale=None, lengths=None, state=None, dstate=None,
                 stream=None):
        """(dq, dk, dv, gradient of the initial state or None).  ``dstate`` is
        the gradient of the final state (None: zero)."""
        ptrs = self._qkv(q, k, v, log_decay, self._shapes)
        lp = _maybe(lengths, torch.int32, (self.batch,), "lengths")
        sp = _maybe(state, torch.float32, self.state_shape, "state")
        dop = _field(do, self.torch_dtype, self.o_shape, "do")
        dsp = _maybe(dstate, torch.float32, self.state_shape, "dstate")
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        ds0 = torch.empty_like(state) if state is not None else None
        check(capi.fno_linattn_backward(self.handle, *ptrs, self._scale(scale), lp, sp, dop, dsp,
                                        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(ds0),
                                        self._workspace(), _stream(stream, q)),
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
        sp = _field(state, torch.float32, (n,) + self.state_shape[1:], "state")
        tp = _maybe(slots, torch.int32, (self.batch,), "slots")
        np_ = sp if new_state is None else _field(new_state, torch.float32, state.shape,
                                                  "new_state")
        shape = (self.batch, self.heads, self.dv)
        if out is None:
            out = torch.empty(shape, dtype=self.torch_dtype, device=q.device)
        op = _field(out, self.torch_dtype, shape, "out")
        check(capi.fno_linattn_step(self.handle, *ptrs, self._scale(scale), tp, n, sp, np_,
                                    op, _stream(stream, q)), "fno_linattn_step")
        return out
