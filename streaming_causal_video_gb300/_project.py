"""ctypes binding of the operators in include/sdv2_project.h (argument marshalling only)."""
import ctypes

import torch

from . import _binding as _b
from ._block import _FP, _TYPE, _U8, _Config, _current_device, _Operands, _stream

NO_ACTIVATION, GELU = 0, 1     # sdv2_activation

# Every symbol that include/sdv2_project.h declares.
PROJECT_EXPORTS = ["sdv2_mx4_codes_bytes", "sdv2_mx4_scales_bytes", "sdv2_mx4_quantize", "sdv2_mx4_dequantize",
                   "sdv2_mx4_workspace_bytes", "sdv2_mx4_workspace_init", "sdv2_mx4_product", "sdv2_axes_rope",
                   "sdv2_axes_rope_backward"]

_i32, _i64, _f64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_double, ctypes.c_void_p


class Mx4Config(_Config):
    """Mirror of sdv2_mx4_cfg."""
    _fields_ = [("rows", _i64), ("cols", _i64), ("x_dtype", _i32), ("transposed", _i32), ("x_row_stride", _i64)]

    def _derive(self):
        """Bytes of codes and of scales; shape, strides, type and bytes of x."""
        shape = (self.cols, self.rows) if self.transposed else (self.rows, self.cols)
        kind, size = _TYPE.get(self.x_dtype, (None, 4))
        stride = self.x_row_stride or shape[1]
        return mx4_codes_bytes(self), mx4_scales_bytes(self), (kind, shape, (stride, 1), _b._row_span(shape[0], stride, shape[1], size))


class Mx4ProductConfig(_Config):
    """Mirror of sdv2_mx4_product_cfg."""
    _fields_ = [("rows", _i64), ("cols", _i64), ("depth", _i64), ("out_dtype", _i32), ("activation", _i32), ("out_row_stride", _i64)]

    def _derive(self):
        """Bytes of codes and scales of a and of b, of the bias and of the workspace; type, shape, strides and bytes of out."""
        a, b = (Mx4Config.make(rows=n, cols=self.depth) for n in (self.rows, self.cols))
        kind, size = _TYPE.get(self.out_dtype, (None, 4))
        stride = self.out_row_stride or self.cols
        return (mx4_codes_bytes(a), mx4_scales_bytes(a), mx4_codes_bytes(b), mx4_scales_bytes(b), max(self.cols, 0) * 4,
                mx4_workspace_bytes(self), (kind, (self.rows, self.cols), (stride, 1), _b._row_span(self.rows, stride, self.cols, size)))


class RopeStrides(ctypes.Structure):
    """Mirror of sdv2_rope_strides."""
    _fields_ = [("token_stride", _i64), ("head_stride", _i64), ("batch_stride", _i64)]


class AxesRopeConfig(_Config):
    """Mirror of sdv2_axes_rope_cfg.  make() takes dims and scale as sequences of one value per axis, and strides as
    mappings of token_stride, head_stride and batch_stride.  To change strides later, assign a new RopeStrides."""
    _fields_ = [("batch", _i32), ("heads", _i32), ("kv_heads", _i32), ("head_dim", _i32), ("tokens", _i64), ("dtype", _i32),
                ("axes", _i32), ("dims", _i32 * 4), ("halves", _i32), ("shared_positions", _i32), ("base", _f64),
                ("scale", _f64 * 4), ("q_in", RopeStrides), ("q_out", RopeStrides), ("k_in", RopeStrides), ("k_out", RopeStrides)]

    @classmethod
    def make(cls, dims=(), scale=(), base=10000.0, **kw):
        dims, scale = [int(d) for d in dims], [float(s) for s in scale]
        if not 1 <= len(dims) <= 4 or len(scale) not in (0, len(dims)):
            raise ValueError("dims must name one to four axes, and scale none or each of them")
        for name in ("q_in", "q_out", "k_in", "k_out"):
            if name in kw:
                kw[name] = RopeStrides(**kw[name])
        return super().make(axes=len(dims), dims=(_i32 * 4)(*dims), scale=(_f64 * 4)(*scale), base=base, **kw)

    def _derive(self):
        """Type; shape, strides and bytes of q in, q out, k in and k out; bytes of the positions."""
        kind, size = _TYPE.get(self.dtype, (None, 4))

        def operand(heads, s):
            hd = s.head_stride or self.head_dim
            tok = s.token_stride or heads * self.head_dim
            batch = s.batch_stride or max(self.tokens * tok, heads * hd)
            span = 0
            if min(self.batch, self.tokens, heads) > 0:
                span = size * ((self.batch - 1) * batch + (self.tokens - 1) * tok + (heads - 1) * hd + self.head_dim)
            return (self.batch, self.tokens, heads, self.head_dim), (batch, tok, hd, 1), span
        places = max(self.tokens, 0) * (1 if self.shared_positions else max(self.batch, 0))
        return (kind, operand(self.heads, self.q_in), operand(self.heads, self.q_out), operand(self.kv_heads, self.k_in),
                operand(self.kv_heads, self.k_out), places * max(self.axes, 0) * 4)


_Tensor = torch.Tensor


def _here(t):
    """The current device if t is a tensor on it, else a number that is no tensor's device."""
    if t.__class__ is _Tensor:
        d = t.get_device()
        if d >= 0 and d == _current_device():
            return d
    return -2


def _buffer(t, name, dtype, nbytes, device):
    """Pointer of a dense tensor of at least nbytes bytes.  What is as it should be is seen at once; anything else goes to
    the checks that say what is wrong with it (or find that nothing is)."""
    if t.__class__ is _Tensor and t.dtype is dtype and t.get_device() == device and t.nbytes >= nbytes and t.is_contiguous():
        return t.data_ptr()
    return _Operands()(t, name, dtype, nbytes, True)


def _view(t, name, kind, shape, strides, nbytes, device):
    """The same for a view of a configuration's shape and strides."""
    if t.__class__ is _Tensor and t.dtype is kind and t.get_device() == device and t.shape == shape and t.stride() == strides:
        return t.data_ptr()
    return _Operands().view(t, name, kind, shape, strides, nbytes)


_LIB = None


def _lib():
    global _LIB
    L = _b.lib()
    if _LIB is not L:
        mx4p, prodp, ropep = ctypes.POINTER(Mx4Config), ctypes.POINTER(Mx4ProductConfig), ctypes.POINTER(AxesRopeConfig)
        types = {"sdv2_mx4_codes_bytes": (ctypes.c_size_t, [mx4p]),
                 "sdv2_mx4_scales_bytes": (ctypes.c_size_t, [mx4p]),
                 "sdv2_mx4_quantize": (ctypes.c_int, [mx4p] + [_vp] * 4),
                 "sdv2_mx4_dequantize": (ctypes.c_int, [mx4p] + [_vp] * 4),
                 "sdv2_mx4_workspace_bytes": (ctypes.c_size_t, [prodp]),
                 "sdv2_mx4_workspace_init": (ctypes.c_int, [prodp, _vp, _vp]),
                 "sdv2_mx4_product": (ctypes.c_int, [prodp] + [_vp] * 8),
                 "sdv2_axes_rope": (ctypes.c_int, [ropep] + [_vp] * 6),
                 "sdv2_axes_rope_backward": (ctypes.c_int, [ropep] + [_vp] * 6)}
        for name, (res, args) in types.items():
            getattr(L, name).restype = res
            getattr(L, name).argtypes = args
        _LIB = L
    return _LIB


def mx4_codes_bytes(cfg: Mx4Config) -> int:
    return _lib().sdv2_mx4_codes_bytes(ctypes.byref(cfg))


def mx4_scales_bytes(cfg: Mx4Config) -> int:
    return _lib().sdv2_mx4_scales_bytes(ctypes.byref(cfg))


def mx4_workspace_bytes(cfg: Mx4ProductConfig) -> int:
    return _lib().sdv2_mx4_workspace_bytes(ctypes.byref(cfg))


def mx4_workspace_init(cfg, ws, stream=None):
    _b._check(_lib().sdv2_mx4_workspace_init(ctypes.byref(cfg), _Operands()(ws, "ws", _U8, 256), _stream(stream)),
              "sdv2_mx4_workspace_init")


def mx4_quantize(cfg, x, codes, scales, stream=None):
    """x: [rows][cols] (transposed: [cols][rows]) of cfg.x_dtype; codes, scales: uint8, of mx4_codes_bytes(cfg) and
    mx4_scales_bytes(cfg) bytes."""
    dev = _here(x)
    nc, ns, plan = cfg.derived()
    status = _lib().sdv2_mx4_quantize(cfg, _view(x, "x", *plan, dev), _buffer(codes, "codes", _U8, nc, dev),
                                      _buffer(scales, "scales", _U8, ns, dev), _stream(stream))
    if status:
        _b._check(status, "sdv2_mx4_quantize")


def mx4_dequantize(cfg, codes, scales, y, stream=None):
    """y: [rows][cols] of cfg.x_dtype, the values that codes and scales stand for."""
    dev = _here(y)
    nc, ns, plan = cfg.derived()
    status = _lib().sdv2_mx4_dequantize(cfg, _buffer(codes, "codes", _U8, nc, dev), _buffer(scales, "scales", _U8, ns, dev),
                                        _view(y, "y", *plan, dev), _stream(stream))
    if status:
        _b._check(status, "sdv2_mx4_dequantize")


def mx4_product(cfg, a_codes, a_scales, b_codes, b_scales, out, ws, bias=None, stream=None):
    """out [rows][cols] = act(a b^T + bias) of matrices that mx4_quantize wrote: a of `rows` and b of `cols` rows, both of
    `depth` columns; bias: fp32 [cols]; ws: mx4_workspace_bytes(cfg) bytes."""
    dev = _here(out)
    ac, asc, bc, bsc, nb, nw, plan = cfg.derived()
    status = _lib().sdv2_mx4_product(cfg, _buffer(a_codes, "a_codes", _U8, ac, dev), _buffer(a_scales, "a_scales", _U8, asc, dev),
                                     _buffer(b_codes, "b_codes", _U8, bc, dev), _buffer(b_scales, "b_scales", _U8, bsc, dev),
                                     None if bias is None else _buffer(bias, "bias", _FP, nb, dev), _view(out, "out", *plan, dev),
                                     _buffer(ws, "ws", _U8, nw, dev), _stream(stream))
    if status:
        _b._check(status, "sdv2_mx4_product")


def _turn(cfg, positions, q, q_new, k, k_new, backward, stream):
    dev = _here(q)
    kind, q_in, q_out, k_in, k_out, np = cfg.derived()
    if backward:
        q_in, q_out, k_in, k_out = q_out, q_in, k_out, k_in
        names, call = ("dq_out", "dq", "dk_out", "dk"), _lib().sdv2_axes_rope_backward
    else:
        names, call = ("q", "q_out", "k", "k_out"), _lib().sdv2_axes_rope
    pk = pk_new = None
    if cfg.kv_heads:
        pk, pk_new = _view(k, names[2], kind, *k_in, dev), _view(k_new, names[3], kind, *k_out, dev)
    status = call(cfg, _buffer(positions, "positions", torch.int32, np, dev), _view(q, names[0], kind, *q_in, dev),
                  _view(q_new, names[1], kind, *q_out, dev), pk, pk_new, _stream(stream))
    if status:
        _b._check(status, "sdv2_axes_rope_backward" if backward else "sdv2_axes_rope")


def axes_rope(cfg, positions, q, q_out, k=None, k_out=None, stream=None):
    """q, q_out: [batch][tokens][heads][head_dim], k, k_out: [batch][tokens][kv_heads][head_dim] with cfg's strides;
    positions: int32 [batch][tokens][axes], or [tokens][axes] shared by the batch."""
    _turn(cfg, positions, q, q_out, k, k_out, False, stream)


def axes_rope_backward(cfg, positions, dq_out, dq, dk_out=None, dk=None, stream=None):
    """Gradients dq (cfg.q_in's strides) and dk (cfg.k_in's) from those of axes_rope's results."""
    _turn(cfg, positions, dq_out, dq, dk_out, dk, True, stream)
