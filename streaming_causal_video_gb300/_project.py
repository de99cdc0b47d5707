"""ctypes binding of the operators in include/sdv2_project.h (argument marshalling only)."""
import ctypes

import torch

from . import _binding as _b
from ._block import _FP, _TYPE, _U8, _Config, _current_device, _Operands, _raw_stream, _stream

_I32 = torch.int32

NO_ACTIVATION, GELU = 0, 1     # sdv2_activation

# Every symbol that include/sdv2_project.h declares.
PROJECT_EXPORTS = ["sdv2_mx4_codes_bytes", "sdv2_mx4_scales_bytes", "sdv2_mx4_quantize", "sdv2_mx4_dequantize",
                   "sdv2_mx4_workspace_bytes", "sdv2_mx4_workspace_init", "sdv2_mx4_product", "sdv2_debug_mx4_plan",
                   "sdv2_axes_rope", "sdv2_axes_rope_backward"]

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
    """Mirror of sdv2_rope_strides.  Those in a configuration change as a whole, so that what is derived from them does as well."""
    _fields_ = [("token_stride", _i64), ("head_stride", _i64), ("batch_stride", _i64)]

    def __setattr__(self, name, value):
        if self._b_base_ is not None:
            raise AttributeError("assign a new RopeStrides to the configuration")
        super().__setattr__(name, value)


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
        """Type; shape, strides and bytes of q in, q out, k in and k out; bytes of the positions; whether there is a k."""
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
                operand(self.kv_heads, self.k_out), places * max(self.axes, 0) * 4, self.kv_heads != 0)


def _stream_on(device, stream):
    return _raw_stream(device) if stream is None and _raw_stream is not None else _stream(stream)


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
                 "sdv2_debug_mx4_plan": (ctypes.c_int, [prodp, ctypes.POINTER(_i32)]),
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


def debug_mx4_plan(cfg: Mx4ProductConfig):
    """(width, parts, rounds): how mx4_product runs a configuration, as sdv2_debug_mx4_plan tells; host only."""
    plan = (_i32 * 3)()
    _b._check(_lib().sdv2_debug_mx4_plan(cfg, plan), "sdv2_debug_mx4_plan")
    return tuple(plan)


def mx4_workspace_init(cfg, ws, stream=None):
    _b._check(_lib().sdv2_mx4_workspace_init(ctypes.byref(cfg), _Operands()(ws, "ws", _U8, 256), _stream(stream)),
              "sdv2_mx4_workspace_init")


# The calls below see at once, operand by operand, that all is as it should be, as most of a small call's time on the host goes
# there.  Anything else goes to the checks of _Operands, which say what is wrong or find that nothing is.

def _matrix(plan, x, name, codes, scales, stream):
    """Pointers of x or y, codes and scales, and the stream."""
    nc, ns, (kind, shape, strides, nbytes) = plan
    try:
        dev = x.get_device()
        if (dev >= 0 and dev == _current_device() and x.dtype is kind and x.shape == shape and x.stride() == strides
                and codes.dtype is _U8 and codes.get_device() == dev and codes.nbytes >= nc and codes.is_contiguous()
                and scales.dtype is _U8 and scales.get_device() == dev and scales.nbytes >= ns and scales.is_contiguous()):
            return x.data_ptr(), codes.data_ptr(), scales.data_ptr(), _stream_on(dev, stream)
    except AttributeError:             # a pointer in a tensor's place
        pass
    op = _Operands()
    return (op.view(x, name, kind, shape, strides, nbytes), op(codes, "codes", _U8, nc, True), op(scales, "scales", _U8, ns, True),
            _stream(stream))


def mx4_quantize(cfg, x, codes, scales, stream=None):
    """x: [rows][cols] (transposed: [cols][rows]) of cfg.x_dtype; codes, scales: uint8, of mx4_codes_bytes(cfg) and
    mx4_scales_bytes(cfg) bytes."""
    px, pc, ps, st = _matrix(cfg.derived(), x, "x", codes, scales, stream)
    status = _lib().sdv2_mx4_quantize(cfg, px, pc, ps, st)
    if status:
        _b._check(status, "sdv2_mx4_quantize")


def mx4_dequantize(cfg, codes, scales, y, stream=None):
    """y: [rows][cols] of cfg.x_dtype, the values that codes and scales stand for."""
    py, pc, ps, st = _matrix(cfg.derived(), y, "y", codes, scales, stream)
    status = _lib().sdv2_mx4_dequantize(cfg, pc, ps, py, st)
    if status:
        _b._check(status, "sdv2_mx4_dequantize")


def _product(plan, a_codes, a_scales, b_codes, b_scales, out, ws, bias, stream):
    """Pointers of a product's operands, its result and its workspace, and the stream."""
    nac, nas, nbc, nbs, nb, nw, (kind, shape, strides, nbytes) = plan
    try:
        dev = out.get_device()
        if (dev >= 0 and dev == _current_device() and out.dtype is kind and out.shape == shape and out.stride() == strides
                and a_codes.dtype is _U8 and a_codes.get_device() == dev and a_codes.nbytes >= nac and a_codes.is_contiguous()
                and a_scales.dtype is _U8 and a_scales.get_device() == dev and a_scales.nbytes >= nas and a_scales.is_contiguous()
                and b_codes.dtype is _U8 and b_codes.get_device() == dev and b_codes.nbytes >= nbc and b_codes.is_contiguous()
                and b_scales.dtype is _U8 and b_scales.get_device() == dev and b_scales.nbytes >= nbs and b_scales.is_contiguous()
                and ws.dtype is _U8 and ws.get_device() == dev and ws.nbytes >= nw and ws.is_contiguous()
                and (bias is None or bias.dtype is _FP and bias.get_device() == dev and bias.nbytes >= nb and bias.is_contiguous())):
            return (a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(), b_scales.data_ptr(),
                    None if bias is None else bias.data_ptr(), out.data_ptr(), ws.data_ptr(), _stream_on(dev, stream))
    except AttributeError:
        pass
    op = _Operands()
    return (op(a_codes, "a_codes", _U8, nac, True), op(a_scales, "a_scales", _U8, nas, True), op(b_codes, "b_codes", _U8, nbc, True),
            op(b_scales, "b_scales", _U8, nbs, True), op(bias, "bias", _FP, nb, True),
            op.view(out, "out", kind, shape, strides, nbytes), op(ws, "ws", _U8, nw, True), _stream(stream))


def mx4_product(cfg, a_codes, a_scales, b_codes, b_scales, out, ws, bias=None, stream=None):
    """out [rows][cols] = act(a b^T + bias) of matrices that mx4_quantize wrote: a of `rows` and b of `cols` rows, both of
    `depth` columns; bias: fp32 [cols]; ws: mx4_workspace_bytes(cfg) bytes."""
    status = _lib().sdv2_mx4_product(cfg, *_product(cfg.derived(), a_codes, a_scales, b_codes, b_scales, out, ws, bias, stream))
    if status:
        _b._check(status, "sdv2_mx4_product")


def _multiply(cfg, operands):
    """The product of operands that _product has seen, between which and this the caller may have quantised a."""
    status = _lib().sdv2_mx4_product(cfg, *operands)
    if status:
        _b._check(status, "sdv2_mx4_product")


_FORWARD, _BACKWARD = ("q", "q_out", "k", "k_out"), ("dq_out", "dq", "dk_out", "dk")


def _turn(plan, names, positions, q, q_new, k, k_new, stream):
    """Pointers of the positions, of q and its result and of k and its result (None without a k), and the stream."""
    kind, (qs, qt, qn), (rs, rt, rn), (ks, kt, kn), (ls, lt, ln), np, with_k = plan
    try:
        dev = q.get_device()
        if (dev >= 0 and dev == _current_device() and positions.dtype is _I32 and positions.get_device() == dev and positions.nbytes >= np
                and positions.is_contiguous() and q.dtype is kind and q.shape == qs and q.stride() == qt
                and q_new.dtype is kind and q_new.get_device() == dev and q_new.shape == rs and q_new.stride() == rt
                and (not with_k or k.dtype is kind and k.get_device() == dev and k.shape == ks and k.stride() == kt
                     and k_new.dtype is kind and k_new.get_device() == dev and k_new.shape == ls and k_new.stride() == lt)):
            return (positions.data_ptr(), q.data_ptr(), q_new.data_ptr(), k.data_ptr() if with_k else None,
                    k_new.data_ptr() if with_k else None, _stream_on(dev, stream))
    except AttributeError:
        pass
    op = _Operands()
    return (op(positions, "positions", _I32, np, True), op.view(q, names[0], kind, qs, qt, qn), op.view(q_new, names[1], kind, rs, rt, rn),
            op.view(k, names[2], kind, ks, kt, kn) if with_k else None, op.view(k_new, names[3], kind, ls, lt, ln) if with_k else None,
            _stream(stream))


def axes_rope(cfg, positions, q, q_out, k=None, k_out=None, stream=None):
    """q, q_out: [batch][tokens][heads][head_dim], k, k_out: [batch][tokens][kv_heads][head_dim] with cfg's strides;
    positions: int32 [batch][tokens][axes], or [tokens][axes] shared by the batch."""
    status = _lib().sdv2_axes_rope(cfg, *_turn(cfg.derived(), _FORWARD, positions, q, q_out, k, k_out, stream))
    if status:
        _b._check(status, "sdv2_axes_rope")


def axes_rope_backward(cfg, positions, dq_out, dq, dk_out=None, dk=None, stream=None):
    """Gradients dq (cfg.q_in's strides) and dk (cfg.k_in's) from those of axes_rope's results."""
    kind, q_in, q_out, k_in, k_out, nbytes, with_k = cfg.derived()
    status = _lib().sdv2_axes_rope_backward(cfg, *_turn((kind, q_out, q_in, k_out, k_in, nbytes, with_k), _BACKWARD, positions, dq_out, dq,
                                                        dk_out, dk, stream))
    if status:
        _b._check(status, "sdv2_axes_rope_backward")
