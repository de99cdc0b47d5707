"""ctypes binding of the operators in include/sdv2_block.h (argument marshalling only)."""
import ctypes

import torch

from . import _binding as _b

BF16, F32 = 0, 1               # sdv2_dtype

# Every symbol that include/sdv2_block.h declares.
BLOCK_EXPORTS = ["sdv2_cross_workspace_bytes", "sdv2_cross_workspace_init", "sdv2_cross_attention",
                 "sdv2_cross_attention_backward", "sdv2_layer_norm", "sdv2_norm_workspace_bytes",
                 "sdv2_layer_norm_backward"]

_i32, _i64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class _Config(ctypes.Structure):
    """A configuration and, until a field is set, what the binding derives from it."""

    @classmethod
    def make(cls, **kw):
        names = {n for n, _ in cls._fields_}
        for k in kw:
            if k not in names:
                raise TypeError("%s has no field %r" % (cls.__name__, k))
        return cls(**kw)

    def __setattr__(self, name, value):
        self.__dict__.pop("plan", None)
        super().__setattr__(name, value)

    def derived(self):
        plan = self.__dict__.get("plan")
        if plan is None:
            plan = self.__dict__["plan"] = self._derive()
        return plan


class CrossConfig(_Config):
    """Mirror of sdv2_cross_cfg."""
    _fields_ = [("batch", _i32), ("heads", _i32), ("kv_heads", _i32), ("head_dim", _i32), ("q_len", _i64),
                ("kv_len", _i64), ("q_token_stride", _i64), ("q_head_stride", _i64), ("q_batch_stride", _i64),
                ("kv_token_stride", _i64), ("kv_head_stride", _i64), ("kv_batch_stride", _i64)]

    def _derive(self):
        """Shape, strides and bytes of q and of k and v; bytes of dense rows of q, of
        log-sum-exps and of k; bytes of the workspace for a backward pass."""
        B, H, Hk = self.batch, self.heads, self.kv_heads or self.heads
        rows, kv_rows = max(B, 0) * max(H, 0) * max(self.q_len, 0), max(B, 0) * max(Hk, 0) * max(self.kv_len, 0)

        def operand(length, heads, tok, hd, batch):
            hd = hd or 128
            tok = tok or heads * 128
            batch = batch or max(max(length, 1) * tok, heads * hd)
            span = 2 * ((B - 1) * batch + (length - 1) * tok + (heads - 1) * hd + 128) if min(B, length, heads) > 0 else 0
            return (B, length, heads, 128), (batch, tok, hd, 1), span
        return (operand(self.q_len, H, self.q_token_stride, self.q_head_stride, self.q_batch_stride),
                operand(self.kv_len, Hk, self.kv_token_stride, self.kv_head_stride, self.kv_batch_stride),
                rows * 256, rows * 4, kv_rows * 256, cross_workspace_bytes(self, True))


class NormConfig(_Config):
    """Mirror of sdv2_norm_cfg."""
    _fields_ = [("rows", _i64), ("cols", _i32), ("x_dtype", _i32), ("y_dtype", _i32), ("weight_plus_one", _i32),
                ("x_row_stride", _i64), ("y_row_stride", _i64), ("rows_per_group", _i64), ("group_stride", _i64),
                ("eps", _f32)]

    def _derive(self):
        """Shape, strides, type and bytes of x and of y; shape, stride and bytes of the parameters;
        bytes of their gradients, of a value per row, and of the workspace."""
        def operand(dtype, stride):
            kind, size = _TYPE.get(dtype, (None, 4))
            stride = stride or self.cols
            return (self.rows, self.cols), (stride, 1), kind, _b._row_span(self.rows, stride, self.cols, size)
        per = self.rows_per_group or self.rows
        groups = (self.rows + per - 1) // per if per > 0 else 0
        stride = self.group_stride or self.cols
        return (operand(self.x_dtype, self.x_row_stride), operand(self.y_dtype, self.y_row_stride),
                ((groups, self.cols), stride, _b._row_span(groups, stride, self.cols, 4)), groups * self.cols * 4, self.rows * 4,
                norm_workspace_bytes(self))


_LIB = None


def _lib():
    global _LIB
    L = _b.lib()
    if _LIB is not L:
        crossp, normp = ctypes.POINTER(CrossConfig), ctypes.POINTER(NormConfig)
        types = {"sdv2_cross_workspace_bytes": (ctypes.c_size_t, [crossp, _i32]),
                 "sdv2_cross_workspace_init": (ctypes.c_int, [crossp, _vp, _vp]),
                 "sdv2_cross_attention": (ctypes.c_int, [crossp, ctypes.POINTER(_i64)] + [_vp] * 3 + [_f32] + [_vp] * 4),
                 "sdv2_cross_attention_backward": (ctypes.c_int, [crossp, ctypes.POINTER(_i64)] + [_vp] * 6 + [_f32] +
                                                   [_vp] * 5),
                 "sdv2_layer_norm": (ctypes.c_int, [normp] + [_vp] * 7),
                 "sdv2_norm_workspace_bytes": (ctypes.c_size_t, [normp]),
                 "sdv2_layer_norm_backward": (ctypes.c_int, [normp] + [_vp] * 10)}
        for name, (res, args) in types.items():
            getattr(L, name).restype = res
            getattr(L, name).argtypes = args
        _LIB = L
    return L


# The current device and its current stream as integers.  torch's own accessors build a Python object
# per call, which costs more than a small kernel; its raw ones are used where the build has them.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None and _raw_stream is not None:
        return _raw_stream(_current_device())
    return _b._stream(stream)


class _Operands:
    """Pointers of one call's tensors, each checked for its type, its extent and its device: one CUDA
    device, the current one.  Raw integer pointers and None pass through unchecked."""
    __slots__ = ("device",)

    def __init__(self):
        self.device = -2

    def __call__(self, t, name, dtype, nbytes, dense=False):
        if t is None or type(t) is int:
            return t
        device = t.get_device()
        if device != self.device:
            if device < 0:
                raise ValueError("%s must be a CUDA tensor" % name)
            if self.device != -2:
                raise ValueError("%s is on device %d, not on device %d" % (name, device, self.device))
            if device != _current_device():
                raise ValueError("%s is on device %d, the current device is %d" % (name, device, _current_device()))
            self.device = device
        if t.dtype is not dtype:
            raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
        if t.is_contiguous():
            if t.nbytes >= nbytes:
                return t.data_ptr()
        elif dense:
            raise ValueError("%s must be contiguous" % name)
        return _b._dev(t, name, nbytes)

    def view(self, t, name, dtype, shape, strides, nbytes):
        """A view of the configuration's rank must have its shape and strides; a contiguous tensor of another rank
        is a buffer that they are applied to, and any other has to have them when it is seen in that shape."""
        if t is not None and type(t) is not int:
            if t.dim() == len(shape):
                if t.shape != shape:
                    raise ValueError("%s is %s, the configuration says %s" % (name, tuple(t.shape), shape))
                _check_strides(t, name, shape, strides)
            elif not t.is_contiguous():
                _check_strides(_seen_as(t, name, shape), name, shape, strides)
        return self(t, name, dtype, nbytes)

    def parameters(self, t, name, shape, stride, nbytes):
        """fp32 rows of shape (groups, cols), `stride` apart.  Two-dimensional parameters must have that stride (rows
        behind the last group may follow); a contiguous tensor of another shape is a buffer."""
        p = self(t, name, _FP, nbytes)
        if t is not None and type(t) is not int and not (stride == shape[1] and t.is_contiguous()):
            if t.dim() == 2 and t.shape[1] == shape[1] and t.shape[0] >= shape[0]:
                _check_strides(t, name, shape, (stride, 1))
            elif not t.is_contiguous():
                _check_strides(_seen_as(t, name, shape), name, shape, (stride, 1))
        return p


def _check_strides(t, name, shape, strides):
    have = t.stride()
    if have != strides and any(n > 1 and h != w for n, h, w in zip(shape, have, strides)):
        raise ValueError("%s has strides %s, the configuration says %s" % (name, have, strides))


def _seen_as(t, name, shape):
    try:
        return t.view(shape)
    except RuntimeError:
        raise ValueError("%s (%s, strides %s) must be contiguous or a view of %s" % (name, tuple(t.shape), t.stride(), shape)) from None


_BF, _FP, _U8 = torch.bfloat16, torch.float32, torch.uint8
_TYPE = {BF16: (_BF, 2), F32: (_FP, 4)}


def cross_workspace_bytes(cfg: CrossConfig, backward: bool = False) -> int:
    return _lib().sdv2_cross_workspace_bytes(ctypes.byref(cfg), 1 if backward else 0)


def norm_workspace_bytes(cfg: NormConfig) -> int:
    return _lib().sdv2_norm_workspace_bytes(ctypes.byref(cfg))


def cross_workspace_init(cfg, ws, stream=None):
    _b._check(_lib().sdv2_cross_workspace_init(ctypes.byref(cfg), _Operands()(ws, "ws", _U8, 256), _stream(stream)),
              "sdv2_cross_workspace_init")


def _lens(cfg, kv_lens):
    return None if kv_lens is None else _b._i64_array(kv_lens, cfg.batch)


def _cross_inputs(op, q, k, v, qs, ks):
    return op.view(q, "q", _BF, *qs), op.view(k, "k", _BF, *ks), op.view(v, "v", _BF, *ks)


def cross_attention(cfg, q, k, v, out, ws, kv_lens=None, lse=None, scale=0.0, stream=None):
    """q: [B][Nq][H][128], k, v: [B][Nk][Hk][128] bf16 with cfg's strides; out: [B][Nq][H][128] bf16 and
    lse: fp32 [B][H][Nq], dense; kv_lens: valid rows of k and v per stream (host integers)."""
    op = _Operands()
    qs, ks, rows, stats, _, _ = cfg.derived()
    status = _lib().sdv2_cross_attention(ctypes.byref(cfg), _lens(cfg, kv_lens), *_cross_inputs(op, q, k, v, qs, ks), scale,
                                         op(out, "out", _BF, rows, True), op(lse, "lse", _FP, stats, True),
                                         op(ws, "ws", _U8, 256), _stream(stream))
    if status:
        _b._check(status, "sdv2_cross_attention")


def cross_attention_backward(cfg, q, k, v, out, lse, dout, dq, dk, dv, ws, kv_lens=None, scale=0.0, stream=None):
    """Gradients dq [B][Nq][H][128] and dk, dv [B][Nk][Hk][128] (bf16, dense) of cross_attention, whose out
    and lse are given with the gradient dout of out; ws: cross_workspace_bytes(cfg, backward=True) bytes."""
    op = _Operands()
    qs, ks, rows, stats, kv_rows, scratch = cfg.derived()
    status = _lib().sdv2_cross_attention_backward(
        ctypes.byref(cfg), _lens(cfg, kv_lens), *_cross_inputs(op, q, k, v, qs, ks), op(out, "out", _BF, rows, True),
        op(lse, "lse", _FP, stats, True), op(dout, "dout", _BF, rows, True), scale, op(dq, "dq", _BF, rows, True),
        op(dk, "dk", _BF, kv_rows, True), op(dv, "dv", _BF, kv_rows, True), op(ws, "ws", _U8, scratch), _stream(stream))
    if status:
        _b._check(status, "sdv2_cross_attention_backward")


def layer_norm(cfg, x, y, weight=None, bias=None, mean=None, rstd=None, stream=None):
    """x: [rows][cols] of cfg.x_dtype; y: of cfg.y_dtype; weight, bias: fp32 [groups][cols], group_stride
    apart; mean, rstd: fp32 [rows], written for the backward pass."""
    op = _Operands()
    (shape, xs, xt, xb), (_, ys, yt, yb), par, _, stats, _ = cfg.derived()
    status = _lib().sdv2_layer_norm(ctypes.byref(cfg), op.view(x, "x", xt, shape, xs, xb),
                                    op.parameters(weight, "weight", *par), op.parameters(bias, "bias", *par), op.view(y, "y", yt, shape, ys, yb),
                                    op(mean, "mean", _FP, stats, True), op(rstd, "rstd", _FP, stats, True), _stream(stream))
    if status:
        _b._check(status, "sdv2_layer_norm")


def layer_norm_backward(cfg, dy, x, mean, rstd, dx, ws, weight=None, dweight=None, dbias=None, stream=None):
    """dx (of x's type and stride), and fp32 dweight, dbias [groups][cols] (dense, or None), from the
    gradient dy of y and what layer_norm read and wrote; ws: norm_workspace_bytes(cfg) bytes."""
    op = _Operands()
    (shape, xs, xt, xb), (_, ys, yt, yb), par, grads, stats, scratch = cfg.derived()
    status = _lib().sdv2_layer_norm_backward(
        ctypes.byref(cfg), op.view(dy, "dy", yt, shape, ys, yb), op.view(x, "x", xt, shape, xs, xb), op.parameters(weight, "weight", *par),
        op(mean, "mean", _FP, stats, True), op(rstd, "rstd", _FP, stats, True), op.view(dx, "dx", xt, shape, xs, xb),
        op(dweight, "dweight", _FP, grads, True), op(dbias, "dbias", _FP, grads, True),
        op(ws, "ws", _U8, scratch if (dweight is not None or dbias is not None) else 0), _stream(stream))
    if status:
        _b._check(status, "sdv2_layer_norm_backward")
