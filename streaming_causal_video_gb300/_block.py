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
    @classmethod
    def make(cls, **kw):
        names = {n for n, _ in cls._fields_}
        for k in kw:
            if k not in names:
                raise TypeError("%s has no field %r" % (cls.__name__, k))
        return cls(**kw)


class CrossConfig(_Config):
    """Mirror of sdv2_cross_cfg."""
    _fields_ = [("batch", _i32), ("heads", _i32), ("kv_heads", _i32), ("head_dim", _i32), ("q_len", _i64),
                ("kv_len", _i64), ("q_token_stride", _i64), ("q_head_stride", _i64), ("q_batch_stride", _i64),
                ("kv_token_stride", _i64), ("kv_head_stride", _i64), ("kv_batch_stride", _i64)]


class NormConfig(_Config):
    """Mirror of sdv2_norm_cfg."""
    _fields_ = [("rows", _i64), ("cols", _i32), ("x_dtype", _i32), ("y_dtype", _i32), ("weight_plus_one", _i32),
                ("x_row_stride", _i64), ("y_row_stride", _i64), ("rows_per_group", _i64), ("group_stride", _i64),
                ("eps", _f32)]


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
        self.device = -1

    def __call__(self, t, name, dtype, nbytes, dense=False):
        if t is None or type(t) is int:
            return t
        if not t.is_cuda:
            raise ValueError("%s must be a CUDA tensor" % name)
        if t.dtype is not dtype:
            raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
        device = t.get_device()
        if device != self.device:
            if self.device >= 0:
                raise ValueError("%s is on device %d, not on device %d" % (name, device, self.device))
            if device != _current_device():
                raise ValueError("%s is on device %d, the current device is %d" % (name, device, _current_device()))
            self.device = device
        if not t.is_contiguous():
            if dense:
                raise ValueError("%s must be contiguous" % name)
        elif t.nbytes >= nbytes:
            return t.data_ptr()
        return _b._dev(t, name, nbytes)


_BF, _FP, _U8 = torch.bfloat16, torch.float32, torch.uint8
_TYPE = {BF16: (_BF, 2), F32: (_FP, 4)}


def cross_workspace_bytes(cfg: CrossConfig, backward: bool = False) -> int:
    return _lib().sdv2_cross_workspace_bytes(ctypes.byref(cfg), 1 if backward else 0)


def norm_workspace_bytes(cfg: NormConfig) -> int:
    return _lib().sdv2_norm_workspace_bytes(ctypes.byref(cfg))


def cross_workspace_init(cfg, ws, stream=None):
    _b._check(_lib().sdv2_cross_workspace_init(ctypes.byref(cfg), _Operands()(ws, "ws", _U8, 256), _stream(stream)),
              "sdv2_cross_workspace_init")


def _strides(heads, length, tok, hd, batch):
    hd = hd or 128
    tok = tok or heads * 128
    return tok, hd, batch or max(max(length, 1) * tok, heads * hd)


def _span(batch, length, heads, st):
    """Bytes from an operand's first element to past its last."""
    if batch < 1 or length < 1 or heads < 1:
        return 0
    return 2 * ((batch - 1) * st[2] + (length - 1) * st[0] + (heads - 1) * st[1] + 128)


def _cross_operand(op, t, name, batch, length, heads, st):
    """A [B][length][heads][128] view must have the configuration's strides; a tensor of another rank is
    a buffer that they are applied to."""
    if t is not None and type(t) is not int and t.dim() == 4:
        if t.shape != (batch, length, heads, 128):
            raise ValueError("%s is %s, the configuration says %s" % (name, tuple(t.shape), (batch, length, heads, 128)))
        want, have = (st[2], st[0], st[1], 1), t.stride()
        if want != have and any(n > 1 and w != h for n, w, h in zip(t.shape, want, have)):
            raise ValueError("%s has strides %s, the configuration says %s" % (name, have, want))
    return op(t, name, _BF, _span(batch, length, heads, st))


def _lens(cfg, kv_lens):
    return None if kv_lens is None else _b._i64_array(kv_lens, cfg.batch)


def _cross_inputs(cfg, op, q, k, v):
    B, H, Hk = cfg.batch, cfg.heads, cfg.kv_heads or cfg.heads
    qs = _strides(H, cfg.q_len, cfg.q_token_stride, cfg.q_head_stride, cfg.q_batch_stride)
    ks = _strides(Hk, cfg.kv_len, cfg.kv_token_stride, cfg.kv_head_stride, cfg.kv_batch_stride)
    return (_cross_operand(op, q, "q", B, cfg.q_len, H, qs), _cross_operand(op, k, "k", B, cfg.kv_len, Hk, ks),
            _cross_operand(op, v, "v", B, cfg.kv_len, Hk, ks))


def cross_attention(cfg, q, k, v, out, ws, kv_lens=None, lse=None, scale=0.0, stream=None):
    """q: [B][Nq][H][128], k, v: [B][Nk][Hk][128] bf16 with cfg's strides; out: [B][Nq][H][128] bf16 and
    lse: fp32 [B][H][Nq], dense; kv_lens: valid rows of k and v per stream (host integers)."""
    op = _Operands()
    rows = max(cfg.batch, 0) * max(cfg.heads, 0) * max(cfg.q_len, 0)
    _b._check(_lib().sdv2_cross_attention(ctypes.byref(cfg), _lens(cfg, kv_lens), *_cross_inputs(cfg, op, q, k, v),
                                          float(scale), op(out, "out", _BF, rows * 256, True),
                                          op(lse, "lse", _FP, rows * 4, True),
                                          op(ws, "ws", _U8, 256), _stream(stream)), "sdv2_cross_attention")


def cross_attention_backward(cfg, q, k, v, out, lse, dout, dq, dk, dv, ws, kv_lens=None, scale=0.0, stream=None):
    """Gradients dq [B][Nq][H][128] and dk, dv [B][Nk][Hk][128] (bf16, dense) of cross_attention, whose out
    and lse are given with the gradient dout of out; ws: cross_workspace_bytes(cfg, backward=True) bytes."""
    op = _Operands()
    rows = max(cfg.batch, 0) * max(cfg.heads, 0) * max(cfg.q_len, 0)
    kv_rows = max(cfg.batch, 0) * (cfg.kv_heads or cfg.heads) * max(cfg.kv_len, 0)
    _b._check(_lib().sdv2_cross_attention_backward(
        ctypes.byref(cfg), _lens(cfg, kv_lens), *_cross_inputs(cfg, op, q, k, v), op(out, "out", _BF, rows * 256, True),
        op(lse, "lse", _FP, rows * 4, True), op(dout, "dout", _BF, rows * 256, True), float(scale),
        op(dq, "dq", _BF, rows * 256, True), op(dk, "dk", _BF, kv_rows * 256, True),
        op(dv, "dv", _BF, kv_rows * 256, True), op(ws, "ws", _U8, cross_workspace_bytes(cfg, True)),
        _stream(stream)), "sdv2_cross_attention_backward")


def _rows(cfg, op, t, name, dtype, stride):
    """Rows of x or y: a 2-D tensor must be [rows][cols] with the configuration's row stride."""
    kind, size = _TYPE.get(dtype, (None, 4))
    stride = stride or cfg.cols
    if t is not None and type(t) is not int and t.dim() == 2:
        if t.shape != (cfg.rows, cfg.cols) or (cfg.cols > 1 and t.stride(1) != 1) or \
                (cfg.rows > 1 and t.stride(0) != stride):
            raise ValueError("%s is %s with strides %s, the configuration says %s and row stride %d" %
                             (name, tuple(t.shape), tuple(t.stride()), (cfg.rows, cfg.cols), stride))
    return op(t, name, kind, _b._row_span(cfg.rows, stride, cfg.cols, size))


def _groups(cfg):
    per = cfg.rows_per_group or cfg.rows
    return (cfg.rows + per - 1) // per if per > 0 else 0


def layer_norm(cfg, x, y, weight=None, bias=None, mean=None, rstd=None, stream=None):
    """x: [rows][cols] of cfg.x_dtype; y: of cfg.y_dtype; weight, bias: fp32 [groups][cols], group_stride
    apart; mean, rstd: fp32 [rows], written for the backward pass."""
    op = _Operands()
    par = _b._row_span(_groups(cfg), cfg.group_stride or cfg.cols, cfg.cols, 4)
    _b._check(_lib().sdv2_layer_norm(ctypes.byref(cfg), _rows(cfg, op, x, "x", cfg.x_dtype, cfg.x_row_stride),
                                     op(weight, "weight", _FP, par), op(bias, "bias", _FP, par),
                                     _rows(cfg, op, y, "y", cfg.y_dtype, cfg.y_row_stride),
                                     op(mean, "mean", _FP, cfg.rows * 4, True), op(rstd, "rstd", _FP, cfg.rows * 4, True),
                                     _stream(stream)), "sdv2_layer_norm")


def layer_norm_backward(cfg, dy, x, mean, rstd, dx, ws, weight=None, dweight=None, dbias=None, stream=None):
    """dx (of x's type and stride), and fp32 dweight, dbias [groups][cols] (dense, or None), from the
    gradient dy of y and what layer_norm read and wrote; ws: norm_workspace_bytes(cfg) bytes."""
    op = _Operands()
    par = _b._row_span(_groups(cfg), cfg.group_stride or cfg.cols, cfg.cols, 4)
    grads = _groups(cfg) * cfg.cols * 4
    _b._check(_lib().sdv2_layer_norm_backward(
        ctypes.byref(cfg), _rows(cfg, op, dy, "dy", cfg.y_dtype, cfg.y_row_stride),
        _rows(cfg, op, x, "x", cfg.x_dtype, cfg.x_row_stride), op(weight, "weight", _FP, par),
        op(mean, "mean", _FP, cfg.rows * 4, True), op(rstd, "rstd", _FP, cfg.rows * 4, True),
        _rows(cfg, op, dx, "dx", cfg.x_dtype, cfg.x_row_stride), op(dweight, "dweight", _FP, grads, True),
        op(dbias, "dbias", _FP, grads, True),
        op(ws, "ws", _U8, norm_workspace_bytes(cfg) if (dweight is not None or dbias is not None) else 0),
        _stream(stream)), "sdv2_layer_norm_backward")
