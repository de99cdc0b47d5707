"""Device buffers for a stream batch, allocated with torch, and the per-layer call sequence.

A StreamSession owns the workspace, one LayerCache (k, v, slot metadata) per DiT layer and the
q_rot / out buffers; layer_step() issues sdv2_rope_append_kv then sdv2_chunk_attention for one
layer of one denoise step.  Around it, norm_step() normalises a chunk's tokens (before the
projections) and cross_step() attends to the layer's prompt states, which set_prompt() names and
which stay for all chunks and steps until the prompt changes.  project_step() multiplies tokens by
weights held in 4 bits (Mx4Matrix), and rope_step() turns queries and keys that do not go into the
cache.  Nothing here computes: it allocates and calls the library.  Steps of one session share its
buffers and error word: steps, or graphs of them, that run at the same time need sessions of their own.
What a session allocates is the memory of the stream that the call names (the current one by default):
before a session is dropped, any other stream that it was used on has to be waited for.
"""
import contextlib

import torch

from . import _binding as sd
from . import _block as block
from . import _project as project

_KINDS = {torch.bfloat16: block.BF16, torch.float32: block.F32}


def _memory_of(stream, device):
    """A context in which new memory is that of `stream`, where it is first written.  The allocator hands out what the current
    stream has freed at once, in the order of that stream alone: on another one such memory may still be in use."""
    device = torch.device(device)
    if stream is None or device.type != "cuda":
        return contextlib.nullcontext()
    handle = sd._stream(stream)
    # 0 and 1 are the names of the legacy default stream
    return torch.cuda.stream(torch.cuda.default_stream(device) if handle in (0, 1) else torch.cuda.ExternalStream(handle, device))


class LayerCache:
    """One layer's KV cache: k and v [B][H][(F_s+W)*HW][D] bf16, meta [B][F_s+W][2] int64."""

    def __init__(self, cfg: sd.StreamConfig, device, stream=None):
        B, H, D = cfg.batch, cfg.heads, cfg.head_dim
        rows = cfg.slots * cfg.hw
        assert sd.cache_bytes(cfg) == B * H * rows * D * 2
        with _memory_of(stream, device):
            self.k = torch.empty((B, H, rows, D), dtype=torch.bfloat16, device=device)
            self.v = torch.empty((B, H, rows, D), dtype=torch.bfloat16, device=device)
            self.meta = torch.empty((B, cfg.slots, 2), dtype=torch.int64, device=device)
        sd.cache_reset(cfg, self.k, self.v, self.meta, stream)


def _rows_of(t, name, groups, cols):
    """A norm's parameters as [groups][cols] and the stride between rows (0 where there is one row or none)."""
    if t is None or isinstance(t, int):
        return t, 0
    if t.dim() != 2 or t.shape[0] != groups or t.shape[1] != cols:
        if t.shape[-1:] != (cols,) or t.numel() != groups * cols:
            raise ValueError("%s is %s, not [%d][%d]" % (name, tuple(t.shape), groups, cols))
        try:
            t = t.view(groups, cols)
        except RuntimeError:
            raise ValueError("%s (strides %s) has no stride between its rows" % (name, t.stride())) from None
    stride = t.stride(0) if groups > 1 else 0
    if groups > 1 and stride < cols:
        raise ValueError("%s has a stride of %d between rows of %d" % (name, stride, cols))
    return t, stride


class Mx4Matrix:
    """A matrix of microscaled 4-bit numbers: codes and scales as sdv2_mx4_quantize writes them.

    A weight [N][K] is loaded once; activations [M][K] are loaded for every product.  For gradients a matrix can be loaded from its
    transpose: with y = x w^T, dx is the product of dy [M][N] and w loaded as [K][N], dw that of dy and x loaded as [N][M] and [K][M].
    """

    def __init__(self, rows: int, cols: int, device="cuda"):
        cfg = project.Mx4Config.make(rows=rows, cols=cols)
        if not project.mx4_codes_bytes(cfg):
            raise ValueError("a matrix has at least one row and one column, not %d and %d" % (rows, cols))
        self.rows, self.cols = rows, cols
        self.codes = torch.empty(project.mx4_codes_bytes(cfg), dtype=torch.uint8, device=device)
        self.scales = torch.empty(project.mx4_scales_bytes(cfg), dtype=torch.uint8, device=device)
        self.configs = {}              # of load and values, which follow from type, stride and direction

    def _first(self, rows):
        """A matrix of that many rows at the start of this one's memory."""
        m = object.__new__(Mx4Matrix)
        cfg = project.Mx4Config.make(rows=rows, cols=self.cols)
        m.rows, m.cols, m.configs = rows, self.cols, {}
        m.codes, m.scales = self.codes[:project.mx4_codes_bytes(cfg)], self.scales[:project.mx4_scales_bytes(cfg)]
        return m

    @classmethod
    def of(cls, x, transposed=False, stream=None):
        """A new matrix loaded from x [rows][cols], or from x [cols][rows].  Its memory is the current stream's, which another
        `stream` has to follow."""
        if x.dim() != 2:
            raise ValueError("x must have two dimensions, not %d" % x.dim())
        rows, cols = reversed(x.shape) if transposed else x.shape
        return cls(rows, cols, x.device).load(x, transposed, stream)

    def _config(self, x, transposed):
        shape = (self.cols, self.rows) if transposed else (self.rows, self.cols)
        if x.dtype not in _KINDS or tuple(x.shape) != shape:
            raise ValueError("expected bf16 or fp32 %s, got %s %s" % (shape, x.dtype, tuple(x.shape)))
        if x.stride(1) != 1 and shape[1] > 1:
            raise ValueError("rows must be dense, not %d elements apart" % x.stride(1))
        stride = x.stride(0) if shape[0] > 1 else 0
        if shape[0] > 1 and stride < shape[1]:
            raise ValueError("rows of %d elements cannot lie %d apart" % (shape[1], stride))
        key = (x.dtype, stride, transposed)
        cfg = self.configs.get(key)
        if cfg is None:
            cfg = self.configs[key] = project.Mx4Config.make(rows=self.rows, cols=self.cols, x_dtype=_KINDS[x.dtype],
                                                             transposed=int(transposed), x_row_stride=stride)
        return cfg

    def load(self, x, transposed=False, stream=None):
        """Quantises x [rows][cols] (transposed: [cols][rows]), bf16 or fp32 with any stride between rows."""
        project.mx4_quantize(self._config(x, transposed), x, self.codes, self.scales, stream)
        return self

    def values(self, out, stream=None):
        """Writes the values that the matrix stands for into out [rows][cols], bf16 or fp32."""
        project.mx4_dequantize(self._config(out, False), self.codes, self.scales, out, stream)
        return out


class StreamSession:
    def __init__(self, cfg: sd.StreamConfig, layers: int, start_frames, device="cuda", stream=None):
        self.cfg = cfg
        self.start_frames = [int(s) for s in start_frames]
        B, H, D, nq = cfg.batch, cfg.heads, cfg.head_dim, cfg.nq
        with _memory_of(stream, device):
            self.ws = torch.zeros(sd.workspace_bytes(cfg), dtype=torch.uint8, device=device)
            self.q_rot = torch.empty((B, H, nq, D), dtype=torch.bfloat16, device=device)
            self.out = torch.empty((B, nq, H, D), dtype=torch.bfloat16, device=device)
        sd.workspace_init(cfg, self.ws, stream)
        self.layers = [LayerCache(cfg, device, stream) for _ in range(layers)]
        self.prompts = [None] * layers
        self.cross_ws = None
        self.norms = {}                # norm_step's configurations, which follow from shapes, types and strides
        self.products = {}             # project_step's
        self.loaded = {}               # the 4-bit forms of its activations by their sizes, and the memory that those share
        self.scratch = {}
        self.ropes = {}                # rope_step's

    def layer_step(self, layer: int, chunk_index, q, k, v, out=None, lse=None, stream=None):
        """Causal-RoPE + cache append, then chunk attention, for one layer.  q, k, v: [B][Nq][H][D]."""
        L = self.layers[layer]
        out = self.out if out is None else out
        sd.rope_append_kv(self.cfg, self.start_frames, chunk_index, q, k, v, self.q_rot, L.k, L.v, L.meta,
                          self.ws, stream)
        sd.chunk_attention(self.cfg, chunk_index, self.q_rot, L.k, L.v, out, self.ws, lse=lse, stream=stream)
        return out

    def set_prompt(self, layer: int, k, v, lens=None, stream=None):
        """States of the prompt encoder that cross_step(layer, ...) attends to: k, v [B][Nk][Hk][128] bf16, views
        with any strides of whole 16 bytes (the same for both), kept by reference; lens: valid rows of each stream."""
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride():
            raise ValueError("k and v must be [B][Nk][Hk][128] with the same shape and strides")
        if k.stride(3) != 1:
            raise ValueError("k and v must be dense in their last dimension")
        c = self.cfg
        B, nk, hk, D = k.shape
        if B != c.batch:
            raise ValueError("k and v hold %d streams, the session %d" % (B, c.batch))
        if B > 1 and k.stride(0) == 0:
            raise ValueError("streams that share a prompt need a copy of it each")
        # a dimension of size one has no stride to speak of
        tok = k.stride(1) if nk > 1 else 0
        hd = k.stride(2) if hk > 1 else 0
        batch = k.stride(0) if B > 1 else 0
        cross = block.CrossConfig.make(batch=B, heads=c.heads, kv_heads=hk, head_dim=D, q_len=c.nq, kv_len=nk,
                                       kv_token_stride=tok, kv_head_stride=hd, kv_batch_stride=batch)
        lens = [nk] * B if lens is None else [int(n) for n in lens]
        need = block.cross_workspace_bytes(cross)
        if self.cross_ws is None or not need:          # init names what is wrong with a configuration without a size
            with _memory_of(stream, self.ws.device):
                ws = torch.empty(max(need, 256), dtype=torch.uint8, device=self.ws.device)
            block.cross_workspace_init(cross, ws, stream)
            self.cross_ws = ws
        self.prompts[layer] = (cross, k, v, lens)

    def cross_step(self, layer: int, q, out=None, lse=None, stream=None):
        """The chunk's queries q [B][Nq][H][128] attend to the layer's prompt; out as q (the session's by default)."""
        if self.prompts[layer] is None:
            raise ValueError("layer %d has no prompt: call set_prompt first" % layer)
        cross, k, v, lens = self.prompts[layer]
        out = self.out if out is None else out
        block.cross_attention(cross, q, k, v, out, self.cross_ws, kv_lens=lens, lse=lse, stream=stream)
        return out

    def norm_step(self, x, out, weight=None, bias=None, modulated=False, eps=1e-6, stream=None):
        """Layer norm of a chunk's tokens x [B][Nq][C] (bf16 or fp32) into out [B][Nq][C].  weight, bias fp32: [C], the
        learned affine; or, modulated, [B*F][C], the scale and shift of every latent frame: xhat * (1 + weight) + bias.
        Those may be slices of one modulation tensor such as [B*F][6][C] (of the same one, as they share a stride)."""
        if x.dtype not in _KINDS or out.dtype not in _KINDS:
            raise ValueError("x and out must be bf16 or fp32")
        if x.shape != out.shape or not x.is_contiguous() or not out.is_contiguous():
            raise ValueError("x and out must be contiguous and of one shape")
        C = x.shape[-1]
        rows = x.numel() // C
        groups = -(-rows // self.cfg.hw) if modulated else 1
        weight, stride = _rows_of(weight, "weight", groups, C)
        bias, bias_stride = _rows_of(bias, "bias", groups, C)
        if stride and bias_stride and stride != bias_stride:
            raise ValueError("weight and bias must have one stride between rows, not %d and %d" % (stride, bias_stride))
        key = (rows, C, x.dtype, out.dtype, modulated, stride or bias_stride, eps)
        cfg = self.norms.get(key)
        if cfg is None:
            cfg = self.norms[key] = block.NormConfig.make(
                rows=rows, cols=C, x_dtype=_KINDS[x.dtype], y_dtype=_KINDS[out.dtype], weight_plus_one=int(modulated),
                rows_per_group=self.cfg.hw if modulated else 0, group_stride=stride or bias_stride, eps=eps)
        block.layer_norm(cfg, x, out, weight=weight, bias=bias, stream=stream)
        return out

    def quantize_step(self, x, stream=None):
        """x [...][K] (bf16 or fp32, contiguous) in 4 bits, for several products of the same activations.  What it returns is the
        session's and holds until its next activations of K columns."""
        return self._activations(x, stream).load(x.view(-1, x.shape[-1]), stream=stream)

    def _activations(self, x, stream):
        """The session's matrix for activations of x's size, whatever it holds.  Its memory is that of the stream of its first use."""
        if x.dim() < 1 or not x.is_contiguous() or not x.numel():
            raise ValueError("x must be contiguous and hold at least one row")
        rows, cols = x.numel() // x.shape[-1], x.shape[-1]
        m = self.loaded.get((rows, cols))
        if m is None:
            # Memory for 128 * 2^n rows, so that any number of lengths takes at most four times what the longest does, or 128 rows
            # where that is shorter.  It is kept as long as the session, as graphs may hold it.
            room = max(128, 1 << (rows - 1).bit_length())
            if (room, cols) not in self.scratch:
                with _memory_of(stream, self.ws.device):
                    self.scratch[room, cols] = Mx4Matrix(room, cols, self.ws.device)
            m = self.loaded[rows, cols] = self.scratch[room, cols]._first(rows)
        return m

    def project_step(self, weight: Mx4Matrix, x, out, bias=None, activation=project.NO_ACTIVATION, stream=None):
        """out [...][N] = act(x w^T + bias) for a weight [N][K] in 4 bits; x: [...][K], bf16 or fp32, or what quantize_step made of
        it; out: contiguous, bf16 or fp32; bias: fp32 [N]; activation: NO_ACTIVATION or GELU.  A call that is refused has quantised
        nothing, so that what quantize_step returned before still holds."""
        if out.dtype not in _KINDS or out.dim() < 1 or not out.is_contiguous():
            raise ValueError("out must be contiguous bf16 or fp32")
        loaded = isinstance(x, Mx4Matrix)
        cols = x.cols if loaded else x.shape[-1] if x.dim() else 0
        if cols != weight.cols:
            raise ValueError("x has %d columns, the weight %d" % (cols, weight.cols))
        a = x if loaded else self._activations(x, stream)
        if out.shape[-1] != weight.rows or out.numel() != a.rows * weight.rows:
            raise ValueError("out is %s, not %d rows of %d" % (tuple(out.shape), a.rows, weight.rows))
        if bias is not None and bias.numel() != weight.rows:
            raise ValueError("bias has %d values, not %d" % (bias.numel(), weight.rows))
        key = (a.rows, weight.rows, a.cols, out.dtype, activation)
        cfg = self.products.get(key)
        if cfg is None:
            if activation not in (project.NO_ACTIVATION, project.GELU):
                raise ValueError("activation must be NO_ACTIVATION or GELU, not %r" % (activation,))
            cfg = self.products[key] = project.Mx4ProductConfig.make(rows=a.rows, cols=weight.rows, depth=a.cols,
                                                                     out_dtype=_KINDS[out.dtype], activation=activation)
        # (a product needs the error word alone, which is where the session's workspace has it)
        operands = project._product(cfg.derived(), a.codes, a.scales, weight.codes, weight.scales, out.view(a.rows, weight.rows), self.ws,
                                    bias, stream)
        if not loaded:
            if (operands[2] | operands[3] | (operands[4] or 0) | operands[5]) & 15:
                raise ValueError("the weight, bias and out must begin on 16 bytes")
            a.load(x.view(a.rows, cols), stream=stream)
        project._multiply(cfg, operands)
        return out

    def chunk_positions(self, chunk_index):
        """int32 [B][Nq][3]: time index, row and column of a chunk's tokens, the places that layer_step turns them by."""
        c = self.cfg
        if len(chunk_index) != c.batch:
            raise ValueError("%d chunk indexes for %d streams" % (len(chunk_index), c.batch))
        if min(chunk_index) < 0:
            raise ValueError("chunk indexes must be >= 0, not %s" % (list(chunk_index),))
        n = torch.arange(c.nq)
        grid = torch.stack([n // c.hw, n % c.hw // c.grid_w, n % c.grid_w], -1)
        pos = grid.expand(c.batch, c.nq, 3).clone()
        for b, (start, chunk) in enumerate(zip(self.start_frames, chunk_index)):
            pos[b, :, 0] += start + c.chunk_frames * (chunk % c.refresh_chunks if c.refresh_chunks else chunk)
        if int(pos.max()) >= 1 << 31:
            raise ValueError("time index %d is past 32 bits" % int(pos.max()))
        return pos.to(device=self.ws.device, dtype=torch.int32)

    def rope_step(self, positions, q, q_out, k=None, k_out=None, stream=None):
        """Turns q [B][N][H][D], and k, by their places on the session's three axes: positions int32 [B][N][3], or [N][3] for all of
        the batch.  bf16 or fp32 views with any strides of whole 16 bytes; q_out may be q itself, k_out k."""
        c = self.cfg
        if (k is None) != (k_out is None):
            raise ValueError("k and k_out go together")
        if q.dim() != 4 or q.dtype not in _KINDS or q.shape != q_out.shape or (k is not None and (k.dim() != 4 or k.shape != k_out.shape)):
            raise ValueError("q, k and their results must be bf16 or fp32 [B][N][H][D], each of one shape with its result")
        if k is not None and (k.shape[0], k.shape[1], k.shape[3]) != (q.shape[0], q.shape[1], q.shape[3]):
            raise ValueError("k must have q's batch, tokens and head dim")
        if q.shape[3] != c.head_dim:
            raise ValueError("q has heads of %d dims, the session of %d" % (q.shape[3], c.head_dim))
        if tuple(positions.shape) not in ((q.shape[0], q.shape[1], 3), (q.shape[1], 3)):
            raise ValueError("positions must be [B][N][3] or [N][3], not %s" % (tuple(positions.shape),))
        tensors = (q, q_out, k, k_out)
        key = (q.shape, q.dtype, positions.dim(), *(None if t is None else (t.shape[2], t.stride()) for t in tensors))
        cfg = self.ropes.get(key)
        if cfg is None:
            def strides(t):            # a dimension of size one has no stride to speak of
                if t is None:
                    return {}
                of = lambda i: t.stride(i) if t.shape[i] > 1 else 0
                return dict(token_stride=of(1), head_stride=of(2), batch_stride=of(0))
            names = ("q_in", "q_out", "k_in", "k_out")
            cfg = self.ropes[key] = project.AxesRopeConfig.make(
                batch=q.shape[0], tokens=q.shape[1], heads=q.shape[2], kv_heads=0 if k is None else k.shape[2], head_dim=q.shape[3],
                dims=(c.rope_t, c.rope_h, c.rope_w), base=c.rope_base, dtype=_KINDS[q.dtype], shared_positions=int(positions.dim() == 2),
                **{n: strides(t) for n, t in zip(names, tensors)})
        project.axes_rope(cfg, positions, q, q_out, k, k_out, stream)
        return q_out
