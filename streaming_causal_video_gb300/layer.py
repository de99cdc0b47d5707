"""Device buffers for a stream batch, allocated with torch, and the per-layer call sequence.

A StreamSession owns the workspace, one LayerCache (k, v, slot metadata) per DiT layer and the
q_rot / out buffers; layer_step() issues sdv2_rope_append_kv then sdv2_chunk_attention for one
layer of one denoise step.  Around it, norm_step() normalises a chunk's tokens (before the
projections) and cross_step() attends to the layer's prompt states, which set_prompt() names and
which stay for all chunks and steps until the prompt changes.  Nothing here computes: it allocates
and calls the library.
"""
import torch

from . import _binding as sd
from . import _block as block


class LayerCache:
    """One layer's KV cache: k and v [B][H][(F_s+W)*HW][D] bf16, meta [B][F_s+W][2] int64."""

    def __init__(self, cfg: sd.StreamConfig, device, stream=None):
        B, H, D = cfg.batch, cfg.heads, cfg.head_dim
        rows = cfg.slots * cfg.hw
        assert sd.cache_bytes(cfg) == B * H * rows * D * 2
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


class StreamSession:
    def __init__(self, cfg: sd.StreamConfig, layers: int, start_frames, device="cuda", stream=None):
        self.cfg = cfg
        self.start_frames = [int(s) for s in start_frames]
        B, H, D, nq = cfg.batch, cfg.heads, cfg.head_dim, cfg.nq
        self.ws = torch.zeros(sd.workspace_bytes(cfg), dtype=torch.uint8, device=device)
        sd.workspace_init(cfg, self.ws, stream)
        self.layers = [LayerCache(cfg, device, stream) for _ in range(layers)]
        self.q_rot = torch.empty((B, H, nq, D), dtype=torch.bfloat16, device=device)
        self.out = torch.empty((B, nq, H, D), dtype=torch.bfloat16, device=device)
        self.prompts = [None] * layers
        self.cross_ws = None
        self.norms = {}                # norm_step's configurations, which follow from shapes, types and strides

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
        kinds = {torch.bfloat16: block.BF16, torch.float32: block.F32}
        if x.dtype not in kinds or out.dtype not in kinds:
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
                rows=rows, cols=C, x_dtype=kinds[x.dtype], y_dtype=kinds[out.dtype], weight_plus_one=int(modulated),
                rows_per_group=self.cfg.hw if modulated else 0, group_stride=stride or bias_stride, eps=eps)
        block.layer_norm(cfg, x, out, weight=weight, bias=bias, stream=stream)
        return out
