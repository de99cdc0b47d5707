"""GB300 (sm_103a) streaming causal-video chunk attention: thin Python binding of libsdv2.so.

The functions below have the names of the C ABI in include/sdv2.h and only marshal arguments:
torch tensors become device pointers, Python sequences become host int64 arrays, and a
non-zero status becomes an SDV2Error.  Every step of the path runs in the library's kernels;
there is no fallback -- if the library is missing or cannot be loaded, the calls raise.
"""
from ._binding import (  # noqa: F401
    NoiseCtl,
    SDV2Error,
    StreamConfig,
    cache_bytes,
    cache_reset,
    check_device_error,
    chunk_attention,
    chunk_attention_noalloc,
    debug_drop_kv_tile,
    debug_kv_schedule,
    debug_set_kv_splits,
    last_kv_splits,
    exported_symbols,
    lib,
    lib_path,
    meta_bytes,
    motion_l2,
    noalloc_check_device_error,
    noise_from_motion,
    qkv_rope_append,
    rope_append_kv,
    rope_refresh_rerotate,
    set_wait_timeout_ns,
    sink_update,
    visible_tokens,
    workspace_bytes,
    workspace_init,
)
from ._block import (  # noqa: F401
    BF16,
    F32,
    CrossConfig,
    NormConfig,
    cross_attention,
    cross_attention_backward,
    cross_workspace_bytes,
    cross_workspace_init,
    layer_norm,
    layer_norm_backward,
    norm_workspace_bytes,
)
from ._project import (  # noqa: F401
    GELU,
    NO_ACTIVATION,
    AxesRopeConfig,
    Mx4Config,
    Mx4ProductConfig,
    RopeStrides,
    axes_rope,
    axes_rope_backward,
    debug_mx4_plan,
    mx4_codes_bytes,
    mx4_dequantize,
    mx4_product,
    mx4_quantize,
    mx4_scales_bytes,
    mx4_workspace_bytes,
    mx4_workspace_init,
)
from .layer import LayerCache, Mx4Matrix, StreamSession  # noqa: F401
