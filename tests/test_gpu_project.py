"""GPU tests of 4-bit matrices, their products and rotary positions, forward and backward, against plain 64-bit implementations
with derived bounds (project_common.py)."""
import math

import pytest
import torch

import streaming_causal_video_gb300 as sd
from project_common import HALF, packed, product_reference, quantized, rope_reference, special, values, within

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
KIND = {BF: sd.BF16, FP: sd.F32}


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build_library()


def cpu_gen(seed):
    return torch.Generator().manual_seed(seed)


def buffers(cfg):
    """Room for codes and scales, filled with what a kernel that leaves bytes out would leave."""
    return (torch.full((sd.mx4_codes_bytes(cfg),), 0xA5, dtype=torch.uint8, device="cuda"),
            torch.full((sd.mx4_scales_bytes(cfg),), 0xA5, dtype=torch.uint8, device="cuda"))


def strided(x, pad):
    """x on the GPU as a view whose rows lie `pad` elements further apart, with NaN between them."""
    base = torch.full((x.shape[0], x.shape[1] + pad), math.nan, dtype=x.dtype, device="cuda")
    base[:, :x.shape[1]] = x
    return base[:, :x.shape[1]], base


# ---- quantisation and values ------------------------------------------------------------------------

QUANT = [(1, 1, 0), (1, 31, 0), (2, 32, 0), (3, 33, 3), (16, 128, 0), (17, 129, 8), (33, 1050, 0), (127, 96, 4), (128, 256, 0),
         (129, 1001, 7), (300, 40, 0), (20, 1536, 16), (260, 5120, 0), (1, 20480, 0), (15, 8200, 8)]


@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad", QUANT)
def test_quantize_and_values(rows, cols, pad, dtype, transposed):
    g = cpu_gen(rows + cols)
    x = special(torch.randn(rows, cols, generator=g) * torch.exp(4 * torch.randn(rows, 1, generator=g)), g).to(dtype)
    view, _ = strided(x.t().contiguous() if transposed else x, pad)
    cfg = sd.Mx4Config.make(rows=rows, cols=cols, x_dtype=KIND[dtype], transposed=transposed, x_row_stride=view.stride(0) if pad else 0)
    codes, scales = buffers(cfg)
    sd.mx4_quantize(cfg, view, codes, scales)
    code, byte, bad = quantized(x)
    want_codes, want_scales = packed(code, byte, rows, cols)
    assert torch.equal(scales.cpu(), want_scales.flatten())
    got = codes.cpu().view(rows, -1)
    sound = ~bad.repeat_interleave(32, 1)                       # a NaN's codes do not matter
    sound = torch.nn.functional.pad(sound, (0, got.shape[1] * 2 - sound.shape[1]), value=True)[:, 0::2]
    assert torch.equal(got[sound], want_codes[sound])
    for out_dtype, out_pad in ((BF, 0), (FP, 0), (BF, 5), (FP, 8)):
        y, base = strided(torch.zeros(rows, cols, dtype=out_dtype), out_pad)
        back = sd.Mx4Config.make(rows=rows, cols=cols, x_dtype=KIND[out_dtype], x_row_stride=cols + out_pad)
        sd.mx4_dequantize(back, codes, scales, y)
        ref = values(code, byte)
        ref[bad.repeat_interleave(32, 1)[:, :cols]] = math.nan
        ref[ref.abs() >= 2.0 ** 128] *= math.inf                # what no 32-bit number holds
        assert torch.equal(y.cpu().double().nan_to_num(nan=12345.0), ref.nan_to_num(nan=12345.0))
        assert out_pad == 0 or bool(base[:, cols:].isnan().all())


# ---- products ---------------------------------------------------------------------------------------

class Product:
    """Operands as 64-bit values and as the library's bytes, quantised by the plain implementation."""

    def __init__(self, M, N, K, out_dtype, bias=True, gelu=False, pad=0, seed=0):
        g = cpu_gen(seed)
        self.M, self.N, self.K = M, N, K
        spread = lambda n: torch.exp(torch.randn(n, 1, generator=g))
        self.a, self.a4 = self.operand(torch.randn(M, K, generator=g) * spread(M))
        self.b, self.b4 = self.operand(torch.randn(N, K, generator=g) * spread(N) / math.sqrt(K))
        self.bias = torch.randn(N, generator=g).cuda() if bias else None
        self.gelu = gelu
        self.out_dtype = out_dtype
        self.out, self.base = strided(torch.full((M, N), math.nan, dtype=out_dtype), pad)
        self.pad = pad
        self.cfg = sd.Mx4ProductConfig.make(rows=M, cols=N, depth=K, out_dtype=KIND[out_dtype],
                                            activation=sd.GELU if gelu else sd.NO_ACTIVATION, out_row_stride=N + pad if pad else 0)
        self.ws = torch.full((sd.mx4_workspace_bytes(self.cfg),), 0xA5, dtype=torch.uint8, device="cuda")
        sd.mx4_workspace_init(self.cfg, self.ws)

    @staticmethod
    def operand(x):
        code, byte, _ = quantized(x)
        codes, scales = packed(code, byte, *x.shape)
        return values(code, byte).cuda(), (codes.cuda().flatten(), scales.cuda().flatten())

    def run(self, stream=None):
        sd.mx4_product(self.cfg, *self.a4, *self.b4, self.out, self.ws, bias=self.bias, stream=stream)

    def check(self):
        sd.check_device_error(self.ws)
        ref, tol = product_reference(self.a, self.b, self.bias, self.gelu, self.out_dtype)
        within(self.out, ref, tol, "out")
        assert not self.pad or bool(self.base[:, self.N:].isnan().all())


FEW = [(1, 1, 1), (1, 128, 128), (2, 33, 129), (3, 9216, 1536), (4, 127, 31), (5, 257, 1050), (8, 1000, 2080), (1, 40, 20480),
       (7, 300, 9000), (9, 130, 640), (16, 257, 9000), (17, 1000, 1100), (31, 129, 256), (32, 513, 4096), (33, 640, 1280), (64, 300, 7001)]
TILES = [(65, 1, 1), (70, 7, 32), (256, 256, 256), (128, 128, 128), (129, 255, 257), (100, 130, 1), (255, 257, 64), (257, 256, 127),
         (300, 500, 700), (1001, 777, 1050), (600, 300, 1280), (520, 1536, 1536)]
DEEP = [(65, 300, 8200), (77, 1536, 8960), (512, 700, 4096), (300, 260, 20480), (256, 250, 7001)]


@pytest.mark.parametrize("out_dtype", [FP, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", FEW, ids=str)
def test_products_of_few_rows(size, out_dtype):
    for bias, gelu, pad in ((False, False, 0), (True, False, 3), (True, True, 8)):
        p = Product(*size, out_dtype, bias, gelu, pad, seed=sum(size))
        p.run()
        p.check()


@pytest.mark.parametrize("out_dtype", [FP, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", TILES + DEEP, ids=str)
def test_products(size, out_dtype):
    for bias, gelu, pad in ((False, False, 0), (True, False, 3), (True, True, 8)):
        p = Product(*size, out_dtype, bias, gelu, pad, seed=sum(size))
        p.run()
        p.check()


# ---- rotary positions ---------------------------------------------------------------------------------

def rows(gen, B, N, H, D, dtype, layout):
    """A [B][N][H][D] view in a layout, and its strides."""
    if layout == "dense":
        return torch.randn(B, N, H, D, generator=gen, device="cuda").to(dtype), {}
    if layout == "heads_first":
        t = torch.randn(B, H, N, D, generator=gen, device="cuda").to(dtype).transpose(1, 2)
        return t, dict(token_stride=D, head_stride=N * D, batch_stride=H * N * D)
    base = torch.full((B, N, 3, H, D + 8), math.nan, dtype=dtype, device="cuda")     # q beside k and v, rows with room behind
    base[:, :, 1, :, :D] = torch.randn(B, N, H, D, generator=gen, device="cuda").to(dtype)
    return base[:, :, 1, :, :D], dict(token_stride=3 * H * (D + 8), head_stride=D + 8, batch_stride=N * 3 * H * (D + 8))


class Rope:
    def __init__(self, B, N, H, Hk, D, dims, halves, dtype, layouts, far=False, shared=False, scale=(), base=10000.0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dims, self.halves, self.scale, self.base = dims, halves, scale, base
        (self.q, qi), (self.q_new, qo) = rows(g, B, N, H, D, dtype, layouts[0]), rows(g, B, N, H, D, dtype, layouts[1])
        (self.k, ki), (self.k_new, ko) = rows(g, B, N, max(Hk, 1), D, dtype, layouts[1]), rows(g, B, N, max(Hk, 1), D, dtype, layouts[0])
        self.Hk = Hk
        high = 2 ** 31 - 1 if far else 200
        self.positions = torch.randint(-high, high, (N, len(dims)) if shared else (B, N, len(dims)), generator=g, device="cuda", dtype=torch.int32)
        self.cfg = sd.AxesRopeConfig.make(batch=B, tokens=N, heads=H, kv_heads=Hk, head_dim=D, dims=dims, scale=scale, base=base,
                                          halves=int(halves), dtype=KIND[dtype], shared_positions=int(shared), q_in=qi, q_out=qo,
                                          k_in=ki, k_out=ko)

    def reference(self, x, backward=False):
        return rope_reference(x, self.positions, self.dims, self.base, self.scale, self.halves, backward)

    def pair(self, k, k_new):
        return (k, k_new) if self.Hk else (None, None)

    def check(self):
        sd.axes_rope(self.cfg, self.positions, self.q, self.q_new, *self.pair(self.k, self.k_new))
        within(self.q_new, *self.reference(self.q), "q")
        if self.Hk:
            within(self.k_new, *self.reference(self.k), "k")
        # the gradient, whose layouts are the other way round
        dq_out, dk_out = self.q_new.clone(memory_format=torch.preserve_format), self.k_new
        self.q_new.copy_(torch.randn_like(self.q_new.float()))
        ref_q, ref_k = self.reference(self.q_new, True), self.reference(dk_out, True)
        sd.axes_rope_backward(self.cfg, self.positions, self.q_new, self.q, *self.pair(dk_out, self.k))
        within(self.q, *ref_q, "dq")
        if self.Hk:
            within(self.k, *ref_k, "dk")
        del dq_out


ROPE = [
    # B, N, H, Hk, D, dims, halves, layouts
    (1, 1, 1, 0, 8, (2,), False, ("dense", "dense")),
    (1, 1, 40, 40, 128, (44, 42, 42), False, ("dense", "dense")),
    (2, 5, 3, 1, 128, (44, 42, 42), False, ("packed", "heads_first")),
    (1, 77, 12, 12, 128, (44, 42, 42), False, ("dense", "heads_first")),
    (3, 33, 4, 2, 64, (16, 24, 24), True, ("heads_first", "dense")),
    (1, 130, 5, 5, 128, (64, 64), True, ("packed", "dense")),
    (2, 19, 9, 3, 80, (36, 36), True, ("dense", "packed")),
    (1, 300, 2, 1, 256, (64, 64, 64, 64), False, ("heads_first", "heads_first")),
    (1, 257, 7, 0, 96, (96,), True, ("dense", "dense")),
    (4, 11, 6, 6, 40, (2, 2, 4, 10), False, ("packed", "packed")),
    (1, 2000, 3, 3, 16, (6, 10), True, ("dense", "dense")),
    (2, 3, 2, 2, 136, (100,), False, ("dense", "packed")),
]


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", ROPE, ids=lambda c: "B%d-N%d-H%d-%d-D%d-%s" % (*c[:5], "halves" if c[6] else "pairs"))
def test_rotary_positions_and_their_gradient(case, dtype):
    B, N, H, Hk, D, dims, halves, layouts = case
    Rope(B, N, H, Hk, D, dims, halves, dtype, layouts, seed=N).check()
    Rope(B, N, H, Hk, D, dims, halves, dtype, layouts, far=True, shared=True, scale=[0.5, -2.0, 7.25, 1.0][:len(dims)], base=500.0,
         seed=N + 1).check()
