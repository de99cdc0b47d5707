"""GPU tests of 4-bit matrices, their products and rotary positions, forward and backward, against plain 64-bit implementations
with derived bounds (project_common.py)."""
import math
import subprocess
import sys
import threading
from pathlib import Path

import pytest
import torch

import streaming_causal_video_gb300 as sd
from block_common import cross_reference
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


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad", [(2500, 1800, 0), (2500, 1800, 8), (2500, 1793, 0), (2500, 1793, 1), (2600, 1922, 0), (2600, 1921, 3),
                                           (1300, 1150, 0), (1300, 1151, 0), (2500, 1152, 0), (9800, 2, 0), (9800, 1, 0), (9800, 1, 2)])
def test_rows_enough_for_several_tiles_of_a_thread(rows, cols, pad, dtype):
    """Rows that begin on even and odd places, whole and cut tiles at the end of a thread's, and results between guard bytes."""
    g = cpu_gen(rows + cols)
    x = special(torch.randn(rows, cols, generator=g) * torch.exp(4 * torch.randn(rows, 1, generator=g)), g).to(dtype)
    view, _ = strided(x, pad)
    cfg = sd.Mx4Config.make(rows=rows, cols=cols, x_dtype=KIND[dtype], x_row_stride=cols + pad)
    codes, scales = buffers(cfg)
    sd.mx4_quantize(cfg, view, codes, scales)
    code, byte, bad = quantized(x)
    want_codes, want_scales = packed(code, byte, rows, cols)
    assert torch.equal(scales.cpu(), want_scales.flatten())
    sound = torch.nn.functional.pad(~bad.repeat_interleave(32, 1), (0, -bad.shape[1] % 4 * 32), value=True)[:, 0::2]
    assert torch.equal(codes.cpu().view(rows, -1)[sound], want_codes[sound])
    ref = values(code, byte)
    ref[bad.repeat_interleave(32, 1)[:, :cols]] = math.nan
    ref[ref.abs() >= 2.0 ** 128] *= math.inf
    base = torch.full((16 + rows * (cols + pad) + 16,), 77.0, dtype=dtype, device="cuda")
    inner = base[16:-16].view(rows, cols + pad)
    sd.mx4_dequantize(cfg, codes, scales, inner[:, :cols])
    assert torch.equal(inner[:, :cols].cpu().double().nan_to_num(nan=12345.0), ref.nan_to_num(nan=12345.0))
    assert bool((base[:16] == 77).all()) and bool((base[-16:] == 77).all()) and bool((inner[:, cols:] == 77).all())


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
DEEP = [(65, 300, 8200), (77, 1536, 8960), (512, 700, 4096), (300, 260, 20480), (256, 250, 7001),
        (700, 650, 8300)]


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


@pytest.mark.parametrize("out_dtype", [FP, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [(4100, 1600, 600), (4500, 1530, 1300), (4100, 1600, 2900), (4100, 1603, 2900), (9000, 2100, 2100), (260, 40000, 520)],
                         ids=str)
def test_products_of_several_tiles_of_a_pair(size, out_dtype):
    """Tiles of 128, 192 and 256 rows one after the other, whose operands the library quantises."""
    M, N, K = size
    g = torch.Generator(device="cuda").manual_seed(M)
    a, b = (torch.randn(n, K, generator=g, device="cuda") for n in (M, N))
    a4, b4 = sd.Mx4Matrix.of(a), sd.Mx4Matrix.of(b)
    a, b = a4.values(a).double(), b4.values(b).double()
    bias = torch.randn(N, generator=g, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for gelu in (False, True):
        cfg = sd.Mx4ProductConfig.make(rows=M, cols=N, depth=K, out_dtype=KIND[out_dtype], activation=sd.GELU if gelu else sd.NO_ACTIVATION)
        out = torch.full((M, N), math.nan, dtype=out_dtype, device="cuda")
        sd.mx4_product(cfg, a4.codes, a4.scales, b4.codes, b4.scales, out, ws, bias=bias)
        sd.check_device_error(ws)
        within(out, *product_reference(a, b, bias, gelu, out_dtype), "out")


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


# ---- products: exact sums, NaN, places, graphs, errors ---------------------------------------------

SHAPES = [(3, 200, 2048), (40, 130, 2048), (70, 300, 2048), (90, 260, 9000), (300, 260, 1300), (600, 700, 2048), (300, 1030, 8200),
          (1560, 1530, 700), (2040, 2050, 300), (4100, 1600, 300)]
# few rows in one part and in several; tiles of 128 rows, their depth shared by four pairs and by two; tiles of 192 and of 256 rows,
# and several tiles of a pair


@pytest.mark.parametrize("size", SHAPES, ids=str)
def test_sums_that_32_bits_hold_are_exact(size):
    """Codes and scales 2^0 to 2^1 at random: every partial sum is a multiple of 1/4 below 2^24 quarters (36 * 4 * K / 1 quarters
    at most 1.3 million), which no order of additions and no cutting off at 2^-24 of the largest changes."""
    M, N, K = size
    g = cpu_gen(M)

    def operand(rows):
        code = torch.randint(0, 16, (rows, K), generator=g)
        byte = torch.randint(127, 129, (rows, -(-K // 32)), generator=g)
        codes, scales = packed(code, byte, rows, K)
        return values(code, byte).cuda(), (codes.cuda().flatten(), scales.cuda().flatten())
    (a, a4), (b, b4) = operand(M), operand(N)
    cfg = sd.Mx4ProductConfig.make(rows=M, cols=N, depth=K, out_dtype=sd.F32)
    ws, out = torch.zeros(256, dtype=torch.uint8, device="cuda"), torch.empty((M, N), device="cuda")
    sd.mx4_product(cfg, *a4, *b4, out, ws)
    sd.check_device_error(ws)
    assert torch.equal(out.double(), a @ b.t())


@pytest.mark.parametrize("size", SHAPES, ids=str)
def test_a_scale_of_nan_reaches_its_row_and_its_column_only(size):
    p = Product(*size, FP, bias=False, seed=2)
    tiles = -(-p.K // 128)

    def spoil(scales, row, block):
        at = (((row // 128) * tiles + block // 4) * 32 + row % 32) * 16 + row % 128 // 32 * 4 + block % 4
        scales[at] = 255
    spoil(p.a4[1], p.M - 1, 0)
    spoil(p.b4[1], p.N // 2, (p.K - 1) // 32)
    p.run()
    sd.check_device_error(p.ws)
    nan = torch.zeros((p.M, p.N), dtype=torch.bool, device="cuda")
    nan[p.M - 1], nan[:, p.N // 2] = True, True
    assert torch.equal(p.out.isnan(), nan)
    ref, tol = product_reference(p.a, p.b, None, False, FP)
    within(torch.where(nan, ref.float(), p.out), ref, tol, "out")


@pytest.mark.parametrize("size", SHAPES, ids=str)
def test_a_nan_leaves_its_neighbours_with_an_activation(size):
    """The activation takes columns two at a time."""
    for dtype in (FP, BF):
        p = Product(*size, dtype, gelu=True, seed=7)
        nan = torch.zeros((p.M, p.N), dtype=torch.bool, device="cuda")
        for n, value in ((1, math.nan), (p.N // 2, math.nan), (p.N // 2 + 3, math.inf), (p.N - 1, -math.inf)):
            p.bias[n] = value
            nan[:, n] = math.isnan(value)
        p.run()
        sd.check_device_error(p.ws)
        assert torch.equal(p.out.isnan(), nan)
        assert bool((p.out[:, p.N // 2 + 3] == math.inf).all())
        ref, tol = product_reference(p.a, p.b, torch.where(p.bias.isfinite(), p.bias, torch.zeros_like(p.bias)), True, dtype)
        sound = p.bias.isfinite()
        within(p.out[:, sound], ref[:, sound], tol[:, sound], "out")
        assert bool((p.out[:, p.N - 1].abs() <= 2.0 ** -40).all())


def test_extreme_scales():
    """Scales of 2^-127 and 2^126 that cancel: no intermediate leaves the range of 32 bits, in few rows and in tiles."""
    K = 256
    for M in (2, 80):
        code = torch.full((M, K), 7)                       # 6
        one = values(code, torch.full((M, K // 32), 127)).cuda()
        for ea, eb in ((253, 1), (0, 253), (250, 4), (127, 127)):
            a4 = [t.cuda().flatten() for t in packed(code, torch.full((M, K // 32), ea), M, K)]
            b4 = [t.cuda().flatten() for t in packed(code, torch.full((M, K // 32), eb), M, K)]
            cfg = sd.Mx4ProductConfig.make(rows=M, cols=M, depth=K, out_dtype=sd.F32)
            ws, out = torch.zeros(256, dtype=torch.uint8, device="cuda"), torch.empty((M, M), device="cuda")
            sd.mx4_product(cfg, *a4, *b4, out, ws)
            assert torch.equal(out.double(), one @ one.t() * 2.0 ** (ea + eb - 254)), (M, ea, eb)


@pytest.mark.parametrize("size", SHAPES, ids=str)
def test_products_are_deterministic_and_replay_from_graphs_that_share_a_workspace(size):
    p, q = Product(*size, BF, gelu=True, seed=1), Product(*size, BF, seed=5)
    q.ws = p.ws
    p.run()
    q.run()
    want = p.out.clone(), q.out.clone()
    graphs = []
    for x in (p, q):
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            x.run()
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        p.out.fill_(0)
        q.out.fill_(0)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):              # at the same time
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.out, want[0]) and torch.equal(q.out, want[1])
    p.check()


@pytest.mark.parametrize("size", SHAPES + [(5, 7, 100), (65, 129, 129)], ids=str)
def test_calls_write_only_their_outputs(size):
    """Every buffer lies between guard bytes; operands stay as they were."""
    M, N, K = size
    guard = 4096

    def guarded(n):
        base = torch.full((n + 2 * guard,), 0x5A, dtype=torch.uint8, device="cuda")
        return base, base[guard:guard + n]
    for kind, dtype, trans in ((sd.BF16, BF, 0), (sd.F32, FP, 1)):
        cfg = sd.Mx4Config.make(rows=M, cols=K, x_dtype=kind, transposed=trans)
        nc, ns = sd.mx4_codes_bytes(cfg), sd.mx4_scales_bytes(cfg)
        (cb, codes), (sb, scales) = guarded(nc), guarded(ns)
        x = torch.randn((K, M) if trans else (M, K), device="cuda").to(dtype)
        before = x.clone()
        sd.mx4_quantize(cfg, x, codes, scales)
        yb, y = guarded(M * K * 4)
        sd.mx4_dequantize(sd.Mx4Config.make(rows=M, cols=K, x_dtype=sd.F32), codes, scales, y.view(torch.float32).view(M, K))
        ob, o = guarded(M * N * dtype.itemsize)
        p = Product(M, N, K, dtype, seed=3)
        kept = [t.clone() for t in (*p.a4, *p.b4, p.bias)]
        wb, ws = guarded(256)
        ws.zero_()
        sd.mx4_product(p.cfg, *p.a4, *p.b4, o.view(dtype).view(M, N), ws, bias=p.bias)
        torch.cuda.synchronize()
        for base in (cb, sb, yb, ob, wb):
            assert bool((base[:guard] == 0x5A).all()) and bool((base[-guard:] == 0x5A).all())
        assert torch.equal(x, before) and all(torch.equal(a, b) for a, b in zip(kept, (*p.a4, *p.b4, p.bias)))
        assert not ws.any()


@pytest.mark.parametrize("size", [(20, 300), (300, 520), (700, 8300)], ids=str)
def test_a_matrix_with_itself(size):
    """Both operands may be the same matrix."""
    M, K = size
    a = sd.Mx4Matrix.of(torch.randn(M, K, generator=cpu_gen(M)).cuda())
    v = a.values(torch.empty(M, K, device="cuda")).double()
    cfg = sd.Mx4ProductConfig.make(rows=M, cols=M, depth=K, out_dtype=sd.F32)
    ws, out = torch.zeros(256, dtype=torch.uint8, device="cuda"), torch.empty(M, M, device="cuda")
    sd.mx4_product(cfg, a.codes, a.scales, a.codes, a.scales, out, ws)
    sd.check_device_error(ws)
    within(out, *product_reference(v, v, None, False, FP), "out")


def test_rows_from_a_multiple_of_128_are_a_matrix_of_their_own():
    """One projection's part of a packed weight, and the tokens of one stream of a batch."""
    K, N, first, count = 300, 700, 256, 333
    p = Product(130, N, K, FP, seed=9)
    tiles = -(-K // 128)
    codes, scales = p.b4[0][first * tiles * 64:], p.b4[1][first // 128 * tiles * 512:]
    cfg = sd.Mx4ProductConfig.make(rows=130, cols=count, depth=K, out_dtype=sd.F32)
    out = torch.empty((130, count), device="cuda")
    sd.mx4_product(cfg, *p.a4, codes, scales, out, p.ws, bias=p.bias[first:first + count].clone())
    ref, tol = product_reference(p.a, p.b[first:first + count], p.bias[first:first + count], False, FP)
    within(out, ref, tol, "part")


@pytest.mark.parametrize("size,step", [((3, 200, 2048), 3), ((16, 300, 9000), 30), ((70, 300, 2048), 0), ((90, 260, 9000), 20), ((600, 700, 2048), 7),
                                       ((300, 1030, 8200), 12), ((1560, 1530, 700), 1), ((2040, 2050, 300), 0), ((4100, 1600, 300), 1)],
                         ids=str)
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(size, step):
    p = Product(*size, BF, seed=4)
    p.run()
    p.check()
    try:
        sd.set_wait_timeout_ns(20_000_000)
        sd.debug_drop_kv_tile(step)
        p.run()
        with pytest.raises(sd.SDV2Error) as e:
            sd.check_device_error(p.ws)
        assert e.value.status == 4
    finally:
        sd.debug_drop_kv_tile(-1)
        sd.set_wait_timeout_ns(2_000_000_000)
    p.out.fill_(0)
    p.run()
    p.check()


def test_results_follow_what_copies_and_other_streams_bring():
    """Quantisation, product and rotation chained behind copies, kernels and another stream's work, eagerly and captured; the inputs
    change right in front of every call."""
    g = torch.Generator(device="cuda").manual_seed(3)
    M, N, K, H = 300, 256, 512, 2
    x0 = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    w = sd.Mx4Matrix.of(torch.randn(N, K, generator=g, device="cuda").bfloat16())
    pos0 = torch.randint(0, 1000, (1, M, 2), generator=g, device="cuda", dtype=torch.int32)
    x, pos = torch.empty_like(x0), torch.empty_like(pos0)
    x4 = sd.Mx4Matrix(M, K)
    cfg = sd.Mx4ProductConfig.make(rows=M, cols=N, depth=K)
    ws, y = torch.zeros(256, dtype=torch.uint8, device="cuda"), torch.empty(M, N, dtype=BF, device="cuda")
    rc = sd.AxesRopeConfig.make(batch=1, tokens=M, heads=H, head_dim=N // H, dims=(64, 64))
    z = torch.empty_like(y)
    busy, other = torch.zeros(64 << 20, device="cuda"), torch.cuda.Stream()

    def run(kind):
        main = torch.cuda.current_stream()
        x.fill_(7.0)
        pos.fill_(5)
        busy.add_(1.0)
        if kind == "stream":
            other.wait_stream(main)
            with torch.cuda.stream(other):
                x.copy_(x0 * 1.0)
                pos.copy_(pos0 + 0)
            main.wait_stream(other)
        elif kind == "copy":
            x.copy_(x0)
            pos.copy_(pos0)
        else:
            torch.mul(x0, 1.0, out=x)
            torch.add(pos0, 0, out=pos)
        x4.load(x)
        sd.mx4_product(cfg, x4.codes, x4.scales, w.codes, w.scales, y, ws)
        sd.axes_rope(rc, pos, y.view(1, M, H, N // H), z.view(1, M, H, N // H))
        return z.clone()
    want = run("copy")
    torch.cuda.synchronize()
    assert float(want.float().abs().max()) > 0
    for kind in ("copy", "kernel", "stream"):
        for _ in range(3):
            assert torch.equal(run(kind), want), kind
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            got = run(kind)
        for _ in range(3):
            graph.replay()
            assert torch.equal(got, want), "captured " + kind


FIRST_CALLS = """
import sys, torch
sys.path.insert(0, sys.argv[1])
import streaming_causal_video_gb300 as sd
g = torch.Generator(device="cuda").manual_seed(1)
cases = []
for M, N, K in ((3, 200, 2048), (70, 300, 2048), (90, 260, 9000), (600, 700, 2048)):
    a, b = (sd.Mx4Matrix(n, K) for n in (M, N))
    cfg = sd.Mx4ProductConfig.make(rows=M, cols=N, depth=K)
    cases.append((torch.randn(M, K, generator=g, device="cuda"), torch.randn(K, N, generator=g, device="cuda"), a, b, cfg,
                  torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"), torch.zeros(M, N, device="cuda")))
ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
rc = sd.AxesRopeConfig.make(batch=1, tokens=9, heads=2, head_dim=64, dims=(20, 20), halves=1)
pos, q = torch.arange(18, device="cuda", dtype=torch.int32).view(1, 9, 2), torch.randn(1, 9, 2, 64, generator=g, device="cuda").bfloat16()
r = torch.zeros_like(q)
def work():
    for x, w, a, b, cfg, y, v in cases:
        a.load(x)
        b.load(w, transposed=True)
        sd.mx4_product(cfg, a.codes, a.scales, b.codes, b.scales, y, ws)
    sd.axes_rope(rc, pos, q, r)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):                # the first calls of the process are captured
    work()
graph.replay()
torch.cuda.synchronize()
got = [c[5].clone() for c in cases] + [r.clone()]
for c in cases:
    c[5].zero_()
r.zero_()
work()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, [c[5] for c in cases] + [r]))
assert all(float(t.float().abs().max()) > 0 for t in got)
sd.check_device_error(ws)
print("same")
"""


def test_first_calls_of_a_process_inside_a_capture():
    run = subprocess.run([sys.executable, "-c", FIRST_CALLS, str(Path(__file__).resolve().parents[1])], capture_output=True,
                         text=True, timeout=240)
    assert run.returncode == 0 and run.stdout.strip().endswith("same"), run.stderr[-2000:]


def test_calls_from_several_host_threads():
    """First and later calls of several kernels from threads with streams of their own; the results are those of the calls alone."""
    cases = [Product(*SHAPES[i % len(SHAPES)], (BF, FP)[i % 2], seed=40 + i) for i in range(8)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    failed = []

    def body(p, s):
        try:
            for _ in range(50):
                p.run(stream=s)
        except Exception as e:                     # noqa: BLE001 (reported by the test's thread)
            failed.append(e)
    threads = [threading.Thread(target=body, args=a) for a in zip(cases, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed[0]
    for p in cases:
        p.check()


def test_matrices_beyond_2_to_the_31_elements():
    """Offsets past 32 bits in x, its values and a product's result; rows at both ends against the plain implementation."""
    rows, cols = 66000, 32800
    x = torch.empty((rows, cols), dtype=BF, device="cuda")
    pick = torch.tensor([0, 1, rows // 2, rows - 2, rows - 1])
    x.view(-1).copy_(torch.arange(97, device="cuda").sub(48).bfloat16().repeat(rows * cols // 97 + 1)[:rows * cols])
    m = sd.Mx4Matrix.of(x)
    code, byte, _ = quantized(x[pick])
    want = values(code, byte)
    y = torch.empty((rows, cols), dtype=BF, device="cuda")
    m.values(y)
    assert torch.equal(y[pick].cpu().double(), want)
    t = sd.Mx4Matrix.of(x, transposed=True)                    # 32800 rows of 66000 columns
    ends = torch.tensor([0, 17, cols - 1])
    code, byte, _ = quantized(x[:, ends].t())
    want_codes, _ = packed(code, byte, 3, rows)
    assert torch.equal(t.codes.view(cols, -1)[ends].cpu(), want_codes)
    del y, t
    a, b = (Product.operand(torch.randn(n, 40, generator=cpu_gen(n))) for n in (rows, cols))
    cfg = sd.Mx4ProductConfig.make(rows=rows, cols=cols, depth=40)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sd.mx4_product(cfg, *a[1], *b[1], x, ws)
    sd.check_device_error(ws)
    ref, tol = product_reference(a[0][pick], b[0], None, False, BF)
    within(x[pick], ref, tol, "rows at the ends")


@pytest.mark.parametrize("size", [(200, 96, 130), (1001, 300, 257)], ids=str)
def test_gradients_of_a_product_are_products(size):
    """dx = dy w and dw = dy^T x from matrices quantised along the contracted side, against the formula on the quantised values."""
    M, N, K = size
    g = cpu_gen(M)
    x, w, dy = (torch.randn(s, generator=g).bfloat16() for s in ((M, K), (N, K), (M, N)))
    on = lambda t: t.cuda()
    dy4, wt4 = sd.Mx4Matrix.of(on(dy)), sd.Mx4Matrix.of(on(w), transposed=True)
    dyt4, xt4 = sd.Mx4Matrix.of(on(dy), transposed=True), sd.Mx4Matrix.of(on(x), transposed=True)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    plain = lambda t: values(*quantized(t)[:2]).cuda()
    for a4, b4, a, b, shape, dtype in ((dy4, wt4, plain(dy), plain(w.t()), (M, K), BF), (dyt4, xt4, plain(dy.t()), plain(x.t()), (N, K), FP)):
        out = torch.empty(shape, dtype=dtype, device="cuda")
        cfg = sd.Mx4ProductConfig.make(rows=a4.rows, cols=b4.rows, depth=a4.cols, out_dtype=KIND[dtype])
        sd.mx4_product(cfg, a4.codes, a4.scales, b4.codes, b4.scales, out, ws)
        within(out, *product_reference(a, b, None, False, dtype), "gradient")
    # and against differences: the product is linear in its operands' values, so a difference of any size is the gradient's
    dx = torch.empty((M, K), device="cuda")
    cfg = sd.Mx4ProductConfig.make(rows=M, cols=K, depth=N, out_dtype=sd.F32)
    sd.mx4_product(cfg, dy4.codes, dy4.scales, wt4.codes, wt4.scales, dx, ws)
    bump = torch.randn(M, K, generator=g).double().cuda()
    wv, dyv = plain(w.t()).t(), plain(dy)
    loss = lambda v: float((v @ wv.t() * dyv).sum())
    xv = plain(x)
    step = loss(xv + bump) - loss(xv - bump)
    slack = float(product_reference(dyv, wv.t(), None, False, FP)[1].mul(bump.abs()).sum())
    assert abs(step / 2 - float((dx.double() * bump).sum())) <= slack + 1e-9 * abs(step)


# ---- rotary positions: places, values and use ----------------------------------------------------------

@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "f32"])
def test_rotation_in_place_and_back(dtype, halves):
    r = Rope(2, 70, 5, 2, 96, (36, 20), halves, dtype, ("packed", "packed"), seed=1)
    sd.axes_rope(r.cfg, r.positions, r.q, r.q_new, r.k, r.k_new)
    q, k = r.q.clone(), r.k.clone()
    sd.axes_rope(r.cfg, r.positions, r.q, r.q, r.k, r.k)
    assert torch.equal(r.q, r.q_new) and torch.equal(r.k, r.k_new)
    sd.axes_rope_backward(r.cfg, r.positions, r.q, r.q, r.k, r.k)
    # two rotations that undo each other: two bounds, each of at most 2^-21 of both dims and a rounding of what has their size
    for back, was in ((r.q, q), (r.k, k)):
        size = was.double().abs().amax(-1, keepdim=True) * 2 ** 0.5 + 1e-9
        within(back, was.double(), 2 * (2.0 ** -20 + 2 * HALF[dtype]) * size.expand(was.shape), "back")
    # dims behind the axes are copied, whatever they hold
    r.q[..., 56:] = torch.tensor(math.inf, dtype=dtype)
    r.q[..., 57] = math.nan
    sd.axes_rope(r.cfg, r.positions, r.q, r.q_new, r.k, r.k_new)
    assert torch.equal(r.q_new[..., 56:].nan_to_num(nan=5.0), r.q[..., 56:].nan_to_num(nan=5.0)) and bool(r.q_new[..., :56].isfinite().all())


def test_gradient_of_the_rotation_against_differences():
    """The rotation is linear: a difference of any size is the gradient's, up to the bounds of both."""
    r = Rope(1, 40, 3, 1, 64, (20, 30), False, FP, ("dense", "heads_first"), far=True, seed=2)
    g = torch.Generator(device="cuda").manual_seed(5)
    for x, x_new, heads in ((r.q, r.q_new, 3), (r.k, r.k_new, 1)):
        bump, dy = (torch.randn(x.shape, generator=g, device="cuda") for _ in range(2))
        outs = []
        for sign in (1, -1):
            xq, xk = (x + sign * bump if t is x else t.clone() for t in (r.q, r.k))
            yq, yk = torch.empty_like(r.q_new), torch.empty_like(r.k_new)
            cfg = r.cfg
            sd.axes_rope(cfg, r.positions, xq, yq, torch.empty_like(r.k).copy_(xk), yk)
            outs.append((yq if x is r.q else yk).double())
        step = float(((outs[0] - outs[1]) * dy.double()).sum()) / 2
        dq_out, dk_out = torch.zeros_like(r.q_new), torch.zeros_like(r.k_new)
        (dq_out if x is r.q else dk_out).copy_(dy)
        dq, dk = torch.empty_like(r.q), torch.empty_like(r.k)
        sd.axes_rope_backward(r.cfg, r.positions, dq_out, dq, dk_out, dk)
        got = float(((dq if x is r.q else dk).double() * bump.double()).sum())
        # each of the three rotations is off by at most 2^-21 + 2^-23 of both dims of a pair
        slack = 3 * 2.0 ** -20 * float((x.abs() + bump.abs()).double().sum(-1).mul(dy.abs().double().sum(-1)).sum())
        assert abs(step - got) <= slack


@pytest.mark.parametrize("B,H,Hk", [(65535, 1, 1), (1, 65535, 65535), (1, 65535, 0)])
def test_rotation_of_the_most_streams_and_heads(B, H, Hk):
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k = (torch.randn(B, 1, n, 8, generator=g, device="cuda").bfloat16() for n in (H, max(Hk, 1)))
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, 1, 1), generator=g, device="cuda", dtype=torch.int64).int()
    cfg = sd.AxesRopeConfig.make(batch=B, tokens=1, heads=H, kv_heads=Hk, head_dim=8, dims=(6,))
    new = [torch.full_like(t, math.nan) for t in (q, k)]
    sd.axes_rope(cfg, pos, q, new[0], k, new[1])
    for x, y in list(zip((q, k), new))[:2 if Hk else 1]:
        within(y, *rope_reference(x, pos, (6,), 10000.0, (), False), "rotated")
    assert Hk or bool(new[1].isnan().all())


def test_rotation_beyond_2_to_the_31_elements():
    B, N, H, D = 1, 600000, 30, 128
    q = torch.empty((B, N, H, D), dtype=BF, device="cuda")
    q.view(-1).copy_(torch.arange(97, device="cuda").sub(48).bfloat16().repeat(q.numel() // 97 + 1)[:q.numel()])
    pos = torch.arange(N, device="cuda", dtype=torch.int32)[:, None].repeat(1, 3).contiguous()
    cfg = sd.AxesRopeConfig.make(batch=B, tokens=N, heads=H, head_dim=D, dims=(44, 42, 42), shared_positions=1)
    out = torch.empty_like(q)
    sd.axes_rope(cfg, pos, q, out)
    for n in (0, N // 2, N - 1):
        ref, tol = rope_reference(q[:, n:n + 1], pos[n:n + 1], (44, 42, 42), 10000.0, (), False)
        within(out[:, n:n + 1], ref, tol, "token %d" % n)


def test_a_session_turns_tokens_as_the_append_does():
    """The chunk's positions and rope_step give what the append to the cache writes for q, up to a rounding of the sine and cosine:
    a step of bf16 where that decides it."""
    cfg = sd.StreamConfig.make(batch=2, heads=3, head_dim=128, rope_t=44, rope_h=42, rope_w=42, rope_base=1e4, grid_h=5, grid_w=7,
                               chunk_frames=3, sink_frames=3, window_frames=6, refresh_chunks=4, qkv_token_stride=0)
    sess = sd.StreamSession(cfg, 1, [0, 100000], "cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k, v = (torch.randn(2, cfg.nq, 3, 128, generator=g, device="cuda").bfloat16() for _ in range(3))
    for chunk in (0, 5):
        sess.layer_step(0, [chunk, chunk], q, k, v)
        pos = sess.chunk_positions([chunk, chunk])
        mine, heads = torch.empty_like(q), torch.empty_like(sess.q_rot)
        sess.rope_step(pos, q, mine)
        sess.rope_step(pos, q, heads.transpose(1, 2))
        assert torch.equal(mine, heads.transpose(1, 2))
        ref, tol = rope_reference(q, pos, (44, 42, 42), 1e4, (), False)
        within(sess.q_rot.transpose(1, 2), ref, tol, "append")
        within(mine, ref, tol, "rope_step")
    one = sess.rope_step(pos[:, :1].contiguous(), q[:, :1], torch.empty_like(q[:, :1]))
    assert torch.equal(one, mine[:, :1])


def test_a_layer_as_a_session_runs_it():
    """norm -> 4-bit query projection -> rotation by the places of an image -> cross attention to its tokens, and the feed-forward
    pair with its activation, each step against a 64-bit implementation of the step on the same inputs."""
    cfg = sd.StreamConfig.make(batch=2, heads=2, head_dim=128, rope_t=44, rope_h=42, rope_w=42, rope_base=1e4, grid_h=6, grid_w=8,
                               chunk_frames=2, sink_frames=2, window_frames=4, refresh_chunks=0, qkv_token_stride=0)
    sess = sd.StreamSession(cfg, 1, [0, 9], "cuda")
    g = torch.Generator(device="cuda").manual_seed(6)
    f32 = lambda *s: torch.randn(s, generator=g, device="cuda")
    B, nq, H, D, C, Cf = 2, cfg.nq, 2, 128, 256, 640
    x, y = f32(B, nq, C), torch.empty(B, nq, C, dtype=BF, device="cuda")
    sess.norm_step(x, y, 0.3 * f32(B * 2, C), 0.3 * f32(B * 2, C), modulated=True)
    weights = {n: f32(*s) / s[1] ** 0.5 for n, s in (("q", (C, C)), ("k", (C, C)), ("up", (Cf, C)), ("down", (C, Cf)))}
    held = {n: sd.Mx4Matrix.of(w) for n, w in weights.items()}
    plain = lambda t: values(*quantized(t.reshape(-1, t.shape[-1]))[:2]).cuda()
    # one quantisation for both projections of the normed tokens
    y4 = sess.quantize_step(y)
    q, k = (torch.empty(B, nq, H, D, dtype=BF, device="cuda") for _ in range(2))
    bias = 0.1 * f32(C)
    sess.project_step(held["q"], y4, q.view(B, nq, C), bias=bias)
    sess.project_step(held["k"], y4, k.view(B, nq, C))
    for got, n, b in ((q, "q", bias), (k, "k", None)):
        within(got.view(-1, C), *product_reference(plain(y), plain(weights[n]), b, False, BF), n)
    pos = sess.chunk_positions([3, 3])
    refs = [rope_reference(t, pos, (44, 42, 42), 1e4, (), False) for t in (q, k)]
    sess.rope_step(pos, q, q, k, k)
    for got, ref in zip((q, k), refs):
        within(got, *ref, "rotated")
    v = f32(B, nq, H, D).bfloat16()
    sess.set_prompt(0, k, v, [nq, 50])
    out = sess.cross_step(0, q)
    out_ref, _, out_tol, _ = cross_reference(q, k, v, [nq, 50], 1 / math.sqrt(D))
    within(out, out_ref, out_tol, "cross attention")
    up, down = torch.empty(B, nq, Cf, dtype=BF, device="cuda"), torch.empty(B, nq, C, device="cuda")
    sess.project_step(held["up"], out.view(B, nq, C), up, bias=f32(Cf).mul_(0.1).clone(), activation=sd.GELU)
    sess.project_step(held["down"], up, down)
    within(down.view(-1, C), *product_reference(plain(up), plain(weights["down"]), None, False, FP), "down")
    # a pooled token goes the way of few rows
    few = torch.empty(B, C, device="cuda")
    sess.project_step(held["q"], x[:, 0].contiguous(), few)
    within(few, *product_reference(plain(x[:, 0]), plain(weights["q"]), None, False, FP), "one token of each stream")
    sd.check_device_error(sess.ws)
    with pytest.raises(ValueError, match="columns"):
        sess.project_step(held["down"], y, down)


def test_a_session_reports_its_products_and_captures_its_first_ones():
    cfg = sd.StreamConfig.make(batch=1, heads=2, head_dim=128, rope_t=44, rope_h=42, rope_w=42, rope_base=1e4, grid_h=6, grid_w=8,
                               chunk_frames=2, sink_frames=2, window_frames=4, refresh_chunks=0, qkv_token_stride=0)
    sess = sd.StreamSession(cfg, 1, [0], "cuda")
    g = torch.Generator(device="cuda").manual_seed(8)
    w = sd.Mx4Matrix.of(torch.randn(200, 520, generator=g, device="cuda"))
    x = [torch.randn(rows, 520, generator=g, device="cuda") for rows in (96, 100, 3)]
    y = [torch.zeros(len(t), 200, device="cuda") for t in x]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for a, b in zip(x, y):
            sess.project_step(w, a, b)
    sd.check_device_error(sess.ws)                             # nothing has run
    want = [sess.project_step(w, a, torch.empty_like(b)) for a, b in zip(x, y)]
    for t in y:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(y, want))
    try:
        sd.set_wait_timeout_ns(20_000_000)
        sd.debug_drop_kv_tile(1)
        sess.project_step(w, x[0], y[0])
        with pytest.raises(sd.SDV2Error):
            sd.check_device_error(sess.ws)
    finally:
        sd.debug_drop_kv_tile(-1)
        sd.set_wait_timeout_ns(2_000_000_000)
    assert torch.equal(sess.project_step(w, x[0], y[0]), want[0])
    sd.check_device_error(sess.ws)
