"""CPU tests of the C ABI of 4-bit matrices, their products and rotary positions: the library exports what
include/sdv2_project.h declares, bad arguments are refused on the host with a status and a message, and the binding and the session
refuse tensors that do not match the configuration.  No kernel is launched here."""
import ctypes
import os
import pickle
import re
import subprocess

import pytest
import torch

import streaming_causal_video_gb300 as sd
from project_common import packed, quantized, special, values
from streaming_causal_video_gb300 import _project

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20          # an aligned non-null address; every call below is rejected before use


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build_library()


def test_library_exports_every_declared_function():
    text = open(os.path.join(ROOT, "include", "sdv2_project.h")).read()
    declared = sorted(set(re.findall(r"\b(sdv2_[a-z0-9_]+)\s*\(const", text)))
    assert declared == sorted(_project.PROJECT_EXPORTS)
    for n in declared:
        assert hasattr(sd.lib(), n), n


def test_struct_layouts(tmp_path):
    """Sizes and offsets of the mirrors, against a C compiler's."""
    probes = [("sdv2_mx4_cfg", sd.Mx4Config, ["x_dtype", "x_row_stride"]),
              ("sdv2_mx4_product_cfg", sd.Mx4ProductConfig, ["out_dtype", "out_row_stride"]),
              ("sdv2_axes_rope_cfg", sd.AxesRopeConfig, ["tokens", "dims", "halves", "base", "scale", "q_in", "k_out"]),
              ("sdv2_rope_strides", sd.RopeStrides, ["head_stride", "batch_stride"])]
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "sdv2_project.h"', "int main(void) {"]
    for name, _, fields in probes:
        lines.append('printf("%%zu", sizeof(%s));' % name)
        lines += ['printf(" %%zu", offsetof(%s, %s));' % (name, f) for f in fields]
        lines.append('printf("\\n");')
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.split("\n")
    for line, (_, cls, fields) in zip(out, probes):
        assert [int(x) for x in line.split()] == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fields]


def mx4(**over):
    d = dict(rows=6, cols=40)
    d.update(over)
    return sd.Mx4Config.make(**d)


def product(**over):
    d = dict(rows=6, cols=40, depth=100)
    d.update(over)
    return sd.Mx4ProductConfig.make(**d)


def rope(**over):
    d = dict(batch=2, tokens=5, heads=4, kv_heads=2, head_dim=128, dims=(44, 42, 42))
    d.update(over)
    return sd.AxesRopeConfig.make(**d)


def status(fn, *a, **k):
    with pytest.raises(sd.SDV2Error) as e:
        fn(*a, **k)
    return e.value.status


def past_checks(call, *a, **k):
    """Valid arguments end at the device check.  With a GPU nothing is called: their addresses are none of it."""
    return torch.cuda.is_available() or call(*a, **k) in (2, 3)


def quantize(c, x=FAKE, codes=FAKE, scales=FAKE):
    return status(sd.mx4_quantize, c, x, codes, scales, stream=0)


def dequantize(c, codes=FAKE, scales=FAKE, y=FAKE):
    return status(sd.mx4_dequantize, c, codes, scales, y, stream=0)


def multiply(c, a_codes=FAKE, a_scales=FAKE, b_codes=FAKE, b_scales=FAKE, out=FAKE, ws=FAKE, **kw):
    return status(sd.mx4_product, c, a_codes, a_scales, b_codes, b_scales, out, ws, stream=0, **kw)


def turn(c, positions=FAKE, q=FAKE, q_out=2 * FAKE, k=3 * FAKE, k_out=4 * FAKE, fn=None):
    return status(fn or sd.axes_rope, c, positions, q, q_out, k, k_out, stream=0)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (128, 129), (129, 5120), (4680, 1536), (1 << 30, 1 << 10)])
def test_sizes(rows, cols):
    c = mx4(rows=rows, cols=cols)
    tiles = -(-cols // 128)
    assert sd.mx4_codes_bytes(c) == rows * tiles * 64
    assert sd.mx4_scales_bytes(c) == -(-rows // 128) * tiles * 512
    assert sd.mx4_workspace_bytes(product(rows=rows, depth=cols)) == 256


@pytest.mark.parametrize("over,want", [
    (dict(rows=0), 1), (dict(rows=-1), 1), (dict(cols=0), 1), (dict(rows=(1 << 30) + 1), 1), (dict(cols=(1 << 30) + 1), 1),
    (dict(x_dtype=2), 1), (dict(x_dtype=-1), 1), (dict(transposed=2), 1), (dict(x_row_stride=39), 1), (dict(x_row_stride=-40), 1),
    (dict(transposed=1, x_row_stride=5), 1), (dict(x_row_stride=(1 << 38) + 1), 2),
])
def test_invalid_matrices(over, want):
    c = mx4(**over)
    assert sd.mx4_codes_bytes(c) == 0 and sd.mx4_scales_bytes(c) == 0
    assert quantize(c) == want and dequantize(c) == want
    assert sd.lib().sdv2_last_error()


def test_invalid_matrix_arguments():
    c = mx4()
    for bad in (None, FAKE + 8):
        for name in ("x", "codes", "scales"):
            assert quantize(c, **{name: bad}) == 1, name
        for name in ("y", "codes", "scales"):
            assert dequantize(c, **{name: bad}) == 1, name
    assert dequantize(mx4(transposed=1)) == 2
    assert past_checks(quantize, c) and past_checks(dequantize, c) and past_checks(quantize, mx4(transposed=1, x_row_stride=6))


@pytest.mark.parametrize("over,want", [
    (dict(rows=0), 1), (dict(cols=0), 1), (dict(depth=0), 1), (dict(rows=-5), 1), (dict(depth=(1 << 30) + 1), 1), (dict(out_dtype=7), 1),
    (dict(activation=2), 1), (dict(activation=-1), 1), (dict(out_row_stride=39), 1), (dict(out_row_stride=-1), 1),
    (dict(out_row_stride=(1 << 38) + 1), 2), (dict(rows=1 << 30, cols=1 << 30), 2),
])
def test_invalid_products(over, want):
    c = product(**over)
    assert sd.mx4_workspace_bytes(c) == 0
    assert status(sd.mx4_workspace_init, c, FAKE, stream=0) == want
    assert multiply(c) == want


def test_invalid_product_arguments():
    c = product()
    for bad in (None, FAKE + 8):
        for name in ("a_codes", "a_scales", "b_codes", "b_scales", "out", "ws"):
            assert multiply(c, **{name: bad}) == 1, name
        assert status(sd.mx4_workspace_init, c, bad, stream=0) == 1
    assert multiply(c, bias=FAKE + 4) == 1
    assert past_checks(multiply, c) and past_checks(multiply, c, bias=FAKE) and past_checks(multiply, product(out_row_stride=41))


@pytest.mark.parametrize("over,want", [
    (dict(batch=0), 1), (dict(batch=65536), 1), (dict(heads=0), 1), (dict(heads=65536), 1), (dict(kv_heads=-1), 1), (dict(tokens=0), 1),
    (dict(tokens=(1 << 30) + 1), 1), (dict(head_dim=0), 1), (dict(head_dim=130), 1), (dict(head_dim=264), 1), (dict(dtype=2), 1),
    (dict(dims=(44, 42, 44)), 1), (dict(dims=(43, 42)), 1), (dict(dims=(-2, 42)), 1), (dict(halves=2), 1), (dict(shared_positions=-1), 1),
    (dict(base=1.0), 1), (dict(base=float("nan")), 1), (dict(base=float("inf")), 1), (dict(scale=(1.0, float("nan"), 1.0)), 1),
    (dict(scale=(1.0, 1.0, 2.0 ** 21)), 1),
    (dict(q_in=dict(token_stride=-8)), 1), (dict(q_in=dict(token_stride=120)), 1), (dict(q_out=dict(head_stride=64)), 1),
    (dict(k_in=dict(head_stride=132)), 1), (dict(k_out=dict(batch_stride=4)), 1), (dict(q_in=dict(batch_stride=(1 << 38) + 8)), 2),
    (dict(tokens=1 << 30, q_in=dict(token_stride=1 << 37)), 2),
])
def test_invalid_rotations(over, want):
    c = rope(**over)
    assert turn(c) == want and turn(c, fn=sd.axes_rope_backward) == want


def test_invalid_rotation_arguments():
    c = rope()
    for bad in (None, FAKE + 8):
        for name in ("positions", "q", "q_out", "k", "k_out"):
            assert turn(c, **{name: bad}) == 1, name
    # in place only with the same strides
    assert turn(rope(q_out=dict(token_stride=1024)), q=FAKE, q_out=FAKE) == 1
    assert b"in place" in sd.lib().sdv2_last_error()
    assert past_checks(turn, c) and past_checks(turn, c, q=FAKE, q_out=FAKE) and past_checks(turn, rope(dims=(0, 42, 42)))
    assert past_checks(turn, rope(kv_heads=0), k=None, k_out=None)
    with pytest.raises(ValueError, match="one to four axes"):
        rope(dims=())
    with pytest.raises(ValueError, match="one to four axes"):
        rope(scale=(1.0,))
    with pytest.raises(TypeError, match="no field"):
        rope(head=3)


def test_the_binding_refuses_tensors_that_do_not_match():
    bf, u8 = torch.bfloat16, torch.uint8
    c = mx4()
    for x in (torch.zeros(6, 40, dtype=bf), torch.zeros(6, 41), torch.zeros(6, 40, dtype=torch.float16)):
        with pytest.raises(ValueError):
            sd.mx4_quantize(c, x, FAKE, FAKE, stream=0)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sd.mx4_quantize(c, FAKE, torch.zeros(384, dtype=u8), FAKE, stream=0)
    with pytest.raises(ValueError):
        sd.mx4_product(product(), FAKE, FAKE, FAKE, FAKE, torch.zeros(6, 40, dtype=bf), FAKE, stream=0)
    with pytest.raises(ValueError):
        sd.axes_rope(rope(), torch.zeros(2, 5, 3, dtype=torch.int64), FAKE, FAKE, FAKE, FAKE, stream=0)


def test_a_changed_configuration_is_derived_again():
    c = mx4()
    assert c.derived()[0] == 6 * 64
    c.rows = 7
    assert c.derived()[0] == 7 * 64 and pickle.loads(pickle.dumps(c)).derived() == c.derived()
    r = rope()
    assert r.derived()[1][1] == (5 * 512, 512, 128, 1)
    r.q_in = sd.RopeStrides(token_stride=1024)
    assert r.derived()[1][1] == (5 * 1024, 1024, 128, 1)


def test_the_plain_quantiser_on_known_numbers():
    """The tests' own implementation: levels and ties, the scale's bound, and the documented bytes."""
    x = torch.zeros(2, 64)
    x[0, :16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 0.26, 0.74, 1.26, 1.74, 2.51, 3.49, 5.1, -6.5])
    x[0, 32] = 7.0000005
    code, byte, bad = quantized(x)
    assert byte.tolist() == [[127, 128], [0, 0]] and not bad.any()
    assert values(code, byte)[0, :16].tolist() == [0, 1, 1, 2, 2, 4, 4, 6, 0.5, 0.5, 1.5, 1.5, 3, 3, 6, -6]
    assert values(code, byte)[0, 32] == 8.0 and not values(code, byte)[1].any()
    codes, scales = packed(code, byte, 2, 64)
    # 0.25 and 0.75 become 0 and 1 (codes 0 and 2, the even column in the low bits), 1.25 and 1.75 become 1 and 2 (2 and 4), ...
    assert codes.shape == (2, 64) and codes[0, :8].tolist() == [0x20, 0x42, 0x64, 0x76, 0x11, 0x33, 0x55, 0xF7]
    assert scales.shape == (1, 1, 32, 4, 4) and scales[0, 0, 0, 0].tolist() == [127, 128, 0, 0] and scales[0, 0, 1, 0].tolist() == [0] * 4
    g = torch.Generator().manual_seed(1)
    y = special(torch.randn(40, 70, generator=g), g)
    code, byte, bad = quantized(y)
    assert bad.sum() == 2 and byte[bad].tolist() == [255, 255]
    back, n = values(code, byte), y.double()
    scale = torch.exp2(byte.double() - 127).repeat_interleave(32, 1)[:, :70]
    ok = ~bad.repeat_interleave(32, 1)[:, :70]
    # the nearest level is at most half of the step at 4 to 6 away, and at most 1 where a magnitude above 6 is cut off
    assert bool(((back - n).abs()[ok] <= scale[ok]).all())


def session(**over):
    """A session's shape without its buffers (there is no GPU here)."""
    s = object.__new__(sd.StreamSession)
    s.cfg = sd.StreamConfig.make(batch=1, heads=2, head_dim=128, rope_t=44, rope_h=42, rope_w=42, rope_base=1e4, grid_h=2, grid_w=3,
                                 chunk_frames=2, sink_frames=1, window_frames=3, refresh_chunks=5, qkv_token_stride=0)
    s.ws = torch.zeros(1, dtype=torch.uint8)
    s.start_frames = [7]
    s.products, s.loaded, s.scratch, s.ropes = {}, {}, {}, {}
    return s


def test_session_positions():
    s = session()
    pos = s.chunk_positions([6])
    assert pos.shape == (1, 12, 3) and pos.dtype == torch.int32
    # chunk 6 of a stream that starts at frame 7 and starts over every 5 chunks: frames 7 + 2 * 1 and one on
    assert pos[0, :, 0].tolist() == [9] * 6 + [10] * 6
    assert pos[0, :6, 1].tolist() == [0, 0, 0, 1, 1, 1] and pos[0, :6, 2].tolist() == [0, 1, 2] * 2


def test_session_and_matrix_refuse_what_does_not_fit():
    s = session()
    m = sd.Mx4Matrix(6, 40, "cpu")
    assert m.codes.numel() == 384 and m.scales.numel() == 512
    with pytest.raises(ValueError, match="at least one row"):
        sd.Mx4Matrix(0, 3, "cpu")
    for bad in (torch.zeros(6, 41), torch.zeros(40, 6), torch.zeros(6, 40, dtype=torch.float16), torch.zeros(40, 6).t(),
                torch.zeros(1, 40).expand(6, 40)):
        with pytest.raises(ValueError):
            m.load(bad)
    with pytest.raises(ValueError, match="two dimensions"):
        sd.Mx4Matrix.of(torch.zeros(2, 3, 4))
    with pytest.raises(ValueError, match="contiguous"):
        s.quantize_step(torch.zeros(40, 6).t())
    with pytest.raises(ValueError, match="columns"):
        s.project_step(m, sd.Mx4Matrix(3, 39, "cpu"), torch.zeros(3, 6))
    with pytest.raises(ValueError, match="rows of 6"):
        s.project_step(m, sd.Mx4Matrix(3, 40, "cpu"), torch.zeros(4, 6))
    with pytest.raises(ValueError, match="contiguous"):
        s.project_step(m, sd.Mx4Matrix(3, 40, "cpu"), torch.zeros(6, 3).t())
    with pytest.raises(ValueError, match="bias has"):
        s.project_step(m, sd.Mx4Matrix(3, 40, "cpu"), torch.zeros(3, 6), bias=torch.zeros(5))
    q = torch.zeros(1, 12, 2, 128)
    pos = torch.zeros(1, 12, 3, dtype=torch.int32)
    for args in ((pos, q, torch.zeros(1, 12, 2, 64)), (pos, q[..., :64], q[..., :64]), (pos[:, :5], q, q), (pos, q, q, q[:, :5], q[:, :5]),
                 (pos, q.half(), q.half()), (pos, q, q, q, q[:, :, :1]), (pos, q, q, q), (pos, q, q, None, q)):
        with pytest.raises(ValueError):
            s.rope_step(*args)
    for chunks in ([1, 2], []):
        with pytest.raises(ValueError, match="chunk indexes"):
            s.chunk_positions(chunks)
    s.cfg.refresh_chunks = 0
    with pytest.raises(ValueError, match="past 32 bits"):
        s.chunk_positions([1 << 30])


def test_activations_of_many_lengths_share_memory():
    s = session()
    s.ws = torch.zeros(1, dtype=torch.uint8)
    for rows in range(1, 700):
        with pytest.raises(ValueError):                        # there is no GPU to load it on
            s.quantize_step(torch.zeros(rows, 40))
        m, whole = s.loaded[rows, 40], sd.Mx4Matrix(rows, 40, "cpu")
        assert (m.rows, m.cols, m.codes.numel(), m.scales.numel()) == (rows, 40, whole.codes.numel(), whole.scales.numel())
    assert sorted(s.scratch) == [(n, 40) for n in (128, 256, 512, 1024)]
