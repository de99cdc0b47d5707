"""CPU tests of the block operators' C ABI: the library exports what include/sdv2_block.h declares,
bad arguments are refused on the host with a status and a message, and the binding refuses tensors
that do not match the configuration.  No kernel is launched here."""
import copy
import ctypes
import os
import pickle
import re
import subprocess

import pytest
import torch

import streaming_causal_video_gb300 as sd
from streaming_causal_video_gb300 import _block

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20          # an aligned non-null address; every call below is rejected before use


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build_library()


def test_library_exports_every_declared_function():
    text = open(os.path.join(ROOT, "include", "sdv2_block.h")).read()
    declared = sorted(set(re.findall(r"\b(sdv2_[a-z0-9_]+)\s*\(const", text)))
    assert declared == sorted(_block.BLOCK_EXPORTS)
    for n in declared:
        assert hasattr(sd.lib(), n), n


def test_struct_layouts():
    assert ctypes.sizeof(sd.CrossConfig) == 80 and sd.CrossConfig.q_len.offset == 16
    assert sd.CrossConfig.kv_batch_stride.offset == 72
    assert ctypes.sizeof(sd.NormConfig) == 64 and sd.NormConfig.x_row_stride.offset == 24
    assert sd.NormConfig.eps.offset == 56
    with pytest.raises(TypeError, match="no field"):
        sd.CrossConfig.make(head=3)


def test_a_changed_configuration_is_derived_again():
    c = norm(rows=6)
    assert c.derived()[0][0] == (6, 40)
    d = copy.copy(c)
    c.rows = 7
    assert c.derived()[0][0] == (7, 40) and d.derived()[0][0] == (6, 40) and d.rows == 6
    assert pickle.loads(pickle.dumps(c)).derived() == c.derived()


def cross(**over):
    d = dict(batch=2, heads=4, kv_heads=2, head_dim=128, q_len=5, kv_len=7)
    d.update(over)
    return sd.CrossConfig.make(**d)


def norm(**over):
    d = dict(rows=6, cols=40, eps=1e-6)
    d.update(over)
    return sd.NormConfig.make(**d)


def status(fn, *a, **k):
    with pytest.raises(sd.SDV2Error) as e:
        fn(*a, **k)
    return e.value.status


def forward(c, q=FAKE, k=FAKE, v=FAKE, out=FAKE, ws=FAKE, **kw):
    return status(sd.cross_attention, c, q, k, v, out, ws, stream=0, **kw)


def backward(c, q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE, dout=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, ws=FAKE, **kw):
    return status(sd.cross_attention_backward, c, q, k, v, out, lse, dout, dq, dk, dv, ws, stream=0, **kw)


@pytest.mark.parametrize("over,want", [
    (dict(batch=0), 1), (dict(heads=0), 1), (dict(kv_heads=3), 1), (dict(kv_heads=-1), 1), (dict(kv_heads=8), 1),
    (dict(head_dim=64), 2), (dict(q_len=0), 1), (dict(q_len=-1), 1), (dict(q_len=(1 << 30) + 1), 1),
    (dict(kv_len=-1), 1), (dict(kv_len=(1 << 30) + 1), 1), (dict(q_token_stride=-8), 1),
    (dict(q_token_stride=120), 1), (dict(q_token_stride=516), 1), (dict(kv_head_stride=132), 1),
    (dict(kv_batch_stride=4), 1), (dict(kv_token_stride=(1 << 38) + 8), 2), (dict(batch=65536), 2),
    (dict(q_token_stride=1 << 37, q_len=1 << 30), 2),
])
def test_invalid_cross_configurations(over, want):
    c = cross(**over)
    assert sd.cross_workspace_bytes(c) == 0 and sd.cross_workspace_bytes(c, True) == 0
    assert status(sd.cross_workspace_init, c, FAKE, stream=0) == want
    if c.batch > 0 and c.batch < 100:
        assert forward(c) == want and backward(c) == want


def test_invalid_cross_arguments():
    c = cross()
    for bad in (None, FAKE + 8):
        for name in ("q", "k", "v", "out", "ws"):
            assert forward(c, **{name: bad}) == 1, name
        for name in ("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv", "ws"):
            assert backward(c, **{name: bad}) == 1, name
    assert forward(c, lse=FAKE + 4) == 1
    for lens in ([7, 8], [-1, 0]):
        assert forward(c, kv_lens=lens) == 1 and backward(c, kv_lens=lens) == 1
        assert b"kv_lens" in sd.lib().sdv2_last_error()
    with pytest.raises(ValueError, match="expected 2 values"):
        sd.cross_attention(c, FAKE, FAKE, FAKE, FAKE, FAKE, kv_lens=[1], stream=0)
    assert forward(c, scale=float("inf")) == 1 and backward(c, scale=float("inf")) == 1
    assert b"scale" in sd.lib().sdv2_last_error()
    # valid arguments reach the device check (no GPU here): 2 or 3, not 1
    if not torch.cuda.is_available():
        assert forward(c, kv_lens=[0, 7]) in (2, 3) and forward(cross(kv_len=0), k=None, v=None) in (2, 3)
        assert backward(cross(kv_len=0), k=None, v=None, dk=None, dv=None) in (2, 3)


@pytest.mark.parametrize("heads,nq,nk", [(1, 200, 140), (4, 300, 512), (12, 4680, 512), (2, 5000, 60)])
def test_cross_workspace_holds_every_launch_of_a_large_batch(heads, nq, nk):
    """32 streams go into a launch.  The streams left over are cut into more ranges than a whole launch is, and the
    partial sums of theirs need their room as well."""
    make = lambda b: sd.CrossConfig.make(batch=b, heads=heads, head_dim=128, q_len=nq, kv_len=nk)
    stats = lambda b: b * heads * -(-nq // 128) * 1024
    scratch = lambda b: sd.cross_workspace_bytes(make(b), True) - stats(min(b, 32))
    for rest in (1, 2, 5, 31):
        for whole in (32, 64):
            assert scratch(whole + rest) >= max(scratch(32), scratch(rest))


def test_cross_workspace_sizes():
    c = cross(batch=3, heads=5, kv_heads=5, q_len=11)
    assert sd.cross_workspace_bytes(c) >= 256
    assert sd.cross_workspace_bytes(c, True) >= sd.cross_workspace_bytes(c) + 3 * 5 * 11 * 4


@pytest.mark.parametrize("over,want", [
    (dict(rows=0), 1), (dict(rows=1 << 31), 1), (dict(cols=0), 1), (dict(cols=16385), 2), (dict(x_dtype=2), 1),
    (dict(y_dtype=-1), 1), (dict(weight_plus_one=2), 1), (dict(x_row_stride=39), 1), (dict(y_row_stride=39), 1),
    (dict(group_stride=-1), 1), (dict(rows_per_group=-1), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1), (dict(x_row_stride=1 << 40), 2),
])
def test_invalid_norm_configurations(over, want):
    c = norm(**over)
    assert sd.norm_workspace_bytes(c) == 0
    assert status(sd.layer_norm, c, FAKE, FAKE, stream=0) == want
    assert status(sd.layer_norm_backward, c, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, stream=0) == want


def test_invalid_norm_arguments():
    c = norm()
    for bad in (None, FAKE + 4):
        assert status(sd.layer_norm, c, bad, FAKE, stream=0) == 1
        assert status(sd.layer_norm, c, FAKE, bad, stream=0) == 1
        for i in range(5):
            args = [FAKE] * 6
            args[i] = bad
            assert status(sd.layer_norm_backward, c, *args, stream=0) == 1
    for name in ("weight", "bias", "mean", "rstd"):
        assert status(sd.layer_norm, c, FAKE, FAKE, stream=0, **{name: FAKE + 4}) == 1
    for name in ("weight", "dweight", "dbias"):
        assert status(sd.layer_norm_backward, c, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, stream=0, **{name: FAKE + 4}) == 1
    assert status(sd.layer_norm_backward, c, FAKE, FAKE, FAKE, FAKE, FAKE, None, dweight=FAKE, stream=0) == 1
    assert b"ws" in sd.lib().sdv2_last_error()


class FakeTensor:
    """What the binding reads of a CUDA tensor, for its checks."""

    def __init__(self, shape, dtype=torch.bfloat16, strides=None, device=0, offset=0):
        self._t = torch.empty(shape, dtype=dtype)
        if strides is not None:
            need = sum((n - 1) * s for n, s in zip(shape, strides)) + 1
            self._t = torch.empty(need, dtype=dtype).as_strided(shape, strides)
        self.dtype, self.shape, self.is_cuda = dtype, self._t.shape, True
        self.get_device = lambda: device

    def __getattr__(self, name):
        return getattr(self._t, name)


def test_binding_refuses_tensors_that_do_not_fit(monkeypatch):
    monkeypatch.setattr(_block, "_current_device", lambda: 0)
    c = cross()
    q, k, v, out = (FakeTensor(s) for s in ((2, 5, 4, 128), (2, 7, 2, 128), (2, 7, 2, 128), (2, 5, 4, 128)))
    ws = FakeTensor((256,), torch.uint8)

    def call(**o):
        a = dict(q=q, k=k, v=v, out=out, ws=ws)
        a.update(o)
        lse = a.pop("lse", None)
        sd.cross_attention(c, a["q"], a["k"], a["v"], a["out"], a["ws"], lse=lse, stream=0)
    for o, match in ((dict(q=FakeTensor((2, 5, 4, 128), torch.float16)), "q must be torch.bfloat16"),
                     (dict(k=FakeTensor((2, 7, 4, 128))), "configuration says"),
                     (dict(v=FakeTensor((2, 7, 2, 128), strides=(1792, 128, 896, 1))), "has strides"),
                     (dict(k=FakeTensor((7 * 2 * 128,))), "the call touches"),
                     (dict(out=FakeTensor((2, 5, 4, 128), strides=(2560, 128, 640, 1))), "out must be contiguous"),
                     (dict(lse=FakeTensor((2, 4, 5), torch.float64)), "lse must be torch.float32"),
                     (dict(lse=FakeTensor((2, 4, 4), torch.float32)), "the call touches"),
                     (dict(v=FakeTensor((2, 7, 2, 128), device=1)), "v is on device 1, not on device 0"),
                     (dict(q=torch.empty((2, 5, 4, 128), dtype=torch.bfloat16)), "q must be a CUDA tensor")):
        with pytest.raises(ValueError, match=match):
            call(**o)
    monkeypatch.setattr(_block, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="the current device is 1"):
        call()
    monkeypatch.setattr(_block, "_current_device", lambda: 0)
    n = norm(rows_per_group=4)
    x, y = FakeTensor((6, 40)), FakeTensor((6, 40))
    w = FakeTensor((2, 40), torch.float32)
    for a, kw, match in (((FakeTensor((6, 40), torch.float32), y), {}, "x must be torch.bfloat16"),
                         ((x, FakeTensor((6, 40), strides=(48, 1))), {}, "y has strides"),
                         ((x, FakeTensor((6, 40), strides=(1, 6))), {}, "y has strides"),
                         ((FakeTensor((40, 6)), y), {}, "x is"),
                         ((x, y), dict(weight=FakeTensor((1, 40), torch.float32)), "weight: "),
                         ((x, y), dict(weight=w, mean=FakeTensor((5,), torch.float32)), "mean: ")):
        with pytest.raises(ValueError, match=match):
            sd.layer_norm(n, *a, stream=0, **kw)


def reached(call):
    """The call passes the binding's checks and reaches the library's device check (no GPU here) or its own checks."""
    try:
        call()
    except sd.SDV2Error as e:
        assert e.status in (2, 3), e
    return True


def wide(shape, strides, dtype=torch.float32):
    return FakeTensor(shape, dtype, strides=strides)


@pytest.mark.parametrize("name", ["weight", "bias"])
def test_binding_refuses_parameters_with_other_strides(monkeypatch, name):
    """A modulation's scale and shift are slices of one tensor: read as if they were dense they would be other rows."""
    monkeypatch.setattr(_block, "_current_device", lambda: 0)
    monkeypatch.setattr(_block, "_raw_stream", lambda device: 0)
    x, y = FakeTensor((6, 40)), FakeTensor((6, 40))
    ok = FakeTensor((3, 40), torch.float32)
    stats = FakeTensor((6,), torch.float32)
    ws = FakeTensor((1 << 16,), torch.uint8)

    def calls(c, t):
        yield lambda: sd.layer_norm(c, x, y, **{name: t})
        if name == "weight":
            yield lambda: sd.layer_norm_backward(c, y, x, stats, stats, FakeTensor((6, 40)), ws, weight=t)
    dense, spaced = norm(rows_per_group=2), norm(rows_per_group=2, group_stride=240)
    for c, t in ((dense, wide((3, 40), (240, 1))), (dense, wide((3, 40), (1, 3))), (dense, wide((3, 40), (80, 2))),
                 (dense, wide((1, 3, 40), (1, 240, 1))), (dense, wide((4, 40), (240, 1))), (dense, wide((40, 3), (3, 2))),
                 (spaced, wide((3, 40), (80, 1))), (spaced, wide((3, 40, 2), (240, 2, 1))),
                 (norm(), wide((40,), (2,))), (norm(), wide((1, 40), (80, 2)))):
        t._t = torch.empty(4096).as_strided(t._t.shape, t._t.stride())       # long enough for any reading
        for call in calls(c, t):
            with pytest.raises(ValueError, match=name):
                call()
    if not torch.cuda.is_available():
        for c, t in ((dense, ok), (dense, FakeTensor((120,), torch.float32)), (dense, FakeTensor((5, 40), torch.float32)),
                     (spaced, wide((3, 40), (240, 1))), (spaced, wide((1, 3, 40), (720, 240, 1))), (spaced, wide((4, 40), (240, 1))),
                     (spaced, FakeTensor((3, 240), torch.float32)), (spaced, FakeTensor((3, 6, 40), torch.float32)),
                     (norm(), FakeTensor((40,), torch.float32)), (norm(), wide((1, 40), (999, 1)))):
            for call in calls(c, t):
                assert reached(call)


def test_binding_refuses_operands_of_another_rank_with_other_strides(monkeypatch):
    """A packed projection's slice in three dimensions is no dense [B][Nq][H][128]."""
    monkeypatch.setattr(_block, "_current_device", lambda: 0)
    monkeypatch.setattr(_block, "_raw_stream", lambda device: 0)
    q, kv, out = FakeTensor((2, 5, 4, 128)), FakeTensor((2, 7, 2, 128)), FakeTensor((2, 5, 4, 128))
    ws = FakeTensor((256,), torch.uint8)
    packed = FakeTensor((2, 5, 512), strides=(5 * 1536, 1536, 1))
    for bad in (packed, FakeTensor((10, 512), strides=(1, 10)), FakeTensor((5120,), strides=(2,))):
        with pytest.raises(ValueError, match="q "):
            sd.cross_attention(cross(), bad, kv, kv, out, ws)
    y = FakeTensor((6, 40))
    for bad in (FakeTensor((2, 3, 40), strides=(144, 48, 1)), FakeTensor((2, 3, 40), strides=(200, 40, 1))):
        with pytest.raises(ValueError, match="x "):
            sd.layer_norm(norm(), bad, y)
    if not torch.cuda.is_available():
        assert reached(lambda: sd.cross_attention(cross(q_token_stride=1536), packed, kv, kv, out, ws))
        assert reached(lambda: sd.cross_attention(cross(), FakeTensor((10, 512)), kv, kv, out, ws))
        assert reached(lambda: sd.layer_norm(norm(x_row_stride=48), FakeTensor((2, 3, 40), strides=(144, 48, 1)), y))
        assert reached(lambda: sd.layer_norm(norm(x_row_stride=48), FakeTensor((6 * 48,)), y))


def test_norm_step_takes_the_parameters_stride_and_refuses_other_shapes(monkeypatch):
    sess = sd.StreamSession.__new__(sd.StreamSession)        # its configuration only: nothing is allocated or launched
    sess.cfg = sd.StreamConfig.make(batch=2, heads=2, head_dim=128, rope_t=44, rope_h=42, rope_w=42, rope_base=1e4, grid_h=4,
                                    grid_w=6, chunk_frames=3, sink_frames=3, window_frames=4, refresh_chunks=0, qkv_token_stride=0)
    sess.norms = {}
    C, groups = 256, 6
    x = torch.zeros(2, sess.cfg.nq, C)
    y = torch.zeros(2, sess.cfg.nq, C, dtype=torch.bfloat16)
    seen = []
    monkeypatch.setattr(_block, "layer_norm", lambda cfg, x, y, weight=None, bias=None, stream=None: seen.append((cfg, weight, bias)))
    mod = torch.arange(groups * 6 * C, dtype=torch.float32).view(groups, 6, C)
    halves = mod.view(groups, 6 * C)[:, :2 * C].chunk(2, -1)
    frames = mod.view(2, 3, 6, C)
    for w, b, stride in ((mod[:, 1], mod[:, 0], 6 * C), (*halves, 6 * C), (frames[:, :, 2], frames[:, :, 5], 6 * C),
                         (mod[:, 1].contiguous(), None, C), (None, mod[:, 3], 6 * C), (mod[:, 1].contiguous().view(2, 3, C), None, C)):
        assert sess.norm_step(x, y, w, b, modulated=True) is y
        cfg, gw, gb = seen.pop()
        assert (cfg.rows, cfg.cols, cfg.rows_per_group, cfg.weight_plus_one, cfg.group_stride) == (2 * sess.cfg.nq, C, 24, 1, stride)
        for given, got in ((w, gw), (b, gb)):
            assert given is None and got is None or (torch.equal(got, given.reshape(groups, C)) and got.data_ptr() == given.data_ptr())
    sess.norm_step(x, y, mod[0, 0], mod[:1, 1])
    cfg, gw, gb = seen.pop()
    assert (cfg.rows_per_group, cfg.weight_plus_one, cfg.group_stride) == (0, 0, 0) and torch.equal(gw[0], mod[0, 0])
    sess.norm_step(x, y)
    assert seen.pop()[1:] == (None, None)
    whole = mod[:, 0].contiguous()
    for args, modulated in (((whole, whole), False),                    # one row is used: the others would be lost
                            ((whole[:1], whole[:1]), True), ((whole[0], None), True), ((mod[0, 0].expand(groups, C), None), True),
                            ((whole, mod[:, 1]), True), ((mod[:, 1], whole), True), ((None, whole[:, :128]), True),
                            ((whole.t().contiguous().t(), None), True), ((whole.view(C, groups), None), True),
                            ((frames[:, :2, 0].expand(2, 2, C)[:, :, ::2], None), True)):
        with pytest.raises(ValueError):
            sess.norm_step(x, y, *args, modulated=modulated)
    assert not seen


def test_a_preparation_that_fails_is_tried_again(tmp_path):
    """What a kernel needs once per device is kept only where it succeeded."""
    exe = tmp_path / "per_device"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I",
                    os.path.join(ROOT, "streaming_causal_video_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "c_abi", "per_device.cpp"), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0 and run.stdout == "ok\n", run.stdout
    for name in ("cross_attention.cu", "cross_backward.cu"):
        text = open(os.path.join(ROOT, "streaming_causal_video_gb300", "csrc", name)).read()
        assert "call_once" not in text and "PerDevice" in text
