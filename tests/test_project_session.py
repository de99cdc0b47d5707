"""CPU tests of what the session and the binding do around 4-bit products and rotations: what they check before anything is
computed, and where a session's memory comes from.  Nothing is computed here: there is no GPU."""
import contextlib

import pytest
import torch

import streaming_causal_video_gb300 as sd
from streaming_causal_video_gb300 import _binding, _block, _project, layer


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build_library()


def session(**over):
    """A session's shape without its buffers."""
    s = object.__new__(sd.StreamSession)
    d = dict(batch=1, heads=2, head_dim=128, rope_t=44, rope_h=42, rope_w=42, rope_base=1e4, grid_h=2, grid_w=3, chunk_frames=2,
             sink_frames=1, window_frames=3, refresh_chunks=5, qkv_token_stride=0)
    d.update(over)
    s.cfg = sd.StreamConfig.make(**d)
    s.ws = torch.zeros(256, dtype=torch.uint8)
    s.start_frames = [7] * s.cfg.batch
    s.products, s.loaded, s.scratch, s.ropes = {}, {}, {}, {}
    s.prompts, s.cross_ws = [None], None
    return s


@pytest.fixture
def steps(monkeypatch):
    """Records quantisations and products instead of calling the library, behind the binding's checks of the bias."""
    done = []

    def operands(plan, a_codes, a_scales, b_codes, b_scales, out, ws, bias, stream):
        if bias is not None and (bias.dtype is not torch.float32 or not bias.is_contiguous()):
            raise ValueError("bias")
        return (a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(), b_scales.data_ptr(), None if bias is None else bias.data_ptr(),
                out.data_ptr(), ws.data_ptr(), 0)
    monkeypatch.setattr(sd.Mx4Matrix, "load", lambda self, x, transposed=False, stream=None: done.append(("load", self.codes.data_ptr())) or self)
    monkeypatch.setattr(_project, "_product", operands, raising=False)
    monkeypatch.setattr(_project, "_multiply", lambda cfg, args: done.append(("multiply", args[0])), raising=False)
    return done


def test_a_refused_product_has_quantised_nothing(steps):
    """What quantize_step returned is the session's memory for all activations of its columns: a call that ends in an error may not
    have overwritten it."""
    s = session()
    w = sd.Mx4Matrix(24, 40, "cpu")
    kept = s.quantize_step(torch.zeros(5, 40))
    assert steps == [("load", kept.codes.data_ptr())]
    del steps[:]
    x, out = torch.zeros(6, 40), torch.zeros(6, 24)
    odd = torch.zeros(6 * 24 + 1)[1:].view(6, 24)
    long = torch.zeros(25)
    for args, kw in (((w, torch.zeros(6, 41), out), {}), ((w, torch.tensor(1.0), out), {}), ((w, x, torch.zeros(6, 25)), {}),
                     ((w, x, torch.zeros(5, 24)), {}), ((w, x, torch.zeros(24, 6).t()), {}), ((w, x, out.half()), {}), ((w, x, odd), {}),
                     ((w, x, out), dict(bias=torch.zeros(25))), ((w, x, out), dict(bias=torch.zeros(24, dtype=torch.bfloat16))),
                     ((w, x, out), dict(bias=torch.zeros(24, 2)[:, 0])), ((w, x, out), dict(bias=long[1:])),
                     ((w, x, out), dict(activation=2)), ((w, x, out), dict(activation=-1)), ((w, torch.zeros(40, 6).t(), out), {})):
        with pytest.raises(ValueError):
            s.project_step(*args, **kw)
        assert not steps, (args[1].shape, kw)
    assert all(cols == 40 for _, cols in s.scratch)
    assert s.project_step(w, x, out, bias=torch.zeros(24), activation=sd.GELU) is out
    assert [name for name, _ in steps] == ["load", "multiply"] and steps[0][1] == steps[1][1]
    del steps[:]
    s.project_step(w, kept, out[:5])
    assert steps == [("multiply", kept.codes.data_ptr())]


def test_memory_that_a_session_makes_is_that_of_the_stream_it_is_first_written_on(steps, monkeypatch):
    """Memory of another stream may be what that stream's kernels still use: the allocator orders its reuse on one stream only."""
    inside, made = [None], []

    @contextlib.contextmanager
    def memory_of(stream, device):
        inside[0] = stream
        yield
        inside[0] = None

    def recorded(make):
        def wrapped(*a, **k):
            made.append(inside[0])
            return make(*a, **k)
        return wrapped
    monkeypatch.setattr(layer, "_memory_of", memory_of, raising=False)
    for call in ("workspace_init", "cache_reset"):
        monkeypatch.setattr(_binding, call, lambda *a: None)
    monkeypatch.setattr(_block, "cross_workspace_init", lambda *a: None)
    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, recorded(getattr(torch, name)))
    x, w, out, kv = torch.ones(200, 40), sd.Mx4Matrix(24, 40, "cpu"), torch.ones(200, 24), torch.ones(1, 9, 2, 128)

    def made_by(f, *a, **k):
        del made[:]
        f(*a, **k)
        return set(made), len(made)
    s = session()
    assert made_by(s.quantize_step, x, stream=11) == ({11}, 2)
    assert made_by(s.quantize_step, x[:150], stream=12) == (set(), 0)
    assert made_by(s.project_step, w, x[:100], out[:100], stream=13) == ({13}, 2)
    assert made_by(s.set_prompt, 0, kv, kv, stream=14) == ({14}, 1)
    assert made_by(sd.StreamSession, s.cfg, 2, [0], "cpu", 15) == ({15}, 9)
    assert made_by(sd.StreamSession, s.cfg, 1, [0], "cpu") == ({None}, 6)


def test_memory_of_no_stream_and_of_no_gpu():
    for stream, device in ((None, "cuda"), (None, "cuda:1"), (7, "cpu"), (None, torch.device("cpu"))):
        with layer._memory_of(stream, device):
            pass


def test_strides_of_a_rotation_change_as_a_whole():
    """What the binding checks tensors by is derived from them: a stride that changed behind its back would let a tensor pass that
    the call runs beyond."""
    cfg = sd.AxesRopeConfig.make(batch=2, tokens=5, heads=4, head_dim=128, dims=(64, 64))
    assert cfg.derived()[1][1] == (5 * 512, 512, 128, 1)
    for name in ("q_in", "q_out", "k_in", "k_out"):
        for field in ("token_stride", "head_stride", "batch_stride"):
            with pytest.raises(AttributeError, match="assign a new RopeStrides"):
                setattr(getattr(cfg, name), field, 4096)
    assert cfg.q_in.token_stride == 0
    alone = sd.RopeStrides(token_stride=1024)
    alone.head_stride = 256
    cfg.q_in = alone
    assert (cfg.q_in.token_stride, cfg.q_in.head_stride) == (1024, 256) and cfg.derived()[1][1] == (5 * 1024, 1024, 256, 1)
    alone.token_stride = 8192                              # the configuration holds a copy
    assert cfg.q_in.token_stride == 1024


@pytest.mark.parametrize("refresh", [0, 5])
def test_there_are_no_places_before_the_first_chunk(refresh):
    """layer_step refuses such a chunk; with a refresh every 5 chunks, chunk -1 would look like chunk 4."""
    s = session(batch=2, refresh_chunks=refresh)
    for chunks in ([0, -1], [-5, 0], (-1, -1)):
        with pytest.raises(ValueError, match="must be >= 0"):
            s.chunk_positions(chunks)
    assert s.chunk_positions((0, 3))[1, 0].tolist() == [13, 0, 0]
