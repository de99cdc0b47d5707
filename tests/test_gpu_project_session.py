"""GPU tests of a session's 4-bit products: refused calls, and streams."""
import pytest
import torch

import streaming_causal_video_gb300 as sd
from test_gpu_project import gpu_ready  # noqa: F401

pytestmark = pytest.mark.gpu


def session():
    cfg = sd.StreamConfig.make(batch=1, heads=2, head_dim=128, rope_t=44, rope_h=42, rope_w=42, rope_base=1e4, grid_h=6, grid_w=8,
                               chunk_frames=2, sink_frames=2, window_frames=4, refresh_chunks=0, qkv_token_stride=0)
    return sd.StreamSession(cfg, 1, [0], "cuda")


@pytest.mark.parametrize("rows", [3, 100])
def test_a_refused_product_leaves_quantised_activations(rows):
    s = session()
    g = torch.Generator(device="cuda").manual_seed(rows)
    w = sd.Mx4Matrix.of(torch.randn(200, 520, generator=g, device="cuda"))
    x, other = (torch.randn(rows, 520, generator=g, device="cuda") for _ in range(2))
    out, bias = torch.empty(rows, 200, device="cuda"), torch.zeros(201, device="cuda")
    kept = s.quantize_step(x)
    want = s.project_step(w, kept, torch.empty_like(out))
    held = kept.codes.clone(), kept.scales.clone()
    for kw in (dict(out=out[:, :199].contiguous()), dict(out=out.half()), dict(out=out.cpu()), dict(out=out, bias=bias),
               dict(out=out, bias=bias[:200].bfloat16()), dict(out=out, bias=bias[1:]), dict(out=out, bias=bias[:200].cpu()),
               dict(out=out, activation=2), dict(out=torch.empty(rows * 200 + 1, device="cuda")[1:].view(rows, 200))):
        with pytest.raises(ValueError):
            s.project_step(w, other, **kw)
    for bad in (other.cpu(), other.half(), other.t(), other[:, :519].contiguous()):
        with pytest.raises(ValueError):
            s.project_step(w, bad, out)
    assert torch.equal(kept.codes, held[0]) and torch.equal(kept.scales, held[1])
    assert torch.equal(s.project_step(w, kept, out), want)
    assert not torch.equal(s.project_step(w, other, out), want)
    sd.check_device_error(s.ws)


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("rows", [3, 700])
def test_first_products_on_another_stream_leave_memory_in_use_alone(rows, raw):
    """The current stream is busy, and what it will write last lies in memory that is free again on the host's side."""
    s, other = session(), torch.cuda.Stream()
    g = torch.Generator(device="cuda").manual_seed(rows)
    w = sd.Mx4Matrix.of(torch.randn(200, 1500, generator=g, device="cuda"))
    x = torch.randn(rows, 1500, generator=g, device="cuda")
    out, again = torch.empty(rows, 200, device="cuda"), torch.empty(rows, 200, device="cuda")
    want = session().project_step(w, x, torch.empty_like(out))
    k, v = (torch.randn(1, 64, 2, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(1, s.cfg.nq, 2, 128, generator=g, device="cuda").bfloat16()
    torch.cuda.synchronize()
    room = max(128, 1 << (rows - 1).bit_length())
    sizes = {"codes": room * 12 * 64, "scales": -(-room // 128) * 12 * 512, "workspace": 256}
    torch.cuda._sleep(50_000_000)                          # some 25 ms
    held = {n: [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(3)] for n, size in sizes.items()}
    spans = [(t.data_ptr(), t.data_ptr() + t.nbytes) for ts in held.values() for t in ts]
    for ts in held.values():
        for t in ts:
            t.fill_(0x5A)
    del held, t, ts
    stream = other.cuda_stream if raw else other
    s.project_step(w, x, out, stream=stream)
    s.set_prompt(0, k, v, stream=stream)
    made = s.quantize_step(x, stream=stream)
    rows_out = s.cross_step(0, q, torch.empty_like(q), stream=stream)
    s.project_step(w, made, again, stream=stream)
    for t in (made.codes, made.scales, s.cross_ws):
        assert all(t.data_ptr() + t.nbytes <= a or t.data_ptr() >= b for a, b in spans)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(again, want) and bool(rows_out.isfinite().all())
    sd.check_device_error(s.ws)
    sd.check_device_error(s.cross_ws)


def test_first_products_captured_on_a_stream_that_is_named():
    s, stream = session(), torch.cuda.Stream()
    g = torch.Generator(device="cuda").manual_seed(1)
    w = sd.Mx4Matrix.of(torch.randn(200, 520, generator=g, device="cuda"))
    x, out = torch.randn(90, 520, generator=g, device="cuda"), torch.zeros(90, 200, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.project_step(w, x, out, stream=stream)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, s.project_step(w, x, torch.empty_like(out))) and bool(out.any())


def test_a_session_made_on_another_stream():
    stream = torch.cuda.Stream()
    cfg = session().cfg
    torch.cuda.synchronize()
    for st in (stream, stream.cuda_stream, 0):
        s = sd.StreamSession(cfg, 1, [0], "cuda", stream=st)
        g = torch.Generator(device="cuda").manual_seed(2)
        q, k, v = (torch.randn(1, cfg.nq, 2, 128, generator=g, device="cuda").bfloat16() for _ in range(3))
        torch.cuda.synchronize()
        s.layer_step(0, [0], q, k, v, stream=st)
        torch.cuda.synchronize()
        got = s.out.clone()
        want = session().layer_step(0, [0], q, k, v)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
