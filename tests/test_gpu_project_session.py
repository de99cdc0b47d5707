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
