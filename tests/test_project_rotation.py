"""CPU tests of the rotation's refusals: results whose rows would share memory.  No kernel is launched here."""
import pytest
import torch

import streaming_causal_video_gb300 as sd

FAKE = 1 << 20          # an aligned non-null address; every call below is rejected before use


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build_library()


def rotated(fn, **over):
    """Status of a rotation, and what it says."""
    d = dict(batch=2, tokens=5, heads=4, kv_heads=2, head_dim=128, dims=(64, 64))
    d.update(over)
    with pytest.raises(sd.SDV2Error) as e:
        fn(sd.AxesRopeConfig.make(**d), FAKE, FAKE, 2 * FAKE, 3 * FAKE, 4 * FAKE, stream=0)
    return e.value.status, str(e.value)


OVERLAPS = [                                                # of q's four heads, five tokens and two streams of 128 dims
    dict(token_stride=128),                                 # heads and tokens in one place
    dict(token_stride=384),                                 # a token's last head is the next one's first
    dict(head_stride=256),                                  # heads two rows apart, tokens four
    dict(token_stride=512, head_stride=512),
    dict(batch_stride=8), dict(batch_stride=2048), dict(batch_stride=2552),
    dict(token_stride=128, head_stride=640, batch_stride=2048),
]
APART = [
    dict(), dict(token_stride=512), dict(token_stride=520, batch_stride=2600), dict(batch_stride=2560),
    dict(token_stride=128, head_stride=640, batch_stride=2560),                         # heads first
    dict(token_stride=256, head_stride=1280, batch_stride=128),                         # streams side by side
    dict(token_stride=1024, head_stride=256, batch_stride=128),
    dict(token_stride=1536, batch_stride=7680),                                         # q of a packed q|k|v
]


@pytest.mark.parametrize("strides", OVERLAPS, ids=str)
def test_a_result_whose_rows_overlap_is_refused(strides):
    assert rotated(sd.axes_rope, q_out=strides)[0] == 1 and "q_out overlap" in rotated(sd.axes_rope, q_out=strides)[1]
    assert rotated(sd.axes_rope_backward, q_in=strides)[0] == 1 and "q_in overlap" in rotated(sd.axes_rope_backward, q_in=strides)[1]
    same = dict(heads=1, kv_heads=4)
    assert "k_out overlap" in rotated(sd.axes_rope, k_out=strides, **same)[1]
    assert "k_in overlap" in rotated(sd.axes_rope_backward, k_in=strides, **same)[1]
    if torch.cuda.is_available():              # the calls below pass all checks: their addresses are no GPU's memory
        return
    # what is only read may overlap, and an axis of one row has no stride to speak of
    assert rotated(sd.axes_rope, q_in=strides)[0] in (2, 3) and rotated(sd.axes_rope_backward, q_out=strides)[0] in (2, 3)
    assert rotated(sd.axes_rope, q_out=strides, batch=1, tokens=1, heads=1)[0] in (2, 3)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls pass all checks: their addresses are no GPU's memory")
@pytest.mark.parametrize("strides", APART, ids=str)
def test_results_whose_rows_lie_apart_pass(strides):
    for fn in (sd.axes_rope, sd.axes_rope_backward):
        assert rotated(fn, q_in=strides, q_out=strides)[0] in (2, 3)


def test_the_rule_covers_every_overlap():
    """Against all addresses of small layouts: what passes has no two rows in one place."""
    g = torch.Generator().manual_seed(3)
    refused = shared = 0
    for _ in range(400):
        batch, tokens, heads = (int(torch.randint(1, 5, (), generator=g)) for _ in range(3))
        ts, hs, bs = (8 * int(torch.randint(1, 33, (), generator=g)) for _ in range(3))
        spots = {b * bs + n * ts + h * hs for b in range(batch) for n in range(tokens) for h in range(heads)}     # rows of 8
        overlap = len(spots) < batch * tokens * heads
        strides = dict(token_stride=ts, head_stride=hs, batch_stride=bs)
        # (positions that are not on 16 bytes end the call behind the check of the rows)
        with pytest.raises(sd.SDV2Error) as e:
            sd.axes_rope(sd.AxesRopeConfig.make(batch=batch, tokens=tokens, heads=heads, head_dim=8, dims=(8,), q_out=strides), FAKE + 8, FAKE,
                         2 * FAKE, stream=0)
        assert e.value.status == 1
        said = "overlap" in str(e.value)
        assert said or not overlap, strides
        refused, shared = refused + said, shared + overlap
    assert 0 < shared <= refused < 400
