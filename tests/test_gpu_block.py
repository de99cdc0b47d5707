"""GPU tests of cross attention and layer norm, forward and backward, against plain 64-bit
implementations with derived bounds (block_common.py)."""
import ctypes
import math
import subprocess
import sys
import threading
from pathlib import Path

import pytest
import torch

import streaming_causal_video_gb300 as sd
from block_common import (BF, F32, cross_backward_reference, cross_reference, norm_backward_reference, norm_reference,
                          within)

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build_library()


def randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def operand(gen, B, N, H, layout):
    """A [B][N][H][D] view of random rows in one of the supported layouts, with NaN between the rows, and
    the configuration's (token, head, batch) strides."""
    if layout == "dense":
        return randn(gen, B, N, H, D), (0, 0, 0)
    if layout == "head_major":
        base = randn(gen, B, H, N, D)
        return base.transpose(1, 2), (D, N * D, 0)
    if layout == "packed":                      # one of two projections that lie side by side
        base = torch.full((B, N, 2, H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        base[:, :, 1] = randn(gen, B, N, H, D)
        return base[:, :, 1], (2 * H * D, 0, 0)
    base = torch.full((B, N * (H * 136 + 24) + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = base[:, 16:].as_strided((B, N, H, D), (base.shape[1], H * 136 + 24, 136, 1), 16)   # odd strides
    view.copy_(randn(gen, B, N, H, D))
    return view, (H * 136 + 24, 136, base.shape[1])


class Cross:
    def __init__(self, B, H, Hk, nq, nk, lens, layout="dense", scale=0.0, seed=0, backward=True):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens = list(lens)
        kv_layout = layout
        self.q, qs = operand(g, B, nq, H, layout)
        self.k, ks = operand(g, B, nk, Hk, kv_layout)
        self.v, _ = operand(g, B, nk, Hk, kv_layout)
        for b, n in enumerate(self.lens):       # what lies behind a stream's last row has no influence
            if n < nk:
                self.k[b, n:] = float("nan")
                self.v[b, n:] = float("inf")
        self.cfg = sd.CrossConfig.make(batch=B, heads=H, kv_heads=Hk if Hk != H else 0, head_dim=D, q_len=nq, kv_len=nk,
                                       q_token_stride=qs[0], q_head_stride=qs[1], q_batch_stride=qs[2],
                                       kv_token_stride=ks[0], kv_head_stride=ks[1], kv_batch_stride=ks[2])
        self.scale = scale
        self.real_scale = scale if scale > 0 else 1 / math.sqrt(D)
        self.ws = torch.full((sd.cross_workspace_bytes(self.cfg, backward),), 0xA5, dtype=torch.uint8, device="cuda")
        sd.cross_workspace_init(self.cfg, self.ws)
        nan = float("nan")
        self.out = torch.full((B, nq, H, D), nan, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((B, H, nq), nan, dtype=torch.float32, device="cuda")
        self.dout = randn(g, B, nq, H, D)
        self.dq = torch.full_like(self.out, nan)
        self.dk = torch.full((B, nk, Hk, D), nan, dtype=torch.bfloat16, device="cuda")
        self.dv = torch.full_like(self.dk, nan)

    def forward(self, stream=None, lens=True):
        sd.cross_attention(self.cfg, self.q, self.k, self.v, self.out, self.ws, kv_lens=self.lens if lens else None,
                           lse=self.lse, scale=self.scale, stream=stream)

    def backward(self, stream=None, lens=True):
        sd.cross_attention_backward(self.cfg, self.q, self.k, self.v, self.out, self.lse, self.dout, self.dq, self.dk,
                                    self.dv, self.ws, kv_lens=self.lens if lens else None, scale=self.scale,
                                    stream=stream)

    def check_forward(self):
        sd.check_device_error(self.ws)
        out, lse, tol, lse_tol = cross_reference(self.q, self.k, self.v, self.lens, self.real_scale)
        within(self.out, out, tol, "out")
        within(self.lse, lse, lse_tol, "lse")

    def check_backward(self):
        sd.check_device_error(self.ws)
        refs, tols = cross_backward_reference(self.q, self.k, self.v, self.dout, self.lens, self.real_scale)
        for got, ref, tol, what in zip((self.dq, self.dk, self.dv), refs, tols, ("dq", "dk", "dv")):
            within(got, ref, tol, what)


CROSS = [
    # B, H, Hk, Nq, Nk, lens, layout
    (1, 1, 1, 1, 1, [1], "dense"),
    (1, 2, 2, 1, 512, [512], "dense"),
    (2, 3, 3, 4, 77, [77, 0], "packed"),
    (1, 4, 1, 1, 130, [130], "head_major"),
    (3, 4, 2, 17, 257, [257, 1, 2], "odd"),
    (2, 2, 2, 127, 128, [128, 127], "dense"),
    (1, 3, 3, 128, 129, [129], "odd"),
    (2, 2, 1, 129, 300, [300, 255], "packed"),
    (1, 2, 2, 256, 512, [512], "head_major"),
    (4, 3, 1, 300, 512, [512, 77, 0, 301], "dense"),
    (1, 12, 12, 700, 769, [769], "dense"),
    (2, 6, 2, 1000, 5, [5, 4], "packed"),
    (1, 1, 1, 3, 3001, [3001], "dense"),
    (2, 4, 2, 40, 2000, [2000, 1], "head_major"),
    (33, 2, 1, 20, 40, [(7 * b) % 41 for b in range(33)], "dense"),
    (33, 1, 1, 200, 140, [(37 * b) % 141 for b in range(33)], "packed"),
    (2, 2, 2, 50, 64, [0, 0], "dense"),
    (34, 4, 4, 260, 300, [300 - b for b in range(34)], "dense"),       # the last two streams in more ranges than the others
]


@pytest.mark.parametrize("case", CROSS, ids=lambda c: "B%d-H%d-%d-q%d-k%d-%s" % (*c[:5], c[6]))
def test_cross_attention_and_its_gradients(case):
    B, H, Hk, nq, nk, lens, layout = case
    c = Cross(B, H, Hk, nq, nk, lens, layout, seed=nq + nk)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()
    for b, n in enumerate(lens):
        assert not c.dk[b, n:].any() and not c.dv[b, n:].any()
        if n < 2:
            assert not c.dq[b].any() and not c.dk[b].any()


def test_cross_attention_without_keys():
    c = sd.CrossConfig.make(batch=2, heads=2, kv_heads=0, head_dim=D, q_len=9, kv_len=0)
    ws = torch.zeros(sd.cross_workspace_bytes(c, True), dtype=torch.uint8, device="cuda")
    q = torch.randn(2, 9, 2, D, device="cuda").bfloat16()
    out, dq = torch.full_like(q, 3.0), torch.full_like(q, 3.0)
    lse = torch.zeros((2, 2, 9), device="cuda")
    sd.cross_attention(c, q, None, None, out, ws, lse=lse)
    sd.cross_attention_backward(c, q, None, None, out, lse, q, dq, None, None, ws)
    assert not out.any() and not dq.any() and bool((lse == -math.inf).all())


@pytest.mark.parametrize("nq,nk", [(2, 600), (140, 600)])
def test_cross_attention_scale_and_optional_lse(nq, nk):
    c = Cross(1, 2, 2, nq, nk, [nk], scale=0.25, seed=5)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()
    out = c.out.clone()
    c.out.fill_(float("nan"))
    sd.cross_attention(c.cfg, c.q, c.k, c.v, c.out, c.ws, scale=0.25)       # no lse, no lengths
    assert torch.equal(out, c.out)


@pytest.mark.parametrize("nq,nk", [(3, 700), (150, 700)])
def test_cross_attention_follows_growing_scores(nq, nk):
    """Scores that climb by far more than 2^8 along the keys: the running maximum has to follow, and what
    came before has to vanish; and scores that fall, where the first keys stay."""
    for sign in (1.0, -1.0):
        c = Cross(1, 2, 2, nq, nk, [nk], scale=1.0, seed=3)
        c.q.zero_()
        c.k.zero_()
        c.q[..., 0] = 1.0
        c.k[..., 0] = sign * torch.arange(nk, device="cuda").to(torch.bfloat16)[None, :, None]
        c.forward()
        s = c.q.double().transpose(1, 2) @ c.k.double().transpose(1, 2).transpose(2, 3)
        p = torch.softmax(s, -1)
        v = c.v.double().transpose(1, 2)
        # the scores are whole numbers, exact in fp32: only the probabilities' rounding is left
        ref, tol = p @ v, (BF + 2.0 ** -10) * (p @ v.abs())
        within(c.out.transpose(1, 2), ref, tol + BF * ref.abs(), "out")
        within(c.lse, torch.logsumexp(s, -1), 2.0 ** -20 * (1 + s.abs().amax(-1)), "lse")


@pytest.mark.parametrize("nq,nk,lens", [(3, 5, [5]), (150, 130, [130]), (70, 300, [300, 31])])
def test_cross_attention_of_scores_far_below_zero(nq, nk, lens):
    """Every score near -280: exp(-lse) is out of range, so a place behind the last key must not reach a sum."""
    c = Cross(len(lens), 2, 2, nq, nk, lens, seed=4)
    c.q.copy_(5.0 + 0.1 * c.q.float())
    c.k.copy_(-5.0 + 0.1 * c.k.float())
    c.forward()
    c.check_forward()
    assert float(c.lse.max()) < -150
    c.backward()
    c.check_backward()


@pytest.mark.parametrize("heads,kv_heads,nq,nk", [(3, 1, 60, 128), (10, 2, 40, 300), (7, 1, 100, 256), (100, 1, 3, 384)])
def test_gradients_where_heads_do_not_fill_a_tile_and_the_last_rows_of_key_tiles_matter(heads, kv_heads, nq, nk):
    """Heads that share a key head in numbers that do not divide 128: a query tile has rows that no load writes, while
    key tiles have all 128, the last of which hold nearly all the probability here."""
    c = Cross(1, heads, kv_heads, nq, nk, [nk], seed=heads)
    last = torch.arange(nk, device="cuda") % 128 >= 120
    c.q.copy_((1.0 + 0.1 * c.q.float()))
    c.k.copy_(torch.where(last[None, :, None, None], 0.5, -0.5) + 0.1 * c.k.float())
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()
    first = [t.clone() for t in (c.dq, c.dk, c.dv)]
    for _ in range(10):
        c.backward()
        assert all(torch.equal(a, b) for a, b in zip(first, (c.dq, c.dk, c.dv)))


@pytest.mark.parametrize("H,nq,nk,hidden", [(2, 1, 400, 200), (2, 2, 400, 200), (2, 3, 700, 128), (2, 3, 700, 560), (2, 150, 700, 300),
                                            (2, 150, 128, 100), (40, 700, 300, 140), (40, 1000, 700, 520), (3, 300, 100, 60)])
def test_keys_of_the_types_lowest_value_have_no_influence(H, nq, nk, hidden):
    """Keys that a caller has hidden by the type's lowest value: their scores run over to -infinity, a row's whole first
    key tile at once or one half of its keys.  The others' softmax is what is left, and no gradient reaches the hidden."""
    c = Cross(1, H, H, nq, nk, [nk], seed=hidden)
    c.q.copy_(c.q.abs() + 0.1)
    c.k[:, :hidden] = torch.finfo(torch.bfloat16).min
    c.forward()
    rest = [t[:, hidden:] for t in (c.k, c.v)]
    out, lse, tol, lse_tol = cross_reference(c.q, *rest, [nk - hidden], c.real_scale)
    within(c.out, out, tol, "out")
    within(c.lse, lse, lse_tol, "lse")
    c.backward()
    sd.check_device_error(c.ws)
    assert (nk <= 128) == (nk - hidden <= 128)      # delta by the same rule for the rest alone
    refs, tols = cross_backward_reference(c.q, *rest, c.dout, [nk - hidden], c.real_scale)
    within(c.dq, refs[0], tols[0], "dq")
    within(c.dk[:, hidden:], refs[1], tols[1], "dk")
    within(c.dv[:, hidden:], refs[2], tols[2], "dv")
    assert not c.dk[:, :hidden].any() and not c.dv[:, :hidden].any()


@pytest.mark.parametrize("heads,kv_heads,nq,nk,lens", [(4, 4, 2, 3, [3]), (2, 2, 300, 3, [3, 2]), (6, 2, 9, 128, [128, 4, 127]),
                                                       (3, 1, 40, 600, [2, 600, 33])])
def test_gradients_of_few_keys_do_not_carry_the_rounding_of_out(heads, kv_heads, nq, nk, lens):
    """With 128 keys or fewer delta comes from P and dP.  An out that is one bf16 step off in one direction would
    move delta by a step of rowsum(|dO * O|), which the bound for so few keys has no room for."""
    c = Cross(len(lens), heads, kv_heads, nq, nk, lens, seed=6)
    c.forward()
    for b, n in enumerate(lens):
        if n <= 128:
            c.out[b] = (c.out[b].float() * (1 + 2.0 ** -7)).to(torch.bfloat16)
    c.backward()
    c.check_backward()


def test_nan_and_infinity_in_valid_rows_reach_only_what_reads_them():
    c = Cross(2, 2, 2, 140, 300, [300, 200], seed=9)
    c.forward()
    clean = c.out.clone()
    c.q[0, 5, 1] = float("nan")
    c.v[1, 3, 0, 7] = float("nan")
    c.forward()
    expect = clean.clone()
    expect[0, 5, 1] = float("nan")
    expect[1, :, 0, 7] = float("nan")
    assert torch.equal(torch.isnan(c.out), torch.isnan(expect))
    keep = ~torch.isnan(expect)
    assert torch.equal(c.out[keep], expect[keep])


@pytest.mark.parametrize("nq,nk,lens", [(4, 900, [900, 33]), (400, 520, [520, 130]), (129, 1500, [1500, 0])])
def test_cross_attention_is_deterministic(nq, nk, lens):
    c = Cross(2, 4, 2, nq, nk, lens, seed=21)
    c.forward()
    c.backward()
    first = [t.clone() for t in (c.out, c.lse, c.dq, c.dk, c.dv)]
    for _ in range(3):
        for t in (c.out, c.lse, c.dq, c.dk, c.dv):
            t.fill_(float("nan"))
        c.forward()
        c.backward()
        for a, b in zip(first, (c.out, c.lse, c.dq, c.dk, c.dv)):
            assert torch.equal(a, b)


def guarded(shape, dtype, fill):
    pad = 4096 // torch.tensor([], dtype=dtype).element_size()
    n = math.prod(shape)
    base = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")
    return base, base[pad:pad + n].view(shape), pad, fill


def check_bands(*bands):
    for base, _, pad, fill in bands:
        ref = torch.full((pad,), fill, dtype=base.dtype, device="cuda")
        assert torch.equal(base[:pad], ref) and torch.equal(base[-pad:], ref)


@pytest.mark.parametrize("nq,nk,lens", [(3, 70, [70, 11]), (131, 259, [259, 0])])
def test_cross_attention_writes_only_its_outputs(nq, nk, lens):
    c = Cross(2, 3, 3, nq, nk, lens, seed=2)
    bands = {n: guarded(getattr(c, n).shape, getattr(c, n).dtype, 7.0) for n in ("out", "lse", "dq", "dk", "dv")}
    ws = guarded((c.ws.numel(),), torch.uint8, 0x5A)
    for n, b in bands.items():
        setattr(c, n, b[1])
    c.ws = ws[1]
    sd.cross_workspace_init(c.cfg, c.ws)
    inputs = [t.clone() for t in (c.q, c.k, c.v, c.dout)]
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()
    check_bands(ws, *bands.values())
    for a, b in zip(inputs, (c.q, c.k, c.v, c.dout)):
        assert torch.equal(a.view(torch.int16) if a.is_contiguous() else a.contiguous().view(torch.int16),
                           b.contiguous().view(torch.int16))


@pytest.mark.parametrize("nq", [4, 300])
def test_cross_attention_captured_and_replayed_beside_another_graph(nq):
    """Two graphs that share one workspace, replayed in turn on changed inputs, on a stream of their own."""
    a = Cross(2, 2, 1, nq, 300, [300, 40], seed=1)
    b = Cross(2, 2, 1, nq, 300, [17, 300], seed=2)
    b.ws = a.ws
    s = torch.cuda.Stream()
    graphs = []
    for c in (a, b):
        c.forward(s)
        c.backward(s)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            c.forward()
            c.backward()
        graphs.append(graph)
    for turn in range(2):
        for c, graph in zip((a, b), graphs):
            c.q.mul_(0.5)
            c.dout.mul_(2.0)
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                graph.replay()
        s.synchronize()
    for c in (a, b):
        c.check_forward()
        c.check_backward()


def test_two_streams_with_their_own_workspaces():
    cases = [Cross(1, 4, 4, 600, 400, [400], seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cases, streams):
            c.forward(s)
            c.backward(s)
    torch.cuda.synchronize()
    for c in cases:
        c.check_forward()
        c.check_backward()


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right():
    """The copy of one key tile is left out: the waits for it run out, the kernel returns, the error word says
    so, and the workspace serves the next call."""
    c = Cross(2, 3, 3, 300, 500, [500, 400], seed=8)
    few = Cross(1, 2, 2, 20, 900, [900], seed=8)          # key ranges shared by a cluster
    for case in (c, few):
        try:
            sd.set_wait_timeout_ns(50_000_000)
            sd.debug_drop_kv_tile(1)
            case.forward()
            with pytest.raises(sd.SDV2Error) as e:
                sd.check_device_error(case.ws)
            assert e.value.status == 4
        finally:
            sd.debug_drop_kv_tile(-1)
            sd.set_wait_timeout_ns(2_000_000_000)
        case.forward()
        case.check_forward()


@pytest.mark.parametrize("H,Hk,nq,nk,waits", [(2, 2, 2, 1024, False), (4, 2, 1, 900, False), (2, 2, 2, 1025, True), (3, 1, 1, 900, True)])
def test_a_tile_is_left_out_only_where_tiles_are_copied(H, Hk, nq, nk, waits):
    c = Cross(1, H, Hk, nq, nk, [nk], seed=8, backward=False)
    try:
        sd.set_wait_timeout_ns(50_000_000)
        sd.debug_drop_kv_tile(1)
        c.forward()
        if waits:
            with pytest.raises(sd.SDV2Error):
                sd.check_device_error(c.ws)
    finally:
        sd.debug_drop_kv_tile(-1)
        sd.set_wait_timeout_ns(2_000_000_000)
    if waits:
        c.forward()
    c.check_forward()


@pytest.mark.parametrize("shape", [(1, 2, 2, 300, 100), (1, 2, 2, 100, 300), (2, 6, 2, 700, 500), (2, 40, 40, 300, 300)],
                         ids=["dkv", "dq", "both", "many units"])
def test_waits_of_the_backward_pass_that_run_out_are_reported_and_the_next_call_is_right(shape):
    """The copy of one streamed tile is left out: key tile 1 for dQ, query tile 1 for dK and dV."""
    B, H, Hk, nq, nk = shape
    c = Cross(B, H, Hk, nq, nk, [nk] * B, seed=8)
    c.forward()
    try:
        sd.set_wait_timeout_ns(50_000_000)
        sd.debug_drop_kv_tile(1)
        c.backward()
        with pytest.raises(sd.SDV2Error) as e:
            sd.check_device_error(c.ws)
        assert e.value.status == 4
    finally:
        sd.debug_drop_kv_tile(-1)
        sd.set_wait_timeout_ns(2_000_000_000)
    refs, tols = cross_backward_reference(c.q, c.k, c.v, c.dout, c.lens, c.real_scale)
    if nk <= 128:                              # the other launch had no such tile
        within(c.dq, refs[0], tols[0], "dq")
    if nq <= 128:                              # and does not count dQ's wait as its own
        within(c.dk, refs[1], tols[1], "dk")
        within(c.dv, refs[2], tols[2], "dv")
    c.backward()
    c.check_backward()


def test_cross_gradients_against_differences():
    """<gradient, direction> against central differences of the 64-bit forward."""
    c = Cross(1, 2, 1, 150, 200, [200], seed=31)
    c.forward()
    c.backward()
    g = torch.Generator(device="cuda").manual_seed(7)
    _, tols = cross_backward_reference(c.q, c.k, c.v, c.dout, c.lens, c.real_scale)
    ins = [c.q.double(), c.k.double(), c.v.double()]
    h = 1e-4
    for i, (grad, tol) in enumerate(zip((c.dq, c.dk, c.dv), tols)):
        d = torch.randn(ins[i].shape, generator=g, device="cuda", dtype=torch.float64)
        loss = []
        for sign in (1, -1):
            a = list(ins)
            a[i] = a[i] + sign * h * d
            loss.append(float((cross_reference(*a, c.lens, c.real_scale)[0] * c.dout.double()).sum()))
        diff = (loss[0] - loss[1]) / (2 * h)
        # the bound is the sum of the elements' bounds; the difference's own error is of order h^2
        assert abs(float((grad.double() * d).sum()) - diff) <= float((tol * d.abs()).sum()) + 1e-5 * abs(diff) + 1e-5


# ---------------------------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------------------------

TYPES = {"bf16": (sd.BF16, torch.bfloat16, BF), "f32": (sd.F32, torch.float32, F32)}


class Norm:
    def __init__(self, rows, cols, per=0, plus_one=False, xt="bf16", yt="bf16", xpad=0, ypad=0, gpad=0, affine=True,
                 offset=0.0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rows, self.cols, self.per = rows, cols, per or rows
        groups = (rows + self.per - 1) // self.per
        xd, self.xtype, self.x_step = TYPES[xt]
        yd, self.ytype, self.y_step = TYPES[yt]
        self.plus_one, self.eps = plus_one, 1e-6

        def rows_of(dtype, pad, fill):
            base = torch.full((rows, cols + pad), fill, dtype=dtype, device="cuda")
            return base, base[:, :cols]
        self.x_base, self.x = rows_of(self.xtype, xpad, 55.0)
        self.x.copy_(torch.randn((rows, cols), generator=g, device="cuda") * 2 + offset)
        self.y_base, self.y = rows_of(self.ytype, ypad, 55.0)
        self.dy_base, self.dy = rows_of(self.ytype, ypad, 55.0)
        self.dy.copy_(torch.randn((rows, cols), generator=g, device="cuda"))
        self.dx_base, self.dx = rows_of(self.xtype, xpad, 55.0)
        self.weight = self.bias = None
        if affine:
            w = torch.randn((groups, cols + gpad), generator=g, device="cuda")
            b = torch.randn((groups, cols + gpad), generator=g, device="cuda")
            self.weight, self.bias = w[:, :cols], b[:, :cols]
        self.mean, self.rstd = (torch.full((rows,), float("nan"), device="cuda") for _ in range(2))
        self.dweight, self.dbias = (torch.full((groups, cols), float("nan"), device="cuda") for _ in range(2))
        self.cfg = sd.NormConfig.make(rows=rows, cols=cols, x_dtype=xd, y_dtype=yd, weight_plus_one=int(plus_one),
                                      x_row_stride=cols + xpad if xpad else 0, y_row_stride=cols + ypad if ypad else 0,
                                      rows_per_group=per, group_stride=cols + gpad if gpad else 0, eps=self.eps)
        self.ws = torch.full((sd.norm_workspace_bytes(self.cfg),), 0xFF, dtype=torch.uint8, device="cuda")

    def forward(self, stream=None):
        sd.layer_norm(self.cfg, self.x, self.y, weight=self.weight, bias=self.bias, mean=self.mean, rstd=self.rstd,
                      stream=stream)

    def backward(self, stream=None):
        sd.layer_norm_backward(self.cfg, self.dy, self.x, self.mean, self.rstd, self.dx, self.ws, weight=self.weight,
                               dweight=self.dweight, dbias=self.dbias, stream=stream)

    def check_forward(self):
        refs, tols = norm_reference(self.x, self.weight, self.bias, self.per, self.eps, self.plus_one, self.y_step)
        for got, ref, tol, what in zip((self.y, self.mean, self.rstd), refs, tols, ("y", "mean", "rstd")):
            within(got, ref, tol, what)

    def check_backward(self):
        refs, tols = norm_backward_reference(self.x, self.weight, self.dy, self.per, self.eps, self.plus_one, self.x_step)
        for got, ref, tol, what in zip((self.dx, self.dweight, self.dbias), refs, tols, ("dx", "dweight", "dbias")):
            within(got, ref, tol, what)


NORMS = [dict(rows=1, cols=1), dict(rows=1, cols=1536), dict(rows=3, cols=7, xt="f32", yt="f32"),
         dict(rows=72, cols=256), dict(rows=5, cols=257, per=2, plus_one=True), dict(rows=300, cols=512, per=77),
         dict(rows=301, cols=1000, xt="f32"), dict(rows=64, cols=1001, per=10, plus_one=True, yt="f32"),
         dict(rows=700, cols=1536, affine=False), dict(rows=41, cols=2048, yt="f32"), dict(rows=33, cols=2056),
         dict(rows=19, cols=4096, per=5), dict(rows=23, cols=4104, xt="f32"), dict(rows=31, cols=5120, per=8, plus_one=True, xt="f32"),
         dict(rows=9, cols=8192), dict(rows=9, cols=8193, xt="f32", yt="f32"), dict(rows=6, cols=16384, per=4),
         dict(rows=5, cols=16383), dict(rows=40, cols=640, xpad=8, ypad=16, gpad=24, per=13),
         dict(rows=40, cols=640, xpad=3, ypad=0, per=13), dict(rows=40, cols=96, ypad=5, gpad=1, per=40),
         dict(rows=2000, cols=64, per=1), dict(rows=999, cols=128, per=333, offset=30.0, xt="f32"),
         dict(rows=1500, cols=1536, offset=-8.0), dict(rows=700, cols=16384, xt="f32", yt="f32", per=300),
         dict(rows=330, cols=15000, xt="f32", yt="f32"), dict(rows=340, cols=8192, xt="f32", yt="f32", plus_one=True),
         dict(rows=2500, cols=640, per=700, plus_one=True), dict(rows=2501, cols=768, xt="f32"), dict(rows=1801, cols=1024)]


@pytest.mark.parametrize("case", NORMS, ids=lambda c: "-".join("%s%s" % i for i in c.items()))
def test_layer_norm_and_its_gradients(case):
    n = Norm(**case, seed=case["rows"])
    n.forward()
    n.check_forward()
    n.backward()
    n.check_backward()
    for base, pad in ((n.y_base, case.get("ypad", 0)), (n.dx_base, case.get("xpad", 0))):
        assert not pad or bool((base[:, n.cols:] == 55.0).all())


def test_layer_norm_optional_outputs_and_in_place():
    n = Norm(50, 768, seed=1)
    n.forward()
    n.backward()
    y, dx, dw, db = n.y.clone(), n.dx.clone(), n.dweight.clone(), n.dbias.clone()
    for keep in ("weight", "bias"):
        m = Norm(50, 768, seed=1)
        setattr(m, keep, None)
        sd.layer_norm(m.cfg, m.x, m.y, weight=m.weight, bias=m.bias)
        refs, tols = norm_reference(m.x, m.weight, m.bias, m.per, m.eps, False, BF)
        within(m.y, refs[0], tols[0], "y without " + keep)
    for w, b in ((None, None), (n.dweight, None), (None, n.dbias)):
        n.dx.zero_(); n.dweight.zero_(); n.dbias.zero_()
        sd.layer_norm_backward(n.cfg, n.dy, n.x, n.mean, n.rstd, n.dx, n.ws if (w is not None or b is not None) else None,
                               weight=n.weight, dweight=w, dbias=b)
        assert torch.equal(n.dx, dx)
        assert torch.equal(n.dweight, dw) if w is not None else not n.dweight.any()
        assert torch.equal(n.dbias, db) if b is not None else not n.dbias.any()
    x = n.x.clone()
    sd.layer_norm(n.cfg, x, x, weight=n.weight, bias=n.bias)
    assert torch.equal(x, y)
    for target in ("x", "dy"):
        x, dy = n.x.clone(), n.dy.clone()
        dst = x if target == "x" else dy
        sd.layer_norm_backward(n.cfg, dy, x, n.mean, n.rstd, dst, n.ws, weight=n.weight, dweight=n.dweight, dbias=n.dbias)
        assert torch.equal(dst, dx) and torch.equal(n.dweight, dw)


def test_layer_norm_keeps_nan_and_infinity_in_their_rows():
    n = Norm(30, 512, seed=4)
    n.forward()
    clean = n.y.clone()
    n.x[3, 9] = float("nan")
    n.x[7, 100] = float("inf")
    n.forward()
    rows = torch.arange(30, device="cuda")
    hurt = (rows == 3) | (rows == 7)
    assert bool(torch.isnan(n.y[hurt]).any(1).all()) and torch.equal(n.y[~hurt], clean[~hurt])


def test_layer_norm_is_deterministic_and_replays_from_a_graph():
    n = Norm(1200, 1536, per=500, plus_one=True, seed=6)
    n.forward()
    n.backward()
    first = [t.clone() for t in (n.y, n.dx, n.dweight, n.dbias)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        n.forward()
        n.backward()
    for _ in range(3):
        for t in (n.y, n.dx, n.dweight, n.dbias, n.mean):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, (n.y, n.dx, n.dweight, n.dbias)):
            assert torch.equal(a, b)


def test_layer_norm_backward_does_not_report_or_clear_an_error_of_another_part():
    """An error that its owner has not asked for yet; calls whose parameter gradients need no second kernel."""
    n, one = Norm(64, 250, seed=1), Norm(4, 250, seed=2)
    for m in (n, one):
        m.forward()
    dx = torch.empty_like(n.dx)
    stream = torch.cuda.current_stream().cuda_stream
    rt = ctypes.CDLL(next(l.split()[-1] for l in open("/proc/self/maps") if "libcudart" in l))
    torch.cuda.synchronize()
    left = rt.cudaSetDevice(4096)              # no such device: an error code, nothing else
    assert left != 0 and rt.cudaPeekAtLastError() == left
    sd.layer_norm_backward(n.cfg, n.dy, n.x, n.mean, n.rstd, dx, None, weight=n.weight, stream=stream)
    one.backward(stream)
    assert rt.cudaGetLastError() == left and rt.cudaGetLastError() == 0
    one.check_backward()


def test_layer_norm_writes_only_its_outputs():
    n = Norm(37, 200, per=10, seed=8)
    bands = {k: guarded(getattr(n, k).shape, getattr(n, k).dtype, 7.0)
             for k in ("y", "dx", "mean", "rstd", "dweight", "dbias")}
    for k, b in bands.items():
        setattr(n, k, b[1])
    ws = guarded((n.ws.numel(),), torch.uint8, 0x5A)
    n.ws = ws[1]
    n.forward()
    n.backward()
    n.check_forward()
    n.check_backward()
    check_bands(ws, *bands.values())


def test_layer_norm_gradients_against_differences():
    n = Norm(40, 300, per=15, xt="f32", yt="f32", seed=12)
    n.forward()
    n.backward()
    g = torch.Generator(device="cuda").manual_seed(3)
    _, tols = norm_backward_reference(n.x, n.weight, n.dy, n.per, n.eps, False, F32)
    ins = [n.x.double(), n.weight.double(), n.bias.double()]
    h = 1e-4
    for i, (grad, tol) in enumerate(zip((n.dx, n.dweight, n.dbias), tols)):
        d = torch.randn(ins[i].shape, generator=g, device="cuda", dtype=torch.float64)
        loss = []
        for sign in (1, -1):
            a = list(ins)
            a[i] = a[i] + sign * h * d
            loss.append(float((norm_reference(*a, n.per, n.eps, False, F32)[0][0] * n.dy.double()).sum()))
        diff = (loss[0] - loss[1]) / (2 * h)
        assert abs(float((grad.double() * d).sum()) - diff) <= float((tol * d.abs()).sum()) + 1e-5 * abs(diff) + 1e-5


# ---------------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------------

def test_norm_projection_and_cross_attention_as_a_layer_runs_them():
    """x -> affine layer norm -> query projection -> cross attention to two prompts, and back: the gradients
    of the norm's input and parameters and of the prompt's keys and values, against 64-bit autograd of
    the whole run.  The run rounds xhat, q, out, their gradients to bf16 (2^-8 each, six in a row at most
    on any path), so whole tensors agree to 6 * 2^-8 in the 2-norm."""
    B, H, nq, nk, lens = 2, 3, 200, 150, [150, 64]
    C = H * D
    g = torch.Generator(device="cuda").manual_seed(17)
    n = Norm(B * nq, C, seed=5)
    n.weight, n.bias = 1 + 0.1 * torch.randn((1, C), generator=g, device="cuda"), 0.1 * torch.randn((1, C), generator=g, device="cuda")
    wq = (torch.randn((C, C), generator=g, device="cuda") / C ** 0.5).bfloat16()
    c = Cross(B, H, H, nq, nk, lens, seed=6)
    n.forward()
    q = (n.y.float() @ wq.float().t()).bfloat16()
    c.q = q.view(B, nq, H, D)
    c.forward()
    c.backward()
    n.dy = (c.dq.view(B * nq, C).float() @ wq.float()).bfloat16()
    n.backward()

    leaf = lambda t: t.double().detach().requires_grad_()
    x, w, b, k, v = leaf(n.x), leaf(n.weight), leaf(n.bias), leaf(torch.nan_to_num(c.k, 0, 0, 0)), leaf(torch.nan_to_num(c.v, 0, 0, 0))
    var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
    y = (x - mean) / torch.sqrt(var + n.eps) * w + b
    qq = (y @ wq.double().t()).view(B, nq, H, D)
    outs = []
    for i, length in enumerate(lens):
        s = torch.einsum("ihd,jhd->hij", qq[i], k[i, :length]) / math.sqrt(D)
        outs.append(torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v[i, :length]))
    out = torch.stack(outs)
    grads = torch.autograd.grad(out, (x, w, b, k, v), c.dout.double())
    rel = lambda a, r: float((a.double() - r).norm() / r.norm())
    assert rel(c.out, out.detach()) <= 6 * BF
    for what, a, r in zip(("dx", "dweight", "dbias", "dk", "dv"), (n.dx, n.dweight, n.dbias, c.dk, c.dv), grads):
        assert rel(a, r) <= 6 * BF, what


def test_session_runs_a_layer_with_norms_and_a_prompt():
    """A session's layer as a model calls it: modulated norm -> fused projection -> chunk attention -> affine norm ->
    query projection -> cross attention, for two chunks and a prompt that changes between them."""
    B, H, D, F = 2, 2, 128, 3
    C = H * D
    cfg = sd.StreamConfig.make(batch=B, heads=H, head_dim=D, rope_t=44, rope_h=42, rope_w=42, rope_base=1e4, grid_h=4, grid_w=6,
                               chunk_frames=F, sink_frames=3, window_frames=4, refresh_chunks=0, qkv_token_stride=0)
    sess = sd.StreamSession(cfg, 1, [0, 50], "cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    f32 = lambda *s: torch.randn(s, generator=g, device="cuda")
    w_qkv, w_q = (f32(3 * C, C) / C ** 0.5).bfloat16(), (f32(C, C) / C ** 0.5).bfloat16()
    scale, shift = 0.3 * f32(B * F, C), 0.3 * f32(B * F, C)
    weight, bias = 1 + 0.1 * f32(1, C), 0.1 * f32(1, C)
    y, z = (torch.empty((B, cfg.nq, C), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    with pytest.raises(ValueError, match="no prompt"):
        sess.cross_step(0, y.view(B, cfg.nq, H, D))
    one = torch.zeros((1, 5, H, D), dtype=torch.bfloat16, device="cuda")
    for k in (one, one.expand(B, -1, -1, -1), one.expand(B, -1, -1, -1).repeat(1, 1, 1, 2)[..., ::2]):
        with pytest.raises(ValueError):
            sess.set_prompt(0, k, k)
    for chunk in range(2):
        x = f32(B, cfg.nq, C)
        sess.norm_step(x, y, scale, shift, modulated=True)
        refs, tols = norm_reference(x.view(-1, C), scale, shift, cfg.hw, 1e-6, True, BF)
        within(y.view(-1, C), refs[0], tols[0], "modulated norm")
        L = sess.layers[0]
        sd.qkv_rope_append(cfg, sess.start_frames, [chunk] * B, y, w_qkv, sess.q_rot, L.k, L.v, L.meta, sess.ws)
        sd.chunk_attention(cfg, [chunk] * B, sess.q_rot, L.k, L.v, sess.out, sess.ws)
        h = x + sess.out.view(B, cfg.nq, C).float()
        sess.norm_step(h, z, weight, bias)
        refs, tols = norm_reference(h.view(-1, C), weight, bias, B * cfg.nq, 1e-6, False, BF)
        within(z.view(-1, C), refs[0], tols[0], "affine norm")
        q = (z.float() @ w_q.float().t()).bfloat16().view(B, cfg.nq, H, D)
        kv = torch.randn((B, 90 + chunk, 2, H, D), generator=g, device="cuda").bfloat16()     # packed keys and values
        lens = [90, 31 + chunk]
        sess.set_prompt(0, kv[:, :, 0], kv[:, :, 1], lens)
        lse = torch.empty((B, H, cfg.nq), device="cuda")
        out = sess.cross_step(0, q, lse=lse)
        sd.check_device_error(sess.ws)
        sd.check_device_error(sess.cross_ws)
        ref, lse_ref, tol, lse_tol = cross_reference(q, kv[:, :, 0], kv[:, :, 1], lens, 1 / math.sqrt(D))
        within(out, ref, tol, "cross attention")
        within(lse, lse_ref, lse_tol, "lse")


def test_norm_step_reads_scale_and_shift_out_of_one_modulation_tensor():
    B, F, C = 2, 3, 384
    cfg = sd.StreamConfig.make(batch=B, heads=C // D, head_dim=D, rope_t=44, rope_h=42, rope_w=42, rope_base=1e4, grid_h=5, grid_w=7,
                               chunk_frames=F, sink_frames=3, window_frames=4, refresh_chunks=0, qkv_token_stride=0)
    sess = sd.StreamSession(cfg, 1, [0, 0], "cuda")
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn((B, cfg.nq, C), generator=g, device="cuda")
    y = torch.empty((B, cfg.nq, C), dtype=torch.bfloat16, device="cuda")
    mod = 0.3 * torch.randn((B * F, 6, C), generator=g, device="cuda")
    scale, shift = mod.view(B * F, 6 * C)[:, :2 * C].chunk(2, -1)
    for w, b in ((mod[:, 1], mod[:, 4]), (scale, shift), (mod.view(B, F, 6, C)[:, :, 5], mod.view(B, F, 6, C)[:, :, 3])):
        y.fill_(float("nan"))
        sess.norm_step(x, y, w, b, modulated=True)
        refs, tols = norm_reference(x.view(-1, C), w.reshape(B * F, C), b.reshape(B * F, C), cfg.hw, 1e-6, True, BF)
        within(y.view(-1, C), refs[0], tols[0], "modulated norm")


FIRST_CALLS = """
import sys, torch
sys.path.insert(0, sys.argv[1])
import streaming_causal_video_gb300 as sd
g = torch.Generator(device="cuda").manual_seed(1)
bf = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
cfgs = [sd.CrossConfig.make(batch=1, heads=2, head_dim=128, q_len=nq, kv_len=200) for nq in (1, 300)]
ws = torch.zeros(max(sd.cross_workspace_bytes(c, True) for c in cfgs), dtype=torch.uint8, device="cuda")
norm = sd.NormConfig.make(rows=300, cols=256, eps=1e-6)
wsn = torch.zeros(sd.norm_workspace_bytes(norm), dtype=torch.uint8, device="cuda")
k, v = bf(1, 200, 2, 128), bf(1, 200, 2, 128)
def buffers(c):
    n = c.q_len
    return dict(q=bf(1, n, 2, 128), out=bf(1, n, 2, 128), lse=torch.zeros((1, 2, n), device="cuda"), dout=bf(1, n, 2, 128),
                dq=bf(1, n, 2, 128), dk=bf(1, 200, 2, 128), dv=bf(1, 200, 2, 128))
sets = [buffers(c) for c in cfgs]
x, y, dy, dx = (bf(300, 256) for _ in range(4))
mean, rstd = (torch.zeros(300, device="cuda") for _ in range(2))
dw, db = (torch.zeros((1, 256), device="cuda") for _ in range(2))
def work(i):
    c, t = cfgs[i], sets[i]
    sd.cross_attention(c, t["q"], k, v, t["out"], ws, lse=t["lse"])
    sd.cross_attention_backward(c, t["q"], k, v, t["out"], t["lse"], t["dout"], t["dq"], t["dk"], t["dv"], ws)
    sd.layer_norm(norm, x, y, mean=mean, rstd=rstd)
    sd.layer_norm_backward(norm, dy, x, mean, rstd, dx, wsn, dweight=dw, dbias=db)
torch.cuda.synchronize()
graphs, stream = [], torch.cuda.Stream()
for i in range(2):                       # the first calls of the process are captured; the graphs share the workspaces
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        work(i)
    graphs.append(graph)
names = ("out", "lse", "dq", "dk", "dv")
for graph in graphs + graphs:
    graph.replay()
torch.cuda.synchronize()
got = [[t[n].clone() for n in names] for t in sets] + [[y.clone(), dx.clone(), dw.clone(), db.clone()]]
for i in range(2):
    work(i)
torch.cuda.synchronize()
want = [[t[n] for n in names] for t in sets] + [[y, dx, dw, db]]
assert all(torch.equal(a, b) for p, q in zip(got, want) for a, b in zip(p, q))
assert float(got[1][0].float().abs().max()) > 0 and float(got[2][2].abs().max()) > 0
sd.check_device_error(ws)
print("same")
"""


def test_first_calls_of_a_process_inside_a_capture():
    run = subprocess.run([sys.executable, "-c", FIRST_CALLS, str(Path(__file__).resolve().parents[1])], capture_output=True,
                         text=True, timeout=240)
    assert run.returncode == 0 and run.stdout.strip().endswith("same"), run.stderr[-2000:]


def test_calls_from_several_host_threads():
    """Each thread has its stream, workspace and buffers; the results are those of the same calls alone."""
    def one(i):
        return Cross(1 + i % 2, 2, 2, 40 + 90 * i, 130 + i, [130 + i] * (1 + i % 2), seed=20 + i)
    want, cases = [one(i) for i in range(4)], [one(i) for i in range(4)]
    for c in want:
        c.forward()
        c.backward()
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()

    def body(c, s):
        for _ in range(20):
            c.forward(stream=s)
            c.backward(stream=s)
    threads = [threading.Thread(target=body, args=a) for a in zip(cases, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        sd.check_device_error(c.ws)
        assert all(torch.equal(getattr(c, n), getattr(w, n)) for n in ("out", "lse", "dq", "dk", "dv"))


def test_norms_of_several_widths_from_several_host_threads():
    """Widths that run in one kernel with different amounts of shared memory, called at the same time, past the binding
    so that the calls meet inside the library."""
    L = sd.lib()
    wide, narrow = (lambda i: Norm(152, 8192, xt="f32", yt="f32", seed=i)), (lambda i: Norm(1000, 512, xt="f32", yt="f32", seed=i))
    cases = [(wide, narrow)[i % 2](i) for i in range(8)]
    for n in cases:
        n.forward()
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    failed = []

    def body(n, s):
        cfg, ptr = ctypes.byref(n.cfg), [t.data_ptr() for t in (n.x, n.weight, n.bias, n.y, n.mean, n.rstd, n.dy, n.dx, n.dweight, n.dbias, n.ws)]
        x, w, b, y, mean, rstd, dy, dx, dw, db, ws = ptr
        for _ in range(3000):
            for status in (L.sdv2_layer_norm(cfg, x, w, b, y, mean, rstd, s.cuda_stream),
                           L.sdv2_layer_norm_backward(cfg, dy, x, w, mean, rstd, dx, dw, db, ws, s.cuda_stream)):
                if status:
                    failed.append(L.sdv2_last_error())
    threads = [threading.Thread(target=body, args=a) for a in zip(cases, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, (len(failed), failed[0])
    for n in cases:
        n.check_forward()
        n.check_backward()


def test_results_follow_what_other_streams_and_copies_bring():
    """The launches start early and wait for what is before them: a kernel, a copy, a fill, another stream's event;
    eagerly and captured.  The inputs change right in front of every call, and the outputs are read right behind."""
    c, want = Cross(1, 2, 2, 300, 260, [260], seed=31), Cross(1, 2, 2, 300, 260, [260], seed=32)
    n = Norm(rows=300, cols=512, per=100)
    want.forward()
    want.backward()
    n.forward()
    n.backward()
    ref = [t.clone() for t in (n.y, n.dx, n.dweight, n.dbias)]
    x, dy = n.x.clone(), n.dy.clone()
    other = torch.cuda.Stream()
    busy = torch.zeros(64 << 20, device="cuda")
    torch.cuda.synchronize()

    def spoil():
        for t in (c.q, c.k, c.v, c.dout, c.out, c.dq, c.dk, c.dv, n.x, n.dy, n.y, n.dx):
            t.fill_(7.0)

    def run(kind):
        main = torch.cuda.current_stream()
        spoil()
        busy.add_(1.0)                         # long enough for a launch that does not wait to overtake
        if kind == "stream":
            other.wait_stream(main)
            with torch.cuda.stream(other):
                for a, b in ((c.q, want.q), (c.k, want.k), (c.v, want.v), (c.dout, want.dout), (n.x, x), (n.dy, dy)):
                    a.copy_(b * 1.0)
            main.wait_stream(other)
        else:                                  # copies (device to device) or kernels
            for a, b in ((c.q, want.q), (c.k, want.k), (c.v, want.v), (c.dout, want.dout), (n.x, x), (n.dy, dy)):
                a.copy_(b) if kind == "copy" else torch.mul(b, 1.0, out=a)
        c.forward()
        c.backward()
        n.forward()
        n.backward()
        return [t.clone() for t in (c.out, c.lse, c.dq, c.dk, c.dv, n.y, n.dx, n.dweight, n.dbias)]

    expect = [want.out, want.lse, want.dq, want.dk, want.dv] + ref
    for kind in ("copy", "kernel", "stream"):
        for _ in range(3):
            got = run(kind)
            assert all(torch.equal(a, b) for a, b in zip(got, expect)), kind
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            got = run(kind)
        for _ in range(3):
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(got, expect)), "captured " + kind
    sd.check_device_error(c.ws)
