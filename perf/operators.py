"""What the operators around the chunk attention cost: cross attention to the prompt encoder's
states and layer norm, each with its backward pass.

A DiT layer of a streamed video model normalises its tokens (per-frame scale and shift, or a
learned affine), attends to the chunk's cache, and then attends to the states of a prompt
encoder, whose length is another one than the chunk's and differs from stream to stream.  The
cases below are those calls at this repository's workload shapes, from one token to a 14B layer.

With own = False, run() computes each operator with elementary torch operations in 32 bits;
with own = True it makes the framework's calls.
"""
import math

import torch

own = False

D = 128                       # head dim of every workload


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _cross(name, op, batch, heads, kv_heads, q_len, kv_len, lens):
    return {"name": name, "op": op, "batch": batch, "heads": heads, "kv_heads": kv_heads, "q_len": q_len,
            "kv_len": kv_len, "lens": ",".join(str(n) for n in lens)}


def _norm(name, op, rows, cols, rows_per_group, modulated, x_type, y_type):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "rows_per_group": rows_per_group,
            "modulated": modulated, "x_type": x_type, "y_type": y_type}


def listed():
    return [
        # one query (a pooled or register token) against a full prompt of 512 states: latency
        _cross("cross_fwd_token", "cross_fwd", 1, 12, 12, 1, 512, [512]),
        # one 480p chunk of the 1.3B model (3 frames of 30 x 52 tokens) and a full prompt
        _cross("cross_fwd_480p", "cross_fwd", 1, 12, 12, 4680, 512, [512]),
        # four 480p streams whose prompts have their own lengths; one has no prompt at all
        _cross("cross_fwd_batch", "cross_fwd", 4, 12, 12, 4680, 512, [512, 77, 301, 0]),
        # one 720p chunk and a prompt followed by the states of a conditioning image (512 + 257)
        _cross("cross_fwd_720p", "cross_fwd", 1, 12, 12, 10800, 769, [769]),
        # a few query tokens against the long states of a reference clip, shared key heads
        _cross("cross_fwd_long", "cross_fwd", 2, 16, 4, 17, 20001, [20001, 12345]),
        # backward pass of the 480p chunk: a training step's cross attention
        _cross("cross_bwd_480p", "cross_bwd", 1, 12, 12, 4680, 512, [512]),
        # backward pass over one latent frame of four streams with their own prompt lengths
        _cross("cross_bwd_batch", "cross_bwd", 4, 12, 12, 1560, 512, [512, 77, 301, 1]),
        # backward pass of the 14B model's 480p chunk (40 heads)
        _cross("cross_bwd_14b", "cross_bwd", 1, 40, 40, 4680, 512, [512]),
        # the tiny stream's chunk (72 tokens of 2 heads) with a learned affine: latency
        _norm("norm_fwd_tiny", "norm_fwd", 72, 256, 0, False, "bf16", "bf16"),
        # 14B 480p chunk: 32-bit residual in, bf16 out, scale and shift per latent frame
        _norm("norm_fwd_14b", "norm_fwd", 4680, 5120, 1560, True, "f32", "bf16"),
        # backward pass of the 1.3B 480p chunk's affine norm, with the weight's gradient
        _norm("norm_bwd_480p", "norm_bwd", 4680, 1536, 0, False, "bf16", "bf16"),
        # backward pass at an odd width and a ragged last group, 32-bit residual
        _norm("norm_bwd_odd", "norm_bwd", 3001, 1001, 700, True, "f32", "bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _estimate(case):
    """Seconds that the case's bytes and operations stand for, to compare cases by."""
    w = work(case)
    return w["bytes"] / 6e12 + w["flops"] / 1.5e15


def draw(rng):
    """One more case of the ranges above: queries from one to a 720p chunk, states from none to a long
    clip's, 1 to 40 heads with shared key heads, rows and widths of any size."""
    most = max(_estimate(c) for c in listed())
    while True:
        op = rng.choice(["cross_fwd", "cross_fwd", "cross_bwd", "norm_fwd", "norm_bwd"])
        if op.startswith("cross"):
            kv_heads = rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 40])
            heads = kv_heads * rng.choice([1, 1, 1, 2, 3, 4])
            batch = rng.choice([1, 1, 2, 3, 4, 6])
            q_len = _log_int(rng, 1, 10800)
            kv_len = _log_int(rng, 1, 20001 if q_len < 600 else 1500)
            if heads > 40:
                continue
            kind = rng.choice(["full", "ragged", "ragged"])
            lens = [kv_len if kind == "full" else rng.randint(0, kv_len) for _ in range(batch)]
            lens[0] = kv_len
            case = _cross("", op, batch, heads, kv_heads, q_len, kv_len, lens)
        else:
            rows = _log_int(rng, 1, 18720)
            cols = rng.choice([rng.randint(3, 8192), 8 * _log_int(rng, 8, 1024), 128 * rng.randint(1, 40)])
            group = rng.choice([0, rng.randint(1, rows)]) if rows < 64 else rng.choice([0, rng.randint(rows // 12 + 1, rows)])
            case = _norm("", op, rows, cols, group, rng.random() < 0.5, rng.choice(["bf16", "f32"]),
                         rng.choice(["bf16", "f32"]))
        if _estimate(case) <= most:
            del case["name"]
            return case


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


def _groups(case):
    """(rows in a group, groups)"""
    per = case["rows_per_group"] or case["rows"]
    return per, (case["rows"] + per - 1) // per


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if case["op"].startswith("cross"):
        B, H, Hk, nq, nk = case["batch"], case["heads"], case["kv_heads"], case["q_len"], case["kv_len"]
        # queries and keys come from a normalised projection: rows of about unit mean square,
        # with a spread between heads that makes some of them attend sharply
        sharp = 0.5 + 1.5 * torch.rand((1, 1, H, 1), generator=g, device="cuda")
        d = {"q": (randn(B, nq, H, D) * sharp).to(torch.bfloat16), "k": randn(B, nk, Hk, D).to(torch.bfloat16),
             "v": randn(B, nk, Hk, D).to(torch.bfloat16)}
        if case["op"] == "cross_bwd":
            # the gradient of a mean-like loss: small
            d["dout"] = (randn(B, nq, H, D) * 0.02).to(torch.bfloat16)
        return d
    rows, cols = case["rows"], case["cols"]
    _, groups = _groups(case)
    # a residual stream: rows of their own size and offset, and a few loud columns
    x = randn(rows, cols) * (0.5 + 2.0 * torch.rand((rows, 1), generator=g, device="cuda")) + 0.5 * randn(rows, 1)
    x *= 1.0 + 4.0 * (torch.rand((1, cols), generator=g, device="cuda") > 0.98).float()
    d = {"x": x.to(_TYPES[case["x_type"]])}
    if case["modulated"]:          # y = xhat * (1 + weight) + bias, a row of each for every group
        d["weight"], d["bias"] = 0.3 * randn(groups, cols), 0.3 * randn(groups, cols)
    else:                          # y = xhat * weight + bias
        d["weight"], d["bias"] = 1.0 + 0.1 * randn(groups, cols), 0.1 * randn(groups, cols)
    if case["op"] == "norm_bwd":
        d["dy"] = (0.02 * randn(rows, cols)).to(_TYPES[case["y_type"]])
    return d


EPS = 1e-6


def prepare(case, seed):
    """Inputs of the call; for a backward pass what its forward pass left behind (output and
    log-sum-exp, mean and inverse deviation); for the framework its configuration, workspace and
    output buffers."""
    st = dict(_inputs(case, seed), case=case)
    op = case["op"]
    if op == "cross_bwd":
        out, st["lse"] = _plain_cross(case, st)
        st["out"] = out
    if op == "norm_bwd":
        xf = st["x"].float()
        mean = xf.mean(1)
        st["mean"] = mean
        st["rstd"] = 1.0 / torch.sqrt(((xf - mean[:, None]) ** 2).mean(1) + EPS)
    if own:
        _prepare_own(case, st)
    return st


def _prepare_own(case, st):
    import streaming_causal_video_gb300 as sd
    op = case["op"]
    if op.startswith("cross"):
        B, H, Hk, nq, nk = case["batch"], case["heads"], case["kv_heads"], case["q_len"], case["kv_len"]
        cfg = sd.CrossConfig.make(batch=B, heads=H, kv_heads=Hk, head_dim=D, q_len=nq, kv_len=nk)
        backward = op == "cross_bwd"
        st["ws"] = torch.empty(sd.cross_workspace_bytes(cfg, backward), dtype=torch.uint8, device="cuda")
        sd.cross_workspace_init(cfg, st["ws"])
        st["lens"] = _lens(case)
        if backward:
            st["dq"], st["dk"], st["dv"] = (torch.empty_like(st[n]) for n in ("q", "k", "v"))
        else:
            st["out"] = torch.empty_like(st["q"])
            st["lse"] = torch.empty((B, H, nq), dtype=torch.float32, device="cuda")
    else:
        cfg = sd.NormConfig.make(rows=case["rows"], cols=case["cols"], rows_per_group=case["rows_per_group"],
                                 weight_plus_one=int(case["modulated"]), eps=EPS,
                                 x_dtype={"bf16": sd.BF16, "f32": sd.F32}[case["x_type"]],
                                 y_dtype={"bf16": sd.BF16, "f32": sd.F32}[case["y_type"]])
        if op == "norm_bwd":
            st["ws"] = torch.empty(sd.norm_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
            st["dx"] = torch.empty_like(st["x"])
            st["dweight"], st["dbias"] = torch.empty_like(st["weight"]), torch.empty_like(st["bias"])
        else:
            st["y"] = torch.empty((case["rows"], case["cols"]), dtype=_TYPES[case["y_type"]], device="cuda")
            st["mean"], st["rstd"] = (torch.empty(case["rows"], dtype=torch.float32, device="cuda") for _ in range(2))
    st["cfg"] = cfg


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(op, state)
    if op == "cross_fwd":
        out, lse = _plain_cross(state["case"], state)
        return {"out": out, "lse": lse}
    if op == "cross_bwd":
        return _plain_cross_backward(state["case"], state)
    if op == "norm_fwd":
        return _plain_norm(state["case"], state)
    return _plain_norm_backward(state["case"], state)


def _run_own(op, st):
    import streaming_causal_video_gb300 as sd
    if op == "cross_fwd":
        sd.cross_attention(st["cfg"], st["q"], st["k"], st["v"], st["out"], st["ws"], kv_lens=st["lens"], lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    if op == "cross_bwd":
        sd.cross_attention_backward(st["cfg"], st["q"], st["k"], st["v"], st["out"], st["lse"], st["dout"], st["dq"],
                                    st["dk"], st["dv"], st["ws"], kv_lens=st["lens"])
        return {"dq": st["dq"], "dk": st["dk"], "dv": st["dv"]}
    if op == "norm_fwd":
        sd.layer_norm(st["cfg"], st["x"], st["y"], weight=st["weight"], bias=st["bias"], mean=st["mean"], rstd=st["rstd"])
        return {"y": st["y"], "mean": st["mean"], "rstd": st["rstd"]}
    sd.layer_norm_backward(st["cfg"], st["dy"], st["x"], st["mean"], st["rstd"], st["dx"], st["ws"], weight=st["weight"],
                           dweight=st["dweight"], dbias=st["dbias"])
    return {"dx": st["dx"], "dweight": st["dweight"], "dbias": st["dbias"]}


def _heads_first(t, n, heads):
    """[tokens][heads of keys][D] -> 32-bit [heads][n][D], key heads repeated for the queries that share them."""
    t = t[:n].float().transpose(0, 1)
    return t.repeat_interleave(heads // t.shape[0], 0)


def _plain_cross(case, st):
    B, H, nq = case["batch"], case["heads"], case["q_len"]
    out = torch.zeros_like(st["q"])
    lse = torch.full((B, H, nq), -math.inf, dtype=torch.float32, device="cuda")
    for b, n in enumerate(_lens(case)):
        if n == 0:
            continue
        q = st["q"][b].float().transpose(0, 1)
        k, v = _heads_first(st["k"][b], n, H), _heads_first(st["v"][b], n, H)
        s = (q @ k.transpose(1, 2)) * (1.0 / math.sqrt(D))
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        total = p.sum(-1, keepdim=True)
        out[b] = ((p @ v) / total).transpose(0, 1).to(torch.bfloat16)
        lse[b] = (m + torch.log(total))[..., 0]
    return out, lse


def _plain_cross_backward(case, st):
    H, Hk = case["heads"], case["kv_heads"]
    scale = 1.0 / math.sqrt(D)
    dq, dk, dv = torch.zeros_like(st["q"]), torch.zeros_like(st["k"]), torch.zeros_like(st["v"])
    for b, n in enumerate(_lens(case)):
        if n == 0:
            continue
        q, dout = st["q"][b].float().transpose(0, 1), st["dout"][b].float().transpose(0, 1)
        k, v = _heads_first(st["k"][b], n, H), _heads_first(st["v"][b], n, H)
        s = (q @ k.transpose(1, 2)) * scale
        p = torch.exp(s - s.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        dp = dout @ v.transpose(1, 2)
        ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
        dq[b] = (ds @ k).transpose(0, 1).to(torch.bfloat16)
        dk[b, :n] = (ds.transpose(1, 2) @ q).view(Hk, H // Hk, n, D).sum(1).transpose(0, 1).to(torch.bfloat16)
        dv[b, :n] = (p.transpose(1, 2) @ dout).view(Hk, H // Hk, n, D).sum(1).transpose(0, 1).to(torch.bfloat16)
    return {"dq": dq, "dk": dk, "dv": dv}


def _by_row(case, t):
    """A group's row of weights for every row of x."""
    per, groups = _groups(case)
    if groups == 1:
        return t
    return t.repeat_interleave(per, 0)[:case["rows"]]


def _plain_norm(case, st):
    x = st["x"].float()
    mean = x.mean(1)
    centred = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((centred * centred).mean(1) + EPS)
    gain = st["weight"] + 1.0 if case["modulated"] else st["weight"]
    y = centred * rstd[:, None] * _by_row(case, gain) + _by_row(case, st["bias"])
    return {"y": y.to(_TYPES[case["y_type"]]), "mean": mean, "rstd": rstd}


def _by_group(case, t):
    """Sums over the rows of each group."""
    per, groups = _groups(case)
    if groups == 1:
        return t.sum(0, keepdim=True)
    pad = groups * per - case["rows"]
    if pad:
        t = torch.cat([t, t.new_zeros((pad, t.shape[1]))])
    return t.view(groups, per, -1).sum(1)


def _plain_norm_backward(case, st):
    dy = st["dy"].float()
    xhat = (st["x"].float() - st["mean"][:, None]) * st["rstd"][:, None]
    gain = st["weight"] + 1.0 if case["modulated"] else st["weight"]
    g = dy * _by_row(case, gain)
    dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * st["rstd"][:, None]
    return {"dx": dx.to(st["x"].dtype), "dweight": _by_group(case, dy * xhat), "dbias": _by_group(case, dy)}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits, and what a pass has to move and compute
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    d = _inputs(case, seed)
    if case["op"].startswith("cross"):
        return _exact_cross(case, d)
    x = d["x"].double().requires_grad_()
    weight, bias = d["weight"].double().requires_grad_(), d["bias"].double().requires_grad_()
    per, _ = _groups(case)
    group = torch.arange(case["rows"], device="cuda") // per
    var, mean = torch.var_mean(x, dim=1, unbiased=False)
    rstd = (var + EPS) ** -0.5
    y = (x - mean[:, None]) * rstd[:, None] * (weight + float(case["modulated"]))[group] + bias[group]
    if case["op"] == "norm_fwd":
        return {"y": y.detach(), "mean": mean.detach(), "rstd": rstd.detach()}
    dx, dweight, dbias = torch.autograd.grad(y, (x, weight, bias), d["dy"].double())
    return {"dx": dx, "dweight": dweight, "dbias": dbias}


def _exact_cross(case, d):
    H, Hk = case["heads"], case["kv_heads"]
    backward = case["op"] == "cross_bwd"
    q, k, v = (d[n].double() for n in ("q", "k", "v"))
    if backward:
        res = {"dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v)}
    else:
        res = {"out": torch.zeros_like(q),
               "lse": torch.full((case["batch"], H, case["q_len"]), -math.inf, dtype=torch.float64, device="cuda")}
    for b, n in enumerate(_lens(case)):
        for h in range(H if n else 0):
            j = h // (H // Hk)
            qh, kh, vh = (t.clone().requires_grad_(backward) for t in (q[b, :, h], k[b, :n, j], v[b, :n, j]))
            logits = torch.einsum("id,jd->ij", qh, kh) / D ** 0.5
            out = torch.softmax(logits, 1) @ vh
            if backward:
                gq, gk, gv = torch.autograd.grad(out, (qh, kh, vh), d["dout"][b, :, h].double())
                res["dq"][b, :, h] = gq
                res["dk"][b, :n, j] += gk
                res["dv"][b, :n, j] += gv
            else:
                res["out"][b, :, h] = out
                res["lse"][b, h] = torch.logsumexp(logits, 1)
    return res


def work(case):
    if case["op"].startswith("cross"):
        B, H, Hk, nq, nk = case["batch"], case["heads"], case["kv_heads"], case["q_len"], case["kv_len"]
        pairs = H * nq * sum(_lens(case))
        rows_q = B * nq * H * D * 2
        rows_kv = sum(_lens(case)) * Hk * D * 2
        stats = B * H * nq * 4
        if case["op"] == "cross_fwd":        # q, k, v in; out and log-sum-exp out; two products
            return {"bytes": 2 * rows_q + 2 * rows_kv + stats, "flops": 4 * D * pairs}
        # q, out, dout, log-sum-exp, k, v in; dq, dk, dv (whole) out; five products
        return {"bytes": 4 * rows_q + 2 * rows_kv + 2 * B * nk * Hk * D * 2 + stats, "flops": 10 * D * pairs}
    size = {"bf16": 2, "f32": 4}
    n, x, y = case["rows"] * case["cols"], size[case["x_type"]], size[case["y_type"]]
    params = 2 * _groups(case)[1] * case["cols"] * 4
    if case["op"] == "norm_fwd":             # x, weight, bias in; y, mean, rstd out
        return {"bytes": n * (x + y) + params + 8 * case["rows"], "flops": 8 * n}
    # dy, x, mean, rstd, weight in; dx, dweight, dbias out
    return {"bytes": n * (2 * x + y) + params + params // 2 + 8 * case["rows"], "flops": 14 * n}
