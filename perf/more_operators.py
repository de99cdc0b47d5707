"""What a layer's products in microscaled 4-bit numbers and its rotary positions cost.

Next to the chunk attention, the cross attention and the norms, a DiT layer of a streamed video
model multiplies its tokens by weights (the modulation from the time embedding, the prompt's
projection, the feed-forward pair) and turns queries and keys by their place in time, height and
width.  A matrix is held in 4 bits as e2m1 numbers with one power of two for every 32 of a row;
products run between two such matrices.  The cases are those calls at this repository's workload
shapes, from one token to a 14B layer, forward and backward.

With own = False, run() computes each operator with elementary torch operations in 32 bits;
with own = True it makes the framework's calls.
"""
import math

import torch

own = False

BLOCK = 32                    # numbers that share a scale
BASE = 10000.0                # of the rotary frequencies


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _quantize(name, rows, cols, x_type, transposed):
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "x_type": x_type, "transposed": transposed}


def _product(name, op, rows, cols, depth, x_type, out_type, bias, gelu):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "depth": depth, "x_type": x_type, "out_type": out_type,
            "bias": bias, "gelu": gelu}


def _rope(name, op, batch, tokens, heads, kv_heads, head_dim, dims, halves, head_major, far, x_type):
    return {"name": name, "op": op, "batch": batch, "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "dims": ",".join(str(d) for d in dims), "halves": halves, "head_major": head_major,
            "far": far, "x_type": x_type}


def listed():
    return [
        # the 32-bit activations of a 14B 480p chunk (3 frames of 30 x 52 tokens) to 4 bits and back to bf16
        _quantize("quantize_14b", 4680, 5120, "f32", False),
        # a gradient whose rows are contracted in the weight's gradient: blocks run down its columns, odd sizes
        _quantize("quantize_transposed_odd", 3001, 1001, "bf16", True),
        # six modulation vectors for each of a chunk's 3 frames from the time embedding: latency
        _product("linear_frames", "linear", 3, 9216, 1536, "f32", "f32", True, False),
        # projection of a prompt's 512 states to the 1.3B width
        _product("linear_prompt", "linear", 512, 1536, 4096, "bf16", "bf16", True, False),
        # first product of the 1.3B 480p feed-forward, with its activation
        _product("linear_480p", "linear", 4680, 6144, 1536, "bf16", "bf16", True, True),
        # second product of the 14B 480p feed-forward; its input is already quantised
        _product("product_14b", "product", 4680, 5120, 20480, "bf16", "bf16", True, False),
        # odd sizes everywhere, 32-bit result, no bias
        _product("product_odd", "product", 1001, 777, 1050, "f32", "f32", False, False),
        # backward pass of the 1.3B 480p query projection: gradients of its input and of its weight
        _product("linear_bwd_480p", "linear_bwd", 4680, 1536, 1536, "bf16", "bf16", False, False),
        # one token of 40 heads far into a stream: latency
        _rope("rope_fwd_token", "rope_fwd", 1, 1, 40, 40, 128, (44, 42, 42), False, False, True, "bf16"),
        # queries and keys of one 480p chunk of the 1.3B model
        _rope("rope_fwd_480p", "rope_fwd", 1, 4680, 12, 12, 128, (44, 42, 42), False, False, False, "bf16"),
        # backward pass of the 14B chunk, gradients head by head as the attention leaves them
        _rope("rope_bwd_14b", "rope_bwd", 1, 4680, 40, 40, 128, (44, 42, 42), False, True, True, "bf16"),
        # backward pass over the patches of two images: two axes, pairs half a segment apart, dims that do
        # not turn, shared key heads, 32 bits
        _rope("rope_bwd_images", "rope_bwd", 2, 1023, 9, 3, 80, (36, 36), True, False, False, "f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _estimate(case):
    """Seconds that the case's bytes and operations stand for, to compare cases by."""
    w = work(case)
    return w["bytes"] / 6e12 + w["flops"] / 5e15


def draw(rng):
    """One more case of the ranges above: rows from one to a 720p chunk, widths of any size up to a
    14B feed-forward's, heads of 16 to 256 dims with one to four axes."""
    most = max(_estimate(c) for c in listed())
    while True:
        op = rng.choice(["quantize", "quantize", "linear", "linear", "product", "linear_bwd", "rope_fwd", "rope_bwd"])
        x_type = rng.choice(["bf16", "f32"])
        if op == "quantize":
            case = _quantize("", _log_int(rng, 1, 10800), _log_int(rng, 1, 20480), x_type, rng.random() < 0.4)
        elif not op.startswith("rope"):
            def width():
                return rng.choice([_log_int(rng, 1, 20480), 128 * _log_int(rng, 1, 160)])
            rows = _log_int(rng, 1, 10800)
            if op == "linear_bwd":
                case = _product("", op, rows, width(), width(), x_type, rng.choice(["bf16", "f32"]), False, False)
            else:
                case = _product("", op, rows, width(), width(), x_type, rng.choice(["bf16", "f32"]), rng.random() < 0.7,
                                rng.random() < 0.3)
        else:
            head_dim = rng.choice([128, 128, 8 * rng.randint(2, 32)])
            axes = rng.randint(1, 4)
            left, dims = head_dim, []
            for a in range(axes):
                dims.append(2 * rng.randint(1, max(1, left // 2 // (axes - a))))
                left -= dims[-1]
            kv = rng.choice([1, 2, 3, 4, 8, 12, 16, 40])
            heads = kv * rng.choice([1, 1, 2, 4])
            if heads > 40:
                continue
            case = _rope("", op, rng.choice([1, 1, 2, 4]), _log_int(rng, 1, 10800), heads, kv, head_dim, dims,
                         rng.random() < 0.4, rng.random() < 0.4, rng.random() < 0.4, x_type)
        if _estimate(case) <= most:
            del case["name"]
            return case


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _dims(case):
    return [int(d) for d in case["dims"].split(",")]


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def activations(rows, cols):
        # what a norm leaves: rows of about unit mean square and a few loud columns
        x = randn(rows, cols)
        x *= 1.0 + 4.0 * (torch.rand((1, cols), generator=g, device="cuda") > 0.98).float()
        return x

    if case["op"] == "quantize":
        rows, cols = case["rows"], case["cols"]
        x = activations(cols, rows) if case["transposed"] else activations(rows, cols)
        return {"x": x.to(_TYPES[case["x_type"]])}
    if not case["op"].startswith("rope"):
        M, N, K = case["rows"], case["cols"], case["depth"]
        d = {"x": activations(M, K).to(_TYPES[case["x_type"]]), "w": (randn(N, K) / math.sqrt(K)).to(torch.bfloat16)}
        if case["bias"]:
            d["bias"] = 0.1 * randn(N)
        if case["op"] == "linear_bwd":
            # the gradient of a mean-like loss: small
            d["dy"] = (0.02 * randn(M, N)).to(_TYPES[case["x_type"]])
        return d
    B, T, dims = case["batch"], case["tokens"], _dims(case)
    kind = _TYPES[case["x_type"]]

    def rows(heads):
        if case["head_major"]:
            return randn(B, heads, T, case["head_dim"]).to(kind).transpose(1, 2)
        return randn(B, T, heads, case["head_dim"]).to(kind)

    # frames first, then the places of a grid whose last axes are about square
    grid = max(1, math.isqrt(max(1, T // 3))) if len(dims) > 1 else T
    n = torch.arange(T, device="cuda")
    pos = torch.stack([n // (grid ** (len(dims) - 1 - a)) % (grid if a else T) for a in range(len(dims))], -1)
    pos = pos[None].expand(B, T, len(dims)).clone()
    start = torch.randint(0, 1000000 if case["far"] else 64, (B, 1), generator=g, device="cuda")
    pos[:, :, 0] += start
    return {"positions": pos.to(torch.int32).contiguous(), "q": rows(case["heads"]), "k": rows(case["kv_heads"])}


def prepare(case, seed):
    """Inputs of the call and, as a program has them at hand, weights in 4 bits; for the framework its
    configurations, workspace and output buffers."""
    st = dict(_inputs(case, seed), case=case)
    op = case["op"]
    if own:
        _prepare_own(case, st)
    elif op in ("linear", "product"):
        st["w"] = _pack(*_plain_quantize(st["w"].float()))
        if op == "product":
            st["x"] = _pack(*_plain_quantize(st["x"].float()))
    elif op == "linear_bwd":
        st["wt"] = _pack(*_plain_quantize(st.pop("w").float().t()))
    return st


def _prepare_own(case, st):
    import streaming_causal_video_gb300 as sd
    op = case["op"]
    kinds = {"bf16": sd.BF16, "f32": sd.F32}

    def matrix(rows, cols, kind, transposed=0):
        cfg = sd.Mx4Config.make(rows=rows, cols=cols, x_dtype=kinds[kind], transposed=transposed)
        return (cfg, torch.empty(sd.mx4_codes_bytes(cfg), dtype=torch.uint8, device="cuda"),
                torch.empty(sd.mx4_scales_bytes(cfg), dtype=torch.uint8, device="cuda"))

    def product(rows, cols, depth, kind, gelu=False):
        cfg = sd.Mx4ProductConfig.make(rows=rows, cols=cols, depth=depth, out_dtype=kinds[kind],
                                       activation=sd.GELU if gelu else sd.NO_ACTIVATION)
        ws = torch.empty(sd.mx4_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
        sd.mx4_workspace_init(cfg, ws)
        return cfg, torch.empty((rows, cols), dtype=_TYPES[kind], device="cuda"), ws

    if op == "quantize":
        st["x4"] = matrix(case["rows"], case["cols"], case["x_type"], int(case["transposed"]))
        st["back"] = sd.Mx4Config.make(rows=case["rows"], cols=case["cols"], x_dtype=sd.BF16)
        st["y"] = torch.empty((case["rows"], case["cols"]), dtype=torch.bfloat16, device="cuda")
    elif not op.startswith("rope"):
        M, N, K = case["rows"], case["cols"], case["depth"]
        if op == "linear_bwd":
            st["wt4"] = matrix(K, N, "bf16", 1)
            sd.mx4_quantize(st["wt4"][0], st.pop("w"), *st["wt4"][1:])
            st["dy4"], st["dyt4"], st["xt4"] = (matrix(M, N, case["x_type"]), matrix(N, M, case["x_type"], 1),
                                                matrix(K, M, case["x_type"], 1))
            st["dx"], st["dw"] = product(M, K, N, case["out_type"]), product(N, K, M, "f32")
        else:
            st["w4"] = matrix(N, K, "bf16")
            sd.mx4_quantize(st["w4"][0], st.pop("w"), *st["w4"][1:])
            st["x4"] = matrix(M, K, case["x_type"])
            if op == "product":
                sd.mx4_quantize(st["x4"][0], st.pop("x"), *st["x4"][1:])
            st["y"] = product(M, N, K, case["out_type"], case["gelu"])
    else:
        q, k = st["q"], st["k"]
        one = {"token_stride": q.stride(1), "head_stride": q.stride(2), "batch_stride": q.stride(0)}
        two = {"token_stride": k.stride(1), "head_stride": k.stride(2), "batch_stride": k.stride(0)}
        st["cfg"] = sd.AxesRopeConfig.make(batch=case["batch"], tokens=case["tokens"], heads=case["heads"],
                                           kv_heads=case["kv_heads"], head_dim=case["head_dim"], dims=_dims(case),
                                           halves=int(case["halves"]), base=BASE, dtype=kinds[case["x_type"]],
                                           q_in=one, q_out=one, k_in=two, k_out=two)
        st["q_new"], st["k_new"] = torch.empty_like(q), torch.empty_like(k)


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(state):
    case, op = state["case"], state["case"]["op"]
    if own:
        return _run_own(op, state)
    if op == "quantize":
        x = state["x"].float()
        codes, scales = _plain_quantize(x.t() if case["transposed"] else x)
        return {"values": _plain_values(codes, scales)[:, :case["cols"]].to(torch.bfloat16)}
    if op == "linear":
        return {"y": _plain_product(case, _plain_values(*_plain_quantize(state["x"].float())), _unpack(state["w"]),
                                    state.get("bias"))}
    if op == "product":
        return {"y": _plain_product(case, _unpack(state["x"]), _unpack(state["w"]), state.get("bias"))}
    if op == "linear_bwd":
        dy, x = state["dy"].float(), state["x"].float()
        dx = _plain_values(*_plain_quantize(dy)) @ _unpack(state["wt"]).t()
        dw = _plain_values(*_plain_quantize(dy.t())) @ _plain_values(*_plain_quantize(x.t())).t()
        return {"dx": dx.to(_TYPES[case["out_type"]]), "dw": dw}
    sign = 1.0 if op == "rope_fwd" else -1.0
    return {"q": _plain_rope(case, state["q"], state["positions"], sign),
            "k": _plain_rope(case, state["k"], state["positions"], sign)}


def _run_own(op, st):
    import streaming_causal_video_gb300 as sd
    if op == "quantize":
        cfg, codes, scales = st["x4"]
        sd.mx4_quantize(cfg, st["x"], codes, scales)
        sd.mx4_dequantize(st["back"], codes, scales, st["y"])
        return {"values": st["y"]}
    if op in ("linear", "product"):
        if op == "linear":
            sd.mx4_quantize(st["x4"][0], st["x"], *st["x4"][1:])
        cfg, y, ws = st["y"]
        sd.mx4_product(cfg, *st["x4"][1:], *st["w4"][1:], y, ws, bias=st.get("bias"))
        return {"y": y}
    if op == "linear_bwd":
        sd.mx4_quantize(st["dy4"][0], st["dy"], *st["dy4"][1:])
        sd.mx4_quantize(st["dyt4"][0], st["dy"], *st["dyt4"][1:])
        sd.mx4_quantize(st["xt4"][0], st["x"], *st["xt4"][1:])
        (dx_cfg, dx, dx_ws), (dw_cfg, dw, dw_ws) = st["dx"], st["dw"]
        sd.mx4_product(dx_cfg, *st["dy4"][1:], *st["wt4"][1:], dx, dx_ws)
        sd.mx4_product(dw_cfg, *st["dyt4"][1:], *st["xt4"][1:], dw, dw_ws)
        return {"dx": dx, "dw": dw}
    rotate = sd.axes_rope if op == "rope_fwd" else sd.axes_rope_backward
    rotate(st["cfg"], st["positions"], st["q"], st["q_new"], st["k"], st["k_new"])
    return {"q": st["q_new"], "k": st["k_new"]}


_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _plain_quantize(x):
    """Codes [rows][cols to a whole block] (0 to 7, plus 8 where negative) and exponents [rows][blocks] of
    32-bit x: the power of two by which the block's largest magnitude comes to lie in (3.5, 7]."""
    rows, cols = x.shape
    pad = -cols % BLOCK
    if pad:
        x = torch.cat([x, x.new_zeros((rows, pad))], 1)
    x = x.reshape(rows, -1, BLOCK)
    mantissa, exponent = torch.frexp(x.abs().amax(-1))           # mantissa in [0.5, 1)
    e = torch.clamp(exponent - 3 + (mantissa > 0.875).int(), -127, 127)
    e = torch.where(mantissa == 0, torch.full_like(e, -127), e)
    a = torch.ldexp(x, -e[..., None]).abs()
    # ties go to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + 8 * (x < 0).to(torch.uint8)
    return code.reshape(rows, -1), e


def _plain_values(code, e):
    """32-bit values of codes and exponents."""
    level = torch.tensor(_LEVELS + tuple(-v for v in _LEVELS), device=code.device)[code.long()]
    return torch.ldexp(level.view(code.shape[0], -1, BLOCK), e[..., None]).reshape(code.shape)


def _pack(code, e):
    """Two codes a byte, and the exponents as bytes."""
    return code[:, 0::2] + 16 * code[:, 1::2], (e + 127).to(torch.uint8)


def _unpack(packed):
    both, e = packed
    code = torch.stack([both & 15, both >> 4], -1).view(both.shape[0], -1)
    return _plain_values(code, e.int() - 127)


def _plain_product(case, a, b, bias):
    y = a @ b.t()
    if bias is not None:
        y = y + bias
    if case["gelu"]:
        y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    return y.to(_TYPES[case["out_type"]])


def _plain_rope(case, x, positions, sign):
    x = x.float()
    out = x.clone()
    first = 0
    for a, d in enumerate(_dims(case)):
        # angles in 64 bits: positions are far, and only what is left of whole turns counts
        freq = BASE ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device=x.device) / d)
        angle = positions[:, :, a].double()[..., None] * freq
        cos, sin = torch.cos(angle).float()[:, :, None], sign * torch.sin(angle).float()[:, :, None]
        if case["halves"]:
            i, j = slice(first, first + d // 2), slice(first + d // 2, first + d)
        else:
            i, j = slice(first, first + d, 2), slice(first + 1, first + d, 2)
        u, v = x[..., i], x[..., j]
        out[..., i] = u * cos - v * sin
        out[..., j] = u * sin + v * cos
        first += d
    return out.to(_TYPES[case["x_type"]])


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits, and what a pass has to move and compute
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    d = _inputs(case, seed)
    op = case["op"]
    if op == "quantize":
        x = d["x"].double()
        return {"values": _nearest(x.t() if case["transposed"] else x)}
    if op == "linear_bwd":
        dy, x, w = d["dy"].double(), d["x"].double(), d["w"].double()
        return {"dx": _nearest(dy) @ _nearest(w.t()).t(), "dw": _nearest(dy.t()) @ _nearest(x.t()).t()}
    if not op.startswith("rope"):
        y = _nearest(d["x"].double()) @ _nearest(d["w"].double()).t()
        if case["bias"]:
            y += d["bias"].double()
        if case["gelu"]:
            # (1 + tanh u) / 2 is the logistic function of 2u
            y = y * torch.sigmoid(y * (1.0 + 0.044715 * y ** 2) * math.sqrt(8.0 / math.pi))
        return {"y": y}
    out = {}
    for name in ("q", "k"):
        x = d[name].double()
        B, T, H, D = x.shape
        y = x.clone()
        first = 0
        for a, n in enumerate(_dims(case)):
            seg = x[..., first:first + n]
            pairs = seg.unflatten(-1, (2, n // 2)).movedim(-2, -1) if case["halves"] else seg.unflatten(-1, (n // 2, 2))
            angle = torch.einsum("bt,j->btj", d["positions"][:, :, a].double(),
                                 torch.tensor([BASE ** (-2.0 * j / n) for j in range(n // 2)], dtype=torch.float64,
                                              device=x.device))
            turn = torch.polar(torch.ones_like(angle), angle if op == "rope_fwd" else -angle)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, :, None])
            y[..., first:first + n] = z.movedim(-1, -2).flatten(-2) if case["halves"] else z.flatten(-2)
            first += n
        out[name] = y
    return out


def _nearest(x):
    """64-bit values that the rows of x have in 4 bits: of each block of 32, e is the least power of two with
    amax <= 7 * 2^e (2^-127 at least), and a number goes to the nearest of 2^e times 0, 0.5, 1, 1.5, 2, 3, 4, 6, and
    from the middle of two to the one at an even place of that list."""
    rows, cols = x.shape
    padded = torch.nn.functional.pad(x, (0, -cols % BLOCK)).view(rows, -1, BLOCK)
    top = padded.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(top / 7.0)).clamp(-128, 127)      # 2^e may still be off by one step either way
    e = torch.where(7.0 * torch.exp2(e - 1) >= top, e - 1, e)
    e = torch.where(7.0 * torch.exp2(e) < top, e + 1, e).clamp(min=-127)
    unit = torch.exp2(e)
    v = padded / unit
    size = v.abs()
    # steps of a half below 2, of one below 4, of two above; torch rounds middles to even
    step = 0.5 + 0.5 * (size >= 2) + (size >= 4)
    near = torch.round(size / step) * step
    near = torch.clamp(near, max=6.0)
    return (torch.copysign(near, v) * unit).view(rows, -1)[:, :cols]


def work(case):
    size = {"bf16": 2, "f32": 4}
    op = case["op"]
    four = 0.5 + 1.0 / BLOCK                     # bytes of a number and its share of a scale
    if op == "quantize":                         # x in, 4 bits out and in again, bf16 out
        n = case["rows"] * case["cols"]
        return {"bytes": n * (size[case["x_type"]] + 2 * four + 2), "flops": 4 * n}
    if not op.startswith("rope"):
        M, N, K = case["rows"], case["cols"], case["depth"]
        out, x = size[case["out_type"]], size[case["x_type"]]
        if op == "linear_bwd":                   # dy, x and the weight in; dx and dw out; two products
            return {"bytes": M * N * x + M * K * (x + out) + N * K * (four + 4), "flops": 4 * M * N * K}
        given = M * K * (x if op == "linear" else four)
        return {"bytes": given + N * K * four + M * N * out + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    rows = case["batch"] * case["tokens"] * (case["heads"] + case["kv_heads"])
    return {"bytes": 2 * rows * case["head_dim"] * size[case["x_type"]] + case["batch"] * case["tokens"] * 4 * len(_dims(case)),
            "flops": 3 * rows * sum(_dims(case))}
