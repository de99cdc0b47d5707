"""Plain 64-bit implementations of cross attention and layer norm, with the error bounds that the
kernels' roundings allow, for the tests of those operators.

Bounds (all sums below are computed beside the reference, per element):
* a rounding to bf16 is off by at most half a step, 2^-8 of the value; to fp32 by 2^-24;
* an fp32 sum of 128 products in any order is off by at most 128 * 2^-23 = 2^-16 of the sum of the
  products' magnitudes (2^-23 per addition covers accumulators that truncate);
* so a score is off by 2^-16 of the scaled sum of |q||k|, and a probability by twice that relative to
  itself (its own score, the normaliser's); the exponential and the division add a few 2^-22.
"""
import math

import torch

BF = 2.0 ** -8
F32 = 2.0 ** -24
SUM = 2.0 ** -16


def score_size(q, k, scale):
    """Largest scaled sum of |q||k| over the pairs."""
    return float((q.abs() @ k.abs().transpose(-1, -2)).max()) * scale


def prob_error(top):
    """Relative error of a probability whose scores' sums of magnitudes are at most `top`."""
    return 2 * SUM * top + 2.0 ** -20


def heads_first(t, heads):
    """[B][N][Hk][D] -> 64-bit [B][heads][N][D]."""
    t = t.double().transpose(1, 2)
    return t.repeat_interleave(heads // t.shape[1], 1)


def cross_reference(q, k, v, lens, scale):
    """out [B][Nq][H][D], lse [B][H][Nq] in 64 bits and the bounds of both.  q, k, v: [B][N][H][D] views."""
    B, nq, H, D = q.shape
    out = torch.zeros((B, nq, H, D), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    lse = torch.full((B, H, nq), -math.inf, dtype=torch.float64, device=q.device)
    lse_tol = torch.zeros_like(lse)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        qb = q[b:b + 1].double().transpose(1, 2)[0]
        kb, vb = (heads_first(t[b:b + 1, :n], H)[0] for t in (k, v))
        top = score_size(qb, kb, scale)
        s = qb @ kb.transpose(1, 2) * scale
        p = torch.softmax(s, -1)
        o = p @ vb
        out[b] = o.transpose(0, 1)
        # the output's rounding, then the probabilities' rounding and error
        tol[b] = (BF * o.abs() + (BF + prob_error(top)) * (p @ vb.abs())).transpose(0, 1)
        lse[b] = torch.logsumexp(s, -1)
        lse_tol[b] = SUM * top + 2.0 ** -20 * (1 + lse[b].abs())
    return out, lse, tol, lse_tol


def cross_backward_reference(q, k, v, dout, lens, scale):
    """dq [B][Nq][H][D], dk, dv [B][Nk][Hk][D] in 64 bits and their bounds, when the kernel is given the
    forward kernel's out (whose bound enters through delta = rowsum(dO * O)); a stream of 128 keys or fewer
    takes delta = rowsum(P * dP), in 32 bits from the same P and dP."""
    B, nq, H, D = q.shape
    nk, Hk = k.shape[1], k.shape[2]
    mk = lambda *s: torch.zeros(s, dtype=torch.float64, device=q.device)
    dq, dk, dv = mk(B, nq, H, D), mk(B, nk, Hk, D), mk(B, nk, Hk, D)
    tq, tk, tv = torch.zeros_like(dq), torch.zeros_like(dk), torch.zeros_like(dv)
    _, _, out_tol, _ = cross_reference(q, k, v, lens, scale)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        qb, db = q[b].double().transpose(0, 1), dout[b].double().transpose(0, 1)
        kb, vb = (heads_first(t[b:b + 1, :n], H)[0] for t in (k, v))
        prob = prob_error(score_size(qb, kb, scale))
        p = torch.softmax(qb @ kb.transpose(1, 2) * scale, -1)
        dp = db @ vb.transpose(1, 2)
        delta = (p * dp).sum(-1, keepdim=True)
        ds = p * (dp - delta)
        dp_size = db.abs() @ vb.abs().transpose(1, 2)
        if n <= 128:
            delta_err = (p * ((prob + SUM) * dp.abs() + SUM * dp_size)).sum(-1, keepdim=True)
        else:
            delta_err = (db.abs() * out_tol[b].transpose(0, 1)).sum(-1, keepdim=True)
        ds_err = (BF + prob) * ds.abs() + (1 + BF) * p * (delta_err + SUM * dp_size + SUM * delta_err)
        if n == 1:
            ds, ds_err = torch.zeros_like(ds), torch.zeros_like(ds_err)
        fold = lambda t: t.view(Hk, H // Hk, n, D).sum(1).transpose(0, 1)
        g = scale * ds @ kb
        dq[b] = g.transpose(0, 1)
        tq[b] = (BF * g.abs() + scale * (ds_err + SUM * ds.abs()) @ kb.abs()).transpose(0, 1)
        # sums over the queries: at most 2^-23 per addition of the longest chain
        chain = 2.0 ** -23 * (H // Hk) * nq
        g = fold(scale * ds.transpose(1, 2) @ qb)
        dk[b, :n] = g
        tk[b, :n] = BF * g.abs() + fold(scale * (ds_err + chain * ds.abs()).transpose(1, 2) @ qb.abs())
        g = fold(p.transpose(1, 2) @ db)
        dv[b, :n] = g
        tv[b, :n] = BF * g.abs() + fold(((BF + prob + chain) * p).transpose(1, 2) @ db.abs())
    return (dq, dk, dv), (tq, tk, tv)


def norm_reference(x, weight, bias, per, eps, plus_one, y_step):
    """y, mean, rstd in 64 bits and their bounds.  y_step: half a step of y's type.  A row's sum is at
    most 2^7 additions deep (64 columns of a thread, 5 shuffles, 16 warps), so it is off by at most
    2^-17 of the sum of magnitudes."""
    xd = x.double()
    rows, cols = xd.shape
    group = torch.arange(rows, device=x.device) // per
    mean = xd.mean(1)
    var = ((xd - mean[:, None]) ** 2).mean(1)
    rstd = (var + eps) ** -0.5
    gain = torch.ones((int(group[-1]) + 1, cols), dtype=torch.float64, device=x.device) if weight is None else \
        weight.double() + float(plus_one)
    xhat = (xd - mean[:, None]) * rstd[:, None]
    y = xhat * gain[group]
    size = y.abs()
    if bias is not None:
        y = y + bias.double()[group]
        size = size + bias.double().abs()[group]
    mean_tol = 2.0 ** -17 * xd.abs().mean(1)
    # a mean that is off by d adds d^2 to the variance; the rest is the depth of its sum
    rstd_rel = 2.0 ** -16 + (mean_tol * rstd) ** 2
    y_tol = y_step * y.abs() + gain[group].abs() * ((mean_tol * rstd)[:, None] + (rstd_rel[:, None] + 2.0 ** -22) *
                                                    xhat.abs()) + 4 * F32 * size + 2 * F32 * (xd.abs() * rstd[:, None] *
                                                                                             gain[group].abs())
    return (y, mean, rstd), (y_tol, mean_tol, rstd_rel * rstd)


def norm_backward_reference(x, weight, dy, per, eps, plus_one, x_step):
    """dx, dweight, dbias in 64 bits and their bounds, when the kernel is given the forward kernel's mean
    and rstd."""
    (_, mean, rstd), (_, mean_tol, rstd_tol) = norm_reference(x, weight, None, per, eps, plus_one, F32)
    xd, dyd = x.double(), dy.double()
    rows, cols = xd.shape
    group = torch.arange(rows, device=x.device) // per
    groups = int(group[-1]) + 1
    gain = torch.ones((groups, cols), dtype=torch.float64, device=x.device) if weight is None else \
        weight.double() + float(plus_one)
    r = rstd[:, None]
    xh = (xd - mean[:, None]) * r
    xh_err = (mean_tol * rstd)[:, None] + ((rstd_tol / rstd)[:, None] + 2.0 ** -22) * xh.abs() + 2 * F32 * xd.abs() * r
    g = dyd * gain[group]
    m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - m1 - xh * m2)
    a1, a2 = g.abs().mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
    dx_tol = x_step * dx.abs() + r * (2.0 ** -15 * (g.abs() + a1 + xh.abs() * a2) + xh_err * a2 +
                                      xh.abs() * (g.abs() * xh_err).mean(1, keepdim=True))
    dx_tol = dx_tol + (rstd_tol / rstd)[:, None] * dx.abs()
    put = lambda t: torch.zeros((groups, cols), dtype=torch.float64, device=x.device).index_add_(0, group, t)
    # a column's sum over the rows: at most `per` additions, in fact split over slices and teams
    chain = F32 * min(rows, per) + 2 * F32
    return (dx, put(dyd * xh), put(dyd)), (dx_tol, put(dyd.abs() * xh_err + chain * (dyd * xh).abs()),
                                            put(chain * dyd.abs()))


def within(got, ref, tol, what):
    """|got - ref| <= tol everywhere (and got is finite where the reference is)."""
    got = got.double()
    bad = ~((got - ref).abs() <= tol) & ~(got == ref)
    if bool(bad.any()):
        i = tuple(int(j) for j in bad.nonzero()[0])
        raise AssertionError("%s: %d of %d outside the bound, first at %s: %r, reference %r, bound %.3g" %
                             (what, int(bad.sum()), bad.numel(), i, float(got[i]), float(ref[i]), float(tol[i])))
