"""fp64 numpy definitions of the operators around the mixer: the channel-wise
gated recurrence and its gradients, the seam between two blocks (post-norm,
gate, scaled residual, pre-norm) and its gradients, rotary positions.

Plain restatements of the formulas, sharing no code with the CUDA path.  Each
function also returns, where asked, a magnitude of the same shape as a result:
the result's own sum with every term replaced by its absolute value (and, for
the recurrences, with the error that a relative perturbation of every factor
would build up).  A result computed with relative errors of at most delta per
factor and term is within delta times that magnitude of the exact one, to
first order; a decay a = exp(la) counts 1 + |la| times, since a relative error
delta of its exponent is one of |la| delta of itself.
"""
from __future__ import annotations

import numpy as np

PLAIN, STEP, UNIT = 0, 1, 2


def softplus(z):
    return np.logaddexp(z, 0.0)


def sigmoid(z):
    return np.where(z >= 0, 1.0 / (1.0 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1.0 + np.exp(-np.abs(z))))


def gates(dt, A_log, dt_bias=None, scale=PLAIN):
    """z, Delta, log a, a, beta of every (sequence, token, channel)."""
    z = np.asarray(dt, np.float64) + (0.0 if dt_bias is None else np.asarray(dt_bias, np.float64))
    delta = softplus(z)
    la = -delta * np.exp(np.asarray(A_log, np.float64))
    a = np.exp(la)
    beta = np.ones_like(a) if scale == PLAIN else delta if scale == STEP else np.sqrt(-np.expm1(2.0 * la))
    return z, delta, la, a, beta


def _lengths(lengths, B, L):
    n = np.full(B, L) if lengths is None else np.clip(np.asarray(lengths, np.int64), 0, L)
    return n, np.arange(L)[None, :] < n[:, None]


def gated_scan(x, dt, A_log, dt_bias=None, h0=None, lengths=None, scale=PLAIN):
    """(y, h_out, magnitude of y): y rows behind a sequence's end are zero."""
    x = np.asarray(x, np.float64)
    B, L, D = x.shape
    _, _, la, a, beta = gates(dt, A_log, dt_bias, scale)
    _, on = _lengths(lengths, B, L)
    h = np.zeros((B, D)) if h0 is None else np.asarray(h0, np.float64).copy()
    m, e = np.abs(h), np.zeros((B, D))
    y, mag = np.zeros_like(x), np.zeros_like(x)
    for t in range(L):
        live = on[:, t, None]
        u = beta[:, t] * x[:, t]
        m2 = a[:, t] * m + np.abs(u)
        e = np.where(live, a[:, t] * (e + m * (1 - la[:, t])) + np.abs(u), e)
        h = np.where(live, a[:, t] * h + u, h)
        m = np.where(live, m2, m)
        y[:, t], mag[:, t] = np.where(live, h, 0.0), np.where(live, e, 0.0)
    return y, h, mag


def gated_scan_bwd(x, dt, dy, A_log, dt_bias=None, h0=None, lengths=None, scale=PLAIN, dh_out=None):
    """Gradients of sum(dy * y) + sum(dh_out * h_out): dict of (value, magnitude) for
    dx, ddt, dA_log, d_dt_bias, dh0.  Rows behind a sequence's end are zero."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    B, L, D = x.shape
    z, delta, la, a, beta = gates(dt, A_log, dt_bias, scale)
    rate = np.exp(np.asarray(A_log, np.float64))
    _, on = _lengths(lengths, B, L)
    h = np.zeros((B, D)) if h0 is None else np.asarray(h0, np.float64).copy()
    m, e = np.abs(h), np.abs(h)
    hb, mb, eb = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)      # h_{t-1}, its magnitudes
    for t in range(L):
        live = on[:, t, None]
        hb[:, t], mb[:, t], eb[:, t] = h, m, e
        u = beta[:, t] * x[:, t]
        m2 = a[:, t] * m + np.abs(u)
        e = np.where(live, a[:, t] * (e + m * (1 - la[:, t])) + np.abs(u), e)
        h = np.where(live, a[:, t] * h + u, h)
        m = np.where(live, m2, m)
    c = np.zeros((B, D)) if dh_out is None else np.asarray(dh_out, np.float64).copy()
    cm, ce = np.abs(c), np.abs(c)
    g, gm, ge = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    for t in range(L - 1, -1, -1):
        live = on[:, t, None]
        gt, gmt = dy[:, t] + c, np.abs(dy[:, t]) + cm
        get = ce + gmt
        g[:, t], gm[:, t], ge[:, t] = (np.where(live, v, 0.0) for v in (gt, gmt, get))
        c, cm = (np.where(live, a[:, t] * v, w) for v, w in ((gt, c), (gmt, cm)))
        ce = np.where(live, a[:, t] * (get + gmt * (1 - la[:, t])), ce)
    dla, dlam = g * a * hb, a * (ge * mb + gm * eb + gm * mb * (1 - la))
    if scale == UNIT:
        k = np.where(beta > 0, a * a / np.where(beta > 0, beta, 1.0), 0.0)
        dla, dlam = dla - g * x * k, dlam + (ge + gm * (1 - la)) * np.abs(x) * k
    dd, ddm = -rate * dla, rate * dlam
    if scale == STEP:
        dd, ddm = dd + g * x, ddm + ge * np.abs(x)
    s = sigmoid(z)
    return {"dx": (g * beta, ge * beta), "ddt": (dd * s, ddm * s),
            "dA_log": ((dla * la).sum((0, 1)), (dlam * -la).sum((0, 1))),
            "d_dt_bias": ((dd * s).sum((0, 1)), (ddm * s).sum((0, 1))), "dh0": (c, ce)}


def _norm(u, w, b, layer, eps):
    """norm(u) w + b, the normalised rows, 1 / sqrt(var + eps), magnitude."""
    D = u.shape[-1]
    mean = u.mean(-1, keepdims=True) if layer else 0.0
    rstd = 1.0 / np.sqrt(((u - mean) ** 2).sum(-1, keepdims=True) / D + eps)
    n = (u - mean) * rstd
    w = 1.0 if w is None else np.asarray(w, np.float64)
    b = 0.0 if b is None else np.asarray(b, np.float64)
    return n * w + b, n, rstd


def norm_gate(y, r, gate=None, layer=False, post=True, eps=1e-5, alpha=1.0, scale=None, post_w=None, post_b=None,
              pre_w=None, pre_b=None):
    """(r_out, xn)."""
    n = np.asarray(y, np.float64)
    if post:
        n = _norm(n, post_w, post_b, layer, eps)[0]
    if gate is not None:
        g = np.asarray(gate, np.float64)
        n = n * g * sigmoid(g)
    s = 1.0 if scale is None else np.asarray(scale, np.float64)
    out = (0.0 if r is None else np.asarray(r, np.float64)) + alpha * s * n
    return out, _norm(out, pre_w, pre_b, layer, eps)[0]


def _norm_bwd(d, w, n, rstd, layer):
    """Gradient of the norm's input from that of its output."""
    d = d * (1.0 if w is None else np.asarray(w, np.float64))
    c = d - n * (d * n).mean(-1, keepdims=True)
    return (c - d.mean(-1, keepdims=True) if layer else c) * rstd


def norm_gate_bwd(y, r_out, dr_out, dxn, gate=None, layer=False, post=True, eps=1e-5, alpha=1.0, scale=None,
                  post_w=None, post_b=None, pre_w=None):
    """Gradients of sum(dr_out * r_out) + sum(dxn * xn): dict of dy, dgate, dr and the
    parameters' (dscale, dpost_w, dpost_b, dpre_w, dpre_b)."""
    y = np.asarray(y, np.float64)
    dr = np.zeros_like(y) if dr_out is None else np.asarray(dr_out, np.float64)
    out = {"dpre_w": np.zeros(y.shape[-1]), "dpre_b": np.zeros(y.shape[-1])}
    if dxn is not None:
        dxn = np.asarray(dxn, np.float64)
        _, n, rstd = _norm(np.asarray(r_out, np.float64), None, None, layer, eps)
        out["dpre_w"], out["dpre_b"] = (dxn * n).sum(0), dxn.sum(0)
        dr = dr + _norm_bwd(dxn, pre_w, n, rstd, layer)
    s = 1.0 if scale is None else np.asarray(scale, np.float64)
    u, v, rstd = y, y, 1.0
    if post:
        v, u, rstd = _norm(y, post_w, post_b, layer, eps)
    dm = alpha * s * dr
    if gate is None:
        m, dn, out["dgate"] = v, dm, None
    else:
        g = np.asarray(gate, np.float64)
        sg = sigmoid(g)
        m, dn = v * g * sg, dm * g * sg
        out["dgate"] = dm * v * sg * (1.0 + g * (1.0 - sg))
    out["dscale"] = alpha * (dr * m).sum(0)
    out["dpost_w"], out["dpost_b"] = (dn * u).sum(0), dn.sum(0)
    out["dy"] = _norm_bwd(dn, post_w, u, rstd, layer) if post else dn
    out["dr"] = dr
    return out


def rotary_theta(rot, base=10000.0, scaling="none", factor=1.0, orig_len=0.0, beta_slow=1.0, beta_fast=32.0):
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    th = base ** (-2.0 * i / rot)
    if scaling == "linear":
        th = th / factor
    if scaling == "by_parts":
        w = np.clip((orig_len * th / (2 * np.pi) - beta_slow) / (beta_fast - beta_slow), 0.0, 1.0)
        th = th * ((1 - w) / factor + w)
    return th


def rotary(x, positions, rot=0, interleaved=False, transpose=False, mscale=1.0, **kw):
    """x [B, L, H, d] turned at positions [B, L] (broadcast); kw as rotary_theta."""
    x = np.asarray(x, np.float64)
    rot = rot or x.shape[-1]
    ang = np.broadcast_to(np.asarray(positions), x.shape[:2]).astype(np.float64)[..., None, None] * \
        rotary_theta(rot, **kw)
    cs, sn = mscale * np.cos(ang), mscale * np.sin(ang) * (-1.0 if transpose else 1.0)
    u, v = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    out = x.copy()
    out[..., u] = x[..., u] * cs - x[..., v] * sn
    out[..., v] = x[..., u] * sn + x[..., v] * cs
    return out
