"""The layer operators in fp64 (oracle side): layer norm, the short causal
convolution, the selective state space scan, one token of the delta rule.

TEST INFRASTRUCTURE ONLY.

Each is its definition written out token by token or row by row, with its
gradient by the chain rule; no code is shared with the GPU path.  Sequences are
given as (batch row, first token, last token + 1) spans (`spans`), so batches
and packed batches are one code path.
"""
from __future__ import annotations

import numpy as np

__all__ = ["spans", "layer_norm", "layer_norm_backward", "causal_conv", "causal_conv_backward", "selective_scan",
           "selective_scan_backward", "delta_step", "sigmoid", "softplus"]


def f64(x):
    return np.asarray(x, dtype=np.float64)


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def softplus(x):
    return np.logaddexp(0.0, x)


def spans(B, T, cu=None):
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, int(cu[i]), int(cu[i + 1])) for i in range(len(cu) - 1)]


def layer_norm(x, w=None, b=None, eps=1e-5):
    """(y, mean, rstd) over the last axis."""
    x = f64(x)
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    xh = (x - mean[..., None]) * rstd[..., None]
    y = xh * (1.0 if w is None else f64(w)) + (0.0 if b is None else f64(b))
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, w=None):
    """(dx, dw, db) for rows [R, D], from the given mean and rstd."""
    dy, x, r = f64(dy), f64(x), f64(rstd)[:, None]
    xh = (x - f64(mean)[:, None]) * r
    g = dy * (1.0 if w is None else f64(w))
    dx = r * (g - g.mean(-1, keepdims=True) - xh * (g * xh).mean(-1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def causal_conv(x, w, b=None, state=None, seqs=None, silu=True):
    """(y, final states [n, W - 1, D]) of x [B, T, D]."""
    x, w = f64(x), f64(w)
    D, W = w.shape
    seqs = seqs or spans(*x.shape[:2])
    y = np.zeros(x.shape)
    last = np.zeros((len(seqs), W - 1, D))
    for n, (r, t0, t1) in enumerate(seqs):
        rows = np.concatenate([np.zeros((W - 1, D)) if state is None else f64(state)[n], x[r, t0:t1]])
        for t in range(t1 - t0):
            u = (rows[t:t + W] * w.T).sum(0) + (0.0 if b is None else f64(b))
            y[r, t0 + t] = u * sigmoid(u) if silu else u
        last[n] = rows[len(rows) - (W - 1):]
    return y, last


def causal_conv_backward(dy, x, w, b=None, state=None, seqs=None, silu=True, d_last=None):
    """(dx, dw, db, d_state)."""
    dy, x, w = f64(dy), f64(x), f64(w)
    D, W = w.shape
    seqs = seqs or spans(*x.shape[:2])
    dx, dw, db = np.zeros(x.shape), np.zeros((D, W)), np.zeros(D)
    ds = np.zeros((len(seqs), W - 1, D))
    for n, (r, t0, t1) in enumerate(seqs):
        rows = np.concatenate([np.zeros((W - 1, D)) if state is None else f64(state)[n], x[r, t0:t1]])
        dr = np.zeros(rows.shape)
        if d_last is not None:
            dr[len(rows) - (W - 1):] += f64(d_last)[n]
        for t in range(t1 - t0):
            du = dy[r, t0 + t].copy()
            if silu:
                u = (rows[t:t + W] * w.T).sum(0) + (0.0 if b is None else f64(b))
                s = sigmoid(u)
                du *= s + u * s * (1.0 - s)
            dr[t:t + W] += w.T * du
            dw += (rows[t:t + W] * du).T
            db += du
        dx[r, t0:t1], ds[n] = dr[W - 1:], dr[:W - 1]
    return dx, dw, db, ds


def _step(dt, bias, use_softplus):
    pre = f64(dt) + (0.0 if bias is None else f64(bias))
    return pre, softplus(pre) if use_softplus else pre


def selective_scan(x, dt, A, B, C, D=None, z=None, bias=None, use_softplus=True, state=None, seqs=None):
    """(y, final states [n, D, N]) of x, dt, z [Bt, T, D], B, C [Bt, T, N]."""
    x, A, B, C = f64(x), f64(A), f64(B), f64(C)
    seqs = seqs or spans(*x.shape[:2])
    _, s = _step(dt, bias, use_softplus)
    y = np.zeros(x.shape)
    last = np.zeros((len(seqs), *A.shape))
    for n, (r, t0, t1) in enumerate(seqs):
        h = np.zeros(A.shape) if state is None else f64(state)[n].copy()
        for t in range(t0, t1):
            h = np.exp(s[r, t][:, None] * A) * h + (s[r, t] * x[r, t])[:, None] * B[r, t]
            y[r, t] = h @ C[r, t]
        last[n] = h
    if D is not None:
        y = y + f64(D) * x
    if z is not None:
        y = y * f64(z) * sigmoid(f64(z))
    return y, last


def selective_scan_backward(dy, x, dt, A, B, C, D=None, z=None, bias=None, use_softplus=True, state=None, seqs=None,
                            d_last=None, magnitude=False):
    """(dx, ddt, dA, dB, dC, dD, dz, dbias, d_state).  magnitude: for inputs
    that are all given as absolute values (A and dt as they are), the sums of
    the absolute values of the gradients' terms."""
    dy, x, A, B, C = f64(dy), f64(x), f64(A), f64(B), f64(C)
    seqs = seqs or spans(*x.shape[:2])
    pre, s = _step(dt, bias, use_softplus)
    skip = 0.0 if D is None else f64(D)
    dx, ds, dz = np.zeros(x.shape), np.zeros(x.shape), np.zeros(x.shape)
    dA, dB, dC = np.zeros(A.shape), np.zeros(B.shape), np.zeros(C.shape)
    dD, dst = np.zeros(x.shape[2]), np.zeros((len(seqs), *A.shape))
    for n, (r, t0, t1) in enumerate(seqs):
        h = [np.zeros(A.shape) if state is None else f64(state)[n]]
        for t in range(t0, t1):
            h.append(np.exp(s[r, t][:, None] * A) * h[-1] + (s[r, t] * x[r, t])[:, None] * B[r, t])
        dh = np.zeros(A.shape) if d_last is None else f64(d_last)[n].copy()
        for t in range(t1 - 1, t0 - 1, -1):
            now, before = h[t - t0 + 1], h[t - t0]
            g = dy[r, t]
            if z is not None:
                zz = f64(z)[r, t]
                sg = sigmoid(zz)
                dz[r, t] = g * (now @ C[r, t] + skip * x[r, t]) * (sg + zz * sg * (1.0 - sg))
                g = g * zz * sg
            dD += g * x[r, t]
            dC[r, t] = g @ now
            dh = dh + g[:, None] * C[r, t]
            a = np.exp(s[r, t][:, None] * A)
            q = dh * a * before
            dB[r, t] = (s[r, t] * x[r, t]) @ dh
            du = dh @ B[r, t]
            dA += q * s[r, t][:, None]
            ds[r, t] = (q * (np.abs(A) if magnitude else A)).sum(1) + du * x[r, t]
            dx[r, t] = du * s[r, t] + skip * g
            dh = dh * a
        dst[n] = dh
    ddt = ds * sigmoid(pre) if use_softplus else ds
    return dx, ddt, dA, dB, dC, dD, dz, ddt.sum((0, 1)), dst


def delta_step(q, k, v, g, beta, S, scale=None, l2norm=False, eps=1e-6):
    """(o [N, H, dv], new S [N, H, dk, dv]) of one token."""
    q, k, v, g, beta, S = (f64(t) for t in (q, k, v, g, beta, S))
    if l2norm:
        q = q / np.sqrt((q * q).sum(-1, keepdims=True) + eps)
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + eps)
    S = S * np.exp(g)[..., None, None]
    u = beta[..., None] * (v - np.einsum("nhj,nhji->nhi", k, S))
    S = S + np.einsum("nhj,nhi->nhji", k, u)
    scale = scale or q.shape[-1] ** -0.5
    return scale * np.einsum("nhj,nhji->nhi", q, S), S
