"""The operators between and beside a layer's recurrence in fp64 (oracle side): the
block norm and the gated feed-forward block.

TEST INFRASTRUCTURE ONLY.

Each is its definition with its gradient by the chain rule; no code is shared with
the GPU path.  Rows are [R, D].
"""
from __future__ import annotations

import numpy as np

from .layer_ops import f64, sigmoid

__all__ = ["gate_value", "block_norm", "block_norm_backward", "ffn_activation", "gated_ffn", "gated_ffn_backward"]


def gate_value(z, activation):
    """(a(z), a'(z)); (1, 0) without a gate."""
    if z is None:
        return 1.0, 0.0
    z = f64(z)
    s = sigmoid(z)
    if activation == "sigmoid":
        return s, s * (1.0 - s)
    return z * s, s + z * s * (1.0 - s)


def block_norm(y, r=None, z=None, w_post=None, scale=None, w_pre=None, post=True, pre=True, activation="silu", eps=1e-5):
    """(x, h, rstd_post, rstd_pre), None for what is left out."""
    n = f64(y)
    rp = rn = h = None
    if post:
        rp = 1.0 / np.sqrt((n * n).mean(-1) + eps)
        n = n * rp[:, None] * (1.0 if w_post is None else f64(w_post))
    x = n * gate_value(z, activation)[0] * (1.0 if scale is None else f64(scale)) + (0.0 if r is None else f64(r))
    if pre:
        rn = 1.0 / np.sqrt((x * x).mean(-1) + eps)
        h = x * rn[:, None] * (1.0 if w_pre is None else f64(w_pre))
    return x, h, rp, rn


def block_norm_backward(dx, dh, y, x, rp, rn, z=None, w_post=None, scale=None, w_pre=None, activation="silu",
                        magnitude=False):
    """(dy, dr, dz, dw_post, dscale, dw_pre).  magnitude: for inputs that are all given
    as absolute values (z as it is), the sums of the absolute values of the terms."""
    sign = -1.0 if not magnitude else 1.0
    y = f64(y)
    one = np.ones(y.shape[1])
    wp, sc, wn = (one if w is None else f64(w) for w in (w_post, scale, w_pre))
    d = np.zeros(y.shape) if dx is None else f64(dx)
    dwn = np.zeros(y.shape[1])
    if rn is not None:
        r = f64(rn)[:, None]
        xh, g = f64(x) * r, f64(dh) * wn
        dwn = (f64(dh) * xh).sum(0)
        d = d + r * (g + sign * xh * (g * xh).mean(-1, keepdims=True))
    a, slope = gate_value(z, activation)
    if magnitude:
        a, slope = np.abs(a), np.abs(slope) + np.abs(a) + 1.0   # a' moves by up to this times the sigmoid's error
    yh = y if rp is None else y * f64(rp)[:, None]
    e = d * sc * a * wp
    dz = d * sc * wp * yh * slope
    dwp, ds = (d * sc * a * yh).sum(0), (d * a * wp * yh).sum(0)
    dy = e if rp is None else f64(rp)[:, None] * (e + sign * yh * (e * yh).mean(-1, keepdims=True))
    return dy, d, dz, dwp, ds, dwn


def ffn_activation(g, activation):
    """(act(g), act'(g))."""
    g = f64(g)
    if activation == "silu":
        return gate_value(g, "silu")
    u = np.sqrt(2.0 / np.pi) * (g + 0.044715 * g ** 3)
    t = np.tanh(u)
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * np.sqrt(2.0 / np.pi) * (1.0 + 3.0 * 0.044715 * g * g)


def gated_ffn(x, wg, wu, wd, activation="silu"):
    """(y, g, u, h)."""
    x, wg, wu, wd = f64(x), f64(wg), f64(wu), f64(wd)
    g, u = x @ wg.T, x @ wu.T
    h = ffn_activation(g, activation)[0] * u
    return h @ wd.T, g, u, h


def gated_ffn_backward(dy, x, wg, wu, wd, g, u, activation="silu"):
    """(dx, dwg, dwu, dwd) and (dg, du, h)."""
    dy, x, wg, wu, wd, u = f64(dy), f64(x), f64(wg), f64(wu), f64(wd), f64(u)
    a, slope = ffn_activation(g, activation)
    dh = dy @ wd
    dg, du, h = dh * u * slope, dh * a, a * u
    return (dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ h), (dg, du, h)
