"""The fp64 oracle of the layer operators: gradients against central
differences, the scan and the convolution against a sequence cut in two, the
single token against the recurrence's oracle.

Central differences with step e have an error of about e^2 f''' / 6 + 1e-16 |f| / e;
e = 1e-5 and values of order one leave 1e-9, so 1e-6 of the gradient's size is
a bar that only a wrong formula misses."""
import numpy as np
import pytest

import oracle
from oracle.layer_ops import (causal_conv, causal_conv_backward, delta_step, layer_norm, layer_norm_backward,
                              selective_scan, selective_scan_backward, spans)


def differences(f, args, name, e=1e-5):
    """Central differences of the scalar f(**args) in the array args[name]."""
    x = args[name]
    g = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        up, dn = x.copy(), x.copy()
        up[i] += e
        dn[i] -= e
        g[i] = (f(**dict(args, **{name: up})) - f(**dict(args, **{name: dn}))) / (2 * e)
    return g


def same(got, want):
    assert np.abs(got - want).max() <= 1e-6 * max(1.0, np.abs(want).max())


def test_layer_norm_backward_is_the_gradient():
    r = np.random.default_rng(0)
    x, w, b, dy = r.normal(size=(3, 5)), r.normal(size=5), r.normal(size=5), r.normal(size=(3, 5))
    f = lambda x, w, b: float((layer_norm(x, w, b)[0] * dy).sum())   # noqa: E731
    _, mean, rstd = layer_norm(x, w, b)
    got = layer_norm_backward(dy, x, mean, rstd, w)
    for g, name in zip(got, ("x", "w", "b")):
        same(g, differences(f, dict(x=x, w=w, b=b), name))


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("cu", [None, [0, 0, 1, 5, 5, 7]])
def test_conv_backward_is_the_gradient(W, silu, cu):
    r = np.random.default_rng(1)
    B, T, D = (2, 4, 3) if cu is None else (1, 7, 3)
    seqs = spans(B, T, cu)
    a = dict(x=r.normal(size=(B, T, D)), w=r.normal(size=(D, W)), b=r.normal(size=D),
             state=r.normal(size=(len(seqs), W - 1, D)))
    dy, dl = r.normal(size=(B, T, D)), r.normal(size=(len(seqs), W - 1, D))

    def f(x, w, b, state):
        y, last = causal_conv(x, w, b, state, seqs, silu)
        return float((y * dy).sum() + (last * dl).sum())

    got = causal_conv_backward(dy, a["x"], a["w"], a["b"], a["state"], seqs, silu, dl)
    for g, name in zip(got, ("x", "w", "b", "state")):
        same(g, differences(f, a, name))


@pytest.mark.parametrize("use_softplus", [True, False])
@pytest.mark.parametrize("cu", [None, [0, 1, 1, 5]])
def test_scan_backward_is_the_gradient(use_softplus, cu):
    r = np.random.default_rng(2)
    Bt, T, D, N = (2, 3, 2, 3) if cu is None else (1, 5, 2, 3)
    seqs = spans(Bt, T, cu)
    a = dict(x=r.normal(size=(Bt, T, D)), dt=0.3 * r.normal(size=(Bt, T, D)), A=-np.exp(r.normal(size=(D, N))),
             B=r.normal(size=(Bt, T, N)), C=r.normal(size=(Bt, T, N)), D=r.normal(size=D), z=r.normal(size=(Bt, T, D)),
             bias=r.normal(size=D), state=r.normal(size=(len(seqs), D, N)))
    dy, dl = r.normal(size=(Bt, T, D)), r.normal(size=(len(seqs), D, N))

    def f(**k):
        y, last = selective_scan(use_softplus=use_softplus, seqs=seqs, **k)
        return float((y * dy).sum() + (last * dl).sum())

    got = selective_scan_backward(dy, use_softplus=use_softplus, seqs=seqs, d_last=dl, **a)
    for g, name in zip(got, ("x", "dt", "A", "B", "C", "D", "z", "bias", "state")):
        same(g, differences(f, a, name))


def test_conv_and_scan_continue_from_their_states():
    r = np.random.default_rng(3)
    x, w, b = r.normal(size=(1, 9, 2)), r.normal(size=(2, 4)), r.normal(size=2)
    y, last = causal_conv(x, w, b)
    y0, s0 = causal_conv(x[:, :2], w, b)
    y1, s1 = causal_conv(x[:, 2:], w, b, s0)
    assert np.allclose(np.concatenate([y0, y1], 1), y, atol=1e-14) and np.allclose(s1, last, atol=0)
    dt, B, C = r.normal(size=(1, 9, 2)), r.normal(size=(1, 9, 3)), r.normal(size=(1, 9, 3))
    A = -np.exp(r.normal(size=(2, 3)))
    y, last = selective_scan(x, dt, A, B, C)
    y0, s0 = selective_scan(x[:, :4], dt[:, :4], A, B[:, :4], C[:, :4])
    y1, s1 = selective_scan(x[:, 4:], dt[:, 4:], A, B[:, 4:], C[:, 4:], state=s0)
    assert np.allclose(np.concatenate([y0, y1], 1), y, atol=1e-13) and np.allclose(s1, last, atol=1e-13)


def test_delta_step_is_the_recurrence():
    r = np.random.default_rng(4)
    T, H, dk, dv = 6, 2, 4, 3
    q, k = r.normal(size=(1, T, H, dk)), r.normal(size=(1, T, H, dk))
    q, k = q / np.linalg.norm(q, axis=-1, keepdims=True), k / np.linalg.norm(k, axis=-1, keepdims=True)
    v, g, beta = r.normal(size=(1, T, H, dv)), -r.random((1, T, H)), r.random((1, T, H))
    S = r.normal(size=(1, H, dk, dv))
    o_ref, S_ref = oracle.gdn_reference(q, k, v, g, beta, S, None, scale=0.5)
    for t in range(T):
        o, S = delta_step(q[:, t], k[:, t], v[:, t], g[:, t], beta[:, t], S, 0.5)
        assert np.allclose(o[0], o_ref.reshape(T, H, dv)[t], atol=1e-12)
    assert np.allclose(S, S_ref, atol=1e-12)
