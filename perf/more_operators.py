"""The two halves of a layer around its recurrence: what is timed, on which
inputs, their plain forms and their values in 64 bits.

Operators (see include/gdn.h for the definitions):
  block_norm  what lies between two blocks, in one pass: the RMS norm after a
              block, its gate and scale, the residual sum, the RMS norm before
              the next block; forward and backward.  Without the residual and the
              second norm it is the gated norm of the recurrence's heads
  gated_ffn   the gated feed-forward block: both projections, the activation and
              the product, then the projection back; prompts, single tokens,
              training forward (keeps the projections) and backward

`run` computes the plain form (elementary torch operations in fp32, rounded
once) or, when `own` is set, calls the package.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # between two blocks of the layer workload (4 x 8192 tokens, 32 heads x 128)
        dict(name="norm fwd layer", op="norm", mode="fwd", rows=32768, H=0, D=4096, parts="pgrsn", dtype="bf16"),
        # its backward pass in training
        dict(name="norm bwd layer", op="norm", mode="bwd", rows=32768, H=0, D=4096, parts="pgrsn", dtype="bf16"),
        # the gated norm of the recurrence's output, head by head, the gate a slice of a projection
        dict(name="norm fwd heads", op="norm", mode="fwd", rows=16384, H=32, D=128, parts="pg", dtype="bf16"),
        # the same in training, a batch of an odd length
        dict(name="norm bwd heads", op="norm", mode="bwd", rows=8191, H=32, D=128, parts="pg", dtype="bf16"),
        # one token of 16 sequences being served: latency
        dict(name="norm fwd tokens", op="norm", mode="fwd", rows=16, H=0, D=4096, parts="pgrsn", dtype="bf16"),
        # a prompt of 8192 tokens through the feed-forward block of that layer
        dict(name="ffn fwd prompt", op="ffn", mode="fwd", M=8192, D=4096, F=12288, act="silu", dtype="bf16"),
        # training on a sequence of an odd length
        dict(name="ffn bwd train", op="ffn", mode="bwd", M=8191, D=4096, F=12288, act="silu", dtype="bf16"),
        # the forward pass of a smaller model in training
        dict(name="ffn save small", op="ffn", mode="save", M=4096, D=1024, F=4096, act="silu", dtype="bf16"),
        # one token of one sequence: latency, bound by the weights
        dict(name="ffn fwd token", op="ffn", mode="fwd", M=1, D=4096, F=12288, act="silu", dtype="bf16"),
        # one token of a serving batch
        dict(name="ffn fwd batch", op="ffn", mode="fwd", M=64, D=4096, F=12288, act="silu", dtype="bf16"),
        # fp32 training of a small model whose sizes fit no tile
        dict(name="ffn bwd f32 odd", op="ffn", mode="bwd", M=1999, D=1030, F=2750, act="gelu_tanh", dtype="f32"),
        # a packed batch of short prompts in fp32
        dict(name="ffn fwd f32", op="ffn", mode="fwd", M=2048, D=2048, F=6144, act="silu", dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng: random.Random):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if rng.random() < 0.5:
        H = rng.choice([0, 0, rng.randint(1, 40)])
        D = rng.choice([32, 64, 128, 256]) if H else rng.choice([1, 8, 8]) * _log(rng, 33, 1024)
        rows = _log(rng, 1, min(32768, 2 ** 26 // (max(H, 1) * D)))
        parts = "pg" if H else rng.choice(["pgrsn", "prn", "rn", "prsn", "grsn", "p", "pgr"])
        return dict(op="norm", mode=rng.choice(["fwd", "bwd"]), rows=rows, H=H, D=D, parts=parts, dtype=dtype)
    mode = rng.choice(["fwd", "save", "bwd"])
    e = rng.choice([1, 8, 8, 64])
    D = max(1, _log(rng, 64, 4096) // e) * e
    F = max(1, _log(rng, 64, 12288) // e) * e
    most = 2 ** 38 if dtype == "bf16" else 2 ** 35
    M = _log(rng, 1, max(1, min(8192, most // (D * F))))
    return dict(op="ffn", mode=mode, M=M, D=D, F=F, act=rng.choice(["silu", "silu", "gelu_tanh"]), dtype=dtype)


# ----------------------------------------------------------------- the inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(int(seed))
    dt = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, to=dt):
        return torch.randn(*shape, generator=gen, device=DEVICE).mul_(std).to(to)

    s = dict(case=dict(case))
    if case["op"] == "norm":
        rows, H, D, parts = case["rows"], case["H"], case["D"], case["parts"]
        shape = (rows, H, D) if H else (rows, D)
        spread = torch.rand(*shape[:-1], 1, generator=gen, device=DEVICE) * 2.7 + 0.3
        s["y"] = (torch.randn(*shape, generator=gen, device=DEVICE) * spread).to(dt)
        s["z"] = s["r"] = s["w_post"] = s["w_pre"] = s["scale"] = None
        if "g" in parts:                             # the gate: the second half of a projection
            wide = normal(rows, 2 * max(H, 1) * D)
            s["z"] = wide[:, max(H, 1) * D:].view(shape)
        if "r" in parts:
            s["r"] = normal(*shape, std=2.0)
        if "p" in parts:
            s["w_post"] = 1.0 + normal(D, std=0.2, to=torch.float32)
        if "n" in parts:
            s["w_pre"] = 1.0 + normal(D, std=0.2, to=torch.float32)
        if "s" in parts:
            s["scale"] = 0.5 + normal(D, std=0.1, to=torch.float32)
        if case["mode"] == "bwd":
            out = _norm_forward(s, torch.float32)    # what the forward pass left
            s["x"], s["rstd_post"], s["rstd_pre"] = out["x"].to(dt), out["rstd_post"], out["rstd_pre"]
            s["dx"] = normal(*shape)
            s["dh"] = normal(*shape) if "n" in parts else None
        return s
    M, D, F = case["M"], case["D"], case["F"]
    s["x"] = normal(M, D)
    s["w_gate"], s["w_up"] = normal(F, D, std=D ** -0.5), normal(F, D, std=D ** -0.5)
    s["w_down"] = normal(D, F, std=F ** -0.5)
    if case["mode"] == "bwd":
        s["gate"], s["up"] = s["x"] @ s["w_gate"].t(), s["x"] @ s["w_up"].t()   # kept by the forward pass
        s["dy"] = normal(M, D)
    return s


# -------------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import chunked_prefill_gdn_gb300 as gdn
    c = s["case"]
    if c["op"] == "norm" and c["mode"] == "fwd":
        x, h, rstd_post, rstd_pre = gdn.block_norm_fwd(
            s["y"], residual=s["r"], gate=s["z"], post_weight=s["w_post"], scale=s["scale"], pre_weight=s["w_pre"],
            post_norm="p" in c["parts"], pre_norm="n" in c["parts"], activation="silu", eps=EPS)
        return dict(x=x, h=h, rstd_post=rstd_post, rstd_pre=rstd_pre)
    if c["op"] == "norm":
        g = gdn.block_norm_bwd(s["dx"], s["dh"], s["y"], s["x"], s["rstd_post"], s["rstd_pre"], gate=s["z"],
                               post_weight=s["w_post"], scale=s["scale"], pre_weight=s["w_pre"], activation="silu",
                               residual="r" in c["parts"])
        return dict(zip(("dy", "dresidual", "dgate", "dpost", "dscale", "dpre"), g))
    weights = s["w_gate"], s["w_up"], s["w_down"]
    if c["mode"] == "bwd":
        g = gdn.gated_ffn_bwd(s["dy"], s["x"], *weights, s["gate"], s["up"], activation=c["act"])
        return dict(zip(("dx", "dw_gate", "dw_up", "dw_down"), g))
    y, gate, up = gdn.gated_ffn_fwd(s["x"], *weights, activation=c["act"], save=c["mode"] == "save")
    return dict(y=y, gate=gate, up=up)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "ffn":
        return _plain_ffn(s, c)
    dt = s["y"].dtype
    if c["mode"] == "bwd":
        return _plain_norm_bwd(s, dt)
    out = _norm_forward(s, torch.float32)
    return dict(x=out["x"].to(dt), h=out["h"].to(dt) if out["h"] is not None else None, rstd_post=out["rstd_post"],
                rstd_pre=out["rstd_pre"])


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _rstd(x):
    return 1.0 / torch.sqrt(x.square().mean(-1) + EPS)


def _norm_forward(s, to):
    t, rstd_post, rstd_pre, h = s["y"].to(to), None, None, None
    if "p" in s["case"]["parts"]:
        rstd_post = _rstd(t)
        t = t * rstd_post[..., None] * s["w_post"]
    if s["z"] is not None:
        z = s["z"].to(to)
        t = t * z * _sigmoid(z)
    if s["scale"] is not None:
        t = t * s["scale"]
    if s["r"] is not None:
        t = t + s["r"].to(to)
    if "n" in s["case"]["parts"]:
        rstd_pre = _rstd(t)
        h = t * rstd_pre[..., None] * s["w_pre"]
    return dict(x=t, h=h, rstd_post=rstd_post, rstd_pre=rstd_pre)


def _plain_norm_bwd(s, dt):
    lead = tuple(range(s["y"].dim() - 1))
    d, y = s["dx"].float(), s["y"].float()
    out = dict.fromkeys(("dy", "dresidual", "dgate", "dpost", "dscale", "dpre"))
    if s["dh"] is not None:
        dh, r = s["dh"].float(), s["rstd_pre"][..., None]
        xh = s["x"].float() * r
        out["dpre"] = (dh * xh).sum(lead)
        g = dh * s["w_pre"]
        d = d + r * (g - xh * (g * xh).mean(-1, keepdim=True))
    if s["r"] is not None:
        out["dresidual"] = d.to(dt)
    n = yh = y
    if s["rstd_post"] is not None:
        yh = y * s["rstd_post"][..., None]
        n = yh * s["w_post"]
    a = 1.0
    if s["z"] is not None:
        z = s["z"].float()
        sg = _sigmoid(z)
        a = z * sg
    if s["scale"] is not None:
        out["dscale"] = (d * n * a).sum(lead)
        d = d * s["scale"]
    if s["z"] is not None:
        out["dgate"] = (d * n * (sg * (1.0 + z * (1.0 - sg)))).to(dt)
    d = d * a
    if s["rstd_post"] is not None:
        out["dpost"] = (d * yh).sum(lead)
        g = d * s["w_post"]
        d = s["rstd_post"][..., None] * (g - yh * (g * yh).mean(-1, keepdim=True))
    out["dy"] = d.to(dt)
    return out


C1, C3 = math.sqrt(8.0 / math.pi), 0.044715    # gelu_tanh(g) = g sigmoid(C1 (g + C3 g^3))


def _plain_ffn(s, c):
    dt = s["x"].dtype
    x, wg, wu, wd = (s[k].float() for k in ("x", "w_gate", "w_up", "w_down"))
    gelu = c["act"] == "gelu_tanh"
    if c["mode"] != "bwd":
        g, u = x @ wg.t(), x @ wu.t()
        h = g * _sigmoid(C1 * (g + C3 * g * g * g) if gelu else g) * u
        keep = c["mode"] == "save"
        return dict(y=(h @ wd.t()).to(dt), gate=g.to(dt) if keep else None, up=u.to(dt) if keep else None)
    g, u, dy = s["gate"].float(), s["up"].float(), s["dy"].float()
    sg = _sigmoid(C1 * (g + C3 * g * g * g) if gelu else g)
    slope = C1 * (1.0 + 3.0 * C3 * g * g) if gelu else 1.0
    a = g * sg
    dh = dy @ wd
    dg, du = dh * u * (sg + a * (1.0 - sg) * slope), dh * a
    return dict(dx=(dg @ wg + du @ wu).to(dt), dw_gate=(dg.t() @ x).to(dt), dw_up=(du.t() @ x).to(dt),
                dw_down=(dy.t() @ (a * u)).to(dt))


# ------------------------------------------------------- what a pass cannot avoid

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        parts, rows, D = case["parts"], case["rows"] * max(case["H"], 1), case["D"]
        n = rows * D
        stats, params = 4 * rows * ("p" in parts) + 4 * rows * ("n" in parts), 4 * D * sum(k in parts for k in "psn")
        if case["mode"] == "fwd":
            tensors = 2 + ("g" in parts) + ("r" in parts) + ("n" in parts)
            return dict(bytes=tensors * n * e + stats + params, flops=n * (4 + 3 * ("p" in parts) + 4 * ("n" in parts) + 6 * ("g" in parts)))
        tensors = 3 + 2 * ("g" in parts) + 2 * ("n" in parts) + ("r" in parts)
        return dict(bytes=tensors * n * e + stats + 2 * params, flops=n * (6 + 8 * ("p" in parts) + 10 * ("n" in parts) + 12 * ("g" in parts)))
    M, D, F = case["M"], case["D"], case["F"]
    if case["mode"] == "bwd":
        return dict(bytes=e * (3 * M * D + 2 * M * F + 6 * D * F), flops=12 * M * D * F)
    kept = 2 * M * F if case["mode"] == "save" else 0
    return dict(bytes=e * (2 * M * D + 3 * D * F + kept), flops=6 * M * D * F)


# -------------------------------------------------------- the values in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if torch.is_tensor(v) else v for k, v in s.items()}
    return _exact_ffn(s, case) if case["op"] == "ffn" else _exact_norm(s, case)


def _exact_norm(s, c):
    D, parts = c["D"], c["parts"]
    one = torch.ones(D, dtype=torch.float64, device=DEVICE)
    wp, wn, sc = (s[k] if s[k] is not None else one for k in ("w_post", "w_pre", "scale"))
    e = 1 / (1 + torch.exp(-s["z"])) if s["z"] is not None else None
    gate = s["z"] * e if e is not None else torch.ones_like(s["y"])
    if c["mode"] == "fwd":
        rp = rn = h = None
        n = s["y"]
        if "p" in parts:
            rp = torch.rsqrt(torch.einsum("...d,...d->...", n, n) / D + EPS)
            n = wp * n * rp.unsqueeze(-1)
        x = sc * gate * n + (s["r"] if s["r"] is not None else 0)
        if "n" in parts:
            rn = torch.rsqrt(torch.einsum("...d,...d->...", x, x) / D + EPS)
            h = wn * x * rn.unsqueeze(-1)
        return dict(x=x, h=h, rstd_post=rp, rstd_pre=rn)

    def through(g, x, r):
        """The Jacobian r (I - x x' r^2 / D) of x r applied to g."""
        r = r.unsqueeze(-1)
        return r * g - x * r ** 3 * torch.einsum("...d,...d->...", x, g).unsqueeze(-1) / D

    flat = lambda t: t.reshape(-1, D)                                         # noqa: E731
    total, dpre = s["dx"], None
    if "n" in parts:
        dpre = torch.einsum("rd,rd->d", flat(s["dh"]), flat(s["x"] * s["rstd_pre"].unsqueeze(-1)))
        total = total + through(s["dh"] * wn, s["x"], s["rstd_pre"])
    yh = s["y"] * s["rstd_post"].unsqueeze(-1) if "p" in parts else s["y"]
    dyh = total * sc * gate * wp
    return dict(dy=through(dyh, s["y"], s["rstd_post"]) if "p" in parts else dyh,
                dresidual=total if "r" in parts else None,
                dgate=total * sc * wp * yh * (e + gate * (1 - e)) if e is not None else None,
                dpost=torch.einsum("rd,rd->d", flat(total * sc * gate), flat(yh)) if "p" in parts else None,
                dscale=torch.einsum("rd,rd->d", flat(total * gate), flat(wp * yh)) if "s" in parts else None,
                dpre=dpre)


def _exact_ffn(s, c):
    def activation(g):
        """The activation and its slope, from tanh and from the logistic function."""
        if c["act"] == "silu":
            e = torch.sigmoid(g)
            return g * e, e * (1 + g * (1 - e))
        inner = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
        t = torch.tanh(inner)
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)

    if c["mode"] != "bwd":
        g, u = torch.einsum("md,fd->mf", s["x"], s["w_gate"]), torch.einsum("md,fd->mf", s["x"], s["w_up"])
        y = torch.einsum("mf,df->md", activation(g)[0] * u, s["w_down"])
        keep = c["mode"] == "save"
        return dict(y=y, gate=g if keep else None, up=u if keep else None)
    a, slope = activation(s["gate"])
    dw_down = torch.einsum("md,mf->df", s["dy"], a * s["up"])
    dh = torch.einsum("md,df->mf", s["dy"], s["w_down"])
    dg, du = dh * s["up"] * slope, dh * a
    return dict(dx=torch.einsum("mf,fd->md", dg, s["w_gate"]) + torch.einsum("mf,fd->md", du, s["w_up"]),
                dw_gate=torch.einsum("mf,md->fd", dg, s["x"]), dw_up=torch.einsum("mf,md->fd", du, s["x"]), dw_down=dw_down)
