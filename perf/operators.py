"""The layer operators around the gated delta rule: what is timed, on which
inputs, their plain forms and their values in 64 bits.

Operators (see include/gdn.h for the definitions):
  layer_norm        forward and backward (with the weight and bias gradients)
  causal_conv       the short depthwise convolution: prompts, backward, one token
  selective_scan    the diagonal selective state space scan: prompts, backward, one token
  gated_delta_step  one token of the gated delta rule on a cached state

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


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the norm in front of the layer workload's projections (4 x 8192 tokens, 32 heads x 128)
        dict(name="norm fwd layer", op="norm", mode="fwd", rows=32768, D=4096, dtype="bf16"),
        # its backward pass in training
        dict(name="norm bwd layer", op="norm", mode="bwd", rows=32768, D=4096, dtype="bf16"),
        # one token of 16 sequences being served: latency
        dict(name="norm fwd tokens", op="norm", mode="fwd", rows=16, D=4096, dtype="bf16"),
        # q, k and v (16 heads x 3 x 128 channels) of packed prompts of mixed lengths, from states
        dict(name="conv fwd packed", op="conv", mode="fwd", B=1, T=65536, seqs=64, D=6144, W=4, dtype="bf16"),
        # the same layer in training, one batch of equal sequences of an odd length
        dict(name="conv bwd train", op="conv", mode="bwd", B=4, T=4095, seqs=0, D=4096, W=4, dtype="bf16"),
        # one token of 64 sequences, 32 heads x 3 x 128 channels: latency
        dict(name="conv step", op="conv", mode="step", B=64, T=1, seqs=0, D=12288, W=4, dtype="bf16"),
        # a batch of prompts: enough (sequence, channel) pairs to fill the GPU
        dict(name="scan fwd batch", op="scan", mode="fwd", B=8, T=1024, seqs=0, D=4096, N=16, dtype="bf16"),
        # one long prompt with few channels: the time axis has to be split
        dict(name="scan fwd long", op="scan", mode="fwd", B=1, T=32768, seqs=0, D=1024, N=16, dtype="bf16"),
        # training on packed sequences
        dict(name="scan bwd packed", op="scan", mode="bwd", B=1, T=4099, seqs=5, D=2048, N=16, dtype="bf16"),
        # one token of 32 sequences
        dict(name="scan step", op="scan", mode="step", B=32, T=1, seqs=0, D=4096, N=16, dtype="bf16"),
        # one token of one sequence (32 heads x 128): latency
        dict(name="delta step one", op="delta", mode="step", B=1, H=32, dk=128, dv=128, dtype="bf16"),
        # one token of a full serving batch
        dict(name="delta step batch", op="delta", mode="step", B=128, H=32, dk=128, dv=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng: random.Random):
    op = rng.choice(["norm", "conv", "scan", "delta"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        D = _log(rng, 33, 8192)
        rows = _log(rng, 1, min(32768, 2 ** 26 // D))
        return dict(op=op, mode=rng.choice(["fwd", "bwd"]), rows=rows, D=D, dtype=dtype)
    if op == "delta":
        return dict(op=op, mode="step", B=_log(rng, 1, 100), H=rng.randint(1, 40), dk=rng.choice([32, 64, 128]),
                    dv=rng.choice([32, 64, 128]), dtype=dtype)
    mode = rng.choice(["fwd", "bwd", "step"])
    D = rng.choice([1, 8, 8]) * _log(rng, 12, 512 if op == "conv" else 256)
    seqs = 0 if mode == "step" else rng.choice([0, 0, rng.randint(1, 9)])
    N = rng.choice([8, 16, 16, 24])
    if mode == "step":
        B, T = _log(rng, 1, 256), 1
    else:
        B = 1 if seqs else rng.choice([1, 1, 2, 3])
        most = 2 ** 26 if op == "conv" else 2 ** (29 if mode == "fwd" else 27) // N
        T = min(_log(rng, 1, 16384), most // (B * D))
    if op == "conv":
        return dict(op=op, mode=mode, B=B, T=T, seqs=seqs, D=D, W=rng.choice([2, 3, 4, 4]), dtype=dtype)
    return dict(op=op, mode=mode, B=B, T=T, seqs=seqs, D=D, N=N, dtype=dtype)


# ----------------------------------------------------------------- the inputs

def _cuts(case, seed):
    """Cumulative lengths of the packed sequences (one of them has a single
    token where there is room), as the packer of a batch would give them."""
    r = random.Random(seed * 7919 + 17)
    T, n = case["T"], case["seqs"]
    at = sorted(r.randint(0, T) for _ in range(n - 1))
    cu = [0] + at + [T]
    if n > 1 and cu[1] + 1 <= cu[2]:
        cu[1] = min(cu[1], 1)
    return torch.tensor(cu, dtype=torch.int32, device=DEVICE)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(int(seed))
    dt = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, to=dt):
        return torch.randn(*shape, generator=gen, device=DEVICE).mul_(std).to(to)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=gen, device=DEVICE) * (hi - lo) + lo

    s = dict(case=dict(case))
    op, mode = case["op"], case["mode"]
    if op == "norm":
        rows, D = case["rows"], case["D"]
        s["x"] = (torch.randn(rows, D, generator=gen, device=DEVICE) * uniform(0.3, 3.0, rows, 1) + uniform(-1, 1, rows, 1)).to(dt)
        s["w"] = 1.0 + normal(D, std=0.2, to=torch.float32)
        s["b"] = normal(D, std=0.1, to=torch.float32)
        if mode == "bwd":
            s["dy"] = normal(rows, D)
            x = s["x"].float()
            s["mean"] = x.mean(-1)
            s["rstd"] = 1.0 / torch.sqrt((x - s["mean"][:, None]).square().mean(-1) + 1e-5)
        return s
    if op == "delta":
        B, H, dk, dv = (case[k] for k in ("B", "H", "dk", "dv"))
        q, k = normal(B, H, dk, to=torch.float32), normal(B, H, dk, to=torch.float32)
        s["q"] = (q / q.norm(dim=-1, keepdim=True)).to(dt)
        s["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dt)
        s["v"] = normal(B, H, dv)
        s["beta"] = torch.sigmoid(normal(B, H, to=torch.float32))
        s["g"] = -torch.exp(uniform(-4, -1, H)) * torch.log1p(torch.exp(normal(B, H, to=torch.float32)))
        s["state"] = normal(B, H, dk, dv, std=0.1, to=torch.float32)
        return s
    B, T, D = case["B"], case["T"], case["D"]
    s["cu"] = _cuts(case, seed) if case["seqs"] else None
    n = case["seqs"] or B
    if op == "conv":
        W = case["W"]
        s["w"] = normal(D, W, std=1.0 / W ** 0.5)
        s["b"] = normal(D, std=0.1)
        s["x"] = normal(B, D) if mode == "step" else normal(B, T, D)
        s["state"] = normal(n, W - 1, D)
        if mode == "bwd":
            s["dy"] = normal(B, T, D)
        return s
    N = case["N"]
    lead = (B,) if mode == "step" else (B, T)
    xz = normal(*lead, 2 * D)                       # one projection holds x and the gate, as in a model
    s["x"], s["z"] = xz[..., :D], xz[..., D:]
    s["dt"] = normal(*lead, D, std=0.5)
    bc = normal(*lead, 2 * N)                       # and another B and C
    s["B"], s["C"] = bc[..., :N], bc[..., N:]
    s["A"] = -torch.arange(1, N + 1, device=DEVICE, dtype=torch.float32) * torch.exp(normal(D, N, std=0.1, to=torch.float32))
    s["D"] = 1.0 + normal(D, std=0.1, to=torch.float32)
    step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), D))
    s["bias"] = step + torch.log(-torch.expm1(-step))         # softplus(bias) = step
    s["state"] = normal(n, D, N, std=0.3, to=torch.float32)
    if mode == "bwd":
        s["dy"] = normal(B, T, D)
        s["d_final"] = normal(n, D, N, std=0.1, to=torch.float32)
    return s


# -------------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import chunked_prefill_gdn_gb300 as gdn
    c = s["case"]
    op, mode = c["op"], c["mode"]
    if op == "norm" and mode == "fwd":
        y, mean, rstd = gdn.layer_norm_fwd(s["x"], s["w"], s["b"], eps=1e-5)
        return dict(y=y, mean=mean, rstd=rstd)
    if op == "norm":
        dx, dw, db = gdn.layer_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
        return dict(dx=dx, dw=dw, db=db)
    if op == "conv" and mode == "fwd":
        y, state = gdn.causal_conv_fwd(s["x"], s["w"], s["b"], initial_state=s["state"], cu_seqlens=s["cu"],
                                       activation="silu", output_final_state=True)
        return dict(y=y, state=state)
    if op == "conv" and mode == "bwd":
        dx, dw, db, ds = gdn.causal_conv_bwd(s["dy"], s["x"], s["w"], s["b"], initial_state=s["state"],
                                             cu_seqlens=s["cu"], activation="silu")
        return dict(dx=dx, dw=dw, db=db, dstate=ds)
    if op == "conv":
        y = gdn.causal_conv_step(s["x"], s["state"], s["w"], s["b"], activation="silu")
        return dict(y=y, state=s["state"])
    if op == "scan" and mode == "fwd":
        y, state = gdn.selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
                                          dt_bias=s["bias"], dt_softplus=True, initial_state=s["state"],
                                          cu_seqlens=s["cu"])
        return dict(y=y, state=state)
    if op == "scan" and mode == "bwd":
        g = gdn.selective_scan_bwd(s["dy"], s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
                                   dt_bias=s["bias"], dt_softplus=True, initial_state=s["state"],
                                   cu_seqlens=s["cu"], d_final_state=s["d_final"])
        return dict(zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dstate"), g))
    if op == "scan":
        y = gdn.selective_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], D=s["D"], z=s["z"],
                                    dt_bias=s["bias"], dt_softplus=True)
        return dict(y=y, state=s["state"])
    o = gdn.gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"])
    return dict(o=o, state=s["state"])


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _softplus(x):
    return torch.where(x > 20.0, x, torch.log1p(torch.exp(torch.minimum(x, torch.full_like(x, 20.0)))))


def _places(cu, B, T):
    """Per flattened token: its sequence and its position in it; per sequence:
    its first token and length."""
    if cu is None:
        cu = torch.arange(0, (B + 1) * T, T, device=DEVICE)
    cu = cu.long()
    t = torch.arange(B * T, device=DEVICE)
    seq = torch.searchsorted(cu[1:], t, right=True)
    return seq, t - cu[seq], cu[:-1], cu[1:] - cu[:-1]


def _run_plain(s):
    c = s["case"]
    return {"norm": _plain_norm, "conv": _plain_conv, "scan": _plain_scan, "delta": _plain_delta}[c["op"]](s, c)


def _plain_norm(s, c):
    x = s["x"].float()
    if c["mode"] == "fwd":
        mean = x.mean(-1)
        xc = x - mean[:, None]
        rstd = 1.0 / torch.sqrt(xc.square().mean(-1) + 1e-5)
        return dict(y=(xc * rstd[:, None] * s["w"] + s["b"]).to(s["x"].dtype), mean=mean, rstd=rstd)
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    gy = dy * s["w"]
    dx = rstd * (gy - gy.mean(-1, keepdim=True) - xh * (gy * xh).mean(-1, keepdim=True))
    return dict(dx=dx.to(s["x"].dtype), dw=(dy * xh).sum(0), db=dy.sum(0))


def _plain_conv(s, c):
    W, D, dt = c["W"], c["D"], s["x"].dtype
    w, b = s["w"].float(), s["b"].float()
    if c["mode"] == "step":
        win = torch.cat([s["state"], s["x"][:, None]], dim=1)             # [B, W, D]
        u = (win.float() * w.t()).sum(1) + b
        s["state"].copy_(win[:, 1:])
        return dict(y=(u * _sigmoid(u)).to(dt), state=s["state"])
    seq, pos, first, length = _places(s["cu"], c["B"], c["T"])
    Tt = seq.numel()
    rows = torch.cat([s["x"].reshape(Tt, D), s["state"].reshape(-1, D)])  # tokens, then the states' rows
    t = torch.arange(Tt, device=DEVICE)

    def back(j):                                                          # the row j tokens earlier
        return torch.where(pos >= j, t - j, Tt + seq * (W - 1) + (W - 1) + pos - j)

    u = b + sum(w[:, W - 1 - j] * rows[back(j)].float() for j in range(W))
    if c["mode"] == "fwd":
        p = length[:, None] - (W - 1) + torch.arange(W - 1, device=DEVICE)
        n = torch.arange(length.numel(), device=DEVICE)[:, None]
        last = torch.where(p >= 0, first[:, None] + p, Tt + n * (W - 1) + (W - 1) + p)
        return dict(y=(u * _sigmoid(u)).to(dt).reshape(s["x"].shape), state=rows[last])
    sg = _sigmoid(u)
    du = s["dy"].reshape(Tt, D).float() * sg * (1.0 + u * (1.0 - sg))
    d = torch.zeros(rows.shape, device=DEVICE)
    dw = torch.empty(D, W, device=DEVICE)
    for j in range(W):
        d.index_add_(0, back(j), w[:, W - 1 - j] * du)
        dw[:, W - 1 - j] = (du * rows[back(j)].float()).sum(0)
    return dict(dx=d[:Tt].to(dt).reshape(s["x"].shape), dw=dw, db=du.sum(0), dstate=d[Tt:].to(dt).reshape(s["state"].shape))


def _doubling(a, b, span):
    """h_t = a_t h_{t-1} + b_t along dim 0, by doubling the reach of each step."""
    reach = 1
    while reach < span:
        b = torch.cat([b[:reach], b[reach:] + a[reach:] * b[:-reach]])
        a = torch.cat([a[:reach], a[reach:] * a[:-reach]])
        reach *= 2
    return b


def _plain_scan(s, c):
    D, N, dt = c["D"], c["N"], s["x"].dtype
    flat = lambda t, n: t.reshape(-1, n).float()                          # noqa: E731
    x, z = flat(s["x"], D), flat(s["z"], D)
    pre = flat(s["dt"], D) + s["bias"]
    step = _softplus(pre)
    Bm, Cm = flat(s["B"], N)[:, None, :], flat(s["C"], N)[:, None, :]     # [T, 1, N]
    sz = _sigmoid(z)
    if c["mode"] == "step":
        h = torch.exp(step[..., None] * s["A"]) * s["state"] + (step * x)[..., None] * Bm
        s["state"].copy_(h)
        y = (h * Cm).sum(-1) + s["D"] * x
        return dict(y=(y * z * sz).to(dt), state=s["state"])
    seq, pos, first, length = _places(s["cu"], c["B"], c["T"])
    Tt = seq.numel()
    some = length > 0
    starts, ends = first[some], (first + length - 1)[some]
    a = torch.exp(step[..., None] * s["A"])                               # [T, D, N]
    b = (step * x)[..., None] * Bm
    a0 = a[starts]
    b[starts] += a0 * s["state"][some]
    cut = a.clone()
    cut[starts] = 0.0                                                     # nothing crosses a sequence's start
    h = _doubling(cut, b, c["T"])
    y = (h * Cm).sum(-1) + s["D"] * x
    if c["mode"] == "fwd":
        final = s["state"].clone()
        final[some] = h[ends]
        return dict(y=(y * z * sz).to(dt).reshape(s["x"].shape), state=final)
    do = flat(s["dy"], D)
    dy = do * z * sz
    dz = do * y * sz * (1.0 + z * (1.0 - sz))
    after = torch.cat([cut[1:], torch.zeros_like(cut[:1])])               # a of the next token of the sequence
    r = dy[..., None] * Cm
    r[ends] += s["d_final"][some]
    dh = _doubling(after.flip(0), r.flip(0), c["T"]).flip(0)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[starts] = s["state"][some]
    da = dh * before * a                                                  # d of the exponent
    dB, dC = (dh * (step * x)[..., None]).sum(1), (h * dy[..., None]).sum(1)
    du = (dh * Bm).sum(-1)
    dstep = (da * s["A"]).sum(-1) + du * x
    dpre = dstep * _sigmoid(pre)
    dstate = s["d_final"].clone()
    dstate[some] = dh[starts] * a0
    like = s["x"].shape
    return dict(dx=(du * step + s["D"] * dy).to(dt).reshape(like), ddt=dpre.to(dt).reshape(like),
                dA=(da * step[..., None]).sum(0), dB=dB.to(dt).reshape(s["B"].shape), dC=dC.to(dt).reshape(s["C"].shape),
                dD=(dy * x).sum(0), dz=dz.to(dt).reshape(like), dbias=dpre.sum(0), dstate=dstate)


def _plain_delta(s, c):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    S = s["state"] * torch.exp(s["g"])[..., None, None]
    u = s["beta"][..., None] * (v - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    s["state"].copy_(S)
    o = c["dk"] ** -0.5 * (S * q[..., None]).sum(-2)
    return dict(o=o.to(s["v"].dtype), state=s["state"])


# ------------------------------------------------------- what a pass cannot avoid

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op, mode = case["op"], case["mode"]
    if op == "norm":
        n = case["rows"] * case["D"]
        if mode == "fwd":
            return dict(bytes=2 * n * e + 8 * case["rows"] + 8 * case["D"], flops=8 * n)
        return dict(bytes=3 * n * e + 8 * case["rows"] + 12 * case["D"], flops=14 * n)
    if op == "delta":
        n, d = case["B"] * case["H"], case["dk"] * case["dv"]
        return dict(bytes=n * (8 * d + e * (2 * case["dk"] + 2 * case["dv"]) + 8), flops=n * 7 * d)
    B, T, D = case["B"], case["T"], case["D"]
    n, seqs = B * T * D, case["seqs"] or B
    if op == "conv":
        W = case["W"]
        side = seqs * (W - 1) * D * e
        if mode in ("fwd", "step"):
            return dict(bytes=2 * n * e + 2 * side + (W + 1) * D * e, flops=n * (2 * W + 5))
        return dict(bytes=3 * n * e + 2 * side + (W + 1) * D * (e + 4), flops=n * (6 * W + 10))
    N = case["N"]
    state, bc, par = seqs * D * N * 4, B * T * N * e, D * N * 4 + 8 * D
    if mode in ("fwd", "step"):
        return dict(bytes=4 * n * e + 2 * bc + 2 * state + par, flops=n * (7 * N + 12))
    return dict(bytes=7 * n * e + 4 * bc + 3 * state + 2 * par, flops=n * (18 * N + 30))


# -------------------------------------------------------- the values in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    return {"norm": _exact_norm, "conv": _exact_conv, "scan": _exact_scan, "delta": _exact_delta}[case["op"]](s, case)


def _spans(s, c):
    """(batch row, first token, last token + 1) of each sequence."""
    if s["cu"] is None:
        return [(b, 0, c["T"]) for b in range(c["B"])]
    cu = s["cu"].tolist()
    return [(0, cu[i], cu[i + 1]) for i in range(len(cu) - 1)]


def _exact_norm(s, c):
    x, D = s["x"], c["D"]
    xc = x - x.sum(1, keepdim=True) / D
    sd = torch.sqrt((xc * xc).sum(1, keepdim=True) / D + 1e-5)
    xh = xc / sd
    if c["mode"] == "fwd":
        return dict(y=xh * s["w"] + s["b"], mean=x.sum(1) / D, rstd=1.0 / sd[:, 0])
    g = s["dy"] * s["w"]
    # the Jacobian (I - 11'/D - xh xh'/D) / sd applied to g
    dx = (g - g.sum(1, keepdim=True) / D - xh * (g * xh).sum(1, keepdim=True) / D) / sd
    return dict(dx=dx, dw=torch.einsum("rd,rd->d", s["dy"], xh), db=s["dy"].sum(0))


def _exact_conv(s, c):
    W = c["W"]
    if c["mode"] == "step":
        win = torch.cat([s["state"], s["x"][:, None]], 1)
        u = torch.einsum("bwd,dw->bd", win, s["w"]) + s["b"]
        return dict(y=u / (1 + torch.exp(-u)), state=win[:, 1:])
    bwd = c["mode"] == "bwd"
    out, last = torch.empty_like(s["x"]), torch.empty_like(s["state"])
    dw, db, dst = torch.zeros_like(s["w"]), torch.zeros_like(s["b"]), torch.empty_like(s["state"])
    for n, (r, t0, t1) in enumerate(_spans(s, c)):
        full = torch.cat([s["state"][n], s["x"][r, t0:t1]])              # [W - 1 + L, D]
        last[n] = full[full.shape[0] - (W - 1):]
        taps = full.unfold(0, W, 1)                                       # [L, D, W]
        u = (taps * s["w"]).sum(-1) + s["b"]
        e = 1 / (1 + torch.exp(-u))
        if not bwd:
            out[r, t0:t1] = u * e
            continue
        du = s["dy"][r, t0:t1] * (e + u * e * (1 - e))
        dfull = torch.zeros_like(full)
        for i in range(W):
            dfull[i:i + t1 - t0] += du * s["w"][:, i]
        dw += (taps * du[..., None]).sum(0)
        db += du.sum(0)
        out[r, t0:t1], dst[n] = dfull[W - 1:], dfull[:W - 1]
    return dict(dx=out, dw=dw, db=db, dstate=dst) if bwd else dict(y=out, state=last)


def _exact_scan(s, c):
    D, A = c["D"], s["A"]
    pre = s["dt"] + s["bias"]
    step = torch.nn.functional.softplus(pre, threshold=100.0)
    sig = 1 / (1 + torch.exp(-s["z"]))
    if c["mode"] == "step":
        h = torch.exp(step[:, :, None] * A) * s["state"] + (step * s["x"])[:, :, None] * s["B"][:, None]
        y = torch.einsum("bdn,bn->bd", h, s["C"]) + s["D"] * s["x"]
        return dict(y=y * s["z"] * sig, state=h)
    bwd = c["mode"] == "bwd"
    y = torch.empty(s["x"].shape, dtype=torch.float64, device=DEVICE)
    final = s["state"].clone()
    names = ("dx", "ddt", "dz")
    g = {k: torch.empty_like(y) for k in names} if bwd else {}
    if bwd:
        g |= dict(dB=torch.empty(s["B"].shape, dtype=torch.float64, device=DEVICE),
                  dC=torch.empty(s["C"].shape, dtype=torch.float64, device=DEVICE), dA=torch.zeros_like(A), dstate=s["d_final"].clone())
    for n, (r, t0, t1) in enumerate(_spans(s, c)):
        h, kept = s["state"][n], []
        for t in range(t0, t1):
            kept.append(h) if bwd else None
            h = torch.exp(step[r, t][:, None] * A) * h + torch.outer(step[r, t] * s["x"][r, t], s["B"][r, t])
            y[r, t] = h @ s["C"][r, t]
        final[n] = h
        if not bwd:
            continue
        dh = s["d_final"][n]
        for t in range(t1 - 1, t0 - 1, -1):
            gate = s["z"][r, t] * sig[r, t]
            ypre = y[r, t] + s["D"] * s["x"][r, t]
            dy = s["dy"][r, t] * gate
            g["dz"][r, t] = s["dy"][r, t] * ypre * (sig[r, t] + gate * (1 - sig[r, t]))
            p = kept.pop()
            a = torch.exp(step[r, t][:, None] * A)
            g["dC"][r, t] = dy @ h
            dh = dh + torch.outer(dy, s["C"][r, t])
            g["dB"][r, t] = (step[r, t] * s["x"][r, t]) @ dh
            du = dh @ s["B"][r, t]
            q = dh * p * a
            g["dA"] += q * step[r, t][:, None]
            g["ddt"][r, t] = ((q * A).sum(1) + du * s["x"][r, t]) / (1 + torch.exp(-pre[r, t]))
            g["dx"][r, t] = du * step[r, t] + s["D"] * dy
            h, dh = p, dh * a
        g["dstate"][n] = dh
    if not bwd:
        return dict(y=(y + s["D"] * s["x"]) * s["z"] * sig, state=final)
    dy = s["dy"] * s["z"] * sig
    return dict(g, dD=(dy * s["x"]).reshape(-1, D).sum(0), dbias=g["ddt"].reshape(-1, D).sum(0))


def _exact_delta(s, c):
    S = torch.exp(s["g"])[..., None, None] * s["state"]
    k, q = s["k"], s["q"]
    u = s["beta"][..., None] * (s["v"] - torch.einsum("bhj,bhji->bhi", k, S))
    S = S + torch.einsum("bhj,bhi->bhji", k, u)
    return dict(o=torch.einsum("bhj,bhji->bhi", q, S) / c["dk"] ** 0.5, state=S)
