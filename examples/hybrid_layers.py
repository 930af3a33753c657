"""Two linear-attention layers, of the delta rule and of the selective scan, in
the three ways they are used: a packed batch of prompts, one token at a time on
the cached states, and a training step.

    python examples/hybrid_layers.py            # needs the built library and a GPU

Each layer is norm -> projection -> short causal convolution -> recurrence ->
projection, added to its input.  The weights are random; what is checked is that
the single tokens continue the prompts as one longer prompt would, and that a
training step lowers its loss.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import chunked_prefill_gdn_gb300 as gdn  # noqa: E402


class Layer:
    """What both layers share: the norm, the convolution and their caches."""

    def __init__(self, model, conv_channels, gen, width=4):
        dev = "cuda"
        self.model, self.width = model, width
        self.p = dict(norm_w=torch.ones(model, device=dev), norm_b=torch.zeros(model, device=dev),
                      conv_w=torch.randn(conv_channels, width, generator=gen).to(dev, torch.bfloat16) / width ** 0.5,
                      conv_b=torch.zeros(conv_channels, dtype=torch.bfloat16, device=dev))
        self.conv_channels = conv_channels

    def matrix(self, rows, cols, gen):
        return (torch.randn(rows, cols, generator=gen) / rows ** 0.5).to("cuda", torch.bfloat16)

    def parameters(self):
        return list(self.p.values())

    def norm(self, x):
        return gdn.layer_norm(x, self.p["norm_w"], self.p["norm_b"])


class DeltaLayer(Layer):
    def __init__(self, model, heads, d, gen):
        super().__init__(model, 3 * heads * d, gen)
        self.heads, self.d = heads, d
        self.p["w_qkv"] = self.matrix(model, 3 * heads * d, gen)
        self.p["w_gate"] = self.matrix(model, 2 * heads, gen)
        self.p["w_out"] = self.matrix(heads * d, model, gen)

    def new_state(self, slots):
        return dict(conv=torch.zeros(slots, self.width - 1, self.conv_channels, dtype=torch.bfloat16, device="cuda"),
                    s=torch.zeros(slots, self.heads, self.d, self.d, device="cuda"))

    def split(self, u):
        return u.view(*u.shape[:-1], 3, self.heads, self.d).unbind(-3)

    def gates(self, h):
        a, b = (h @ self.p["w_gate"]).float().chunk(2, -1)
        return -torch.nn.functional.softplus(a), torch.sigmoid(b)

    def prompt(self, x, cu):
        """x [1, T, model]; returns the output and the states of the sequences."""
        h = self.norm(x)
        u, conv = gdn.causal_conv(h @ self.p["w_qkv"], self.p["conv_w"], self.p["conv_b"], cu_seqlens=cu,
                                  output_final_state=True)
        o, s = gdn.chunk_gated_delta_rule(*self.split(u), *self.gates(h), output_final_state=True, cu_seqlens=cu,
                                          use_qk_l2norm_in_kernel=True)
        return x + o.flatten(-2) @ self.p["w_out"], dict(conv=conv, s=s)

    def token(self, x, state, slots):
        """x [N, model], one token of the sequences whose states are in `slots`."""
        h = self.norm(x)
        u = gdn.causal_conv_step(h @ self.p["w_qkv"], state["conv"], self.p["conv_w"], self.p["conv_b"],
                                 state_indices=slots)
        o = gdn.gated_delta_step(*self.split(u), *self.gates(h), state["s"], use_qk_l2norm_in_kernel=True,
                                 state_indices=slots)
        return x + o.flatten(-2) @ self.p["w_out"]


class ScanLayer(Layer):
    def __init__(self, model, channels, n, gen, rank=16):
        super().__init__(model, channels, gen)
        self.channels, self.n, self.rank = channels, n, rank
        dev = "cuda"
        self.p["w_in"] = self.matrix(model, 2 * channels, gen)
        self.p["w_bc"] = self.matrix(channels, rank + 2 * n, gen)
        self.p["w_dt"] = self.matrix(rank, channels, gen)
        self.p["w_out"] = self.matrix(channels, model, gen)
        self.p["a_log"] = torch.log(torch.arange(1, n + 1, device=dev).float()).repeat(channels, 1)
        self.p["skip"] = torch.ones(channels, device=dev)
        self.p["dt_bias"] = torch.full((channels,), -4.0, device=dev)

    def new_state(self, slots):
        return dict(conv=torch.zeros(slots, self.width - 1, self.conv_channels, dtype=torch.bfloat16, device="cuda"),
                    s=torch.zeros(slots, self.channels, self.n, device="cuda"))

    def inputs(self, u):
        """dt, B and C of the convolved rows: slices of one projection, used as they lie."""
        dbc = u @ self.p["w_bc"]
        return (dbc[..., :self.rank] @ self.p["w_dt"], -torch.exp(self.p["a_log"]),
                dbc[..., self.rank:self.rank + self.n], dbc[..., self.rank + self.n:])

    def prompt(self, x, cu):
        xz = self.norm(x) @ self.p["w_in"]
        u, conv = gdn.causal_conv(xz[..., :self.channels], self.p["conv_w"], self.p["conv_b"], cu_seqlens=cu,
                                  output_final_state=True)
        y, s = gdn.selective_scan(u, *self.inputs(u), self.p["skip"], xz[..., self.channels:], self.p["dt_bias"],
                                  output_final_state=True, cu_seqlens=cu)
        return x + y @ self.p["w_out"], dict(conv=conv, s=s)

    def token(self, x, state, slots):
        xz = self.norm(x) @ self.p["w_in"]
        u = gdn.causal_conv_step(xz[..., :self.channels], state["conv"], self.p["conv_w"], self.p["conv_b"],
                                 state_indices=slots)
        y = gdn.selective_scan_step(u, *self.inputs(u), state["s"], self.p["skip"], xz[..., self.channels:],
                                    self.p["dt_bias"], state_indices=slots)
        return x + y @ self.p["w_out"]


def make_model(model=256, heads=2, d=128, channels=512, n=16, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return [DeltaLayer(model, heads, d, gen), ScanLayer(model, channels, n, gen)]


@torch.no_grad()
def serve(layers, lengths=(37, 1, 150), new_tokens=4, slots=8, seed=1):
    """Prompts of the given lengths, packed, then `new_tokens` single tokens of
    each on states kept in a cache of `slots` rows; returns the outputs of the
    single tokens and those of the same tokens in one longer prompt."""
    gen = torch.Generator().manual_seed(seed)
    model = layers[0].model
    seqs = [torch.randn(n + new_tokens, model, generator=gen).to("cuda", torch.bfloat16) for n in lengths]

    def run(parts):
        x = torch.cat(parts)[None]
        cu = torch.tensor([0] + [len(p) for p in parts], device="cuda").cumsum(0).to(torch.int32)
        states = []
        for layer in layers:
            x, st = layer.prompt(x, cu)
            states.append(st)
        return x[0], cu, states

    whole, cu, _ = run(seqs)
    rows = torch.tensor(list(range(slots - 1, slots - 1 - len(seqs), -1)), dtype=torch.int32, device="cuda")
    _, _, states = run([s[:n] for s, n in zip(seqs, lengths)])
    cache = []
    for layer, st in zip(layers, states):
        c = layer.new_state(slots)
        for k in c:
            c[k][rows.long()] = st[k]
        cache.append(c)
    # one padded row, as a server fills its batch up
    index = torch.cat([rows, torch.tensor([-1], dtype=torch.int32, device="cuda")])
    got, want = [], []
    for t in range(new_tokens):
        x = torch.stack([s[n + t] for s, n in zip(seqs, lengths)] + [torch.zeros_like(seqs[0][0])])
        for layer, c in zip(layers, cache):
            x = layer.token(x, c, index)
        got.append(x[:-1])
        want.append(torch.stack([whole[int(cu[i]) + n + t] for i, n in enumerate(lengths)]))
    return torch.stack(got), torch.stack(want)


def train(layers, steps=3, lengths=(100, 29), lr=2e-3, seed=2):
    """Gradient steps on a fixed packed batch towards random targets; returns
    the losses."""
    gen = torch.Generator().manual_seed(seed)
    model, T = layers[0].model, sum(lengths)
    x = torch.randn(1, T, model, generator=gen).to("cuda", torch.bfloat16)
    target = torch.randn(1, T, model, generator=gen).to("cuda")
    cu = torch.tensor([0, *lengths], device="cuda").cumsum(0).to(torch.int32)
    params = [p for layer in layers for p in layer.parameters()]
    for p in params:
        p.requires_grad_()
    opt = torch.optim.AdamW(params, lr=lr)
    losses = []
    for _ in range(steps):
        h = x
        for layer in layers:
            h, _ = layer.prompt(h, cu)
        loss = (h.float() - target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


def main():
    layers = make_model()
    got, want = serve(layers)
    err = float((got.float() - want.float()).norm() / want.float().norm())
    print("single tokens against one longer prompt: relative difference %.2e" % err)
    losses = train(layers)
    print("training: loss " + " -> ".join("%.4f" % v for v in losses))
    return err, losses


if __name__ == "__main__":
    main()
