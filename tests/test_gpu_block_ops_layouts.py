"""Layouts and calls of the block operators beside the usual ones: heads before tokens, rows
further apart than 32 bits count, a workspace that captured graphs share.  The same bits as
from contiguous copies, from rows of the same alignment near to one another (rows of odd
alignment are summed in another order than vectors), or from calls alone."""
import pytest
import torch

import chunked_prefill_gdn_gb300 as gdn
from chunked_prefill_gdn_gb300 import build as gdn_build

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def lib():
    gdn_build.build()
    return gdn.load_library()


def equal(got, want):
    for a, b in zip(got, want):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,T,D", [(5, 700, 128), (3, 37, 33), (4, 50, 96), (2, 9, 9001), (7, 1, 64), (1, 7, 64)])
def test_heads_before_tokens(H, T, D, dtype):
    """[T, H, D] views of [H, T, D] memory: the outer rows are closer together than the inner ones."""
    g = torch.Generator(device="cuda").manual_seed(H * T + D)
    n = lambda: torch.randn(H, T, D, generator=g, device="cuda").to(TORCH[dtype])   # noqa: E731
    w = 1 + 0.2 * torch.randn(D, generator=g, device="cuda")
    y, r, z, dx, dh = (n().transpose(0, 1) for _ in range(5))
    z = z.contiguous()          # and one input in the other order
    args = dict(gate=z, post_weight=w, scale=w, pre_weight=w)
    got = gdn.block_norm_fwd(y, r, **args)
    flat = lambda t: t.contiguous()   # noqa: E731
    want = gdn.block_norm_fwd(flat(y), flat(r), **args)
    equal(got, want)
    x, _, rp, rn = want
    xt = x.transpose(0, 1).contiguous().transpose(0, 1)
    equal(gdn.block_norm_bwd(dx, dh, y, xt, rp, rn, **args), gdn.block_norm_bwd(flat(dx), flat(dh), flat(y), x, rp, rn, **args))


def far(t, apart):
    """The rows of t `apart` elements from one another."""
    buf = torch.empty((t.shape[0] - 1) * apart + t.shape[1], dtype=t.dtype, device=t.device)
    view = buf.as_strided(t.shape, (apart, 1))
    view.copy_(t)
    return view


@pytest.mark.parametrize("apart", [2 ** 31 + 8, 2 ** 31 + 9])
def test_rows_far_apart(apart):
    g = torch.Generator(device="cuda").manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
    near = lambda t: far(t, (t.shape[1] // 16 + 1) * 16 + apart % 16)   # noqa: E731
    for rows, D in ((3, 136), (3, 9001)):
        y, w = near(n(rows, D)), 1 + 0.2 * torch.randn(D, generator=g, device="cuda")
        f = far(y, apart)
        x, h, rp, rn = want = gdn.block_norm_fwd(y, y, y, w, w, w)
        equal(gdn.block_norm_fwd(f, f, f, w, w, w), want)
        equal(gdn.block_norm_bwd(f, f, f, x, rp, rn, f, w, w, w), gdn.block_norm_bwd(y, y, y, x, rp, rn, y, w, w, w))
        del f
    D, F, O = 136, 72, 40
    w = [n(F, D) / 12, n(F, D) / 12, n(O, F) / 8]
    for M in (3, 18):          # a few tokens, tiles
        x, dy = near(n(M, D)), n(M, O)
        if M > 3:
            fx = far(x, (2 ** 32 + apart) // M // 8 * 8 + apart % 8)    # the last rows past 2^31
        else:
            fx = far(x, apart)
        y, gate, up = gdn.gated_ffn_fwd(x, *w, save=True, check=True)
        equal(gdn.gated_ffn_fwd(fx, *w, save=True, check=True), (y, gate, up))
        want = gdn.gated_ffn_bwd(dy, x, *w, gate, up, check=True)
        equal(gdn.gated_ffn_bwd(dy, fx, *w, gate, up, check=True), want)
        del fx


def test_graphs_that_share_a_workspace():
    """Two captured calls with one workspace, replayed in turn on one stream."""
    g = torch.Generator(device="cuda").manual_seed(9)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
    D, F = 130, 264
    w = [n(F, D) / 12, n(F, D) / 12, n(D, F) / 16]
    xs = [n(300, D), n(70, D)]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    want = []
    for x in xs:
        y, gate, up = gdn.gated_ffn_fwd(x, *w, save=True)
        want.append((y, *gdn.gated_ffn_bwd(y, x, *w, gate, up)))
    graphs, out = [], []
    for x in xs:
        def step():
            y, gate, up = gdn.gated_ffn_fwd(x, *w, save=True, workspace=ws)
            return (y, *gdn.gated_ffn_bwd(y, x, *w, gate, up, workspace=ws))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            out.append(step())
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    for got, alone in zip(out, want):
        equal(got, alone)


def test_beside_the_recurrence_on_another_stream():
    """The feed-forward block's and the recurrence's tensor-core kernels at the same time: the
    bits of each alone."""
    g = torch.Generator(device="cuda").manual_seed(2)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    q, k, v = (torch.nn.functional.normalize(n(2, 2000, 16, 128), dim=-1).bfloat16() for _ in range(3))
    decay, beta = -0.1 * torch.rand(2, 2000, 16, generator=g, device="cuda"), torch.rand(2, 2000, 16, generator=g, device="cuda")
    cases = []
    for M, D, F in ((1500, 512, 2048), (100, 1024, 4096), (40, 512, 512)):
        x, w = n(M, D).bfloat16(), [(n(*s) / s[1] ** 0.5).bfloat16() for s in ((F, D), (F, D), (D, F))]
        cases.append((x, w))

    def recurrence(stream=None):
        return gdn.chunk_fwd(q, k, v, decay, beta, stream=stream)

    def block(stream=None):
        out = []
        for x, w in cases:
            y, gate, up = gdn.gated_ffn_fwd(x, *w, save=True, stream=stream)
            out += [y, *gdn.gated_ffn_bwd(y, x, *w, gate, up, stream=stream)]
        return out

    want = recurrence(), block()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(10):
        for i, (call, s) in enumerate(zip((recurrence, block), streams)):
            with torch.cuda.stream(s):
                got[i].append(call())
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for i in range(2):
        for again in got[i]:
            equal(again, want[i])
