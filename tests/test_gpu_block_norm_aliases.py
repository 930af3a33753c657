"""Outputs of the block norm in the memory of its inputs, as include/gdn.h allows them through
the C entry points: x or h in that of y, gate or residual, and backward dresidual or dy in that
of dx, dh or x, dgate in that of gate.  The same bits as with memory of their own, with more
rows than the grid holds: vectors, rows of odd alignment (whose 16-byte copies reach into
the neighbouring row, which another block writes), a single stage of copies, rows read
several times."""
import itertools

import pytest
import torch

import chunked_prefill_gdn_gb300 as gdn
from chunked_prefill_gdn_gb300 import build as gdn_build

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
CASES = [(20000, 33, "bf16", 0), (20001, 33, "f32", 1), (6000, 128, "bf16", 0), (6000, 128, "bf16", 1), (1500, 4096, "bf16", 0),
         (1501, 4095, "bf16", 0), (900, 4095, "f32", 1), (500, 8192, "f32", 0), (500, 8191, "f32", 0), (500, 8192, "bf16", 3),
         (400, 9008, "bf16", 0), (401, 9001, "f32", 0)]


@pytest.fixture(scope="module")
def lib():
    gdn_build.build()
    return gdn.load_library()


def pointer(t):
    return t.data_ptr() if t is not None else None


class Case:
    def __init__(self, lib, rows, D, dtype, offset):
        self.lib, self.rows, self.D, self.dtype, self.offset = lib, rows, D, dtype, offset
        g = torch.Generator(device="cuda").manual_seed(rows + D)
        self.given = {n: torch.randn(rows, D, generator=g, device="cuda").to(TORCH[dtype]) for n in ("y", "gate", "residual", "dx", "dh")}
        self.w = {n: 1 + 0.2 * torch.randn(D, generator=g, device="cuda") for n in ("post", "scale", "pre")}

    def empty(self):
        """Rows at `offset` elements from a 16-byte boundary."""
        return torch.empty(self.rows * self.D + self.offset, dtype=TORCH[self.dtype], device="cuda")[self.offset:].view(self.rows, self.D)

    def inputs(self, names):
        out = {}
        for n in names:
            out[n] = self.empty()
            out[n].copy_(self.given[n])
        return out

    def desc(self, t):
        w = [pointer(self.w[n]) for n in ("post", "scale", "pre")]
        return gdn.GdnBlockNormDesc(pointer(t["y"]), pointer(t["gate"]), *w, self.rows, 1, self.D, *[self.D] * 4, 1e-5, 1, 1, 0,
                                    0 if self.dtype == "bf16" else 1, 1)

    def forward(self, place=()):
        """place: (output, input) pairs."""
        t = self.inputs(("y", "gate", "residual"))
        out = {n: self.empty() for n in ("x", "h")}
        for o, i in place:
            out[o] = t[i]
        stats = [torch.empty(self.rows, device="cuda") for _ in range(2)]
        rc = self.lib.gdn_block_norm_fwd(self.desc(t), pointer(t["residual"]), self.D, self.D, pointer(out["x"]), pointer(out["h"]),
                                         *(pointer(s) for s in stats), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        return [out["x"], out["h"], *stats]

    def backward(self, x, rp, rn, place=()):
        t = self.inputs(("y", "gate", "dx", "dh"))
        t["x"] = self.empty()
        t["x"].copy_(x)
        out = {n: self.empty() for n in ("dy", "dresidual", "dgate")}
        for o, i in place:
            out[o] = t[i]
        params = [torch.empty(self.D, device="cuda") for _ in range(3)]
        d = self.desc(t)
        ws = torch.empty(self.lib.gdn_block_norm_bwd_workspace_size(d), dtype=torch.uint8, device="cuda")
        rc = self.lib.gdn_block_norm_bwd(d, pointer(t["dx"]), self.D, self.D, pointer(t["dh"]), self.D, self.D, pointer(t["x"]), self.D, self.D,
                                         pointer(rp), pointer(rn), pointer(out["dy"]), pointer(out["dresidual"]), pointer(out["dgate"]),
                                         *(pointer(p) for p in params), pointer(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        return [out["dy"], out["dresidual"], out["dgate"], *params]


FORWARD = [[(o, i)] for o, i in itertools.product(("x", "h"), ("y", "gate", "residual"))] + [
    [("x", "residual"), ("h", "y")], [("x", "y"), ("h", "gate")]]
BACKWARD = [[(o, i)] for o, i in itertools.product(("dresidual", "dy"), ("dx", "dh", "x"))] + [
    [("dgate", "gate")], [("dresidual", "dx"), ("dy", "dh"), ("dgate", "gate")], [("dresidual", "dh"), ("dy", "x")]]


@pytest.mark.parametrize("rows,D,dtype,offset", CASES)
def test_outputs_in_the_memory_of_inputs(lib, rows, D, dtype, offset):
    c = Case(lib, rows, D, dtype, offset)
    want = c.forward()
    assert all(torch.isfinite(t).all() for t in want)
    for place in FORWARD:
        for a, b in zip(c.forward(place), want):
            assert torch.equal(a, b), place
    x, _, rp, rn = want
    wantg = c.backward(x, rp, rn)
    assert all(torch.isfinite(t).all() for t in wantg)
    for place in BACKWARD:
        for a, b in zip(c.backward(x, rp, rn, place), wantg):
            assert torch.equal(a, b), place
