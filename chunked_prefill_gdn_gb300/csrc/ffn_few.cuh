// The feed-forward block's forward products for a few tokens (single-token serving):
// bound by the weights' bytes.
#pragma once

#include "elem.cuh"

namespace gdn {
namespace ffn {

constexpr int kFewBf16 = 16, kFewF32 = 32;   // at most so many tokens

struct FewArgs {
    const void *x, *w0, *w1;   // tokens; weights (up: w_gate and w_up; else w_down)
    long long x_stride, K;     // K: the length of a row of weights
    int M, rows, act;          // rows of w0 that there are (up: F; else D_out)
    int wpr;                   // one token: warps per pair of rows (set by launch_few)
    void *out;                 // up: h, else y; [M, out_ld]
    long long out_ld;
    void *gate, *up;           // up: [M, rows] or null
};

// up: h = act(x w_gate^T) (x w_up^T), else y = h w_down^T; vec: 16-byte vectors.
cudaError_t launch_few(const FewArgs &a, bool up, bool f32, bool vec, cudaStream_t s);

}  // namespace ffn
}  // namespace gdn
