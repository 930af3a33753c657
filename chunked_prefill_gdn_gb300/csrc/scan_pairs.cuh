// What the selective scan's kernels share: softplus, the arguments, and where a
// tile of tokens lies among the sequences.
#pragma once

#include "elem.cuh"

namespace gdn {

constexpr int kTile = 16;   // tokens per tile

// log(1 + exp(x)) = max(x, 0) + log(1 + t), t = exp(-|x|) in [0, 1], with
// log(1 + t) = 2 artanh(r), r = t / (2 + t) <= 1/3: no cancellation at either
// end.  2 artanh(r) / r is a polynomial of degree 4 in r^2 (interpolated at the
// Chebyshev points of [0, 1/9], 8e-9 relative).  What is off is t: 2^-22 and the
// rounded argument of its exponential, 5e-7 relatively at x = -7 (a step of 1e-3),
// 1e-6 at -20.  About a quarter of the instructions of the library's expf and
// log1pf.
__device__ __forceinline__ F2 softplus_pair(F2 x) {
    const F2 t = exp2_pair(mul2(x & 0x7FFFFFFF7FFFFFFFull, both(-kLog2e)));
    const F2 r = mul2(t, rcp_pair(add2(t, both(2.f)))), w = mul2(r, r);
    F2 p = fma2(both(0.2815778f), w, both(0.27965158f));
    p = fma2(p, w, both(0.40024596f));
    p = fma2(p, w, both(0.6666632f));
    p = fma2(p, w, both(2.f));
    return fma2(r, p, pair(fmaxf(lo(x), 0.f), fmaxf(hi(x), 0.f)));
}
__device__ __forceinline__ float softplus_f32(float x) { return lo(softplus_pair(pair(x, 0.f))); }

struct ScanArgs {
    const void *x, *dt, *z, *Bm, *Cm, *dy;
    const float *A, *skip, *bias, *init, *d_final;
    const int32_t *cu, *slots;
    int32_t *status;
    void *out;                       // y; or dx
    float *final_state;
    void *ddt, *dz;
    float *dinit;
    // workspace: the segments' maps, [segments][D][NP] and [segments][D]
    float *hloc, *gloc, *sums;
    int32_t *flags;                  // [segments]: bit 0 a sequence starts at its first token, bit 1 at a later one
    // backward: every tile's start state and the steps before it, from a zero start
    // of its segment, [tiles][D][NP] and [tiles][D] (nothing for a segment's first)
    float *htile, *stile;
    int32_t *exact;                  // [tiles]: a sequence starts in the segment before the tile
    float *part_a, *part_v, *part_bc;   // [segments][D][NP], [segments][2][D], [chan_blocks][tokens][2][NP]
    long long x_batch, x_token, dt_batch, dt_token, z_batch, z_token, b_batch, b_token, c_batch, c_token, dy_batch,
        dy_token;
    int B, T, D, N, n_seqs, softplus, vec, bc_vec, chan_blocks, segs, seg_tokens, row_tiles, span_tokens, pool, has_carry;
};

// Tokens [t0, t1) of row b, and the sequence that holds the current one.
struct Span {
    int b, t0, t1, n, begin, end;
};

// The bounds of sequence r.n, made to contain token t whatever cu_seqlens holds.
__device__ __forceinline__ void span_bounds(const ScanArgs &a, Span &r, int t) {
    if (a.cu) {
        r.begin = min(max(__ldg(a.cu + r.n), 0), t);
        r.end = min(max(__ldg(a.cu + r.n + 1), t + 1), a.T);
    } else {
        r.begin = 0;
        r.end = a.T;
    }
}
__device__ __forceinline__ void span_find(const ScanArgs &a, Span &r) {
    r.n = a.cu ? find_seq(a.cu, a.n_seqs, r.t0) : r.b;
    span_bounds(a, r, r.t0);
}
// The sequence that starts at token t, where the last one ended.
__device__ __forceinline__ void span_next(const ScanArgs &a, Span &r, int t) {
    if (!a.cu) return;
    while (r.n + 1 < a.n_seqs && __ldg(a.cu + r.n + 1) <= t) ++r.n;
    span_bounds(a, r, t);
}

// Eight neighbouring elements of which `live` exist.
template <typename T>
__device__ __forceinline__ Raw<T, 8> load8(const T *p, int live, bool vec) {
    if (live <= 0) return zero_raw<T, 8>();
    if (vec && live >= 8) return load_raw<T, 8>(p);
    return load_some<T, 8>(p, live);
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float *v, int live, bool vec) {
    if (live <= 0) return;
    if (vec && live >= 8) store_raw<T, 8>(p, pack<T, 8>(v));
    else store_some<T, 8>(p, v, live);
}

// M pairs of consecutive n from n0 of a row of N values (null: zero).
template <int M>
__device__ __forceinline__ void load_pairs(const float *row, int n0, int N, bool live, F2 (&h)[M]) {
#pragma unroll
    for (int i = 0; i < M; ++i) {
        const int n = n0 + 2 * i;
        h[i] = pair(row && live && n < N ? row[n] : 0.f, row && live && n + 1 < N ? row[n + 1] : 0.f);
    }
}
template <int M>
__device__ __forceinline__ void store_pairs(float *row, int n0, int N, const F2 (&h)[M]) {
#pragma unroll
    for (int i = 0; i < M; ++i) {
        const int n = n0 + 2 * i;
        if (n < N) row[n] = lo(h[i]);
        if (n + 1 < N) row[n + 1] = hi(h[i]);
    }
}

// The backward pass with its maps, partial sums and outputs placed in `a`;
// channels per block of its main kernel.
cudaError_t launch_scan_bwd(const ScanArgs &a, int dtype, void *dB, void *dC, float *dA, float *dskip, float *dbias,
                            cudaStream_t s);
int scan_bwd_channels(int N);
// The segments' maps and the tiles' start states for the backward pass.
cudaError_t launch_scan_maps(const ScanArgs &a, int dtype, cudaStream_t s);
// A row of padded n, 16-byte aligned.
template <int M>
__device__ __forceinline__ void store_aligned(float *row, const F2 (&h)[M]) {
#pragma unroll
    for (int i = 0; i < M / 2; ++i) reinterpret_cast<ulonglong2 *>(row)[i] = make_ulonglong2(h[2 * i], h[2 * i + 1]);
}
template <int M>
__device__ __forceinline__ void load_aligned(const float *row, bool live, F2 (&h)[M]) {
#pragma unroll
    for (int i = 0; i < M / 2; ++i) {
        const ulonglong2 v = live ? reinterpret_cast<const ulonglong2 *>(row)[i] : make_ulonglong2(0, 0);
        h[2 * i] = v.x, h[2 * i + 1] = v.y;
    }
}

cudaError_t launch_scan_combine(const ScanArgs &a, int maps, bool grad, cudaStream_t s);

// Eights of n, rounded up to a power of two: the state of a channel is padded to
// that many in the workspace and in registers.
inline int scan_parts(int N) { return N <= 8 ? 1 : N <= 16 ? 2 : N <= 32 ? 4 : 8; }

}  // namespace gdn
