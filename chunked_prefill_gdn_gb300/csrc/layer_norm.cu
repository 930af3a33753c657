// Layer norm over the last axis, forward and backward.
//
//     mean = sum_d x_d / D,   rstd = (sum_d (x_d - mean)^2 / D + eps)^-1/2,
//     xh = (x - mean) rstd,   y = xh w + b
//
// and, for an upstream gradient dy with g = dy w,
//
//     dx = rstd (g - sum_d g_d / D - xh sum_d g_d xh_d / D),
//     dw = sum_rows dy xh,    db = sum_rows dy.
//
// Both passes are streams bound by HBM: x (and dy) are read once, y (or dx)
// written once.  A row is held in registers (by a warp up to 512 columns, by a
// block of 128, 256 or 512 threads above), so the variance is the two-pass one
// around the exact fp32 mean without a second read.  The blocks are persistent
// and own their columns: the weights stay in registers over all rows of a block,
// and in the backward pass so do the sums of dw and db, which leave the block
// once, as one partial row per block; a second kernel adds those rows in a fixed
// order, so the result does not depend on the launch.  The next rows come in by
// asynchronous copies (up to four in flight, each thread reading back what it
// copied) while the current one is reduced.  The arithmetic is on pairs of
// columns (two-wide FP32): unpaired, the backward pass was held up by its own
// instructions between the barriers (163 us where the pairs took 142).  Rows wider
// than 8192 are read three times instead (layer_norm_wide_*).  Rows that only their
// type aligns, or of an odd length, go element by element through the same
// kernels, 16 elements per thread of which spill up to 200 bytes.
//
// Measured (bf16, fp32 weights, 32768 x 4096): forward 95 us, 5.7 TB/s, 85% of
// the measured copy rate; backward 139 us, 5.8 TB/s (87%), of it 6 us the sum
// over the blocks; fp32 178 and 236 us, 6.0 and 6.8 TB/s; 16 rows of 4096 2.4 us.
// Element by element (4095 columns) 113 and 339 us.  Rows of 16384 columns (8192 of
// them, bf16) 274 and 827 us, 2.0 and 1.0 TB/s: single elements, read three times.
#include <algorithm>

#include "elem.cuh"

namespace gdn {

namespace {

struct NormArgs {
    const void *x, *dy, *w, *b;
    void *out;               // y or dx
    float *mean, *rstd;      // outputs of the forward pass (may be null), inputs of the backward pass
    float *partial;          // [grid][2][D] partial dw, db or null
    long long rows, x_stride, dy_stride;
    int D, w_f32;
    float eps;
};

__device__ __forceinline__ float load_param(const void *p, int i, int f32) {
    return f32 ? static_cast<const float *>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

// Sums over the TPR threads of a row (a warp, or the whole block).
template <int TPR, int NSUM>
__device__ __forceinline__ void row_sums(float (&v)[NSUM], float (*red)[32]) {
#pragma unroll
    for (int s = 0; s < NSUM; ++s) v[s] = warp_sum(v[s]);
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) {
#pragma unroll
            for (int s = 0; s < NSUM; ++s) red[s][warp] = v[s];
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < NSUM; ++s) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < TPR / 32; ++i) t += red[s][i];
            v[s] = t;
        }
    }
}

// Threads per block for TPR threads per row, and the blocks per SM that the
// registers are budgeted for: 768 threads per SM in the forward pass (85
// registers), 512 in the backward pass (128), which holds two rows of inputs
// and two rows of sums.
constexpr int norm_threads(int tpr) { return tpr == 32 ? 256 : tpr; }
constexpr int norm_blocks_per_sm(int tpr, bool bwd) { return (bwd ? 512 : 768) / norm_threads(tpr); }

// Rows in flight per row of threads: as many as 64 KB per block hold, at most
// four.  (Unaligned rows are loaded element by element, one row ahead.)
template <typename T, int TPR, int VEC, int NV, int ARRAYS>
struct NormStages {
    static constexpr bool async = VEC * sizeof(T) == 16;
    static constexpr int bytes = norm_threads(TPR) * NV * ARRAYS * 16;   // one stage of a block
    static constexpr int count = !async ? 1 : 65536 / bytes >= 4 ? 4 : 65536 / bytes;
    static constexpr int smem = async ? count * bytes : 0;
};

__device__ __forceinline__ void copy16(uint4 *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

// A thread's element e of a row (of NV vectors of VEC elements, TPR vectors
// apart) is in the row; elements 2p and 2p + 1 are pair p.
template <int TPR, int VEC>
__device__ __forceinline__ bool live_col(int e, int t, int D) {
    return (e / VEC * TPR + t) * VEC + (VEC > 1 ? 0 : e % VEC) < D;   // a vector lies in the row or past it
}
__device__ __forceinline__ float half(F2 v, int e) { return e & 1 ? hi(v) : lo(v); }

template <int TPR, int VEC, int NV>
__device__ __forceinline__ void load_param_pairs(const void *p, int f32, int D, int t, float none, F2 (&v)[NV * VEC / 2]) {
    float x[NV * VEC];
#pragma unroll
    for (int e = 0; e < NV * VEC; ++e)
        x[e] = p && live_col<TPR, VEC>(e, t, D) ? load_param(p, (e / VEC * TPR + t) * VEC + e % VEC, f32) : none;
#pragma unroll
    for (int i = 0; i < NV * VEC / 2; ++i) v[i] = pair(x[2 * i], x[2 * i + 1]);
}

template <typename T, int TPR, int VEC, int NV, typename F>
__device__ __forceinline__ void unpack_row(int D, int t, F2 (&v)[NV * VEC / 2], F load) {
    if constexpr (VEC > 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            F2 u[VEC / 2];
            unpack_pairs<T, VEC>(live_col<TPR, VEC>(i * VEC, t, D) ? load(i) : zero_raw<T, VEC>(), u);
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) v[i * (VEC / 2) + j] = u[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV / 2; ++i) {
            float a, b;
            unpack<T, 1>(load(2 * i), &a);
            unpack<T, 1>(load(2 * i + 1), &b);
            v[i] = pair(a, b);
        }
    }
}

template <typename T, int TPR, int VEC, int NV>
__device__ __forceinline__ void store_row(T *row, int D, int t, const F2 (&v)[NV * VEC / 2]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * VEC;
        if (c >= D) continue;
        if constexpr (VEC > 1) {
            F2 u[VEC / 2];
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) u[j] = v[i * (VEC / 2) + j];
            store_raw<T, VEC>(row + c, pack_pairs<T, VEC>(u));
        } else {
            row[c] = from_f32<T>(half(v[i / 2], i));
        }
    }
}

// TPR threads per row, NV vectors of VEC elements per thread.
template <typename T, int TPR, int VEC, int NV>
__global__ void __launch_bounds__(norm_threads(TPR), norm_blocks_per_sm(TPR, false)) layer_norm_fwd_kernel(NormArgs a) {
    using St = NormStages<T, TPR, VEC, NV, 1>;
    constexpr int RPB = norm_threads(TPR) / TPR;   // rows per block
    constexpr int S = St::count, NT = norm_threads(TPR), NP = NV * VEC / 2;
    __shared__ float red[2][1][32];
    extern __shared__ uint4 stages[];              // [S][NV][thread]
    const int t = threadIdx.x % TPR;
    const long long step = (long long)gridDim.x * RPB;
    grid_dependency_wait();
    long long row = (long long)blockIdx.x * RPB + threadIdx.x / TPR;
    const T *x = static_cast<const T *>(a.x);
    T *y = static_cast<T *>(a.out);
    Raw<T, VEC> next[St::async ? 1 : NV];
    auto load_row = [&](long long r, int slot) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            const bool in = r < a.rows && c < a.D;
            if constexpr (St::async) {
                if (in) copy16(stages + (slot * NV + i) * NT + threadIdx.x, x + r * a.x_stride + c);
            } else {
                next[i] = in ? load_raw<T, VEC>(x + r * a.x_stride + c) : zero_raw<T, VEC>();
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int k = 0; k < (S > 1 ? S - 1 : 1); ++k) load_row(row + k * step, k);
    F2 w[NP], b[NP];
    load_param_pairs<TPR, VEC, NV>(a.w, a.w_f32, a.D, t, 1.f, w);
    load_param_pairs<TPR, VEC, NV>(a.b, a.w_f32, a.D, t, 0.f, b);
    const float inv_d = 1.f / (float)a.D;
    // (with several rows per block a row is a warp's own: it may leave the loop alone)
    for (int slot = 0; row < a.rows; row += step, slot = slot + 1 == S ? 0 : slot + 1) {
        F2 v[NP];
        if constexpr (St::async) {
            load_row(row + (S - 1) * step, slot == 0 ? S - 1 : slot - 1);
            copy_wait<S - 1>();
            unpack_row<T, TPR, VEC, NV>(a.D, t, v, [&](int i) {
                return load_raw<T, VEC>(reinterpret_cast<const T *>(stages + (slot * NV + i) * NT + threadIdx.x));
            });
        } else {
            unpack_row<T, TPR, VEC, NV>(a.D, t, v, [&](int i) { return next[i]; });
            load_row(row + step, 0);
        }
        F2 s2 = v[0];
#pragma unroll
        for (int p = 1; p < NP; ++p) s2 = add2(s2, v[p]);
        float s[1] = {lo(s2) + hi(s2)};
        row_sums<TPR, 1>(s, red[0]);
        const float mean = s[0] * inv_d;
        F2 q2 = both(0.f);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            v[p] = add2(v[p], both(-mean));
            if (!live_col<TPR, VEC>(2 * p, t, a.D)) v[p] = v[p] & 0xFFFFFFFF00000000ull;
            if (!live_col<TPR, VEC>(2 * p + 1, t, a.D)) v[p] = v[p] & 0x00000000FFFFFFFFull;
            q2 = fma2(v[p], v[p], q2);
        }
        float q[1] = {lo(q2) + hi(q2)};
        row_sums<TPR, 1>(q, red[1]);
        const float rstd = rsqrtf(q[0] * inv_d + a.eps);
#pragma unroll
        for (int p = 0; p < NP; ++p) v[p] = fma2(mul2(v[p], both(rstd)), w[p], b[p]);
        store_row<T, TPR, VEC, NV>(y + row * a.D, a.D, t, v);
        if (t == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

template <typename T, int TPR, int VEC, int NV>
__global__ void __launch_bounds__(norm_threads(TPR), norm_blocks_per_sm(TPR, true)) layer_norm_bwd_kernel(NormArgs a) {
    using St = NormStages<T, TPR, VEC, NV, 2>;
    constexpr int RPB = norm_threads(TPR) / TPR;
    constexpr int S = St::count, NT = norm_threads(TPR), NP = NV * VEC / 2;
    __shared__ float red[2][2][32];
    extern __shared__ uint4 stages[];              // [S][x, dy][NV][thread]
    const int t = threadIdx.x % TPR;
    const long long step = (long long)gridDim.x * RPB;
    grid_dependency_wait();
    long long row = (long long)blockIdx.x * RPB + threadIdx.x / TPR;
    const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy);
    T *dx = static_cast<T *>(a.out);
    Raw<T, VEC> nx[St::async ? 1 : NV], ng[St::async ? 1 : NV];
    auto load_row = [&](long long r, int slot) {
        const bool live = r < a.rows;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            const bool in = live && c < a.D;
            if constexpr (St::async) {
                uint4 *at = stages + (slot * 2 * NV + i) * NT + threadIdx.x;
                if (in) copy16(at, x + r * a.x_stride + c), copy16(at + NV * NT, dy + r * a.dy_stride + c);
            } else {
                nx[i] = in ? load_raw<T, VEC>(x + r * a.x_stride + c) : zero_raw<T, VEC>();
                ng[i] = in ? load_raw<T, VEC>(dy + r * a.dy_stride + c) : zero_raw<T, VEC>();
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int k = 0; k < (S > 1 ? S - 1 : 1); ++k) load_row(row + k * step, k);
    float nmean = row < a.rows ? a.mean[row] : 0.f, nrstd = row < a.rows ? a.rstd[row] : 0.f;
    F2 w[NP], dw[NP], db[NP];
    load_param_pairs<TPR, VEC, NV>(a.w, a.w_f32, a.D, t, 1.f, w);
#pragma unroll
    for (int p = 0; p < NP; ++p) dw[p] = db[p] = both(0.f);
    const float inv_d = 1.f / (float)a.D;
    int phase = 0;
    for (int slot = 0; row < a.rows; row += step, slot = slot + 1 == S ? 0 : slot + 1, phase ^= 1) {
        F2 xh[NP], g[NP];
        const float mean = nmean, rstd = nrstd;
        if (row + step < a.rows) nmean = a.mean[row + step], nrstd = a.rstd[row + step];
        if constexpr (St::async) {
            load_row(row + (S - 1) * step, slot == 0 ? S - 1 : slot - 1);
            copy_wait<S - 1>();
            const uint4 *at = stages + slot * 2 * NV * NT + threadIdx.x;
            unpack_row<T, TPR, VEC, NV>(a.D, t, xh, [&](int i) { return load_raw<T, VEC>(reinterpret_cast<const T *>(at + i * NT)); });
            unpack_row<T, TPR, VEC, NV>(a.D, t, g, [&](int i) { return load_raw<T, VEC>(reinterpret_cast<const T *>(at + (NV + i) * NT)); });
        } else {
            unpack_row<T, TPR, VEC, NV>(a.D, t, xh, [&](int i) { return nx[i]; });
            unpack_row<T, TPR, VEC, NV>(a.D, t, g, [&](int i) { return ng[i]; });
            load_row(row + step, 0);
        }
        // Past D g is zero and xh = -mean rstd, which adds nothing unless it overflows:
        // then 0 times it is no longer 0.  With vectors that is branched on per row:
        // those columns take the mean itself (139 us at 32768 x 4096 bf16, as without;
        // the sum taken again on the branch 171).  Element by element the mean is
        // masked (4095 columns 339 us, 332 without; the branch 424).
        if constexpr (VEC > 1) {
            if (!(fabsf(mean * rstd) < INFINITY)) {
#pragma unroll
                for (int p = 0; p < NP; ++p)
                    xh[p] = pair(live_col<TPR, VEC>(2 * p, t, a.D) ? lo(xh[p]) : mean,
                                 live_col<TPR, VEC>(2 * p + 1, t, a.D) ? hi(xh[p]) : mean);
            }
        }
        F2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const F2 m = VEC > 1 ? both(-mean) : pair(live_col<TPR, VEC>(2 * p, t, a.D) ? -mean : 0.f,
                                                      live_col<TPR, VEC>(2 * p + 1, t, a.D) ? -mean : 0.f);
            xh[p] = mul2(add2(xh[p], m), both(rstd));
            dw[p] = fma2(g[p], xh[p], dw[p]);
            db[p] = add2(db[p], g[p]);
            g[p] = mul2(g[p], w[p]);
            s0 = add2(s0, g[p]);
            s1 = fma2(g[p], xh[p], s1);
        }
        float s[2] = {lo(s0) + hi(s0), lo(s1) + hi(s1)};
        row_sums<TPR, 2>(s, red[phase]);
        const float m1 = s[0] * inv_d, m2 = s[1] * inv_d;
#pragma unroll
        for (int p = 0; p < NP; ++p) g[p] = mul2(fma2(xh[p], both(-m2), add2(g[p], both(-m1))), both(rstd));
        store_row<T, TPR, VEC, NV>(dx + row * a.D, a.D, t, g);
    }
    if (!a.partial) return;
    float *pw = a.partial + 2ll * blockIdx.x * a.D, *pb = pw + a.D;
    if constexpr (RPB == 1) {
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i) {
            const int c = (i / VEC * TPR + t) * VEC + i % VEC;
            if (c < a.D) pw[c] = half(dw[i / 2], i), pb[c] = half(db[i / 2], i);
        }
    } else {
        // the warps' sums, added in the warps' order
        constexpr int COLS = TPR * NV * VEC;
        __shared__ float sum[2][COLS];
        for (int r = 0; r < RPB; ++r) {
            if ((int)threadIdx.x / TPR == r) {
#pragma unroll
                for (int i = 0; i < NV * VEC; ++i) {
                    const int c = (i / VEC * TPR + t) * VEC + i % VEC;
                    sum[0][c] = (r ? sum[0][c] : 0.f) + half(dw[i / 2], i);
                    sum[1][c] = (r ? sum[1][c] : 0.f) + half(db[i / 2], i);
                }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.D; c += blockDim.x) pw[c] = sum[0][c], pb[c] = sum[1][c];
    }
}

// Rows wider than the register-resident kernels take: a block per row, three
// reads of it (the later two mostly from L2).
template <typename T>
__global__ void __launch_bounds__(1024) layer_norm_wide_fwd_kernel(NormArgs a) {
    __shared__ float red[2][1][32];
    const float inv_d = 1.f / (float)a.D;
    grid_dependency_wait();
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
        T *y = static_cast<T *>(a.out) + row * a.D;
        float s[1] = {0.f}, q[1] = {0.f};
        for (int c = threadIdx.x; c < a.D; c += 1024) s[0] += to_f32(x[c]);
        row_sums<1024, 1>(s, red[0]);
        const float mean = s[0] * inv_d;
        for (int c = threadIdx.x; c < a.D; c += 1024) {
            const float d = to_f32(x[c]) - mean;
            q[0] = fmaf(d, d, q[0]);
        }
        row_sums<1024, 1>(q, red[1]);
        const float rstd = rsqrtf(q[0] * inv_d + a.eps);
        for (int c = threadIdx.x; c < a.D; c += 1024)
            y[c] = from_f32<T>(fmaf((to_f32(x[c]) - mean) * rstd, a.w ? load_param(a.w, c, a.w_f32) : 1.f,
                                    a.b ? load_param(a.b, c, a.w_f32) : 0.f));
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

// The block's partial sums of dw and db live in its partial row (L2-resident).
template <typename T>
__global__ void __launch_bounds__(1024) layer_norm_wide_bwd_kernel(NormArgs a) {
    __shared__ float red[2][2][32];
    const float inv_d = 1.f / (float)a.D;
    float *pw = a.partial ? a.partial + 2ll * blockIdx.x * a.D : nullptr;
    int phase = 0;
    grid_dependency_wait();
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, phase ^= 1) {
        const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
        const T *dy = static_cast<const T *>(a.dy) + row * a.dy_stride;
        T *dx = static_cast<T *>(a.out) + row * a.D;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s[2] = {0.f, 0.f};
        for (int c = threadIdx.x; c < a.D; c += 1024) {
            const float g = to_f32(dy[c]), xh = (to_f32(x[c]) - mean) * rstd;
            const float gw = g * (a.w ? load_param(a.w, c, a.w_f32) : 1.f);
            s[0] += gw;
            s[1] = fmaf(gw, xh, s[1]);
            if (pw) {
                const bool first = row == blockIdx.x;
                pw[c] = first ? g * xh : fmaf(g, xh, pw[c]);
                pw[a.D + c] = first ? g : pw[a.D + c] + g;
            }
        }
        row_sums<1024, 2>(s, red[phase]);
        const float m1 = s[0] * inv_d, m2 = s[1] * inv_d;
        for (int c = threadIdx.x; c < a.D; c += 1024) {
            const float gw = to_f32(dy[c]) * (a.w ? load_param(a.w, c, a.w_f32) : 1.f);
            dx[c] = from_f32<T>(rstd * (gw - m1 - (to_f32(x[c]) - mean) * rstd * m2));
        }
    }
}

// dw (blockIdx.y = 0) and db from the blocks' partial rows, in the blocks' order:
// 32 row groups of 32 columns per block, then the groups in order.
__global__ void __launch_bounds__(1024) layer_norm_reduce_kernel(const float *partial, int rows, int D, float *dw,
                                                                 float *db) {
    __shared__ float sum[32][32];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.f;
    grid_dependency_wait();
    if (c < D) {
        const float *p = partial + (long long)blockIdx.y * D + c;
#pragma unroll 8
        for (int r = grp; r < rows; r += 32) s += p[2ll * r * D];
    }
    sum[grp][lane] = s;
    __syncthreads();
    float *out = blockIdx.y ? db : dw;
    if (grp == 0 && c < D && out) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += sum[i][lane];
        out[c] = s;
    }
}

// Threads per row by its columns: at most 16 elements per thread.  Rows wider
// than kNormMaxCols take the three-read kernels.
constexpr int kNormMaxCols = 8192;
int threads_per_row(int D) { return D <= 512 ? 32 : D <= 1024 ? 128 : D <= 4096 ? 256 : 512; }

// Blocks of the persistent grid.
int norm_grid(long long rows, int D, bool bwd) {
    if (D > kNormMaxCols) return (int)std::min<long long>(rows, device_sm_count());
    const int tpr = threads_per_row(D), rpb = norm_threads(tpr) / tpr;
    return (int)std::min<long long>((rows + rpb - 1) / rpb, (long long)device_sm_count() * norm_blocks_per_sm(tpr, bwd));
}

template <typename T, int TPR, int VEC, int NV, bool BWD>
cudaError_t launch_norm_one(const NormArgs &a, int grid, cudaStream_t s) {
    constexpr int smem = NormStages<T, TPR, VEC, NV, BWD ? 2 : 1>::smem;
    void (*kernel)(NormArgs);
    if constexpr (BWD) kernel = layer_norm_bwd_kernel<T, TPR, VEC, NV>;
    else kernel = layer_norm_fwd_kernel<T, TPR, VEC, NV>;
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(kernel, dim3(grid), dim3(norm_threads(TPR)), smem, s, a);
}

template <typename T, int VEC, bool BWD>
cudaError_t launch_norm(const NormArgs &a, int grid, cudaStream_t s) {
#define GDN_NORM(TPR, EPT) return launch_norm_one<T, TPR, VEC, (EPT) / VEC, BWD>(a, grid, s)
    if (a.D <= 256) GDN_NORM(32, 8);
    else if (a.D <= 512) GDN_NORM(32, 16);
    else if (a.D <= 1024) GDN_NORM(128, 8);
    else if (a.D <= 2048) GDN_NORM(256, 8);
    else if (a.D <= 4096) GDN_NORM(256, 16);
    else if (a.D <= kNormMaxCols) GDN_NORM(512, 16);
    void (*wide)(NormArgs);
    if constexpr (BWD) wide = layer_norm_wide_bwd_kernel<T>;
    else wide = layer_norm_wide_fwd_kernel<T>;
    return launch_dependent(wide, dim3(grid), dim3(1024), 0, s, a);
#undef GDN_NORM
}

template <typename T, bool BWD>
cudaError_t launch_norm_typed(const NormArgs &a, int grid, cudaStream_t s) {
    constexpr int VEC = 16 / (int)sizeof(T);
    const bool vec = aligned16(a.x) && aligned16(a.out) && (!BWD || aligned16(a.dy)) && a.D % VEC == 0 &&
                     a.x_stride % VEC == 0 && (!BWD || a.dy_stride % VEC == 0);
    return vec ? launch_norm<T, VEC, BWD>(a, grid, s) : launch_norm<T, 1, BWD>(a, grid, s);
}

bool elem_aligned(const void *p, int dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (dtype == GDN_F32 ? 3u : 1u)) == 0;
}

gdn_status norm_args_ok(int64_t rows, int D, int dtype, int w_dtype, int64_t stride) {
    if (rows < 0 || D < 1 || stride < D) return GDN_ERR_INVALID_ARG;
    if (D > (1 << 30)) return GDN_ERR_UNSUPPORTED;   // columns are counted in 32 bits
    if ((dtype != GDN_BF16 && dtype != GDN_F32) || (w_dtype != GDN_BF16 && w_dtype != GDN_F32)) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

}  // namespace

}  // namespace gdn

extern "C" gdn_status gdn_layer_norm_fwd(const void *x, int64_t x_stride, const void *weight, const void *bias,
                                         gdn_dtype w_dtype, float eps, int64_t rows, int D, gdn_dtype dtype, void *y,
                                         float *mean, float *rstd, gdn_stream_t stream) {
    const gdn_status st = gdn::norm_args_ok(rows, D, dtype, w_dtype, x_stride);
    if (st != GDN_OK) return st;
    if (!(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
    if (rows == 0) return GDN_OK;
    if (!x || !y || !gdn::elem_aligned(x, dtype) || !gdn::elem_aligned(y, dtype) ||
        !gdn::elem_aligned(weight, w_dtype) || !gdn::elem_aligned(bias, w_dtype) ||
        !gdn::elem_aligned(mean, GDN_F32) || !gdn::elem_aligned(rstd, GDN_F32))
        return GDN_ERR_INVALID_ARG;
    gdn::NormArgs a = {};
    a.x = x, a.w = weight, a.b = bias, a.out = y, a.mean = mean, a.rstd = rstd;
    a.rows = rows, a.x_stride = x_stride, a.D = D, a.w_f32 = w_dtype == GDN_F32, a.eps = eps;
    const int grid = gdn::norm_grid(rows, D, false);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == GDN_BF16 ? gdn::launch_norm_typed<__nv_bfloat16, false>(a, grid, s)
                                            : gdn::launch_norm_typed<float, false>(a, grid, s);
    if (e != cudaSuccess) {
        gdn::set_error_detail("launch layer_norm_fwd", e);
        return GDN_ERR_CUDA;
    }
    return GDN_OK;
}

extern "C" size_t gdn_layer_norm_bwd_workspace_size(int64_t rows, int D) {
    if (rows < 0 || D < 1) return 0;
    return std::max<size_t>(16, (size_t)gdn::norm_grid(rows, D, true) * 2 * (size_t)D * sizeof(float));
}

extern "C" gdn_status gdn_layer_norm_bwd(const void *dy, int64_t dy_stride, const void *x, int64_t x_stride,
                                         const float *mean, const float *rstd, const void *weight, gdn_dtype w_dtype,
                                         int64_t rows, int D, gdn_dtype dtype, void *dx, float *dweight, float *dbias,
                                         void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    const gdn_status st = gdn::norm_args_ok(rows, D, dtype, w_dtype, x_stride);
    if (st != GDN_OK) return st;
    if (dy_stride < D) return GDN_ERR_INVALID_ARG;
    const bool params = dweight || dbias;
    if (!gdn::elem_aligned(dweight, GDN_F32) || !gdn::elem_aligned(dbias, GDN_F32) ||
        !gdn::elem_aligned(weight, w_dtype))
        return GDN_ERR_INVALID_ARG;
    if (rows > 0 && (!dy || !x || !mean || !rstd || !dx || !gdn::elem_aligned(dy, dtype) ||
                     !gdn::elem_aligned(x, dtype) || !gdn::elem_aligned(dx, dtype) ||
                     !gdn::elem_aligned(mean, GDN_F32) || !gdn::elem_aligned(rstd, GDN_F32)))
        return GDN_ERR_INVALID_ARG;
    const int grid = gdn::norm_grid(rows, D, true);
    if (params && rows > 0) {
        if (!workspace || !gdn::aligned16(workspace)) return GDN_ERR_INVALID_ARG;
        if (workspace_bytes < gdn_layer_norm_bwd_workspace_size(rows, D)) return GDN_ERR_WORKSPACE;
    }
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (rows > 0) {
        gdn::NormArgs a = {};
        a.x = x, a.dy = dy, a.w = weight, a.out = dx;
        a.mean = const_cast<float *>(mean), a.rstd = const_cast<float *>(rstd);
        a.partial = params ? static_cast<float *>(workspace) : nullptr;
        a.rows = rows, a.x_stride = x_stride, a.dy_stride = dy_stride, a.D = D, a.w_f32 = w_dtype == GDN_F32;
        e = dtype == GDN_BF16 ? gdn::launch_norm_typed<__nv_bfloat16, true>(a, grid, s)
                              : gdn::launch_norm_typed<float, true>(a, grid, s);
    }
    if (e == cudaSuccess && params) {  // no rows: the sums are zero
        e = gdn::launch_dependent(gdn::layer_norm_reduce_kernel, dim3((D + 31) / 32, 2), dim3(1024), 0, s,
                                  static_cast<const float *>(workspace), rows > 0 ? grid : 0, D, dweight, dbias);
    }
    if (e != cudaSuccess) {
        gdn::set_error_detail("launch layer_norm_bwd", e);
        return GDN_ERR_CUDA;
    }
    return GDN_OK;
}
