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
// written once.  A row is held in registers (by a warp up to 512 columns, by
// a block of 128, 256 or 512 threads above), so the variance is the two-pass one
// around the exact fp32 mean without a second read.  The blocks are persistent
// and own their columns: the weights stay in registers over all rows of a
// block, and in the backward pass so do the sums of dw and db, which leave the
// block once, as one partial row per block; a second kernel adds those rows in
// a fixed order, so the result does not depend on the launch.  The next row is
// loaded before the current one is reduced.  Rows wider than 8192 are read
// three times instead (layer_norm_wide_*).
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

// TPR threads per row, NV vectors of VEC elements per thread.
template <typename T, int TPR, int VEC, int NV>
__global__ void __launch_bounds__(norm_threads(TPR), norm_blocks_per_sm(TPR, false)) layer_norm_fwd_kernel(NormArgs a) {
    constexpr int RPB = norm_threads(TPR) / TPR;   // rows per block
    __shared__ float red[2][1][32];
    const int t = threadIdx.x % TPR;
    const long long step = (long long)gridDim.x * RPB;
    long long row = (long long)blockIdx.x * RPB + threadIdx.x / TPR;
    const T *x = static_cast<const T *>(a.x);
    T *y = static_cast<T *>(a.out);
    Raw<T, VEC> next[NV];
    auto load_row = [&](long long r) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            next[i] = r < a.rows && c < a.D ? load_raw<T, VEC>(x + r * a.x_stride + c) : zero_raw<T, VEC>();
        }
    };
    load_row(row);
    float w[NV * VEC], b[NV * VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int c = (i * TPR + t) * VEC + j;
            w[i * VEC + j] = a.w && c < a.D ? load_param(a.w, c, a.w_f32) : 1.f;
            b[i * VEC + j] = a.b && c < a.D ? load_param(a.b, c, a.w_f32) : 0.f;
        }
    }
    const float inv_d = 1.f / (float)a.D;
    // a row group without a row of its own still takes part in the block's sums
    for (long long first = (long long)blockIdx.x * RPB; first < a.rows; first += step, row += step) {
        float v[NV * VEC];
#pragma unroll
        for (int i = 0; i < NV; ++i) unpack<T, VEC>(next[i], v + i * VEC);
        load_row(row + step);
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i) s[0] += v[i];
        row_sums<TPR, 1>(s, red[0]);
        const float mean = s[0] * inv_d;
        float q[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = (i * TPR + t) * VEC < a.D;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                v[i * VEC + j] = in ? v[i * VEC + j] - mean : 0.f;
                q[0] = fmaf(v[i * VEC + j], v[i * VEC + j], q[0]);
            }
        }
        row_sums<TPR, 1>(q, red[1]);
        const float rstd = rsqrtf(q[0] * inv_d + a.eps);
        if (row >= a.rows) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (c >= a.D) continue;
            float o[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) o[j] = fmaf(v[i * VEC + j] * rstd, w[i * VEC + j], b[i * VEC + j]);
            store_raw<T, VEC>(y + row * a.D + c, pack<T, VEC>(o));
        }
        if (t == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

template <typename T, int TPR, int VEC, int NV>
__global__ void __launch_bounds__(norm_threads(TPR), norm_blocks_per_sm(TPR, true)) layer_norm_bwd_kernel(NormArgs a) {
    constexpr int RPB = norm_threads(TPR) / TPR;
    __shared__ float red[2][2][32];
    const int t = threadIdx.x % TPR;
    const long long step = (long long)gridDim.x * RPB;
    long long row = (long long)blockIdx.x * RPB + threadIdx.x / TPR;
    const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy);
    T *dx = static_cast<T *>(a.out);
    Raw<T, VEC> nx[NV], ng[NV];
    float nmean = 0.f, nrstd = 0.f;
    auto load_row = [&](long long r) {
        const bool live = r < a.rows;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            nx[i] = live && c < a.D ? load_raw<T, VEC>(x + r * a.x_stride + c) : zero_raw<T, VEC>();
            ng[i] = live && c < a.D ? load_raw<T, VEC>(dy + r * a.dy_stride + c) : zero_raw<T, VEC>();
        }
        nmean = live ? a.mean[r] : 0.f;
        nrstd = live ? a.rstd[r] : 0.f;
    };
    load_row(row);
    float w[NV * VEC], dw[NV * VEC], db[NV * VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int c = (i * TPR + t) * VEC + j;
            w[i * VEC + j] = a.w && c < a.D ? load_param(a.w, c, a.w_f32) : 1.f;
            dw[i * VEC + j] = db[i * VEC + j] = 0.f;
        }
    }
    const float inv_d = 1.f / (float)a.D;
    int phase = 0;
    for (long long first = (long long)blockIdx.x * RPB; first < a.rows; first += step, row += step, phase ^= 1) {
        float xh[NV * VEC], g[NV * VEC];
        const float mean = nmean, rstd = nrstd;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack<T, VEC>(nx[i], xh + i * VEC);
            unpack<T, VEC>(ng[i], g + i * VEC);
        }
        load_row(row + step);
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = (i * TPR + t) * VEC < a.D;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int e = i * VEC + j;
                xh[e] = in ? (xh[e] - mean) * rstd : 0.f;
                dw[e] = fmaf(g[e], xh[e], dw[e]);
                db[e] += g[e];
                g[e] *= w[e];
                s[0] += g[e];
                s[1] = fmaf(g[e], xh[e], s[1]);
            }
        }
        row_sums<TPR, 2>(s, red[phase]);
        if (row >= a.rows) continue;
        const float m1 = s[0] * inv_d, m2 = s[1] * inv_d;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (c >= a.D) continue;
            float o[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int e = i * VEC + j;
                o[j] = rstd * (g[e] - m1 - xh[e] * m2);
            }
            store_raw<T, VEC>(dx + row * a.D + c, pack<T, VEC>(o));
        }
    }
    if (!a.partial) return;
    float *pw = a.partial + 2ll * blockIdx.x * a.D, *pb = pw + a.D;
    if constexpr (RPB == 1) {
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i) {
            const int c = (i / VEC * TPR + t) * VEC + i % VEC;
            if (c < a.D) pw[c] = dw[i], pb[c] = db[i];
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
                    sum[0][c] = (r ? sum[0][c] : 0.f) + dw[i];
                    sum[1][c] = (r ? sum[1][c] : 0.f) + db[i];
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

// dw, db from the blocks' partial rows, in the blocks' order: eight row groups
// of 32 columns per block, then the groups in order.
__global__ void __launch_bounds__(256) layer_norm_reduce_kernel(const float *partial, int rows, int D, float *dw,
                                                                float *db) {
    __shared__ float sum[2][8][32];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s0 = 0.f, s1 = 0.f;
    if (c < D) {
#pragma unroll 4
        for (int r = grp; r < rows; r += 8) {
            s0 += partial[2ll * r * D + c];
            s1 += partial[(2ll * r + 1) * D + c];
        }
    }
    sum[0][grp][lane] = s0;
    sum[1][grp][lane] = s1;
    __syncthreads();
    if (grp < 2 && c < D) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sum[grp][i][lane];
        float *out = grp ? db : dw;
        if (out) out[c] = s;
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

template <typename T, int VEC, bool BWD>
cudaError_t launch_norm(const NormArgs &a, int grid, cudaStream_t s) {
#define GDN_NORM(TPR, EPT)                                                                                      \
    do {                                                                                                        \
        if constexpr (BWD) layer_norm_bwd_kernel<T, TPR, VEC, (EPT) / VEC><<<grid, norm_threads(TPR), 0, s>>>(a); \
        else layer_norm_fwd_kernel<T, TPR, VEC, (EPT) / VEC><<<grid, norm_threads(TPR), 0, s>>>(a);               \
    } while (0)
    if (a.D <= 256) GDN_NORM(32, 8);
    else if (a.D <= 512) GDN_NORM(32, 16);
    else if (a.D <= 1024) GDN_NORM(128, 8);
    else if (a.D <= 2048) GDN_NORM(256, 8);
    else if (a.D <= 4096) GDN_NORM(256, 16);
    else if (a.D <= kNormMaxCols) GDN_NORM(512, 16);
    else if constexpr (BWD) layer_norm_wide_bwd_kernel<T><<<grid, 1024, 0, s>>>(a);
    else layer_norm_wide_fwd_kernel<T><<<grid, 1024, 0, s>>>(a);
#undef GDN_NORM
    return cudaGetLastError();
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
    if ((dtype != GDN_BF16 && dtype != GDN_F32) || (w_dtype != GDN_BF16 && w_dtype != GDN_F32)) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

}  // namespace

}  // namespace gdn

extern "C" gdn_status gdn_layer_norm_fwd(const void *x, int64_t x_stride, const void *weight, const void *bias,
                                         gdn_dtype w_dtype, float eps, int64_t rows, int D, gdn_dtype dtype, void *y,
                                         float *mean, float *rstd, gdn_stream_t stream) {
    if (gdn::norm_args_ok(rows, D, dtype, w_dtype, x_stride) != GDN_OK || !(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
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
    if (gdn::norm_args_ok(rows, D, dtype, w_dtype, x_stride) != GDN_OK || dy_stride < D) return GDN_ERR_INVALID_ARG;
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
        gdn::layer_norm_reduce_kernel<<<(D + 31) / 32, 256, 0, s>>>(static_cast<const float *>(workspace),
                                                                   rows > 0 ? grid : 0, D, dweight, dbias);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) {
        gdn::set_error_detail("launch layer_norm_bwd", e);
        return GDN_ERR_CUDA;
    }
    return GDN_OK;
}
