// One token of the gated delta rule on a cached state, the serving form of the
// chunked pass: for every sequence n and head h, with S the [dk, dv] state as
// stored (S[j][i], key index j outer),
//
//     S' = alpha S,  u_i = beta (v_i - sum_j k_j S'_ji),
//     S_ji <- S'_ji + k_j u_i,  o_i = scale sum_j q_j S_ji,   alpha = exp(g).
//
// The state is read once and written once (8 dk dv bytes against a few
// hundred for the token), so the step is bound by HBM.  A block holds all dk
// rows of `cols` neighbouring columns in registers, four columns per thread;
// since o_i = scale (alpha sum_j q_j S_ji + (q.k) u_i), both sums over the
// rows are taken in one pass and one exchange through shared memory, and the
// updated rows leave from the registers.  A whole state per block (cols = dv)
// makes the longest contiguous runs; when the (sequence, head) pairs do not
// give every SM a block or two, blocks of 32 columns spread a state over up to
// four SMs.
//
// Measured (bf16, 128 x 128 states): 128 sequences x 32 heads 86 us, 6.3 TB/s, 94%
// of the measured copy rate (fp32 88 us); one sequence x 32 heads (4.2 MB) 2.4 us.
#include <algorithm>

#include "elem.cuh"

namespace gdn {

namespace {

struct DeltaArgs {
    const void *q, *k, *v;
    const float *g, *beta;
    float *state;
    const int32_t *slots;
    void *o;
    int H, dk, dv, pool, l2norm;
    long long units, q_token, k_token, v_token;
    float scale;
};

constexpr int kDeltaThreads = 256;

// DK rows, COLS columns per block.
template <typename T, int DK, int COLS>
__global__ void __launch_bounds__(kDeltaThreads) delta_step_kernel(DeltaArgs a) {
    constexpr int CG = COLS / 4;                       // threads across a row
    constexpr int RG = kDeltaThreads / CG;             // rows of one sweep
    constexpr int R = DK / RG;                         // rows per thread (RG is 8, 16 or 32)
    constexpr int WARPS = kDeltaThreads / 32;
    constexpr int RPW = 32 / CG;                       // rows of one warp's sweep
    __shared__ float qs[DK], ks[DK], dots[3];
    __shared__ float4 sum[2][WARPS][CG];
    grid_dependency_wait();
    const int parts = a.dv / COLS;
    const long long unit = blockIdx.x / parts;         // n * H + h
    const int col0 = (int)(blockIdx.x % parts) * COLS;
    const long long n = unit / a.H;
    const int h = (int)(unit % a.H);
    T *o = static_cast<T *>(a.o) + unit * a.dv + col0;
    const int slot = a.slots ? __ldg(a.slots + n) : (int)n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (slot < 0 || slot >= a.pool) {                  // a padded row
        if (tid < COLS) o[tid] = from_f32<T>(0.f);
        return;
    }
    float *S = a.state + ((long long)slot * a.H + h) * DK * a.dv + col0;
    const int cg = tid % CG, row0 = tid / CG;
    float4 s[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        s[i] = *reinterpret_cast<const float4 *>(S + (long long)(row0 + i * RG) * a.dv + cg * 4);
    if (warp == 0) {                                   // q, k, their norms and their product
        float qv[DK / 32], kv[DK / 32], qq = 0.f, kk = 0.f, qk = 0.f;
#pragma unroll
        for (int i = 0; i < DK / 32; ++i) {
            qv[i] = to_f32(static_cast<const T *>(a.q)[n * a.q_token + h * DK + i * 32 + lane]);
            kv[i] = to_f32(static_cast<const T *>(a.k)[n * a.k_token + h * DK + i * 32 + lane]);
            qq = fmaf(qv[i], qv[i], qq);
            kk = fmaf(kv[i], kv[i], kk);
        }
        float fq = 1.f, fk = 1.f;
        if (a.l2norm) {
            fq = rsqrtf(warp_sum(qq) + kQkNormEps);
            fk = rsqrtf(warp_sum(kk) + kQkNormEps);
        }
#pragma unroll
        for (int i = 0; i < DK / 32; ++i) {
            qv[i] *= fq, kv[i] *= fk;
            qk = fmaf(qv[i], kv[i], qk);
            qs[i * 32 + lane] = qv[i];
            ks[i * 32 + lane] = kv[i];
        }
        qk = warp_sum(qk);
        if (lane == 0) dots[0] = qk, dots[1] = expf(a.g[unit]), dots[2] = a.beta[unit];
    }
    __syncthreads();
    float4 sk = make_float4(0.f, 0.f, 0.f, 0.f), sq = sk;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float kj = ks[row0 + i * RG], qj = qs[row0 + i * RG];
        sk.x = fmaf(kj, s[i].x, sk.x), sk.y = fmaf(kj, s[i].y, sk.y);
        sk.z = fmaf(kj, s[i].z, sk.z), sk.w = fmaf(kj, s[i].w, sk.w);
        sq.x = fmaf(qj, s[i].x, sq.x), sq.y = fmaf(qj, s[i].y, sq.y);
        sq.z = fmaf(qj, s[i].z, sq.z), sq.w = fmaf(qj, s[i].w, sq.w);
    }
    if constexpr (RPW > 1) {
#pragma unroll
        for (int off = CG; off < 32; off <<= 1) {
            sk.x += __shfl_xor_sync(0xffffffffu, sk.x, off), sk.y += __shfl_xor_sync(0xffffffffu, sk.y, off);
            sk.z += __shfl_xor_sync(0xffffffffu, sk.z, off), sk.w += __shfl_xor_sync(0xffffffffu, sk.w, off);
            sq.x += __shfl_xor_sync(0xffffffffu, sq.x, off), sq.y += __shfl_xor_sync(0xffffffffu, sq.y, off);
            sq.z += __shfl_xor_sync(0xffffffffu, sq.z, off), sq.w += __shfl_xor_sync(0xffffffffu, sq.w, off);
        }
    }
    if (lane < CG) sum[0][warp][cg] = sk, sum[1][warp][cg] = sq;
    __syncthreads();
    sk = sq = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        const float4 x = sum[0][w][cg], y = sum[1][w][cg];
        sk.x += x.x, sk.y += x.y, sk.z += x.z, sk.w += x.w;
        sq.x += y.x, sq.y += y.y, sq.z += y.z, sq.w += y.w;
    }
    const float qk = dots[0], alpha = dots[1], beta = dots[2];
    float vv[4];
    const T *v = static_cast<const T *>(a.v) + n * a.v_token + (long long)h * a.dv + col0 + cg * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) vv[e] = to_f32(v[e]);
    float4 u;
    u.x = beta * fmaf(-alpha, sk.x, vv[0]), u.y = beta * fmaf(-alpha, sk.y, vv[1]);
    u.z = beta * fmaf(-alpha, sk.z, vv[2]), u.w = beta * fmaf(-alpha, sk.w, vv[3]);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float kj = ks[row0 + i * RG];
        float4 x;
        x.x = fmaf(alpha, s[i].x, kj * u.x), x.y = fmaf(alpha, s[i].y, kj * u.y);
        x.z = fmaf(alpha, s[i].z, kj * u.z), x.w = fmaf(alpha, s[i].w, kj * u.w);
        *reinterpret_cast<float4 *>(S + (long long)(row0 + i * RG) * a.dv + cg * 4) = x;
    }
    if (row0 == 0) {
        o[cg * 4 + 0] = from_f32<T>(a.scale * fmaf(alpha, sq.x, qk * u.x));
        o[cg * 4 + 1] = from_f32<T>(a.scale * fmaf(alpha, sq.y, qk * u.y));
        o[cg * 4 + 2] = from_f32<T>(a.scale * fmaf(alpha, sq.z, qk * u.z));
        o[cg * 4 + 3] = from_f32<T>(a.scale * fmaf(alpha, sq.w, qk * u.w));
    }
}

template <typename T, int DK>
cudaError_t launch_delta_dk(const DeltaArgs &a, int cols, cudaStream_t s) {
    void (*kernel)(DeltaArgs) = cols == 32 ? delta_step_kernel<T, DK, 32>
                              : cols == 64 ? delta_step_kernel<T, DK, 64> : delta_step_kernel<T, DK, 128>;
    return launch_dependent(kernel, dim3((unsigned)(a.units * (a.dv / cols))), dim3(kDeltaThreads), 0, s, a);
}

template <typename T>
cudaError_t launch_delta(const DeltaArgs &a, cudaStream_t s) {
    int cols = a.dv;
    while (cols > 32 && a.units * (a.dv / cols) < 2ll * device_sm_count()) cols >>= 1;
    return a.dk == 32 ? launch_delta_dk<T, 32>(a, cols, s)
         : a.dk == 64 ? launch_delta_dk<T, 64>(a, cols, s) : launch_delta_dk<T, 128>(a, cols, s);
}

}  // namespace

}  // namespace gdn

extern "C" gdn_status gdn_delta_step(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                     int64_t v_stride, const float *g, const float *beta, float *state, const int32_t *state_indices, int n_states, float scale,
                                     int qk_l2norm, int N, int H, int dk, int dv, gdn_dtype dtype, void *o,
                                     gdn_stream_t stream) {
    using namespace gdn;
    const auto head = [](int d) { return d == 32 || d == 64 || d == 128; };
    if (N < 0 || H < 1 || n_states < 0 || (!state_indices && n_states < N)) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    if (!head(dk) || !head(dv)) return GDN_ERR_UNSUPPORTED;
    if ((long long)N * H > (1ll << 28)) return GDN_ERR_UNSUPPORTED;
    if (N == 0) return GDN_OK;
    if (!q || !k || !v || !g || !beta || !state || !o) return GDN_ERR_INVALID_ARG;
    if (q_stride < (int64_t)H * dk || k_stride < (int64_t)H * dk || v_stride < (int64_t)H * dv) return GDN_ERR_INVALID_ARG;
    const uintptr_t em = dtype == GDN_F32 ? 3 : 1;
    const void *elems[] = {q, k, v, o}, *f32[] = {g, beta, state_indices};
    for (const void *p : elems)
        if (reinterpret_cast<uintptr_t>(p) & em) return GDN_ERR_INVALID_ARG;
    for (const void *p : f32)
        if (reinterpret_cast<uintptr_t>(p) & 3) return GDN_ERR_INVALID_ARG;
    if (!aligned16(state)) return GDN_ERR_INVALID_ARG;
    DeltaArgs a = {};
    a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.state = state, a.slots = state_indices, a.o = o;
    a.H = H, a.dk = dk, a.dv = dv, a.pool = n_states, a.l2norm = qk_l2norm != 0;
    a.units = (long long)N * H, a.q_token = q_stride, a.k_token = k_stride, a.v_token = v_stride;
    a.scale = scale > 0.f ? scale : 1.f / sqrtf((float)dk);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == GDN_BF16 ? launch_delta<__nv_bfloat16>(a, s) : launch_delta<float>(a, s);
    if (e != cudaSuccess) {
        set_error_detail("launch delta_step", e);
        return GDN_ERR_CUDA;
    }
    return GDN_OK;
}
