// Few tokens through the feed-forward block: every row of the weights times up to 16
// tokens (8 where the weights are large; fp32: 32), bound by the weights' bytes (4096 x 12288 bf16: 45 us at the measured
// copy rate, fp32 90).
//
// One token: a group of one to eight warps owns two rows of weights, the gate's and the
// projection's of one h, or two of w_down, and reads them once in 16-byte vectors, eight
// in flight per thread; sums in fp32 on pairs.  49 us (fp32 91).
//
// More tokens: with each token's vector loaded and converted again for every pair of rows
// that form took 62, 88 and 174 us for 2, 4 and 8 tokens, so these run on the warp-level
// tensor instructions, whose rate (unlike that of tcgen05, which would want tiles in shared
// memory and 128 rows a tile) is above what the bytes ask for.  A block owns 16 rows of
// w_gate and of w_up, or of w_down, its eight warps take turns along K.  The order of K
// within a product is free as long as both operands share it, so a lane's 16-byte vector of
// a row is its part of two instructions' fragments: no shuffles, no shared memory, tokens
// come from L1.  2 to 8 tokens 50 us; 16 would take 66, so from nine on the tiles of ffn_gemm.cuh
// take over (57 us), but for weights of up to 134 MB (4096 x 1024: 16 tokens 9.4 of 3.8).  Beyond
// 16 the tokens no longer fit L1 (32: 159 us, on tiles 58; small blocks 18).  fp32 is split into three bf16 terms a value, six products: 122 us for 2, 173
// for 16, 305 for 32 tokens, where laying the weights out for tiles takes 490; (errors
// against 64 bits 7e-7 and less, as of products in fp32).
//
// h is rounded to the activations' type here too, so that a token's h does not depend on how
// many come with it.
//
// The second product's blocks start while the first one's last are at work.
#include <algorithm>

#include "ffn_few.cuh"
#include "ffn_gemm.cuh"

namespace gdn {
namespace ffn {
namespace {

constexpr int kFewThreads = 256;

template <typename T, int V, bool UP>
__global__ void __launch_bounds__(kFewThreads, 4) ffn_one_kernel(const FewArgs a) {
    constexpr int U = V > 1 ? 4 : 8, NP = (V + 1) / 2;
    __shared__ float red[kFewThreads / 32][2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = kFewThreads / 32 / a.wpr, slice = warp % a.wpr;
    const long long unit = (long long)blockIdx.x * per + warp / a.wpr;
    const long long r0 = UP ? unit : 2 * unit;
    const int live = r0 >= a.rows ? 0 : UP || r0 + 1 < a.rows ? 2 : 1;   // rows that exist
    // a row that does not exist is read as row 0
    const T *w0 = static_cast<const T *>(a.w0) + (live > 0 ? r0 * a.K : 0);
    const T *w1 = UP ? static_cast<const T *>(a.w1) + (live > 0 ? r0 * a.K : 0) : static_cast<const T *>(a.w0) + (live > 1 ? (r0 + 1) * a.K : 0);
    const int K = (int)a.K, step = 32 * V * a.wpr;
    int k = (slice * 32 + lane) * V;
    Raw<T, V> p[U], q[U];
    auto load = [&]() {
#pragma unroll
        for (int u = 0; u < U; ++u) p[u] = load_raw<T, V>(w0 + k + u * step), q[u] = load_raw<T, V>(w1 + k + u * step);
    };
    // The second product's blocks start while the first one's last are at work (below),
    // and their weights are not that kernel's output: they set out for them at once.
    bool full = live && k + (U - 1) * step < K, loaded = false;
    if (!UP && full) load(), loaded = true;
    grid_dependency_wait();
    if (UP) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const T *x = static_cast<const T *>(a.x);
    F2 acc[2] = {both(0.f), both(0.f)};
    auto add = [&](const Raw<T, V> &ra, const Raw<T, V> &rb, int at) {
        F2 f[NP], g[NP], t[NP];
        unpack_pairs<T, V>(ra, f);
        unpack_pairs<T, V>(rb, g);
        unpack_pairs<T, V>(load_raw<T, V>(x + at), t);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            acc[0] = fma2(f[i], t[i], acc[0]);
            acc[1] = fma2(g[i], t[i], acc[1]);
        }
    };
    while (full) {
        if (!loaded) load();
        loaded = false;
#pragma unroll
        for (int u = 0; u < U; ++u) add(p[u], q[u], k + u * step);
        k += U * step;
        full = k + (U - 1) * step < K;
    }
    if (live)
        for (; k < K; k += step) add(load_raw<T, V>(w0 + k), load_raw<T, V>(w1 + k), k);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float s = warp_sum(lo(acc[i]) + hi(acc[i]));
        if (lane == 0) red[warp][i] = s;
    }
    __syncthreads();
    const int u = threadIdx.x;   // a thread per unit
    if (u >= per) return;
    const long long mine = (long long)blockIdx.x * per + u, row = UP ? mine : 2 * mine;
    float s[2] = {0.f, 0.f};
    for (int w = 0; w < a.wpr; ++w) s[0] += red[u * a.wpr + w][0], s[1] += red[u * a.wpr + w][1];
    if (row >= a.rows) return;
    T *out = static_cast<T *>(a.out) + row;
    if constexpr (UP) {
        if (a.gate) {
            static_cast<T *>(a.gate)[row] = from_f32<T>(s[0]);
            static_cast<T *>(a.up)[row] = from_f32<T>(s[1]);
        }
        out[0] = from_f32<T>(act_times(s[0], s[1], a.act));
    } else {
        out[0] = from_f32<T>(s[0]);
        if (row + 1 < a.rows) out[1] = from_f32<T>(s[1]);
    }
}

// d += a b: 16 rows x 8 tokens, 16 of K.
__device__ __forceinline__ void mma_step(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four fp32 values as three bf16 terms each, two values to a register.
__device__ __forceinline__ void split_pairs(const uint32_t (&x)[4], uint32_t (&p)[3][2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float v0 = __uint_as_float(x[2 * i]), v1 = __uint_as_float(x[2 * i + 1]);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            p[k][i] = tc::pack_bf16x2(v0, v1);
            v0 -= tc::bf16_lo(p[k][i]), v1 -= tc::bf16_hi(p[k][i]);
        }
    }
}

// Up to 8 NT tokens; SETS of 16 rows: w_gate's and w_up's, or w_down's.
template <typename T, int NT, bool VEC, bool UP>
__global__ void __launch_bounds__(kFewThreads, sizeof(T) == 4 && NT == 4 ? 2 : 3) ffn_few_kernel(const FewArgs a) {
    constexpr int V = 16 / (int)sizeof(T), KC = 4 * V, SETS = UP ? 2 : 1, U = UP ? 2 : 4, WARPS = kFewThreads / 32;
    constexpr bool F32 = sizeof(T) == 4;
    __shared__ float red[WARPS][SETS][16][9];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gi = lane >> 2, ti = lane & 3;
    const int K = (int)a.K;
    const long long r0 = (long long)blockIdx.x * 16;
    // rows and tokens that do not exist are read as the last ones, and their results left
    const T *w[SETS][2];
#pragma unroll
    for (int i = 0; i < SETS; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            w[i][h] = static_cast<const T *>(i ? a.w1 : a.w0) + min(r0 + gi + 8 * h, (long long)a.rows - 1) * a.K;
    const T *x[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) x[j] = static_cast<const T *>(a.x) + min(8 * j + gi, a.M - 1) * a.x_stride;
    // 16 bytes of a row from k on, zero past its end
    auto vector = [&](const T *row, int k) {
        if constexpr (VEC) return k < K ? load_raw<T, V>(row + k) : zero_raw<T, V>();
        else return load_some<T, V>(row + (k < K ? k : 0), K - k);
    };
    Raw<T, V> p[U][SETS][2];
    auto load = [&](int k) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < SETS; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) p[u][i][h] = vector(w[i][h], k + u * WARPS * KC);
    };
    int k = warp * KC + ti * V;
    // The second product's blocks start while the first one's last are at work, and their
    // weights are not that kernel's output: they set out for them at once.
    if (!UP) load(k);
    grid_dependency_wait();
    if (UP) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    float d[SETS][NT][4], total[F32 ? SETS : 1][F32 ? NT : 1][4];
#pragma unroll
    for (int i = 0; i < SETS; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[i][j][e] = total[F32 ? i : 0][F32 ? j : 0][e] = 0.f;
    for (bool loaded = !UP; k - ti * V < K; k += U * WARPS * KC, loaded = false) {
        if (!loaded) load(k);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = k + u * WARPS * KC;
            uint32_t t[F32 ? SETS : 1][2][3][2];
            if constexpr (F32) {
#pragma unroll
                for (int i = 0; i < SETS; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) split_pairs(p[u][i][h].w, t[i][h]);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const Raw<T, V> b = vector(x[j], at);
                if constexpr (F32) {
                    uint32_t tb[3][2];
                    split_pairs(b.w, tb);
#pragma unroll
                    for (int i = 0; i < SETS; ++i)
#pragma unroll
                        for (int sum = 2; sum >= 0; --sum)   // the terms x_v y_(sum - v), smallest first
#pragma unroll
                            for (int v = sum; v >= 0; --v)
                                mma_step(d[i][j], t[i][0][v][0], t[i][1][v][0], t[i][0][v][1], t[i][1][v][1], tb[sum - v][0], tb[sum - v][1]);
                } else {
#pragma unroll
                    for (int i = 0; i < SETS; ++i) {
                        const uint32_t *g0 = p[u][i][0].w, *g1 = p[u][i][1].w;
#pragma unroll
                        for (int e = 0; e < 4; e += 2) mma_step(d[i][j], g0[e], g1[e], g0[e + 1], g1[e + 1], b.w[e], b.w[e + 1]);
                    }
                }
            }
        }
        // the tensor instructions cut what an addition leaves over, so their sums are short
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < SETS; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) total[i][j][e] += d[i][j][e], d[i][j][e] = 0.f;
        }
    }
    if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < SETS; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) d[i][j][e] = total[i][j][e];
    }
    // the warps' sums, in order, eight tokens at a time
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        if (8 * j >= a.M) break;
        if (j) __syncthreads();
#pragma unroll
        for (int i = 0; i < SETS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) red[warp][i][gi + 8 * (e >> 1)][2 * ti + (e & 1)] = d[i][j][e];
        __syncthreads();
        const int row = threadIdx.x & 15, m = 8 * j + (threadIdx.x >> 4);
        if (threadIdx.x < 128 && m < a.M && r0 + row < a.rows) {
            float s[SETS];
#pragma unroll
            for (int i = 0; i < SETS; ++i) {
                s[i] = 0.f;
#pragma unroll
                for (int v = 0; v < WARPS; ++v) s[i] += red[v][i][row][threadIdx.x >> 4];
            }
            if constexpr (UP) {
                const long long at = (long long)m * a.rows + r0 + row;
                if (a.gate) static_cast<T *>(a.gate)[at] = from_f32<T>(s[0]), static_cast<T *>(a.up)[at] = from_f32<T>(s[SETS - 1]);
                s[0] = act_times(s[0], s[SETS - 1], a.act);
            }
            static_cast<T *>(a.out)[m * a.out_ld + r0 + row] = from_f32<T>(s[0]);
        }
    }
}

template <typename T, bool VEC, bool UP>
cudaError_t launch_v(const FewArgs &args, cudaStream_t s) {
    FewArgs a = args;
    if (a.M == 1) {
        // warps per unit: as few as fill the GPU (24 warps an SM hold the memory's latency)
        const long long units = UP ? a.rows : (a.rows + 1) / 2;
        a.wpr = 1;
        while (a.wpr < 8 && units * a.wpr < 24ll * device_sm_count()) a.wpr *= 2;
        const long long per = kFewThreads / 32 / a.wpr;
        return launch_dependent(ffn_one_kernel<T, VEC ? 16 / (int)sizeof(T) : 1, UP>, dim3((unsigned)((units + per - 1) / per)), dim3(kFewThreads), 0, s, a);
    }
    void (*kernel)(const FewArgs) = a.M <= 8 ? ffn_few_kernel<T, 1, VEC, UP> : ffn_few_kernel<T, 2, VEC, UP>;
    if constexpr (sizeof(T) == 4)
        if (a.M > 16) kernel = ffn_few_kernel<T, 4, VEC, UP>;
    return launch_dependent(kernel, dim3((unsigned)((a.rows + 15) / 16)), dim3(kFewThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_few(const FewArgs &a, bool up, bool f32, bool vec, cudaStream_t s) {
    if (f32) return up ? (vec ? launch_v<float, true, true>(a, s) : launch_v<float, false, true>(a, s))
                       : (vec ? launch_v<float, true, false>(a, s) : launch_v<float, false, false>(a, s));
    return up ? (vec ? launch_v<__nv_bfloat16, true, true>(a, s) : launch_v<__nv_bfloat16, false, true>(a, s))
              : (vec ? launch_v<__nv_bfloat16, true, false>(a, s) : launch_v<__nv_bfloat16, false, false>(a, s));
}

}  // namespace ffn
}  // namespace gdn
