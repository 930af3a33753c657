// What lies between two blocks of a layer, in one pass, forward and backward:
//
//     n = y rstd_post w_post,          rstd_post = (sum y^2 / D + eps)^-1/2,
//     x = r + s n a(z),                a(z) = z sigmoid(z), or sigmoid(z),
//     h = x rstd_pre w_pre,            rstd_pre = (sum x^2 / D + eps)^-1/2,
//
// of which the first norm, the gate z, the scale s, the residual r and the second
// norm may each be left out; and, for upstream gradients dx and dh,
//
//     d  = dx + rstd_pre (g - xh sum g xh / D),       g = dh w_pre, xh = x rstd_pre,
//     dr = d,   dz = d s n a'(z),
//     dy = rstd_post (e - yh sum e yh / D),           e = d s a(z) w_post, yh = y rstd_post,
//     dw_pre = sum_rows dh xh,   P = sum_rows d a(z) yh,   dw_post = s P,   ds = w_post P.
//
// Statistics and h are taken from x before it is rounded.  Both passes are streams
// bound by HBM: every tensor is read once and written once (five tensors forward,
// eight backward).  A row is held by 8 to 1024 threads, 8 or 16 columns each; the
// blocks are persistent and own their columns, so the parameters and the sums P and
// dw_pre stay in registers over all rows of a block.  The next rows come in by
// asynchronous copies; what is needed twice is read again from those copies instead
// of being held.  The blocks' sums leave as partial rows that a second kernel adds in
// a fixed order.
//
// Measured (all parts, fp32 parameters; of the measured copy rate): 32768 x 4096 bf16
// forward 201 us, backward 321 (both 100%); 2^27 elements of 8192 columns 236 and 365, of
// 1024 210 and 326, of 256 245 and 372; fp32 4096 columns (16384 rows) 227 and 361.  The
// gated norm of 16384 x 32 heads of 128 62 us (97%), its backward pass on 8191 x 32 58 (86%,
// 4 of it the sum over the blocks).  Rows that are not 16-byte aligned come in the 16-byte
// chunks they touch and leave element by element: 32776 x 4095 bf16 363 and 648 us, fp32
// (16388) 230 and 459.  Rows wider than 8192 columns are read two or three times: 8192 x
// 16384 bf16 489 and 905 us.  16 rows 5.4 us (a call takes 28 to 32, on the host).
#include <algorithm>
#include <type_traits>

#include "elem.cuh"

namespace gdn {
namespace {

// Rows [outer][inner]: row i starts at (i / inner) so + (i % inner) si elements.  From
// a row to the one `step` rows on it is `ahead` elements, and `wrap` more where the inner
// index passes its end.
struct View {
    const void *p;
    long long so, si, ahead, wrap;
    const void *end;          // past the last row
};
struct BlockNormArgs {
    View y, z, r, dx, dh;             // r: the residual, or x in the backward pass
    void *x, *h, *dy, *dr, *dz;       // outputs, contiguous
    const void *w_post, *w_pre, *scale;
    float *rstd_post, *rstd_pre;
    float *partial;                   // [grid][P, dw_pre][D] or null
    long long rows;
    uint32_t inner, magic, shift;     // division by inner
    uint32_t inner_step;              // of a block's step from row to row
    int D, w_f32, post, pre, gate, res;   // gate: 0 none, 1 silu, 2 sigmoid
    float eps;
};

__device__ __forceinline__ long long row_at(const BlockNormArgs &a, const View &v, long long row) {
    if (a.inner == 1) return row * v.so;
    const uint32_t n = (uint32_t)row, q = (__umulhi(a.magic, n) + n) >> a.shift;
    return (long long)q * v.so + (long long)(n - q * a.inner) * v.si;
}
__device__ __forceinline__ uint32_t inner_of(const BlockNormArgs &a, long long row) {
    if (a.inner == 1) return 0u;
    const uint32_t n = (uint32_t)row;
    return n - ((__umulhi(a.magic, n) + n) >> a.shift) * a.inner;
}
__device__ __forceinline__ float param_at(const void *p, int i, int f32) {
    return f32 ? static_cast<const float *>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

// Sum over the TPR threads of a row.  Each use takes the other of the two arrays: who
// writes one again has passed the barrier of the use in between, by which all have
// read it.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (*both_red)[32], int &phase) {
    float *red = both_red[phase];
    phase ^= 1;
#pragma unroll
    for (int off = (TPR < 32 ? TPR : 32) / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) v += red[i];
    }
    return v;
}

constexpr int bn_threads(int tpr) { return tpr <= 32 ? 256 : tpr; }

// Rows in flight per row of threads: as many as a block's share of shared memory holds,
// at most MOST; a single one where not even two fit.  Blocks per SM that the registers are
// budgeted for: THREADS threads.
template <typename T, int TPR, int VEC, int NV, int ARRAYS, int THREADS, int MOST>
struct BnStages {
    // Vectors: each thread reads back what it copied.  Else a row comes as the 16-byte
    // chunks that it touches, and its threads read from all of them.
    static constexpr bool async = VEC * sizeof(T) == 16;
    static constexpr int row_bytes = TPR * NV * VEC * (int)sizeof(T) + 16;
    static constexpr int bytes = async ? bn_threads(TPR) * NV * ARRAYS * 16 : bn_threads(TPR) / TPR * ARRAYS * row_bytes;
    static constexpr int by_threads = THREADS >= bn_threads(TPR) ? THREADS / bn_threads(TPR) : 1;
    static constexpr int fit = (225 * 1024 / by_threads - 1024) / bytes;
    static constexpr int count = fit >= MOST ? MOST : fit >= 2 ? fit : 2 * bytes <= 224 * 1024 ? 2 : 1;
    static constexpr int smem = count * bytes;
    static constexpr int by_smem = 225 * 1024 / (smem + 1024);
    static constexpr int blocks = by_smem < by_threads ? by_smem : by_threads;
    static_assert(smem <= 226 * 1024 && blocks >= 1, "shared memory");
};

__device__ __forceinline__ void bn_copy16(uint4 *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

// More rows in flight than these are slower, not only useless (forward, 2^27 elements in
// bf16, all parts: 2048 columns 208 us with two rows, 225 with three or four, 1024 columns 210
// and 243; the gated norm of heads 127 with three, 132 with four, 137 with two; backward, 256
// columns 371 with two, 390 with four, 2048 columns 362 and 374), and so are more threads of
// fewer registers (backward, 1024 columns 326 us at 640 threads, 365 at 768).
template <typename T, int TPR, int VEC, int NV>
using FwdStages = BnStages<T, TPR, VEC, NV, 3, (TPR >= 512 ? 1024 : 768), (TPR >= 128 ? 2 : 3)>;
template <typename T, int TPR, int VEC, int NV, bool PRE>
using BwdStages = BnStages<T, TPR, VEC, NV, PRE ? 5 : 3, (NV * VEC > 8 ? 512 : PRE && TPR >= 128 ? 640 : 768), (PRE ? 2 : 4)>;

// The threads of a row, which read what any of them copied.
template <int TPR>
__device__ __forceinline__ void row_sync() {
    if constexpr (TPR > 32) __syncthreads();
    else __syncwarp();
}
// Copies the 16-byte chunks that a row of D elements at src touches; of chunks that reach
// past the tensor's ends its elements only.
template <typename T, int TPR>
__device__ __forceinline__ void window_copy(uint8_t *dst, const T *src, const View &v, int D, int t) {
    const uintptr_t first = reinterpret_cast<uintptr_t>(src) & ~(uintptr_t)15, lo = reinterpret_cast<uintptr_t>(v.p),
                    hi = reinterpret_cast<uintptr_t>(v.end);
    const int n = (int)((reinterpret_cast<uintptr_t>(src + D) - first + 15) >> 4);
    for (int j = t; j < n; j += TPR) {
        const uintptr_t at = first + 16ull * j;
        if (at >= lo && at + 16 <= hi) {
            bn_copy16(reinterpret_cast<uint4 *>(dst + 16 * j), reinterpret_cast<const void *>(at));
        } else {
            for (int b = 0; b < 16; b += (int)sizeof(T)) {
                const T *el = reinterpret_cast<const T *>(at + b);
                if (el >= src && el < src + D) *reinterpret_cast<T *>(dst + 16 * j + b) = *el;
            }
        }
    }
}

// Column of a thread's element e (of NV vectors of VEC, TPR vectors apart).
template <int TPR, int VEC>
__device__ __forceinline__ int col_of(int e, int t) {
    return (e / VEC * TPR + t) * VEC + e % VEC;
}
template <int TPR, int VEC, int NV>
__device__ __forceinline__ void params(const void *p, const void *q, int f32, int D, int t, F2 (&v)[NV * VEC / 2]) {
    float x[NV * VEC];
#pragma unroll
    for (int e = 0; e < NV * VEC; ++e) {
        const int c = col_of<TPR, VEC>(e, t);
        x[e] = 1.f;
        if (c < D && p) x[e] = param_at(p, c, f32);
        if (c < D && q) x[e] *= param_at(q, c, f32);
    }
#pragma unroll
    for (int i = 0; i < NV * VEC / 2; ++i) v[i] = pair(x[2 * i], x[2 * i + 1]);
}

// A thread's part of one array's row, from the copies: its vectors, or its elements of
// the row; zero past the row's end.
template <typename T, int TPR, int VEC, int NV, bool ASYNC>
struct Part {
    const uint4 *at;     // [NV] vectors, NT apart
    const T *row;
    int t, D;
    bool live;
    template <int NT>
    __device__ __forceinline__ void get(F2 (&v)[NV * VEC / 2]) const {
        if constexpr (ASYNC) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const bool in = live && (i * TPR + t) * VEC < D;
                F2 u[VEC / 2];
                unpack_pairs<T, VEC>(in ? load_raw<T, VEC>(reinterpret_cast<const T *>(at + i * NT)) : zero_raw<T, VEC>(), u);
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) v[i * (VEC / 2) + j] = u[j];
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV * VEC / 2; ++i) {
                const int c0 = col_of<TPR, VEC>(2 * i, t), c1 = col_of<TPR, VEC>(2 * i + 1, t);
                v[i] = pair(live && c0 < D ? to_f32(row[c0]) : 0.f, live && c1 < D ? to_f32(row[c1]) : 0.f);
            }
        }
    }
};

template <typename T, int TPR, int VEC, int NV>
__device__ __forceinline__ void put_row(T *row, int D, int t, bool live, const F2 (&v)[NV * VEC / 2]) {
    if (!live) return;
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
            row[c] = from_f32<T>(i & 1 ? hi(v[i / 2]) : lo(v[i / 2]));
        }
    }
}

template <typename T, int TPR, int VEC, int NV>
__global__ void __launch_bounds__(bn_threads(TPR), FwdStages<T, TPR, VEC, NV>::blocks) block_norm_fwd_kernel(const BlockNormArgs a) {
    using St = FwdStages<T, TPR, VEC, NV>;
    constexpr int NT = bn_threads(TPR), RPB = NT / TPR, S = St::count, NP = NV * VEC / 2;
    __shared__ float red[2][32];
    extern __shared__ uint4 stages[];              // [S][y, z, r][NV][thread], or [S][y, z, r][row][chunk]
    uint8_t *const windows = reinterpret_cast<uint8_t *>(stages) + threadIdx.x / TPR * St::row_bytes;
    constexpr int kArray = RPB * St::row_bytes;
    const int t = threadIdx.x % TPR;
    const long long step = (long long)gridDim.x * RPB;
    grid_dependency_wait();
    long long row = (long long)blockIdx.x * RPB + threadIdx.x / TPR;
    const int behind = TPR < 32 ? (threadIdx.x & 31) / TPR : 0;   // rows of a warp go together
    // the rows are loaded in turn: pointers walk instead of being computed
    const T *src[3] = {static_cast<const T *>(a.y.p) + row_at(a, a.y, row), a.gate ? static_cast<const T *>(a.z.p) + row_at(a, a.z, row) : nullptr,
                       a.res ? static_cast<const T *>(a.r.p) + row_at(a, a.r, row) : nullptr};
    uint32_t rem = inner_of(a, row);
    auto load_row = [&](long long r, int slot) {
        if (r < a.rows) {
            if constexpr (St::async) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = (i * TPR + t) * VEC;
                    uint4 *at = stages + (slot * 3 * NV + i) * NT + threadIdx.x;
                    if (c < a.D) {
                        bn_copy16(at, src[0] + c);
                        if (a.gate) bn_copy16(at + NV * NT, src[1] + c);
                        if (a.res) bn_copy16(at + 2 * NV * NT, src[2] + c);
                    }
                }
            } else {
                uint8_t *at = windows + slot * 3 * kArray;
                window_copy<T, TPR>(at, src[0], a.y, a.D, t);
                if (a.gate) window_copy<T, TPR>(at + kArray, src[1], a.z, a.D, t);
                if (a.res) window_copy<T, TPR>(at + 2 * kArray, src[2], a.r, a.D, t);
            }
        }
        copy_commit();
        rem += a.inner_step;
        const bool wrap = rem >= a.inner;
        if (wrap) rem -= a.inner;
        src[0] += a.y.ahead + (wrap ? a.y.wrap : 0);
        src[1] += a.z.ahead + (wrap ? a.z.wrap : 0);
        src[2] += a.r.ahead + (wrap ? a.r.wrap : 0);
    };
    if constexpr (S > 1 || St::async) {
#pragma unroll
        for (int k = 0; k < (S > 1 ? S - 1 : 1); ++k) load_row(row + k * step, k);
    }
    F2 c[NP], wn[NP];
    params<TPR, VEC, NV>(a.w_post, a.scale, a.w_f32, a.D, t, c);
    params<TPR, VEC, NV>(a.w_pre, nullptr, a.w_f32, a.D, t, wn);
    const float inv_d = 1.f / (float)a.D;
    int phase = 0;
    for (int slot = 0; row - behind < a.rows; row += step, slot = slot + 1 == S ? 0 : slot + 1) {
        const bool live = row < a.rows;
        Part<T, TPR, VEC, NV, St::async> y, z, r;
        y.t = z.t = r.t = t, y.D = z.D = r.D = a.D, y.live = z.live = r.live = live;
        if constexpr (St::async) {
            if constexpr (S > 1) load_row(row + (S - 1) * step, slot == 0 ? S - 1 : slot - 1);
            copy_wait<S - 1>();
            y.at = stages + slot * 3 * NV * NT + threadIdx.x;
            z.at = y.at + NV * NT, r.at = z.at + NV * NT;
        } else {
            if constexpr (S == 1) row_sync<TPR>(), load_row(row, 0);
            copy_wait<(S > 1 ? S - 2 : 0)>();
            row_sync<TPR>();   // all have this row, and none reads the last one any more
            if constexpr (S > 1) load_row(row + (S - 1) * step, slot == 0 ? S - 1 : slot - 1);
            const uint8_t *at = windows + slot * 3 * kArray;
            auto place = [&](const View &w, int k) {
                return reinterpret_cast<const T *>(at + k * kArray + ((reinterpret_cast<uintptr_t>(w.p) + row_at(a, w, row) * sizeof(T)) & 15));
            };
            y.row = place(a.y, 0), z.row = place(a.z, 1), r.row = place(a.r, 2);
        }
        F2 v[NP], u[NP];
        y.template get<NT>(v);
        float rstd = 1.f;
        if (a.post) {
            F2 q = mul2(v[0], v[0]);
#pragma unroll
            for (int p = 1; p < NP; ++p) q = fma2(v[p], v[p], q);
            rstd = rsqrtf(row_sum<TPR>(lo(q) + hi(q), red, phase) * inv_d + a.eps);
            if (t == 0 && live) a.rstd_post[row] = rstd;
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) v[p] = mul2(mul2(v[p], both(rstd)), c[p]);
        if (a.gate) {
            z.template get<NT>(u);
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const F2 s = sigmoid_pair(u[p]);
                v[p] = mul2(v[p], a.gate == 1 ? mul2(u[p], s) : s);
            }
        }
        if (a.res) {
            r.template get<NT>(u);
#pragma unroll
            for (int p = 0; p < NP; ++p) v[p] = add2(v[p], u[p]);
        }
        if constexpr (S == 1 && St::async) load_row(row + step, 0);
        put_row<T, TPR, VEC, NV>(static_cast<T *>(a.x) + row * a.D, a.D, t, live, v);
        if (a.pre) {
            F2 q = both(0.f);
#pragma unroll
            for (int p = 0; p < NP; ++p) q = fma2(v[p], v[p], q);
            const float r2 = rsqrtf(row_sum<TPR>(lo(q) + hi(q), red, phase) * inv_d + a.eps);
            if (t == 0 && live) a.rstd_pre[row] = r2;
#pragma unroll
            for (int p = 0; p < NP; ++p) v[p] = mul2(mul2(v[p], both(r2)), wn[p]);
            put_row<T, TPR, VEC, NV>(static_cast<T *>(a.h) + row * a.D, a.D, t, live, v);
        }
    }
}

// PRE: with the second norm (kept apart: without it a third of the registers go).
template <typename T, int TPR, int VEC, int NV, bool PRE>
__global__ void __launch_bounds__(bn_threads(TPR), BwdStages<T, TPR, VEC, NV, PRE>::blocks) block_norm_bwd_kernel(const BlockNormArgs a) {
    using St = BwdStages<T, TPR, VEC, NV, PRE>;
    constexpr int ARR = PRE ? 5 : 3;
    constexpr int NT = bn_threads(TPR), RPB = NT / TPR, S = St::count, NP = NV * VEC / 2;
    __shared__ float red[2][32];
    extern __shared__ uint4 stages[];              // [S][y, z, dx(, dh, x)][NV][thread], or [..][row][chunk]
    uint8_t *const windows = reinterpret_cast<uint8_t *>(stages) + threadIdx.x / TPR * St::row_bytes;
    constexpr int kArray = RPB * St::row_bytes;
    const int t = threadIdx.x % TPR;
    const long long step = (long long)gridDim.x * RPB;
    grid_dependency_wait();
    long long row = (long long)blockIdx.x * RPB + threadIdx.x / TPR;
    const int behind = TPR < 32 ? (threadIdx.x & 31) / TPR : 0;
    const bool has_dx = a.dx.p != nullptr;
    const View *view[5] = {&a.y, &a.z, &a.dx, &a.dh, &a.r};
    const bool there[5] = {true, a.gate != 0, has_dx, true, true};
    const T *src[ARR];
#pragma unroll
    for (int k = 0; k < ARR; ++k) src[k] = static_cast<const T *>(view[k]->p) + (there[k] ? row_at(a, *view[k], row) : 0);
    uint32_t rem = inner_of(a, row);
    auto load_row = [&](long long r, int slot) {
        if (r < a.rows) {
#pragma unroll
            for (int k = 0; k < ARR; ++k) {
                if (!there[k]) continue;
                if constexpr (St::async) {
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const int c = (i * TPR + t) * VEC;
                        if (c < a.D) bn_copy16(stages + ((slot * ARR + k) * NV + i) * NT + threadIdx.x, src[k] + c);
                    }
                } else {
                    window_copy<T, TPR>(windows + (slot * ARR + k) * kArray, src[k], *view[k], a.D, t);
                }
            }
        }
        copy_commit();
        rem += a.inner_step;
        const bool wrap = rem >= a.inner;
        if (wrap) rem -= a.inner;
#pragma unroll
        for (int k = 0; k < ARR; ++k) src[k] += view[k]->ahead + (wrap ? view[k]->wrap : 0);
    };
    if constexpr (S > 1 || St::async) {
#pragma unroll
        for (int k = 0; k < (S > 1 ? S - 1 : 1); ++k) load_row(row + k * step, k);
    }
    F2 c[NP], P[NP], wn[PRE ? NP : 1], Q[PRE ? NP : 1];
    params<TPR, VEC, NV>(a.w_post, a.scale, a.w_f32, a.D, t, c);
    if constexpr (PRE) params<TPR, VEC, NV>(a.w_pre, nullptr, a.w_f32, a.D, t, wn);
#pragma unroll
    for (int p = 0; p < NP; ++p) P[p] = Q[PRE ? p : 0] = both(0.f);
    // a row's rstd is loaded a row ahead (heads 65.5 -> 60.2 us); with the second norm its
    // loads are hidden, and the register is not (324 us, 328 ahead)
    float next_rp = !PRE && a.post && row < a.rows ? a.rstd_post[row] : 1.f;
    const float inv_d = 1.f / (float)a.D;
    int phase = 0;
    for (int slot = 0; row - behind < a.rows; row += step, slot = slot + 1 == S ? 0 : slot + 1) {
        const bool live = row < a.rows;
        const float rp = !PRE ? next_rp : a.post && live ? a.rstd_post[row] : 1.f, rn = PRE && live ? a.rstd_pre[row] : 1.f;
        if (!PRE && a.post && row + step < a.rows) next_rp = a.rstd_post[row + step];
        Part<T, TPR, VEC, NV, St::async> part[ARR];
#pragma unroll
        for (int k = 0; k < ARR; ++k) part[k].t = t, part[k].D = a.D, part[k].live = live;
        if constexpr (St::async) {
            if constexpr (S > 1) load_row(row + (S - 1) * step, slot == 0 ? S - 1 : slot - 1);
            copy_wait<S - 1>();
#pragma unroll
            for (int k = 0; k < ARR; ++k) part[k].at = stages + (slot * ARR + k) * NV * NT + threadIdx.x;
        } else {
            if constexpr (S == 1) row_sync<TPR>(), load_row(row, 0);
            copy_wait<(S > 1 ? S - 2 : 0)>();
            row_sync<TPR>();   // all have this row, and none reads the last one any more
            if constexpr (S > 1) load_row(row + (S - 1) * step, slot == 0 ? S - 1 : slot - 1);
#pragma unroll
            for (int k = 0; k < ARR; ++k)
                part[k].row = reinterpret_cast<const T *>(windows + (slot * ARR + k) * kArray +
                                                          ((reinterpret_cast<uintptr_t>(view[k]->p) + row_at(a, *view[k], row) * sizeof(T)) & 15));
        }
        F2 d[NP], u[NP], v[NP];
        if constexpr (PRE) {
            part[3].template get<NT>(u);
            part[4].template get<NT>(v);
            F2 q = both(0.f);
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                v[p] = mul2(v[p], both(rn));
                Q[p] = fma2(u[p], v[p], Q[p]);
                u[p] = mul2(u[p], wn[p]);
                q = fma2(u[p], v[p], q);
            }
            const float m = row_sum<TPR>(lo(q) + hi(q), red, phase) * inv_d;
#pragma unroll
            for (int p = 0; p < NP; ++p) d[p] = mul2(fma2(v[p], both(-m), u[p]), both(rn));
            if (has_dx) {
                part[2].template get<NT>(u);
#pragma unroll
                for (int p = 0; p < NP; ++p) d[p] = add2(d[p], u[p]);
            }
        } else {
            part[2].template get<NT>(d);
        }
        if (a.dr) put_row<T, TPR, VEC, NV>(static_cast<T *>(a.dr) + row * a.D, a.D, t, live, d);
        part[0].template get<NT>(v);
#pragma unroll
        for (int p = 0; p < NP; ++p) v[p] = mul2(v[p], both(rp));      // yh
        if (a.gate) {
            part[1].template get<NT>(u);
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const F2 s = sigmoid_pair(u[p]), one = fma2(s, both(-1.f), both(1.f));   // 1 - s
                const F2 g = a.gate == 1 ? mul2(u[p], s) : s;                              // a(z)
                const F2 slope = a.gate == 1 ? fma2(g, one, s) : mul2(s, one);             // a'(z)
                const F2 dc = mul2(d[p], c[p]);
                P[p] = fma2(mul2(d[p], g), v[p], P[p]);
                u[p] = mul2(mul2(dc, v[p]), slope);
                d[p] = mul2(dc, g);
            }
            put_row<T, TPR, VEC, NV>(static_cast<T *>(a.dz) + row * a.D, a.D, t, live, u);
        } else {
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                P[p] = fma2(d[p], v[p], P[p]);
                d[p] = mul2(d[p], c[p]);
            }
        }
        if constexpr (S == 1 && St::async) load_row(row + step, 0);
        if (a.post) {
            F2 q = both(0.f);
#pragma unroll
            for (int p = 0; p < NP; ++p) q = fma2(d[p], v[p], q);
            const float m = row_sum<TPR>(lo(q) + hi(q), red, phase) * inv_d;
#pragma unroll
            for (int p = 0; p < NP; ++p) d[p] = mul2(fma2(v[p], both(-m), d[p]), both(rp));
        }
        put_row<T, TPR, VEC, NV>(static_cast<T *>(a.dy) + row * a.D, a.D, t, live, d);
    }
    if (!a.partial) return;
    float *pp = a.partial + 2ll * blockIdx.x * a.D, *pq = pp + a.D;
    if constexpr (RPB == 1) {
#pragma unroll
        for (int e = 0; e < NV * VEC; ++e) {
            const int col = col_of<TPR, VEC>(e, t);
            if (col < a.D) {
                pp[col] = e & 1 ? hi(P[e / 2]) : lo(P[e / 2]);
                if constexpr (PRE) pq[col] = e & 1 ? hi(Q[e / 2]) : lo(Q[e / 2]);
            }
        }
    } else {
        // the sums of the block's rows of threads, in order
        constexpr int COLS = TPR * NV * VEC;
        __shared__ float sum[PRE ? 2 : 1][COLS];
        for (int r = 0; r < RPB; ++r) {
            if ((int)threadIdx.x / TPR == r) {
#pragma unroll
                for (int e = 0; e < NV * VEC; ++e) {
                    const int col = col_of<TPR, VEC>(e, t);
                    sum[0][col] = (r ? sum[0][col] : 0.f) + (e & 1 ? hi(P[e / 2]) : lo(P[e / 2]));
                    if constexpr (PRE) sum[1][col] = (r ? sum[1][col] : 0.f) + (e & 1 ? hi(Q[e / 2]) : lo(Q[e / 2]));
                }
            }
            __syncthreads();
        }
        for (int col = threadIdx.x; col < a.D; col += blockDim.x) {
            pp[col] = sum[0][col];
            if constexpr (PRE) pq[col] = sum[1][col];
        }
    }
}

// Rows wider than the register-resident kernels take: a block per row, which it reads
// twice or three times (the later ones mostly from L2), V columns a thread at a time.
template <typename T, int V>
__device__ __forceinline__ void wide_load(const T *row, int c, float (&v)[V]) {
    unpack<T, V>(load_raw<T, V>(row + c), v);
}
template <int V>
__device__ __forceinline__ void wide_param(const void *p, int f32, int c, float (&v)[V], bool times) {
    float w[V];
    if (p && f32 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {   // V columns: V > 1 in rows of a multiple of V
        wide_load<float, V>(static_cast<const float *>(p), c, w);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) w[e] = p ? param_at(p, c + e, f32) : 1.f;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = times ? v[e] * w[e] : w[e];
}
template <typename T, int V>
__global__ void __launch_bounds__(1024) block_norm_wide_fwd_kernel(const BlockNormArgs a) {
    __shared__ float red[2][32];
    const float inv_d = 1.f / (float)a.D;
    int phase = 0;
    grid_dependency_wait();
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *y = static_cast<const T *>(a.y.p) + row_at(a, a.y, row);
        const T *z = a.gate ? static_cast<const T *>(a.z.p) + row_at(a, a.z, row) : nullptr;
        const T *r = a.res ? static_cast<const T *>(a.r.p) + row_at(a, a.r, row) : nullptr;
        float rstd = 1.f, q = 0.f;
        if (a.post) {
            for (int c = threadIdx.x * V; c < a.D; c += 1024 * V) {
                float v[V];
                wide_load<T, V>(y, c, v);
#pragma unroll
                for (int e = 0; e < V; ++e) q = fmaf(v[e], v[e], q);
            }
            rstd = rsqrtf(row_sum<1024>(q, red, phase) * inv_d + a.eps);
            if (threadIdx.x == 0) a.rstd_post[row] = rstd;
        }
        auto value = [&](int c, float (&v)[V]) {
            float t[V];
            wide_load<T, V>(y, c, v);
            wide_param<V>(a.w_post, a.w_f32, c, v, true);
            wide_param<V>(a.scale, a.w_f32, c, v, true);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] *= rstd;
            if (a.gate) {
                wide_load<T, V>(z, c, t);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float s = sigmoid_f32(t[e]);
                    v[e] *= a.gate == 1 ? t[e] * s : s;
                }
            }
            if (a.res) {
                wide_load<T, V>(r, c, t);
#pragma unroll
                for (int e = 0; e < V; ++e) v[e] += t[e];
            }
        };
        float r2 = 1.f;
        if (a.pre) {
            q = 0.f;
            for (int c = threadIdx.x * V; c < a.D; c += 1024 * V) {
                float v[V];
                value(c, v);
#pragma unroll
                for (int e = 0; e < V; ++e) q = fmaf(v[e], v[e], q);
            }
            r2 = rsqrtf(row_sum<1024>(q, red, phase) * inv_d + a.eps);
            if (threadIdx.x == 0) a.rstd_pre[row] = r2;
        }
        for (int c = threadIdx.x * V; c < a.D; c += 1024 * V) {   // x may be the memory of y, z or r: written last
            float v[V];
            value(c, v);
            store_raw<T, V>(static_cast<T *>(a.x) + row * a.D + c, pack<T, V>(v));
            if (a.pre) {
                wide_param<V>(a.w_pre, a.w_f32, c, v, true);
#pragma unroll
                for (int e = 0; e < V; ++e) v[e] *= r2;
                store_raw<T, V>(static_cast<T *>(a.h) + row * a.D + c, pack<T, V>(v));
            }
        }
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(1024) block_norm_wide_bwd_kernel(const BlockNormArgs a) {
    __shared__ float red[2][32];
    const float inv_d = 1.f / (float)a.D;
    int phase = 0;
    float *pp = a.partial ? a.partial + 2ll * blockIdx.x * a.D : nullptr;
    grid_dependency_wait();
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *y = static_cast<const T *>(a.y.p) + row_at(a, a.y, row);
        const T *z = a.gate ? static_cast<const T *>(a.z.p) + row_at(a, a.z, row) : nullptr;
        const T *dx = a.dx.p ? static_cast<const T *>(a.dx.p) + row_at(a, a.dx, row) : nullptr;
        const T *dh = a.pre ? static_cast<const T *>(a.dh.p) + row_at(a, a.dh, row) : nullptr;
        const T *x = a.pre ? static_cast<const T *>(a.r.p) + row_at(a, a.r, row) : nullptr;
        const float rp = a.post ? a.rstd_post[row] : 1.f, rn = a.pre ? a.rstd_pre[row] : 1.f;
        float m = 0.f, q = 0.f;
        if (a.pre) {
            for (int c = threadIdx.x * V; c < a.D; c += 1024 * V) {
                float g[V], t[V];
                wide_load<T, V>(dh, c, g);
                wide_load<T, V>(x, c, t);
                wide_param<V>(a.w_pre, a.w_f32, c, g, true);
#pragma unroll
                for (int e = 0; e < V; ++e) q = fmaf(g[e], t[e] * rn, q);
            }
            m = row_sum<1024>(q, red, phase) * inv_d;
        }
        // d, d's part of P (d a yh), dh xh; e = d s a w_post, dz
        auto value = [&](int c, float (&d)[V], float (&yh)[V], float (&e)[V], float (&dz)[V], float (&p)[V], float (&qq)[V]) {
            float t[V], w[V];
#pragma unroll
            for (int i = 0; i < V; ++i) d[i] = 0.f, qq[i] = 0.f;
            if (dx) wide_load<T, V>(dx, c, d);
            if (a.pre) {
                float g[V];
                wide_load<T, V>(dh, c, g);
                wide_load<T, V>(x, c, t);
                wide_param<V>(a.w_pre, a.w_f32, c, w, false);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float xh = t[i] * rn;
                    qq[i] = g[i] * xh;
                    d[i] += rn * (g[i] * w[i] - xh * m);
                }
            }
            wide_load<T, V>(y, c, yh);
            wide_param<V>(a.w_post, a.w_f32, c, w, false);
            wide_param<V>(a.scale, a.w_f32, c, w, true);
            if (a.gate) wide_load<T, V>(z, c, t);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                yh[i] *= rp;
                float act = 1.f, slope = 0.f;
                if (a.gate) {
                    const float s = sigmoid_f32(t[i]);
                    act = a.gate == 1 ? t[i] * s : s;
                    slope = a.gate == 1 ? fmaf(act, 1.f - s, s) : s * (1.f - s);
                }
                const float dc = d[i] * w[i];
                p[i] = d[i] * act * yh[i], dz[i] = dc * yh[i] * slope, e[i] = dc * act;
            }
        };
        float m2 = 0.f;
        if (a.post) {
            q = 0.f;
            for (int c = threadIdx.x * V; c < a.D; c += 1024 * V) {
                float d[V], yh[V], e[V], dz[V], p[V], qq[V];
                value(c, d, yh, e, dz, p, qq);
#pragma unroll
                for (int i = 0; i < V; ++i) q = fmaf(e[i], yh[i], q);
            }
            m2 = row_sum<1024>(q, red, phase) * inv_d;
        }
        for (int c = threadIdx.x * V; c < a.D; c += 1024 * V) {
            float d[V], yh[V], e[V], dz[V], p[V], qq[V];
            value(c, d, yh, e, dz, p, qq);
            if (a.dr) store_raw<T, V>(static_cast<T *>(a.dr) + row * a.D + c, pack<T, V>(d));
            if (a.gate) store_raw<T, V>(static_cast<T *>(a.dz) + row * a.D + c, pack<T, V>(dz));
#pragma unroll
            for (int i = 0; i < V; ++i) e[i] = rp * (e[i] - yh[i] * m2);
            store_raw<T, V>(static_cast<T *>(a.dy) + row * a.D + c, pack<T, V>(e));
            if (pp) {   // the block's sums, in its partial row (L2)
                if (row != blockIdx.x) {
                    float t[V];
                    wide_load<float, V>(pp, c, t);
#pragma unroll
                    for (int i = 0; i < V; ++i) p[i] += t[i];
                    wide_load<float, V>(pp + a.D, c, t);
#pragma unroll
                    for (int i = 0; i < V; ++i) qq[i] += t[i];
                }
                store_raw<float, V>(pp + c, pack<float, V>(p));
                store_raw<float, V>(pp + a.D + c, pack<float, V>(qq));
            }
        }
    }
}

// The blocks' partial rows added in their order (32 groups of rows of blocks, then the
// groups), and the parameters' gradients from the sums.
__global__ void __launch_bounds__(1024) block_norm_reduce_kernel(const BlockNormArgs a, int blocks, float *dpost, float *dscale,
                                                                 float *dpre) {
    __shared__ float sum[32][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    grid_dependency_wait();
    if (c < a.D) {
        const float *p = a.partial + (long long)blockIdx.y * a.D + c;
#pragma unroll 8
        for (int r = grp; r < blocks; r += 32) s += p[2ll * r * a.D];
    }
    sum[grp][lane] = s;
    __syncthreads();
    if (grp != 0 || c >= a.D) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += sum[i][lane];
    if (blockIdx.y) {
        if (dpre) dpre[c] = s;
    } else {
        if (dpost) dpost[c] = a.scale ? s * param_at(a.scale, c, a.w_f32) : s;
        if (dscale) dscale[c] = a.w_post ? s * param_at(a.w_post, c, a.w_f32) : s;
    }
}

constexpr int kBnMaxCols = 8192;

// Calls f<TPR, EPT>: the threads of a row and the columns of each by the row's length.
// The forward pass is held up by its two sums over a block: more threads of fewer
// columns (32768 x 4096 bf16: 512 x 8 columns at two blocks an SM 201 us, 256 x 16 at two
// 235).  The backward pass has more bytes to a sum and is not (321 us with 256 x 16).
template <bool FWD, typename F>
auto by_columns(int D, F f) {
    if (D <= 64) return f.template operator()<8, 8>();
    if (D <= 128) return f.template operator()<16, 8>();
    if (D <= 256) return f.template operator()<32, 8>();
    if (D <= 512) return f.template operator()<32, 16>();
    if (D <= 1024) return f.template operator()<128, 8>();
    if (D <= 2048) return f.template operator()<256, 8>();
    if (D <= 4096) return f.template operator()<FWD ? 512 : 256, FWD ? 8 : 16>();
    return f.template operator()<FWD ? 1024 : 512, FWD ? 8 : 16>();
}

// What a launch is: forward, backward without and with the second norm.
enum BnPass { kBnFwd = 0, kBnBwd = 1, kBnBwdPre = 2 };
template <typename T, int TPR, int EPT, int PASS, bool VECTORS>
struct BnKernel {
    static constexpr int VEC = VECTORS ? 16 / (int)sizeof(T) : 1, NV = EPT / VEC;
    using St = std::conditional_t<PASS == kBnFwd, FwdStages<T, TPR, VEC, NV>, BwdStages<T, TPR, VEC, NV, PASS == kBnBwdPre>>;
    static auto get() {
        if constexpr (PASS == kBnFwd) return block_norm_fwd_kernel<T, TPR, VEC, NV>;
        else return block_norm_bwd_kernel<T, TPR, VEC, NV, PASS == kBnBwdPre>;
    }
};
template <typename T, int PASS, bool VECTORS>
struct GridOf {
    long long rows;
    template <int TPR, int EPT>
    int operator()() const {   // blocks of the persistent grid
        constexpr int rpb = bn_threads(TPR) / TPR;
        return (int)std::min<long long>((rows + rpb - 1) / rpb, (long long)device_sm_count() * BnKernel<T, TPR, EPT, PASS, VECTORS>::St::blocks);
    }
};
template <typename T, int PASS, bool VECTORS>
struct Launch {
    const BlockNormArgs &a;
    int grid;
    cudaStream_t s;
    template <int TPR, int EPT>
    cudaError_t operator()() const {
        using K = BnKernel<T, TPR, EPT, PASS, VECTORS>;
        constexpr int smem = K::St::smem;
        void (*kernel)(const BlockNormArgs) = K::get();
        if (smem > 40 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
        }
        BlockNormArgs b = a;
        const long long step = (long long)grid * (bn_threads(TPR) / TPR), q = step / b.inner, r = step % b.inner;
        b.inner_step = (uint32_t)r;
        for (View *v : {&b.y, &b.z, &b.r, &b.dx, &b.dh}) {
            v->ahead = q * v->so + r * v->si, v->wrap = v->so - (long long)b.inner * v->si;
            if (v->p) v->end = static_cast<const T *>(v->p) + (b.rows / b.inner - 1) * v->so + (b.inner - 1ll) * v->si + b.D;
        }
        return launch_dependent(kernel, dim3(grid), dim3(bn_threads(TPR)), smem, s, b);
    }
};

template <typename T, int PASS>
int grid_of(long long rows, int D, bool vec) {
    if (D > kBnMaxCols) return (int)std::min<long long>(rows, device_sm_count());
    return vec ? by_columns<PASS == kBnFwd>(D, GridOf<T, PASS, true>{rows}) : by_columns<PASS == kBnFwd>(D, GridOf<T, PASS, false>{rows});
}
int bwd_grid(long long rows, int D, int dtype, bool vec, bool pre) {
    if (dtype == GDN_BF16) return pre ? grid_of<__nv_bfloat16, kBnBwdPre>(rows, D, vec) : grid_of<__nv_bfloat16, kBnBwd>(rows, D, vec);
    return pre ? grid_of<float, kBnBwdPre>(rows, D, vec) : grid_of<float, kBnBwd>(rows, D, vec);
}

template <typename T, int PASS>
cudaError_t launch_rows(const BlockNormArgs &a, bool vec, cudaStream_t s) {
    const int grid = grid_of<T, PASS>(a.rows, a.D, vec);
    if (a.D > kBnMaxCols) {
        void (*wide)(const BlockNormArgs);
        constexpr int V = 16 / (int)sizeof(T);
        if constexpr (PASS != kBnFwd) wide = vec ? block_norm_wide_bwd_kernel<T, V> : block_norm_wide_bwd_kernel<T, 1>;
        else wide = vec ? block_norm_wide_fwd_kernel<T, V> : block_norm_wide_fwd_kernel<T, 1>;
        return launch_dependent(wide, dim3(grid), dim3(1024), 0, s, a);
    }
    return vec ? by_columns<PASS == kBnFwd>(a.D, Launch<T, PASS, true>{a, grid, s}) : by_columns<PASS == kBnFwd>(a.D, Launch<T, PASS, false>{a, grid, s});
}
cudaError_t launch_bwd(const BlockNormArgs &a, int dtype, bool vec, cudaStream_t s) {
    if (dtype == GDN_BF16) return a.pre ? launch_rows<__nv_bfloat16, kBnBwdPre>(a, vec, s) : launch_rows<__nv_bfloat16, kBnBwd>(a, vec, s);
    return a.pre ? launch_rows<float, kBnBwdPre>(a, vec, s) : launch_rows<float, kBnBwd>(a, vec, s);
}

bool bn_elem_aligned(const void *p, int dtype) { return (reinterpret_cast<uintptr_t>(p) & (dtype == GDN_F32 ? 3u : 1u)) == 0; }

gdn_status bn_args(const gdn_block_norm_desc *d, BlockNormArgs &a) {
    if (!d) return GDN_ERR_INVALID_ARG;
    if (d->outer < 0 || d->inner < 1 || d->D < 1 || !(d->eps >= 0.f)) return GDN_ERR_INVALID_ARG;
    if ((d->dtype != GDN_BF16 && d->dtype != GDN_F32) || (d->w_dtype != GDN_BF16 && d->w_dtype != GDN_F32)) return GDN_ERR_INVALID_ARG;
    if (d->w_dtype == GDN_BF16 && d->dtype == GDN_F32) return GDN_ERR_INVALID_ARG;
    if (d->gate_activation != GDN_GATE_SILU && d->gate_activation != GDN_GATE_SIGMOID) return GDN_ERR_INVALID_ARG;
    // rows are counted in 32 bits, columns too
    if (d->D > (1 << 30) || d->inner > 0x7fffffff || (d->outer > 0 && d->inner > 0x7fffffff / d->outer)) return GDN_ERR_UNSUPPORTED;
    if (!d->post_norm && d->post_weight) return GDN_ERR_INVALID_ARG;
    if (!d->pre_norm && d->pre_weight) return GDN_ERR_INVALID_ARG;
    for (const void *p : {d->post_weight, d->scale, d->pre_weight})
        if (!bn_elem_aligned(p, d->w_dtype)) return GDN_ERR_INVALID_ARG;
    a = {};
    a.y = {d->y, d->y_outer_stride, d->y_inner_stride};
    a.z = {d->gate, d->gate_outer_stride, d->gate_inner_stride};
    a.w_post = d->post_weight, a.scale = d->scale, a.w_pre = d->pre_weight;
    a.rows = d->outer * d->inner, a.D = (int)d->D, a.w_f32 = d->w_dtype == GDN_F32, a.eps = d->eps;
    a.post = d->post_norm != 0, a.pre = d->pre_norm != 0;
    a.gate = d->gate ? (d->gate_activation == GDN_GATE_SILU ? 1 : 2) : 0;
    a.inner = (uint32_t)d->inner;
    if (a.inner > 1) {   // n / inner = (umulhi(magic, n) + n) >> shift for n < 2^31
        uint32_t l = 0;
        while ((1ull << l) < a.inner) ++l;
        a.shift = l;
        a.magic = (uint32_t)((((1ull << l) - a.inner) << 32) / a.inner + 1);
    }
    return GDN_OK;
}
// Strides: rows may not overlap (a single row, or a single one per outer row, has none).
bool bn_view_ok(const gdn_block_norm_desc &d, const void *p, int64_t so, int64_t si) {
    if (!bn_elem_aligned(p, d.dtype)) return false;
    return (d.inner <= 1 || si >= d.D) && (d.outer <= 1 || so >= d.D);
}
bool bn_view_vec(const gdn_block_norm_desc &d, const void *p, int64_t so, int64_t si) {
    const int v = d.dtype == GDN_F32 ? 4 : 8;
    return aligned16(p) && (d.inner <= 1 || si % v == 0) && (d.outer <= 1 || so % v == 0);
}

}  // namespace
}  // namespace gdn

extern "C" gdn_status gdn_block_norm_fwd(const gdn_block_norm_desc *desc, const void *residual, int64_t r_outer_stride,
                                         int64_t r_inner_stride, void *x, void *h, float *rstd_post, float *rstd_pre,
                                         gdn_stream_t stream) {
    using namespace gdn;
    BlockNormArgs a;
    const gdn_status st = bn_args(desc, a);
    if (st != GDN_OK) return st;
    const gdn_block_norm_desc &d = *desc;
    if (a.rows == 0) return GDN_OK;
    if (!d.y || !x || !bn_elem_aligned(x, d.dtype) || !bn_elem_aligned(h, d.dtype) || !bn_elem_aligned(rstd_post, GDN_F32) ||
        !bn_elem_aligned(rstd_pre, GDN_F32) || (a.pre && (!h || !rstd_pre)) || (a.post && !rstd_post))
        return GDN_ERR_INVALID_ARG;
    if (!bn_view_ok(d, d.y, a.y.so, a.y.si) || (a.gate && !bn_view_ok(d, d.gate, a.z.so, a.z.si)) ||
        (residual && !bn_view_ok(d, residual, r_outer_stride, r_inner_stride)))
        return GDN_ERR_INVALID_ARG;
    a.r = {residual, r_outer_stride, r_inner_stride};
    a.res = residual != nullptr;
    a.x = x, a.h = h, a.rstd_post = rstd_post, a.rstd_pre = rstd_pre;
    const bool vec = d.D % (d.dtype == GDN_F32 ? 4 : 8) == 0 && bn_view_vec(d, d.y, a.y.so, a.y.si) &&
                     (!a.gate || bn_view_vec(d, d.gate, a.z.so, a.z.si)) && (!a.res || bn_view_vec(d, residual, r_outer_stride, r_inner_stride)) &&
                     aligned16(x) && (!a.pre || aligned16(h));
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = d.dtype == GDN_BF16 ? launch_rows<__nv_bfloat16, kBnFwd>(a, vec, s) : launch_rows<float, kBnFwd>(a, vec, s);
    if (e != cudaSuccess) {
        set_error_detail("launch block_norm_fwd", e);
        return GDN_ERR_CUDA;
    }
    return GDN_OK;
}

extern "C" size_t gdn_block_norm_bwd_workspace_size(const gdn_block_norm_desc *desc) {
    using namespace gdn;
    BlockNormArgs a;
    if (bn_args(desc, a) != GDN_OK) return 0;
    // alignment is not known here: the larger of both grids
    const int grid = std::max(bwd_grid(a.rows, a.D, desc->dtype, true, a.pre), bwd_grid(a.rows, a.D, desc->dtype, false, a.pre));
    return std::max<size_t>(16, (size_t)grid * 2 * (size_t)a.D * sizeof(float));
}

extern "C" gdn_status gdn_block_norm_bwd(const gdn_block_norm_desc *desc, const void *dx, int64_t dx_outer_stride,
                                         int64_t dx_inner_stride, const void *dh, int64_t dh_outer_stride,
                                         int64_t dh_inner_stride, const void *x, int64_t x_outer_stride,
                                         int64_t x_inner_stride, const float *rstd_post, const float *rstd_pre, void *dy,
                                         void *dresidual, void *dgate, float *dpost_weight, float *dscale,
                                         float *dpre_weight, void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    using namespace gdn;
    BlockNormArgs a;
    const gdn_status st = bn_args(desc, a);
    if (st != GDN_OK) return st;
    const gdn_block_norm_desc &d = *desc;
    for (const float *p : {dpost_weight, dscale, dpre_weight, (float *)rstd_post, (float *)rstd_pre})
        if (!bn_elem_aligned(p, GDN_F32)) return GDN_ERR_INVALID_ARG;
    for (const void *p : {(const void *)dy, (const void *)dresidual, (const void *)dgate})
        if (!bn_elem_aligned(p, d.dtype)) return GDN_ERR_INVALID_ARG;
    if ((dpost_weight && !a.post) || (dpre_weight && !a.pre)) return GDN_ERR_INVALID_ARG;
    const bool params = dpost_weight || dscale || dpre_weight;
    bool vec = false;
    if (a.rows > 0) {
        if (!d.y || !dy || (a.post && !rstd_post) || (a.pre && (!rstd_pre || !dh || !x)) || (!a.pre && !dx) || (a.gate && !dgate))
            return GDN_ERR_INVALID_ARG;
        if (!bn_view_ok(d, d.y, a.y.so, a.y.si) || (a.gate && !bn_view_ok(d, d.gate, a.z.so, a.z.si)) ||
            (dx && !bn_view_ok(d, dx, dx_outer_stride, dx_inner_stride)) ||
            (a.pre && (!bn_view_ok(d, dh, dh_outer_stride, dh_inner_stride) || !bn_view_ok(d, x, x_outer_stride, x_inner_stride))))
            return GDN_ERR_INVALID_ARG;
        if (params) {
            if (!workspace || !aligned16(workspace)) return GDN_ERR_INVALID_ARG;
            if (workspace_bytes < gdn_block_norm_bwd_workspace_size(desc)) return GDN_ERR_WORKSPACE;
        }
        a.dx = {dx, dx_outer_stride, dx_inner_stride};
        a.dh = {dh, dh_outer_stride, dh_inner_stride};
        a.r = {x, x_outer_stride, x_inner_stride};
        a.dy = dy, a.dr = dresidual, a.dz = dgate;
        a.rstd_post = const_cast<float *>(rstd_post), a.rstd_pre = const_cast<float *>(rstd_pre);
        a.partial = params ? static_cast<float *>(workspace) : nullptr;
        vec = d.D % (d.dtype == GDN_F32 ? 4 : 8) == 0 && bn_view_vec(d, d.y, a.y.so, a.y.si) &&
              (!a.gate || (bn_view_vec(d, d.gate, a.z.so, a.z.si) && aligned16(dgate))) &&
              (!dx || bn_view_vec(d, dx, dx_outer_stride, dx_inner_stride)) &&
              (!a.pre || (bn_view_vec(d, dh, dh_outer_stride, dh_inner_stride) && bn_view_vec(d, x, x_outer_stride, x_inner_stride))) &&
              aligned16(dy) && aligned16(dresidual);
    }
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (a.rows > 0) e = launch_bwd(a, d.dtype, vec, s);
    if (e == cudaSuccess && params) {   // no rows: the sums are zero
        const int blocks = a.rows > 0 ? bwd_grid(a.rows, a.D, d.dtype, vec, a.pre) : 0;
        e = launch_dependent(block_norm_reduce_kernel, dim3((a.D + 31) / 32, a.pre ? 2 : 1), dim3(1024), 0, s, a, blocks, dpost_weight, dscale, dpre_weight);
    }
    if (e != cudaSuccess) {
        set_error_detail("launch block_norm_bwd", e);
        return GDN_ERR_CUDA;
    }
    return GDN_OK;
}
