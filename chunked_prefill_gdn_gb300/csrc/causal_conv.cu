// Short causal depthwise convolution along the tokens of a sequence, the step
// between a linear-attention layer's projections and its recurrence:
//
//     u_t = bias + sum_{i < W} w_i x_{t - (W-1) + i},   y_t = act(u_t),
//
// per channel, W = 2, 3 or 4, act the identity or SiLU.  Rows before a
// sequence's first token are those of its state (the last W - 1 inputs of what
// came before, oldest first) or zero.  With du_t = dy_t act'(u_t),
//
//     dx_q = sum_i w_i du_{q + (W-1) - i},  dw_i = sum_t du_t x_{t - (W-1) + i},
//     dbias = sum_t du_t,
//
// where the state's rows count as x_{-(W-1)} .. x_{-1}.
//
// All three forms are streams bound by HBM: a thread owns four neighbouring
// channels (one without alignment), a warp a run of tokens that it walks with
// the window of the last W - 1 inputs in registers, so that a row is read once
// from memory (W - 1 rows of halo per run come from L2); the next kSub rows are
// loaded while the current ones are computed.  A sequence boundary inside a run
// only replaces the window.  In the backward pass the walk also carries the
// W partial sums of the dx that are not complete yet, so dy and x are read
// once; dw and dbias stay in registers over the run, are added over the block's
// warps and leave as one partial row per block that a second kernel adds in
// order.  All arithmetic is on pairs of channels (two-wide FP32).
//
// Measured (bf16, W = 4, SiLU): 65536 packed tokens x 6144 channels 264 us, 6.1
// TB/s, 92% of the measured copy rate; backward 4 x 4095 x 4096 87 us, 4.6 TB/s
// (69%): there the 116 registers of a thread leave 16 warps per SM, which issue 2.3
// instructions per clock, 28 per element; one token of 64 sequences x 12288
// channels 3.3 us, 3.8 TB/s.  fp32: 489 us (6.6 TB/s), 130 us (6.2) and 5.2 us (4.9).
#include <algorithm>

#include "elem.cuh"

namespace gdn {

namespace {

// Measured at 65536 packed tokens x 6144 channels forward, 4 x 4095 x 4096
// backward (bf16).  Forward: 4 warps and runs of 64 give 313 us, 8 warps 289, with
// runs of 128 too 275 (16 warps 361, runs of 256 279; four rows ahead 318, 16 348;
// eight channels per thread instead of four 320), with the run's last rows on the
// boundary-free path 266.  Backward: rows in registers 102 us (eight channels per
// thread 135), eight rows on their way into shared memory 93 (four or twelve 96;
// steps of eight rows 98, of two 100).
constexpr int kConvWarps = 8;   // token runs per block
constexpr int kConvRun = 128;   // tokens of a run, at most
constexpr int kSub = 8;         // rows loaded ahead (forward)
constexpr int kSubB = 4;        // rows of an unrolled step (backward)
constexpr int kAheadBytes = 16; // element size x rows of x and dy on their way (backward)

struct ConvArgs {
    const void *x, *dy, *w, *bias, *init, *d_final;
    void *out, *last;           // y and final state; or dx and d_init
    float *partial;             // [groups][W + 1][D]
    const int32_t *cu, *slots;
    int32_t *status;
    long long x_batch, x_token, dy_batch, dy_token;
    int B, T, D, n_seqs, w_f32, w_vec, silu, run, groups, chan_blocks, pool;
};

__device__ __forceinline__ float conv_param(const void *p, long long i, int f32) {
    return f32 ? static_cast<const float *>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

// Weights and bias of a thread's VEC channels, as pairs of channels.
template <int W, int VEC>
__device__ __forceinline__ void load_weights(const ConvArgs &a, int c, bool live, F2 (&w)[W][(VEC + 1) / 2],
                                             F2 (&b)[(VEC + 1) / 2]) {
    if constexpr (VEC == 4) {
        if (a.w_vec && live) {   // the channels' taps are neighbours: 4 W values in words of four
            float f[4 * W];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const long long at = (long long)c * W + 4 * i;
                if (a.w_f32) unpack<float, 4>(load_raw<float, 4>(static_cast<const float *>(a.w) + at), f + 4 * i);
                else unpack<__nv_bfloat16, 4>(load_raw<__nv_bfloat16, 4>(static_cast<const __nv_bfloat16 *>(a.w) + at), f + 4 * i);
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) {
#pragma unroll
                for (int i = 0; i < W; ++i) w[i][p] = pair(f[2 * p * W + i], f[(2 * p + 1) * W + i]);
                b[p] = pair(a.bias ? conv_param(a.bias, c + 2 * p, a.w_f32) : 0.f,
                            a.bias ? conv_param(a.bias, c + 2 * p + 1, a.w_f32) : 0.f);
            }
            return;
        }
    }
#pragma unroll
    for (int p = 0; p < (VEC + 1) / 2; ++p) {
        const bool two = live && VEC > 1;
#pragma unroll
        for (int i = 0; i < W; ++i)
            w[i][p] = pair(live ? conv_param(a.w, (long long)(c + 2 * p) * W + i, a.w_f32) : 0.f,
                           two ? conv_param(a.w, (long long)(c + 2 * p + 1) * W + i, a.w_f32) : 0.f);
        b[p] = pair(live && a.bias ? conv_param(a.bias, c + 2 * p, a.w_f32) : 0.f,
                    two && a.bias ? conv_param(a.bias, c + 2 * p + 1, a.w_f32) : 0.f);
    }
}

// Row r of sequence n's state.
template <typename T, int W, int VEC>
__device__ __forceinline__ void state_row(const ConvArgs &a, const void *state, int n, int r, int c, bool live,
                                          F2 (&v)[(VEC + 1) / 2]) {
    unpack_pairs<T, VEC>(live && state ? load_raw<T, VEC>(static_cast<const T *>(state) + ((long long)n * (W - 1) + r) * a.D + c)
                                       : zero_raw<T, VEC>(), v);
}

// Where a run of tokens [t0, t1) of batch row b lies.
struct Run {
    int b, t0, t1, n, begin, end;   // begin, end: of the sequence that holds the current token
};

__device__ __forceinline__ void enter_seq(const ConvArgs &a, Run &r, int t) {
    if (a.cu) {
        r.begin = min(max(__ldg(a.cu + r.n), 0), t);
        r.end = min(max(__ldg(a.cu + r.n + 1), t + 1), a.T);
    }
}

// The window before token t0: rows of the run's sequence, or of its state.
template <typename T, int W, int VEC>
__device__ __forceinline__ void first_window(const ConvArgs &a, const Run &r, int c, bool live,
                                             F2 (&win)[W - 1][(VEC + 1) / 2]) {
    const T *x = static_cast<const T *>(a.x) + r.b * a.x_batch + c;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        const int t = r.t0 - (W - 1) + i;
        if (t >= r.begin) unpack_pairs<T, VEC>(live ? load_raw<T, VEC>(x + t * a.x_token) : zero_raw<T, VEC>(), win[i]);
        else state_row<T, W, VEC>(a, a.init, r.n, (W - 1) + t - r.begin, c, live, win[i]);
    }
}

// VEC elements on their way into shared memory (a single 2-byte one by way of a
// register).
template <typename T, int VEC>
__device__ __forceinline__ void copy_piece(T *dst, const T *src) {
    constexpr int bytes = VEC * (int)sizeof(T);
    if constexpr (bytes >= 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "n"(bytes) : "memory");
    else
        *dst = *src;
}

// u of a token whose row is x, and the window moved on.
template <int W, int P>
__device__ __forceinline__ void conv_sum(const F2 (&w)[W][P], const F2 (&bias)[P], const F2 (&win)[W - 1][P],
                                         const F2 (&x)[P], F2 (&u)[P]) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
        u[p] = fma2(w[W - 1][p], x[p], bias[p]);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) u[p] = fma2(w[k][p], win[k][p], u[p]);
    }
}
template <int W, int P>
__device__ __forceinline__ void move_window(F2 (&win)[W - 1][P], const F2 (&x)[P]) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
        for (int k = 0; k < W - 2; ++k) win[k][p] = win[k + 1][p];
        win[W - 2][p] = x[p];
    }
}

template <typename T, int W, int VEC>
__global__ void __launch_bounds__(32 * kConvWarps) conv_fwd_kernel(ConvArgs a) {
    constexpr int P = (VEC + 1) / 2;
    grid_dependency_wait();
    if (a.status && a.cu && blockIdx.x == 0) check_cu(a.cu, a.n_seqs, a.T, a.status);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = ((blockIdx.x % a.chan_blocks) * 32 + lane) * VEC;
    const int tile = (blockIdx.x / a.chan_blocks) * kConvWarps + warp;   // over all batch rows
    const bool live = c < a.D;
    const int per_row = a.groups / a.B * kConvWarps;
    Run r;
    r.b = tile / per_row;
    r.t0 = (tile % per_row) * a.run;
    r.t1 = min(a.T, r.t0 + a.run);
    T *last = static_cast<T *>(a.last);
    // a sequence without a token keeps its state: packed ones are dealt over the runs
    if (last && live) {
        auto keep = [&](int n) {
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                F2 v[P];
                state_row<T, W, VEC>(a, a.init, n, i, c, true, v);
                store_raw<T, VEC>(last + ((long long)n * (W - 1) + i) * a.D + c, pack_pairs<T, VEC>(v));
            }
        };
        for (int n = tile; a.cu && n < a.n_seqs; n += a.groups * kConvWarps)
            if (__ldg(a.cu + n) >= __ldg(a.cu + n + 1)) keep(n);
        if (!a.cu && a.T == 0 && r.t0 == 0) keep(r.b);
    }
    if (r.t0 >= r.t1 || !live) return;
    const T *x = static_cast<const T *>(a.x) + r.b * a.x_batch + r.t0 * a.x_token + c;   // the next row to load
    T *y = static_cast<T *>(a.out) + ((long long)r.b * a.T + r.t0) * a.D + c;            // the next to store
    Raw<T, VEC> ring[kSub];
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
        ring[i] = r.t0 + i < r.t1 ? load_raw<T, VEC>(x) : zero_raw<T, VEC>();
        x += a.x_token;
    }
    F2 w[W][P], bias[P], win[W - 1][P];
    load_weights<W, VEC>(a, c, live, w, bias);
    r.n = a.cu ? find_seq(a.cu, a.n_seqs, r.t0) : r.b;
    r.begin = 0, r.end = a.T;
    enter_seq(a, r, r.t0);
    first_window<T, W, VEC>(a, r, c, live, win);
    auto token = [&](int i) {   // computes row i of the ring
        F2 xv[P], u[P];
        unpack_pairs<T, VEC>(ring[i], xv);
        conv_sum<W, P>(w, bias, win, xv, u);
        move_window<W, P>(win, xv);
        if (a.silu) {
#pragma unroll
            for (int p = 0; p < P; ++p) u[p] = mul2(u[p], sigmoid_pair(u[p]));
        }
        store_raw<T, VEC>(y, pack_pairs<T, VEC>(u));
        y += a.D;
    };
    for (int t = r.t0; t < r.t1; t += kSub) {
        if (t + kSub <= r.t1 && t + kSub < r.end) {   // no boundary among these rows
            const int more = r.t1 - t - kSub;
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
                token(i);
                if (i < more) ring[i] = load_raw<T, VEC>(x);
                x += a.x_token;
            }
            continue;
        }
#pragma unroll
        for (int i = 0; i < kSub; ++i) {
            const int q = t + i;
            if (q >= r.t1) break;
            if (q == r.end) {   // the next sequence that has a token
                while (r.n + 1 < a.n_seqs && __ldg(a.cu + r.n + 1) <= q) ++r.n;
                enter_seq(a, r, q);
#pragma unroll
                for (int k = 0; k < W - 1; ++k) state_row<T, W, VEC>(a, a.init, r.n, k, c, true, win[k]);
            }
            token(i);
            if (q + kSub < r.t1) ring[i] = load_raw<T, VEC>(x);
            x += a.x_token;
            if (last && q + 1 == r.end) {
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
                    store_raw<T, VEC>(last + ((long long)r.n * (W - 1) + k) * a.D + c, pack_pairs<T, VEC>(win[k]));
            }
        }
    }
}

template <typename T, int W, int VEC>
__global__ void __launch_bounds__(32 * kConvWarps) conv_bwd_kernel(ConvArgs a) {
    constexpr int P = (VEC + 1) / 2;
    constexpr int kAhead = kAheadBytes / (int)sizeof(T);
    static_assert(kAhead % kSubB == 0, "a step's rows in neighbouring slots");
    using Piece = T[VEC];
    using Rows = Piece[kAhead][2][32];               // of a warp
    using Sums = float[W + 1][32 * VEC];             // of a warp, when it is done with its rows
    __shared__ __align__(16) unsigned char shared[kConvWarps * (sizeof(Rows) > sizeof(Sums) ? sizeof(Rows) : sizeof(Sums))];
    Piece *ring = reinterpret_cast<Rows *>(shared)[threadIdx.x >> 5][0][0];
    Sums *sum = reinterpret_cast<Sums *>(shared);
    grid_dependency_wait();
    if (a.status && a.cu && blockIdx.x == 0) check_cu(a.cu, a.n_seqs, a.T, a.status);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = ((blockIdx.x % a.chan_blocks) * 32 + lane) * VEC;
    const int group = blockIdx.x / a.chan_blocks;
    const int tile = group * kConvWarps + warp;
    const bool live = c < a.D;
    const int per_row = a.groups / a.B * kConvWarps;
    Run r;
    r.b = tile / per_row;
    r.t0 = (tile % per_row) * a.run;
    r.t1 = min(a.T, r.t0 + a.run);
    T *dinit = static_cast<T *>(a.last);
    // a sequence without a token hands the gradient of its final state on
    if (dinit && live) {
        auto pass_on = [&](int n) {
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                F2 v[P];
                state_row<T, W, VEC>(a, a.d_final, n, i, c, true, v);
                store_raw<T, VEC>(dinit + ((long long)n * (W - 1) + i) * a.D + c, pack_pairs<T, VEC>(v));
            }
        };
        for (int n = tile; a.cu && n < a.n_seqs; n += a.groups * kConvWarps)
            if (__ldg(a.cu + n) >= __ldg(a.cu + n + 1)) pass_on(n);
        if (!a.cu && a.T == 0 && r.t0 == 0) pass_on(r.b);
    }
    F2 dw[W][P], db[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        db[p] = both(0.f);
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k][p] = both(0.f);
    }
    if (r.t0 < r.t1 && live) {
        // dx of a token needs the W - 1 tokens after it: the walk goes on past the run
        const int stop = min(a.T, r.t1 + W - 1);
        const T *x = static_cast<const T *>(a.x) + r.b * a.x_batch + r.t0 * a.x_token + c;
        const T *dy = static_cast<const T *>(a.dy) + r.b * a.dy_batch + r.t0 * a.dy_token + c;
        T *dx = static_cast<T *>(a.out) + (long long)r.b * a.T * a.D + c;
        // rows of x and dy come in kAhead ahead, asynchronously where the address allows,
        // row t in slot t - t0 modulo kAhead; a lane reads back what it copied
        auto load_row = [&](Piece *at, int t) {
            if (t < stop) {
                copy_piece<T, VEC>(at[0], x);
                copy_piece<T, VEC>(at[32], dy);
            }
            copy_commit();
            x += a.x_token, dy += a.dy_token;
        };
        Piece *slots = ring + lane;   // the unrolled step's first slot
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load_row(slots + i * 64, r.t0 + i);
        F2 w[W][P], bias[P], win[W - 1][P], acc[W][P];
        load_weights<W, VEC>(a, c, live, w, bias);
        r.n = a.cu ? find_seq(a.cu, a.n_seqs, r.t0) : r.b;
        r.begin = 0, r.end = a.T;
        enter_seq(a, r, r.t0);
        first_window<T, W, VEC>(a, r, c, live, win);
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int k = 0; k < W; ++k) acc[k][p] = both(0.f);
        // row i of the step, that of token t; acc[k] gathers dx of position t - (W - 1) + k
        auto token = [&](int i, int t, bool mine) {
            F2 xv[P], u[P], du[P];
            Piece *at = slots + i * 64;
            copy_wait<kAhead - 1>();
            unpack_pairs<T, VEC>(load_raw<T, VEC>(at[0]), xv);
            unpack_pairs<T, VEC>(load_raw<T, VEC>(at[32]), du);
            load_row(at, t + kAhead);
            if (a.silu) {
                conv_sum<W, P>(w, bias, win, xv, u);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    // silu' = s + u s (1 - s) = s (1 + u (1 - s))
                    const F2 s = sigmoid_pair(u[p]);
                    const F2 g = fma2(u[p], fma2(s, both(-1.f), both(1.f)), both(1.f));
                    du[p] = mul2(du[p], mul2(s, g));
                }
            }
#pragma unroll
            for (int p = 0; p < P; ++p) {
#pragma unroll
                for (int k = 0; k < W; ++k) acc[k][p] = fma2(w[k][p], du[p], acc[k][p]);
                if (mine) {   // tokens past the run belong to the next one's sums
                    db[p] = add2(db[p], du[p]);
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) dw[k][p] = fma2(du[p], win[k][p], dw[k][p]);
                    dw[W - 1][p] = fma2(du[p], xv[p], dw[W - 1][p]);
                }
            }
            move_window<W, P>(win, xv);
        };
        auto shift = [&] {
#pragma unroll
            for (int p = 0; p < P; ++p) {
#pragma unroll
                for (int k = 0; k < W - 1; ++k) acc[k][p] = acc[k + 1][p];
                acc[W - 1][p] = both(0.f);
            }
        };
        // the complete sum of position q, to whom it belongs
        auto emit = [&](int q, const F2 (&v)[P]) {
            if (q >= r.begin) {
                if (q >= r.t0 && q < r.t1) store_raw<T, VEC>(dx + (long long)q * a.D, pack_pairs<T, VEC>(v));
            } else if (dinit && r.begin >= r.t0 && r.begin < r.t1) {
                store_raw<T, VEC>(dinit + ((long long)r.n * (W - 1) + (W - 1) + q - r.begin) * a.D + c, pack_pairs<T, VEC>(v));
            }
        };
        // the last W - 1 positions before a sequence's end (at t): no token follows
        auto flush = [&](int t) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                F2 f[P];
                state_row<T, W, VEC>(a, a.d_final, r.n, k, c, true, f);
#pragma unroll
                for (int p = 0; p < P; ++p) acc[k][p] = add2(acc[k][p], f[p]);
                emit(t - (W - 1) + k, acc[k]);
#pragma unroll
                for (int p = 0; p < P; ++p) acc[k][p] = both(0.f);
            }
        };
        bool done = false;
        for (int t = r.t0; t < stop && !done; t += kSubB, slots = kAhead == kSubB ? slots : ring + lane + (t - r.t0) % kAhead * 64) {
            // tokens and the positions they complete in the run and the sequence
            if (t - (W - 1) >= max(r.begin, r.t0) && t + kSubB <= min(r.end, r.t1)) {
                T *out = dx + (long long)(t - (W - 1)) * a.D;
#pragma unroll
                for (int i = 0; i < kSubB; ++i) {
                    token(i, t + i, true);
                    store_raw<T, VEC>(out, pack_pairs<T, VEC>(acc[0]));
                    out += a.D;
                    shift();
                }
                continue;
            }
            for (int i = 0; i < kSubB; ++i) {
                const int q = t + i;
                if (q >= stop || done) break;
                if (q == r.end) {
                    flush(q);
                    if (q >= r.t1) {
                        done = true;
                        break;
                    }
                    while (r.n + 1 < a.n_seqs && __ldg(a.cu + r.n + 1) <= q) ++r.n;
                    enter_seq(a, r, q);
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) state_row<T, W, VEC>(a, a.init, r.n, k, c, true, win[k]);
                }
                token(i, q, q < r.t1);
                emit(q - (W - 1), acc[0]);
                shift();
            }
        }
        copy_wait<0>();
        if (!done && stop == r.end) flush(stop);
    }
    if (!a.partial) return;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
#pragma unroll
        for (int k = 0; k < W; ++k) sum[warp][k][lane * VEC + e] = e & 1 ? hi(dw[k][e / 2]) : lo(dw[k][e / 2]);
        sum[warp][W][lane * VEC + e] = e & 1 ? hi(db[e / 2]) : lo(db[e / 2]);
    }
    __syncthreads();
    const int c0 = (blockIdx.x % a.chan_blocks) * 32 * VEC;
    for (int i = threadIdx.x; i < (W + 1) * 32 * VEC; i += blockDim.x) {
        const int k = i / (32 * VEC), j = i % (32 * VEC);
        if (c0 + j >= a.D) continue;
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < kConvWarps; ++v) s += sum[v][k][j];
        a.partial[((long long)group * (W + 1) + k) * a.D + c0 + j] = s;
    }
}

// dw [D][W] and dbias [D] from the blocks' partial rows, in the blocks' order.
__global__ void __launch_bounds__(256) conv_reduce_kernel(const float *partial, int groups, int W, int D, float *dw,
                                                          float *dbias) {
    __shared__ float sum[8][32];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, k = blockIdx.y;
    float s = 0.f;
    grid_dependency_wait();
    if (c < D) {
#pragma unroll 4
        for (int g = grp; g < groups; g += 8) s += partial[((long long)g * (W + 1) + k) * D + c];
    }
    sum[grp][lane] = s;
    __syncthreads();
    if (grp == 0 && c < D) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sum[i][lane];
        if (k < W && dw) dw[(long long)c * W + k] = s;
        if (k == W && dbias) dbias[c] = s;
    }
}

// One token of each sequence: the window is the cached state, which moves on
// by one row in place.
template <typename T, int W, int VEC>
__global__ void __launch_bounds__(128) conv_step_kernel(ConvArgs a) {
    const int c = (blockIdx.x * 128 + threadIdx.x) * VEC;
    const int n = blockIdx.y;
    grid_dependency_wait();
    if (c >= a.D) return;
    T *y = static_cast<T *>(a.out) + (long long)n * a.D + c;
    const int slot = a.slots ? __ldg(a.slots + n) : n;
    if (slot < 0 || slot >= a.pool) {   // a padded row
        store_raw<T, VEC>(y, zero_raw<T, VEC>());
        return;
    }
    T *state = static_cast<T *>(a.last) + (long long)slot * (W - 1) * a.D + c;
    Raw<T, VEC> row[W];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) row[k] = load_raw<T, VEC>(state + (long long)k * a.D);
    row[W - 1] = load_raw<T, VEC>(static_cast<const T *>(a.x) + n * a.x_batch + c);
    constexpr int P = (VEC + 1) / 2;
    F2 w[W][P], u[P];
    load_weights<W, VEC>(a, c, true, w, u);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        F2 v[P];
        unpack_pairs<T, VEC>(row[k], v);
#pragma unroll
        for (int p = 0; p < P; ++p) u[p] = fma2(w[k][p], v[p], u[p]);
    }
    if (a.silu) {
#pragma unroll
        for (int p = 0; p < P; ++p) u[p] = mul2(u[p], sigmoid_pair(u[p]));
    }
    store_raw<T, VEC>(y, pack_pairs<T, VEC>(u));
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store_raw<T, VEC>(state + (long long)k * a.D, row[k + 1]);
}

enum class Conv { kFwd, kBwd, kStep };

template <Conv OP, typename T, int W, int VEC>
cudaError_t launch_conv_one(const ConvArgs &a, cudaStream_t s) {
    if constexpr (OP == Conv::kStep) {
        return launch_dependent(conv_step_kernel<T, W, VEC>, dim3((a.D + 128 * VEC - 1) / (128 * VEC), a.B), dim3(128), 0, s, a);
    } else {
        const dim3 grid((unsigned)((long long)a.groups * a.chan_blocks)), block(32 * kConvWarps);
        if constexpr (OP == Conv::kFwd) return launch_dependent(conv_fwd_kernel<T, W, VEC>, grid, block, 0, s, a);
        else return launch_dependent(conv_bwd_kernel<T, W, VEC>, grid, block, 0, s, a);
    }
}

template <Conv OP, typename T>
cudaError_t launch_conv(ConvArgs a, int W, bool vec, cudaStream_t s) {
    const int per_block = 32 * (vec ? 4 : 1);
    a.chan_blocks = (a.D + per_block - 1) / per_block;
#define GDN_CONV(WW) (vec ? launch_conv_one<OP, T, WW, 4>(a, s) : launch_conv_one<OP, T, WW, 1>(a, s))
    return W == 2 ? GDN_CONV(2) : W == 3 ? GDN_CONV(3) : GDN_CONV(4);
#undef GDN_CONV
}

// Tokens per warp: the run that gives the shortest schedule when an SM holds
// `resident` blocks, counting for each run its tokens and about 24 more (halo,
// weights, filling and draining the ring of rows).  At 4 x 4095 tokens x 4096
// channels the backward pass runs 1.7 waves of blocks with runs of 128 and 2.95
// with runs of 76.
int conv_run(int B, int T, int D, int vec, int resident) {
    const long long chan = (D + 32 * vec - 1) / (32 * vec), slots = (long long)resident * device_sm_count();
    long long best = -1;
    int run = kSub;
    for (int r = kSub; r <= kConvRun; r += 4) {
        const long long blocks = B * chan * ((T + r * kConvWarps - 1) / (r * kConvWarps));
        const long long cost = (blocks + slots - 1) / slots * (r + 24);
        if (best < 0 || cost < best) best = cost, run = r;
    }
    return run;
}
constexpr int kConvResident = 3, kConvResidentB = 2;   // blocks per SM by registers

// Groups of kConvWarps runs over all batch rows (at least one per row).
int conv_groups(int B, int T, int run) { return B * std::max(1, (T + run * kConvWarps - 1) / (run * kConvWarps)); }

struct ConvShape {
    const int32_t *cu;
    int n_seqs, B, T, D, W, dtype, w_dtype;
};

gdn_status conv_shape_ok(const ConvShape &p, int64_t batch_stride, int64_t token_stride) {
    if (p.B < 0 || p.T < 0 || p.D < 1) return GDN_ERR_INVALID_ARG;
    if (p.W < 2 || p.W > 4) return GDN_ERR_UNSUPPORTED;
    // token and channel indices are 32-bit, and so is the number of blocks
    if (p.T > (1 << 30) || p.D > (1 << 30) || (long long)p.B * (p.T / kSub + 1) > (1ll << 30)) return GDN_ERR_UNSUPPORTED;
    if ((p.dtype != GDN_BF16 && p.dtype != GDN_F32) || (p.w_dtype != GDN_F32 && p.w_dtype != p.dtype))
        return GDN_ERR_INVALID_ARG;
    if (p.cu && (p.B != 1 || p.n_seqs < 1)) return GDN_ERR_INVALID_ARG;
    if (token_stride < p.D || batch_stride < 0) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

bool conv_vec(const ConvShape &p, const void *const *ptrs, int n, int64_t s0, int64_t s1) {
    const uintptr_t mask = (p.dtype == GDN_F32 ? 16 : 8) - 1;
    bool ok = p.D % 4 == 0 && s0 % 4 == 0 && s1 % 4 == 0;
    for (int i = 0; i < n; ++i) ok = ok && (reinterpret_cast<uintptr_t>(ptrs[i]) & mask) == 0;
    return ok;
}

bool conv_elems(const void *const *ptrs, int n, int dtype) {
    for (int i = 0; i < n; ++i)
        if (reinterpret_cast<uintptr_t>(ptrs[i]) & (dtype == GDN_F32 ? 3u : 1u)) return false;
    return true;
}

}  // namespace

}  // namespace gdn

extern "C" gdn_status gdn_causal_conv_fwd(const void *x, int64_t x_batch_stride, int64_t x_token_stride,
                                          const void *weight, const void *bias, gdn_dtype w_dtype,
                                          const void *initial_state, const int32_t *cu_seqlens, int n_seqs, int B,
                                          int T, int D, int W, int silu, gdn_dtype dtype, void *y, void *final_state,
                                          int32_t *device_status, gdn_stream_t stream) {
    using namespace gdn;
    const ConvShape p = {cu_seqlens, n_seqs, B, T, D, W, dtype, w_dtype};
    const gdn_status st = conv_shape_ok(p, x_batch_stride, x_token_stride);
    if (st != GDN_OK) return st;
    if (B == 0) return GDN_OK;
    if (!weight || (T > 0 && (!x || !y))) return GDN_ERR_INVALID_ARG;
    const void *act[] = {x, y, initial_state, final_state}, *par[] = {weight, bias};
    if (!conv_elems(act, 4, dtype) || !conv_elems(par, 2, w_dtype)) return GDN_ERR_INVALID_ARG;
    const bool vec = conv_vec(p, act, 4, x_batch_stride, x_token_stride);
    ConvArgs a = {};
    a.x = x, a.w = weight, a.bias = bias, a.init = initial_state, a.out = y, a.last = final_state;
    a.cu = cu_seqlens, a.status = device_status, a.x_batch = x_batch_stride, a.x_token = x_token_stride;
    a.B = B, a.T = T, a.D = D, a.n_seqs = cu_seqlens ? n_seqs : B, a.w_f32 = w_dtype == GDN_F32, a.w_vec = aligned16(weight), a.silu = silu != 0;
    a.run = conv_run(B, T, D, vec ? 4 : 1, kConvResident);
    a.groups = conv_groups(B, T, a.run);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == GDN_BF16 ? launch_conv<Conv::kFwd, __nv_bfloat16>(a, W, vec, s)
                                            : launch_conv<Conv::kFwd, float>(a, W, vec, s);
    if (e != cudaSuccess) {
        set_error_detail("launch causal_conv_fwd", e);
        return GDN_ERR_CUDA;
    }
    return GDN_OK;
}

extern "C" size_t gdn_causal_conv_bwd_workspace_size(int B, int T, int D, int W) {
    if (B < 0 || T < 0 || D < 1 || W < 2 || W > 4) return 0;
    // the narrower of the two layouts needs more groups: room for either
    const int g4 = gdn::conv_groups(B, T, gdn::conv_run(B, T, D, 4, gdn::kConvResidentB));
    const int g1 = gdn::conv_groups(B, T, gdn::conv_run(B, T, D, 1, gdn::kConvResidentB));
    return std::max<size_t>(16, (size_t)std::max(g4, g1) * (W + 1) * (size_t)D * sizeof(float));
}

extern "C" gdn_status gdn_causal_conv_bwd(const void *dy, int64_t dy_batch_stride, int64_t dy_token_stride,
                                          const void *x, int64_t x_batch_stride, int64_t x_token_stride,
                                          const void *weight, const void *bias, gdn_dtype w_dtype,
                                          const void *initial_state, const void *d_final_state,
                                          const int32_t *cu_seqlens, int n_seqs, int B, int T, int D, int W, int silu,
                                          gdn_dtype dtype, void *dx, float *dweight, float *dbias,
                                          void *d_initial_state, int32_t *device_status, void *workspace,
                                          size_t workspace_bytes, gdn_stream_t stream) {
    using namespace gdn;
    const ConvShape p = {cu_seqlens, n_seqs, B, T, D, W, dtype, w_dtype};
    gdn_status st = conv_shape_ok(p, x_batch_stride, x_token_stride);
    if (st == GDN_OK) st = conv_shape_ok(p, dy_batch_stride, dy_token_stride);
    if (st != GDN_OK) return st;
    if (!weight || (B > 0 && T > 0 && (!x || !dy || !dx))) return GDN_ERR_INVALID_ARG;
    const void *act[] = {x, dy, dx, initial_state, d_final_state, d_initial_state}, *par[] = {weight, bias};
    const void *f32[] = {dweight, dbias};
    if (!conv_elems(act, 6, dtype) || !conv_elems(par, 2, w_dtype) || !conv_elems(f32, 2, GDN_F32))
        return GDN_ERR_INVALID_ARG;
    const bool vec = conv_vec(p, act, 6, x_batch_stride | dy_batch_stride, x_token_stride | dy_token_stride);
    const bool params = dweight || dbias;
    if (params && B > 0) {
        if (!workspace || !aligned16(workspace)) return GDN_ERR_INVALID_ARG;
        if (workspace_bytes < gdn_causal_conv_bwd_workspace_size(B, T, D, W)) return GDN_ERR_WORKSPACE;
    }
    ConvArgs a = {};
    a.x = x, a.dy = dy, a.w = weight, a.bias = bias, a.init = initial_state, a.d_final = d_final_state;
    a.out = dx, a.last = d_initial_state, a.partial = params ? static_cast<float *>(workspace) : nullptr;
    a.cu = cu_seqlens, a.status = device_status;
    a.x_batch = x_batch_stride, a.x_token = x_token_stride, a.dy_batch = dy_batch_stride, a.dy_token = dy_token_stride;
    a.B = B, a.T = T, a.D = D, a.n_seqs = cu_seqlens ? n_seqs : B, a.w_f32 = w_dtype == GDN_F32, a.w_vec = aligned16(weight), a.silu = silu != 0;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (B > 0) {
        a.run = conv_run(B, T, D, vec ? 4 : 1, kConvResidentB);
        a.groups = conv_groups(B, T, a.run);
        e = dtype == GDN_BF16 ? launch_conv<Conv::kBwd, __nv_bfloat16>(a, W, vec, s)
                              : launch_conv<Conv::kBwd, float>(a, W, vec, s);
    }
    if (e == cudaSuccess && params) {
        e = launch_dependent(conv_reduce_kernel, dim3((D + 31) / 32, W + 1), dim3(256), 0, s,
                             static_cast<const float *>(workspace), B > 0 ? a.groups : 0, W, D, dweight, dbias);
    }
    if (e != cudaSuccess) {
        set_error_detail("launch causal_conv_bwd", e);
        return GDN_ERR_CUDA;
    }
    return GDN_OK;
}

extern "C" gdn_status gdn_causal_conv_step(const void *x, int64_t x_stride, void *state, const int32_t *state_indices,
                                           int n_states, const void *weight, const void *bias, gdn_dtype w_dtype,
                                           int N, int D, int W, int silu, gdn_dtype dtype, void *y,
                                           gdn_stream_t stream) {
    using namespace gdn;
    const ConvShape p = {nullptr, 0, N, 1, D, W, dtype, w_dtype};
    const gdn_status st = conv_shape_ok(p, 0, x_stride);
    if (st != GDN_OK) return st;
    if (N > 65535 || n_states < 0 || (!state_indices && n_states < N)) return GDN_ERR_INVALID_ARG;
    if (N == 0) return GDN_OK;
    if (!x || !state || !weight || !y) return GDN_ERR_INVALID_ARG;
    const void *act[] = {x, state, y}, *par[] = {weight, bias};
    if (!conv_elems(act, 3, dtype) || !conv_elems(par, 2, w_dtype)) return GDN_ERR_INVALID_ARG;
    const bool vec = conv_vec(p, act, 3, x_stride, x_stride);
    ConvArgs a = {};
    a.x = x, a.w = weight, a.bias = bias, a.out = y, a.last = state, a.slots = state_indices, a.pool = n_states;
    a.x_batch = x_stride, a.B = N, a.T = 1, a.D = D, a.w_f32 = w_dtype == GDN_F32, a.w_vec = aligned16(weight), a.silu = silu != 0;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == GDN_BF16 ? launch_conv<Conv::kStep, __nv_bfloat16>(a, W, vec, s)
                                            : launch_conv<Conv::kStep, float>(a, W, vec, s);
    if (e != cudaSuccess) {
        set_error_detail("launch causal_conv_step", e);
        return GDN_ERR_CUDA;
    }
    return GDN_OK;
}
