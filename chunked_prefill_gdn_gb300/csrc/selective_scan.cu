// Selective state space scan with a diagonal transition: per channel d and
// state index n of a sequence,
//
//     h_t = a_t h_{t-1} + s_t x_t B_t[n],  a_t = exp(s_t A[d][n]),
//     y_t = sum_n C_t[n] h_t + D x_t,      out_t = y_t silu(z_t),
//
// with the step s_t = dt_t + dt_bias (through softplus when asked).  This file
// holds the forward pass, the single-token form and the entry points.
//
// What bounds the forward pass is arithmetic, not memory: one exponential and
// four multiply-adds per (token, channel, n) against about 8 bytes per (token,
// channel).  ex2 runs at 32 lanes per clock and SM, FP32 FMA at 128 (measured on
// a GB300), so both pipes are full at the same rate, 32 (token, channel, n) per
// clock and SM; a loop of exactly these instructions, with B and C in shared
// memory, reaches 20 of them with four warps per scheduler, 16 with two, 11 with
// one.  The arithmetic is written on pairs (two-wide FP32), which leaves issue
// slots for the rest.  B and C of a tile of tokens are read from shared memory by
// all channels of a block at once, and what is per (token, channel) only
// (softplus, the gate) is computed once, by a warp of its own.
//
// Measured (bf16, 16 n): 8 x 1024 tokens x 4096 channels 171 us (11 per clock and
// SM): 6.7 scanning warps per SM are what 32768 channels give, and without the
// feeding warps' work they alone take 136 us.  A row of 32768 tokens x 1024
// channels 287 us, of it 118 the maps and 7 their combination.  24 n, padded to 32,
// 332 us on the batch, 32 n 302, 64 n 584, 8 n 118.  Tried and dropped: eight n per
// thread and twice the warps (lanes or warps sharing a channel: 213 and 199 us
// where 16 n took 197, before the feeding warp; not measured with it), two channels
// x eight n per thread, which halves the reads of B and C (201 / 298 us: the same
// rate per SM, but blocks of 64 channels fill the SMs less evenly), tiles of 8 or 32
// tokens, the exponentials of the next token computed ahead (181 us).
//
// When the (sequence, channel) pairs do not fill the GPU, the token axis is cut
// into segments: a first pass gives every segment's end state from a zero
// start, a short pass combines them (the map of a segment is h -> exp(A sum s)
// h + end), and the full pass starts every segment from its exact state.  Each
// exponential is then taken twice.
#include <algorithm>
#include <type_traits>

#include "scan_pairs.cuh"

namespace gdn {

namespace {

// kFull: the outputs and final states.  kState: the end state from a zero start
// and the sum of the steps of every segment.  kMaps: the same for the backward
// pass, whose segments are shorter than what a block of this kernel walks
// (span_tokens), with the gradient at a segment's start that the outputs of its
// tokens give, and the state and the sum so far before each of its tiles.
enum ScanMode { kFull, kState, kMaps };

// 32 channels per block.  NW warps scan, a lane per channel, sharing out the n,
// NPT per thread; one more warp feeds them: it copies the raw rows in
// asynchronously (three tiles in flight, each piece read back by the lane that
// copied it), prepares the steps and B and C of the next tile in fp32, and
// finishes the outputs of the last one, all while the current tile is scanned.
template <typename T, int NPT, int NW, int MODE>
struct ScanShape {
    static constexpr int CW = 32;
    static constexpr int NP = NPT * NW;                     // n, padded
    static constexpr int VPR = CW / 8;                      // vectors of eight channels per row
    static constexpr int RPP = 32 / VPR;                    // rows per pass of the feeding warp
    static constexpr int PASSES = kTile / RPP;
    static constexpr int BCR = NP / 4;                      // vectors of eight n per row of B and C
    static constexpr int BCP = 32 / BCR;                    // rows of B and C per pass
    static constexpr int BCV = kTile / BCP;
    static constexpr int ARRAYS = MODE == kState ? 2 : MODE == kFull ? 3 : 4;
    // rows of a value per channel, shifted by a quarter of a bank row so that the four
    // rows that a pass writes or reads together do not meet in a bank
    static constexpr int ROW = CW + 8;
    static constexpr size_t rows_bytes = 3 * ARRAYS * PASSES * 32 * 8 * sizeof(T);
    static constexpr size_t bcr_bytes = 2 * BCV * 32 * 8 * sizeof(T);
    static constexpr size_t smem = rows_bytes + bcr_bytes + 2 * kTile * (2 * ROW + 2 * NP + (MODE == kFull ? NW * ROW : MODE == kMaps ? ROW : 0)) * 4;
};

template <typename T, int NPT, int NW, int MODE>
__global__ void __launch_bounds__(32 * (NW + 1), NW == 1 ? (MODE == kMaps ? 6 : 7) : NW == 2 ? 4 : 2) scan_kernel(ScanArgs a) {
    using S = ScanShape<T, NPT, NW, MODE>;
    constexpr int CW = S::CW, NP = S::NP, VPR = S::VPR, RPP = S::RPP, PASSES = S::PASSES, M = NPT / 2, TILE = kTile;
    extern __shared__ __align__(16) unsigned char smem[];
    using Piece = T[8];
    Piece *rows = reinterpret_cast<Piece *>(smem);                              // [3][ARRAYS][PASSES][lane]
    Piece *bcr = reinterpret_cast<Piece *>(smem + S::rows_bytes);               // [2][BCV][lane]
    float *sd = reinterpret_cast<float *>(smem + S::rows_bytes + S::bcr_bytes); // [2][TILE][2][ROW]: step, step * x
    float *bc = sd + 2 * TILE * 2 * S::ROW;                                     // [2][TILE][2][NP]
    float *ys = bc + 2 * TILE * 2 * NP;                                         // kFull: [2][NW][TILE][ROW], y
    float *gs = ys;                                                             // kMaps: [2][TILE][ROW], dy through the gate

    grid_dependency_wait();
    if (MODE == kFull && a.status && a.cu && blockIdx.x == 0) check_cu(a.cu, a.n_seqs, a.T, a.status);
    const int lane = threadIdx.x & 31;
    int warp = threadIdx.x >> 5;
    if (NW == 1) {
        // Two warps of a block lie on neighbouring schedulers of the SM's four: were the
        // first one always the scanning one, half of the schedulers would feed only.
        __shared__ unsigned slot;
        if (threadIdx.x == 0) asm volatile("mov.u32 %0, %%warpid;" : "=r"(slot));
        __syncthreads();
        warp ^= slot >> 2 & 1;
    }
    const int chan0 = (blockIdx.x % a.chan_blocks) * CW;
    // the last segment of a row needs no map
    const int spr = MODE == kState ? a.segs - 1 : a.segs;
    Span r;
    r.b = blockIdx.x / a.chan_blocks / spr;
    const int seg = r.b * a.segs + blockIdx.x / a.chan_blocks % spr;
    const int walked = MODE == kMaps ? a.span_tokens : a.seg_tokens;
    r.t0 = (seg - r.b * a.segs) * walked;
    r.t1 = min(a.T, r.t0 + walked);
    const int tiles = r.t0 < r.t1 ? (r.t1 - r.t0 + TILE - 1) / TILE : 0;

    if (warp == NW) {   // the feeding warp: lane -> (row of the pass, eight channels)
        if (tiles == 0) return;
        const int lv = lane % VPR, lrow = lane / VPR, lc = chan0 + lv * 8, lrest = a.D - lc;
        const bool gated = MODE != kState && a.z != nullptr;
        const long long first = r.t0 + lrow;
        const T *px = static_cast<const T *>(a.x) + r.b * a.x_batch + first * a.x_token + lc;
        const T *pd = static_cast<const T *>(a.dt) + r.b * a.dt_batch + first * a.dt_token + lc;
        const T *pz = static_cast<const T *>(a.z) + r.b * a.z_batch + first * a.z_token + lc;
        const T *pg = MODE == kMaps ? static_cast<const T *>(a.dy) + r.b * a.dy_batch + first * a.dy_token + lc : nullptr;
        T *py = MODE != kFull ? nullptr : static_cast<T *>(a.out) + ((long long)r.b * a.T + first) * a.D + lc;
        const int bcc = lane / (NP / 8) % 2, bcn = lane % (NP / 8) * 8, bcrow = lane / S::BCR;
        const long long bc_token = bcc ? a.c_token : a.b_token;
        const T *pbc = (bcc ? static_cast<const T *>(a.Cm) + r.b * a.c_batch : static_cast<const T *>(a.Bm) + r.b * a.b_batch) +
                       (r.t0 + bcrow) * bc_token + bcn;
        const bool whole = a.vec && lrest >= 8 && a.bc_vec && a.N - bcn >= 8;
        auto piece = [&](int k, int array, int i) -> T * { return rows[((k % 3 * S::ARRAYS + array) * PASSES + i) * 32 + lane]; };
        auto bc_piece = [&](int k, int i) -> T * { return bcr[(k % 2 * S::BCV + i) * 32 + lane]; };
        F2 bias[4], skip[4];
        load_pairs(a.bias ? a.bias + lc : nullptr, 0, lrest, true, bias);
        load_pairs(MODE == kFull && a.skip ? a.skip + lc : nullptr, 0, lrest, true, skip);
        auto stage = [&](int k) {   // copies tile k and moves the pointers on to the next
            const int t = r.t0 + k * TILE;
            if (whole && t + TILE <= r.t1) {
#pragma unroll
                for (int i = 0; i < PASSES; ++i) {
                    copy8_whole<T>(piece(k, 0, i), px + i * RPP * a.x_token);
                    copy8_whole<T>(piece(k, 1, i), pd + i * RPP * a.dt_token);
                    if (gated) copy8_whole<T>(piece(k, 2, i), pz + i * RPP * a.z_token);
                    if (MODE == kMaps) copy8_whole<T>(piece(k, 3, i), pg + i * RPP * a.dy_token);
                }
#pragma unroll
                for (int i = 0; i < S::BCV; ++i) copy8_whole<T>(bc_piece(k, i), pbc + i * S::BCP * bc_token);
            } else if (t < r.t1) {
#pragma unroll
                for (int i = 0; i < PASSES; ++i) {
                    const int n = t + i * RPP + lrow < r.t1 ? lrest : 0;
                    copy8_async<T>(piece(k, 0, i), px + i * RPP * a.x_token, n, a.vec);
                    copy8_async<T>(piece(k, 1, i), pd + i * RPP * a.dt_token, n, a.vec);
                    if (gated) copy8_async<T>(piece(k, 2, i), pz + i * RPP * a.z_token, n, a.vec);
                    if (MODE == kMaps) copy8_async<T>(piece(k, 3, i), pg + i * RPP * a.dy_token, n, a.vec);
                }
#pragma unroll
                for (int i = 0; i < S::BCV; ++i)
                    copy8_async<T>(bc_piece(k, i), pbc + i * S::BCP * bc_token,
                                   t + i * S::BCP + bcrow < r.t1 ? a.N - bcn : 0, a.bc_vec);
            }
            px += TILE * a.x_token, pd += TILE * a.dt_token, pz += TILE * a.z_token;
            if (MODE == kMaps) pg += TILE * a.dy_token;
            pbc += TILE * bc_token;
            copy_commit();
        };
        auto prepare = [&](int k) {
            float *s_at = sd + k % 2 * TILE * 2 * S::ROW, *bc_at = bc + k % 2 * TILE * 2 * NP;
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                float *at = s_at + (i * RPP + lrow) * 2 * S::ROW + lv * 2;
                F2 x[4], d[4];
                unpack_pairs<T>(load_raw<T, 8>(piece(k, 0, i)), x);
                unpack_pairs<T>(load_raw<T, 8>(piece(k, 1, i)), d);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    d[e] = add2(d[e], bias[e]);
                    const F2 s = a.softplus ? softplus_pair(d[e]) : d[e];
                    *reinterpret_cast<F2 *>(at + e * VPR * 2) = s;
                    *reinterpret_cast<F2 *>(at + S::ROW + e * VPR * 2) = mul2(s, x[e]);
                }
                if (MODE == kMaps) {
                    float *g_at = gs + (k % 2 * TILE + i * RPP + lrow) * S::ROW + lv * 2;
                    F2 g[4], z[4];
                    unpack_pairs<T>(load_raw<T, 8>(piece(k, 3, i)), g);
                    if (gated) unpack_pairs<T>(load_raw<T, 8>(piece(k, 2, i)), z);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (gated) g[e] = mul2(g[e], mul2(z[e], sigmoid_pair(z[e])));
                        *reinterpret_cast<F2 *>(g_at + e * VPR * 2) = g[e];
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < S::BCV; ++i) {
                F2 f[4];
                unpack_pairs<T>(load_raw<T, 8>(bc_piece(k, i)), f);
                ulonglong2 *at = reinterpret_cast<ulonglong2 *>(bc_at + ((i * S::BCP + bcrow) * 2 + bcc) * NP + bcn);
                at[0] = make_ulonglong2(f[0], f[1]);
                at[1] = make_ulonglong2(f[2], f[3]);
            }
        };
        auto finish = [&](int k) {
            const float *y_at = ys + k % 2 * NW * TILE * S::ROW + lv * 2;
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                const int q = i * RPP + lrow;
                if (r.t0 + k * TILE + q >= r.t1) continue;
                F2 x[4], z[4];
                float o[8];
                unpack_pairs<T>(load_raw<T, 8>(piece(k, 0, i)), x);
                if (gated) unpack_pairs<T>(load_raw<T, 8>(piece(k, 2, i)), z);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float *at = y_at + q * S::ROW + e * VPR * 2;
                    F2 y = *reinterpret_cast<const F2 *>(at);
#pragma unroll
                    for (int w = 1; w < NW; ++w) y = add2(y, *reinterpret_cast<const F2 *>(at + w * TILE * S::ROW));
                    y = fma2(skip[e], x[e], y);
                    if (gated) y = mul2(y, mul2(z[e], sigmoid_pair(z[e])));
                    o[2 * e] = lo(y), o[2 * e + 1] = hi(y);
                }
                store8<T>(py + (long long)i * RPP * a.D, o, lrest, a.vec);
            }
            py += (long long)TILE * a.D;
        };
        stage(0);
        stage(1);
        copy_wait<1>();
        prepare(0);
        __syncthreads();
        for (int k = 0; k < tiles; ++k) {
            if (MODE == kFull && k > 0) finish(k - 1);
            stage(k + 2);
            copy_wait<1>();
            if (k + 1 < tiles) prepare(k + 1);
            __syncthreads();
        }
        if (MODE == kFull) finish(tiles - 1);
        return;
    }

    // a scanning warp: the channels in the order in which the feeding lanes lay them
    // down, pair e of vector v at place e VPR + v
    const int n0 = warp * NPT, ch = chan0 + lane / 2 % VPR * 8 + lane / 2 / VPR * 2 + lane % 2;
    const bool live = ch < a.D;
    if (MODE == kFull && a.final_state && live) {    // a sequence without a token keeps its state
        auto keep = [&](int n) {
            const long long at = ((long long)n * a.D + ch) * a.N;
            F2 v[M];
            load_pairs(a.init ? a.init + at : nullptr, n0, a.N, true, v);
            store_pairs(a.final_state + at, n0, a.N, v);
        };
        if (!a.cu && a.T == 0) keep(r.b);
        for (int n = seg; a.cu && n < a.n_seqs; n += a.segs)
            if (__ldg(a.cu + n) >= __ldg(a.cu + n + 1)) keep(n);
    }
    if (tiles == 0) return;
    F2 A2[M], h[M];
    load_pairs(a.A + (long long)ch * a.N, n0, a.N, live, A2);
#pragma unroll
    for (int i = 0; i < M; ++i) A2[i] = mul2(A2[i], both(kLog2e));
    span_find(a, r);
    bool starts = r.begin == r.t0, inside = false;
    auto initial = [&](int n) {
        load_pairs(a.init ? a.init + ((long long)n * a.D + ch) * a.N : nullptr, n0, a.N, live, h);
    };
    if (starts) initial(r.n);
    else load_aligned(a.hloc + ((long long)seg * a.D + ch) * NP + n0, live && MODE == kFull && a.has_carry, h);
    float step_sum = 0.f;
    F2 p[M], G[M];   // kMaps: the product of the a's so far, the gradient at the tile's start
    auto token = [&](auto with_g, int j, const float *s_at, const float *bc_at, float *y_at) {
        const float step = s_at[j * 2 * S::ROW];
        const F2 ss = both(step), sx = both(s_at[j * 2 * S::ROW + S::ROW]);
        const ulonglong2 *Bk = reinterpret_cast<const ulonglong2 *>(bc_at + j * 2 * NP);
        const ulonglong2 *Ck = reinterpret_cast<const ulonglong2 *>(bc_at + j * 2 * NP + NP);
        F2 y0 = both(0.f), y1 = both(0.f), gg = both(0.f);
        if (with_g) gg = both(y_at[j * S::ROW]);
#pragma unroll
        for (int i = 0; i < M / 2; ++i) {
            const ulonglong2 b = Bk[i];
            const F2 e0 = exp2_pair(mul2(ss, A2[2 * i])), e1 = exp2_pair(mul2(ss, A2[2 * i + 1]));
            h[2 * i] = fma2(e0, h[2 * i], mul2(sx, b.x));
            h[2 * i + 1] = fma2(e1, h[2 * i + 1], mul2(sx, b.y));
            if (MODE == kFull) {
                const ulonglong2 c = Ck[i];
                y0 = i ? fma2(c.x, h[2 * i], y0) : mul2(c.x, h[0]);
                y1 = i ? fma2(c.y, h[2 * i + 1], y1) : mul2(c.y, h[1]);
            }
            if (with_g) {
                const ulonglong2 c = Ck[i];
                p[2 * i] = mul2(p[2 * i], e0);
                p[2 * i + 1] = mul2(p[2 * i + 1], e1);
                G[2 * i] = fma2(p[2 * i], mul2(gg, c.x), G[2 * i]);
                G[2 * i + 1] = fma2(p[2 * i + 1], mul2(gg, c.y), G[2 * i + 1]);
            }
        }
        if (MODE == kFull) {
            y0 = add2(y0, y1);
            y_at[j * S::ROW] = lo(y0) + hi(y0);
        } else {
            step_sum += step;
        }
    };
    using Yes = std::integral_constant<bool, MODE == kMaps>;
    using No = std::integral_constant<bool, false>;
    __syncthreads();
    for (int k = 0; k < tiles; ++k) {
        const int t = r.t0 + k * TILE, stop = min(r.t1, t + TILE);
        const float *s_at = sd + k % 2 * TILE * 2 * S::ROW + lane, *bc_at = bc + k % 2 * TILE * 2 * NP + n0;
        float *y_at = MODE == kFull ? ys + (k % 2 * NW + warp) * TILE * S::ROW + lane : gs + k % 2 * TILE * S::ROW + lane;
        if (MODE == kMaps) {
            const bool here = r.begin == t;
            if (t % a.seg_tokens == 0) {   // a new segment
                starts = here, inside = false, step_sum = 0.f;
#pragma unroll
                for (int i = 0; i < M; ++i) p[i] = both(1.f), G[i] = h[i] = both(0.f);
            } else if (here) {
                inside = true;
            }
            if (here) initial(r.n);
            if (live && t % a.seg_tokens != 0) {
                const long long tile = (long long)r.b * a.row_tiles + t / TILE;
                store_aligned(a.htile + (tile * a.D + ch) * NP + n0, h);
                if (warp == 0) a.stile[tile * a.D + ch] = step_sum;
                if (chan0 == 0 && warp == 0 && lane == 0) a.exact[tile] = starts || inside;
            }
        }
        for (int q = t; q < stop;) {
            const int run_end = min(stop, r.end);
            if (run_end - q == TILE && !(MODE == kMaps && inside)) {
                // the usual case, with addresses known: unrolled whole (179 us on the batch
                // of prompts where four at a time take 197), but for the longer token of
                // kMaps (16 at a time miss the instruction cache: 322 us against 314)
#pragma unroll(MODE == kMaps ? 4 : TILE)
                for (int j = 0; j < TILE; ++j) token(Yes(), j, s_at, bc_at, y_at);
            } else if (MODE == kMaps && !inside) {
                for (int j = q - t; j < run_end - t; ++j) token(Yes(), j, s_at, bc_at, y_at);
            } else {
                for (int j = q - t; j < run_end - t; ++j) token(No(), j, s_at, bc_at, y_at);
            }
            q = run_end;
            if (q == r.end) {   // the sequence is complete
                const long long at = ((long long)r.n * a.D + ch) * a.N;
                if (MODE == kFull && a.final_state && live) store_pairs(a.final_state + at, n0, a.N, h);
                if (MODE == kMaps && !inside && a.d_final) {
                    F2 f[M];
                    load_pairs(a.d_final + at, n0, a.N, live, f);
#pragma unroll
                    for (int i = 0; i < M; ++i) G[i] = fma2(p[i], f[i], G[i]);
                }
                if (q < r.t1) {
                    span_next(a, r, q);
                    if (MODE != kMaps || q < stop) initial(r.n), inside = true;   // (a tile's start: at its top)
                }
            }
        }
        if (MODE == kMaps && live && (stop % a.seg_tokens == 0 || stop == a.T)) {   // the segment is complete
            const long long at = (long long)r.b * ((a.T + a.seg_tokens - 1) / a.seg_tokens) + t / a.seg_tokens;
            store_aligned(a.hloc + (at * a.D + ch) * NP + n0, h);
            store_aligned(a.gloc + (at * a.D + ch) * NP + n0, G);
            if (warp == 0) a.sums[at * a.D + ch] = step_sum;
            if (chan0 == 0 && warp == 0 && lane == 0) a.flags[at] = (starts ? 1 : 0) | (inside ? 2 : 0);
        }
        __syncthreads();
    }
    if (MODE == kState) {
        if (live) {
            store_aligned(a.hloc + ((long long)seg * a.D + ch) * NP + n0, h);
            if (warp == 0) a.sums[(long long)seg * a.D + ch] = step_sum;
        }
        if (chan0 == 0 && warp == 0 && lane == 0) a.flags[seg] = (starts ? 1 : 0) | (inside ? 2 : 0);
    }
}

// Replaces every map's end state by the state before it, and (GRAD) every
// map's start gradient by the gradient at its end.  A thread per (row, channel,
// n); eight maps are loaded ahead.
template <bool GRAD>
__global__ void __launch_bounds__(64) scan_combine_kernel(ScanArgs a, int maps, int NP) {
    constexpr int AHEAD = 8;
    grid_dependency_wait();
    const long long at = (long long)blockIdx.x * 64 + threadIdx.x, size = (long long)a.D * NP;
    if (at >= size) return;
    const int ch = (int)(at / NP), n = (int)(at % NP);
    const float A2 = n < a.N ? a.A[(long long)ch * a.N + n] * kLog2e : 0.f;
    const bool back = GRAD && blockIdx.z == 1;
    // the walk's first map and its direction
    const long long m0 = (long long)blockIdx.y * maps + (back ? maps - 1 : 0), dir = back ? -1 : 1;
    float *at_map = (back ? a.gloc : a.hloc) + m0 * size + at;
    const float *at_sum = a.sums + m0 * a.D + ch;
    const int32_t *at_flag = a.flags + m0;
    const long long map_step = dir * size, sum_step = dir * a.D;
    const int there = GRAD ? maps : maps - 1;   // forward only: the last map is not there
    float v[AHEAD], s[AHEAD], carry = 0.f;
    int f[AHEAD];
    float *ahead = at_map;
    auto load = [&](int i, int m) {
        const bool in = m < there;
        v[i] = in ? *ahead : 0.f;
        s[i] = in ? *at_sum : 0.f;
        f[i] = in ? *at_flag : 0;
        ahead += map_step, at_sum += sum_step, at_flag += dir;
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) load(i, i);
    for (int m = 0; m < maps; m += AHEAD) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (m + i >= maps) break;
            *at_map = carry;
            at_map += map_step;
            const float through = fmaf(exp2_f32(A2 * s[i]), carry, v[i]);
            carry = back ? (f[i] & 1 ? 0.f : f[i] & 2 ? v[i] : through) : f[i] ? v[i] : through;
            load(i, m + AHEAD + i);
        }
    }
}

// One token of each sequence: 4 n per thread, LANES threads per channel, so that a
// warp reads and writes 512 contiguous bytes of the states; bound by their traffic
// (32 x 4096 x 16, 18 MB: 6.0 us with the states in HBM, 3.0 TB/s, 45% of the
// measured copy rate: a thread has one 16-byte load of its state in flight).
template <typename T, int LANES>
__global__ void __launch_bounds__(128) scan_step_kernel(ScanArgs a, int vec) {
    const int part = threadIdx.x % LANES, ch = (int)((blockIdx.x * 128ll + threadIdx.x) / LANES);
    const int b = blockIdx.y, n0 = part * 4;
    const bool live = ch < a.D;
    grid_dependency_wait();
    const int slot = a.slots ? __ldg(a.slots + b) : b;
    if (slot < 0 || slot >= a.pool) {   // a padded row
        if (live && part == 0) static_cast<T *>(a.out)[(long long)b * a.D + ch] = from_f32<T>(0.f);
        return;
    }
    float y = 0.f, x = 0.f;
    if (live) {
        float *state = a.final_state + ((long long)slot * a.D + ch) * a.N + n0;
        const float *A = a.A + (long long)ch * a.N + n0;
        float h[4], av[4], Bv[4], Cv[4];
        const T *B = static_cast<const T *>(a.Bm) + b * a.b_batch + n0, *C = static_cast<const T *>(a.Cm) + b * a.c_batch + n0;
        if (vec && n0 < a.N) {
            const float4 hv = *reinterpret_cast<const float4 *>(state), aw = *reinterpret_cast<const float4 *>(A);
            h[0] = hv.x, h[1] = hv.y, h[2] = hv.z, h[3] = hv.w;
            av[0] = aw.x, av[1] = aw.y, av[2] = aw.z, av[3] = aw.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = n0 + i < a.N ? state[i] : 0.f, av[i] = n0 + i < a.N ? A[i] : 0.f;
        }
        if (a.bc_vec && n0 + 4 <= a.N) {
            unpack<T, 4>(load_raw<T, 4>(B), Bv);
            unpack<T, 4>(load_raw<T, 4>(C), Cv);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) Bv[i] = n0 + i < a.N ? to_f32(B[i]) : 0.f, Cv[i] = n0 + i < a.N ? to_f32(C[i]) : 0.f;
        }
        x = to_f32(static_cast<const T *>(a.x)[b * a.x_batch + ch]);
        float s = to_f32(static_cast<const T *>(a.dt)[b * a.dt_batch + ch]) + (a.bias ? a.bias[ch] : 0.f);
        if (a.softplus) s = softplus_f32(s);
        const float sx = s * x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] = fmaf(exp2_f32(s * kLog2e * av[i]), h[i], sx * Bv[i]);
            y = fmaf(Cv[i], h[i], y);
        }
        if (vec && n0 < a.N) {
            *reinterpret_cast<float4 *>(state) = make_float4(h[0], h[1], h[2], h[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n0 + i < a.N) state[i] = h[i];
        }
    }
#pragma unroll
    for (int off = 1; off < LANES; off <<= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
    if (live && part == 0) {
        y = fmaf(a.skip ? a.skip[ch] : 0.f, x, y);
        if (a.z) {
            const float z = to_f32(static_cast<const T *>(a.z)[b * a.z_batch + ch]);
            y *= z * sigmoid_f32(z);
        }
        static_cast<T *>(a.out)[(long long)b * a.D + ch] = from_f32<T>(y);
    }
}

// Blocks of the scanning kernels that the plans count on per SM, by N: what
// registers and shared memory leave for bf16 inputs.  The plans do not know the
// type: with fp32 inputs and N <= 16 shared memory holds 5 of the 7, so a row cut
// for 7 runs as a wave and a part of one (8 x 1024 tokens x 4096 channels 225 us,
// bf16 171; a row of 32768 x 1024 342 us, bf16 287).
int scan_resident(int N) { return N <= 16 ? 7 : N <= 32 ? 4 : 2; }

template <typename T, int NPT, int NW, int MODE>
cudaError_t launch_scan_one(const ScanArgs &a, int segs, cudaStream_t s) {
    using S = ScanShape<T, NPT, NW, MODE>;
    if (S::smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(scan_kernel<T, NPT, NW, MODE>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::smem);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)((long long)a.chan_blocks * a.B * segs));
    return launch_dependent(scan_kernel<T, NPT, NW, MODE>, grid, dim3(32 * (NW + 1)), S::smem, s, a);
}

template <typename T, int NPT, int NW>
cudaError_t launch_scan_parts(ScanArgs a, cudaStream_t s) {
    a.chan_blocks = (a.D + 31) / 32;
    a.has_carry = a.segs > 1;
    if (a.segs > 1) {
        cudaError_t e = launch_scan_one<T, NPT, NW, kState>(a, a.segs - 1, s);
        if (e == cudaSuccess) e = launch_scan_combine(a, a.segs, false, s);
        if (e != cudaSuccess) return e;
    }
    return launch_scan_one<T, NPT, NW, kFull>(a, a.segs, s);
}

template <typename T>
cudaError_t launch_scan_typed(const ScanArgs &a, cudaStream_t s) {
    if (a.N <= 8) return launch_scan_parts<T, 8, 1>(a, s);
    if (a.N <= 16) return launch_scan_parts<T, 16, 1>(a, s);
    if (a.N <= 32) return launch_scan_parts<T, 16, 2>(a, s);
    return launch_scan_parts<T, 16, 4>(a, s);
}

template <typename T>
cudaError_t launch_step_typed(const ScanArgs &a, int vec, cudaStream_t s) {
    const int lanes = a.N <= 8 ? 2 : a.N <= 16 ? 4 : a.N <= 32 ? 8 : 16;
    const dim3 grid((unsigned)(((long long)a.D * lanes + 127) / 128), a.B);
    void (*kernel)(ScanArgs, int) = lanes == 2 ? scan_step_kernel<T, 2> : lanes == 4 ? scan_step_kernel<T, 4>
                                  : lanes == 8 ? scan_step_kernel<T, 8> : scan_step_kernel<T, 16>;
    return launch_dependent(kernel, grid, dim3(128), 0, s, a, vec);
}

// Segments per row in the forward pass.  One segment takes each exponential
// once; several take it twice but put that many times the blocks to work: they
// are cut when whole rows leave half of the SMs' room free, as many as fill it
// once (at bf16's room).
int scan_segments(int B, int T, int D, int N) {
    const int tiles = (T + kTile - 1) / kTile;
    const long long blocks = (long long)B * ((D + 31) / 32), room = (long long)scan_resident(N) * device_sm_count();
    if (tiles <= 1 || blocks == 0 || 2 * blocks > room) return 1;
    const int segs = (int)std::min<long long>(room / blocks, tiles);
    const int len = (tiles + segs - 1) / segs;
    return (tiles + len - 1) / len;
}
int scan_segment_tokens(int T, int segs) {
    const int tiles = (T + kTile - 1) / kTile;
    return std::max(1, (tiles + segs - 1) / segs) * kTile;
}

}  // namespace

namespace {

// Segments of `tiles` tiles that a block of the maps walks: what gives the
// shortest schedule on six blocks per SM, with a tile's time for a block's own
// start and end; that schedule's length in tiles.  Six is what an SM holds for bf16
// inputs and N <= 16 (fp32: four; N up to 32 four, above two), for the others it
// only weighs the choices.
int maps_per_block(int B, int row_segs, int tiles, int chan_blocks, long long *cost) {
    const long long slots = 6ll * device_sm_count(), unit = (long long)B * chan_blocks;
    int per = 1;
    *cost = 0;
    if (unit == 0) return per;   // no batch rows
    *cost = (unit * row_segs + slots - 1) / slots * (tiles + 1);
    for (int waves = 1; waves <= 4; ++waves) {   // the fewest segments per block that fit so many waves
        const long long per_row = waves * slots / unit;
        if (per_row < 1 || row_segs < 1) continue;
        const int m = (int)((row_segs + per_row - 1) / per_row);
        const long long c = waves * ((long long)m * tiles + 1);
        if (c < *cost) *cost = c, per = m;
    }
    return per;
}

}  // namespace

cudaError_t launch_scan_maps(const ScanArgs &p, int dtype, cudaStream_t s) {
    ScanArgs a = p;
    a.chan_blocks = (a.D + 31) / 32;
    const int per_seg = a.seg_tokens / kTile, row_segs = (a.row_tiles + per_seg - 1) / per_seg;
    long long cost = 0;
    const int per = maps_per_block(a.B, row_segs, per_seg, a.chan_blocks, &cost);
    a.segs = (row_segs + per - 1) / per;
    a.span_tokens = per * a.seg_tokens;
#define GDN_MAPS(NPT, NW) \
    (dtype == GDN_BF16 ? launch_scan_one<__nv_bfloat16, NPT, NW, kMaps>(a, a.segs, s) : launch_scan_one<float, NPT, NW, kMaps>(a, a.segs, s))
    if (a.N <= 8) return GDN_MAPS(8, 1);
    if (a.N <= 16) return GDN_MAPS(16, 1);
    if (a.N <= 32) return GDN_MAPS(16, 2);
    return GDN_MAPS(16, 4);
#undef GDN_MAPS
}

cudaError_t launch_scan_combine(const ScanArgs &a, int maps, bool grad, cudaStream_t s) {
    const int NP = 8 * scan_parts(a.N);
    const dim3 grid((unsigned)(((long long)a.D * NP + 63) / 64), a.B, grad ? 2 : 1);
    return grad ? launch_dependent(scan_combine_kernel<true>, grid, dim3(64), 0, s, a, maps, NP)
                : launch_dependent(scan_combine_kernel<false>, grid, dim3(64), 0, s, a, maps, NP);
}

namespace {

gdn_status scan_desc_ok(const gdn_scan_desc *p) {
    if (!p || p->B < 0 || p->T < 0 || p->D < 1 || p->N < 1) return GDN_ERR_INVALID_ARG;
    if (p->dtype != GDN_BF16 && p->dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    // token and channel indices are 32-bit
    if (p->N > 64 || p->B > 65535 || p->T > (1 << 30) || p->D > (1 << 26)) return GDN_ERR_UNSUPPORTED;
    if (p->cu_seqlens && (p->B != 1 || p->n_seqs < 1)) return GDN_ERR_INVALID_ARG;
    if (p->B > 0 && (!p->A || (p->T > 0 && (!p->x || !p->dt || !p->B_ || !p->C_)))) return GDN_ERR_INVALID_ARG;
    const int64_t chan[] = {p->x_token_stride, p->dt_token_stride, p->z ? p->z_token_stride : p->D};
    for (int64_t st : chan)
        if (st < p->D) return GDN_ERR_INVALID_ARG;
    if (p->b_token_stride < p->N || p->c_token_stride < p->N) return GDN_ERR_INVALID_ARG;
    const int64_t batch[] = {p->x_batch_stride, p->dt_batch_stride, p->z_batch_stride, p->b_batch_stride,
                             p->c_batch_stride};
    for (int64_t st : batch)
        if (st < 0) return GDN_ERR_INVALID_ARG;
    const uintptr_t em = p->dtype == GDN_F32 ? 3 : 1;
    const void *elems[] = {p->x, p->dt, p->z, p->B_, p->C_};
    for (const void *q : elems)
        if (reinterpret_cast<uintptr_t>(q) & em) return GDN_ERR_INVALID_ARG;
    const void *f32[] = {p->A, p->D_skip, p->dt_bias, p->initial_state, p->cu_seqlens};
    for (const void *q : f32)
        if (reinterpret_cast<uintptr_t>(q) & 3) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

bool all_aligned(const void *const *ptrs, int n, const int64_t *strides, int m, int elems) {
    bool ok = true;
    for (int i = 0; i < n; ++i) ok = ok && aligned16(ptrs[i]);
    for (int i = 0; i < m; ++i) ok = ok && strides[i] % elems == 0;
    return ok;
}

ScanArgs scan_args(const gdn_scan_desc &p) {
    ScanArgs a = {};
    a.x = p.x, a.dt = p.dt, a.z = p.z, a.Bm = p.B_, a.Cm = p.C_;
    a.A = p.A, a.skip = p.D_skip, a.bias = p.dt_bias, a.init = p.initial_state, a.cu = p.cu_seqlens;
    a.x_batch = p.x_batch_stride, a.x_token = p.x_token_stride, a.dt_batch = p.dt_batch_stride;
    a.dt_token = p.dt_token_stride, a.z_batch = p.z_batch_stride, a.z_token = p.z_token_stride;
    a.b_batch = p.b_batch_stride, a.b_token = p.b_token_stride, a.c_batch = p.c_batch_stride;
    a.c_token = p.c_token_stride;
    a.B = p.B, a.T = p.T, a.D = p.D, a.N = p.N, a.n_seqs = p.cu_seqlens ? p.n_seqs : p.B;
    a.softplus = p.dt_softplus != 0;
    const int per = p.dtype == GDN_F32 ? 4 : 8;   // elements of 16 bytes
    const void *wide[] = {p.x, p.dt, p.z};
    const int64_t ws[] = {p.x_batch_stride, p.x_token_stride, p.dt_batch_stride, p.dt_token_stride,
                          p.z ? p.z_batch_stride : 0, p.z ? p.z_token_stride : 0, p.D};
    a.vec = all_aligned(wide, 3, ws, 7, per);
    const void *bc[] = {p.B_, p.C_};
    const int64_t bs[] = {p.b_batch_stride, p.b_token_stride, p.c_batch_stride, p.c_token_stride};
    a.bc_vec = all_aligned(bc, 2, bs, 4, per);
    return a;
}

size_t round16(size_t n) { return (n + 15) & ~(size_t)15; }

// Workspace of the maps: end states (and start gradients), step sums, flags.
size_t maps_bytes(long long maps, int D, int N, int arrays) {
    const size_t np = 8 * (size_t)scan_parts(N);
    return arrays * round16(maps * D * np * 4) + round16(maps * (size_t)D * 4) + round16(maps * 4);
}
char *place_maps(ScanArgs &a, char *p, long long maps, int arrays) {
    const size_t np = 8 * (size_t)scan_parts(a.N);
    a.hloc = reinterpret_cast<float *>(p), p += round16(maps * a.D * np * 4);
    if (arrays == 2) a.gloc = reinterpret_cast<float *>(p), p += round16(maps * a.D * np * 4);
    a.sums = reinterpret_cast<float *>(p), p += round16(maps * (size_t)a.D * 4);
    a.flags = reinterpret_cast<int32_t *>(p), p += round16(maps * 4);
    return p;
}

}  // namespace

}  // namespace gdn

extern "C" size_t gdn_selective_scan_fwd_workspace_size(int B, int T, int D, int N) {
    if (B < 0 || T < 0 || D < 1 || N < 1 || N > 64) return 0;
    const int segs = gdn::scan_segments(B, T, D, N);
    return segs > 1 ? gdn::maps_bytes((long long)B * segs, D, N, 1) : 16;
}

extern "C" gdn_status gdn_selective_scan_fwd(const gdn_scan_desc *desc, void *y, float *final_state,
                                             int32_t *device_status, void *workspace, size_t workspace_bytes,
                                             gdn_stream_t stream) {
    using namespace gdn;
    const gdn_status st = scan_desc_ok(desc);
    if (st != GDN_OK) return st;
    const gdn_scan_desc &p = *desc;
    if (p.B == 0) return GDN_OK;
    const uintptr_t em = p.dtype == GDN_F32 ? 3 : 1;
    if ((p.T > 0 && !y) || (reinterpret_cast<uintptr_t>(y) & em) || (reinterpret_cast<uintptr_t>(final_state) & 3))
        return GDN_ERR_INVALID_ARG;
    ScanArgs a = scan_args(p);
    a.vec = a.vec && aligned16(y);
    a.out = y, a.final_state = final_state, a.status = device_status;
    a.segs = scan_segments(p.B, p.T, p.D, p.N);
    a.seg_tokens = scan_segment_tokens(p.T, a.segs);
    if (a.segs > 1) {
        if (!workspace || !aligned16(workspace)) return GDN_ERR_INVALID_ARG;
        if (workspace_bytes < gdn_selective_scan_fwd_workspace_size(p.B, p.T, p.D, p.N)) return GDN_ERR_WORKSPACE;
        place_maps(a, static_cast<char *>(workspace), (long long)p.B * a.segs, 1);
    }
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = p.dtype == GDN_BF16 ? launch_scan_typed<__nv_bfloat16>(a, s) : launch_scan_typed<float>(a, s);
    if (e != cudaSuccess) {
        set_error_detail("launch selective_scan_fwd", e);
        return GDN_ERR_CUDA;
    }
    return GDN_OK;
}

extern "C" gdn_status gdn_selective_scan_step(const gdn_scan_desc *desc, float *state, const int32_t *state_indices,
                                              int n_states, void *y, gdn_stream_t stream) {
    using namespace gdn;
    const gdn_status st = scan_desc_ok(desc);
    if (st != GDN_OK) return st;
    const gdn_scan_desc &p = *desc;
    if (p.T != 1 || p.cu_seqlens || n_states < 0 || (!state_indices && n_states < p.B)) return GDN_ERR_INVALID_ARG;
    if (p.B == 0) return GDN_OK;
    const uintptr_t em = p.dtype == GDN_F32 ? 3 : 1;
    if (!y || !state || (reinterpret_cast<uintptr_t>(y) & em) || (reinterpret_cast<uintptr_t>(state) & 3))
        return GDN_ERR_INVALID_ARG;
    ScanArgs a = scan_args(p);
    a.out = y, a.final_state = state, a.slots = state_indices, a.pool = n_states;
    const int vec = p.N % 4 == 0 && aligned16(state) && aligned16(p.A);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = p.dtype == GDN_BF16 ? launch_step_typed<__nv_bfloat16>(a, vec, s)
                                              : launch_step_typed<float>(a, vec, s);
    if (e != cudaSuccess) {
        set_error_detail("launch selective_scan_step", e);
        return GDN_ERR_CUDA;
    }
    return GDN_OK;
}

namespace gdn {
namespace {

// How the backward pass cuts a problem: tiles per row, segments of tiles that
// one block of the main kernel walks, blocks of channels.
struct BwdPlan {
    int row_tiles, segs, seg_tokens, chan_blocks;
    size_t maps, htile, stile, exact, part_a, part_v, part_bc;
};
BwdPlan bwd_plan(int B, int T, int D, int N) {
    BwdPlan p;
    const size_t np = 8 * (size_t)scan_parts(N);
    const int ch = scan_bwd_channels(N);
    p.row_tiles = (T + kTile - 1) / kTile;
    p.chan_blocks = (D + ch - 1) / ch;
    // tiles per segment: what gives the shortest schedule of the main kernel (two
    // blocks per SM, half a tile's time for a block's own start and end) and of the
    // maps, whose tile takes about 2/11 as long
    const long long slots = 2ll * device_sm_count();
    int per = 1;
    double best = 0;
    for (int m = 1; m <= 16 && m <= std::max(1, p.row_tiles); ++m) {
        const int row_segs = (p.row_tiles + m - 1) / m;
        const long long blocks = (long long)B * row_segs * p.chan_blocks;
        long long maps = 0;
        maps_per_block(B, row_segs, m, (D + 31) / 32, &maps);
        const double cost = (double)((blocks + slots - 1) / slots) * (m + 0.5) + maps * (2.0 / 11);
        if (m == 1 || cost < best) best = cost, per = m;
    }
    p.segs = std::max(1, (p.row_tiles + per - 1) / per);
    p.seg_tokens = per * kTile;
    const size_t tiles = (size_t)B * p.row_tiles;
    p.maps = maps_bytes((long long)B * p.segs, D, N, 2);
    p.htile = round16(tiles * D * np * 4);
    p.stile = round16(tiles * D * 4);
    p.exact = round16(tiles * 4);
    p.part_a = round16((size_t)B * p.segs * D * np * 4);
    p.part_v = round16((size_t)B * p.segs * 2 * D * 4);
    p.part_bc = round16((size_t)p.chan_blocks * B * T * 2 * np * 4);
    return p;
}

}  // namespace
}  // namespace gdn

extern "C" size_t gdn_selective_scan_bwd_workspace_size(int B, int T, int D, int N) {
    if (B < 0 || T < 0 || D < 1 || N < 1 || N > 64) return 0;
    const gdn::BwdPlan p = gdn::bwd_plan(B, T, D, N);
    return std::max<size_t>(16, p.maps + p.htile + p.stile + p.exact + p.part_a + p.part_v + p.part_bc);
}

extern "C" gdn_status gdn_selective_scan_bwd(const gdn_scan_desc *desc, const void *dy, int64_t dy_batch_stride,
                                             int64_t dy_token_stride, const float *d_final_state, void *dx, void *ddt,
                                             float *dA, void *dB, void *dC, float *dD_skip, void *dz,
                                             float *ddt_bias, float *d_initial_state, int32_t *device_status,
                                             void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    using namespace gdn;
    const gdn_status st = scan_desc_ok(desc);
    if (st != GDN_OK) return st;
    const gdn_scan_desc &p = *desc;
    if (dy_token_stride < p.D || dy_batch_stride < 0 || !dA) return GDN_ERR_INVALID_ARG;
    if (p.B > 0 && p.T > 0 && (!dy || !dx || !ddt || !dB || !dC || (p.z && !dz))) return GDN_ERR_INVALID_ARG;
    const uintptr_t em = p.dtype == GDN_F32 ? 3 : 1;
    const void *elems[] = {dy, dx, ddt, dB, dC, dz};
    for (const void *q : elems)
        if (reinterpret_cast<uintptr_t>(q) & em) return GDN_ERR_INVALID_ARG;
    const void *f32[] = {d_final_state, dA, dD_skip, ddt_bias, d_initial_state, device_status};
    for (const void *q : f32)
        if (reinterpret_cast<uintptr_t>(q) & 3) return GDN_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace)) return GDN_ERR_INVALID_ARG;
    if (workspace_bytes < gdn_selective_scan_bwd_workspace_size(p.B, p.T, p.D, p.N)) return GDN_ERR_WORKSPACE;
    ScanArgs a = scan_args(p);
    const int per = p.dtype == GDN_F32 ? 4 : 8;
    const void *wide[] = {dy, dx, ddt, dz};
    const int64_t ws[] = {dy_batch_stride, dy_token_stride};
    a.vec = a.vec && all_aligned(wide, 4, ws, 2, per);
    a.dy = dy, a.dy_batch = dy_batch_stride, a.dy_token = dy_token_stride, a.d_final = d_final_state;
    a.out = dx, a.ddt = ddt, a.dz = dz, a.dinit = d_initial_state, a.status = device_status;
    const BwdPlan plan = bwd_plan(p.B, p.T, p.D, p.N);
    a.row_tiles = plan.row_tiles, a.segs = plan.segs, a.seg_tokens = plan.seg_tokens, a.chan_blocks = plan.chan_blocks;
    char *at = place_maps(a, static_cast<char *>(workspace), (long long)p.B * plan.segs, 2);
    a.htile = reinterpret_cast<float *>(at), at += plan.htile;
    a.stile = reinterpret_cast<float *>(at), at += plan.stile;
    a.exact = reinterpret_cast<int32_t *>(at), at += plan.exact;
    a.part_a = reinterpret_cast<float *>(at), at += plan.part_a;
    a.part_v = reinterpret_cast<float *>(at), at += plan.part_v;
    a.part_bc = reinterpret_cast<float *>(at);
    const cudaError_t e = launch_scan_bwd(a, p.dtype, dB, dC, dA, dD_skip, ddt_bias, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) {
        set_error_detail("launch selective_scan_bwd", e);
        return GDN_ERR_CUDA;
    }
    return GDN_OK;
}
