// Backward pass of the selective state space scan.  With the forward pass's
// h_t = a_t h_{t-1} + s_t x_t B_t, a_t = exp(s_t A), y_t = C_t.h_t + D x_t,
// out_t = y_t silu(z_t) and g_t = dout_t silu(z_t), per channel and n
//
//     dh_t = C_t g_t + a_{t+1} dh_{t+1}          (+ d_final at a sequence's end),
//     dC_t = sum_channels g_t h_t,     dB_t = sum_channels s_t x_t dh_t,
//     q_t = dh_t a_t h_{t-1},          dA = sum_t s_t q_t,
//     ds_t = sum_n q_t A + x_t u_t,    dx_t = s_t u_t + D g_t,   u_t = sum_n dh_t B_t,
//     dz_t = dout_t y_t silu'(z_t),    dD = sum_t g_t x_t,   ddt = ds softplus'.
//
// Both recurrences run over segments of a few tiles of 16 tokens in parallel.  A
// first kernel (scan_kernel in its kMaps mode) gives every segment's two maps
// from one pass over its exponentials: the end state from a zero start, and the
// gradient at its start from a zero gradient at its end, which needs no reversed
// pass: with the running product p_t of the a's it is sum_t p_t C_t g_t.  It also
// keeps the state before every tile.  scan_combine_kernel turns the maps into
// every segment's exact start state and end gradient; a tile's start state is
// what the first kernel kept plus exp(A sum s) times the segment's.  The main
// kernel takes a segment's tiles from the last to the first: each is walked
// forward, keeping the state at every second token in shared memory, then
// backward two tokens at a time, whose states are recomputed in registers.
//
// What bounds the main kernel is the instructions around its 14 multiply-adds and
// two exponentials per (token, channel, n): the sums over n (for the gradients
// per channel) and over channels (for dB and dC).  A thread holds eight n of CS
// channels, so that both sums are first taken in registers and what is per
// (token, channel) serves eight n; each exchange between lanes then halves the
// values still carried (a reduce-scatter).  The first two exchanges of dB and dC
// need no selection of the half to keep: the lanes hold their n in different
// orders, so that every lane keeps the same registers.  Sums over warps, blocks
// and tokens are added in a fixed order: no atomics, the same inputs give the
// same bits.
//
// Measured (bf16, 16 n, 4099 packed tokens x 2048 channels): 301 us, of it 75 the
// maps, 9 their combination, 8 the sums over blocks, the rest the main kernel
// (26 instructions per (token, channel, n), 1.6 per clock on the eight warps per
// SM that 254 registers leave).  Of the main kernel the gradients' last step (dx,
// ddt, dz) is 27 us, the walk forward 27, the sums over channels 20, over n 11.
// With four n of four channels per thread it took 366 us instead of 225.  fp32
// inputs, which are not staged: 350 us.
#include <algorithm>
#include <type_traits>

#include "scan_pairs.cuh"

namespace gdn {

namespace {

// V values per lane summed over the lanes that differ in the bits MASK, MASK / 2,
// ..., LAST: each exchange hands half of the values over and keeps the other
// half, once a single value is left it is added on both sides.  `base` becomes
// the index of the first value this lane is left with.
template <int V, int MASK, int LAST>
__device__ __forceinline__ void reduce_scatter(float *v, int lane, int &base) {
    if constexpr (MASK >= LAST) {
        const bool up = (lane & MASK) != 0;
        if constexpr (V > 1) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float give = up ? v[i] : v[i + V / 2], keep = up ? v[i + V / 2] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, MASK);
            }
            base += up ? V / 2 : 0;
            reduce_scatter<V / 2, MASK / 2, LAST>(v, lane, base);
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], MASK);
            reduce_scatter<1, MASK / 2, LAST>(v, lane, base);
        }
    }
}

constexpr int kBwdThreads = 128;
constexpr int kBwdWarps = kBwdThreads / 32;
constexpr int kBlock = 2;                      // tokens per block of the backward walk
constexpr int kBlocks = kTile / kBlock;

// NL lanes share a channel (eight n each), CS channels per lane.
template <int NL>
struct BwdShape {
    static constexpr int CS = NL == 1 ? 1 : 2;
    static constexpr int CL = 32 / NL;                   // lanes over channels, four at least
    static constexpr int WC = CL * CS;                   // channels of a warp
    static constexpr int CH = WC * kBwdWarps;            // of the block
    static constexpr int NP = 8 * NL;
    static constexpr int VL = 32 / CL;                   // dB, dC sums left per lane and block of tokens
    // float4 per warp and block of tokens: the states before it, later its dB and
    // dC sums (2 tokens x 2 x NP; those of block 0 behind those of block 1)
    static constexpr int REGION = CS * 2 * 32;
    static constexpr int VPR = CH / 8;                   // vectors of eight channels per row
    static constexpr int PASSES = kBwdThreads / VPR >= kTile ? 1 : kTile * VPR / kBwdThreads;
    static constexpr int BCV = (kTile * 2 * NL + kBwdThreads - 1) / kBwdThreads;
    static constexpr size_t smem = (kBlocks - 1) * kBwdWarps * REGION * 16 + 3 * kTile * CH * 4 + kTile * 2 * NP * 4 +
                                   kTile * 4 + 16;
    // raw x, dt, z, dy, B and C of the next tile: where two blocks per SM have the
    // room (16-bit inputs)
    template <typename T>
    static constexpr size_t staged = sizeof(T) == 2 ? (4 * PASSES + BCV) * kBwdThreads * 8 * sizeof(T) : 0;
    static_assert(2 * 4 * NP <= REGION * 4, "sums of two blocks of tokens in one region");
};

// Pairs of eight n of a row from n0: slot i holds pair i ^ perm.
__device__ __forceinline__ void load_perm(const float *row, int n0, int perm, int N, bool live, F2 (&h)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = n0 + 2 * (i ^ perm);
        h[i] = pair(row && live && n < N ? row[n] : 0.f, row && live && n + 1 < N ? row[n + 1] : 0.f);
    }
}
__device__ __forceinline__ void store_perm(float *row, int n0, int perm, int N, const F2 (&h)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = n0 + 2 * (i ^ perm);
        if (n < N) row[n] = lo(h[i]);
        if (n + 1 < N) row[n + 1] = hi(h[i]);
    }
}
// The same from a padded row, eight bytes at a time.
__device__ __forceinline__ void load_padded(const float *row, int n0, int perm, bool live, F2 (&h)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = live ? *reinterpret_cast<const F2 *>(row + n0 + 2 * (i ^ perm)) : both(0.f);
}
__device__ __forceinline__ F2 shfl_pair(F2 v, int mask) {
    return pair(__shfl_xor_sync(0xffffffffu, lo(v), mask), __shfl_xor_sync(0xffffffffu, hi(v), mask));
}

template <typename T, int NL>
__global__ void __launch_bounds__(kBwdThreads, 2) scan_bwd_kernel(ScanArgs a) {
    using S = BwdShape<NL>;
    constexpr int CS = S::CS, CL = S::CL, CH = S::CH, NP = S::NP, VL = S::VL;
    constexpr int VPR = S::VPR, RPP = kBwdThreads / VPR, PASSES = S::PASSES;
    constexpr bool STAGED = sizeof(T) == 2;
    extern __shared__ __align__(16) unsigned char raw[];
    float4 *ck = reinterpret_cast<float4 *>(raw);                       // [kBlocks - 1][warp][cs][2][lane]
    float *st = reinterpret_cast<float *>(ck + (kBlocks - 1) * kBwdWarps * S::REGION);   // [kTile][CH]: step, then ds
    float *xs = st + kTile * CH;                                        // x, then dx
    float *gs = xs + kTile * CH;                                        // g, then y
    float *bc = gs + kTile * CH;                                        // [kTile][2][NP]
    int *seq = reinterpret_cast<int *>(bc + kTile * 2 * NP);            // [kTile] the token's sequence
    unsigned *masks = reinterpret_cast<unsigned *>(seq + kTile);        // tokens that start / end one
    using Piece = T[8];
    Piece *ahead = reinterpret_cast<Piece *>(masks + 4);                // [4 * PASSES + BCV][thread]

    grid_dependency_wait();
    if (a.status && a.cu && blockIdx.x == 0) check_cu(a.cu, a.n_seqs, a.T, a.status);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nl = lane % NL, cl = lane / NL, n0 = nl * 8, perm = (cl & 1) * 2 | (cl >> 1 & 1);
    const int chan_block = blockIdx.x % a.chan_blocks, chan0 = chan_block * CH;
    const int seg = blockIdx.x / a.chan_blocks;
    const int b = seg / a.segs;
    const int tiles_per_seg = a.seg_tokens / kTile;
    const int first_tile = (seg - b * a.segs) * tiles_per_seg;
    const int last_tile = min(a.row_tiles, first_tile + tiles_per_seg) - 1;
    auto local = [&](int cs) { return warp * S::WC + cs * CL + cl; };
    auto channel = [&](int cs) { return chan0 + local(cs); };

    // a sequence without a token hands the gradient of its final state on
    if (a.dinit) {
        for (int n = a.cu ? seg : (a.T == 0 ? b : a.n_seqs); n < a.n_seqs; n += a.cu ? a.segs : a.n_seqs) {
            if (a.cu && __ldg(a.cu + n) < __ldg(a.cu + n + 1)) continue;
            for (int i = tid; i < CH * a.N; i += kBwdThreads) {
                const long long at = ((long long)n * a.D + chan0) * a.N + i;
                if (chan0 + i / a.N < a.D) a.dinit[at] = a.d_final ? a.d_final[at] : 0.f;
            }
        }
    }
    if (a.T == 0) return;

    F2 A2[CS][4], dA[CS][4], dh[CS][4];
    float skip[CS];
#pragma unroll
    for (int cs = 0; cs < CS; ++cs) {
        const bool live = channel(cs) < a.D;
        load_perm(a.A + (long long)channel(cs) * a.N, n0, perm, a.N, live, A2[cs]);
        load_padded(a.gloc + ((long long)seg * a.D + channel(cs)) * NP, n0, perm, live, dh[cs]);
        skip[cs] = a.skip && live ? a.skip[channel(cs)] : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            A2[cs][i] = mul2(A2[cs][i], both(kLog2e));
            dA[cs][i] = both(0.f);
        }
    }
    const int lv = tid % VPR, lrow = tid / VPR, lc = chan0 + lv * 8, lrest = a.D - lc;
    F2 bias[4], dbias[4], dskip[4];
    load_pairs(a.bias ? a.bias + lc : nullptr, 0, lrest, true, bias);
#pragma unroll
    for (int e = 0; e < 4; ++e) dbias[e] = dskip[e] = both(0.f);
    const T *px = static_cast<const T *>(a.x) + b * a.x_batch + lc, *pd = static_cast<const T *>(a.dt) + b * a.dt_batch + lc;
    const T *pz = static_cast<const T *>(a.z) + b * a.z_batch + lc, *pg = static_cast<const T *>(a.dy) + b * a.dy_batch + lc;

    // raw row pieces of a tile: i = array * PASSES + pass for x, dt, z, dy, then B and C
    auto source = [&](int i, int t0, int &n) -> const T * {
        if (i < 4 * PASSES) {
            const int q = i % PASSES * RPP + lrow, t = t0 + q;
            n = q < kTile && t < a.T ? lrest : 0;
            switch (i / PASSES) {
                case 0: return px + t * a.x_token;
                case 1: return pd + t * a.dt_token;
                case 2: n = a.z ? n : 0; return pz + t * a.z_token;
                default: return pg + t * a.dy_token;
            }
        }
        const int j = (i - 4 * PASSES) * kBwdThreads + tid, v = j % NL, c = j / NL % 2, q = j / (2 * NL), t = t0 + q;
        n = q < kTile && t < a.T ? a.N - v * 8 : 0;
        return v * 8 + (c ? static_cast<const T *>(a.Cm) + b * a.c_batch + t * a.c_token
                          : static_cast<const T *>(a.Bm) + b * a.b_batch + t * a.b_token);
    };
    auto stage = [&](int tile) {
        if constexpr (STAGED) {
#pragma unroll
            for (int i = 0; i < 4 * PASSES + S::BCV; ++i) {
                int n;
                const T *src = source(i, tile * kTile, n);
                copy8_async<T>(ahead[i * kBwdThreads + tid], src, n, i < 4 * PASSES ? a.vec : a.bc_vec);
            }
            copy_commit();
        }
    };
    auto fetch = [&](int i, int t0) -> Raw<T, 8> {
        if constexpr (STAGED) return load_raw<T, 8>(ahead[i * kBwdThreads + tid]);
        int n;
        const T *src = source(i, t0, n);
        return load8<T>(src, n, i < 4 * PASSES ? a.vec : a.bc_vec);
    };
    stage(last_tile);
    for (int tile = last_tile; tile >= first_tile; --tile) {
        const int t0 = tile * kTile, t1 = min(a.T, t0 + kTile);
        if (STAGED) copy_wait<0>();
        __syncthreads();   // the tile after this one has left shared memory
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int q = i * RPP + lrow, t = t0 + q;
            if (q >= kTile) continue;
            F2 x[4], d[4], z[4], g[4];
            unpack_pairs<T>(fetch(i, t0), x);
            unpack_pairs<T>(fetch(PASSES + i, t0), d);
            unpack_pairs<T>(fetch(2 * PASSES + i, t0), z);
            unpack_pairs<T>(fetch(3 * PASSES + i, t0), g);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                d[e] = add2(d[e], bias[e]);
                if (a.softplus) d[e] = softplus_pair(d[e]);
                if (t >= t1) d[e] = both(0.f);   // a token past the end: step 0
                if (a.z) g[e] = mul2(g[e], mul2(z[e], sigmoid_pair(z[e])));
                dskip[e] = fma2(g[e], x[e], dskip[e]);
            }
            const int at = q * CH + lv * 8;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                reinterpret_cast<ulonglong2 *>(st + at)[e] = make_ulonglong2(d[2 * e], d[2 * e + 1]);
                reinterpret_cast<ulonglong2 *>(xs + at)[e] = make_ulonglong2(x[2 * e], x[2 * e + 1]);
                reinterpret_cast<ulonglong2 *>(gs + at)[e] = make_ulonglong2(g[2 * e], g[2 * e + 1]);
            }
        }
#pragma unroll
        for (int i = 0; i < S::BCV; ++i) {
            const int j = i * kBwdThreads + tid;
            if (j >= kTile * 2 * NL) continue;
            F2 f[4];
            unpack_pairs<T>(fetch(4 * PASSES + i, t0), f);
            ulonglong2 *at = reinterpret_cast<ulonglong2 *>(bc + j / NL * NP + j % NL * 8);
            at[0] = make_ulonglong2(f[0], f[1]);
            at[1] = make_ulonglong2(f[2], f[3]);
        }
        if (tile > first_tile) stage(tile - 1);
        if (warp == 0) {
            const int t = min(t0 + lane, a.T - 1);
            const int n = a.cu ? find_seq(a.cu, a.n_seqs, t) : b;
            const bool starts = a.cu ? __ldg(a.cu + n) == t : t == 0, ends = a.cu ? __ldg(a.cu + n + 1) == t + 1 : t == a.T - 1;
            const unsigned ms = __ballot_sync(0xffffffffu, starts && t0 + lane < t1);
            const unsigned me = __ballot_sync(0xffffffffu, ends && t0 + lane < t1);
            if (lane < kTile) seq[lane] = n;
            if (lane == 0) masks[0] = ms, masks[1] = me;
        }
        __syncthreads();
        const unsigned ms = masks[0], me = masks[1];
        auto initial = [&](int j, int cs, F2 (&h)[4]) {
            load_perm(a.init ? a.init + ((long long)seq[j] * a.D + channel(cs)) * a.N : nullptr, n0, perm, a.N,
                      channel(cs) < a.D, h);
        };
        // row j's B (c = 0) or C (c = 1) in the lane's order of pairs
        auto load_bc = [&](int j, int c, F2 (&v)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const F2 *>(bc + (j * 2 + c) * NP + n0 + 2 * (i ^ perm));
        };
        // the tile's start state: the segment's, moved on to the tile
        auto start_state = [&](int cs, F2 (&h)[4]) {
            const bool ok = channel(cs) < a.D;
            if (tile == first_tile) {
                load_padded(a.hloc + ((long long)seg * a.D + channel(cs)) * NP, n0, perm, ok, h);
                return;
            }
            const long long at = ((long long)b * a.row_tiles + tile) * a.D + channel(cs);
            load_padded(a.htile + at * NP, n0, perm, ok, h);
            if (a.exact[(long long)b * a.row_tiles + tile]) return;
            const float sum = ok ? a.stile[at] : 0.f;
            F2 first[4];
            load_padded(a.hloc + ((long long)seg * a.D + channel(cs)) * NP, n0, perm, ok, first);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = fma2(exp2_pair(mul2(both(sum), A2[cs][i])), first[i], h[i]);
        };
        // forward: the state before every block of tokens but the first
        {
            F2 h[CS][4];
#pragma unroll
            for (int cs = 0; cs < CS; ++cs) start_state(cs, h[cs]);
#pragma unroll 1
            for (int kb = 0; kb < kBlocks - 1; ++kb) {
#pragma unroll
                for (int k = 0; k < kBlock; ++k) {
                    const int j = kb * kBlock + k;
                    F2 B[4];
                    load_bc(j, 0, B);
                    if (ms >> j & 1) {
#pragma unroll
                        for (int cs = 0; cs < CS; ++cs) initial(j, cs, h[cs]);
                    }
#pragma unroll
                    for (int cs = 0; cs < CS; ++cs) {
                        const float s = st[j * CH + local(cs)], sx = s * xs[j * CH + local(cs)];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            h[cs][i] = fma2(exp2_pair(mul2(both(s), A2[cs][i])), h[cs][i], mul2(both(sx), B[i]));
                    }
                }
#pragma unroll
                for (int cs = 0; cs < CS; ++cs) {
                    ulonglong2 *at = reinterpret_cast<ulonglong2 *>(ck + (kb * kBwdWarps + warp) * S::REGION + cs * 64 + lane);
                    at[0] = make_ulonglong2(h[cs][0], h[cs][1]);
                    at[32] = make_ulonglong2(h[cs][2], h[cs][3]);
                }
            }
        }
        // backward
        F2 acc[kBlock][2][4];   // dB, dC over this lane's channels
        auto walk = [&](auto plain, int kb) {   // plain: no sequence starts or ends in the block
            F2 B[kBlock][4], C[kBlock][4];
#pragma unroll
            for (int k = 0; k < kBlock; ++k) load_bc(kb * kBlock + k, 0, B[k]), load_bc(kb * kBlock + k, 1, C[k]);
#pragma unroll
            for (int cs = 0; cs < CS; ++cs) {
                const int chl = local(cs), ch = channel(cs);
                F2 h[4], e[kBlock][4], p[kBlock][4];
                float s[kBlock], x[kBlock], g[kBlock], y[kBlock], u[kBlock], w[kBlock];
                if (kb == 0) {
                    start_state(cs, h);
                } else {
                    const ulonglong2 *at = reinterpret_cast<const ulonglong2 *>(ck + ((kb - 1) * kBwdWarps + warp) * S::REGION + cs * 64 + lane);
                    const ulonglong2 v0 = at[0], v1 = at[32];
                    h[0] = v0.x, h[1] = v0.y, h[2] = v1.x, h[3] = v1.y;
                }
#pragma unroll
                for (int k = 0; k < kBlock; ++k) {
                    const int j = kb * kBlock + k;
                    s[k] = st[j * CH + chl], x[k] = xs[j * CH + chl], g[k] = gs[j * CH + chl];
                    const F2 ss = both(s[k]), sx = both(s[k] * x[k]), gg = both(g[k]);
                    if (!plain && (ms >> j & 1)) initial(j, cs, h);
                    F2 yy = both(0.f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        e[k][i] = exp2_pair(mul2(ss, A2[cs][i]));
                        p[k][i] = mul2(e[k][i], h[i]);
                        h[i] = fma2(sx, B[k][i], p[k][i]);
                        yy = i ? fma2(C[k][i], h[i], yy) : mul2(C[k][i], h[i]);
                        acc[k][1][i] = cs ? fma2(gg, h[i], acc[k][1][i]) : mul2(gg, h[i]);
                    }
                    y[k] = lo(yy) + hi(yy);
                }
#pragma unroll
                for (int k = kBlock - 1; k >= 0; --k) {
                    const int j = kb * kBlock + k;
                    const F2 gg = both(g[k]), ss = both(s[k]), sx = both(s[k] * x[k]);
                    if (!plain && (me >> j & 1) && a.d_final) {
                        F2 f[4];
                        load_perm(a.d_final + ((long long)seq[j] * a.D + ch) * a.N, n0, perm, a.N, ch < a.D, f);
#pragma unroll
                        for (int i = 0; i < 4; ++i) dh[cs][i] = add2(dh[cs][i], f[i]);
                    }
                    F2 uu = both(0.f), ww = both(0.f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        dh[cs][i] = fma2(gg, C[k][i], dh[cs][i]);
                        acc[k][0][i] = cs ? fma2(sx, dh[cs][i], acc[k][0][i]) : mul2(sx, dh[cs][i]);
                        uu = i ? fma2(dh[cs][i], B[k][i], uu) : mul2(dh[cs][i], B[k][i]);
                        const F2 q = mul2(dh[cs][i], p[k][i]);
                        dA[cs][i] = fma2(ss, q, dA[cs][i]);
                        ww = i ? fma2(q, A2[cs][i], ww) : mul2(q, A2[cs][i]);
                        dh[cs][i] = mul2(dh[cs][i], e[k][i]);
                    }
                    u[k] = lo(uu) + hi(uu);
                    w[k] = lo(ww) + hi(ww);
                    if (!plain && (ms >> j & 1)) {   // the gradient of the sequence's initial state
                        if (a.dinit && ch < a.D)
                            store_perm(a.dinit + ((long long)seq[j] * a.D + ch) * a.N, n0, perm, a.N, dh[cs]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) dh[cs][i] = both(0.f);
                    }
                }
                // over the lanes of the channel; each is left with its token (or both)
                int k0 = 0, k1 = 0, k2 = 0;
                reduce_scatter<kBlock, NL / 2, 1>(u, lane, k0);
                reduce_scatter<kBlock, NL / 2, 1>(w, lane, k1);
                if (a.z) reduce_scatter<kBlock, NL / 2, 1>(y, lane, k2);
                __syncwarp();
                constexpr int KEPT = NL == 1 ? kBlock : 1;
#pragma unroll
                for (int i = 0; i < KEPT; ++i) {
                    const float sk = k0 + i ? s[1] : s[0], xk = k0 + i ? x[1] : x[0], gk = k0 + i ? g[1] : g[0];
                    const int at = (kb * kBlock + k0 + i) * CH + chl;
                    st[at] = fmaf(u[i], xk, w[i] * kLn2);
                    xs[at] = fmaf(u[i], sk, skip[cs] * gk);
                    gs[at] = fmaf(skip[cs], xk, y[i]);
                }
            }
        };
#pragma unroll 1
        for (int kb = kBlocks - 1; kb >= 0; --kb) {
            if (((ms | me) >> kb * kBlock & ((1u << kBlock) - 1)) == 0) walk(std::true_type(), kb);
            else walk(std::false_type(), kb);
            // dB, dC over the lanes of the warp's channels: every lane keeps its slots 0
            // and 1, then 0, of four
            float v[kBlock * 2 * 2];
#pragma unroll
            for (int k = 0; k < kBlock; ++k)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const F2 a0 = add2(acc[k][c][0], shfl_pair(acc[k][c][2], NL)), a1 = add2(acc[k][c][1], shfl_pair(acc[k][c][3], NL));
                    const F2 a2 = add2(a0, shfl_pair(a1, 2 * NL));
                    v[(k * 2 + c) * 2] = lo(a2), v[(k * 2 + c) * 2 + 1] = hi(a2);
                }
            int base = 0;
            reduce_scatter<kBlock * 4, 16, 4 * NL>(v, lane, base);
            __syncwarp();
            float *res = reinterpret_cast<float *>(ck + ((kb ? kb - 1 : 0) * kBwdWarps + warp) * S::REGION) + (kb ? 0 : 4 * NP);
#pragma unroll
            for (int i = 0; i < VL; ++i) res[((base + i) / 2) * NP + n0 + 2 * perm + (base + i) % 2] = v[i];
        }
        __syncthreads();
        // dB, dC of the tile over the block's channels
        const long long tokens = (long long)a.B * a.T;
        for (int i = tid; i < (t1 - t0) * 2 * NP; i += kBwdThreads) {
            const int n = i % NP, c = i / NP % 2, j = i / (2 * NP), kb = j / kBlock;
            float v = 0.f;
#pragma unroll
            for (int wp = 0; wp < kBwdWarps; ++wp)
                v += (reinterpret_cast<const float *>(ck + ((kb ? kb - 1 : 0) * kBwdWarps + wp) * S::REGION) +
                      (kb ? 0 : 4 * NP))[(j % kBlock * 2 + c) * NP + n];
            a.part_bc[((chan_block * tokens + (long long)b * a.T + t0 + j) * 2 + c) * NP + n] = v;
        }
        // dx, ddt, dz
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int q = i * RPP + lrow, t = t0 + q;
            if (q >= kTile || t >= t1 || lrest <= 0) continue;
            float o[8];
            const long long at = ((long long)b * a.T + t) * a.D + lc;
            const int in = q * CH + lv * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = xs[in + e];
            store8<T>(static_cast<T *>(a.out) + at, o, lrest, a.vec);
            F2 d[4], z[4], g[4];
            unpack_pairs<T>(load8<T>(pd + t * a.dt_token, lrest, a.vec), d);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                F2 v = *reinterpret_cast<const F2 *>(st + in + 2 * e);
                if (a.softplus) v = mul2(v, sigmoid_pair(add2(d[e], bias[e])));
                dbias[e] = add2(dbias[e], v);
                o[2 * e] = lo(v), o[2 * e + 1] = hi(v);
            }
            store8<T>(static_cast<T *>(a.ddt) + at, o, lrest, a.vec);
            if (a.z) {
                unpack_pairs<T>(load8<T>(pz + t * a.z_token, lrest, a.vec), z);
                unpack_pairs<T>(load8<T>(pg + t * a.dy_token, lrest, a.vec), g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const F2 sg = sigmoid_pair(z[e]), y = *reinterpret_cast<const F2 *>(gs + in + 2 * e);
                    const F2 v = mul2(mul2(g[e], y), mul2(sg, fma2(z[e], fma2(sg, both(-1.f), both(1.f)), both(1.f))));
                    o[2 * e] = lo(v), o[2 * e + 1] = hi(v);
                }
                store8<T>(static_cast<T *>(a.dz) + at, o, lrest, a.vec);
            }
        }
    }
    // the segment's sums over tokens
#pragma unroll
    for (int cs = 0; cs < CS; ++cs)
        if (channel(cs) < a.D) store_perm(a.part_a + ((long long)seg * a.D + channel(cs)) * NP, n0, perm, NP, dA[cs]);
    __syncthreads();
    float *sum = reinterpret_cast<float *>(raw);   // [2][RPP][CH]
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        *reinterpret_cast<F2 *>(sum + lrow * CH + lv * 8 + 2 * e) = dskip[e];
        *reinterpret_cast<F2 *>(sum + (RPP + lrow) * CH + lv * 8 + 2 * e) = dbias[e];
    }
    __syncthreads();
    for (int i = tid; i < 2 * CH; i += kBwdThreads) {
        const int c = i % CH, k = i / CH;
        if (chan0 + c >= a.D) continue;
        float v = 0.f;
        for (int q = 0; q < RPP; ++q) v += sum[(k * RPP + q) * CH + c];
        a.part_v[((long long)seg * 2 + k) * a.D + chan0 + c] = v;
    }
}

// The sums over blocks: the first `bc_blocks` blocks add dB and dC, in the
// activations' type, over the blocks of channels; the others dA, dD and ddt_bias
// over the segments, eight groups of segments per 32 values, then the groups in
// order.
template <typename T>
__global__ void __launch_bounds__(256) scan_bwd_sum_kernel(ScanArgs a, int bc_blocks, int chan_blocks, int segs, int NP,
                                                           T *dB, T *dC, float *dA, float *dskip, float *dbias) {
    __shared__ float sum[8][32];
    grid_dependency_wait();
    if ((int)blockIdx.x < bc_blocks) {
        const long long i = (long long)blockIdx.x * 256 + threadIdx.x, size = (long long)a.B * a.T * 2 * NP;
        const int n = (int)(i % NP), c = (int)(i / NP % 2);
        if (i >= size || n >= a.N) return;
        float v = 0.f;
#pragma unroll 4
        for (int k = 0; k < chan_blocks; ++k) v += a.part_bc[k * size + i];
        (c ? dC : dB)[i / (2 * NP) * a.N + n] = from_f32<T>(v);
        return;
    }
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const long long i = (long long)(blockIdx.x - bc_blocks) * 32 + lane, na = (long long)a.D * NP, total = na + 2 * a.D;
    float v = 0.f;
    if (i < total) {
        const float *p = i < na ? a.part_a + i : a.part_v + (i - na);
        const long long step = i < na ? na : 2 * a.D;
#pragma unroll 4
        for (int s = grp; s < segs; s += 8) v += p[s * step];
    }
    sum[grp][lane] = v;
    __syncthreads();
    if (grp != 0 || i >= total) return;
    v = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v += sum[k][lane];
    if (i < na) {
        if (i % NP < a.N) dA[i / NP * a.N + i % NP] = v;
    } else if (i - na < a.D) {
        if (dskip) dskip[i - na] = v;
    } else if (dbias) {
        dbias[i - na - a.D] = v;
    }
}

template <typename T, int NL>
cudaError_t launch_main(ScanArgs a, cudaStream_t s) {
    using S = BwdShape<NL>;
    constexpr size_t smem = S::smem + S::template staged<T>;
    const cudaError_t attr = cudaFuncSetAttribute(scan_bwd_kernel<T, NL>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (attr != cudaSuccess) return attr;
    return launch_dependent(scan_bwd_kernel<T, NL>, dim3((unsigned)((long long)a.chan_blocks * a.B * a.segs)),
                            dim3(kBwdThreads), smem, s, a);
}

template <typename T>
cudaError_t launch_bwd_typed(const ScanArgs &a, T *dB, T *dC, float *dA, float *dskip, float *dbias, cudaStream_t s) {
    const int parts = scan_parts(a.N), NP = 8 * parts;
    const long long tokens = (long long)a.B * a.T;
    cudaError_t e = cudaSuccess;
    if (tokens > 0) {
        e = launch_scan_maps(a, sizeof(T) == 2 ? GDN_BF16 : GDN_F32, s);
        if (e == cudaSuccess) e = launch_scan_combine(a, a.segs, true, s);
        if (e != cudaSuccess) return e;
    }
    if (a.B > 0) {   // (without tokens: the gradients of the states)
        switch (parts) {
            case 1: e = launch_main<T, 1>(a, s); break;
            case 2: e = launch_main<T, 2>(a, s); break;
            case 4: e = launch_main<T, 4>(a, s); break;
            default: e = launch_main<T, 8>(a, s);
        }
    }
    if (e != cudaSuccess) return e;
    const int bc_blocks = (int)((tokens * 2 * NP + 255) / 256);
    return launch_dependent(scan_bwd_sum_kernel<T>, dim3((unsigned)(bc_blocks + ((long long)a.D * (NP + 2) + 31) / 32)), dim3(256), 0, s,
                            a, bc_blocks, a.chan_blocks, tokens > 0 ? a.B * a.segs : 0, NP, dB, dC, dA, dskip, dbias);
}

}  // namespace

int scan_bwd_channels(int N) {
    switch (scan_parts(N)) {
        case 1: return BwdShape<1>::CH;
        case 2: return BwdShape<2>::CH;
        case 4: return BwdShape<4>::CH;
        default: return BwdShape<8>::CH;
    }
}

cudaError_t launch_scan_bwd(const ScanArgs &a, int dtype, void *dB, void *dC, float *dA, float *dskip, float *dbias,
                            cudaStream_t s) {
    return dtype == GDN_BF16 ? launch_bwd_typed<__nv_bfloat16>(a, static_cast<__nv_bfloat16 *>(dB),
                                                               static_cast<__nv_bfloat16 *>(dC), dA, dskip, dbias, s)
                             : launch_bwd_typed<float>(a, static_cast<float *>(dB), static_cast<float *>(dC), dA, dskip,
                                                       dbias, s);
}

}  // namespace gdn
