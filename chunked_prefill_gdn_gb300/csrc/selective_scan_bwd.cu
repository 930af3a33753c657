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
// Both recurrences run over tiles of 32 tokens in parallel.  A first kernel
// gives every tile's two maps from one pass over its exponentials: the end
// state from a zero start, and the gradient at its start from a zero gradient
// at its end, which needs no reversed pass: with the running product p_t of
// the a's it is sum_t p_t C_t g_t.  scan_combine_kernel turns the maps into
// every tile's exact start state and end gradient.  The main kernel walks a
// tile forward, keeping the state at every fourth token in shared memory, then
// backward in blocks of four tokens whose states it recomputes in registers.
//
// The sums over n (for the gradients per channel) and over channels (for dB
// and dC) decide the thread layout: a thread holds four n of CS channels, so
// that both sums are first taken in registers, and each remaining exchange
// between lanes halves the values it still carries (a reduce-scatter); a layout
// with all n or all channels in one lane would pay twice the shuffles.
// Sums over warps, blocks and tokens are added in a fixed order: no atomics,
// the same inputs give the same bits.
#include <algorithm>

#include "scan_pairs.cuh"

namespace gdn {

namespace {

constexpr int kMapThreads = 64;

template <typename T, int LP>
__global__ void __launch_bounds__(kMapThreads) scan_tile_maps_kernel(ScanArgs a) {
    constexpr int CH = kMapThreads / LP;
    constexpr int NP = 8 * LP;
    constexpr int VPR = CH / 8;
    constexpr int RPP = kMapThreads / VPR;
    constexpr int PASSES = RPP >= kTile ? 1 : kTile / RPP;
    __shared__ __align__(16) float4 sd[kTile][CH];   // step, step * x, dy through the gate, -
    __shared__ __align__(16) float bc[kTile][2][NP];
    const int tid = threadIdx.x;
    const int chan0 = (blockIdx.x % a.chan_blocks) * CH;
    const int tile = blockIdx.x / a.chan_blocks;     // over all rows
    Span r;
    r.b = tile / a.row_tiles;
    r.t0 = (tile - r.b * a.row_tiles) * kTile;
    r.t1 = min(a.T, r.t0 + kTile);

    const int lv = tid % VPR, lrow = tid / VPR, lc = chan0 + lv * 8, lrest = a.D - lc;
    const long long row = r.b;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int q = i * RPP + lrow, t = r.t0 + q;
        const int n = q < kTile && t < r.t1 ? lrest : 0;
        float x[8], d[8], z[8], g[8];
        unpack<T, 8>(load8<T>(static_cast<const T *>(a.x) + row * a.x_batch + t * a.x_token + lc, n, a.vec), x);
        unpack<T, 8>(load8<T>(static_cast<const T *>(a.dt) + row * a.dt_batch + t * a.dt_token + lc, n, a.vec), d);
        unpack<T, 8>(load8<T>(static_cast<const T *>(a.z) + row * a.z_batch + t * a.z_token + lc, a.z ? n : 0, a.vec), z);
        unpack<T, 8>(load8<T>(static_cast<const T *>(a.dy) + row * a.dy_batch + t * a.dy_token + lc, n, a.vec), g);
        if (q < kTile) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float pre = d[e] + (a.bias && e < lrest ? a.bias[lc + e] : 0.f);
                const float s = a.softplus ? softplus_f32(pre) : pre;
                const float gate = a.z ? z[e] * sigmoid_f32(z[e]) : 1.f;
                sd[q][lv * 8 + e] = make_float4(s, s * x[e], g[e] * gate, 0.f);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < LP; ++i) {
        const int j = i * kMapThreads + tid, v = j % LP, c = j / LP % 2, q = j / (2 * LP), t = r.t0 + q;
        const T *src = c ? static_cast<const T *>(a.Cm) + row * a.c_batch + t * a.c_token
                         : static_cast<const T *>(a.Bm) + row * a.b_batch + t * a.b_token;
        float f[8];
        unpack<T, 8>(load8<T>(src + v * 8, t < r.t1 ? a.N - v * 8 : 0, a.bc_vec), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) bc[q][c][v * 8 + e] = f[e];
    }
    const int part = tid % LP, n0 = part * 8, chl = tid / LP, ch = chan0 + chl;
    const bool live = ch < a.D;
    F2 A2[4], h[4], p[4], G[4];
    load_pairs(a.A + (long long)ch * a.N, n0, a.N, live, A2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        A2[i] = mul2(A2[i], pair(kLog2e, kLog2e));
        h[i] = G[i] = pair(0.f, 0.f);
        p[i] = pair(1.f, 1.f);
    }
    span_find(a, r);
    const bool starts = r.begin == r.t0;
    bool inside = false;
    auto initial = [&](int n) {
        load_pairs(a.init ? a.init + ((long long)n * a.D + ch) * a.N : nullptr, n0, a.N, live, h);
    };
    if (starts) initial(r.n);
    float sum = 0.f;
    __syncthreads();
    for (int q = r.t0; q < r.t1;) {
        const int run_end = min(r.t1, r.end);
        if (!inside) {
#pragma unroll 4
            for (int k = q - r.t0; k < run_end - r.t0; ++k) {
                const float4 s = sd[k][chl];
                const F2 ss = pair(s.x, s.x), sx = pair(s.y, s.y), gg = pair(s.z, s.z);
                const F2 *Bk = reinterpret_cast<const F2 *>(&bc[k][0][n0]), *Ck = reinterpret_cast<const F2 *>(&bc[k][1][n0]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const F2 e = exp2_pair(mul2(ss, A2[i]));
                    h[i] = fma2(e, h[i], mul2(sx, Bk[i]));
                    p[i] = mul2(p[i], e);
                    G[i] = fma2(p[i], mul2(gg, Ck[i]), G[i]);
                }
                sum += s.x;
            }
        } else {
#pragma unroll 4
            for (int k = q - r.t0; k < run_end - r.t0; ++k) {
                const float4 s = sd[k][chl];
                const F2 ss = pair(s.x, s.x), sx = pair(s.y, s.y);
                const F2 *Bk = reinterpret_cast<const F2 *>(&bc[k][0][n0]);
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = fma2(exp2_pair(mul2(ss, A2[i])), h[i], mul2(sx, Bk[i]));
            }
        }
        q = run_end;
        if (q == r.end) {
            if (!inside && a.d_final) {
                F2 f[4];
                load_pairs(a.d_final + ((long long)r.n * a.D + ch) * a.N, n0, a.N, live, f);
#pragma unroll
                for (int i = 0; i < 4; ++i) G[i] = fma2(p[i], f[i], G[i]);
            }
            if (q < r.t1) {
                span_next(a, r, q);
                initial(r.n);
                inside = true;
            }
        }
    }
    if (live) {
        const long long at = ((long long)tile * a.D + ch) * NP;
        store_pairs(a.hloc + at, n0, NP, h);
        store_pairs(a.gloc + at, n0, NP, G);
        if (part == 0) a.sums[(long long)tile * a.D + ch] = sum;
    }
    if (chan0 == 0 && tid == 0) a.flags[tile] = (starts ? 1 : 0) | (inside ? 2 : 0);
}

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
constexpr int kBlock = 4;                      // tokens per block of the backward walk
constexpr int kBlocks = kTile / kBlock;

// NL lanes share a channel (four n each), CS channels per lane.
template <int NL>
struct BwdShape {
    static constexpr int CS = NL == 2 ? 2 : 4;
    static constexpr int CL = 32 / NL;                   // lanes over channels
    static constexpr int WC = CL * CS;                   // channels of a warp
    static constexpr int CH = WC * kBwdWarps;            // of the block
    static constexpr int NP = 4 * NL;
    static constexpr int VL = 4 * 8 / CL > 0 ? 4 * 8 / CL : 1;   // dB, dC sums left per lane and block of tokens
    // a block's dB and dC sums go where its states were; block 0 has none of its own
    static constexpr int REGIONS = 32 * NL * 2 <= CS * 32 * 4 ? kBlocks - 1 : kBlocks;
    static constexpr int REGION = kBwdWarps * CS * 32;   // float4
    static constexpr size_t smem = REGIONS * REGION * 16 + 3 * kTile * CH * 4 + kTile * 2 * NP * 4 + kTile * 4 + 16;
};

template <typename T, int NL>
__global__ void __launch_bounds__(kBwdThreads, 2) scan_bwd_kernel(ScanArgs a) {
    using S = BwdShape<NL>;
    constexpr int CS = S::CS, CL = S::CL, CH = S::CH, NP = S::NP, VL = S::VL;
    constexpr int VPR = CH / 8, RPP = kBwdThreads / VPR, PASSES = kTile / RPP;
    static_assert(RPP <= kTile && RPP * PASSES == kTile, "rows of the loading threads");
    extern __shared__ __align__(16) unsigned char raw[];
    float4 *ck = reinterpret_cast<float4 *>(raw);                       // [REGIONS][warp][cs][lane]
    float *st = reinterpret_cast<float *>(ck + S::REGIONS * S::REGION); // [kTile][CH]: step, then ds
    float *xs = st + kTile * CH;                                        // x, then dx
    float *gs = xs + kTile * CH;                                        // g, then y
    float *bc = gs + kTile * CH;                                        // [kTile][2][NP]
    int *seq = reinterpret_cast<int *>(bc + kTile * 2 * NP);            // [kTile] the token's sequence
    unsigned *masks = reinterpret_cast<unsigned *>(seq + kTile);        // tokens that start / end one

    if (a.status && a.cu && blockIdx.x == 0) check_cu(a.cu, a.n_seqs, a.T, a.status);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nl = lane % NL, cl = lane / NL, n0 = nl * 4;
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

    F2 A2[CS][2], dA[CS][2], dh[CS][2];
#pragma unroll
    for (int cs = 0; cs < CS; ++cs) {
        const bool live = channel(cs) < a.D;
        load_pairs(a.A + (long long)channel(cs) * a.N, n0, a.N, live, A2[cs]);
        load_pairs(a.gloc + (((long long)b * a.row_tiles + last_tile) * a.D + channel(cs)) * NP, n0, NP, live, dh[cs]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            A2[cs][i] = mul2(A2[cs][i], pair(kLog2e, kLog2e));
            dA[cs][i] = pair(0.f, 0.f);
        }
    }
    const int lv = tid % VPR, lrow = tid / VPR, lc = chan0 + lv * 8, lrest = a.D - lc;
    float bias[8], dbias[8], dskip[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        bias[e] = a.bias && e < lrest ? a.bias[lc + e] : 0.f;
        dbias[e] = dskip[e] = 0.f;
    }
    const T *px = static_cast<const T *>(a.x) + b * a.x_batch + lc, *pd = static_cast<const T *>(a.dt) + b * a.dt_batch + lc;
    const T *pz = static_cast<const T *>(a.z) + b * a.z_batch + lc, *pg = static_cast<const T *>(a.dy) + b * a.dy_batch + lc;

    for (int tile = last_tile; tile >= first_tile; --tile) {
        const int t0 = tile * kTile, t1 = min(a.T, t0 + kTile);
        __syncthreads();   // the tile after this one has left shared memory
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int q = i * RPP + lrow, t = t0 + q;
            const bool in = t < t1;
            const int n = in ? lrest : 0;
            float x[8], d[8], z[8], g[8];
            unpack<T, 8>(load8<T>(px + t * a.x_token, n, a.vec), x);
            unpack<T, 8>(load8<T>(pd + t * a.dt_token, n, a.vec), d);
            unpack<T, 8>(load8<T>(pz + t * a.z_token, a.z ? n : 0, a.vec), z);
            unpack<T, 8>(load8<T>(pg + t * a.dy_token, n, a.vec), g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float pre = d[e] + bias[e];
                d[e] = in ? (a.softplus ? softplus_f32(pre) : pre) : 0.f;   // a token past the end: step 0
                if (a.z) g[e] *= z[e] * sigmoid_f32(z[e]);
                dskip[e] = fmaf(g[e], x[e], dskip[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const int at = q * CH + lv * 8 + e;
                *reinterpret_cast<float4 *>(st + at) = make_float4(d[e], d[e + 1], d[e + 2], d[e + 3]);
                *reinterpret_cast<float4 *>(xs + at) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                *reinterpret_cast<float4 *>(gs + at) = make_float4(g[e], g[e + 1], g[e + 2], g[e + 3]);
            }
        }
        for (int j = tid; j < kTile * 2 * (NP / 8); j += kBwdThreads) {
            const int v = j % (NP / 8), c = j / (NP / 8) % 2, q = j / (2 * (NP / 8)), t = t0 + q;
            const T *src = c ? static_cast<const T *>(a.Cm) + b * a.c_batch + t * a.c_token
                             : static_cast<const T *>(a.Bm) + b * a.b_batch + t * a.b_token;
            float f[8];
            unpack<T, 8>(load8<T>(src + v * 8, t < t1 ? a.N - v * 8 : 0, a.bc_vec), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) bc[(q * 2 + c) * NP + v * 8 + e] = f[e];
        }
        if (warp == 0) {
            const int t = min(t0 + lane, a.T - 1);
            const int n = a.cu ? find_seq(a.cu, a.n_seqs, t) : b;
            const bool starts = a.cu ? __ldg(a.cu + n) == t : t == 0, ends = a.cu ? __ldg(a.cu + n + 1) == t + 1 : t == a.T - 1;
            const unsigned ms = __ballot_sync(0xffffffffu, starts && t0 + lane < t1);
            const unsigned me = __ballot_sync(0xffffffffu, ends && t0 + lane < t1);
            seq[lane] = n;
            if (lane == 0) masks[0] = ms, masks[1] = me;
        }
        __syncthreads();
        const unsigned ms = masks[0], me = masks[1];
        auto initial = [&](int j, int cs, F2 (&h)[2]) {
            load_pairs(a.init ? a.init + ((long long)seq[j] * a.D + channel(cs)) * a.N : nullptr, n0, a.N,
                       channel(cs) < a.D, h);
        };
        const long long map = ((long long)b * a.row_tiles + tile) * a.D;
        // forward: the state before every block of tokens but the first
#pragma unroll
        for (int cs = 0; cs < CS; ++cs) {
            F2 h[2];
            load_pairs(a.hloc + (map + channel(cs)) * NP, n0, NP, channel(cs) < a.D, h);
            for (int kb = 0; kb < kBlocks - 1; ++kb) {
#pragma unroll
                for (int k = 0; k < kBlock; ++k) {
                    const int j = kb * kBlock + k;
                    const float s = st[j * CH + local(cs)], sx = s * xs[j * CH + local(cs)];
                    const ulonglong2 B = *reinterpret_cast<const ulonglong2 *>(bc + j * 2 * NP + n0);
                    if (ms >> j & 1) initial(j, cs, h);
                    h[0] = fma2(exp2_pair(mul2(pair(s, s), A2[cs][0])), h[0], mul2(pair(sx, sx), B.x));
                    h[1] = fma2(exp2_pair(mul2(pair(s, s), A2[cs][1])), h[1], mul2(pair(sx, sx), B.y));
                }
                ck[((kb * kBwdWarps + warp) * CS + cs) * 32 + lane] = make_float4(lo(h[0]), hi(h[0]), lo(h[1]), hi(h[1]));
            }
        }
        // backward
        for (int kb = kBlocks - 1; kb >= 0; --kb) {
            float acc[kBlock * 8];   // [token][dB, dC][four n], over this lane's channels
#pragma unroll
            for (int i = 0; i < kBlock * 8; ++i) acc[i] = 0.f;
            ulonglong2 B[kBlock], C[kBlock];
#pragma unroll
            for (int k = 0; k < kBlock; ++k) {
                B[k] = *reinterpret_cast<const ulonglong2 *>(bc + (kb * kBlock + k) * 2 * NP + n0);
                C[k] = *reinterpret_cast<const ulonglong2 *>(bc + (kb * kBlock + k) * 2 * NP + NP + n0);
            }
#pragma unroll
            for (int cs = 0; cs < CS; ++cs) {
                const int chl = local(cs), ch = channel(cs);
                F2 h[2], e[kBlock][2], p[kBlock][2];
                float s[kBlock], x[kBlock], g[kBlock], y[kBlock], u[kBlock], w[kBlock];
                if (kb == 0) {
                    load_pairs(a.hloc + (map + ch) * NP, n0, NP, ch < a.D, h);
                } else {
                    const float4 v = ck[(((kb - 1) * kBwdWarps + warp) * CS + cs) * 32 + lane];
                    h[0] = pair(v.x, v.y), h[1] = pair(v.z, v.w);
                }
#pragma unroll
                for (int k = 0; k < kBlock; ++k) {
                    const int j = kb * kBlock + k;
                    s[k] = st[j * CH + chl], x[k] = xs[j * CH + chl], g[k] = gs[j * CH + chl];
                    const float sx = s[k] * x[k];
                    if (ms >> j & 1) initial(j, cs, h);
                    e[k][0] = exp2_pair(mul2(pair(s[k], s[k]), A2[cs][0]));
                    e[k][1] = exp2_pair(mul2(pair(s[k], s[k]), A2[cs][1]));
                    p[k][0] = mul2(e[k][0], h[0]);
                    p[k][1] = mul2(e[k][1], h[1]);
                    h[0] = fma2(pair(sx, sx), B[k].x, p[k][0]);
                    h[1] = fma2(pair(sx, sx), B[k].y, p[k][1]);
                    const F2 yy = fma2(C[k].y, h[1], mul2(C[k].x, h[0]));
                    y[k] = lo(yy) + hi(yy);
                    // dC, while the state is at hand
                    const F2 gg = pair(g[k], g[k]);
                    F2 c0 = pair(acc[k * 8 + 4], acc[k * 8 + 5]), c1 = pair(acc[k * 8 + 6], acc[k * 8 + 7]);
                    c0 = fma2(gg, h[0], c0), c1 = fma2(gg, h[1], c1);
                    acc[k * 8 + 4] = lo(c0), acc[k * 8 + 5] = hi(c0), acc[k * 8 + 6] = lo(c1), acc[k * 8 + 7] = hi(c1);
                }
#pragma unroll
                for (int k = kBlock - 1; k >= 0; --k) {
                    const int j = kb * kBlock + k;
                    const float sx = s[k] * x[k];
                    const F2 gg = pair(g[k], g[k]), ss = pair(s[k], s[k]), sxx = pair(sx, sx);
                    if (me >> j & 1 && a.d_final) {
                        F2 f[2];
                        load_pairs(a.d_final + ((long long)seq[j] * a.D + ch) * a.N, n0, a.N, ch < a.D, f);
                        dh[cs][0] = add2(dh[cs][0], f[0]), dh[cs][1] = add2(dh[cs][1], f[1]);
                    }
                    dh[cs][0] = fma2(gg, C[k].x, dh[cs][0]);
                    dh[cs][1] = fma2(gg, C[k].y, dh[cs][1]);
                    F2 b0 = pair(acc[k * 8], acc[k * 8 + 1]), b1 = pair(acc[k * 8 + 2], acc[k * 8 + 3]);
                    b0 = fma2(sxx, dh[cs][0], b0), b1 = fma2(sxx, dh[cs][1], b1);
                    acc[k * 8] = lo(b0), acc[k * 8 + 1] = hi(b0), acc[k * 8 + 2] = lo(b1), acc[k * 8 + 3] = hi(b1);
                    const F2 uu = fma2(dh[cs][1], B[k].y, mul2(dh[cs][0], B[k].x));
                    const F2 q0 = mul2(dh[cs][0], p[k][0]), q1 = mul2(dh[cs][1], p[k][1]);
                    dA[cs][0] = fma2(ss, q0, dA[cs][0]);
                    dA[cs][1] = fma2(ss, q1, dA[cs][1]);
                    const F2 ww = fma2(q1, A2[cs][1], mul2(q0, A2[cs][0]));
                    u[k] = lo(uu) + hi(uu);
                    w[k] = lo(ww) + hi(ww);
                    dh[cs][0] = mul2(dh[cs][0], e[k][0]);
                    dh[cs][1] = mul2(dh[cs][1], e[k][1]);
                    if (ms >> j & 1) {   // the gradient of the sequence's initial state
                        if (a.dinit && ch < a.D)
                            store_pairs(a.dinit + ((long long)seq[j] * a.D + ch) * a.N, n0, a.N, dh[cs]);
                        dh[cs][0] = dh[cs][1] = pair(0.f, 0.f);
                    }
                }
                // over the lanes of the channel; each is left with its token or tokens
                int k0 = 0, k1 = 0, k2 = 0;
                reduce_scatter<kBlock, NL / 2, 1>(u, lane, k0);
                reduce_scatter<kBlock, NL / 2, 1>(w, lane, k1);
                if (a.z) reduce_scatter<kBlock, NL / 2, 1>(y, lane, k2);
                __syncwarp();
                constexpr int KEPT = NL >= kBlock ? 1 : kBlock / NL;
                const float skip = a.skip && ch < a.D ? a.skip[ch] : 0.f;
#pragma unroll
                for (int i = 0; i < KEPT; ++i) {
                    float sk = 0.f, xk = 0.f, gk = 0.f;
#pragma unroll
                    for (int k = 0; k < kBlock; ++k)
                        if (k == k0 + i) sk = s[k], xk = x[k], gk = g[k];
                    const int at = (kb * kBlock + k0 + i) * CH + chl;
                    st[at] = fmaf(u[i], xk, w[i] * kLn2);
                    xs[at] = fmaf(u[i], sk, skip * gk);
                    gs[at] = fmaf(skip, xk, y[i]);
                }
            }
            // dB, dC over the lanes of the warp's channels
            int base = 0;
            reduce_scatter<kBlock * 8, 16, NL>(acc, lane, base);
            __syncwarp();
            constexpr int OWN = S::REGIONS == kBlocks ? kBlocks - 1 : 0;   // where block 0's go
            float *res = reinterpret_cast<float *>(ck + ((kb ? kb - 1 : OWN) * kBwdWarps + warp) * CS * 32) +
                         (kb == 0 && S::REGIONS != kBlocks ? 32 * NL : 0);
#pragma unroll
            for (int i = 0; i < VL; ++i) res[nl * 32 + base + i] = acc[i];
        }
        __syncthreads();
        // dB, dC of the tile over the block's channels
        const long long tokens = (long long)a.B * a.T;
        for (int i = tid; i < (t1 - t0) * 2 * NP; i += kBwdThreads) {
            const int n = i % NP, c = i / NP % 2, j = i / (2 * NP), kb = j / kBlock;
            const int at = (n / 4) * 32 + (j % kBlock) * 8 + c * 4 + n % 4;
            constexpr int OWN = S::REGIONS == kBlocks ? kBlocks - 1 : 0;
            float v = 0.f;
#pragma unroll
            for (int wp = 0; wp < kBwdWarps; ++wp)
                v += (reinterpret_cast<const float *>(ck + ((kb ? kb - 1 : OWN) * kBwdWarps + wp) * CS * 32) +
                      (kb == 0 && S::REGIONS != kBlocks ? 32 * NL : 0))[at];
            a.part_bc[((chan_block * tokens + (long long)b * a.T + t0 + j) * 2 + c) * NP + n] = v;
        }
        // dx, ddt, dz
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int q = i * RPP + lrow, t = t0 + q;
            if (t >= t1 || lrest <= 0) continue;
            float d[8], z[8], g[8], o[8];
            const long long at = ((long long)b * a.T + t) * a.D + lc;
            const int in = q * CH + lv * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = xs[in + e];
            store8<T>(static_cast<T *>(a.out) + at, o, lrest, a.vec);
            unpack<T, 8>(load8<T>(pd + t * a.dt_token, lrest, a.vec), d);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                o[e] = st[in + e] * (a.softplus ? sigmoid_f32(d[e] + bias[e]) : 1.f);
                dbias[e] += o[e];
            }
            store8<T>(static_cast<T *>(a.ddt) + at, o, lrest, a.vec);
            if (a.z) {
                unpack<T, 8>(load8<T>(pz + t * a.z_token, lrest, a.vec), z);
                unpack<T, 8>(load8<T>(pg + t * a.dy_token, lrest, a.vec), g);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float sg = sigmoid_f32(z[e]);
                    o[e] = g[e] * gs[in + e] * sg * fmaf(z[e], 1.f - sg, 1.f);
                }
                store8<T>(static_cast<T *>(a.dz) + at, o, lrest, a.vec);
            }
        }
    }
    // the segment's sums over tokens
#pragma unroll
    for (int cs = 0; cs < CS; ++cs)
        if (channel(cs) < a.D) store_pairs(a.part_a + ((long long)seg * a.D + channel(cs)) * NP, n0, NP, dA[cs]);
    __syncthreads();
    float *sum = reinterpret_cast<float *>(raw);   // [2][RPP][CH]
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        sum[lrow * CH + lv * 8 + e] = dskip[e];
        sum[(RPP + lrow) * CH + lv * 8 + e] = dbias[e];
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

// dB, dC in the activations' type, over the blocks of channels.
template <typename T>
__global__ void __launch_bounds__(256) scan_bwd_bc_kernel(const float *part, int blocks, long long tokens, int N, int NP,
                                                          T *dB, T *dC) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, size = tokens * 2 * NP;
    if (i >= size) return;
    const int n = (int)(i % NP), c = (int)(i / NP % 2);
    if (n >= N) return;
    float v = 0.f;
#pragma unroll 4
    for (int k = 0; k < blocks; ++k) v += part[k * size + i];
    (c ? dC : dB)[i / (2 * NP) * N + n] = from_f32<T>(v);
}

// dA, dD and ddt_bias over the segments: eight groups of segments per 32
// values, then the groups in order.
__global__ void __launch_bounds__(256) scan_bwd_param_kernel(const float *part_a, const float *part_v, int segs, int D,
                                                             int N, int NP, float *dA, float *dskip, float *dbias) {
    __shared__ float sum[8][32];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const long long i = (long long)blockIdx.x * 32 + lane, na = (long long)D * NP, total = na + 2 * D;
    float v = 0.f;
    if (i < total) {
        const float *p = i < na ? part_a + i : part_v + (i - na);
        const long long step = i < na ? na : 2 * D;
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
        if (i % NP < N) dA[i / NP * N + i % NP] = v;
    } else if (i - na < D) {
        if (dskip) dskip[i - na] = v;
    } else if (dbias) {
        dbias[i - na - D] = v;
    }
}

template <typename T, int LP>
cudaError_t launch_maps(ScanArgs a, cudaStream_t s) {
    a.chan_blocks = (a.D + kMapThreads / LP - 1) / (kMapThreads / LP);
    scan_tile_maps_kernel<T, LP><<<(unsigned)((long long)a.chan_blocks * a.B * a.row_tiles), kMapThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int NL>
cudaError_t launch_main(ScanArgs a, cudaStream_t s) {
    using S = BwdShape<NL>;
    const cudaError_t attr =
        cudaFuncSetAttribute(scan_bwd_kernel<T, NL>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::smem);
    if (attr != cudaSuccess) return attr;
    scan_bwd_kernel<T, NL><<<(unsigned)((long long)a.chan_blocks * a.B * a.segs), kBwdThreads, S::smem, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bwd_typed(const ScanArgs &a, T *dB, T *dC, float *dA, float *dskip, float *dbias, cudaStream_t s) {
    const int parts = scan_parts(a.N), NP = 8 * parts;
    const long long tokens = (long long)a.B * a.T;
    cudaError_t e = cudaSuccess;
    if (tokens > 0) {
        switch (parts) {
            case 1: e = launch_maps<T, 1>(a, s); break;
            case 2: e = launch_maps<T, 2>(a, s); break;
            case 4: e = launch_maps<T, 4>(a, s); break;
            default: e = launch_maps<T, 8>(a, s);
        }
        if (e == cudaSuccess) e = launch_scan_combine(a, a.row_tiles, true, s);
        if (e != cudaSuccess) return e;
    }
    switch (parts) {
        case 1: e = launch_main<T, 2>(a, s); break;
        case 2: e = launch_main<T, 4>(a, s); break;
        case 4: e = launch_main<T, 8>(a, s); break;
        default: e = launch_main<T, 16>(a, s);
    }
    if (e != cudaSuccess) return e;
    if (tokens > 0) {
        scan_bwd_bc_kernel<T><<<(unsigned)((tokens * 2 * NP + 255) / 256), 256, 0, s>>>(a.part_bc, a.chan_blocks, tokens,
                                                                                       a.N, NP, dB, dC);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    scan_bwd_param_kernel<<<(unsigned)(((long long)a.D * (NP + 2) + 31) / 32), 256, 0, s>>>(
        a.part_a, a.part_v, tokens > 0 ? a.B * a.segs : 0, a.D, a.N, NP, dA, dskip, dbias);
    return cudaGetLastError();
}

}  // namespace

int scan_bwd_channels(int N) { return N <= 8 ? BwdShape<2>::CH : N <= 16 ? BwdShape<4>::CH : N <= 32 ? BwdShape<8>::CH : BwdShape<16>::CH; }

cudaError_t launch_scan_bwd(const ScanArgs &a, int dtype, void *dB, void *dC, float *dA, float *dskip, float *dbias,
                            cudaStream_t s) {
    return dtype == GDN_BF16 ? launch_bwd_typed<__nv_bfloat16>(a, static_cast<__nv_bfloat16 *>(dB),
                                                               static_cast<__nv_bfloat16 *>(dC), dA, dskip, dbias, s)
                             : launch_bwd_typed<float>(a, static_cast<float *>(dB), static_cast<float *>(dC), dA, dskip,
                                                       dbias, s);
}

}  // namespace gdn
