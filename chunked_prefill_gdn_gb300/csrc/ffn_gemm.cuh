// The matrix products of the gated feed-forward block: one persistent tcgen05
// kernel, out = sum over K of A B^T, with the block's elementwise parts in its
// epilogue, for up to four products in one launch.
//
// Operands are bf16 in memory, [rows][K] (K-major) or [K][rows] (MN-major, for
// the products that sum over rows of what is stored), read by TMA into tiles with
// the 128-byte swizzle; whatever lies past a tensor's edge is zero.  fp32 values
// are three bf16 planes, x = x0 + x1 + x2 exactly to 2^-24 of x, and a product is
// the six terms x_i y_j with i + j <= 2 (the three left out are below 2^-24),
// smallest first.
//
// A tile is 128 rows x BN columns per CTA; with CTAS = 2 two CTAs form a pair
// (cta_group::2) of 256 x 256, each holding its own 128 rows of A and half of B,
// which halves what B costs in L2 and shared memory.  Single CTAs of 128 columns run
// two to an SM, for few rows (bound by the weights' bytes) and for small products.
// The accumulators are in tensor memory, two sets of BN columns, so that the epilogue
// of one tile runs under the products of the next.  Warps: 0 loads, 1 issues the
// products, the others are the epilogue, a quarter of the lanes and CW columns each: eight warps, and 16 where the
// epilogue is the longer part (backward pass's first product of 8192 x 256 x 8192: 190 us,
// with eight 229; the forward one with gate and up kept is 4% faster with eight).
// bf16 outputs leave through a box per warp in shared memory by TMA stores.  A sixth
// stage of operands is worth more than a second box per warp, or than boxes into which
// the backward pass's gate and up are loaded ahead (8191 x 4096 x 12288: first backward
// product 514 us, with those 555).
//
// With PROMOTE (fp32) the tensor cores sum only kPromote blocks of K at a time;
// those sums are added in registers, in fp32 with rounding to nearest.
//
// Every wait is bounded; when one runs out the kernel records GDN_ERR_TIMEOUT,
// lets its copies land, frees its tensor memory and returns.
#pragma once

#include <cuda.h>

#include "elem.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace ffn {

enum Epi { kUp = 0, kBack = 1, kPlain = 2 };

constexpr int kTileM = 128, kBlockK = 64;
// Blocks of 64 along K per sum in tensor memory (fp32).  The tensor cores cut what an
// addition leaves over; errors against 64 bits at 2048 x 2048 x 6144: 1.5e-6 with eight blocks,
// 7e-7 with four (5% slower: 645 us), 4e-7 with two (another 3%); products in fp32 throughout
// 1.9e-6.
constexpr int kPromote = 4;
constexpr int kMaxStages = 6, kMaxGroups = 4;
constexpr uint64_t kTimeoutNs = 2000000000ull;

// One product of the launch: out = sum over its pairs of A B^T.
struct Group {
    int M, N;                 // outputs (kUp: N = F, half a tile's columns)
    int mt, nt;               // tiles
    int kb, pairs, splits;    // K blocks of a pair of operands; pairs summed up; parts of that sum
    int a, b, c;              // first of its maps
    int a_mn, b_mn, tma_out, vec_out;
    void *out;                // kPlain: [M, N], rows ld_out apart
    long long ld_out;
    float *partial;           // or null: parts of sums, [split][kUp ? 2 : 1][M][ld_part]
    long long ld_part;
};
struct GemmArgs {
    CUtensorMap a[kMaxGroups + 1], b[kMaxGroups + 1], c[kMaxGroups], io[2];   // one product may have two pairs
    Group group[kMaxGroups];
    int groups, dual;         // dual: the tile's column halves come from b[0] and b[1]
    // the schedule: the longest units come first, `rest` others follow; see item_of
    int first, rest, ratio;
    int terms;                // 1, or 6 for three planes
    int a_rows, stages;       // few_rows: rows of A's boxes (32, 64, 128) and stages (5, 4, 3)
    int probe;                // GDN_DEBUG_TIMEOUT_PROBE: nothing is loaded, every wait runs out
    int act, tma_io, vec_io;  // kUp: gate and up leave through boxes; rows of both in 16-byte vectors
    __nv_bfloat16 *planes[3]; // kUp: h; kBack: dgate, dup, h: one plane (bf16) or three (fp32)
    long long ld_plane, plane_stride;
    void *gate, *up;          // kUp: outputs or null; kBack: inputs; contiguous
    int *err;
};

// act(g) = g sigmoid(p(g)), p(g) = g or C1 (g + C3 g^3): silu, or gelu with tanh
// (0.5 (1 + tanh(u)) = sigmoid(2 u)).  Returns sigmoid(p) and p'.
constexpr float kGelu1 = 1.5957691216057308f, kGelu3 = 0.044715f;
__device__ __forceinline__ float act_sigmoid(float g, int act, float &slope) {
    float p = g;
    slope = 1.f;
    if (act) {
        const float q = g * g;
        p = kGelu1 * g * fmaf(kGelu3, q, 1.f);
        slope = kGelu1 * fmaf(3.f * kGelu3, q, 1.f);
    }
    return sigmoid_f32(p);
}
__device__ __forceinline__ float act_times(float g, float u, int act) {
    float slope;
    return g * act_sigmoid(g, act, slope) * u;
}
// dg = dh u act'(g), du = dh act(g), h = act(g) u.  Where the sigmoid has reached
// 0 or 1 the slope's term is zero, whatever p' (infinite where g^2 is).
__device__ __forceinline__ void act_back(float dh, float g, float u, int act, float &dg, float &du, float &h) {
    float slope;
    const float s = act_sigmoid(g, act, slope), a = g * s, t = a * (1.f - s);
    dg = dh * u * (t == 0.f ? s : fmaf(t, slope, s));
    du = dh * a;
    h = a * u;
}

// The same on pairs, for an activation that is known (ACT).
template <int ACT>
__device__ __forceinline__ F2 act_sigmoid2(F2 g, F2 &slope) {
    if constexpr (ACT == 0) return sigmoid_pair(g);
    const F2 q = mul2(g, g);
    slope = mul2(both(kGelu1), fma2(both(3.f * kGelu3), q, both(1.f)));
    return sigmoid_pair(mul2(mul2(both(kGelu1), g), fma2(both(kGelu3), q, both(1.f))));
}
// x = act(x) u
template <int ACT, int E>
__device__ __forceinline__ void act_times_cols(float (&x)[E], const float (&u)[E]) {
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        F2 slope;
        const F2 g = pair(x[e], x[e + 1]), h = mul2(mul2(g, act_sigmoid2<ACT>(g, slope)), pair(u[e], u[e + 1]));
        x[e] = lo(h), x[e + 1] = hi(h);
    }
}
// (dh, g, u) = (dg, h, du)
template <int ACT, int E>
__device__ __forceinline__ void act_back_cols(float (&d)[E], float (&x)[E], float (&u)[E]) {
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        F2 slope;
        const F2 g = pair(x[e], x[e + 1]), uu = pair(u[e], u[e + 1]), dh = pair(d[e], d[e + 1]);
        const F2 s = act_sigmoid2<ACT>(g, slope), a = mul2(g, s), t = mul2(a, fma2(s, both(-1.f), both(1.f)));
        F2 f;
        if constexpr (ACT == 0) f = add2(t, s);
        else f = pair(lo(t) == 0.f ? lo(s) : fmaf(lo(t), lo(slope), lo(s)), hi(t) == 0.f ? hi(s) : fmaf(hi(t), hi(slope), hi(s)));
        const F2 dg = mul2(mul2(dh, uu), f), du = mul2(dh, a), h = mul2(a, uu);
        d[e] = lo(dg), d[e + 1] = hi(dg), u[e] = lo(du), u[e + 1] = hi(du), x[e] = lo(h), x[e + 1] = hi(h);
    }
}

// x = p0 + p1 + p2 (three roundings to nearest); what is not finite stays in p0.
__device__ __forceinline__ void split3(float x, float (&p)[3]) {
    p[0] = __bfloat162float(__float2bfloat16_rn(x));
    const bool fine = fabsf(p[0]) < INFINITY;
    const float r1 = fine ? x - p[0] : 0.f;
    p[1] = __bfloat162float(__float2bfloat16_rn(r1));
    p[2] = r1 - p[1];
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_to_cta(uint32_t saddr, uint32_t cta) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(cta));
    return r;
}

template <int CTAS>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z) {
    if constexpr (CTAS == 2)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
            : "memory");
}
template <int CTAS>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (CTAS == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        tc::mma_ss(d, a, b, idesc, accumulate);
}
// Arrives on `bar` (with CTAS = 2 on both CTAs') once all products issued so far are done.
template <int CTAS>
__device__ __forceinline__ void commit(uint64_t *bar) {
    if constexpr (CTAS == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                tc::smem_u32(bar)),
            "h"((unsigned short)3)
            : "memory");
    else
        tc::tc_commit(bar);
}
template <int CTAS, int COLS>
__device__ __forceinline__ void tmem_get(uint32_t *dst) {
    if constexpr (CTAS == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(dst)), "n"(COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tc::tmem_alloc(dst, COLS);
        tc::tmem_relinquish();
    }
}
template <int CTAS, int COLS>
__device__ __forceinline__ void tmem_free(uint32_t addr) {
    if constexpr (CTAS == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "n"(COLS) : "memory");
    else
        tc::tmem_dealloc(addr, COLS);
}
template <int LATER>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(LATER) : "memory");
}

template <int EPI, typename T, int CTAS, int BN>
struct Shape {
    static constexpr bool promote = sizeof(T) == 4;
    // columns per warp of the epilogue: 64 where it holds sums (fp32) or is long (kBack)
    static constexpr int CW = promote || EPI == kBack ? 64 : 128, epi_warps = BN * 4 / CW, threads = 64 + 32 * epi_warps;
    static constexpr int box_cols = CW / 2;                      // of a box of 32 rows
    static constexpr int b_rows = BN / CTAS;                     // of B in this CTA
    static constexpr int a_bytes = kTileM * 128, b_bytes = b_rows * 128, stage = a_bytes + b_bytes;
    static constexpr bool boxes = !promote && BN == 256;
    // Tiles of 128 columns take A in boxes of 32 or 64 rows where there are no more rows, and
    // as many stages as then fit (the products read 128 rows from there on, B's first ones
    // among them; what comes of those is not stored).
    static constexpr bool few_rows = BN == 128;
    static constexpr int stages = few_rows ? 3 : CTAS == 2 ? 6 : 4, area = few_rows ? 102400 : stages * stage;
    static constexpr int box_bytes = boxes ? 64 * box_cols : 1024;   // per warp: the box, or room to turn 32 x 8 values
    static constexpr int smem = 1024 + area + epi_warps * box_bytes;   // 1024: alignment
    static constexpr int per_sm = BN == 128 ? 2 : 1;
    static_assert(stages <= kMaxStages && stages * stage <= area && smem + 512 <= 227 * 1024 / per_sm - (per_sm - 1) * 1024, "shared memory");
};

struct Barriers {
    uint64_t full[kMaxStages], empty[kMaxStages], tmem_full[2], tmem_empty[2];
    uint32_t tmem;
    int abort;
};

// One part of the work: a tile and a range of blocks along K.
struct Item {
    int group, m, n, split, q0, q1;   // tile coordinates; blocks [q0, q1) of pairs * kb
};
// The i-th unit of worker p of P, or none (false).  The longest units (the first groups',
// `first` of them) are dealt out in turn; the workers that get one less take `ratio` units of
// the others instead, which are then dealt out in turn too.  Within a group the tiles go
// in bands of 16 rows of tiles of 128, so that what is at work at one time shares what it
// reads in L2.
template <int CTAS>
__device__ __forceinline__ bool item_of(const GemmArgs &g, int p, int P, int i, Item &it) {
    const int extra = g.first % P, mine = (g.first - p + P - 1) / P, behind = extra ? P - extra : 0;
    int w;
    if (i < mine) {
        w = p + i * P;
    } else {
        i -= mine;
        if (extra && p >= extra) {
            w = i < g.ratio ? i * behind + (p - extra) : g.ratio * behind + p + (i - g.ratio) * P;
        } else {
            w = g.ratio * behind + p + i * P;
        }
        if (w >= g.rest) return false;
        w += g.first;
    }
    int grp = 0;
    while (true) {
        const Group &q = g.group[grp];
        const int units = q.mt * q.nt * q.splits;
        if (w < units) break;
        w -= units;
        ++grp;
    }
    const Group &q = g.group[grp];
    it.group = grp;
    it.split = w % q.splits;
    w /= q.splits;
    constexpr int GM = 16 / CTAS;
    const int band = w / (GM * q.nt), first = band * GM, rows = min(GM, q.mt - first);
    w -= band * GM * q.nt;
    it.m = first + w % rows;
    it.n = w / rows;
    const int blocks = q.kb * q.pairs;
    it.q0 = (int)((long long)blocks * it.split / q.splits);
    it.q1 = (int)((long long)blocks * (it.split + 1) / q.splits);
    return true;
}
// Terms of a product of three planes by three, smallest first.
__device__ __forceinline__ void term_planes(int terms, int t, int &pa, int &pb) {
    if (terms == 1) { pa = pb = 0; return; }
    pa = (0x001012 >> (4 * t)) & 15;   // t = 0..5: 2 1 0 1 0 0
    pb = (0x010210 >> (4 * t)) & 15;   //           0 1 2 0 1 0
}

// E neighbouring columns of a row in type T, in 16-byte vectors where the row has them
// all, else one by one.
template <typename T, int E>
__device__ __forceinline__ void store_cols(T *p, const float *v, int live, bool vec) {
    constexpr int V = 16 / (int)sizeof(T);
    if (vec && live >= E) {
#pragma unroll
        for (int i = 0; i < E / V; ++i) store_raw<T, V>(p + i * V, pack<T, V>(v + i * V));
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (i < live) p[i] = from_f32<T>(v[i]);
    }
}
template <typename T, int E>
__device__ __forceinline__ void load_cols(const T *p, float *v) {
    constexpr int V = 16 / (int)sizeof(T);
    Raw<T, V> r[E / V];
#pragma unroll
    for (int i = 0; i < E / V; ++i) r[i] = load_raw<T, V>(p + i * V);
#pragma unroll
    for (int i = 0; i < E / V; ++i) unpack<T, V>(r[i], v + i * V);
}
// The same for the warp's 32 rows together, where rows are not 16-byte aligned or end
// within the E columns: eight columns at a time are turned in shared memory, so that
// neighbouring lanes access neighbouring columns (a lane per row alone touches 32 lines
// with every access).  The tile's first row and column are given.
template <typename T, int E>
__device__ __forceinline__ void store_turned(T *base, long long ld, int row0, int col, int M, int N, const float *v, float *room, int lane) {
#pragma unroll
    for (int j = 0; j < E; j += 8) {
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) room[lane * 8 + (e ^ (lane & 7))] = v[j + e];
        __syncwarp();
        const int c = lane & 7;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = 4 * k + (lane >> 3);
            if (row0 + r < M && col + j + c < N) base[(long long)(row0 + r) * ld + col + j + c] = from_f32<T>(room[r * 8 + (c ^ (r & 7))]);
        }
    }
}
template <typename T, int E>
__device__ __forceinline__ void load_turned(const T *base, long long ld, int row0, int col, int M, int N, float *v, float *room, int lane) {
    const int c = lane & 7;
    float t[E];
#pragma unroll
    for (int j = 0; j < E; j += 8)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = 4 * k + (lane >> 3);
            t[j + k] = row0 + r < M && col + j + c < N ? to_f32(base[(long long)(row0 + r) * ld + col + j + c]) : 0.f;
        }
#pragma unroll
    for (int j = 0; j < E; j += 8) {
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = 4 * k + (lane >> 3);
            room[r * 8 + (c ^ (r & 7))] = t[j + k];
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j + e] = room[lane * 8 + (e ^ (lane & 7))];
    }
}
// E columns into one plane (bf16) or three (fp32); ld is a multiple of 8, so whole
// vectors lie in the row.
template <typename T, int E>
__device__ __forceinline__ void store_planes(__nv_bfloat16 *p, long long stride, const float *v, int live) {
    if constexpr (sizeof(T) == 2) {
        store_cols<__nv_bfloat16, E>(p, v, live, true);
    } else {
        float s[3][E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float t[3];
            split3(v[e], t);
            s[0][e] = t[0], s[1][e] = t[1], s[2][e] = t[2];
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) store_cols<__nv_bfloat16, E>(p + k * stride, s[k], live, true);
    }
}

template <int EPI, typename T, int CTAS, int BN>
__global__ void __launch_bounds__(Shape<EPI, T, CTAS, BN>::threads, Shape<EPI, T, CTAS, BN>::per_sm)
    ffn_gemm_kernel(const __grid_constant__ GemmArgs g) {
    using S = Shape<EPI, T, CTAS, BN>;
    constexpr bool PROMOTE = S::promote, BOXES = S::boxes;
    constexpr int CW = S::CW, E = PROMOTE ? 16 : 32;   // columns of a step of the epilogue
    extern __shared__ uint8_t raw[];
    __shared__ Barriers bars;
    uint8_t *smem = raw + ((1024u - (tc::smem_u32(raw) & 1023u)) & 1023u);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = CTAS == 2 ? cluster_rank() : 0u;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) tc::mbar_init(&bars.full[i], 1), tc::mbar_init(&bars.empty[i], 1);
        for (int i = 0; i < 2; ++i) tc::mbar_init(&bars.tmem_full[i], 1), tc::mbar_init(&bars.tmem_empty[i], S::epi_warps * CTAS);
        bars.abort = 0;
        tc::fence_barrier_init();
    }
    if (warp == 1) tmem_get<CTAS, 2 * BN>(&bars.tmem);
    tc::tc_fence_before();
    __syncthreads();
    if constexpr (CTAS == 2) cluster_sync_all();
    tc::tc_fence_after();
    const uint32_t tmem = bars.tmem;
    volatile int *abort = &bars.abort;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (tc::mbar_wait(bar, parity, abort, kTimeoutNs)) return true;
        if (*abort == 0 && g.err) report_error(g.err, GDN_ERR_TIMEOUT);
        *abort = 1;
        return false;
    };
    grid_dependency_wait();
    const int P = gridDim.x / CTAS, p = blockIdx.x / CTAS;
    const uint32_t n_stages = S::few_rows ? g.stages : S::stages, a_bytes = S::few_rows ? g.a_rows * 128 : S::a_bytes;
    const uint32_t stage = a_bytes + S::b_bytes;
    const int chunk = PROMOTE ? kPromote : 1 << 30;
    Item i;

    // Loads and products are issued by one lane, but the whole warp goes through their
    // loops: what it decides on is then the warp's, and stays in uniform registers (with
    // only one lane in the loops the copies were issued at half the rate).
    auto warp_wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
    if (warp == 0) {
        const bool leader = tc::elect_one();
        uint32_t s = 0, turn = 0, loads = 0;   // the stage, the parity of its rounds
        bool ok = !g.probe;
        const uint32_t base = tc::smem_u32(smem);
        uint32_t full0 = tc::smem_u32(&bars.full[0]);
        if constexpr (CTAS == 2) full0 = map_to_cta(full0, 0);
        asm volatile("fence.proxy.async;" ::: "memory");   // what earlier kernels stored is read by TMA
        const bool dual = g.dual;
        const int terms = g.terms;
        for (int k = 0; ok && item_of<CTAS>(g, p, P, k, i); ++k) {
            const Group &gr = g.group[i.group];
            const bool a_mn = gr.a_mn, b_mn = gr.b_mn;
            const int row = (i.m * CTAS + (int)rank) * kTileM, kb = gr.kb, a0 = gr.a, b0 = gr.b;
            const int ncol = dual ? i.n * (BN / 2) : i.n * BN + (int)rank * S::b_rows;
            for (int c0 = i.q0; ok && c0 < i.q1; c0 += chunk) {
                const int c1 = min(c0 + chunk, i.q1);
                if (c1 < c0) break;
                for (int t = 0; ok && t < terms; ++t) {
                    int pa, pb;
                    term_planes(terms, t, pa, pb);
                    for (int q = c0; q < c1; ++q) {
                        ok = warp_wait(&bars.empty[s], turn ^ 1);
                        if (!ok) break;
                        const int second = q >= kb ? 1 : 0, kc = (q - second * kb) * kBlockK;
                        const CUtensorMap *ma = &g.a[a0 + second], *mb = &g.b[b0 + (dual && CTAS == 2 ? (int)rank : second)];
                        const uint32_t at = base + s * stage, bt = at + a_bytes, bar = full0 + s * 8;
                        if (leader) {
                            if (CTAS == 1 || rank == 0) tc::mbar_arrive_expect_tx(&bars.full[s], stage * CTAS);
                            if (a_mn) {
#pragma unroll
                                for (int j = 0; j < kTileM / 64; ++j) load_box<CTAS>(at + j * 8192, ma, bar, row + j * 64, kc, pa);
                            } else {
                                load_box<CTAS>(at, ma, bar, kc, row, pa);
                            }
                            // B: boxes of 64 rows where it is MN-major or where a tile has 64 of each half, else of 128
                            if (b_mn) {
#pragma unroll
                                for (int j = 0; j < S::b_rows / 64; ++j) load_box<CTAS>(bt + j * 8192, mb, bar, ncol + j * 64, kc, pb);
                            } else if (CTAS == 1 && dual) {
                                load_box<CTAS>(bt, &g.b[0], bar, kc, ncol, pb);
                                load_box<CTAS>(bt + S::b_bytes / 2, &g.b[1], bar, kc, ncol, pb);
                            } else {
#pragma unroll
                                for (int j = 0; j < S::b_rows / 128; ++j) load_box<CTAS>(bt + j * 16384, mb, bar, kc, ncol + j * 128, pb);
                            }
                        }
                        __syncwarp();
                        ++loads;
                        if (++s == n_stages) s = 0, turn ^= 1;
                    }
                }
            }
        }
        // the products have read every stage before the CTA may leave
        for (uint32_t j = 0; ok && j < min(loads, n_stages); ++j) {
            if (s == 0) s = n_stages, turn ^= 1;
            ok = warp_wait(&bars.empty[--s], turn);
        }
    } else if (warp == 1) {
        const bool leader = tc::elect_one();
        if (rank == 0) {
            uint32_t s = 0, turn = 0, n = 0;
            bool ok = true;
            const uint32_t base = tc::smem_u32(smem);
            const int terms = g.terms;
            for (int k = 0; ok && item_of<CTAS>(g, p, P, k, i); ++k) {
                const int a_mn = g.group[i.group].a_mn, b_mn = g.group[i.group].b_mn;
                const uint32_t idesc = tc::idesc_bf16_f32(kTileM * CTAS, BN, a_mn, b_mn);
                const uint32_t ka = a_mn ? 128 : 2, kbs = b_mn ? 128 : 2;   // 16 of K on, in 16-byte units
                const uint64_t da0 = tc::smem_desc_sw128(base, a_mn ? 8192 : 16, 1024);
                const uint64_t db0 = tc::smem_desc_sw128(base + a_bytes, b_mn ? 8192 : 16, 1024);
                for (int c0 = i.q0; ok && c0 < i.q1; c0 += chunk, ++n) {
                    const int c1 = min(c0 + chunk, i.q1);
                    if (c1 < c0) break;
                    const uint32_t buf = n & 1;
                    ok = n < 2 || warp_wait(&bars.tmem_empty[buf], ((n >> 1) - 1) & 1);
                    if (!ok) break;
                    tc::tc_fence_after();
                    const uint32_t d = tmem + buf * BN;
                    const int count = (c1 - c0) * terms;
                    for (int q = 0; q < count; ++q) {
                        ok = warp_wait(&bars.full[s], turn);
                        if (!ok) break;
                        tc::tc_fence_after();
                        const uint64_t da = da0 + s * (stage / 16), db = db0 + s * (stage / 16);
                        if (leader) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) mma_bf16<CTAS>(d, da + kk * ka, db + kk * kbs, idesc, q > 0 || kk > 0);
                            commit<CTAS>(&bars.empty[s]);
                        }
                        __syncwarp();
                        if (++s == n_stages) s = 0, turn ^= 1;
                    }
                    if (ok && leader) commit<CTAS>(&bars.tmem_full[buf]);
                    __syncwarp();
                }
            }
        }
    } else {
        const int quarter = warp & 3, part_of = (warp - 2) >> 2;   // the warp's lanes, and its CW columns
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        uint8_t *box = smem + S::area + (warp - 2) * S::box_bytes;
        const uint32_t box_at = tc::smem_u32(box);
        const uint32_t release = CTAS == 2 ? map_to_cta(tc::smem_u32(&bars.tmem_empty[0]), 0) : 0u;
        uint32_t n = 0;
        bool ok = true;
        // chunk c of a row of the box, swizzled as TMA reads it; 32 packed columns from chunk 4 part on
        auto put16 = [&](int c, uint4 v) {
            tc::sts_u4(box_at + (S::box_cols == 64 ? tc::sw128_offset(lane, c) : lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)), v);
        };
        auto put = [&](const float *v, int part) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const Raw<__nv_bfloat16, 8> r = pack<__nv_bfloat16, 8>(v + 8 * c);
                put16(4 * part + c, make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]));
            }
        };
        auto box_free = [&]() {   // the last store has read it
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
        };
        auto box_out = [&](const CUtensorMap *map, int col, int row, int ncols, int nrows) {
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && col < ncols && row < nrows) {
                tc::tma_store_3d(map, box, col, row, 0);
                tc::bulk_commit_group();
            }
        };
        for (int k = 0; item_of<CTAS>(g, p, P, k, i); ++k) {
            const Group &gr = g.group[i.group];
            const int row0 = (i.m * CTAS + (int)rank) * kTileM + quarter * 32, row = row0 + lane;
            const bool in = row < gr.M;
            uint32_t from = 0;
            auto column = [&](int j) {   // tensor memory column of the warp's column j
                return EPI == kUp ? (j < CW / 2 ? part_of * (CW / 2) + j : BN / 2 + part_of * (CW / 2) + j - CW / 2) : part_of * CW + j;
            };
            auto done = [&]() {
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CTAS == 2)
                        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(release + (n & 1) * 8) : "memory");
                    else
                        tc::mbar_arrive(&bars.tmem_empty[n & 1]);
                }
                ++n;
            };
            // fp32: all sums but the last are taken out, added up in registers, and the total
            // goes back to where the last one lies
            if constexpr (PROMOTE) {
                float acc[CW];
                const int chunks = (i.q1 - i.q0 + kPromote - 1) / kPromote;
                for (int c = 0; c < chunks; ++c) {
                    ok = __all_sync(0xffffffffu, wait(&bars.tmem_full[n & 1], (n >> 1) & 1));
                    if (!ok) break;
                    tc::tc_fence_after();
                    from = tmem + (n & 1) * BN + lanes;
                    if (chunks == 1) break;
                    const bool last = c + 1 == chunks;
#pragma unroll
                    for (int j = 0; j < CW; j += 16) {
                        uint32_t v[16];
                        tc::tmem_ld16(from + column(j), v);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            acc[j + e] = c == 0 ? __uint_as_float(v[e]) : acc[j + e] + __uint_as_float(v[e]);
                            v[e] = __float_as_uint(acc[j + e]);
                        }
                        if (last) tc::tmem_st16(from + column(j), v);
                    }
                    if (last) tc::tmem_wait_st();
                    else done();
                }
            } else {
                ok = __all_sync(0xffffffffu, wait(&bars.tmem_full[n & 1], (n >> 1) & 1));
                tc::tc_fence_after();
                from = tmem + (n & 1) * BN + lanes;
            }
            if (!ok) break;
            auto get = [&](int j, auto &v) {   // the warp's columns from j on, as many as v holds
                constexpr int W = sizeof(v) / 4;
                if constexpr (W == 16) tc::tmem_ld16(from + column(j), reinterpret_cast<uint32_t *>(v));
                else tc::tmem_ld32(from + column(j), reinterpret_cast<uint32_t *>(v));
                tc::tmem_wait_ld();
            };
            // first output column of the warp
            const int col = EPI == kUp ? i.n * (BN / 2) + part_of * (CW / 2) : i.n * BN + part_of * CW;
            constexpr int kUnroll = PROMOTE ? 1 : 2;
            float *room = reinterpret_cast<float *>(box);
            // E columns of a [M, N] tensor of rows ld apart, from column `at` on
            auto store = [&](T *base, long long ld, int at, const float *v, bool vec) {
                if (vec && at + E <= gr.N) {
                    if (in) store_cols<T, E>(base + row * ld + at, v, E, true);
                } else if (at < gr.N) {
                    store_turned<T, E>(base, ld, row0, at, gr.M, gr.N, v, room, lane);
                }
            };
            auto load = [&](const T *base, int at, auto &v) {
                constexpr int W = sizeof(v) / 4;
                if (g.vec_io && at + W <= gr.N) load_cols<T, W>(base + (long long)(in ? row : 0) * gr.N + at, v);
                else load_turned<T, W>(base, gr.N, row0, at, gr.M, gr.N, v, room, lane);
            };
            if (gr.partial) {
#pragma unroll 1
                for (int j = 0; j < CW; j += E) {
                    float v[E];
                    get(j, v);
                    const int which = EPI == kUp ? j / (CW / 2) : 0, at = EPI == kUp ? col + j % (CW / 2) : col + j;
                    if (in && at < gr.N)
                        store_cols<float, E>(gr.partial + (((long long)i.split * (EPI == kUp ? 2 : 1) + which) * gr.M + row) * gr.ld_part + at,
                                             v, (int)gr.ld_part - at, true);
                }
            } else if constexpr (EPI == kUp) {
                if (g.gate) {
#pragma unroll
                    for (int o = 0; o < 2; ++o) {
                        T *dst = static_cast<T *>(o ? g.up : g.gate);
                        if constexpr (BOXES) box_free();
#pragma unroll kUnroll
                        for (int j = 0; j < CW / 2; j += E) {
                            float v[E];
                            get(CW / 2 * o + j, v);
                            if (BOXES && g.tma_io) put(v, j / 32);
                            else store(dst, gr.N, col + j, v, g.vec_io);
                        }
                        if (BOXES && g.tma_io) box_out(&g.io[o], col, row0, gr.N, gr.M);
                    }
                }
                if constexpr (BOXES) box_free();
#pragma unroll kUnroll
                for (int j = 0; j < CW / 2; j += E) {
                    float x[E], u[E];
                    get(j, x);
                    get(CW / 2 + j, u);
                    if (g.act) act_times_cols<1, E>(x, u);
                    else act_times_cols<0, E>(x, u);
                    if constexpr (BOXES) put(x, j / 32);
                    else if (in && col + j < gr.N)
                        store_planes<T, E>(g.planes[0] + row * g.ld_plane + col + j, g.plane_stride, x, (int)g.ld_plane - col - j);
                }
                if constexpr (BOXES) box_out(&g.c[0], col, row0, gr.N, gr.M);
            } else if constexpr (EPI == kBack) {
                const T *gate = static_cast<const T *>(g.gate), *up = static_cast<const T *>(g.up);
                constexpr int W = 16;   // columns at a time: three values of each in registers
                auto step = [&](int j, float (&d)[W], float (&x)[W], float (&u)[W]) {
                    load(gate, col + j, x);
                    load(up, col + j, u);
                    get(j, d);
                    if (g.act) act_back_cols<1, W>(d, x, u);
                    else act_back_cols<0, W>(d, x, u);
                };
#pragma unroll 1
                for (int j = 0; j < CW; j += BOXES ? 32 : W) {
                    float d[W], x[W], u[W];
                    if constexpr (BOXES) {
                        if (!g.vec_io || col + j + 32 > gr.N) box_free();   // load turns the values there
                        uint32_t pk[3][16];
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            step(j + 16 * half, d, x, u);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                pk[0][8 * half + e] = tc::pack_bf16x2(d[2 * e], d[2 * e + 1]);
                                pk[1][8 * half + e] = tc::pack_bf16x2(u[2 * e], u[2 * e + 1]);
                                pk[2][8 * half + e] = tc::pack_bf16x2(x[2 * e], x[2 * e + 1]);
                            }
                        }
#pragma unroll
                        for (int o = 0; o < 3; ++o) {
                            box_free();
#pragma unroll
                            for (int c = 0; c < 4; ++c) put16(c, make_uint4(pk[o][4 * c], pk[o][4 * c + 1], pk[o][4 * c + 2], pk[o][4 * c + 3]));
                            box_out(&g.c[o], col + j, row0, gr.N, gr.M);
                        }
                    } else {
                        step(j, d, x, u);
                        if (in && col + j < gr.N) {
                            const long long to = row * g.ld_plane + col + j;
                            const int room_left = (int)g.ld_plane - col - j;
                            store_planes<T, W>(g.planes[0] + to, g.plane_stride, d, room_left);
                            store_planes<T, W>(g.planes[1] + to, g.plane_stride, u, room_left);
                            store_planes<T, W>(g.planes[2] + to, g.plane_stride, x, room_left);
                        }
                    }
                }
            } else {
                T *out = static_cast<T *>(gr.out);
                const bool box_it = BOXES && gr.tma_out;
                constexpr int STEP = BOXES ? S::box_cols : CW;
#pragma unroll
                for (int part = 0; part < CW; part += STEP) {
                    if constexpr (BOXES) box_free();
#pragma unroll kUnroll
                    for (int j = 0; j < STEP; j += E) {
                        float v[E];
                        get(part + j, v);
                        if (box_it) put(v, j / 32);
                        else store(out, gr.ld_out, col + part + j, v, gr.vec_out);
                    }
                    if (box_it) box_out(&g.c[gr.c], col + part, row0, gr.N, gr.M);
                }
            }
            done();
        }
        if (lane == 0) tc::bulk_wait_group_all();
    }
    __syncwarp();
    if (*abort) {   // what was under way lands before the shared memory goes
        const uint64_t t0 = tc::global_timer_ns();
        while (tc::global_timer_ns() - t0 < 5000000ull) {
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if constexpr (CTAS == 2) cluster_sync_all();
    tc::tc_fence_after();
    if (warp == 1) tmem_free<CTAS, 2 * BN>(tmem);
}

template <int EPI, typename T, int CTAS, int BN>
cudaError_t launch_gemm(const GemmArgs &g, int grid, cudaStream_t s) {
    using S = Shape<EPI, T, CTAS, BN>;
    cudaError_t e = cudaFuncSetAttribute(ffn_gemm_kernel<EPI, T, CTAS, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(S::threads);
    cfg.dynamicSmemBytes = S::smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CTAS, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CTAS == 2 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, ffn_gemm_kernel<EPI, T, CTAS, BN>, g);
}

// The tile shapes: a pair of 256 x 256, a CTA of 128 x 256, two CTAs to an SM of 128 x 128.
enum Tile { kPair = 0, kWide = 1, kSmall = 2 };

// The instantiations, one translation unit each (ffn_gemm_*.cu).
cudaError_t launch_up(const GemmArgs &g, bool f32, int tile, int grid, cudaStream_t s);
cudaError_t launch_back(const GemmArgs &g, bool f32, int tile, int grid, cudaStream_t s);
cudaError_t launch_plain(const GemmArgs &g, bool f32, int tile, int grid, cudaStream_t s);

template <int EPI, typename T>
cudaError_t launch_tile(const GemmArgs &g, int tile, int grid, cudaStream_t s) {
    return tile == kPair ? launch_gemm<EPI, T, 2, 256>(g, grid, s)
           : tile == kWide ? launch_gemm<EPI, T, 1, 256>(g, grid, s)
                           : launch_gemm<EPI, T, 1, 128>(g, grid, s);
}
#define GDN_FFN_LAUNCHER(NAME, EPI)                                                                                  \
    cudaError_t NAME(const GemmArgs &g, bool f32, int tile, int grid, cudaStream_t s) {                              \
        return f32 ? launch_tile<EPI, float>(g, tile, grid, s) : launch_tile<EPI, __nv_bfloat16>(g, tile, grid, s);  \
    }

}  // namespace ffn
}  // namespace gdn
