// The matrix products of the gated feed-forward block: one persistent tcgen05
// kernel, out = sum over K of A B^T, with the block's elementwise parts in its
// epilogue.
//
// Operands are bf16 in memory, [rows][K] (K-major) or [K][rows] (MN-major, for
// the products that sum over rows of what is stored), read by TMA into tiles with
// the 128-byte swizzle; whatever lies past a tensor's edge is zero.  fp32 values
// are three bf16 planes, x = x0 + x1 + x2 exactly to 2^-24 of x, and a product is
// the six terms x_i y_j with i + j <= 2 (the three left out are below 2^-24),
// smallest first.
//
// A tile is 128 rows x 256 columns per CTA; with CTAS = 2 two CTAs form a pair
// (cta_group::2) of 256 x 256, each holding its own 128 rows of A and half of B,
// which halves what B costs in L2 and shared memory.  The accumulators are in
// tensor memory, two sets of 256 columns, so that the epilogue of one tile runs
// under the products of the next.  Warps: 0 loads, 1 issues the products, 2 to 9
// are the epilogue (two warps per quarter of the lanes, half of the columns each).
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

constexpr int kTileM = 128, kTileN = 256, kBlockK = 64;
constexpr int kEpiWarps = 8, kThreads = 64 + 32 * kEpiWarps;
constexpr int kPromote = 8;   // blocks of 64 along K per sum in tensor memory (fp32)
constexpr uint64_t kTimeoutNs = 2000000000ull;

struct GemmArgs {
    CUtensorMap a[2], b[2], c[3];
    int M, N;                 // outputs of a group (kUp: N = F, half a tile's columns)
    int mt, nt, groups;       // tiles per group, groups (a[g] and out[g], one b)
    int kb, pairs, splits;    // K blocks of one (a[p], b[p]) pair; pairs summed up; parts of that sum
    int terms;                // 1, or 6 for three planes
    int a_mn, b_mn, dual;     // dual: the tile's column halves come from b[0] and b[1]
    int tma_out, vec_out, vec_io, act;
    void *out[2];             // kPlain: [M, N] per group
    long long ld_out;
    __nv_bfloat16 *planes[3]; // kUp: h; kBack: dgate, dup, h: three planes each (fp32)
    long long ld_plane, plane_stride;
    void *gate, *up;          // kUp: outputs or null; kBack: inputs
    long long ld_io;
    float *partial;           // splits > 1: [split][dual ? 2 : groups][M][ld_part]
    long long ld_part;
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
// 0 or 1 the slope's term is zero (p' may be large, not infinite, there).
__device__ __forceinline__ void act_back(float dh, float g, float u, int act, float &dg, float &du, float &h) {
    float slope;
    const float s = act_sigmoid(g, act, slope), a = g * s;
    dg = dh * u * fmaf(a * (1.f - s), slope, s);
    du = dh * a;
    h = a * u;
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
template <int CTAS>
__device__ __forceinline__ void tmem_alloc_all(uint32_t *dst) {
    if constexpr (CTAS == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc::smem_u32(dst)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tc::tmem_alloc(dst, 512);
        tc::tmem_relinquish();
    }
}
template <int CTAS>
__device__ __forceinline__ void tmem_free_all(uint32_t addr) {
    if constexpr (CTAS == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(addr) : "memory");
    else
        tc::tmem_dealloc(addr, 512);
}

template <int CTAS>
struct Shape {
    static constexpr int b_rows = kTileN / CTAS;                 // of B in this CTA
    static constexpr int a_bytes = kTileM * 128, b_bytes = b_rows * 128;
    static constexpr int stage = a_bytes + b_bytes;              // 32 or 48 KB
    static constexpr int stages = CTAS == 2 ? 6 : 4;
    static constexpr int epi = kEpiWarps * 4096;
    static constexpr int smem = 1024 + stages * stage + epi;     // 1024: alignment
};

struct Barriers {
    uint64_t full[6], empty[6], tmem_full[2], tmem_empty[2];
    uint32_t tmem;
    int abort;
};

// One part of the work: a tile and a range of blocks along K.
struct Item {
    int m, n, group, split, q0, q1;   // tile coordinates; blocks [q0, q1) of pairs * kb
};
// Tiles in columns of eight rows of tiles, so that the tiles at work at one time
// share what they read in L2.
template <int CTAS>
__device__ __forceinline__ Item item_of(const GemmArgs &g, int w) {
    Item it;
    it.split = w % g.splits;
    w /= g.splits;
    const int per = g.mt * g.nt;
    it.group = w / per;
    w -= it.group * per;
    constexpr int GM = 16 / CTAS;
    const int band = w / (GM * g.nt), first = band * GM, rows = min(GM, g.mt - first);
    w -= band * GM * g.nt;
    it.m = first + w % rows;
    it.n = w / rows;
    const int q = g.kb * g.pairs;
    it.q0 = (int)((long long)q * it.split / g.splits);
    it.q1 = (int)((long long)q * (it.split + 1) / g.splits);
    return it;
}
// Terms of a product of three planes by three, smallest first.
__device__ __forceinline__ void term_planes(int terms, int t, int &pa, int &pb) {
    if (terms == 1) { pa = pb = 0; return; }
    pa = (0x001012 >> (4 * t)) & 15;   // t = 0..5: 2 1 0 1 0 0
    pb = (0x010210 >> (4 * t)) & 15;   //           0 1 2 0 1 0
}

// 32 neighbouring columns of a row in type T, `live` of which exist.
template <typename T>
__device__ __forceinline__ void store32(T *p, const float *v, int live, bool vec) {
    constexpr int E = 16 / (int)sizeof(T);
    if (vec && live >= 32) {
#pragma unroll
        for (int i = 0; i < 32 / E; ++i) store_raw<T, E>(p + i * E, pack<T, E>(v + i * E));
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < live) p[i] = from_f32<T>(v[i]);
    }
}
template <typename T>
__device__ __forceinline__ void load32(const T *p, float *v, int live, bool vec) {
    constexpr int E = 16 / (int)sizeof(T);
    if (vec && live >= 32) {
        Raw<T, E> r[32 / E];
#pragma unroll
        for (int i = 0; i < 32 / E; ++i) r[i] = load_raw<T, E>(p + i * E);
#pragma unroll
        for (int i = 0; i < 32 / E; ++i) unpack<T, E>(r[i], v + i * E);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = i < live ? to_f32(p[i]) : 0.f;
    }
}

template <int EPI, typename T, int CTAS>
__global__ void __launch_bounds__(kThreads, 1) ffn_gemm_kernel(const __grid_constant__ GemmArgs g) {
    using S = Shape<CTAS>;
    constexpr bool PROMOTE = sizeof(T) == 4;
    extern __shared__ uint8_t raw[];
    __shared__ Barriers bars;
    uint8_t *smem = raw + ((1024u - (tc::smem_u32(raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CTAS == 2 ? cluster_rank() : 0u;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::stages; ++i) tc::mbar_init(&bars.full[i], 1), tc::mbar_init(&bars.empty[i], 1);
        for (int i = 0; i < 2; ++i) tc::mbar_init(&bars.tmem_full[i], 1), tc::mbar_init(&bars.tmem_empty[i], kEpiWarps * CTAS);
        bars.abort = 0;
        tc::fence_barrier_init();
    }
    if (warp == 1) tmem_alloc_all<CTAS>(&bars.tmem);
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
    const int work = g.groups * g.mt * g.nt * g.splits;
    const int step = gridDim.x / CTAS;
    const int chunk = PROMOTE ? kPromote : 1 << 30;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            asm volatile("fence.proxy.async;" ::: "memory");   // what earlier kernels stored is read by TMA
            for (int w = blockIdx.x / CTAS; ok && w < work; w += step) {
                const Item i = item_of<CTAS>(g, w);
                const int row = (i.m * CTAS + (int)rank) * kTileM;
                const int ncol = g.dual ? i.n * (kTileN / 2) : i.n * kTileN + (int)rank * S::b_rows;
                for (int c0 = i.q0; ok && c0 < i.q1; c0 += chunk) {
                    const int c1 = min(c0 + chunk, i.q1);
                    if (c1 < c0) break;
                    for (int t = 0; ok && t < g.terms; ++t) {
                        int pa, pb;
                        term_planes(g.terms, t, pa, pb);
                        for (int q = c0; q < c1; ++q, ++it) {
                            const uint32_t s = it % S::stages, round = it / S::stages;
                            if (round > 0 && !wait(&bars.empty[s], (round - 1) & 1)) { ok = false; break; }
                            const int pair = q >= g.kb ? 1 : 0, k = (q - pair * g.kb) * kBlockK;
                            const CUtensorMap *ma = &g.a[g.groups > 1 ? i.group : pair];
                            const uint32_t at = tc::smem_u32(smem) + s * S::stage, bt = at + S::a_bytes;
                            uint32_t bar = tc::smem_u32(&bars.full[s]);
                            if (CTAS == 1 || rank == 0) tc::mbar_arrive_expect_tx(&bars.full[s], S::stage * CTAS);
                            if constexpr (CTAS == 2) bar = map_to_cta(bar, 0);
                            if (g.a_mn) {
                                for (int j = 0; j < kTileM / 64; ++j) load_box<CTAS>(at + j * 8192, ma, bar, row + j * 64, k, pa);
                            } else {
                                load_box<CTAS>(at, ma, bar, k, row, pa);
                            }
                            if (g.dual) {
                                if constexpr (CTAS == 2) {
                                    load_box<CTAS>(bt, &g.b[rank], bar, k, ncol, pb);
                                } else {
                                    load_box<CTAS>(bt, &g.b[0], bar, k, ncol, pb);
                                    load_box<CTAS>(bt + 16384, &g.b[1], bar, k, ncol, pb);
                                }
                            } else if (g.b_mn) {
                                for (int j = 0; j < S::b_rows / 64; ++j) load_box<CTAS>(bt + j * 8192, &g.b[pair], bar, ncol + j * 64, k, pb);
                            } else {
                                for (int j = 0; j < S::b_rows / 128; ++j) load_box<CTAS>(bt + j * 16384, &g.b[pair], bar, k, ncol + j * 128, pb);
                            }
                        }
                    }
                }
            }
            // the products have read every stage before the CTA may leave
            for (uint32_t j = it > S::stages ? it - S::stages : 0; ok && j < it; ++j)
                ok = wait(&bars.empty[j % S::stages], (j / S::stages) & 1);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = tc::idesc_bf16_f32(kTileM * CTAS, kTileN, g.a_mn, g.b_mn);
            const uint32_t ka = g.a_mn ? 128 : 2, kbs = g.b_mn ? 128 : 2;   // 16 of K on, in 16-byte units
            uint32_t it = 0, n = 0;
            bool ok = true;
            for (int w = blockIdx.x / CTAS; ok && w < work; w += step) {
                const Item i = item_of<CTAS>(g, w);
                for (int c0 = i.q0; ok && c0 < i.q1; c0 += chunk, ++n) {
                    const int c1 = min(c0 + chunk, i.q1);
                    if (c1 < c0) break;
                    const uint32_t buf = n & 1;
                    if (n >= 2 && !wait(&bars.tmem_empty[buf], ((n >> 1) - 1) & 1)) { ok = false; break; }
                    tc::tc_fence_after();
                    const uint32_t d = tmem + buf * kTileN;
                    const int count = (c1 - c0) * g.terms;
                    for (int q = 0; q < count; ++q, ++it) {
                        const uint32_t s = it % S::stages;
                        if (!wait(&bars.full[s], (it / S::stages) & 1)) { ok = false; break; }
                        tc::tc_fence_after();
                        const uint32_t at = tc::smem_u32(smem) + s * S::stage;
                        const uint64_t da = tc::smem_desc_sw128(at, g.a_mn ? 8192 : 16, 1024);
                        const uint64_t db = tc::smem_desc_sw128(at + S::a_bytes, g.b_mn ? 8192 : 16, 1024);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) mma_bf16<CTAS>(d, da + kk * ka, db + kk * kbs, idesc, q > 0 || kk > 0);
                        commit<CTAS>(&bars.empty[s]);
                    }
                    if (ok) commit<CTAS>(&bars.tmem_full[buf]);
                }
            }
        }
    } else {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        uint8_t *box = smem + S::stages * S::stage + (warp - 2) * 4096;
        const uint32_t box_at = tc::smem_u32(box);
        const uint32_t release = CTAS == 2 ? map_to_cta(tc::smem_u32(&bars.tmem_empty[0]), 0) : tc::smem_u32(&bars.tmem_empty[0]);
        uint32_t n = 0;
        bool ok = true;
        // 32 columns of a row, packed, into the swizzled box (part 0 or 1 of its 64)
        auto put = [&](const float *v, int part) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const Raw<__nv_bfloat16, 8> r = pack<__nv_bfloat16, 8>(v + 8 * c);
                tc::sts_u4(box_at + tc::sw128_offset(lane, part * 4 + c), make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]));
            }
        };
        auto box_free = [&]() {
            if (lane == 0) tc::bulk_wait_group_read_all();
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
        for (int w = blockIdx.x / CTAS; ok && w < work; w += step) {
            const Item i = item_of<CTAS>(g, w);
            const int row0 = (i.m * CTAS + (int)rank) * kTileM + quarter * 32, row = row0 + lane;
            // the accumulator: 128 columns per warp; kUp: 64 of the gate's and 64 of the projection's
            constexpr int CW = kTileN / 2;
            float acc[PROMOTE ? CW : 1];
            uint32_t from = 0;
            auto column = [&](int j) {   // tensor memory column of the warp's column j
                return EPI == kUp ? (j < 64 ? half * 64 + j : 128 + half * 64 + j - 64) : half * 128 + j;
            };
            auto done = [&]() {
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    const uint32_t bar = release + (n & 1) * 8;
                    if constexpr (CTAS == 2)
                        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
                    else
                        tc::mbar_arrive(&bars.tmem_empty[n & 1]);
                }
                ++n;
            };
            if constexpr (PROMOTE) {
                for (int c0 = i.q0; c0 < i.q1; c0 += chunk) {
                    ok = __all_sync(0xffffffffu, wait(&bars.tmem_full[n & 1], (n >> 1) & 1));
                    if (!ok) break;
                    tc::tc_fence_after();
                    const uint32_t d = tmem + (n & 1) * kTileN + lanes;
#pragma unroll
                    for (int j = 0; j < CW; j += 32) {
                        uint32_t v[32];
                        tc::tmem_ld32(d + column(j), v);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) acc[j + e] = c0 == i.q0 ? __uint_as_float(v[e]) : acc[j + e] + __uint_as_float(v[e]);
                    }
                    done();
                }
            } else {
                ok = __all_sync(0xffffffffu, wait(&bars.tmem_full[n & 1], (n >> 1) & 1));
                tc::tc_fence_after();
                from = tmem + (n & 1) * kTileN + lanes;
            }
            if (!ok) break;
            auto get = [&](int j, float *v) {   // columns j .. j + 31 of the warp's
                if constexpr (PROMOTE) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = acc[j + e];
                } else {
                    tc::tmem_ld32(from + column(j), reinterpret_cast<uint32_t *>(v));
                    tc::tmem_wait_ld();
                }
            };
            const bool in = row < g.M;
            if (g.splits > 1) {
#pragma unroll
                for (int j = 0; j < CW; j += 32) {
                    float v[32];
                    get(j, v);
                    const int which = EPI == kUp ? j / 64 : i.group;
                    const int col = EPI == kUp ? i.n * 128 + half * 64 + j % 64 : i.n * kTileN + half * 128 + j;
                    if (in && col < g.N)
                        store32<float>(g.partial + (((long long)i.split * (EPI == kUp ? 2 : g.groups) + which) * g.M + row) * g.ld_part + col,
                                       v, (int)g.ld_part - col, true);
                }
            } else if constexpr (EPI == kUp) {
                const int col = i.n * 128 + half * 64;
                if (g.gate) {
#pragma unroll
                    for (int o = 0; o < 2; ++o) {
                        T *dst = static_cast<T *>(o ? g.up : g.gate);
                        if (!PROMOTE && g.tma_out) box_free();
#pragma unroll
                        for (int j = 0; j < 64; j += 32) {
                            float v[32];
                            get(64 * o + j, v);
                            if (!PROMOTE && g.tma_out) put(v, j / 32);
                            else if (in && col + j < g.N) store32<T>(dst + row * g.ld_io + col + j, v, g.N - col - j, g.vec_io);
                        }
                        if (!PROMOTE && g.tma_out) box_out(&g.c[1 + o], col, row0, g.N, g.M);
                    }
                }
                if (!PROMOTE) box_free();
#pragma unroll
                for (int j = 0; j < 64; j += 32) {
                    float a[32], b[32];
                    get(j, a);
                    get(64 + j, b);
#pragma unroll
                    for (int e = 0; e < 32; ++e) a[e] = act_times(a[e], b[e], g.act);
                    if constexpr (!PROMOTE) {
                        put(a, j / 32);
                    } else if (in && col + j < g.N) {
#pragma unroll
                        for (int p = 0; p < 3; ++p) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                float s[3];
                                split3(a[e], s);
                                b[e] = s[p];
                            }
                            store32<__nv_bfloat16>(g.planes[0] + p * g.plane_stride + row * g.ld_plane + col + j, b, (int)g.ld_plane - col - j, true);
                        }
                    }
                }
                if (!PROMOTE) box_out(&g.c[0], col, row0, g.N, g.M);
            } else if constexpr (EPI == kBack) {
                const T *gate = static_cast<const T *>(g.gate), *up = static_cast<const T *>(g.up);
#pragma unroll 1
                for (int part = 0; part < 2; ++part) {
                    const int col = i.n * kTileN + half * 128 + part * 64;
                    uint32_t pk[PROMOTE ? 1 : 3][32];
#pragma unroll
                    for (int j = 0; j < 64; j += 32) {
                        float d[32], x[32], u[32];
                        const int live = in ? g.N - col - j : 0;
                        load32<T>(gate + (live > 0 ? row * g.ld_io + col + j : 0), x, live, g.vec_io);
                        load32<T>(up + (live > 0 ? row * g.ld_io + col + j : 0), u, live, g.vec_io);
                        if constexpr (PROMOTE) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) d[e] = part ? acc[64 + j + e] : acc[j + e];
                        } else {
                            get(part * 64 + j, d);
                        }
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            float dg, du, h;
                            act_back(d[e], x[e], u[e], g.act, dg, du, h);
                            d[e] = dg, u[e] = du, x[e] = h;
                        }
                        if constexpr (!PROMOTE) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                pk[0][j / 2 + e] = tc::pack_bf16x2(d[2 * e], d[2 * e + 1]);
                                pk[1][j / 2 + e] = tc::pack_bf16x2(u[2 * e], u[2 * e + 1]);
                                pk[2][j / 2 + e] = tc::pack_bf16x2(x[2 * e], x[2 * e + 1]);
                            }
                        } else if (live > 0) {
#pragma unroll
                            for (int o = 0; o < 3; ++o) {
#pragma unroll
                                for (int p = 0; p < 3; ++p) {
                                    float v[32];
#pragma unroll
                                    for (int e = 0; e < 32; ++e) {
                                        float s[3];
                                        split3(o == 0 ? d[e] : o == 1 ? u[e] : x[e], s);
                                        v[e] = s[p];
                                    }
                                    store32<__nv_bfloat16>(g.planes[o] + p * g.plane_stride + row * g.ld_plane + col + j, v,
                                                           (int)g.ld_plane - col - j, true);
                                }
                            }
                        }
                    }
                    if constexpr (!PROMOTE) {
#pragma unroll
                        for (int o = 0; o < 3; ++o) {
                            box_free();
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                tc::sts_u4(box_at + tc::sw128_offset(lane, c),
                                           make_uint4(pk[o][4 * c], pk[o][4 * c + 1], pk[o][4 * c + 2], pk[o][4 * c + 3]));
                            box_out(&g.c[o], col, row0, g.N, g.M);
                        }
                    }
                }
            } else {
                const int col = i.n * kTileN + half * 128;
                T *out = static_cast<T *>(g.out[i.group]);
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    if (!PROMOTE && g.tma_out) box_free();
#pragma unroll
                    for (int j = 0; j < 64; j += 32) {
                        float v[32];
                        get(part * 64 + j, v);
                        const int at = col + part * 64 + j;
                        if (!PROMOTE && g.tma_out) put(v, j / 32);
                        else if (in && at < g.N) store32<T>(out + row * g.ld_out + at, v, g.N - at, g.vec_out);
                    }
                    if (!PROMOTE && g.tma_out) box_out(&g.c[i.group], col + part * 64, row0, g.N, g.M);
                }
            }
            if constexpr (!PROMOTE) done();
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
    if (warp == 1) tmem_free_all<CTAS>(tmem);
}

template <int EPI, typename T, int CTAS>
cudaError_t launch_gemm(const GemmArgs &g, int grid, cudaStream_t s) {
    using S = Shape<CTAS>;
    cudaError_t e = cudaFuncSetAttribute(ffn_gemm_kernel<EPI, T, CTAS>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CTAS, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CTAS == 2 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, ffn_gemm_kernel<EPI, T, CTAS>, g);
}

// The instantiations, one translation unit each (ffn_gemm_*.cu).
cudaError_t launch_up(const GemmArgs &g, bool f32, int ctas, int grid, cudaStream_t s);
cudaError_t launch_back(const GemmArgs &g, bool f32, int ctas, int grid, cudaStream_t s);
cudaError_t launch_plain(const GemmArgs &g, bool f32, int ctas, int grid, cudaStream_t s);

#define GDN_FFN_LAUNCHER(NAME, EPI)                                                                          \
    cudaError_t NAME(const GemmArgs &g, bool f32, int ctas, int grid, cudaStream_t s) {                      \
        if (f32) return ctas == 2 ? launch_gemm<EPI, float, 2>(g, grid, s) : launch_gemm<EPI, float, 1>(g, grid, s); \
        return ctas == 2 ? launch_gemm<EPI, __nv_bfloat16, 2>(g, grid, s) : launch_gemm<EPI, __nv_bfloat16, 1>(g, grid, s); \
    }

}  // namespace ffn
}  // namespace gdn
