// The gated feed-forward block, forward and backward:
//
//     g = x Wg^T,  u = x Wu^T,  h = act(g) u,  y = h Wd^T,
//     dh = dy Wd,  dg = dh u act'(g),  du = dh act(g),
//     dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  dWd = dy^T h.
//
// Forward two products, the first with both projections, the activation and the
// product h in one kernel; backward one with dg, du and h in its epilogue, and the
// four gradients' in one launch (ffn_gemm.cuh); few tokens forward by ffn_few.cu.
// Operands that TMA cannot read in place (fp32, or rows
// that are not 16-byte aligned) are first laid out as bf16 planes in the workspace.
// Where a product has too few tiles to fill the GPU its sum over K is split: the
// parts leave as fp32 and a second kernel adds them in order and applies the
// epilogue, so the result does not depend on the launch.
//
// In bf16 what lies between the products (h; backward dg, du and h) is rounded to bf16, the
// type in which the tensor cores read it: as fp32 planes the second product would be six.
// Outputs are 2.35e-3 from 64 bits (rms, relative), 1.66e-3 of which are their own rounding.
#include <algorithm>
#include <mutex>

#include "ffn_few.cuh"
#include "ffn_gemm.cuh"

namespace gdn {
namespace ffn {
namespace {

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                             const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
    static std::once_flag once;
    static EncodeFn fn = nullptr;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(ptr);
        cudaGetLastError();
    });
    return fn;
}

// bf16 planes in memory: [planes][rows][ld], `cols` of each row valid.
struct Mat {
    const void *p;
    long long rows, cols, ld, plane;
    int planes;
};

thread_local int debug_checks = 0;   // gdn_gated_ffn_debug

gdn_status failed(const char *where, cudaError_t e) {
    set_error_detail(where, e);
    return GDN_ERR_CUDA;
}

// box_cols: 64, or 32 for the outputs of kBack (128 or 64 bytes a row, swizzled as wide).
// Records why when it fails.
bool encode(CUtensorMap *map, const Mat &m, int box_rows, int box_cols = 64) {
    const EncodeFn fn = encode_fn();
    if (!fn) {
        set_error_detail("driver entry point cuTensorMapEncodeTiled", cudaErrorNotSupported);
        return false;
    }
    const long long ld = m.rows > 1 ? m.ld : (m.cols + 7) / 8 * 8;
    const cuuint64_t dims[3] = {(cuuint64_t)m.cols, (cuuint64_t)m.rows, (cuuint64_t)m.planes};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(m.planes > 1 ? m.plane : ld * m.rows) * 2};
    const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1}, es[3] = {1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(m.p), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) set_error_detail("encode tensor map", cudaErrorInvalidValue, (int)r);
    return r == CUDA_SUCCESS;
}

long long pad8(long long n) { return (n + 7) / 8 * 8; }

// ---------------------------------------------------------------- laying out
struct StageItem {
    const void *src;
    __nv_bfloat16 *dst;
    long long rows, cols, ld, ld_dst, plane;
};
struct StageArgs {
    StageItem item[5];
};
// Rows of T as bf16 planes (one for bf16, three for fp32): eight columns a thread.
template <typename T>
__global__ void __launch_bounds__(256) ffn_stage_kernel(const StageArgs a) {
    grid_dependency_wait();
    const StageItem &s = a.item[blockIdx.y];
    const long long per = s.ld_dst / 8, total = s.rows * per;
    const T *src = static_cast<const T *>(s.src);
    const bool vec = (reinterpret_cast<uintptr_t>(s.src) & 15) == 0 && s.ld % (16 / (int)sizeof(T)) == 0;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const long long r = i / per, c = (i - r * per) * 8;
        const T *at = src + r * s.ld + c;
        float v[8];
        if (vec && c + 8 <= s.cols) unpack<T, 8>(load_raw<T, 8>(at), v);
        else unpack<T, 8>(load_some<T, 8>(at, (int)(s.cols - c < 8 ? s.cols - c : 8)), v);
        __nv_bfloat16 *dst = s.dst + r * s.ld_dst + c;
        if constexpr (sizeof(T) == 2) {
            store_raw<__nv_bfloat16, 8>(dst, pack<__nv_bfloat16, 8>(v));
        } else {
            float p[3][8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float t[3];
                split3(v[e], t);
                p[0][e] = t[0], p[1][e] = t[1], p[2][e] = t[2];
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) store_raw<__nv_bfloat16, 8>(dst + k * s.plane, pack<__nv_bfloat16, 8>(p[k]));
        }
    }
}

// ------------------------------------------------------ adding a split's parts
struct FinishGroup {
    const float *partial;
    int splits, vec;          // vec: rows of what is read and written beside it in vectors of four
    long long M, N, ld_part, ld_out;
    void *out;
};
struct FinishArgs {
    FinishGroup group[kMaxGroups];
    int act;
    __nv_bfloat16 *planes[3];
    long long ld_plane, plane_stride;
    void *gate, *up;
};
// Four columns a thread; blockIdx.y: the product.
template <int EPI, typename T>
__global__ void __launch_bounds__(256) ffn_finish_kernel(const FinishArgs f) {
    grid_dependency_wait();
    const FinishGroup &a = f.group[blockIdx.y];
    const long long per = (a.N + 3) / 4, total = a.partial ? a.M * per : 0, matrix = a.M * a.ld_part;
    auto sum = [&](long long at, float (&v)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = 0.f;
        for (int s = 0; s < a.splits; ++s) {
            const float4 p = *reinterpret_cast<const float4 *>(a.partial + s * (EPI == kUp ? 2 : 1) * matrix + at);
            v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
        }
    };
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const long long r = i / per, c = (i - r * per) * 4;
        const int live = (int)(a.N - c < 4 ? a.N - c : 4);
        float v[4], w[4];
        sum(r * a.ld_part + c, v);
        // planes have rows of a multiple of eight, so four columns are always there
        auto planes = [&](int o, const float *x) {
            __nv_bfloat16 *to = f.planes[o] + r * f.ld_plane + c;
            if constexpr (sizeof(T) == 2) {
                store_raw<__nv_bfloat16, 4>(to, pack<__nv_bfloat16, 4>(x));
            } else {
                float s[3][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float t[3];
                    split3(x[e], t);
                    s[0][e] = t[0], s[1][e] = t[1], s[2][e] = t[2];
                }
#pragma unroll
                for (int k = 0; k < 3; ++k) store_raw<__nv_bfloat16, 4>(to + k * f.plane_stride, pack<__nv_bfloat16, 4>(s[k]));
            }
        };
        auto load4 = [&](const void *p, float (&x)[4]) {
            const T *at = static_cast<const T *>(p) + r * a.N + c;
            unpack<T, 4>(a.vec ? load_raw<T, 4>(at) : load_some<T, 4>(at, live), x);
        };
        auto store4 = [&](void *p, long long ld, const float *x) {
            T *at = static_cast<T *>(p) + r * ld + c;
            if (a.vec) store_raw<T, 4>(at, pack<T, 4>(x));
            else store_some<T, 4>(at, x, live);
        };
        if constexpr (EPI == kUp) {
            sum(matrix + r * a.ld_part + c, w);
            if (f.gate) {
                store4(f.gate, a.N, v);
                store4(f.up, a.N, w);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = act_times(v[e], w[e], f.act);
            planes(0, v);
        } else if constexpr (EPI == kBack) {
            float g[4], u[4];
            load4(f.gate, g);
            load4(f.up, u);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float dg, du, h;
                act_back(v[e], g[e], u[e], f.act, dg, du, h);
                v[e] = dg, w[e] = du, g[e] = h;
            }
            planes(0, v);
            planes(1, w);
            planes(2, g);
        } else {
            store4(a.out, a.ld_out, v);
        }
    }
}

// ------------------------------------------------------------------- the work
struct Problem {
    long long M, D, F, O;
    bool f32;
    int act, planes, terms;
};
struct Product {
    long long M, N, k;        // k: of one pair
    int pairs;
    Mat a[2], b[2];
    bool a_mn, b_mn;
    void *out;                // contiguous
};
struct Plan {
    int tile, splits[kMaxGroups], mt[kMaxGroups], nt[kMaxGroups], kb[kMaxGroups];
    int order[kMaxGroups], ahead, first, rest, ratio;   // ahead: how many of `order` make up `first`
    size_t part_bytes[kMaxGroups], bytes;
};
// One launch: products that share an epilogue (those without an output are planned
// for, so that a result does not depend on which others are wanted, and left out).
struct Batch {
    int epi, n;
    Product p[kMaxGroups];
    Mat planes[3];            // kUp, kBack: outputs
    void *gate, *up;
    Plan plan;
};

// Tiles of 128 columns: the rows of A that a stage holds, and the stages that then fit.
int rows_of_a(const Batch &b) {
    const bool few = b.n == 1 && !b.p[0].a_mn;
    return few && b.p[0].M <= 32 ? 32 : few && b.p[0].M <= 64 ? 64 : kTileM;
}
int small_stages(int a_rows) { return a_rows == 32 ? 5 : a_rows == 64 ? 4 : 3; }

int blocks(long long k) { return (int)((k + kBlockK - 1) / kBlockK); }
long long up_div(long long a, long long b) { return (a + b - 1) / b; }

// Blocks of K that one sum may have.  Whatever an addition in tensor memory leaves over is
// cut, not rounded: bf16 sums of terms of one sign come out 1.1e-7 of themselves too small
// for each addition of 16 products, and so 7e-3 at 2^20 of K in one sum and 0.11 at 2^24.
// Longer sums are cut into parts (added in fp32, rounded to nearest): at most 8192
// additions, 9e-4, a quarter of what rounding to bf16 may be off.
constexpr long long kLongest = 2048;

// Tile shape and parts of a batch, by a model in clocks (1.9 a ns).  A block of K takes a pair
// or a CTA of 256 columns 512 of the tensor pipe for each term, one of 128 columns 256, or its
// operands' way to the SM longer (a pair 546, a CTA of 256 columns 820, one of 128 columns 546,
// two of them on an SM 1092).
// A tile takes at least its epilogue; a launch 4000 to 7000 to fill and drain; the operands
// come at 3500 bytes a clock, or what the CTAs at work can have in flight; parts cost another
// launch and its traffic.  For fp32 the backward pass's first product may leave as one part:
// its epilogue with three outputs of three planes takes 57 us a tile (8192 x 256 x 2048: 230 us
// in all, 134 with the second kernel, which takes its rows in order), so where K is short.
Plan plan_batch(const Batch &b, const Problem &pr) {
    Plan best = {};
    double best_cost = 1e300;
    const int sms = device_sm_count();
    const int which = b.epi == kUp ? 2 : 1;
    long long kmax = 1;
    double bytes = 0;
    const double beside = (double)b.p[0].M * b.p[0].N * (pr.f32 ? 26 : 10);   // kBack: gate and up in, three outputs
    for (int i = 0; i < b.n; ++i) {
        const Product &p = b.p[i];
        kmax = std::max<long long>(kmax, (long long)blocks(p.k) * p.pairs);
        bytes += 2.0 * pr.planes * p.k * p.pairs * (p.M + (double)p.N * which) + 4.0 * p.M * p.N;
    }
    static const int parts[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32};
    for (int tile = 0; tile < 3; ++tile) {
        const int ctas = tile == kPair ? 2 : 1, bn = tile == kSmall ? 128 : 256, cols = b.epi == kUp ? bn / 2 : bn;
        const int P = tile == kPair ? sms / 2 : tile == kWide ? sms : 2 * sms;
        const double direct = (pr.f32 ? (b.epi == kBack ? 108000 : b.epi == kUp ? 32000 : 12000)
                                      : (b.epi == kBack ? 25000 : b.epi == kUp ? 7000 : 5000) * (tile == kSmall ? 1.6 : 1.0));
        long long last = 0;
        for (int want : parts) {
            const long long target = up_div(kmax, want);
            if (target == last) continue;
            last = target;
            for (int via = 0; via < (pr.f32 && b.epi == kBack ? 2 : 1); ++via) {
                Plan c = {};
                c.tile = tile;
                double len[kMaxGroups], longest = 0;
                long long units[kMaxGroups], all = 0;
                bool split = false, chosen = false;   // chosen: not for the sums' length alone
                double part = 0;
                for (int i = 0; i < b.n; ++i) {
                    const Product &p = b.p[i];
                    const long long q = (long long)blocks(p.k) * p.pairs, least = up_div(q, kLongest);
                    c.kb[i] = blocks(p.k);
                    c.mt[i] = (int)up_div(p.M, kTileM * ctas), c.nt[i] = (int)up_div(p.N, cols);
                    c.splits[i] = (int)std::max(up_div(q, target), least);
                    chosen |= c.splits[i] > least || via;
                    units[i] = (long long)c.mt[i] * c.nt[i] * c.splits[i];
                    all += units[i];
                    len[i] = (double)q / c.splits[i];
                    longest = std::max(longest, len[i]);
                    c.part_bytes[i] = c.splits[i] > 1 || via ? (size_t)c.splits[i] * which * p.M * ((p.N + 3) / 4 * 4) * 4 : 0;
                    split |= c.splits[i] > 1 || via, part += c.part_bytes[i];
                }
                if (chosen && (part > 1e9 || (want > 1 && all > 8ll * P))) break;
                // the longest first
                int n = 0;
                double la = 0, lb = 0;
                for (int i = 0; i < b.n; ++i)
                    if (len[i] >= 0.75 * longest) c.order[n++] = i, c.first += (int)units[i], la = std::max(la, len[i]);
                c.ahead = n;
                for (int i = 0; i < b.n; ++i)
                    if (len[i] < 0.75 * longest) c.order[n++] = i, c.rest += (int)units[i], lb = std::max(lb, len[i]);
                c.ratio = lb > 0 ? std::max(1, (int)(la / lb + 0.5)) : 1;
                // of a block of K: the tensor pipe's, or its bytes at 60 a clock and SM (rows that
                // do not exist are not read)
                const double share = tile == kSmall && all > sms ? 2 : 1, rows = std::min(1.0, (double)b.p[0].M / kTileM);
                const double clock = std::max(tile == kSmall ? 256 * share : 512, (16384 * (b.p[0].a_mn ? 1 : rows) + 128.0 * bn / ctas) / 60 * share);
                const double epi = split ? 12000 : direct;
                auto unit = [&](double l) { return std::max(l * pr.terms * clock, epi) + 300; };
                const int extra = c.first % P, behind = extra ? P - extra : 0;
                double span = 0;
                for (int p : {0, extra, P - 1}) {
                    const long long a = up_div(std::max(c.first - p, 0), P), base = (long long)c.ratio * behind;
                    long long r = up_div(std::max<long long>(c.rest - base - p, 0), P);
                    if (extra && p >= extra) r += std::min<long long>(c.ratio, up_div(std::max(c.rest - (p - extra), 0), behind));
                    span = std::max(span, a * unit(la) + r * unit(lb));
                }
                const double in_flight = (tile == kPair ? 6 * 16384 : tile == kWide ? 4 * 32768 : 3 * 16384) / 1800.0;
                const double active = (double)std::min<long long>(all, P) * ctas;
                double cost = std::max(span, bytes / std::min(3500.0, active * in_flight)) + (tile == kPair ? 7000 : tile == kWide ? 5500 : 4000);
                if (split) cost += 6000 + (part * 2 + (b.epi == kBack ? beside : 0)) / 3500;
                if (cost < best_cost * 0.98) {
                    best_cost = cost;
                    best = c;
                }
            }
        }
    }
    for (int i = 0; i < b.n; ++i) best.bytes += (best.part_bytes[i] + 255) / 256 * 256;
    return best;
}

struct Carve {
    char *base;
    size_t at;
    void *take(size_t bytes) {
        void *p = base ? base + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return p;
    }
};

bool tma_ok(const void *p, long long rows, long long ld) {
    return aligned16(p) && (rows <= 1 || ld % 8 == 0);
}
// The operand as TMA reads it: in place where it can, else planes in the workspace.
Mat operand(Carve &c, StageArgs &st, int &n, const Problem &pr, const void *p, long long rows, long long cols, long long ld) {
    Mat m = {p, rows, cols, ld, 0, pr.planes};
    if (!pr.f32 && tma_ok(p, rows, ld)) return m;
    m.ld = pad8(cols);
    m.plane = rows * m.ld;
    m.p = c.take((size_t)m.plane * pr.planes * 2);
    st.item[n++] = {p, static_cast<__nv_bfloat16 *>(const_cast<void *>(m.p)), rows, cols, ld, m.ld, m.plane};
    return m;
}
Mat intermediate(Carve &c, const Problem &pr, long long rows, long long cols) {
    Mat m = {nullptr, rows, cols, pad8(cols), 0, pr.planes};
    m.plane = rows * m.ld;
    m.p = c.take((size_t)m.plane * pr.planes * 2);
    return m;
}

cudaError_t run_stage(const Problem &pr, const StageArgs &st, int n, cudaStream_t s) {
    if (n == 0) return cudaSuccess;
    long long most = 0;
    for (int i = 0; i < n; ++i) most = std::max(most, st.item[i].rows * st.item[i].ld_dst / 8);
    const int grid = (int)std::min<long long>((most + 255) / 256, 8ll * device_sm_count());
    return pr.f32 ? launch_dependent(ffn_stage_kernel<float>, dim3(grid, n), dim3(256), 0, s, st)
                  : launch_dependent(ffn_stage_kernel<__nv_bfloat16>, dim3(grid, n), dim3(256), 0, s, st);
}

template <int EPI>
cudaError_t run_finish(const Problem &pr, const FinishArgs &f, int n, cudaStream_t s) {
    long long most = 0;
    for (int i = 0; i < n; ++i) most = std::max(most, f.group[i].M * ((f.group[i].N + 3) / 4));
    const int grid = (int)std::min<long long>((most + 255) / 256, 8ll * device_sm_count());
    return pr.f32 ? launch_dependent(ffn_finish_kernel<EPI, float>, dim3(grid, n), dim3(256), 0, s, f)
                  : launch_dependent(ffn_finish_kernel<EPI, __nv_bfloat16>, dim3(grid, n), dim3(256), 0, s, f);
}

gdn_status run_batch(const Batch &b, const Problem &pr, char *partial, int *err, cudaStream_t s, const char *where) {
    const Plan &pl = b.plan;
    GemmArgs g = {};
    const int e = pr.f32 ? 4 : 2;
    auto vec = [&](const void *q, long long ld) { return aligned16(q) && ld * e % 16 == 0; };
    g.dual = b.epi == kUp, g.ratio = pl.ratio;
    g.terms = pr.terms, g.act = pr.act, g.err = err;
    const int a_rows = rows_of_a(b);
    g.a_rows = a_rows, g.stages = small_stages(a_rows);
    g.probe = (debug_checks & GDN_DEBUG_TIMEOUT_PROBE) != 0;
    FinishArgs f = {};
    int na = 0, nb = 0, nc = 0;
    bool split = false;
    for (int k = 0; k < b.n; ++k) {
        const int i = pl.order[k];
        const Product &p = b.p[i];
        if (b.epi == kPlain && !p.out) continue;
        Group &q = g.group[g.groups];
        q.M = (int)p.M, q.N = (int)p.N, q.mt = pl.mt[i], q.nt = pl.nt[i], q.kb = pl.kb[i], q.pairs = p.pairs, q.splits = pl.splits[i];
        q.a = na, q.b = nb, q.c = nc, q.a_mn = p.a_mn, q.b_mn = p.b_mn;
        q.out = p.out, q.ld_out = p.N, q.vec_out = vec(p.out, p.N);
        q.partial = pl.part_bytes[i] ? reinterpret_cast<float *>(partial) : nullptr, q.ld_part = (p.N + 3) / 4 * 4;
        partial += (pl.part_bytes[i] + 255) / 256 * 256;
        (k < pl.ahead ? g.first : g.rest) += q.mt * q.nt * q.splits;
        const int b_maps = g.dual ? 2 : p.pairs;
        if (na + p.pairs > kMaxGroups + 1 || nb + b_maps > kMaxGroups + 1) return failed(where, cudaErrorInvalidValue);
        for (int j = 0; j < p.pairs; ++j)
            if (!encode(&g.a[na++], p.a[j], p.a_mn ? 64 : pl.tile == kSmall ? a_rows : kTileM)) return GDN_ERR_CUDA;
        for (int j = 0; j < b_maps; ++j)
            if (!encode(&g.b[nb++], p.b[j], p.b_mn || (g.dual && pl.tile == kSmall) ? 64 : 128)) return GDN_ERR_CUDA;
        if (b.epi == kPlain && !pr.f32 && !q.partial && q.vec_out) {
            q.tma_out = 1;
            if (!encode(&g.c[nc++], Mat{p.out, p.M, p.N, p.N, 0, 1}, 32)) return GDN_ERR_CUDA;
        }
        split |= q.partial != nullptr;
        const bool four = p.N % 4 == 0 && (b.epi == kPlain ? aligned16(p.out) : aligned16(b.gate) && aligned16(b.up));
        f.group[g.groups++] = {q.partial, q.splits, four, p.M, p.N, q.ld_part, q.ld_out, p.out};
    }
    if (g.groups == 0) return GDN_OK;
    if (b.epi != kPlain) {
        const int n = b.epi == kUp ? 1 : 3;
        for (int i = 0; i < n; ++i) {
            g.planes[i] = static_cast<__nv_bfloat16 *>(const_cast<void *>(b.planes[i].p));
            if (!pr.f32 && !encode(&g.c[i], b.planes[i], 32, b.epi == kBack ? 32 : 64)) return GDN_ERR_CUDA;
        }
        g.ld_plane = b.planes[0].ld, g.plane_stride = b.planes[0].plane;
        g.gate = b.gate, g.up = b.up;
        const Product &p = b.p[0];
        g.vec_io = vec(b.gate, p.N) && vec(b.up, p.N);
        if (b.epi == kUp && b.gate && !pr.f32 && g.vec_io) {
            g.tma_io = 1;
            if (!encode(&g.io[0], Mat{b.gate, p.M, p.N, p.N, 0, 1}, 32) || !encode(&g.io[1], Mat{b.up, p.M, p.N, p.N, 0, 1}, 32))
                return GDN_ERR_CUDA;
        }
    }
    const int sms = device_sm_count(), workers = pl.tile == kPair ? sms / 2 : pl.tile == kWide ? sms : 2 * sms;
    const int grid = std::min(workers, g.first + g.rest) * (pl.tile == kPair ? 2 : 1);
    cudaError_t rc = b.epi == kUp ? launch_up(g, pr.f32, pl.tile, grid, s)
                     : b.epi == kBack ? launch_back(g, pr.f32, pl.tile, grid, s)
                                      : launch_plain(g, pr.f32, pl.tile, grid, s);
    if (rc != cudaSuccess) return failed(where, rc);
    if (!split) return GDN_OK;
    f.act = pr.act;
    for (int i = 0; i < 3; ++i) f.planes[i] = g.planes[i];
    f.ld_plane = g.ld_plane, f.plane_stride = g.plane_stride, f.gate = b.gate, f.up = b.up;
    rc = b.epi == kUp ? run_finish<kUp>(pr, f, g.groups, s) : b.epi == kBack ? run_finish<kBack>(pr, f, g.groups, s) : run_finish<kPlain>(pr, f, g.groups, s);
    return rc == cudaSuccess ? GDN_OK : failed(where, rc);
}

// ------------------------------------------------------------------ the passes
struct Pass {
    Problem pr;
    StageArgs stage;
    int n_stage, n;
    Batch batch[2];
    char *partial;
    size_t bytes;
};

void finish_plan(Pass &p, Carve &c) {
    size_t most = 0;
    for (int i = 0; i < p.n; ++i) {
        p.batch[i].plan = plan_batch(p.batch[i], p.pr);
        most = std::max(most, p.batch[i].plan.bytes);
    }
    p.partial = static_cast<char *>(c.take(most));
    p.bytes = std::max<size_t>(c.at, 16);
}

Problem problem_of(const gdn_ffn_desc &d) {
    Problem pr = {};
    pr.M = d.M, pr.D = d.D, pr.F = d.F, pr.O = d.D_out;
    pr.f32 = d.dtype == GDN_F32, pr.act = d.activation;
    pr.planes = pr.f32 ? 3 : 1, pr.terms = pr.f32 ? 6 : 1;
    return pr;
}

// Whether the forward products are those of ffn_few.cu.  From nine tokens in bf16 on they
// slow down with the weights' bytes, the tiles by their launches alone: 16 tokens, 4096 x 12288
// (302 MB) 66 us, tiles 57; 2048 x 6144 (75 MB) 23 and 27; 1024 x 4096 9.4 and 16.
// Rows that are not 16-byte aligned follow the same rule, although tiles lay them out in every
// call (9 and 16 tokens there, and on tiles): 4095 x 12287 191 and 227, 173; 4096 x 12287
// (w_down's rows alone) 138 and 170, 101; 2500 x 9001 (135 MB) 108 and 120, 87; only with
// w_down's alone aligned is it the other way round, 4095 x 12288 117 and 124, 135.  Of smaller
// weights no copies are made: 2047 x 6143 (75 MB) 73 and 91 (17 tokens, on tiles, 56).
// A warp adds up an eighth of K there, in one sum (kLongest).
bool few(const Problem &pr) {
    if (std::max(pr.D, pr.F) > 8 * kLongest * kBlockK) return false;
    const double weights = 2.0 * (2.0 * pr.F * pr.D + (double)pr.O * pr.F);
    return pr.M <= (pr.f32 ? kFewF32 : weights <= 134e6 ? kFewBf16 : kFewBf16 / 2);
}

gdn_status run_few(const gdn_ffn_desc &d, const Problem &pr, void *y, void *gate, void *up, int32_t *status, void *workspace,
                   cudaStream_t s) {
    const int e = pr.f32 ? 4 : 2;
    auto vec = [&](const void *p, long long rows, long long ld) { return aligned16(p) && (rows <= 1 || ld * e % 16 == 0); };
    FewArgs a = {};
    a.x = d.x, a.x_stride = d.x_stride, a.w0 = d.w_gate, a.w1 = d.w_up, a.K = pr.D, a.M = (int)pr.M, a.rows = (int)pr.F, a.act = pr.act;
    a.out = workspace, a.out_ld = pad8(pr.F), a.gate = gate, a.up = up;
    FewArgs b = {};
    b.x = workspace, b.x_stride = pad8(pr.F), b.w0 = d.w_down, b.K = pr.F, b.M = a.M, b.rows = (int)pr.O, b.out = y, b.out_ld = pr.O;
    cudaError_t rc = status ? cudaMemsetAsync(status, 0, sizeof(int32_t), s) : cudaSuccess;
    const bool va = pr.D * e % 16 == 0 && vec(d.x, pr.M, d.x_stride) && aligned16(d.w_gate) && aligned16(d.w_up);
    const bool vb = pr.F * e % 16 == 0 && aligned16(d.w_down);
    if (rc == cudaSuccess) rc = launch_few(a, true, pr.f32, va, s);
    if (rc == cudaSuccess) rc = launch_few(b, false, pr.f32, vb, s);
    return rc == cudaSuccess ? GDN_OK : failed("launch gated_ffn_fwd", rc);
}

Pass plan_fwd(const gdn_ffn_desc &d, void *y, void *gate, void *up, void *workspace) {
    Pass p = {};
    const Problem pr = p.pr = problem_of(d);
    Carve c = {static_cast<char *>(workspace), 0};
    const Mat x = operand(c, p.stage, p.n_stage, pr, d.x, pr.M, pr.D, d.x_stride);
    const Mat wg = operand(c, p.stage, p.n_stage, pr, d.w_gate, pr.F, pr.D, pr.D);
    const Mat wu = operand(c, p.stage, p.n_stage, pr, d.w_up, pr.F, pr.D, pr.D);
    const Mat wd = operand(c, p.stage, p.n_stage, pr, d.w_down, pr.O, pr.F, pr.F);
    const Mat h = intermediate(c, pr, pr.M, pr.F);
    Batch &a = p.batch[0], &b = p.batch[1];
    p.n = 2;
    a.epi = kUp, a.n = 1, a.planes[0] = h, a.gate = gate, a.up = up;
    a.p[0].M = pr.M, a.p[0].N = pr.F, a.p[0].k = pr.D, a.p[0].pairs = 1, a.p[0].a[0] = x, a.p[0].b[0] = wg, a.p[0].b[1] = wu;
    b.epi = kPlain, b.n = 1;
    b.p[0].M = pr.M, b.p[0].N = pr.O, b.p[0].k = pr.F, b.p[0].pairs = 1, b.p[0].a[0] = h, b.p[0].b[0] = wd, b.p[0].out = y;
    finish_plan(p, c);
    return p;
}

Pass plan_bwd(const gdn_ffn_desc &d, const void *dy, int64_t dy_stride, const void *gate, const void *up, void *dx,
              void *dwg, void *dwu, void *dwd, void *workspace) {
    Pass p = {};
    const Problem pr = p.pr = problem_of(d);
    Carve c = {static_cast<char *>(workspace), 0};
    const Mat gy = operand(c, p.stage, p.n_stage, pr, dy, pr.M, pr.O, dy_stride);
    const Mat wd = operand(c, p.stage, p.n_stage, pr, d.w_down, pr.O, pr.F, pr.F);
    const Mat x = operand(c, p.stage, p.n_stage, pr, d.x, pr.M, pr.D, d.x_stride);
    const Mat wg = operand(c, p.stage, p.n_stage, pr, d.w_gate, pr.F, pr.D, pr.D);
    const Mat wu = operand(c, p.stage, p.n_stage, pr, d.w_up, pr.F, pr.D, pr.D);
    const Mat dg = intermediate(c, pr, pr.M, pr.F), du = intermediate(c, pr, pr.M, pr.F), h = intermediate(c, pr, pr.M, pr.F);
    Batch &a = p.batch[0], &b = p.batch[1];
    a.epi = kBack, a.n = 1, a.planes[0] = dg, a.planes[1] = du, a.planes[2] = h;
    a.gate = const_cast<void *>(gate), a.up = const_cast<void *>(up);
    a.p[0].M = pr.M, a.p[0].N = pr.F, a.p[0].k = pr.O, a.p[0].pairs = 1, a.p[0].a[0] = gy, a.p[0].b[0] = wd, a.p[0].b_mn = true;
    b.epi = kPlain;
    auto add = [&](long long M, long long N, long long k, const Mat &A, const Mat &B, bool a_mn, void *out) -> Product & {
        Product &q = b.p[b.n++];
        q.M = M, q.N = N, q.k = k, q.pairs = 1, q.a[0] = A, q.b[0] = B, q.a_mn = a_mn, q.b_mn = true, q.out = out;
        return q;
    };
    Product &q = add(pr.M, pr.D, pr.F, dg, wg, false, dx);
    q.pairs = 2, q.a[1] = du, q.b[1] = wu;
    add(pr.F, pr.D, pr.M, dg, x, true, dwg);
    add(pr.F, pr.D, pr.M, du, x, true, dwu);
    add(pr.O, pr.F, pr.M, gy, h, true, dwd);
    p.n = 2;
    finish_plan(p, c);
    return p;
}

gdn_status run_pass(const Pass &p, int32_t *status, cudaStream_t s, const char *where) {
    cudaError_t e = cudaSuccess;
    if (status) e = cudaMemsetAsync(status, 0, sizeof(int32_t), s);
    if (e == cudaSuccess && p.n) e = run_stage(p.pr, p.stage, p.n_stage, s);
    if (e != cudaSuccess) return failed(where, e);
    gdn_status st = GDN_OK;
    for (int i = 0; st == GDN_OK && i < p.n; ++i) st = run_batch(p.batch[i], p.pr, p.partial, status, s, where);
    return st;
}

bool elem_ok(const void *p, int dtype) { return (reinterpret_cast<uintptr_t>(p) & (dtype == GDN_F32 ? 3u : 1u)) == 0; }

// Rows and the distance between them: TMA strides have 40 bits of bytes.
bool span_ok(int64_t rows, int64_t stride) { return rows <= 1 || stride <= (1ll << 38) / rows; }
// Sizes: TMA coordinates and the work list count in 32 bits.
gdn_status desc_ok(const gdn_ffn_desc *d) {
    if (!d) return GDN_ERR_INVALID_ARG;
    if (d->dtype != GDN_BF16 && d->dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    if (d->activation != GDN_ACT_SILU && d->activation != GDN_ACT_GELU_TANH) return GDN_ERR_INVALID_ARG;
    if (d->M < 0 || d->D < 1 || d->F < 1 || d->D_out < 1 || (d->M > 1 && d->x_stride < d->D)) return GDN_ERR_INVALID_ARG;
    constexpr int64_t most = 1 << 24;
    if (d->M > most || d->D > most || d->F > most || d->D_out > most) return GDN_ERR_UNSUPPORTED;
    if (!span_ok(d->M, d->x_stride)) return GDN_ERR_UNSUPPORTED;
    const int64_t tensors[][2] = {{d->M, d->D}, {d->M, d->F}, {d->M, d->D_out}, {d->F, d->D}, {d->D_out, d->F}};
    for (const auto &t : tensors)
        if (t[0] * t[1] > (1ll << 38)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}
bool pointers_ok(const gdn_ffn_desc &d) {
    for (const void *p : {d.w_gate, d.w_up, d.w_down})
        if (!p || !elem_ok(p, d.dtype)) return false;
    return d.M == 0 || (d.x && elem_ok(d.x, d.dtype));
}

}  // namespace
}  // namespace ffn
}  // namespace gdn

extern "C" size_t gdn_gated_ffn_fwd_workspace_size(const gdn_ffn_desc *desc) {
    if (gdn::ffn::desc_ok(desc) != GDN_OK) return 0;
    if (desc->M == 0) return 16;
    const gdn::ffn::Problem pr = gdn::ffn::problem_of(*desc);
    if (gdn::ffn::few(pr)) return (size_t)pr.M * gdn::ffn::pad8(pr.F) * (pr.f32 ? 4 : 2);
    return gdn::ffn::plan_fwd(*desc, nullptr, nullptr, nullptr, nullptr).bytes;
}

extern "C" gdn_status gdn_gated_ffn_fwd(const gdn_ffn_desc *desc, void *y, void *gate, void *up, int32_t *device_status,
                                        void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    const gdn_status st = gdn::ffn::desc_ok(desc);
    if (st != GDN_OK) return st;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!gdn::ffn::pointers_ok(*desc) || !gdn::ffn::elem_ok(y, desc->dtype) || !gdn::ffn::elem_ok(gate, desc->dtype) ||
        !gdn::ffn::elem_ok(up, desc->dtype) || (gate == nullptr) != (up == nullptr))
        return GDN_ERR_INVALID_ARG;
    gdn::ffn::Pass p = {};
    if (desc->M > 0) {
        if (!y || !workspace || !gdn::aligned16(workspace)) return GDN_ERR_INVALID_ARG;
        const gdn::ffn::Problem pr = gdn::ffn::problem_of(*desc);
        if (gdn::ffn::few(pr)) {
            if (workspace_bytes < gdn_gated_ffn_fwd_workspace_size(desc)) return GDN_ERR_WORKSPACE;
            return gdn::ffn::run_few(*desc, pr, y, gate, up, device_status, workspace, s);
        }
        p = gdn::ffn::plan_fwd(*desc, y, gate, up, workspace);
        if (workspace_bytes < p.bytes) return GDN_ERR_WORKSPACE;
    }
    return gdn::ffn::run_pass(p, device_status, s, "launch gated_ffn_fwd");
}

extern "C" size_t gdn_gated_ffn_bwd_workspace_size(const gdn_ffn_desc *desc, const void *dy, int64_t dy_stride) {
    if (gdn::ffn::desc_ok(desc) != GDN_OK || (desc->M > 1 && dy_stride < desc->D_out) || !gdn::ffn::span_ok(desc->M, dy_stride)) return 0;
    if (desc->M == 0) return 16;
    return gdn::ffn::plan_bwd(*desc, dy, dy_stride, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr).bytes;
}

extern "C" gdn_status gdn_gated_ffn_bwd(const gdn_ffn_desc *desc, const void *dy, int64_t dy_stride, const void *gate,
                                        const void *up, void *dx, void *dw_gate, void *dw_up, void *dw_down,
                                        int32_t *device_status, void *workspace, size_t workspace_bytes,
                                        gdn_stream_t stream) {
    const gdn_status st = gdn::ffn::desc_ok(desc);
    if (st != GDN_OK) return st;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int dt = desc->dtype;
    if (!gdn::ffn::pointers_ok(*desc) || (desc->M > 1 && dy_stride < desc->D_out)) return GDN_ERR_INVALID_ARG;
    if (!gdn::ffn::span_ok(desc->M, dy_stride)) return GDN_ERR_UNSUPPORTED;
    for (const void *q : {(const void *)dx, (const void *)dw_gate, (const void *)dw_up, (const void *)dw_down, dy, gate, up})
        if (!gdn::ffn::elem_ok(q, dt)) return GDN_ERR_INVALID_ARG;
    gdn::ffn::Pass p = {};
    if (desc->M > 0) {
        if (!dy || !gate || !up || !workspace || !gdn::aligned16(workspace)) return GDN_ERR_INVALID_ARG;
        p = gdn::ffn::plan_bwd(*desc, dy, dy_stride, gate, up, dx, dw_gate, dw_up, dw_down, workspace);
        if (workspace_bytes < p.bytes) return GDN_ERR_WORKSPACE;
        if (!dx && !dw_gate && !dw_up && !dw_down) p.n = 0;
        return gdn::ffn::run_pass(p, device_status, s, "launch gated_ffn_bwd");
    }
    // no tokens: the weights' gradients are zero
    const size_t e = dt == GDN_F32 ? 4 : 2, n = (size_t)desc->F * desc->D * e;
    cudaError_t rc = cudaSuccess;
    if (dw_gate) rc = cudaMemsetAsync(dw_gate, 0, n, s);
    if (rc == cudaSuccess && dw_up) rc = cudaMemsetAsync(dw_up, 0, n, s);
    if (rc == cudaSuccess && dw_down) rc = cudaMemsetAsync(dw_down, 0, (size_t)desc->F * desc->D_out * e, s);
    if (rc != cudaSuccess) {
        gdn::set_error_detail("gated_ffn_bwd memset", rc);
        return GDN_ERR_CUDA;
    }
    return gdn::ffn::run_pass(p, device_status, s, "launch gated_ffn_bwd");
}

extern "C" gdn_status gdn_gated_ffn_plan_query(const gdn_ffn_desc *desc, int backward, const void *dy, int64_t dy_stride,
                                               gdn_ffn_plan_info *info) {
    using namespace gdn::ffn;
    const gdn_status st = desc_ok(desc);
    if (st != GDN_OK) return st;
    if (!info || (backward && desc->M > 1 && dy_stride < desc->D_out)) return GDN_ERR_INVALID_ARG;
    if (backward && !span_ok(desc->M, dy_stride)) return GDN_ERR_UNSUPPORTED;
    *info = {};
    if (desc->M == 0) return GDN_OK;
    info->path = !backward && few(problem_of(*desc)) ? GDN_FFN_FEW : GDN_FFN_TILES;
    if (info->path == GDN_FFN_FEW) return GDN_OK;
    const Pass p = backward ? plan_bwd(*desc, dy, dy_stride, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr)
                            : plan_fwd(*desc, nullptr, nullptr, nullptr, nullptr);
    for (int i = 0; i < p.n; ++i) {
        const Batch &b = p.batch[i];
        info->tile[i] = b.plan.tile, info->products[i] = b.n;
        info->a_rows[i] = b.plan.tile == kSmall ? rows_of_a(b) : kTileM;
        for (int k = 0; k < b.n; ++k) info->parts[i][k] = b.plan.part_bytes[k] ? b.plan.splits[k] : 0;
    }
    return GDN_OK;
}

extern "C" gdn_status gdn_gated_ffn_debug(int checks) {
    if (checks & ~GDN_DEBUG_TIMEOUT_PROBE) return GDN_ERR_INVALID_ARG;
    gdn::ffn::debug_checks = checks;
    return GDN_OK;
}
