// The gated feed-forward block, forward and backward:
//
//     g = x Wg^T,  u = x Wu^T,  h = act(g) u,  y = h Wd^T,
//     dh = dy Wd,  dg = dh u act'(g),  du = dh act(g),
//     dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  dWd = dy^T h.
//
// Forward two products, the first with both projections, the activation and the
// product h in one kernel; backward four, the first with dg, du and h in its
// epilogue (ffn_gemm.cuh).  Operands that TMA cannot read in place (fp32, or rows
// that are not 16-byte aligned) are first laid out as bf16 planes in the workspace.
// Where a product has too few tiles to fill the GPU its sum over K is split: the
// parts leave as fp32 and a second kernel adds them in order and applies the
// epilogue, so the result does not depend on the launch.
#include <algorithm>
#include <mutex>

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

bool encode(CUtensorMap *map, const Mat &m, int box_rows) {
    const EncodeFn fn = encode_fn();
    if (!fn) {
        set_error_detail("driver entry point cuTensorMapEncodeTiled", cudaErrorNotSupported);
        return false;
    }
    const long long ld = m.rows > 1 ? m.ld : (m.cols + 7) / 8 * 8;
    const cuuint64_t dims[3] = {(cuuint64_t)m.cols, (cuuint64_t)m.rows, (cuuint64_t)m.planes};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(m.planes > 1 ? m.plane : ld * m.rows) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, es[3] = {1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(m.p), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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
struct FinishArgs {
    const float *partial;
    int splits, which, groups, act;   // which: partial matrices per split
    long long M, N, ld_part;
    void *out[2];
    long long ld_out;
    __nv_bfloat16 *planes[3];
    long long ld_plane, plane_stride;
    int n_planes;
    void *gate, *up;
    long long ld_io;
};
__device__ __forceinline__ void store_planes(__nv_bfloat16 *p, long long stride, int n, const float *v, int live) {
    float s[3][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float t[3];
        split3(v[e], t);
        s[0][e] = n == 1 ? v[e] : t[0], s[1][e] = t[1], s[2][e] = t[2];
    }
    for (int k = 0; k < n; ++k) store_some<__nv_bfloat16, 4>(p + k * stride, s[k], live);
}
template <int EPI, typename T>
__global__ void __launch_bounds__(256) ffn_finish_kernel(const FinishArgs a) {
    grid_dependency_wait();
    const long long per = (a.N + 3) / 4, total = a.M * per * (EPI == kPlain ? a.groups : 1);
    const long long matrix = a.M * a.ld_part;
    auto sum = [&](long long at, float (&v)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = 0.f;
        for (int s = 0; s < a.splits; ++s) {
            const float4 p = *reinterpret_cast<const float4 *>(a.partial + s * a.which * matrix + at);
            v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
        }
    };
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const long long rr = i / per, c = (i - rr * per) * 4, grp = rr / a.M, r = rr - grp * a.M;
        const int live = (int)(a.N - c < 4 ? a.N - c : 4);
        float v[4], w[4];
        sum(grp * matrix + r * a.ld_part + c, v);
        if constexpr (EPI == kUp) {
            sum(matrix + r * a.ld_part + c, w);
            if (a.gate) {
                store_some<T, 4>(static_cast<T *>(a.gate) + r * a.ld_io + c, v, live);
                store_some<T, 4>(static_cast<T *>(a.up) + r * a.ld_io + c, w, live);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = act_times(v[e], w[e], a.act);
            store_planes(a.planes[0] + r * a.ld_plane + c, a.plane_stride, a.n_planes, v, live);
        } else if constexpr (EPI == kBack) {
            float g[4], u[4];
            unpack<T, 4>(load_some<T, 4>(static_cast<const T *>(a.gate) + r * a.ld_io + c, live), g);
            unpack<T, 4>(load_some<T, 4>(static_cast<const T *>(a.up) + r * a.ld_io + c, live), u);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float dg, du, h;
                act_back(v[e], g[e], u[e], a.act, dg, du, h);
                v[e] = dg, w[e] = du, g[e] = h;
            }
            store_planes(a.planes[0] + r * a.ld_plane + c, a.plane_stride, a.n_planes, v, live);
            store_planes(a.planes[1] + r * a.ld_plane + c, a.plane_stride, a.n_planes, w, live);
            store_planes(a.planes[2] + r * a.ld_plane + c, a.plane_stride, a.n_planes, g, live);
        } else {
            store_some<T, 4>(static_cast<T *>(a.out[grp]) + r * a.ld_out + c, v, live);
        }
    }
}

// ------------------------------------------------------------------- planning
struct Plan {
    int ctas, splits, mt, nt;
    long long ld_part;
    size_t partial_bytes;
};

// One product of M x N outputs per group (cols: a tile's columns of N) over kb
// blocks along K.  The model, in clocks: a block of K costs a CTA or pair 512 of the
// tensor pipe (single CTAs 640: they read twice as much of B), a tile 2500 for its
// first loads and its last epilogue, a split the second kernel and its traffic.
Plan plan_product(long long M, long long N, int cols, int groups, int which, long long kb, int terms) {
    Plan best = {};
    double best_cost = 1e300;
    const int sms = device_sm_count();
    for (int ctas = 2; ctas >= 1; --ctas) {
        const long long mt = (M + kTileM * ctas - 1) / (kTileM * ctas), nt = (N + cols - 1) / cols;
        const long long tiles = mt * nt * groups, slots = sms / ctas;
        for (int s = 1; s <= 32 && s <= kb; ++s) {
            const double part = (double)M * N * which * 4 * s;
            if (s > 1 && (tiles >= 2 * slots || part > 512e6)) break;
            const long long waves = (tiles * s + slots - 1) / slots;
            double cost = (double)waves * ((double)((kb + s - 1) / s) * terms * (ctas == 2 ? 512 : 640) + 2500);
            if (s > 1) cost += 6000 + part * 2 / 4000;   // 4000 bytes per clock to and from L2
            if (cost < best_cost * 0.97) {
                best_cost = cost;
                best.ctas = ctas, best.splits = s, best.mt = (int)mt, best.nt = (int)nt;
            }
        }
    }
    best.ld_part = (N + 3) / 4 * 4;
    best.partial_bytes = best.splits > 1 ? (size_t)best.splits * which * M * best.ld_part * 4 : 0;
    return best;
}

int blocks(long long k) { return (int)((k + kBlockK - 1) / kBlockK); }

struct Carve {
    char *base;
    size_t at;
    void *take(size_t bytes) {
        void *p = base ? base + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return p;
    }
};

// What a call needs besides its arguments: operands as TMA reads them, the
// intermediates, the parts of split sums.
struct Problem {
    long long M, D, F, O;
    bool f32;
    int act, planes, terms;
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

struct Product {
    int epi;
    long long M, N;
    int groups, pairs;
    Mat a[2], b[2];
    bool a_mn, b_mn, dual;
    Mat planes[3];            // kUp, kBack outputs
    void *out[2];
    long long ld_out;
    void *gate, *up;
    long long k;              // of one pair
};

Plan plan_of(const Product &p, const Problem &pr) {
    return plan_product(p.M, p.N, p.dual ? kTileN / 2 : kTileN, p.groups, p.dual ? 2 : p.groups,
                        (long long)blocks(p.k) * p.pairs, pr.terms);
}

template <int EPI>
cudaError_t run_finish(const Problem &pr, const FinishArgs &f, cudaStream_t s) {
    const long long total = f.M * ((f.N + 3) / 4) * f.groups;
    const int grid = (int)std::min<long long>((total + 255) / 256, 8ll * device_sm_count());
    return pr.f32 ? launch_dependent(ffn_finish_kernel<EPI, float>, dim3(grid), dim3(256), 0, s, f)
                  : launch_dependent(ffn_finish_kernel<EPI, __nv_bfloat16>, dim3(grid), dim3(256), 0, s, f);
}

cudaError_t run_product(const Product &p, const Problem &pr, float *partial, int *err, cudaStream_t s) {
    const Plan pl = plan_of(p, pr);
    GemmArgs g = {};
    const int e = pr.f32 ? 4 : 2;
    auto vec = [&](const void *q, long long ld) { return aligned16(q) && ld * e % 16 == 0; };
    const int nb = p.dual ? 2 : p.pairs, na = p.groups > 1 ? p.groups : p.pairs;
    for (int i = 0; i < na; ++i)
        if (!encode(&g.a[i], p.a[i], p.a_mn ? 64 : kTileM)) return cudaErrorInvalidValue;
    for (int i = 0; i < nb; ++i)
        if (!encode(&g.b[i], p.b[i], p.b_mn ? 64 : 128)) return cudaErrorInvalidValue;
    g.M = (int)p.M, g.N = (int)p.N, g.mt = pl.mt, g.nt = pl.nt, g.groups = p.groups;
    g.kb = blocks(p.k), g.pairs = p.pairs, g.splits = pl.splits, g.terms = pr.terms;
    g.a_mn = p.a_mn, g.b_mn = p.b_mn, g.dual = p.dual, g.act = pr.act;
    g.err = err;
    g.partial = partial, g.ld_part = pl.ld_part;
    g.gate = p.gate, g.up = p.up, g.ld_io = p.N;
    g.vec_io = vec(p.gate, g.ld_io) && vec(p.up, g.ld_io);
    for (int i = 0; i < 2; ++i) g.out[i] = p.out[i];
    g.ld_out = p.ld_out;
    g.vec_out = vec(p.out[0], p.ld_out) && (p.groups < 2 || vec(p.out[1], p.ld_out));
    const int np = p.epi == kUp ? 1 : p.epi == kBack ? 3 : 0;
    for (int i = 0; i < np; ++i) g.planes[i] = static_cast<__nv_bfloat16 *>(const_cast<void *>(p.planes[i].p));
    g.ld_plane = p.planes[0].ld, g.plane_stride = p.planes[0].plane;
    if (pl.splits == 1 && !pr.f32) {
        if (p.epi == kPlain) {
            g.tma_out = g.vec_out;
            for (int i = 0; g.tma_out && i < p.groups; ++i)
                if (!encode(&g.c[i], Mat{p.out[i], p.M, p.N, p.ld_out, 0, 1}, 32)) return cudaErrorInvalidValue;
        } else {
            for (int i = 0; i < np; ++i)
                if (!encode(&g.c[i], p.planes[i], 32)) return cudaErrorInvalidValue;
            if (p.epi == kUp && p.gate) {
                g.tma_out = g.vec_io;
                if (g.tma_out && (!encode(&g.c[1], Mat{p.gate, p.M, p.N, p.N, 0, 1}, 32) || !encode(&g.c[2], Mat{p.up, p.M, p.N, p.N, 0, 1}, 32)))
                    return cudaErrorInvalidValue;
            }
        }
    }
    const long long work = (long long)g.groups * g.mt * g.nt * g.splits;
    const int grid = (int)std::min<long long>(work, device_sm_count() / pl.ctas) * pl.ctas;
    cudaError_t rc = p.epi == kUp ? launch_up(g, pr.f32, pl.ctas, grid, s)
                     : p.epi == kBack ? launch_back(g, pr.f32, pl.ctas, grid, s)
                                      : launch_plain(g, pr.f32, pl.ctas, grid, s);
    if (rc != cudaSuccess || pl.splits == 1) return rc;
    FinishArgs f = {};
    f.partial = partial, f.splits = pl.splits, f.which = p.dual ? 2 : p.groups, f.groups = p.groups, f.act = pr.act;
    f.M = p.M, f.N = p.N, f.ld_part = pl.ld_part;
    for (int i = 0; i < 2; ++i) f.out[i] = p.out[i];
    f.ld_out = p.ld_out;
    for (int i = 0; i < 3; ++i) f.planes[i] = g.planes[i];
    f.ld_plane = g.ld_plane, f.plane_stride = g.plane_stride, f.n_planes = pr.planes;
    f.gate = p.gate, f.up = p.up, f.ld_io = g.ld_io;
    return p.epi == kUp ? run_finish<kUp>(pr, f, s) : p.epi == kBack ? run_finish<kBack>(pr, f, s) : run_finish<kPlain>(pr, f, s);
}

// ------------------------------------------------------------------ the passes
struct Pass {
    Problem pr;
    StageArgs stage;
    int n_stage;
    Product product[4];
    int n;
    float *partial;
    size_t bytes;
};

void finish_plan(Pass &p, Carve &c) {
    size_t most = 0;
    for (int i = 0; i < p.n; ++i) most = std::max(most, plan_of(p.product[i], p.pr).partial_bytes);
    p.partial = static_cast<float *>(c.take(most));
    p.bytes = std::max<size_t>(c.at, 16);
}

Problem problem_of(const gdn_ffn_desc &d) {
    Problem pr = {};
    pr.M = d.M, pr.D = d.D, pr.F = d.F, pr.O = d.D_out;
    pr.f32 = d.dtype == GDN_F32, pr.act = d.activation;
    pr.planes = pr.f32 ? 3 : 1, pr.terms = pr.f32 ? 6 : 1;
    return pr;
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
    Product &a = p.product[0], &b = p.product[1];
    a.epi = kUp, a.M = pr.M, a.N = pr.F, a.groups = a.pairs = 1, a.a[0] = x, a.b[0] = wg, a.b[1] = wu, a.dual = true;
    a.planes[0] = h, a.gate = gate, a.up = up, a.k = pr.D;
    b.epi = kPlain, b.M = pr.M, b.N = pr.O, b.groups = b.pairs = 1, b.a[0] = h, b.b[0] = wd;
    b.out[0] = y, b.ld_out = pr.O, b.k = pr.F;
    p.n = 2;
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
    auto add = [&]() -> Product & {
        Product &q = p.product[p.n++];
        q.groups = q.pairs = 1;
        return q;
    };
    Product &a = add();
    a.epi = kBack, a.M = pr.M, a.N = pr.F, a.a[0] = gy, a.b[0] = wd, a.b_mn = true, a.k = pr.O;
    a.planes[0] = dg, a.planes[1] = du, a.planes[2] = h, a.gate = const_cast<void *>(gate), a.up = const_cast<void *>(up);
    if (dx) {
        Product &q = add();
        q.epi = kPlain, q.M = pr.M, q.N = pr.D, q.pairs = 2, q.a[0] = dg, q.a[1] = du, q.b[0] = wg, q.b[1] = wu, q.b_mn = true;
        q.k = pr.F, q.out[0] = dx, q.ld_out = pr.D;
    }
    if (dwg || dwu) {
        Product &q = add();
        q.epi = kPlain, q.M = pr.F, q.N = pr.D, q.a_mn = q.b_mn = true, q.b[0] = x, q.k = pr.M, q.ld_out = pr.D;
        q.groups = 0;
        if (dwg) q.a[q.groups] = dg, q.out[q.groups++] = dwg;
        if (dwu) q.a[q.groups] = du, q.out[q.groups++] = dwu;
    }
    if (dwd) {
        Product &q = add();
        q.epi = kPlain, q.M = pr.O, q.N = pr.F, q.a[0] = gy, q.b[0] = h, q.a_mn = q.b_mn = true, q.k = pr.M;
        q.out[0] = dwd, q.ld_out = pr.F;
    }
    finish_plan(p, c);
    return p;
}

gdn_status run_pass(const Pass &p, int32_t *status, cudaStream_t s, const char *where) {
    cudaError_t e = cudaSuccess;
    if (status) e = cudaMemsetAsync(status, 0, sizeof(int32_t), s);
    if (e == cudaSuccess) e = run_stage(p.pr, p.stage, p.n_stage, s);
    for (int i = 0; e == cudaSuccess && i < p.n; ++i) e = run_product(p.product[i], p.pr, p.partial, status, s);
    if (e != cudaSuccess) {
        set_error_detail(where, e);
        return GDN_ERR_CUDA;
    }
    return GDN_OK;
}

bool elem_ok(const void *p, int dtype) { return (reinterpret_cast<uintptr_t>(p) & (dtype == GDN_F32 ? 3u : 1u)) == 0; }

// Sizes: TMA coordinates and the work list count in 32 bits.
gdn_status desc_ok(const gdn_ffn_desc *d) {
    if (!d) return GDN_ERR_INVALID_ARG;
    if (d->dtype != GDN_BF16 && d->dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    if (d->activation != GDN_ACT_SILU && d->activation != GDN_ACT_GELU_TANH) return GDN_ERR_INVALID_ARG;
    if (d->M < 0 || d->D < 1 || d->F < 1 || d->D_out < 1 || (d->M > 1 && d->x_stride < d->D)) return GDN_ERR_INVALID_ARG;
    constexpr int64_t most = 1 << 24;
    if (d->M > most || d->D > most || d->F > most || d->D_out > most || d->x_stride > (1ll << 36)) return GDN_ERR_UNSUPPORTED;
    const int64_t big = std::max({d->D, d->F, d->D_out});
    if (std::max(d->M, big) * std::max(big, (int64_t)64) > (1ll << 38)) return GDN_ERR_UNSUPPORTED;
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
        p = gdn::ffn::plan_fwd(*desc, y, gate, up, workspace);
        if (workspace_bytes < p.bytes) return GDN_ERR_WORKSPACE;
    }
    return gdn::ffn::run_pass(p, device_status, s, "launch gated_ffn_fwd");
}

extern "C" size_t gdn_gated_ffn_bwd_workspace_size(const gdn_ffn_desc *desc, const void *dy, int64_t dy_stride) {
    if (gdn::ffn::desc_ok(desc) != GDN_OK || (desc->M > 1 && dy_stride < desc->D_out)) return 0;
    if (desc->M == 0) return 16;
    // enough for any choice of gradients (the pair of dw_gate and dw_up is split otherwise than one alone)
    void *some = reinterpret_cast<void *>((uintptr_t)16);   // never dereferenced
    return std::max(gdn::ffn::plan_bwd(*desc, dy, dy_stride, nullptr, nullptr, some, some, some, some, nullptr).bytes,
                    gdn::ffn::plan_bwd(*desc, dy, dy_stride, nullptr, nullptr, some, some, nullptr, some, nullptr).bytes);
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
    if (dy_stride > (1ll << 36)) return GDN_ERR_UNSUPPORTED;
    for (const void *q : {(const void *)dx, (const void *)dw_gate, (const void *)dw_up, (const void *)dw_down, dy, gate, up})
        if (!gdn::ffn::elem_ok(q, dt)) return GDN_ERR_INVALID_ARG;
    gdn::ffn::Pass p = {};
    if (desc->M > 0) {
        if (!dy || !gate || !up || !workspace || !gdn::aligned16(workspace)) return GDN_ERR_INVALID_ARG;
        if (workspace_bytes < gdn_gated_ffn_bwd_workspace_size(desc, dy, dy_stride)) return GDN_ERR_WORKSPACE;
        p = gdn::ffn::plan_bwd(*desc, dy, dy_stride, gate, up, dx, dw_gate, dw_up, dw_down, workspace);
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
