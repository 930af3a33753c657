// Element access shared by the layer operators (norm, convolution, scan, step):
// bf16 or fp32 in memory, fp32 in registers, eight or four neighbouring
// elements at a time where the address allows 16-byte accesses.
//
// Every kernel of these operators is launched with programmatic stream
// serialisation (launch_dependent) and starts with grid_dependency_wait(): its
// launch overlaps the end of whatever kernel is before it on the stream, and it
// reads nothing before that kernel is done (2 to 3 us per kernel boundary).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "gdn_internal.cuh"

namespace gdn {

// E neighbouring elements as they lie in memory.
template <typename T, int E>
struct Raw {
    static constexpr int kWords = (int)sizeof(T) * E / 4 > 0 ? (int)sizeof(T) * E / 4 : 1;
    uint32_t w[kWords];
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
    return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

template <typename T, int E>
__device__ __forceinline__ Raw<T, E> zero_raw() {
    Raw<T, E> r;
#pragma unroll
    for (int i = 0; i < Raw<T, E>::kWords; ++i) r.w[i] = 0u;
    return r;
}

// Aligned load of E elements (E * sizeof(T) a power of two from 2 to 32 bytes;
// the address a multiple of min(that, 16)).
template <typename T, int E>
__device__ __forceinline__ Raw<T, E> load_raw(const T *p) {
    Raw<T, E> r;
    constexpr int kBytes = (int)sizeof(T) * E;
    if constexpr (kBytes == 2) {
        r.w[0] = *reinterpret_cast<const unsigned short *>(p);
    } else if constexpr (kBytes == 4) {
        r.w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (kBytes == 8) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        r.w[0] = v.x, r.w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) {
            const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
            r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
        }
    }
    return r;
}

template <typename T, int E>
__device__ __forceinline__ void store_raw(T *p, const Raw<T, E> &r) {
    constexpr int kBytes = (int)sizeof(T) * E;
    if constexpr (kBytes == 2) {
        *reinterpret_cast<unsigned short *>(p) = (unsigned short)r.w[0];
    } else if constexpr (kBytes == 4) {
        *reinterpret_cast<uint32_t *>(p) = r.w[0];
    } else if constexpr (kBytes == 8) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(r.w[0], r.w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i)
            reinterpret_cast<uint4 *>(p)[i] = make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
    }
}

template <typename T, int E>
__device__ __forceinline__ void unpack(const Raw<T, E> &r, float *x) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = __uint_as_float(r.w[i]);
    } else if constexpr (E == 1) {
        x[0] = __uint_as_float(r.w[0] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            x[2 * i] = __uint_as_float(r.w[i] << 16);
            x[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
        }
    }
}

// Rounded once, to nearest even.
template <typename T, int E>
__device__ __forceinline__ Raw<T, E> pack(const float *x) {
    Raw<T, E> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < E; ++i) r.w[i] = __float_as_uint(x[i]);
    } else if constexpr (E == 1) {
        r.w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(x[0]));
    } else {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            r.w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return r;
}

// E elements of which the first `n` exist (element by element: any alignment).
template <typename T, int E>
__device__ __forceinline__ Raw<T, E> load_some(const T *p, int n) {
    float x[E];
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = i < n ? to_f32(p[i]) : 0.f;
    return pack<T, E>(x);  // exact: the values are of type T
}
template <typename T, int E>
__device__ __forceinline__ void store_some(T *p, const float *x, int n) {
#pragma unroll
    for (int i = 0; i < E; ++i)
        if (i < n) p[i] = from_f32<T>(x[i]);
}

// Eight neighbouring elements of which `live` exist, on their way into shared
// memory: asynchronously where the address allows, else (and for what does not
// exist, which is zero) by plain stores.  The thread that copies is the one that
// reads, after copy_commit and copy_wait.
template <typename T>
__device__ __forceinline__ void copy8_whole(T *dst, const T *src) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(dst);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + 16 * i), "l"(src + i * 16 / (int)sizeof(T)) : "memory");
}
template <typename T>
__device__ __forceinline__ void copy8_async(T *dst, const T *src, int live, bool vec) {
    if (vec && live >= 8) {
        copy8_whole<T>(dst, src);
    } else {
        store_raw<T, 8>(dst, live > 0 ? load_some<T, 8>(src, live) : zero_raw<T, 8>());
    }
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LATER>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LATER) : "memory");
}

// Two fp32 values in one 64-bit register; mul, add and fma act on both.
using F2 = unsigned long long;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
__device__ __forceinline__ F2 pair(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float lo(F2 v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi(F2 v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// 2^x, at most 2^-22 off relatively; results below 2^-126 are zero.  Where e^x is
// wanted the argument x log2(e) is rounded once, which adds |x| 2^-24 or less: 2e-7
// at 5, 1e-6 at 20, 4e-6 at 80.  Kept, because what it scales is as small as that
// error is large: sigmoid(-20), softplus(-20) and a decay e^-20 are 2e-9, so at
// most 2e-15 is off beside terms of order one.  Carrying the remainder along in
// softplus and its slope (four more operations on pairs and a guard for infinities)
// brought no output of the scan nearer its 64-bit value: the states stay at 9e-7,
// dA at 1.5e-6, ddt and dB at 4e-7, for 173 us instead of 171 and 305 instead of 301.
__device__ __forceinline__ float exp2_f32(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ F2 exp2_pair(F2 x) { return pair(exp2_f32(lo(x)), exp2_f32(hi(x))); }

__device__ __forceinline__ float rcp_f32(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ F2 rcp_pair(F2 x) { return pair(rcp_f32(lo(x)), rcp_f32(hi(x))); }
__device__ __forceinline__ F2 both(float x) { return pair(x, x); }

// 1 / (1 + exp(-x)); exp(-x) = inf gives the right zero (below -87 the result is
// zero too, as what is below 2^-126).
__device__ __forceinline__ F2 sigmoid_pair(F2 x) {
    return rcp_pair(add2(exp2_pair(mul2(x, both(-kLog2e))), both(1.f)));
}

// E neighbouring values as pairs (a single value: its pair's second half is
// zero), and back, rounded once.
template <typename T, int E = 8>
__device__ __forceinline__ void unpack_pairs(const Raw<T, E> &r, F2 (&v)[(E + 1) / 2]) {
#pragma unroll
    for (int i = 0; i < (E + 1) / 2; ++i) {
        if constexpr (E == 1)
            v[i] = pair(__uint_as_float(sizeof(T) == 2 ? r.w[0] << 16 : r.w[0]), 0.f);
        else if constexpr (sizeof(T) == 2)
            v[i] = pair(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xFFFF0000u));
        else
            v[i] = pair(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
    }
}
template <typename T, int E>
__device__ __forceinline__ Raw<T, E> pack_pairs(const F2 (&v)[(E + 1) / 2]) {
    float x[E + 1];
#pragma unroll
    for (int i = 0; i < (E + 1) / 2; ++i) x[2 * i] = lo(v[i]), x[2 * i + 1] = hi(v[i]);
    return pack<T, E>(x);
}

// 1 / (1 + exp(-x)), x times which is SiLU.
__device__ __forceinline__ float sigmoid_f32(float x) { return rcp_f32(1.f + exp2_f32(x * -kLog2e)); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// The sequence a packed batch's token t belongs to: the n with cu[n] <= t <
// cu[n + 1].  Whatever cu holds, the answer is in [0, n_seqs).
__device__ __forceinline__ int find_seq(const int32_t *cu, int n_seqs, int t) {
    int lo = 0, hi = n_seqs - 1;  // the answer is in [lo, hi]
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(cu + mid + 1) <= t) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// Writes 0 or GDN_ERR_DEVICE_CHECK for cu_seqlens: cu[0] = 0, no entry below
// its predecessor, cu[n_seqs] = T.  Called by one whole block.
__device__ __forceinline__ void check_cu(const int32_t *cu, int n_seqs, int T, int32_t *status) {
    int bad = 0;
    for (int i = threadIdx.x; i <= n_seqs; i += blockDim.x) {
        const int c = cu[i];
        bad |= (i == 0 && c != 0) || (i == n_seqs && c != T) || (i > 0 && c < cu[i - 1]);
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *status = bad ? GDN_ERR_DEVICE_CHECK : GDN_OK;
}

inline int device_sm_count() {
    // a device attribute does not change: cached per device
    static std::atomic<int> cache[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return 152;
    }
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
            cudaGetLastError();
            n = 152;
        }
        cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace gdn
