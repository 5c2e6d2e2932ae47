// 8-bit rows: a row of C values becomes C signed bytes and one float32 scale, with what comes
// before the rounding fused in -- nothing, a gate (silu(x[c]) * x[C + c]), or a root-mean-square
// norm with the residual's addition.
//
// With v the row's values and A = max_c |v[c]|:
//     q[c] = 127 v[c] / A rounded to the nearest integer, ties to even;   scale = A / 127.
// The norm's row is v[c] * rstd with v[c] = h[c] * weight[c], h = x + residual rounded to the
// tensors' type, rstd = 1 / sqrt(mean(h^2) + eps). rstd is the same factor in v and in A, so it
// cancels in q and only enters the scale, A * rstd / 127: the sum of squares and the maximum are
// two reductions of one pass over the row, and the second pass (the rounding) works on values
// that are still in registers. A row is therefore read once and written once; the kernels are
// bound by HBM bandwidth.
//
// Rounding is that of the real quotient 127 v / A of the float32 values v and A: the float32
// product v * (127 / A) is off by at most 127 * 2^-23 < 2e-5, so only a product within 4e-5 of
// a half can round to the wrong side, and those few are decided in float64, where 127 v and
// (k + 1/2) A are exact (7 + 24 and 8 + 24 bits). The result does not depend on how a row is
// divided among threads.
//
// A row with A = 0 has q = 0 and scale = 0. A row that holds a NaN or an infinity (after the
// gate, the residual and the weight), or whose sum of squares passes the float32 range, has
// q = 0 and scale = NaN: it reads back as NaN instead of as finite numbers that mean nothing.
#pragma once
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace convb200 {

enum I8RowsMode { kI8Plain = 0, kI8Glu = 1, kI8Norm = 2, kI8NormResidual = 3 };

struct I8RowsParams {
    const void *x;         // [M][C], or [M][2C] for the gate
    const void *residual;  // [M][C] (may be h itself)
    const float *weight;   // [C]
    void *h;               // [M][C]
    int8_t *q;             // [M] rows of C bytes, ldq apart
    float *scale;          // [M]
    long long M;
    int C;
    int ldq;
    float eps;
};

__device__ __forceinline__ float i8_to_float(float v) { return v; }
__device__ __forceinline__ float i8_to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float i8_round_to(float v, float) { return v; }
__device__ __forceinline__ float i8_round_to(float v, __nv_bfloat16) { return __bfloat162float(__float2bfloat16_rn(v)); }

// Eight consecutive values; `p` 16-byte aligned.
__device__ __forceinline__ void i8_load8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void i8_load8(const float *p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
// Stores eight values that the type holds exactly.
__device__ __forceinline__ void i8_store8(__nv_bfloat16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __byte_perm(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1]), 0x7632);
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void i8_store8(float *p, const float (&v)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// silu(a) * b in float32, silu(a) = a / (1 + exp(-a)). With e = exp(-|a|) <= 1 the quotient is
// a * (a < 0 ? e : 1) / (1 + e): nothing overflows and the divisor lies in [1, 2]. The exponential
// and the quotient are CUDA's fast forms: their relative error (2^-22 + |a| 2^-23) is far below
// the rounding to 8 bits (2^-8 of the row's largest value) that follows.
__device__ __forceinline__ float i8_glu(float a, float b) {
    const float e = __expf(-fabsf(a));
    return __fdividef(a < 0.0f ? a * e : a, 1.0f + e) * b;
}

// What one row's rounding needs: inv = 127 / (A * up), with `up` a power of two that brings rows
// of tiny values (A < 2^-100, where 127 / A could overflow) into range exactly.
struct I8RowScale {
    float A, inv, up;
    bool dead;   // nothing to round: A = 0, or not finite
};

__device__ __forceinline__ I8RowScale i8_row_scale(uint32_t amax_bits, bool finite) {
    I8RowScale s;
    s.dead = amax_bits == 0u || !finite;
    s.up = amax_bits < 0x0d800000u ? 0x1p+60f : 1.0f;   // 0x0d800000 = 2^-100
    s.A = __uint_as_float(amax_bits) * s.up;
    s.inv = s.dead ? 0.0f : 127.0f / s.A;
    return s;
}

// The nearest integer of 127 t / A where the float32 product r = t * inv lies near a half.
__device__ __noinline__ float i8_round_near_half(float t, float A, float r) {
    const float lo = floorf(r);
    const double have = static_cast<double>(t) * 127.0, half = (static_cast<double>(lo) + 0.5) * static_cast<double>(A);
    if (have > half) return lo + 1.0f;
    if (have < half) return lo;
    return (static_cast<int>(lo) & 1) ? lo + 1.0f : lo;
}

// Rounds one value (the low byte of the result).
__device__ __forceinline__ uint32_t i8_quant1(float t, const I8RowScale &s) {
    constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: adding it rounds to an integer, ties to even
    const float v = s.dead ? 0.0f : t * s.up;
    const float r = v * s.inv;
    float m = r + kMagic;
    if (fabsf(r - (m - kMagic)) > 0.49996f) m = i8_round_near_half(v, s.A, r) + kMagic;
    return __float_as_uint(m);
}

// Rounds eight values of a row to eight bytes (byte i of the pair of words is value i).
__device__ __forceinline__ uint2 i8_quant8(const float (&t)[8], const I8RowScale &s) {
    constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: adding it rounds to an integer, ties to even
    uint32_t b[8];
    float worst = 0.0f;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = s.dead ? 0.0f : t[i] * s.up;
        const float r = v[i] * s.inv;
        const float m = r + kMagic;
        b[i] = __float_as_uint(m);
        worst = fmaxf(worst, fabsf(r - (m - kMagic)));
    }
    if (worst > 0.49996f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float r = v[i] * s.inv;
            if (fabsf(r - (__uint_as_float(b[i]) - kMagic)) > 0.49996f)
                b[i] = __float_as_uint(i8_round_near_half(v[i], s.A, r) + kMagic);
        }
    }
    const uint32_t lo = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    const uint32_t hi = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
    return make_uint2(lo, hi);
}

// One row per group of `tpr` threads: a warp (GROUP_WARP, rows up to 256 * NV values) or a block.
// A thread holds NV groups of eight values in registers, so a row of up to tpr * 8 * NV values
// is read once; a longer row (STREAM) is walked in pieces of that size twice, the second time
// from h (or x), which the first pass left in L2.
// VEC: rows start on 16-byte boundaries and C is a multiple of 8; a thread's eight values are
// neighbours. Otherwise they are tpr apart, one element per access.
template <typename T, int MODE, int NV, bool VEC, bool GROUP_WARP, bool STREAM>
__global__ void __launch_bounds__(GROUP_WARP ? 256 : 512)
i8_rows_kernel(const I8RowsParams p, unsigned int *status) {
    grid_dependents_launch();   // programmatic dependent launch (see ptx.cuh)
    grid_dependency_wait();
    constexpr bool NORM = MODE == kI8Norm || MODE == kI8NormResidual;
    __shared__ float s_sum[32];
    __shared__ uint32_t s_max[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tpr = GROUP_WARP ? 32 : static_cast<int>(blockDim.x);
    const int tid = GROUP_WARP ? lane : static_cast<int>(threadIdx.x);
    const long long row = GROUP_WARP ? 1LL * blockIdx.x * (blockDim.x >> 5) + warp : static_cast<long long>(blockIdx.x);
    if (row >= p.M) return;   // whole warps only, and no block barrier follows for GROUP_WARP
    const int C = p.C;
    const long long x_elems = p.M * C * (MODE == kI8Glu ? 2 : 1), n_elems = p.M * C;   // bounds checks (debug build)
    const T *x = static_cast<const T *>(p.x);
    const T *res = static_cast<const T *>(p.residual);
    T *h = static_cast<T *>(p.h);
    const long long xrow = row * C * (MODE == kI8Glu ? 2 : 1), hrow = row * C;

    // element index of value i of group k in the piece that starts at c0
    auto at = [&](int c0, int k, int i) { return VEC ? c0 + (k * tpr + tid) * 8 + i : c0 + (k * 8 + i) * tpr + tid; };

    // Reads group k: the values t that are rounded, and (norms) adds the squares of h to `sum`.
    // first: the row's first pass, which writes h.
    auto load = [&](int c0, int k, bool first, float (&t)[8], float &sum) {
        if constexpr (VEC) {
            const int c = at(c0, k, 0);
            if (c >= C) {
#pragma unroll
                for (int i = 0; i < 8; ++i) t[i] = 0.0f;
                return;
            }
            const bool from_h = MODE == kI8NormResidual && !first;
            if (!in_bounds(from_h ? hrow + c : xrow + c, 8, x_elems, kSiteI8RowsX, status)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) t[i] = 0.0f;
                return;
            }
            i8_load8(from_h ? h + hrow + c : x + xrow + c, t);
            if constexpr (MODE == kI8Glu) {
                float up[8];
                i8_load8(x + xrow + C + c, up);
#pragma unroll
                for (int i = 0; i < 8; ++i) t[i] = i8_glu(t[i], up[i]);
            }
            if constexpr (MODE == kI8NormResidual) {
                if (first) {
                    float r[8];
                    i8_load8(res + hrow + c, r);
#pragma unroll
                    for (int i = 0; i < 8; ++i) t[i] = i8_round_to(t[i] + r[i], T());
                    i8_store8(h + hrow + c, t);
                }
            }
            if constexpr (NORM) {
                float w[8];
                i8_load8(p.weight + c, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    sum = fmaf(t[i], t[i], sum);
                    t[i] *= w[i];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = at(c0, k, i);
                t[i] = 0.0f;
                if (c >= C || !in_bounds(xrow + c, 1, x_elems, kSiteI8RowsX, status)) continue;
                float v;
                if (MODE == kI8NormResidual && !first) v = i8_to_float(h[hrow + c]);
                else v = i8_to_float(x[xrow + c]);
                if constexpr (MODE == kI8Glu) v = i8_glu(v, i8_to_float(x[xrow + C + c]));
                if constexpr (MODE == kI8NormResidual) {
                    if (first) {
                        v = i8_round_to(v + i8_to_float(res[hrow + c]), T());
                        h[hrow + c] = static_cast<T>(v);
                    }
                }
                if constexpr (NORM) {
                    sum = fmaf(v, v, sum);
                    v *= p.weight[c];
                }
                t[i] = v;
            }
        }
    };
    auto store = [&](int c0, int k, const float (&t)[8], const I8RowScale &s) {
        const uint2 b = i8_quant8(t, s);
        int8_t *qrow = p.q + row * p.ldq;
        if constexpr (VEC) {
            const int c = at(c0, k, 0);
            if (c < C && in_bounds(hrow + c, 8, n_elems, kSiteI8RowsQ, status)) *reinterpret_cast<uint2 *>(qrow + c) = b;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = at(c0, k, i);
                if (c < C && in_bounds(hrow + c, 1, n_elems, kSiteI8RowsQ, status))
                    qrow[c] = static_cast<int8_t>((i < 4 ? b.x : b.y) >> (8 * (i & 3)));
            }
        }
    };

    float t[NV][8];
    float sum = 0.0f;
    uint32_t amax = 0u;   // of the magnitudes' bits: ordered like them, with infinity and NaN above
    const int piece = tpr * 8 * NV;
    for (int c0 = 0; c0 < (STREAM ? C : 1); c0 += piece) {
#pragma unroll
        for (int k = 0; k < NV; ++k) load(c0, k, true, t[k], sum);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(t[k][i]) & 0x7fffffffu);
        if (C - c0 <= piece) break;   // c0 + piece may pass the int range
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    if constexpr (NORM) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if constexpr (!GROUP_WARP) {
        if (lane == 0) {
            s_max[warp] = amax;
            s_sum[warp] = sum;
        }
        __syncthreads();
        const int warps = tpr >> 5;
        amax = __reduce_max_sync(0xffffffffu, lane < warps ? s_max[lane] : 0u);
        if constexpr (NORM) {
            sum = lane < warps ? s_sum[lane] : 0.0f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
    }
    const bool finite = amax < 0x7f800000u && (!NORM || sum < __uint_as_float(0x7f800000u));
    const I8RowScale s = i8_row_scale(amax, finite);
    if (tid == 0) {
        const float A = __uint_as_float(amax);
        float sc = NORM ? A * (1.0f / sqrtf(sum / static_cast<float>(C) + p.eps)) / 127.0f : A / 127.0f;
        if (amax == 0u) sc = 0.0f;
        if (!finite) sc = __uint_as_float(0x7fc00000u);
        if (in_bounds(row, 1, p.M, kSiteI8RowsScale, status)) p.scale[row] = sc;
    }
    for (int c0 = 0; c0 < (STREAM ? C : 1); c0 += piece) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if constexpr (STREAM) {
                float unused = 0.0f;
                load(c0, k, false, t[k], unused);
            }
            store(c0, k, t[k], s);
        }
        if (C - c0 <= piece) break;
    }
}

}  // namespace convb200
