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
// Rounding is that of the real quotient 127 v / A of the float32 values v and A, so the result does
// not depend on how a row is divided among threads. inv = 127 / A is off by 2^-24 relative, so
// v * inv can only round to the wrong side near a half; there the sign of 127 v - (k + 1/2) A is
// taken exactly (a product's rounded part and its error, and two fused multiply-adds). Where v and
// A are bf16 values, exact halves are common (about one value in 300) and nothing else comes
// nearer to a half than 1.5e-5 relative: there v * inv (1 - 2^-20) and v * inv (1 + 2^-20) round
// apart on exact halves only, and the even one is taken by the rounding of their sum.
//
// A row with A = 0 has q = 0 and scale = 0. A row that holds a NaN or an infinity (after the
// gate, the residual and the weight), or whose sum of squares passes the float32 range, has
// q = 0 and scale = NaN: it reads back as NaN instead of as finite numbers that mean nothing.
#pragma once
#include <cuda_bf16.h>

#include <type_traits>

#include "depthwise_plane.cuh"   // bulk_g2s
#include "i8_ptx.cuh"

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
template <typename T>
__device__ __forceinline__ T i8_type(float v) {
    if constexpr (sizeof(T) == 2) return __float2bfloat16_rn(v);
    else return v;
}

// Pairs of float32 in one 64-bit register (sm_100's packed arithmetic: two values an instruction).
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_split(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// The largest of three magnitudes; a NaN stays a NaN (its bits lie above infinity's).
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Eight consecutive values as they lie in memory (16-byte aligned), and as four pairs.
template <typename T>
struct I8Raw {
    uint4 u[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ I8Raw<T> i8_raw_load(const T *p) {
    I8Raw<T> r;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.u[i] = reinterpret_cast<const uint4 *>(p)[i];
    return r;
}
template <typename T>
__device__ __forceinline__ I8Raw<T> i8_raw_zero() {
    I8Raw<T> r;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.u[i] = make_uint4(0, 0, 0, 0);
    return r;
}
template <typename T>
__device__ __forceinline__ void i8_raw_store(T *p, const I8Raw<T> &r) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) reinterpret_cast<uint4 *>(p)[i] = r.u[i];
}
__device__ __forceinline__ void i8_unpack(const I8Raw<__nv_bfloat16> &r, uint64_t (&t)[4]) {
    const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void i8_unpack(const I8Raw<float> &r, uint64_t (&t)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        t[2 * i] = f2_pack(__uint_as_float(r.u[i].x), __uint_as_float(r.u[i].y));
        t[2 * i + 1] = f2_pack(__uint_as_float(r.u[i].z), __uint_as_float(r.u[i].w));
    }
}
// Rounds four pairs to the type.
__device__ __forceinline__ void i8_pack(const uint64_t (&t)[4], I8Raw<__nv_bfloat16> &r) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        f2_split(t[i], lo, hi);
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        w[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    r.u[0] = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void i8_pack(const uint64_t (&t)[4], I8Raw<float> &r) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float a, b, c, d;
        f2_split(t[2 * i], a, b);
        f2_split(t[2 * i + 1], c, d);
        r.u[i] = make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
    }
}

// silu(a) * b for two pairs in float32, silu(a) = a / (1 + 2^(-a log2 e)), by the fast exponential and
// reciprocal: relative error below (9 + 1.25 |a|) 2^-24, far below the rounding to 8 bits (2^-8 of
// the row's largest value) that follows. In units of 2^-24 that is the rounded log2 e (0.224) and the
// rounded product with it, which move the exponential by 1.224 |a|; the exponential 4 (two steps
// of its last place), the addition 1, the reciprocal 2 (one step), and 1 for each product. Gates
// below -87.33, whose exponential passes 2^126 and whose silu is below 1.04e-36, give 0. With an
// exponential and a quotient that keep denormals the gate took 14 instructions a value instead of
// 4, and instructions bound the kernel.
__device__ __forceinline__ uint64_t i8_glu(uint64_t a, uint64_t b) {
    float lo, hi;
    f2_split(f2_mul(a, f2_pack(-1.44269504f, -1.44269504f)), lo, hi);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(lo));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(hi));
    f2_split(f2_add(f2_pack(lo, hi), f2_pack(1.0f, 1.0f)), lo, hi);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(lo));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(hi));
    return f2_mul(f2_mul(a, f2_pack(lo, hi)), b);
}

// What one row's rounding needs: inv = 127 / (A * up), with `up` a power of two that brings rows of
// tiny or huge values, where 127 / A or 127 v could leave the float32 range, back into it. The
// scaling is exact but for values that become denormal, which are 2^-100 of A and round to 0.
struct I8RowScale {
    float A, inv, up;
    bool dead;   // nothing to round: A = 0, or not finite
};

__device__ __forceinline__ I8RowScale i8_row_scale(uint32_t amax_bits, bool finite) {
    I8RowScale s;
    s.dead = amax_bits == 0u || !finite;
    // 0x0d800000 = 2^-100, 0x71800000 = 2^100
    s.up = amax_bits < 0x0d800000u ? 0x1p+60f : amax_bits > 0x71800000u ? 0x1p-60f : 1.0f;
    s.A = __uint_as_float(amax_bits) * s.up;
    s.inv = s.dead ? 0.0f : 127.0f / s.A;
    return s;
}

constexpr float kI8Magic = 12582912.0f;   // 1.5 * 2^23: adding it rounds to an integer, ties to even
constexpr float kI8NearHalf = 0.49999f;   // 1e-5 off a half: v * inv is off by at most 127 * 2^-24 < 7.6e-6
constexpr float kI8Below = 1.0f - 0x1p-20f, kI8Above = 1.0f + 0x1p-20f;

// The integer m = kI8Magic + k, k the nearest to v * inv, made the nearest to 127 v / A. With `side`
// the sign of v * inv - k, k moves by `side` if side * (127 v - (k + side / 2) A) > 0, or = 0 and k
// is odd. p and e hold 127 v exactly; near a half p and (k + side / 2) A agree in their leading 15
// bits and more, so the first fused multiply-add is exact and the last sum has the exact sign.
// Away from a half nothing moves.
__device__ __forceinline__ uint32_t i8_settle(float v, float m, const I8RowScale &s) {
    const float k = m - kI8Magic;
    const float side = fmaf(v, s.inv, -k) > 0.0f ? 1.0f : -1.0f;
    const float p = v * 127.0f, e = fmaf(v, 127.0f, -p);
    const float d = side * (fmaf(-fmaf(side, 0.5f, k), s.A, p) + e);
    const bool move = d > 0.0f || (d == 0.0f && (__float_as_uint(m) & 1u));
    return __float_as_uint(move ? m + side : m);
}

// Rounds one value (the low byte of the result).
__device__ __forceinline__ uint32_t i8_quant1(float t, const I8RowScale &s) {
    const float v = s.dead ? 0.0f : t * s.up;
    return i8_settle(v, fmaf(v, s.inv, kI8Magic), s);
}

// bf16 values t and their inv * (1 -+ 2^-20): magic + k from both sides are equal, or neighbours on
// an exact half. Their sum lies in [2^24, 2^25), where float32 holds even integers only: it is 2
// (magic + k), and on a half rounds to the k that is even. Its low mantissa bits are k's.
__device__ __forceinline__ uint64_t i8_round_bf16(uint64_t t, uint64_t below, uint64_t above) {
    const uint64_t magic = f2_pack(kI8Magic, kI8Magic);
    return f2_add(f2_fma(t, below, magic), f2_fma(t, above, magic));
}

// The low bytes of four words.
__device__ __forceinline__ uint32_t i8_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Rounds the NP pairs of values of a live row, already times `up`, to the low bytes of words. BF16:
// the values are bf16 values.
template <bool BF16, int NP>
__device__ __forceinline__ void i8_quant(const uint64_t (&t)[NP], const I8RowScale &s, uint32_t (&b)[2 * NP]) {
    if constexpr (BF16) {
        const float below = s.inv * kI8Below, above = s.inv * kI8Above;
        const uint64_t inv0 = f2_pack(below, below), inv1 = f2_pack(above, above);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            float lo, hi;
            f2_split(i8_round_bf16(t[i], inv0, inv1), lo, hi);
            b[2 * i] = __float_as_uint(lo);
            b[2 * i + 1] = __float_as_uint(hi);
        }
    } else {
        const uint64_t magic = f2_pack(kI8Magic, kI8Magic), inv = f2_pack(s.inv, s.inv), minus1 = f2_pack(-1.0f, -1.0f);
        uint64_t m[NP];
        float worst = 0.0f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            m[i] = f2_fma(t[i], inv, magic);
            float lo, hi;
            f2_split(f2_fma(t[i], inv, f2_fma(m[i], minus1, magic)), lo, hi);   // t * inv less the integer
            worst = max3_abs(worst, lo, hi);
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            float lo, hi;
            f2_split(m[i], lo, hi);
            b[2 * i] = __float_as_uint(lo);
            b[2 * i + 1] = __float_as_uint(hi);
        }
        if (worst > kI8NearHalf) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                float lo, hi;
                f2_split(t[i], lo, hi);
                b[2 * i] = i8_settle(lo, __uint_as_float(b[2 * i]), s);
                b[2 * i + 1] = i8_settle(hi, __uint_as_float(b[2 * i + 1]), s);
            }
        }
    }
}

// Block totals of the warps' maxima and, for a norm, sums (at most 16 warps).
template <bool NORM>
__device__ __forceinline__ void i8_block_totals(uint32_t &amax, float &sum, uint32_t *s_max, float *s_sum, int warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) {
        s_max[warp] = amax;
        s_sum[warp] = sum;
    }
    __syncthreads();
    amax = __reduce_max_sync(0xffffffffu, lane < warps ? s_max[lane] : 0u);
    if constexpr (NORM) {
        sum = lane < warps ? s_sum[lane] : 0.0f;   // lanes 16 .. 31 hold zeros
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
}

// A row's scale as it is stored. A norm's A * rstd can pass the float32 range where the scale, which is
// 127 times smaller, does not: then rstd is divided first.
template <bool NORM>
__device__ __forceinline__ float i8_stored_scale(uint32_t amax, float sum, bool finite, int C, float eps) {
    const float A = __uint_as_float(amax);
    if (!finite) return __uint_as_float(0x7fc00000u);
    if (amax == 0u) return 0.0f;
    if constexpr (NORM) {
        const float rstd = 1.0f / sqrtf(sum / static_cast<float>(C) + eps), top = A * rstd;
        return top < __uint_as_float(0x7f800000u) ? top / 127.0f : A * (rstd / 127.0f);
    } else {
        return A / 127.0f;
    }
}

// One row per group of threads: a block, or a warp (TPR = 32), which takes RW rows at once. A thread
// holds NV groups of eight values of a row in registers, so a row of up to 8 * NV values a thread is
// read once; a longer row (STREAM) is walked in pieces of that size twice, the second time from h
// (or x), which the first pass left in L2. A streamed norm adds the pieces' sums of squares in
// float64: a float32 sum that a thread carries through a row of 2^27 values (131072 additions) is off
// by up to 1e-3 where the values are alike. All of a thread's loads are issued before the first is
// used: with four groups a thread (of one row or several) that keeps 100 KB and more of loads in
// flight per SM.
// VEC: tensors on 16 bytes and C a multiple of 8; a thread's eight values are neighbours and move in
// 16-byte accesses; a block has the threads that the row needs (TPR = 0). Otherwise any C and any
// pointers: neighbouring lanes hold neighbouring values, an element an access, and a thread's values
// are TPR apart, a constant, so that its accesses need no address arithmetic.
template <typename T, int MODE, int NV, bool VEC, int TPR, int RW, bool STREAM>
__global__ void __launch_bounds__(TPR == 32 ? 128 : 512)
i8_rows_kernel(const I8RowsParams p, unsigned int *status) {
    grid_dependents_launch();   // programmatic dependent launch (see ptx.cuh)
    grid_dependency_wait();
    constexpr bool NORM = MODE == kI8Norm || MODE == kI8NormResidual;
    constexpr bool GROUP_WARP = TPR == 32;
    static_assert(RW == 1 || (GROUP_WARP && !STREAM), "several rows: a warp's, in registers");
    constexpr bool BF16 = MODE == kI8Plain && sizeof(T) == 2;   // the rounded values are bf16 values
    __shared__ float s_sum[16];
    __shared__ uint32_t s_max[16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tpr = TPR != 0 ? TPR : static_cast<int>(blockDim.x);
    const int tid = GROUP_WARP ? lane : static_cast<int>(threadIdx.x);
    const long long row0 = GROUP_WARP ? (1LL * blockIdx.x * (blockDim.x >> 5) + warp) * RW : static_cast<long long>(blockIdx.x);
    if (row0 >= p.M) return;   // whole warps only, and no block barrier follows for GROUP_WARP
    const int C = p.C;
    const long long n_elems = p.M * C, x_elems = n_elems * (MODE == kI8Glu ? 2 : 1);   // bounds checks (debug build)

    const T *x = static_cast<const T *>(p.x);
    const T *second = MODE == kI8Glu ? x : static_cast<const T *>(p.residual);   // up, or the residual
    T *h = static_cast<T *>(p.h);
    // the elements and bytes at which row r of the group's starts
    struct Row {
        long long x, second, h, q;
        bool live;
    };
    auto of = [&](int r) {
        const long long row = row0 + r;
        const long long e = row * C * (MODE == kI8Glu ? 2 : 1);
        return Row{e, MODE == kI8Glu ? e + C : e, row * C, row * p.ldq, RW == 1 || row < p.M};
    };

    // VEC: column of value i of group k in the piece that starts at c0
    auto at = [&](int c0, int k, int i) { return c0 + (k * tpr + tid) * 8 + i; };

    // Reads a piece of the warp's or block's rows: the values t that are rounded; the norms add the
    // squares of h to `sum`. first: the rows' first pass, which writes h.
    auto load = [&](int c0, bool first, uint64_t (&t)[RW][NV][4], uint64_t (&sum)[RW]) {
        const bool from_h = MODE == kI8NormResidual && !first;
        const bool two = MODE == kI8Glu || (MODE == kI8NormResidual && first);
        if constexpr (VEC) {
            I8Raw<T> a[RW][NV], b[RW][NV];
#pragma unroll
            for (int r = 0; r < RW; ++r)
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int c = at(c0, k, 0);
                    const Row w = of(r);
                    const bool in = c < C && w.live && in_bounds(w.x + c, 8, x_elems, kSiteI8RowsX, status);
                    a[r][k] = in ? i8_raw_load((from_h ? h : x) + w.x + c) : i8_raw_zero<T>();
                    if (two) b[r][k] = in ? i8_raw_load(second + w.second + c) : i8_raw_zero<T>();
                }
            uint64_t w[4];
#pragma unroll
            for (int kr = 0; kr < NV * RW; ++kr) {
                const int k = kr / RW, r = kr % RW, c = at(c0, k, 0);
                const Row row = of(r);
                i8_unpack(a[r][k], t[r][k]);
                uint64_t u[4];
                if constexpr (MODE == kI8Glu) {
                    i8_unpack(b[r][k], u);
#pragma unroll
                    for (int i = 0; i < 4; ++i) t[r][k][i] = i8_glu(t[r][k][i], u[i]);
                }
                if constexpr (MODE == kI8NormResidual) {
                    if (first) {
                        i8_unpack(b[r][k], u);
#pragma unroll
                        for (int i = 0; i < 4; ++i) t[r][k][i] = f2_add(t[r][k][i], u[i]);
                        i8_pack(t[r][k], a[r][k]);
                        i8_unpack(a[r][k], t[r][k]);
                        if (c < C && row.live) i8_raw_store(h + row.x + c, a[r][k]);
                    }
                }
                if constexpr (NORM) {
                    if (r == 0) i8_unpack(i8_raw_load(p.weight + (c < C ? c : 0)), w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        sum[r] = f2_fma(t[r][k][i], t[r][k][i], sum[r]);
                        t[r][k][i] = f2_mul(t[r][k][i], w[i]);
                    }
                }
            }
        } else {
            static_assert(VEC || RW == 1, "element accesses: one row");
            const Row row = of(0);
            const T *from = (from_h ? h : x) + row.x + c0 + tid, *from2 = second + row.second + c0 + tid;
            const float *weight = p.weight + c0 + tid;
            const int left = C - c0 - tid;   // element e of the thread is in the row if e * TPR < left
            float a[NV][8], b[NV][8], w[NV][8];
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int e = (k * 8 + i) * TPR;
                    const bool in = e < left && in_bounds(row.x + c0 + tid + e, 1, x_elems, kSiteI8RowsX, status);
                    a[k][i] = in ? i8_to_float(from[e]) : 0.0f;
                    if (two) b[k][i] = in ? i8_to_float(from2[e]) : 0.0f;
                    if (NORM) w[k][i] = in ? weight[e] : 0.0f;
                }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    t[0][k][i] = f2_pack(a[k][2 * i], a[k][2 * i + 1]);
                    if constexpr (MODE == kI8Glu) t[0][k][i] = i8_glu(t[0][k][i], f2_pack(b[k][2 * i], b[k][2 * i + 1]));
                    if constexpr (MODE == kI8NormResidual) {
                        if (first) {
                            float lo, hi;
                            f2_split(f2_add(t[0][k][i], f2_pack(b[k][2 * i], b[k][2 * i + 1])), lo, hi);
                            const T hlo = i8_type<T>(lo), hhi = i8_type<T>(hi);
                            const int e = (k * 8 + 2 * i) * TPR;
                            T *to = h + row.x + c0 + tid;
                            if (e < left) to[e] = hlo;
                            if (e + TPR < left) to[e + TPR] = hhi;
                            t[0][k][i] = f2_pack(i8_to_float(hlo), i8_to_float(hhi));
                        }
                    }
                    if constexpr (NORM) {
                        sum[0] = f2_fma(t[0][k][i], t[0][k][i], sum[0]);
                        t[0][k][i] = f2_mul(t[0][k][i], f2_pack(w[k][2 * i], w[k][2 * i + 1]));
                    }
                }
            }
        }
    };
    auto store = [&](int c0, int r, int k, const uint32_t (&b)[8]) {
        const Row row = of(r);
        if constexpr (VEC) {
            const int c = at(c0, k, 0);
            if (c < C && row.live && in_bounds(row.h + c, 8, n_elems, kSiteI8RowsQ, status))
                *reinterpret_cast<uint2 *>(p.q + row.q + c) =
                    make_uint2(i8_bytes(b[0], b[1], b[2], b[3]), i8_bytes(b[4], b[5], b[6], b[7]));
        } else {
            int8_t *to = p.q + row.q + c0 + tid;
            const int left = C - c0 - tid;
            auto group = [&](auto all) {
                constexpr bool ALL = decltype(all)::value;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int e = (k * 8 + i) * TPR;
                    if ((ALL || e < left) && in_bounds(row.h + c0 + tid + e, 1, n_elems, kSiteI8RowsQ, status))
                        to[e] = static_cast<int8_t>(b[i]);
                }
            };
            if (C - c0 >= (k + 1) * 8 * TPR) group(std::true_type());
            else group(std::false_type());
        }
    };

    uint64_t t[RW][NV][4];
    uint64_t sum2[RW];      // of the squares, even and odd values apart
    double pieces = 0.0;    // of a streamed row's earlier pieces
    float top[RW];          // the largest magnitude, or NaN
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        sum2[r] = 0;
        top[r] = 0.0f;
    }
    const int piece = tpr * 8 * NV;
    for (int c0 = 0; c0 < (STREAM ? C : 1); c0 += piece) {
        load(c0, true, t, sum2);
        if constexpr (NORM && STREAM) {
            float lo, hi;
            f2_split(sum2[0], lo, hi);
            pieces += static_cast<double>(lo) + static_cast<double>(hi);
            sum2[0] = 0;
        }
#pragma unroll
        for (int r = 0; r < RW; ++r)
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float lo, hi;
                    f2_split(t[r][k][i], lo, hi);
                    top[r] = max3_abs(top[r], lo, hi);
                }
        if (C - c0 <= piece) break;   // c0 + piece may pass the int range
    }
    I8RowScale s[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        // magnitudes are ordered as their bits, NaN above infinity
        uint32_t amax = __reduce_max_sync(0xffffffffu, __float_as_uint(top[r]) & 0x7fffffffu);
        float sum = 0.0f;
        if constexpr (NORM) {
            float lo, hi;
            f2_split(sum2[r], lo, hi);
            sum = STREAM ? static_cast<float>(pieces) : lo + hi;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        if constexpr (!GROUP_WARP) i8_block_totals<NORM>(amax, sum, s_max, s_sum, tpr >> 5);
        const bool finite = amax < 0x7f800000u && (!NORM || sum < __uint_as_float(0x7f800000u));
        s[r] = i8_row_scale(amax, finite);
        if (tid == 0 && row0 + r < p.M && in_bounds(row0 + r, 1, p.M, kSiteI8RowsScale, status))
            p.scale[row0 + r] = i8_stored_scale<NORM>(amax, sum, finite, C, p.eps);
    }
    for (int c0 = 0; c0 < (STREAM ? C : 1); c0 += piece) {
        if constexpr (STREAM) {
            uint64_t unused[RW] = {};
            load(c0, false, t, unused);
        }
#pragma unroll
        for (int rk = 0; rk < RW * NV; ++rk) {
            const int r = rk / NV, k = rk % NV;
            if (s[r].up != 1.0f) {
#pragma unroll
                for (int i = 0; i < 4; ++i) t[r][k][i] = f2_mul(t[r][k][i], f2_pack(s[r].up, s[r].up));
            }
            uint32_t b[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (!s[r].dead) i8_quant<BF16>(t[r][k], s[r], b);
            store(c0, r, k, b);
        }
        if (C - c0 <= piece) break;
    }
}

// Rows that start off 16 bytes (odd C, shifted tensors), one per block of TPR threads: bulk copies
// bring the row's 16-byte interior into shared memory, plain loads its edges, and both passes read
// it there, an element a lane. The copies in flight take no registers, so many blocks fit on an SM
// and hide one another's latency (blocks that walk over rows, with the next row's copies ahead, took
// up to twice as long: a row's work is shorter than a copy's latency).
template <typename T>
__host__ __device__ constexpr int i8_staged_bytes(int values) { return (values * static_cast<int>(sizeof(T)) + 31) & ~15; }

template <typename T, int MODE, int TPR>
__global__ void __launch_bounds__(TPR)
i8_rows_staged_kernel(const I8RowsParams p, unsigned int *status) {
    grid_dependents_launch();
    grid_dependency_wait();
    constexpr bool NORM = MODE == kI8Norm || MODE == kI8NormResidual, RES = MODE == kI8NormResidual;
    constexpr bool BF16 = MODE == kI8Plain && sizeof(T) == 2;
    extern __shared__ __align__(16) uint8_t staged_raw[];
    __shared__ float s_sum[16];
    __shared__ uint32_t s_max[16];
    __shared__ __align__(8) uint64_t s_bar;
    const int tid = threadIdx.x;
    const int C = p.C, n_in = MODE == kI8Glu ? 2 * C : C;   // values of x's row
    const long long row = blockIdx.x, n_elems = p.M * C, x_elems = p.M * n_in;
    const uint32_t bar = smem_u32(&s_bar);

    // A row's source, and where its values begin in shared memory: as far past 16 bytes as in memory.
    struct Source {
        const T *from;
        T *to;
        int n, front, inner;   // values; bytes before the first 16-byte boundary, and of whole 16 bytes after it
    };
    auto source = [&](bool second) {
        Source v;
        v.n = second ? C : n_in;
        v.from = static_cast<const T *>(second ? p.residual : p.x) + row * v.n;
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(v.from) & 15);
        v.to = reinterpret_cast<T *>(staged_raw + (second ? i8_staged_bytes<T>(C) : 0) + off);
        v.front = (16 - off) & 15;
        v.inner = (v.n * static_cast<int>(sizeof(T)) - v.front) & ~15;
        return v;
    };
    const Source sx = source(false), sr = source(RES);
    T *xs = sx.to, *h = static_cast<T *>(p.h) + row * C;
    int8_t *q = p.q + row * p.ldq;
    if (tid == 0) {
        mbar_init(bar, 1);
        fence_barrier_init();
        mbar_arrive_expect_tx(bar, sx.inner + (RES ? sr.inner : 0));
        const bool in = in_bounds(row * n_in, n_in, x_elems, kSiteI8RowsX, status);
        auto copy = [&](const Source &v) {
            if (in) bulk_g2s(smem_u32(v.to) + v.front, reinterpret_cast<const uint8_t *>(v.from) + v.front, v.inner, bar);
            else mbar_complete_tx(bar, v.inner);
        };
        copy(sx);
        if (RES) copy(sr);
    }
    // the edges: the first eight threads have those before the interior, the next eight those after it
    auto edge = [&](const Source &v) {
        const int front = v.front / static_cast<int>(sizeof(T)), rest = front + v.inner / static_cast<int>(sizeof(T));
        const int e = tid < 8 ? tid : rest + tid - 8;
        if (tid < 16 && (tid < 8 ? e < front : e < v.n) && in_bounds(row * v.n + e, 1, x_elems, kSiteI8RowsX, status))
            v.to[e] = v.from[e];
    };
    edge(sx);
    if (RES) edge(sr);

    // Four values e, e + TPR, ... of the row (as two pairs) at a time, `all` if they are all in it.
    constexpr int NP = 2;
    auto each = [&](auto body) {
        int e0 = 0;
        for (; C - e0 >= 2 * NP * TPR; e0 += 2 * NP * TPR) body(e0 + tid, std::true_type());
        if (e0 < C) body(e0 + tid, std::false_type());
    };
    auto weights = [&](int e, auto all) {
        constexpr bool ALL = decltype(all)::value;
        return f2_pack(ALL || e < C ? p.weight[e] : 0.0f, ALL || e + TPR < C ? p.weight[e + TPR] : 0.0f);
    };
    auto pair = [&](const T *from, int e, auto all) {
        constexpr bool ALL = decltype(all)::value;
        return f2_pack(ALL || e < C ? i8_to_float(from[e]) : 0.0f, ALL || e + TPR < C ? i8_to_float(from[e + TPR]) : 0.0f);
    };
    __syncthreads();
    const bool landed = mbar_wait(bar, 0);
    if (!landed) atomicOr(status, kStatusTimeout);

    uint64_t sum2 = 0;
    float top = 0.0f;
    each([&](int e, auto all) {
        constexpr bool ALL = decltype(all)::value;
        uint64_t w[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) w[i] = NORM ? weights(e + 2 * i * TPR, all) : 0;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = e + 2 * i * TPR;
            uint64_t t = pair(xs, c, all);
            if constexpr (MODE == kI8Glu) t = i8_glu(t, pair(xs + C, c, all));
            if constexpr (RES) {
                float lo, hi;
                f2_split(f2_add(t, pair(sr.to, c, all)), lo, hi);
                const T hlo = i8_type<T>(lo), hhi = i8_type<T>(hi);
                if (ALL || c < C) h[c] = xs[c] = hlo;
                if (ALL || c + TPR < C) h[c + TPR] = xs[c + TPR] = hhi;
                t = f2_pack(i8_to_float(hlo), i8_to_float(hhi));
            }
            if constexpr (NORM) {
                sum2 = f2_fma(t, t, sum2);
                t = f2_mul(t, w[i]);
            }
            float lo, hi;
            f2_split(t, lo, hi);
            top = max3_abs(top, lo, hi);
        }
    });
    uint32_t amax = __reduce_max_sync(0xffffffffu, __float_as_uint(top) & 0x7fffffffu);
    float sum = 0.0f;
    if constexpr (NORM) {
        float lo, hi;
        f2_split(sum2, lo, hi);
        sum = lo + hi;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    i8_block_totals<NORM>(amax, sum, s_max, s_sum, TPR / 32);
    const bool finite = amax < 0x7f800000u && (!NORM || sum < __uint_as_float(0x7f800000u));
    const I8RowScale s = i8_row_scale(amax, finite);
    if (tid == 0 && in_bounds(row, 1, p.M, kSiteI8RowsScale, status))
        p.scale[row] = i8_stored_scale<NORM>(amax, sum, finite, C, p.eps);
    each([&](int e, auto all) {
        constexpr bool ALL = decltype(all)::value;
        uint64_t t[NP], w[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) w[i] = NORM ? weights(e + 2 * i * TPR, all) : 0;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = e + 2 * i * TPR;
            t[i] = pair(xs, c, all);
            if constexpr (MODE == kI8Glu) t[i] = i8_glu(t[i], pair(xs + C, c, all));
            if constexpr (NORM) t[i] = f2_mul(t[i], w[i]);
            if (s.up != 1.0f) t[i] = f2_mul(t[i], f2_pack(s.up, s.up));
        }
        uint32_t b[2 * NP] = {};
        if (!s.dead) i8_quant<BF16>(t, s, b);
#pragma unroll
        for (int i = 0; i < 2 * NP; ++i)
            if ((ALL || e + i * TPR < C) && in_bounds(row * C + e + i * TPR, 1, n_elems, kSiteI8RowsQ, status))
                q[e + i * TPR] = static_cast<int8_t>(b[i]);
    });
    if (!landed) mbar_wait(bar, 0);   // no copy of this block is in flight when it ends
}

}  // namespace convb200
