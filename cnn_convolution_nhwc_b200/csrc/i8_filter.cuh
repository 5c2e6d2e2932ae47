// Filters to 8 bits, and 8-bit rows back.
//
// A 1 x 1 filter F [Cin][Cout] gets one scale per output channel (column): A[o] = max_c |F[c][o]|,
// q = 127 F[c][o] / A[o] rounded to nearest even (the rules of i8_rows.cuh), scale[o] = A[o] / 127.
// The result is stored transposed, Wq [Cout][Cin], so that both operands of the 8-bit product run
// along the reduction. A column's maximum needs all of Cin before its first byte can be written:
// a cluster of S CTAs holds 32 columns, each CTA a share of the rows in shared memory (staged by
// asynchronous copies, all in flight at once), and the CTAs' maxima meet in distributed shared
// memory. The filter is read once; a share beyond shared memory is walked in pieces twice, the
// second time mostly from L2. Rounded bytes are transposed through a second tile, four rows of a
// column to a word, whose 16-byte chunks are permuted by the column so that neither the words'
// stores nor the chunks' loads meet in a bank, and leave as 16-byte stores. 32 columns (64 bytes of a
// bf16 row) rather than 64 keep a CTA small enough for four on an SM, whose loads, maxima and
// stores overlap: 4096 x 16384 in bf16 took 90 us with 64.
#pragma once
#include "i8_rows.cuh"

namespace convb200 {

struct I8FilterParams {
    const void *F;     // [Cin][Cout]
    int8_t *q;         // [Cout] rows of Cin bytes, ldq apart
    float *scale;      // [Cout]
    int Cin, Cout, ldq;
    int share;         // rows per CTA, a multiple of 128
    int piece;         // rows in shared memory at once, a multiple of 128
};

constexpr int kI8FilterCols = 32;

__host__ __device__ constexpr int i8_filter_smem(int piece, int elem) { return piece * kI8FilterCols * (elem + 1); }

// VEC: rows of F on 16-byte boundaries (Cout a multiple of 8).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256, 4)
i8_filter_kernel(const I8FilterParams p, unsigned int *status) {
    grid_dependents_launch();
    grid_dependency_wait();
    extern __shared__ __align__(128) uint8_t dyn[];
    __shared__ uint32_t s_part[8][kI8FilterCols];
    __shared__ uint32_t s_max[kI8FilterCols];        // this CTA's maxima, read by the cluster
    __shared__ __align__(16) float s_scale[3][kI8FilterCols];   // of the columns: A, inv and up (I8RowScale), inv 0 if dead
    constexpr int ROW = kI8FilterCols * sizeof(T);   // bytes of a staged row
    constexpr int CHUNKS = ROW / 16;
    T *slab = reinterpret_cast<T *>(dyn);                    // [piece][32]
    uint8_t *tile = dyn + static_cast<size_t>(p.piece) * ROW;  // [32][piece] bytes
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t S;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
    const uint32_t rank = cluster_rank();
    const int o0 = static_cast<int>(blockIdx.x / S) * kI8FilterCols;
    const int c0 = static_cast<int>(rank) * p.share;
    const int c1 = p.Cin - c0 < p.share ? p.Cin : c0 + p.share;   // c0 may pass Cin: an empty share
    const int cg = (lane & 7) * 4;                                // this thread's four columns in the block
    const int rg = warp * 4 + (lane >> 3);                        // its row, or group of four rows, modulo 32
    const long long f_elems = 1LL * p.Cin * p.Cout, q_elems = f_elems;
    const T *F = static_cast<const T *>(p.F);
    const bool once = c1 - c0 <= p.piece;   // the share stays in shared memory between the passes

    // Rows b0 .. b1 - 1 into the slab, zeros in the columns past Cout and up to a multiple of four rows.
    auto stage = [&](int b0, int b1) {
        const int rows = (b1 - b0 + 3) & ~3;
        if constexpr (VEC) {
            // a thread keeps its 16-byte chunk of the rows and takes every (256 / CHUNKS)-th
            constexpr int STEP = 256 / CHUNKS, PER = 16 / static_cast<int>(sizeof(T));
            const int e = (threadIdx.x % CHUNKS) * PER;
            int r = threadIdx.x / CHUNKS;
            const T *src = F + 1LL * (b0 + r) * p.Cout + o0 + e;
            uint32_t dst = smem_u32(slab) + r * ROW + e * static_cast<int>(sizeof(T));
            const int live = o0 + e < p.Cout ? b1 - b0 : 0;
#pragma unroll 4
            for (; r < rows; r += STEP, src += 1LL * STEP * p.Cout, dst += STEP * ROW)
                cp_async_16(dst, r < live ? src : F,
                            r < live && in_bounds(src - F, PER, f_elems, kSiteI8FilterF, status) ? 16u : 0u);
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else {
            // a column a lane, eight rows at a time
            const int e = lane;
            for (int r0 = warp; r0 < rows; r0 += 64) {
                T v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int r = r0 + 8 * j;
                    const long long at = 1LL * (b0 + r) * p.Cout + o0 + e;
                    v[j] = static_cast<T>(0.0f);
                    if (b0 + r < b1 && o0 + e < p.Cout && in_bounds(at, 1, f_elems, kSiteI8FilterF, status)) v[j] = F[at];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (r0 + 8 * j < rows) slab[(r0 + 8 * j) * kI8FilterCols + e] = v[j];
            }
        }
        __syncthreads();
    };

    // four neighbouring values of a staged row
    auto four = [&](int r, uint64_t &a, uint64_t &b) {
        if constexpr (sizeof(T) == 2) {
            const uint2 u = *reinterpret_cast<const uint2 *>(slab + r * kI8FilterCols + cg);
            a = f2_pack(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
            b = f2_pack(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
        } else {
            const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(slab + r * kI8FilterCols + cg);
            a = u.x;
            b = u.y;
        }
    };

    float top[4] = {0, 0, 0, 0};
    __nv_bfloat162 top2[2] = {__floats2bfloat162_rn(0.0f, 0.0f), __floats2bfloat162_rn(0.0f, 0.0f)};   // bf16: as they come
    for (int b0 = c0; b0 < c1; b0 += p.piece) {
        const int b1 = c1 - b0 < p.piece ? c1 : b0 + p.piece;
        stage(b0, b1);
        // a staged piece ends with a multiple of four rows, zeros past the last
        const int rows = (b1 - b0 + 3) & ~3;
#pragma unroll 4
        for (int r = rg; r < rows; r += 32) {
            if constexpr (sizeof(T) == 2) {
                const uint2 u = *reinterpret_cast<const uint2 *>(slab + r * kI8FilterCols + cg);
                top2[0] = __hmax2_nan(top2[0], __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x)));
                top2[1] = __hmax2_nan(top2[1], __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y)));
            } else {
                uint64_t a, b;
                four(r, a, b);
                float lo, hi;
                f2_split(a, lo, hi);
                top[0] = max3_abs(top[0], lo, 0.0f);
                top[1] = max3_abs(top[1], hi, 0.0f);
                f2_split(b, lo, hi);
                top[2] = max3_abs(top[2], lo, 0.0f);
                top[3] = max3_abs(top[3], hi, 0.0f);
            }
        }
        if (!once) __syncthreads();   // the next piece goes where this one was
    }
    if constexpr (sizeof(T) == 2) {
        top[0] = __low2float(top2[0]);
        top[1] = __high2float(top2[0]);
        top[2] = __low2float(top2[1]);
        top[3] = __high2float(top2[1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t m = __float_as_uint(top[i]) & 0x7fffffffu;
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 16));
        if (lane < 8) s_part[warp][cg + i] = m;
    }
    __syncthreads();
    if (threadIdx.x < kI8FilterCols) {
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = max(m, s_part[w][threadIdx.x]);
        s_max[threadIdx.x] = m;
    }
    __syncthreads();
    cluster_sync_all();
    if (threadIdx.x < kI8FilterCols) {   // a column a thread: the CTAs' maxima, eight remote loads at once
        uint32_t m = 0;
#pragma unroll
        for (uint32_t r = 0; r < 8; ++r) {
            uint32_t v;
            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_rank(smem_u32(&s_max[threadIdx.x]), r < S ? r : 0u)));
            m = max(m, v);
        }
        const bool finite = m < 0x7f800000u;
        const I8RowScale c = i8_row_scale(m, finite);
        s_scale[0][threadIdx.x] = c.A;
        s_scale[1][threadIdx.x] = c.inv;
        s_scale[2][threadIdx.x] = c.up;
        const int o = o0 + static_cast<int>(threadIdx.x);
        if (rank == 0 && o < p.Cout && in_bounds(o, 1, p.Cout, kSiteI8FilterScale, status))
            p.scale[o] = finite ? __uint_as_float(m) / 127.0f : __uint_as_float(0x7fc00000u);
    }
    __syncthreads();
    I8RowScale sc[4];
    bool plain = true;   // no column of zeros, tiny, huge or not finite
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sc[i].A = s_scale[0][cg + i];
        sc[i].inv = s_scale[1][cg + i];
        sc[i].up = s_scale[2][cg + i];
        sc[i].dead = sc[i].inv == 0.0f;
        plain = plain && !sc[i].dead && sc[i].up == 1.0f;
    }
    cluster_arrive();   // these maxima have been read; nobody leaves before all have (cluster_wait below)

    // bf16: the two sides of inv (i8_rows.cuh); float32: inv
    constexpr bool BF16 = sizeof(T) == 2;
    uint64_t inv0[2], inv1[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float a = sc[2 * i].inv, b = sc[2 * i + 1].inv;
        inv0[i] = BF16 ? f2_pack(a * kI8Below, b * kI8Below) : f2_pack(a, b);
        inv1[i] = f2_pack(a * kI8Above, b * kI8Above);
    }
    const uint64_t magic = f2_pack(kI8Magic, kI8Magic), minus1 = f2_pack(-1.0f, -1.0f);
    for (int b0 = c0; b0 < c1; b0 += p.piece) {
        const int b1 = c1 - b0 < p.piece ? c1 : b0 + p.piece;
        if (!once) stage(b0, b1);
        const int groups = (b1 - b0 + 3) / 4;
        for (int g = rg; g < groups; g += 32) {
            uint32_t m[4][4];
            float worst = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint64_t t[2];
                four(g * 4 + j, t[0], t[1]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float lo, hi;
                    if constexpr (BF16) {
                        f2_split(i8_round_bf16(t[i], inv0[i], inv1[i]), lo, hi);
                    } else {
                        const uint64_t u = f2_fma(t[i], inv0[i], magic);
                        f2_split(f2_fma(t[i], inv0[i], f2_fma(u, minus1, magic)), lo, hi);
                        worst = max3_abs(worst, lo, hi);
                        f2_split(u, lo, hi);
                    }
                    m[j][2 * i] = __float_as_uint(lo);
                    m[j][2 * i + 1] = __float_as_uint(hi);
                }
            }
            if (!plain || (!BF16 && worst > kI8NearHalf)) {
#pragma unroll 1
                for (int j = 0; j < 4; ++j) {   // a row's four values at once: a warp here holds up its CTA
                    uint64_t t[2];
                    four(g * 4 + j, t[0], t[1]);
                    float v[4];
                    f2_split(t[0], v[0], v[1]);
                    f2_split(t[1], v[2], v[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t settled = i8_quant1(v[i], sc[i]);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k == j) m[k][i] = settled;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // rows 4 g .. 4 g + 3 of the column: word g, in chunk g / 4 of its 128-byte run, permuted
                const int col = cg + i;
                const int at = (g & ~31) * 4 + ((((g >> 2) & 7) ^ (col >> 2)) << 4) + (g & 3) * 4;
                *reinterpret_cast<uint32_t *>(tile + static_cast<size_t>(col) * p.piece + at) =
                    i8_bytes(m[0][i], m[1][i], m[2][i], m[3][i]);
            }
        }
        __syncthreads();
        // a column a warp, a 16-byte chunk a lane
        const int chunks = (b1 - b0 + 15) / 16;
        for (int col = warp; col < kI8FilterCols && o0 + col < p.Cout; col += 8) {
            const uint8_t *from = tile + static_cast<size_t>(col) * p.piece;
            int8_t *to = p.q + 1LL * (o0 + col) * p.ldq + b0;
            for (int j = lane; j < chunks; j += 32) {
                const uint4 v = *reinterpret_cast<const uint4 *>(from + (j & ~7) * 16 + (((j & 7) ^ (col >> 2)) << 4));
                const int n = b1 - b0 - j * 16 < 16 ? b1 - b0 - j * 16 : 16;
                if (!in_bounds(1LL * (o0 + col) * p.Cin + b0 + j * 16, n, q_elems, kSiteI8FilterQ, status)) continue;
                if (n == 16) {
                    *reinterpret_cast<uint4 *>(to + j * 16) = v;
                } else {
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 15; ++k)
                        if (k < n) to[j * 16 + k] = static_cast<int8_t>(w[k >> 2] >> (8 * (k & 3)));
                }
            }
        }
        __syncthreads();
    }
    cluster_wait();
}

struct I8DequantParams {
    const int8_t *q;
    const float *scale;
    void *y;               // [M][C]
    long long M;
    int C, ldq;
    int wpr_shift;         // log2 of the warps of a block that share a row
};

__device__ __forceinline__ void i8_put(float *p, float v) { *p = v; }
__device__ __forceinline__ void i8_put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// y = q * scale in float32, rounded to the type. A warp takes a segment of a row, four accesses a lane in flight: 16
// bytes of y each (VEC: rows of y on 16 bytes), so that the warp's stores are whole lines; else 16
// values a lane, one of every 32. blockIdx.y counts the segments that do not fit in one block.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
i8_dequant_kernel(const I8DequantParams p, unsigned int *status) {
    grid_dependents_launch();
    grid_dependency_wait();
    constexpr int PER = 16 / sizeof(T);   // values of a 16-byte store
    constexpr int SEG = VEC ? 4 * 32 * PER : 512;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row = (static_cast<long long>(blockIdx.x) << (3 - p.wpr_shift)) + (warp >> p.wpr_shift);
    const long long start = ((static_cast<long long>(blockIdx.y) << p.wpr_shift) + (warp & ((1 << p.wpr_shift) - 1))) * SEG;
    if (row >= p.M || start >= p.C) return;
    const int c0 = static_cast<int>(start);
    const int8_t *q = p.q + row * p.ldq;
    T *y = static_cast<T *>(p.y) + row * p.C;
    const long long elems = p.M * p.C;
    const float s = p.scale[row];
    if constexpr (VEC) {
        uint2 w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = c0 + (k * 32 + lane) * PER;
            w[k] = make_uint2(0u, 0u);
            if (c < p.C) {
                if constexpr (PER == 8) w[k] = *reinterpret_cast<const uint2 *>(q + c);
                else w[k].x = *reinterpret_cast<const uint32_t *>(q + c);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = c0 + (k * 32 + lane) * PER;
            if (c >= p.C || !in_bounds(row * p.C + c, PER, elems, kSiteI8Dequant, status)) continue;
            uint32_t out[4];
#pragma unroll
            for (int i = 0; i < PER / 2; ++i) {
                const uint32_t u = (i < 2 ? w[k].x : w[k].y) >> (16 * (i & 1));
                float lo, hi;
                f2_split(f2_mul(f2_pack(static_cast<float>(static_cast<int8_t>(u)), static_cast<float>(static_cast<int8_t>(u >> 8))),
                                f2_pack(s, s)), lo, hi);
                if constexpr (PER == 8) {
                    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
                    out[i] = *reinterpret_cast<const uint32_t *>(&v);
                } else {
                    out[2 * i] = __float_as_uint(lo);
                    out[2 * i + 1] = __float_as_uint(hi);
                }
            }
            *reinterpret_cast<uint4 *>(y + c) = make_uint4(out[0], out[1], out[2], out[3]);
        }
    } else {
        int8_t v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int c = c0 + i * 32 + lane;
            v[i] = c < p.C ? q[c] : static_cast<int8_t>(0);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int c = c0 + i * 32 + lane;
            if (c < p.C && in_bounds(row * p.C + c, 1, elems, kSiteI8Dequant, status)) i8_put(y + c, static_cast<float>(v[i]) * s);
        }
    }
}

}  // namespace convb200
