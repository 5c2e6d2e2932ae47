// Filters to 8 bits, and 8-bit rows back.
//
// A 1 x 1 filter F [Cin][Cout] gets one scale per output channel (column): A[o] = max_c |F[c][o]|,
// q = 127 F[c][o] / A[o] rounded to nearest even (the rules of i8_rows.cuh), scale[o] = A[o] / 127.
// The result is stored transposed, Wq [Cout][Cin], so that both operands of the 8-bit product run
// along the reduction. A column's maximum needs all of Cin before its first byte can be written:
// a cluster of S CTAs holds the column block, each CTA a slab of rows; the CTAs' maxima meet in
// distributed shared memory, and the second pass reads the slab again from L2 (the blocks in
// flight hold 148 slabs of a few tens of KB, well inside the 126 MB), so DRAM is read once.
#pragma once
#include "i8_rows.cuh"

namespace convb200 {

struct I8FilterParams {
    const void *F;     // [Cin][Cout]
    int8_t *q;         // [Cout] rows of Cin bytes, ldq apart
    float *scale;      // [Cout]
    int Cin, Cout, ldq;
    int slab;          // rows per CTA, a multiple of kI8FilterRows
};

constexpr int kI8FilterCols = 64;    // columns per cluster: 128 bytes of a bf16 row
constexpr int kI8FilterRows = 128;   // rows per transposed tile: a warp's 4 rows x 8 warps x 4 row groups
constexpr int kI8FilterPitch = kI8FilterRows + 4;   // bytes between a tile's columns: 33 words

// VEC: Cout a multiple of 8 and F 16-byte aligned.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
i8_filter_kernel(const I8FilterParams p, unsigned int *status) {
    grid_dependents_launch();
    grid_dependency_wait();
    __shared__ uint32_t s_part[8][kI8FilterCols];
    __shared__ uint32_t s_max[kI8FilterCols];        // this CTA's maxima, read by the cluster
    __shared__ __align__(16) uint8_t s_tile[kI8FilterCols * kI8FilterPitch];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t S, rank;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
    rank = cluster_rank();
    const int o0 = static_cast<int>(blockIdx.x / S) * kI8FilterCols;
    const int c0 = static_cast<int>(rank) * p.slab;
    const int c1 = p.Cin - c0 < p.slab ? p.Cin : c0 + p.slab;   // c0 may pass Cin: an empty slab
    const int cg = (lane & 7) * 8;                   // this thread's eight columns in the block
    const long long f_elems = 1LL * p.Cin * p.Cout, q_elems = f_elems;
    const T *F = static_cast<const T *>(p.F);

    auto load = [&](int c, float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        if (c >= c1) return;
        const long long at = 1LL * c * p.Cout + o0 + cg;
        if constexpr (VEC) {
            if (o0 + cg < p.Cout && in_bounds(at, 8, f_elems, kSiteI8FilterF, status)) {
                uint64_t t[4];
                i8_unpack(i8_raw_load(F + at), t);
#pragma unroll
                for (int i = 0; i < 4; ++i) f2_split(t[i], v[2 * i], v[2 * i + 1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (o0 + cg + i < p.Cout && in_bounds(at + i, 1, f_elems, kSiteI8FilterF, status))
                    v[i] = i8_to_float(F[at + i]);
        }
    };

    uint32_t amax[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
    for (int c = c0 + warp * 4 + (lane >> 3); c < c1; c += 32) {
        float v[8];
        load(c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax[i] = max(amax[i], __float_as_uint(v[i]) & 0x7fffffffu);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        amax[i] = max(amax[i], __shfl_xor_sync(0xffffffffu, amax[i], 8));
        amax[i] = max(amax[i], __shfl_xor_sync(0xffffffffu, amax[i], 16));
        if (lane < 8) s_part[warp][cg + i] = amax[i];
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
    I8RowScale sc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t m = 0;
        for (uint32_t r = 0; r < S; ++r) {
            uint32_t v;
            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_rank(smem_u32(&s_max[cg + i]), r)));
            m = max(m, v);
        }
        const bool finite = m < 0x7f800000u;
        sc[i] = i8_row_scale(m, finite);
        const int o = o0 + cg + i;
        if (rank == 0 && threadIdx.x < 8 && o < p.Cout && in_bounds(o, 1, p.Cout, kSiteI8FilterScale, status))
            p.scale[o] = finite ? __uint_as_float(m) / 127.0f : __uint_as_float(0x7fc00000u);
    }
    cluster_sync_all();   // nobody leaves while its maxima may still be read

    // Transposed tiles of 128 rows x 64 columns: a thread rounds 4 neighbouring rows of its eight
    // columns to eight words along the rows.
    for (int t0 = c0; t0 < c1; t0 += kI8FilterRows) {
        const int rg = warp * 4 + (lane >> 3);   // row group: rows 4 rg .. 4 rg + 3 of the tile
        uint32_t words[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        float v[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j) load(t0 + rg * 4 + j, v[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) words[i] |= (i8_quant1(v[j][i], sc[i]) & 0xffu) << (8 * j);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint32_t *>(&s_tile[(cg + i) * kI8FilterPitch + rg * 4]) = words[i];
        __syncthreads();
        // 64 columns x 128 bytes, a word a thread (a column's 128 bytes by one warp)
        for (int w = threadIdx.x; w < kI8FilterCols * (kI8FilterRows / 4); w += 256) {
            const int col = w >> 5, c = t0 + (w & 31) * 4, o = o0 + col;
            if (o >= p.Cout || c >= c1) continue;
            const uint32_t val = *reinterpret_cast<const uint32_t *>(&s_tile[col * kI8FilterPitch + (w & 31) * 4]);
            int8_t *dst = p.q + 1LL * o * p.ldq + c;
            if (c + 4 <= c1) {
                if (in_bounds(1LL * o * p.Cin + c, 4, q_elems, kSiteI8FilterQ, status)) *reinterpret_cast<uint32_t *>(dst) = val;
            } else {
                for (int j = 0; j < c1 - c; ++j)
                    if (in_bounds(1LL * o * p.Cin + c + j, 1, q_elems, kSiteI8FilterQ, status))
                        dst[j] = static_cast<int8_t>(val >> (8 * j));
            }
        }
        __syncthreads();
    }
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

// y = q * scale, one rounding. A warp takes a segment of a row, four accesses a lane in flight: 16
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
