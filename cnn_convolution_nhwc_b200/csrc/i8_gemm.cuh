// The 1 x 1 convolution (matrix product) in 8-bit integers:
//     Y[m][n] = (sum_k q[m][k] * Wq[n][k]) * q_scale[m] * w_scale[n] + bias[n]
// with the sum exact in int32 (|q|, |Wq| <= 128 and at most 131071 terms) and converted to float32,
// one float32 rounding for the product with q_scale, one for the fused product with w_scale and
// addition of the bias, and one to the output type; the two kernels round alike. Both operands run along k, so both are
// staged by plain 2-D tensor copies of 128-byte rows (128 values, 128-byte swizzle) and multiplied
// by tcgen05.mma kind::i8, K = 32 values a step; rows, columns and k past the matrices read as
// zeros (the tensor maps' extents are exact), so no size has a special case in the main loop.
//
// Two kernels. With many tokens the tensor cores bound the product, and a CTA pair computes a
// 256 x 256 tile. With few, the filter's bytes bound it: the filter's rows become the 128 rows of
// the MMA, the tokens its 16 to 128 columns, and the reduction is split over a cluster until the
// GPU is full.
#pragma once
#include <cuda_bf16.h>

#include "dense_tc.cuh"
#include "dense_halo.cuh"
#include "i8_rows.cuh"

namespace convb200 {

struct I8GemmParams {
    const float *q_scale;   // [M]
    const float *w_scale;   // [N]
    const float *bias;      // [N] or null
    void *Y;                // [M][N]
    int M, N;
    int num_kblk;           // ceil(Cin / 128)
    int n_tiles;            // tiles along N
    int m_tiles;            // tiles along M
    int split;              // split kernel: CTAs per cluster, each with its share of the k blocks
    int wide;               // split kernel: slots of several k blocks in one copy (Cin a multiple of 128)
    int own_shift;          // split kernel: log2 of the token columns a CTA of a cluster owns
    int num_tiles;
    int vec;                // 16-byte stores: rows of Y on 16-byte boundaries
};

template <int N>
struct I8Int {
    static constexpr int value = N;
};

__device__ __forceinline__ void i8_out(float *p, float v) { *p = v; }
__device__ __forceinline__ void i8_out(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// ---------------------------------------------------------------------------------------
// Few tokens: i8_split_kernel
// ---------------------------------------------------------------------------------------
// One CTA per (128 filter rows, BN tokens, share of the k blocks). Every CTA of a cluster
// accumulates its share in TMEM, sends each token column to the CTA of the cluster that owns it
// (distributed shared memory), and after one cluster barrier the owners add the shares, which are
// integers: the result does not depend on the split.
//   warp 0      TMA: slots of KB k blocks of 128 filter rows and BN token rows. A copy costs its
//               issuing warp 0.08 us whatever its size, so a slot of two k blocks is two copies of
//               3-D boxes (128 values, rows, k blocks) where Cin is a multiple of 128; elsewhere
//               a k block each, whose extent ends at Cin (p.wide).
//   warp 1      TMEM allocation, MMA issue (M = 128, N = BN). TMEM is taken after the dependency wait: a
//               CTA that held columns while it waited could keep a predecessor's CTA on the same SM,
//               which takes its own only once it runs, waiting for good. The first copies, which
//               warp 0 issues meanwhile, hide it
//   warps 2..9  epilogue, two warps per TMEM lane quarter taking alternate groups of 16 tokens
// Two forms: a ring that fills an SM's shared memory, for long shares of k, and a short one (KB = 1)
// that leaves room for a second CTA -- of the same launch where there are more CTAs than SMs, or of
// the next one, which then sets up, and asks L2 for its first k blocks of the filter, while this one
// finishes (1 x 4096 x 4096 split in 4, filters in HBM: 5.7 us without the request, 5.4 with three
// blocks, 5.5 with four; with eight, which then compete with this launch's copies, 6.0). The next
// launch is let in after the dependency wait, not before it, so that it is the next one that sets up
// early and not the one after it (16 x 2048 x 2048 with its rows: 5.6 and 5.3 us; 1 x 1024 x 1024:
// 3.05 and 2.85). The long ring of 16 columns asks too (1 x 4096 x 16384: 13.2 us without, 12.8
// with); wider tiles do not, since behind a kernel that fills the SMs they ask when they could load
// (128 x 4096 x 4096: 7.9 and 8.9 us).
template <int BN_, int STAGES_, int KB_>
struct I8SplitCfg {
    static constexpr int BN = BN_, STAGES = STAGES_, KB = KB_;
    static constexpr int W_BYTES = KB * 128 * 128, Q_BYTES = KB * BN * 128;
    static constexpr int SLOT = W_BYTES + Q_BYTES;
    static constexpr int RECV_BYTES = BN * 128 * 4;   // the owned columns' shares: split x (BN / split) x 128
    static constexpr int TMEM_COLS = BN < 32 ? 32 : BN;
    static constexpr int SMEM = 1024 + STAGES * SLOT + RECV_BYTES + BN * 4 + (2 * STAGES + 1) * 8 + 16;
    static constexpr int THREADS = 320;
    static constexpr uint32_t IDESC = idesc_i8_s32(128, BN);
    static_assert(SMEM <= 232448, "shared memory of one CTA");
};

using I8ShortSplit16 = I8SplitCfg<16, 5, 1>;   // the short forms
using I8ShortSplit32 = I8SplitCfg<32, 4, 1>;

template <class Cfg, typename OUT>
__global__ void __launch_bounds__(Cfg::THREADS)
i8_split_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmQ, const I8GemmParams p,
                unsigned int *status) {
    constexpr int BN = Cfg::BN, STAGES = Cfg::STAGES, KB = Cfg::KB;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw_base);
    const uint32_t recv = base + STAGES * Cfg::SLOT;
    float *s_scale = reinterpret_cast<float *>(smem + STAGES * Cfg::SLOT + Cfg::RECV_BYTES);
    const uint32_t bars = recv + Cfg::RECV_BYTES + BN * 4;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (STAGES + s); };
    const uint32_t accf = bars + 8u * (2 * STAGES);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + (accf + 8u - base));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t S = static_cast<uint32_t>(p.split);
    const uint32_t rank = S > 1 ? cluster_rank() : 0u;
    const int tile = static_cast<int>(blockIdx.x / S);
    const int mt = tile / p.n_tiles;
    const int n0 = (tile - mt * p.n_tiles) * 128, m0 = mt * BN;
    const int num_sb = (p.num_kblk + KB - 1) / KB;   // slots of the whole reduction, and this CTA's share
    const int sb0 = static_cast<int>(1LL * num_sb * rank / S), sb1 = static_cast<int>(1LL * num_sb * (rank + 1) / S);
    const int cols = p.M - m0 < BN ? p.M - m0 : BN;   // tokens of this tile

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(accf, 1);
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmQ);
    }
    __syncthreads();
    // the peers' shared memory may be written once they have arrived here
    if (S > 1) cluster_arrive();
    if constexpr (BN == 16 || (BN == 32 && KB == 1)) {
        if (warp == 2) {
            const uint32_t leader = elect_one_sync();
            for (int sb = sb0; sb < sb1 && sb < sb0 + (KB > 1 ? 8 : 3); ++sb) {
                if (KB > 1 && p.wide) {
                    tma_prefetch_3d_if(&tmW, 0, n0, sb * KB, leader);
                } else {
#pragma unroll
                    for (int b = 0; b < KB; ++b) tma_prefetch_2d_if(&tmW, (sb * KB + b) * 128, n0, leader);
                }
            }
        }
    }
    grid_dependency_wait();
    grid_dependents_launch();

    if (warp == 0) {
        const uint32_t leader = elect_one_sync();
        bool ok = true;
        uint32_t s = 0, ph = 0;
        int issued = 0;
        for (int sb = sb0; sb < sb1; ++sb) {
            if (!mbar_wait_warp(empty(s), ph ^ 1u)) { ok = false; break; }
            const uint32_t slot = base + s * Cfg::SLOT;
            mbar_arrive_expect_tx_if(full(s), Cfg::SLOT, leader);
            if (KB > 1 && p.wide) {
                tma_load_3d_if(slot, &tmW, full(s), 0, n0, sb * KB, leader);
                tma_load_3d_if(slot + Cfg::W_BYTES, &tmQ, full(s), 0, m0, sb * KB, leader);
            } else {
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    tma_load_2d_if(slot + b * 128 * 128, &tmW, full(s), (sb * KB + b) * 128, n0, leader);
                    tma_load_2d_if(slot + Cfg::W_BYTES + b * BN * 128, &tmQ, full(s), (sb * KB + b) * 128, m0, leader);
                }
            }
            ++issued;
            if (++s == STAGES) { s = 0; ph ^= 1u; }
        }
        if (!ok && lane == 0) { atomicOr(status, kStatusTimeout); *abort_flag = 1; }
        // every copy has landed before the CTA may exit
        for (int j = issued > STAGES ? issued - STAGES : 0; j < issued; ++j)
            if (!mbar_wait_warp(full(j % STAGES), (j / STAGES) & 1)) {
                if (lane == 0) { atomicOr(status, kStatusTimeout); *abort_flag = 1; }
                break;
            }
    } else if (warp == 1) {
        tmem_alloc(smem_u32(tmem_holder), Cfg::TMEM_COLS);
        tmem_relinquish();
        __syncwarp();
        const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(tmem_holder);
        const uint32_t leader = elect_one_sync();
        bool ok = true;
        uint32_t s = 0, ph = 0;
        for (int sb = sb0; sb < sb1; ++sb) {
            if (!mbar_wait_warp(full(s), ph)) { ok = false; break; }
            tc_fence_after();
            const uint64_t a = smem_desc_sw128(base + s * Cfg::SLOT, 16, 1024);
            const uint64_t b = smem_desc_sw128(base + s * Cfg::SLOT + Cfg::W_BYTES, 16, 1024);
#pragma unroll
            for (int j = 0; j < 4 * KB; ++j)   // 32 bytes of k a step: +2 in the descriptors' 16-byte units
                umma_i8_ss_if(tmem_base, a + (j / 4) * 1024 + 2 * (j % 4), b + (j / 4) * (BN * 8) + 2 * (j % 4), Cfg::IDESC,
                              (sb > sb0 || j > 0) ? 1u : 0u, leader);
            umma_commit_if(empty(s), leader);
            if (++s == STAGES) { s = 0; ph ^= 1u; }
        }
        if (!ok && lane == 0) { atomicOr(status, kStatusTimeout); *abort_flag = 1; }
        umma_commit_if(accf, leader);
        // all MMAs are complete before TMEM is freed
        if (!mbar_wait_warp(accf, 0) && lane == 0) { atomicOr(status, kStatusTimeout); *abort_flag = 1; }
    } else {
        const int t = threadIdx.x - 64;
        for (int j = t; j < BN; j += 256)
            s_scale[j] = j < cols && in_bounds(m0 + j, 1, p.M, kSiteI8GemmScale, status) ? p.q_scale[m0 + j] : 0.0f;
        if (!mbar_wait_warp(accf, 0) && lane == 0) { atomicOr(status, kStatusTimeout); *abort_flag = 1; }
    }
    tc_fence_before();
    __syncthreads();   // also publishes s_scale and where TMEM starts
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;

    const int quarter = warp & 3;            // TMEM lanes of this warp (warps 2..9)
    const int eg = (warp - 2) >> 2;          // which of the quarter's two warps
    const int n_lane = quarter * 32 + lane;  // filter row inside the tile
    const int n = n0 + n_lane;
    const bool live = warp >= 2 && !*abort_flag;
    float ws = 0.0f, bias = 0.0f;
    const bool has_n = n < p.N;
    if (live && has_n && in_bounds(n, 1, p.N, kSiteI8GemmScale, status)) {
        ws = p.w_scale[n];
        if (p.bias) bias = p.bias[n];
    }
    const long long y_elems = 1LL * p.M * p.N;
    const long long y0 = 1LL * m0 * p.N + n;
    OUT *Y = static_cast<OUT *>(p.Y) + y0;
    // columns j .. j + NB - 1 of the tile: a warp stores 32 neighbouring channels of a token
    auto put = [&](int j, const int *acc, auto nb) {
        constexpr int NB = decltype(nb)::value;
        float v[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) v[i] = static_cast<float>(acc[i]) * s_scale[j + i];
#pragma unroll
        for (int i = 0; i < NB; ++i) v[i] = p.bias ? fmaf(v[i], ws, bias) : v[i] * ws;
#pragma unroll
        for (int i = 0; i < NB; ++i)
            if (has_n && j + i < cols && in_bounds(y0 + 1LL * (j + i) * p.N, 1, y_elems, kSiteI8GemmY, status))
                i8_out(Y + 1LL * (j + i) * p.N, v[i]);
    };
    const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    if (S > 1) cluster_wait();
    if (live) {
#pragma unroll 1
        for (int j0 = eg * 16; j0 < cols; j0 += 32) {
            uint32_t r[16];
            tmem_ld_32x32b_x16(t_row + j0, r);
            tmem_wait_ld();
            if (S == 1) {
                put(j0, reinterpret_cast<const int *>(r), I8Int<16>());
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const uint32_t col = static_cast<uint32_t>(j0 + j), to = col >> p.own_shift;
                    const uint32_t at = recv + (((rank << p.own_shift) + (col - (to << p.own_shift))) * 128 + n_lane) * 4;
                    if (j0 + j < cols) st_cluster_u32(map_rank(at, to), r[j]);
                }
            }
        }
    }
    if (S > 1) {
        cluster_sync_all();
        const int c0 = static_cast<int>(rank << p.own_shift), own = 1 << p.own_shift;   // columns this CTA owns
        if (live) {
            for (int j = 2 * eg; j < own && c0 + j < cols; j += 4) {
                int acc[2] = {0, 0};
                for (uint32_t r = 0; r < S; ++r) {
                    const uint32_t at = recv + (((r << p.own_shift) + j) * 128 + n_lane) * 4;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        int v;
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at + i * 512));
                        acc[i] += v;
                    }
                }
                put(c0 + j, acc, I8Int<2>());
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
}

// ---------------------------------------------------------------------------------------
// Many tokens: i8_pair_kernel
// ---------------------------------------------------------------------------------------
// A persistent CTA pair per 256 x BN tile of Y (M = 256, N = BN MMAs, cta_group::2): each CTA
// stages 128 token rows and BN / 2 filter rows per k block and receives its 128 tokens x BN columns
// of the accumulator. Two accumulators, so tile t + 1 multiplies while tile t is scaled and stored.
//   warp 0      TMA ring of STAGES slots
//   warp 1      TMEM allocation (after the dependency wait, as in the split kernel, while warp 0 issues
//               the first copies); the even CTA's issues the MMAs for both
//   warp 2      first asks L2 for the filter's first four blocks, which a launch behind the kernel
//               that quantises its rows does while that one runs (512 x 4096 x 4096 with the norm: 16.8
//               us without, 16.5 with; behind another product 11.3 and 11.2, and 11.4 with eight)
//   warps 2..17 epilogue, four warps per TMEM lane quarter with a quarter of the columns each, in
//               units of 64 bytes of output a row: tcgen05.ld, scale, round, swizzled staging, one
//               tensor store a unit. A warp has its columns' scales and biases fetched a tile ahead
//               and staged in its own corner of shared memory. With short reductions the epilogue
//               is the bound: 25088 x 512 outputs of 256 terms take 5.1 us without it, 11.6 us with
//               it. Its loop is kept short: unrolled over a tile's units, or with a second form of
//               the conversions, it takes 13 to 16 us, since a launch runs each instruction a few
//               times only and waits for the instruction cache.
template <int BN_, int STAGES_>
struct I8PairCfg {
    static constexpr int BN = BN_, STAGES = STAGES_;   // per CTA: 128 rows; the pair: 256
    static constexpr int NUM_EPI = 16;
    static constexpr int UNIT_BYTES = 32 * 64;           // staging of an epilogue warp: 64 bytes a row
    static constexpr int A_BYTES = 128 * 128, B_BYTES = BN / 2 * 128, SLOT = A_BYTES + B_BYTES;
    static constexpr int EPI_BYTES = NUM_EPI * UNIT_BYTES;
    static constexpr int COLS = BN / 4;                  // columns of an epilogue warp
    static constexpr int SCALE_BYTES = NUM_EPI * COLS * 8;   // their scales and biases
    static constexpr int NUM_BARS = 2 * STAGES + 4 + 1;
    static constexpr int SMEM = 1024 + STAGES * SLOT + EPI_BYTES + SCALE_BYTES + NUM_BARS * 8 + 16;
    static constexpr int THREADS = 32 * (2 + NUM_EPI);
    static constexpr uint32_t IDESC = idesc_i8_s32(256, BN);
    static_assert(SMEM <= 232448, "shared memory of one CTA");
};

constexpr int kI8Group = 8;   // row tiles walked together

// Tile t of the walk: GROUP row tiles together, so that the CTAs in flight share their operands
// in L2 (74 pairs in flight hold about 8 x 9 tiles).
__device__ __forceinline__ void i8_tile(int t, int m_tiles, int n_tiles, int &mt, int &nt) {
    const int per = kI8Group * n_tiles;
    const int g = t / per, r = t - g * per;
    const int m_first = g * kI8Group;
    const int h = m_tiles - m_first < kI8Group ? m_tiles - m_first : kI8Group;
    nt = r / h;
    mt = m_first + (r - nt * h);
}

template <class Cfg, typename OUT>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
i8_pair_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmW,
               const __grid_constant__ CUtensorMap tmY, const I8GemmParams p, unsigned int *status) {
    grid_dependents_launch();
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw_base);
    constexpr uint32_t epi_off = Cfg::STAGES * Cfg::SLOT;
    constexpr uint32_t scale_off = epi_off + Cfg::EPI_BYTES;
    const uint32_t bars = base + scale_off + Cfg::SCALE_BYTES;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (Cfg::STAGES + s); };
    auto accf = [&](int b) { return bars + 8u * (2 * Cfg::STAGES + b); };
    auto acce = [&](int b) { return bars + 8u * (2 * Cfg::STAGES + 2 + b); };
    const uint32_t done_bar = bars + 8u * (2 * Cfg::STAGES + 4);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + scale_off + Cfg::SCALE_BYTES + Cfg::NUM_BARS * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    auto lead = [&](uint32_t a) { return map_rank(a, 0u); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < Cfg::STAGES; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf(b), 1);
            mbar_init(acce(b), 2 * Cfg::NUM_EPI);   // one arrival per epilogue warp of both CTAs
        }
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmW);
        if (p.vec) prefetch_tensormap(&tmY);
    }
    __syncthreads();
    cluster_sync_all();   // both CTAs' barriers exist before either is used
    // Both CTAs' TMEM exists before either is used: warp 1 arrives once it has it, the others here, and
    // those that use TMEM wait for that (warp 0 after its copies).
    if (warp != 1) cluster_arrive();
    if (warp == 2 && static_cast<int>(blockIdx.x >> 1) < p.num_tiles) {   // its first filter blocks into L2
        const uint32_t leader = elect_one_sync();
        int mt, nt;
        i8_tile(static_cast<int>(blockIdx.x >> 1), p.m_tiles, p.n_tiles, mt, nt);
        for (int kb = 0; kb < p.num_kblk && kb < 4; ++kb)
            tma_prefetch_2d_if(&tmW, kb * 128, nt * Cfg::BN + static_cast<int>(rank) * (Cfg::BN / 2), leader);
    }
    grid_dependency_wait();
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_holder), 2 * Cfg::BN);
        tmem_relinquish_pair();
        tc_fence_before();
        cluster_arrive();
    }
    auto tmem_ready = [&]() {
        cluster_wait();
        tc_fence_after();
        return *reinterpret_cast<volatile uint32_t *>(tmem_holder);
    };
    uint32_t tmem_base = 0;

    auto fail = [&]() {
        atomicOr(status, kStatusTimeout);
        *abort_flag = 1;
        st_cluster_u32(map_rank(smem_u32(const_cast<int *>(abort_flag)), rank ^ 1u), 1u);
    };
    const int first = static_cast<int>(blockIdx.x >> 1), step = static_cast<int>(gridDim.x >> 1);

    if (warp == 0) {
        const uint32_t leader = elect_one_sync();
        uint32_t it = 0, s = 0, ph = 0;
        bool ok = true;
        for (int t = first; t < p.num_tiles && ok && !*abort_flag; t += step) {
            int mt, nt;
            i8_tile(t, p.m_tiles, p.n_tiles, mt, nt);
            const int row_q = mt * 256 + static_cast<int>(rank) * 128, row_w = nt * Cfg::BN + static_cast<int>(rank) * (Cfg::BN / 2);
            for (int kb = 0; kb < p.num_kblk; ++kb, ++it) {
                if (!mbar_wait_warp(empty(s), ph ^ 1u)) { ok = false; break; }
                const uint32_t slot = base + s * Cfg::SLOT;
                mbar_arrive_expect_tx_if(full(s), 2 * Cfg::SLOT, leader & (rank ^ 1u));   // both CTAs' copies
                tma_load_2d_pair_if(slot, &tmQ, lead(full(s)), kb * 128, row_q, leader);
                tma_load_2d_pair_if(slot + Cfg::A_BYTES, &tmW, lead(full(s)), kb * 128, row_w, leader);
                if (++s == Cfg::STAGES) { s = 0; ph ^= 1u; }
            }
        }
        if (!ok && lane == 0) fail();
        // drain: every copy issued has been consumed (the even CTA's commits report to both)
        for (uint32_t j = it > (uint32_t)Cfg::STAGES ? it - Cfg::STAGES : 0u; j < it; ++j)
            if (!mbar_wait_warp(empty(j % Cfg::STAGES), (j / Cfg::STAGES) & 1u)) { if (lane == 0) fail(); break; }
        __syncwarp();
        cluster_wait();
    } else if (warp == 1) {
        tmem_base = tmem_ready();
        const uint32_t leader = elect_one_sync();
        constexpr uint16_t kBoth = 0x3;
        if (rank == 0) {
            uint32_t local = 0, s = 0, ph = 0;
            bool ok = true;
            const uint64_t a0 = smem_desc_sw128(base, 16, 1024);
            const uint64_t b0 = smem_desc_sw128(base + Cfg::A_BYTES, 16, 1024);
            for (int t = first; t < p.num_tiles && ok && !__any_sync(0xffffffffu, *abort_flag != 0); t += step, ++local) {
                const uint32_t b = local & 1u;
                if (!mbar_wait_warp(acce(b), ((local >> 1) & 1u) ^ 1u)) { ok = false; break; }
                tc_fence_after();
                const uint32_t d = tmem_base + b * Cfg::BN;
                for (int kb = 0; kb < p.num_kblk; ++kb) {
                    if (!mbar_wait_warp(full(s), ph)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t ad = a0 + s * (Cfg::SLOT >> 4), bd = b0 + s * (Cfg::SLOT >> 4);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        umma_i8_ss_pair_if(d, ad + 2 * j, bd + 2 * j, Cfg::IDESC, (kb > 0 || j > 0) ? 1u : 0u, leader);
                    umma_commit_pair_if(empty(s), kBoth, leader);
                    if (++s == Cfg::STAGES) { s = 0; ph ^= 1u; }
                }
                if (!ok) break;
                umma_commit_pair_if(accf(b), kBoth, leader);
            }
            __syncwarp();
            if (!ok && lane == 0) fail();
            // all MMAs complete before TMEM is released
            umma_commit_pair_if(done_bar, kBoth, leader);
            if (!mbar_wait_warp(done_bar, 0) && lane == 0) fail();
        }
    } else {
        constexpr int UW = 64 / static_cast<int>(sizeof(OUT));    // columns of a unit
        constexpr int UNITS = Cfg::COLS / UW;
        constexpr int V = 16 / static_cast<int>(sizeof(OUT));     // values of 16 bytes
        const int quarter = warp & 3, eg = (warp - 2) >> 2;
        const uint32_t stage = base + epi_off + (warp - 2) * Cfg::UNIT_BYTES;
        float *s_ws = reinterpret_cast<float *>(smem + scale_off) + (warp - 2) * 2 * Cfg::COLS;   // scales, then biases
        float *s_bias = s_ws + Cfg::COLS;
        OUT *Y = static_cast<OUT *>(p.Y);
        const long long y_elems = 1LL * p.M * p.N;
        auto swizzle = [](int row) { return (row >> 1) & 3; };   // of the 16-byte pieces of a 64-byte row
        const uint32_t leader = elect_one_sync();
        // The scales of a tile: the lane's row, and the warp's columns 32 at a time. They are fetched a
        // tile ahead.
        float qs_next = 0.0f, ws_next[Cfg::COLS / 32], bias_next[Cfg::COLS / 32];
        auto fetch = [&](int t) {
            int mt, nt;
            i8_tile(t, p.m_tiles, p.n_tiles, mt, nt);
            const int row = mt * 256 + static_cast<int>(rank) * 128 + quarter * 32 + lane;
            qs_next = row < p.M && in_bounds(row, 1, p.M, kSiteI8GemmScale, status) ? p.q_scale[row] : 0.0f;
#pragma unroll
            for (int i = 0; i < Cfg::COLS / 32; ++i) {
                const int c = nt * Cfg::BN + eg * Cfg::COLS + i * 32 + lane;
                const bool in = c < p.N && in_bounds(c, 1, p.N, kSiteI8GemmScale, status);
                ws_next[i] = in ? p.w_scale[c] : 0.0f;
                bias_next[i] = in && p.bias ? p.bias[c] : 0.0f;
            }
        };
        if (first < p.num_tiles) fetch(first);
        tmem_base = tmem_ready();
        uint32_t local = 0;
        for (int t = first; t < p.num_tiles; t += step, ++local) {
            if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
            const uint32_t b = local & 1u;
            int mt, nt;
            i8_tile(t, p.m_tiles, p.n_tiles, mt, nt);
            const int row0 = mt * 256 + static_cast<int>(rank) * 128 + quarter * 32;   // this warp's 32 rows
            const int n0 = nt * Cfg::BN + eg * Cfg::COLS;                              // its columns
            const uint64_t qs = f2_pack(qs_next, qs_next);
            __syncwarp();   // the previous tile's scales have been read
#pragma unroll
            for (int i = 0; i < Cfg::COLS / 32; ++i) {
                s_ws[i * 32 + lane] = ws_next[i];
                s_bias[i * 32 + lane] = bias_next[i];
            }
            __syncwarp();
            if (t + step < p.num_tiles) fetch(t + step);
            if (!mbar_wait_backoff(accf(b), (local >> 1) & 1u, 32)) { if (lane == 0) fail(); break; }
            tc_fence_after();
            const uint32_t t_row =
                tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + b * Cfg::BN + eg * Cfg::COLS;
#pragma unroll 1
            for (int u = 0; u < UNITS; ++u) {
                const int c0 = n0 + u * UW;
                uint32_t r[UW];
#pragma unroll
                for (int g = 0; g < UW / 16; ++g)
                    tmem_ld_32x32b_x16(t_row + u * UW + g * 16, *reinterpret_cast<uint32_t(*)[16]>(r + g * 16));
                tmem_wait_ld();
                if (u + 1 == UNITS) {   // the accumulator is read: the next tile but one may have it
                    tc_fence_before();
                    __syncwarp();
                    mbar_arrive_cluster_if(lead(acce(b)), leader);
                }
                uint64_t v[UW / 2];
#pragma unroll
                for (int i = 0; i < UW / 2; ++i)
                    v[i] = f2_pack(static_cast<float>(static_cast<int>(r[2 * i])), static_cast<float>(static_cast<int>(r[2 * i + 1])));
                // (the sum times its token's scale) times its channel's plus the bias: two roundings with the
                // conversion's, one more for the fused last step, as in the split kernel
#pragma unroll
                for (int i = 0; i < UW / 4; ++i) {
                    const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(s_ws + u * UW + i * 4);
                    v[2 * i] = f2_mul(v[2 * i], qs);
                    v[2 * i + 1] = f2_mul(v[2 * i + 1], qs);
                    if (p.bias) {
                        const ulonglong2 bb = *reinterpret_cast<const ulonglong2 *>(s_bias + u * UW + i * 4);
                        v[2 * i] = f2_fma(v[2 * i], w.x, bb.x);
                        v[2 * i + 1] = f2_fma(v[2 * i + 1], w.y, bb.y);
                    } else {
                        v[2 * i] = f2_mul(v[2 * i], w.x);
                        v[2 * i + 1] = f2_mul(v[2 * i + 1], w.y);
                    }
                }
                bulk_wait_group_read0();   // the previous unit has left the staging (the leader's store)
                __syncwarp();
                // 16-byte pieces of the lane's 64-byte row, 64-byte swizzle
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float lo, hi;
                        if constexpr (sizeof(OUT) == 2) {
                            f2_split(v[4 * c + j], lo, hi);
                            o[j] = halo_pack_bf16x2(lo, hi);
                        } else {
                            f2_split(v[2 * c + j / 2], lo, hi);
                            o[j] = __float_as_uint(j & 1 ? hi : lo);
                        }
                    }
                    st_shared_v4(stage + lane * 64 + ((c ^ swizzle(lane)) << 4), o[0], o[1], o[2], o[3]);
                }
                if (p.vec) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    // rows and columns past Y are not stored
                    tma_store_2d_commit_if(&tmY, stage, c0, row0, c0 < p.N && row0 < p.M ? leader : 0u);
                } else {   // rows of Y off the 16-byte boundaries: an element a lane
                    __syncwarp();
                    const uint8_t *from = smem + (stage - base);
                    const int rows = p.M - row0 < 32 ? p.M - row0 : 32;
                    constexpr int RPI = 32 / UW;   // rows an instruction
                    const int e = lane % UW, col = c0 + e;
#pragma unroll 4
                    for (int rr = lane / UW; rr < rows; rr += RPI) {
                        const long long at = 1LL * (row0 + rr) * p.N + col;
                        if (col < p.N && in_bounds(at, 1, y_elems, kSiteI8GemmY, status))
                            Y[at] = *reinterpret_cast<const OUT *>(from + rr * 64 + (((e / V) ^ swizzle(rr)) << 4) +
                                                                   (e % V) * sizeof(OUT));
                    }
                    __syncwarp();
                }
            }
        }
        bulk_wait_group_read0();   // the stores have left shared memory before the CTA exits
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();   // neither CTA leaves while the other may still signal its barriers
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem_base, 2 * Cfg::BN);
}

}  // namespace convb200
