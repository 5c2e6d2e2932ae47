// The 8-bit entry points: argument checks, kernel choice, tensor maps, launches. Included at the
// end of capi.cu, whose helpers (device state, launch_k, pointer checks) it uses.
#pragma once

#include <cmath>

namespace convb200 {
namespace {

constexpr int kI8MaxReduce = 131071;   // (131071 + 1) * 128 * 128 = 2^31: the int32 sums are exact below
constexpr int kI8MaxCols = 1 << 27;    // of a quantised row: indices past the row's last piece stay in int
constexpr int kI8MaxRows = 2147483647 - 512;   // of a product and its filter: so do a last tile's rows

constexpr int kI8StagedMax = 220 * 1024;   // bytes of a row in the shared memory of a block that has an SM alone

int i8_elem(int dtype) { return dtype == CONV_F32 ? 4 : 2; }

// Bytes from the first to past the last value of `rows` rows of C bytes, ld apart.
long long i8_extent(long long rows, int C, int ld) { return (rows - 1) * ld + C; }

int check_i8_rows(const void *q, int C, int ld) {
    if (ld < C) return CONV_ERR_INVALID_ARG;
    if (ld % 16 != 0 || !aligned(q, 16)) return CONV_ERR_MISALIGNED;
    return CONV_OK;
}

// ---- rows ------------------------------------------------------------------------------
template <typename T, int MODE, int NV, bool VEC, int TPR, int RW, bool STREAM>
int launch_i8_rows(const I8RowsParams &p, int threads, cudaStream_t stream, DeviceState *d) {
    const long long per = TPR == 32 ? threads / 32 * RW : 1, blocks = (p.M + per - 1) / per;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = stream;
    return launched(launch_k(cfg, i8_rows_kernel<T, MODE, NV, VEC, TPR, RW, STREAM>, p, d->status), "i8_rows_kernel");
}

template <typename T, int MODE, int TPR>
int launch_i8_staged(const I8RowsParams &p, int bytes, cudaStream_t stream, DeviceState *d) {
    auto kern = i8_rows_staged_kernel<T, MODE, TPR>;
    constexpr unsigned bit = 160 + (sizeof(T) == 4 ? 12 : 0) + MODE * 3 + (TPR == 128 ? 0 : TPR == 256 ? 1 : 2);
    if (int rc = ensure_smem_attr(d, bit, kern, kI8StagedMax)) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.M));
    cfg.blockDim = dim3(TPR);
    cfg.dynamicSmemBytes = static_cast<size_t>(bytes);
    cfg.stream = stream;
    return launched(launch_k(cfg, kern, p, d->status), "i8_rows_staged_kernel");
}

template <typename T, int MODE>
int run_i8_rows(const I8RowsParams &p, cudaStream_t stream, DeviceState *d) {
    // A warp holds rows up to 1024 values (two rows of up to 512: 25088 x 256 took 6.9 us with one,
    // 4.9 with two, 5.0 with four; 48000 x 512 15.6, 14.5 and 17.0), a block of up to 512 threads rows
    // up to 16384. Four groups a thread where a group is one load or the norm's sums keep few blocks
    // in flight (8192 x 4096 with a residual 42 us with two, 38 with four); two for the gate, whose
    // arithmetic they do not hide (4096 x 4096: 16.5 us with four, 14.5 with two).
    const int C = p.C;
    if (C % 8 == 0 && aligned(p.x, 16) && aligned(p.residual, 16) && aligned(p.h, 16) && aligned(p.weight, 16)) {
        if (C <= 256) return launch_i8_rows<T, MODE, 1, true, 32, 2, false>(p, 128, stream, d);
        if (C <= 512) return launch_i8_rows<T, MODE, 2, true, 32, 2, false>(p, 128, stream, d);
        if (C <= 1024) return launch_i8_rows<T, MODE, 4, true, 32, 1, false>(p, 128, stream, d);
        if constexpr (MODE == kI8Glu) {
            if (C <= 8192)
                return launch_i8_rows<T, MODE, 2, true, 0, 1, false>(p, (C + 511) / 512 * 32, stream, d);
            // bf16: three groups (52 registers a thread, allocated as 56) unless four (64) let more rows be on
            // an SM: 8192 x 9216 59.6 us with three and 66.0 with four, 8192 x 10240 78.0 and 70.3, 8192 x
            // 12288 84.5 and 92.7. In float32 three take as many registers as four: 8192 x 9216 113.5 and
            // 97.4, 8192 x 12288 131 and 131
            if constexpr (sizeof(T) == 2) {
                const int threads = (C + 767) / 768 * 32, threads4 = (C + 1023) / 1024 * 32;
                if (C <= 12288 && 65536 / (threads * 56) >= 65536 / (threads4 * 64))
                    return launch_i8_rows<T, MODE, 3, true, 0, 1, false>(p, threads, stream, d);
            }
        }
        if (C <= 16384) return launch_i8_rows<T, MODE, 4, true, 0, 1, false>(p, (C + 1023) / 1024 * 32, stream, d);
        return launch_i8_rows<T, MODE, 4, true, 0, 1, true>(p, 512, stream, d);
    }
    // Element by element: in registers up to 2048 values (8192 x 901: 16.4 us with 128 threads a row, 11.4
    // with a warp), in float32 up to 8192 (1031 x 5003 with a norm 8.5 us, staged 10.6; with a residual 14.5 and 17.0;
    // two inputs at four groups a thread would take too many registers); beyond that staged (bf16: 8192 x
    // 4095 30.4 us in registers, 20.3 staged; 4096 x 12343 77.6 streamed, 28.0 staged), in float32 while two
    // blocks fit on an SM (1024 x 17001 27.6 us streamed, 17.2 staged; 1024 x 30001 38.2 and 41.3), in bf16
    // while one does (1024 x 60001 82.6 and 50.7).
    if (C <= 512) return launch_i8_rows<T, MODE, 2, false, 32, 1, false>(p, 128, stream, d);
    if (C <= 1024) return launch_i8_rows<T, MODE, 4, false, 32, 1, false>(p, 128, stream, d);
    if (C <= 2048) return launch_i8_rows<T, MODE, 2, false, 128, 1, false>(p, 128, stream, d);
    if constexpr (sizeof(T) == 4) {
        if (C <= 4096) return launch_i8_rows<T, MODE, 2, false, 256, 1, false>(p, 256, stream, d);
        if (C <= 6144) {   // 4096 x 4097 to 6143 with a norm: 29.0 to 31.1 us in the slots of 8192, 22.3 to 24.6 in those of 6144
            if constexpr (MODE == kI8Plain || MODE == kI8Norm) return launch_i8_rows<T, MODE, 3, false, 256, 1, false>(p, 256, stream, d);
            else return launch_i8_rows<T, MODE, 2, false, 384, 1, false>(p, 384, stream, d);
        }
        if (C <= 8192) {
            if constexpr (MODE == kI8Plain || MODE == kI8Norm) return launch_i8_rows<T, MODE, 4, false, 256, 1, false>(p, 256, stream, d);
            else return launch_i8_rows<T, MODE, 2, false, 512, 1, false>(p, 512, stream, d);
        }
    }
    const long long bytes = 1LL * i8_staged_bytes<T>(MODE == kI8Glu ? 2 * C : C) * (MODE == kI8NormResidual ? 2 : 1);
    if (bytes <= (sizeof(T) == 4 ? kI8StagedMax / 2 : kI8StagedMax)) {
        const int n = static_cast<int>(bytes);
        if constexpr (sizeof(T) == 2)
            if (C <= 4096) return launch_i8_staged<T, MODE, 128>(p, n, stream, d);
        if (C <= 16384) return launch_i8_staged<T, MODE, 256>(p, n, stream, d);
        return launch_i8_staged<T, MODE, 512>(p, n, stream, d);
    }
    return launch_i8_rows<T, MODE, 2, false, 512, 1, true>(p, 512, stream, d);
}

template <int MODE>
int run_i8_rows(const I8RowsParams &p, int dtype, cudaStream_t stream, DeviceState *d) {
    return dtype == CONV_F32 ? run_i8_rows<float, MODE>(p, stream, d) : run_i8_rows<__nv_bfloat16, MODE>(p, stream, d);
}

// ---- filter ------------------------------------------------------------------------------
template <typename T, bool VEC>
int launch_i8_filter(const I8FilterParams &p, int S, cudaStream_t stream, DeviceState *d, unsigned bit) {
    auto kern = i8_filter_kernel<T, VEC>;
    if (int rc = ensure_smem_attr(d, bit, kern, 200 * 1024)) return rc;
    const long long ctas = 1LL * ((p.Cout + kI8FilterCols - 1) / kI8FilterCols) * S;
    if (ctas > kInt32Max) return CONV_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(S);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = static_cast<size_t>(i8_filter_smem(p.piece, sizeof(T)));
    cfg.stream = stream;
    return launched(launch_k(cfg, kern, p, d->status), "i8_filter_kernel");
}

template <typename T>
int run_i8_filter(I8FilterParams p, cudaStream_t stream, DeviceState *d) {
    // 512 rows a CTA (a quarter of an SM's shared memory in bf16), fewer while there are not two CTAs
    // an SM, more beyond 4096: 1024 x 16384 in bf16 took 41.6 us with 128 rows each, 17.9 with 512. A
    // share up to a whole SM's shared memory is read once; a longer one in pieces of a quarter, twice.
    const int tiles = (p.Cin + 127) / 128, blocks = (p.Cout + kI8FilterCols - 1) / kI8FilterCols;
    int S = 1;
    while (S < 8 && S < tiles && (tiles > 4 * S || 1LL * blocks * S < 2 * d->num_sms)) S *= 2;
    p.share = (tiles + S - 1) / S * 128;
    constexpr int tile_bytes = i8_filter_smem(128, sizeof(T));
    const int quarter = 54 * 1024 / tile_bytes * 128, all = 200 * 1024 / tile_bytes * 128;
    p.piece = p.share <= all ? p.share : quarter;
    const bool vec = p.Cout % 8 == 0 && aligned(p.F, 16);
    constexpr unsigned bit = sizeof(T) == 4 ? 130 : 128;
    return vec ? launch_i8_filter<T, true>(p, S, stream, d, bit) : launch_i8_filter<T, false>(p, S, stream, d, bit + 1);
}

// ---- product -----------------------------------------------------------------------------
// A matrix of 8-bit rows in boxes of 128 values x `box_rows` rows, 128-byte swizzle; with kb > 1 the
// values are split into blocks of 128 (C a multiple of 128) and a box has kb of them.
int i8_map(CUtensorMap *m, const int8_t *q, int rows, int C, int ld, int box_rows, int kb = 1) {
    const cuuint64_t dims[3] = {kb > 1 ? 128u : (cuuint64_t)C, (cuuint64_t)rows, (cuuint64_t)C / 128};
    const cuuint64_t strides[2] = {(cuuint64_t)ld, 128};
    const cuuint32_t box[3] = {128, (cuuint32_t)box_rows, (cuuint32_t)kb};
    const cuuint32_t estr[3] = {1, 1, 1};
    return g_encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, kb > 1 ? 3 : 2, const_cast<int8_t *>(q), dims, strides, box,
                          estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? CONV_OK
               : CONV_ERR_CUDA;
}

struct I8Operands {
    const int8_t *q, *Wq;
    int Cin, ldq, ldw;
};

template <class Cfg, typename OUT>
int launch_i8_split(const I8Operands &a, I8GemmParams p, int split, cudaStream_t stream, DeviceState *d, unsigned bit) {
    auto kern = i8_split_kernel<Cfg, OUT>;
    if (int rc = ensure_smem_attr(d, bit, kern, Cfg::SMEM)) return rc;
    CUtensorMap tmW, tmQ;
    p.wide = Cfg::KB > 1 && a.Cin % 128 == 0;
    if (int rc = i8_map(&tmW, a.Wq, p.N, a.Cin, a.ldw, 128, p.wide ? Cfg::KB : 1)) return rc;
    if (int rc = i8_map(&tmQ, a.q, p.M, a.Cin, a.ldq, Cfg::BN, p.wide ? Cfg::KB : 1)) return rc;
    p.n_tiles = (p.N + 127) / 128;
    p.m_tiles = (p.M + Cfg::BN - 1) / Cfg::BN;
    p.split = split;
    p.own_shift = 0;
    while ((Cfg::BN >> (p.own_shift + 1)) >= split) ++p.own_shift;   // BN / split, powers of two
    const long long ctas = 1LL * p.n_tiles * p.m_tiles * split;
    if (ctas > kInt32Max) return CONV_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(Cfg::THREADS);
    cfg.dynamicSmemBytes = Cfg::SMEM;
    cfg.stream = stream;
    if (split > 1) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(split);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return launched(launch_k(cfg, kern, tmW, tmQ, p, d->status), "i8_split_kernel");
}

template <class Cfg, typename OUT>
int launch_i8_pair(const I8Operands &a, I8GemmParams p, cudaStream_t stream, DeviceState *d, unsigned bit) {
    auto kern = i8_pair_kernel<Cfg, OUT>;
    if (int rc = ensure_smem_attr(d, bit, kern, Cfg::SMEM)) return rc;
    CUtensorMap tmQ, tmW, tmY;
    if (int rc = i8_map(&tmQ, a.q, p.M, a.Cin, a.ldq, 128)) return rc;
    if (int rc = i8_map(&tmW, a.Wq, p.N, a.Cin, a.ldw, Cfg::BN / 2)) return rc;
    if (p.vec) {   // Y in boxes of 32 rows x 64 bytes
        const cuuint64_t dims[2] = {(cuuint64_t)p.N, (cuuint64_t)p.M};
        const cuuint64_t strides[1] = {(cuuint64_t)p.N * sizeof(OUT)};
        const cuuint32_t box[2] = {64 / (cuuint32_t)sizeof(OUT), 32};
        const cuuint32_t estr[2] = {1, 1};
        if (g_encode_tiled(&tmY, sizeof(OUT) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
                           p.Y, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                           CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return CONV_ERR_CUDA;
    } else {
        tmY = tmQ;   // not used
    }
    p.m_tiles = (p.M + 255) / 256;
    p.n_tiles = (p.N + Cfg::BN - 1) / Cfg::BN;
    p.split = 1;
    const long long tiles = 1LL * p.m_tiles * p.n_tiles;
    if (tiles > kInt32Max / 2) return CONV_ERR_UNSUPPORTED;
    p.num_tiles = static_cast<int>(tiles);
    const int fit = cluster_fit(d, bit, kern, 2, Cfg::SMEM, Cfg::THREADS);
    if (fit < 1) return CONV_ERR_CUDA;
    const int pairs = p.num_tiles < fit ? p.num_tiles : fit;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(Cfg::THREADS);
    cfg.dynamicSmemBytes = Cfg::SMEM;
    cfg.stream = stream;
    return launched(launch_k(cfg, kern, tmQ, tmW, tmY, p, d->status), "i8_pair_kernel");
}

// The kernel for a product: the pair kernel's tile width, or the split kernel's token columns and its
// split of the reduction.
struct I8Plan {
    bool pair;
    int bn, split;
};

// k blocks of a slot of the split kernel: two, but for the widest tile and the short ring.
constexpr int i8_slot_kblks(int bn, bool shared) { return bn == 128 || shared ? 1 : 2; }

// Whether the split kernel runs with its short ring, two CTAs on an SM.
bool i8_shared(int bn, long long ctas, int num_kblk, int split, int num_sms) {
    return bn <= 32 && (ctas > num_sms || num_kblk <= 8 * split);
}

// Picks the plan whose estimated time (us) is least. The estimate is a start (launch, first copies;
// again for each further round of CTAs), an epilogue per round, and the larger-than-either sum (hypot) of the k loop and of the
// bytes at HBM's rate; a k block takes its own time or what its copies take when every SM's go
// through L2. The constants are a fit to 2200 measured times on a B200, M 1 .. 2048, N 1024 .. 20480,
// Cin 512 .. 10240 (rms error 10 %; the plan it picks is on average 1 % slower than the best one
// measured, the fixed rule it replaced 10 %). Both sides at their limits: 128 x 4096 x 4096 (M, N,
// Cin) 8.3 us in 32-column tiles, 9.4 in 64 and 10.9 by pairs; 256 x 20480 x 4096 26.5 us by pairs
// of 128, 29.1 by pairs of 256 and 39.0 split; 1 x 4096 x 10240 10.3 us split in 4, 13.3 unsplit.
// clusters(bn, S): how many clusters of S CTAs the device holds at once.
template <class Clusters>
I8Plan plan_i8(int M, int N, int num_kblk, int num_sms, Clusters clusters) {
    // CONV_B200_I8 (tests): "pair,BN", or "split,BN,S"
    if (const char *f = env("CONV_B200_I8")) {
        int bn = 0, s = 0;
        if (std::sscanf(f, "pair,%d", &bn) == 1 && (bn == 128 || bn == 256)) return I8Plan{true, bn, 1};
        if (std::sscanf(f, "split,%d,%d", &bn, &s) == 2 && (bn == 16 || bn == 32 || bn == 64 || bn == 128) &&
            (s == 1 || s == 2 || s == 4 || s == 8) && s <= (num_kblk + 1) / 2)
            return I8Plan{false, bn, s};
    }
    auto cdiv = [](long long a, long long b) { return (a + b - 1) / b; };
    const float mbytes = (static_cast<float>(M) + N) * num_kblk * 128e-6f + 2e-6f * M * N;
    const float l2 = 128 / 19.8e6f;   // us a row of 128 bytes through L2
    I8Plan best{true, 256, 1};
    float least = 3.4e38f;
    for (int bn = 256; bn >= 128; bn /= 2) {
        const long long tiles = cdiv(M, 256) * cdiv(N, bn), pairs = tiles < num_sms / 2 ? tiles : num_sms / 2;
        const float rounds = static_cast<float>(cdiv(tiles, num_sms / 2));
        const float kblk = fmaxf(bn == 256 ? 0.293f : 0.174f, l2 * pairs * (256 + bn));
        const float t = 3.4f + rounds * (bn == 256 ? 2.3f : 1.5f) + hypotf(rounds * num_kblk * kblk, mbytes / 10.2f);
        if (t < least) {
            least = t;
            best = I8Plan{true, bn, 1};
        }
    }
    if (M > 512) return best;
    for (int bn = 128; bn >= 16; bn /= 2) {
        if (bn >= 2 * M && bn > 16) continue;   // half of the columns and more would be empty
        const long long tiles = cdiv(M, bn) * cdiv(N, 128);
        const float cols = static_cast<float>(bn < M ? bn : M);
        for (int S = 1; S <= 8; S *= 2) {
            const long long ctas = tiles * S;
            // a split that does not run at once only adds to the work
            if (S > 1 && (ctas > num_sms || 2 * S > num_kblk)) break;
            const int kb = i8_slot_kblks(bn, i8_shared(bn, ctas, num_kblk, S, num_sms));
            const float rounds = static_cast<float>(cdiv(ctas, num_sms));
            const float share = static_cast<float>(cdiv(cdiv(num_kblk, kb), S) * kb);
            const float own = bn == 128 ? 0.177f : bn == 64 ? 0.132f : bn == 32 ? 0.121f : 0.135f;
            const float kblk = fmaxf(own, l2 * (ctas < num_sms ? ctas : num_sms) * (128 + bn));
            const float t = 0.5f + 1.5f * rounds + rounds * (0.019f * cols + (S > 1 ? 0.62f + 0.013f * cols : 0.0f)) +
                            hypotf(rounds * share * kblk, mbytes / 5.9f);
            if (t < least && (S == 1 || tiles <= clusters(bn, S))) {
                least = t;
                best = I8Plan{false, bn, S};
            }
        }
    }
    return best;
}

template <class Cfg, typename OUT>
int i8_split_clusters(DeviceState *d, unsigned bit, int S) {
    auto kern = i8_split_kernel<Cfg, OUT>;
    if (ensure_smem_attr(d, bit, kern, Cfg::SMEM)) return 0;
    return cluster_fit(d, bit, kern, S, Cfg::SMEM, Cfg::THREADS);
}

template <typename OUT>
int run_i8_product(const I8Operands &a, I8GemmParams p, cudaStream_t stream, DeviceState *d) {
    constexpr unsigned bit = sizeof(OUT) == 4 ? 148 : 132;
    using Split16 = I8SplitCfg<16, 6, i8_slot_kblks(16, false)>;
    using Split32 = I8SplitCfg<32, 5, i8_slot_kblks(32, false)>;
    using Split64 = I8SplitCfg<64, 4, i8_slot_kblks(64, false)>;
    using Split128 = I8SplitCfg<128, 5, i8_slot_kblks(128, false)>;
    p.num_kblk = (a.Cin + 127) / 128;
    p.vec = aligned(p.Y, 16) && (1LL * p.N * sizeof(OUT)) % 16 == 0;
    const I8Plan pl = plan_i8(p.M, p.N, p.num_kblk, d->num_sms, [&](int bn, int S) {
        return bn == 16 ? i8_split_clusters<Split16, OUT>(d, bit + 2, S) : bn == 32 ? i8_split_clusters<Split32, OUT>(d, bit + 4, S)
             : bn == 64 ? i8_split_clusters<Split64, OUT>(d, bit + 6, S) : i8_split_clusters<Split128, OUT>(d, bit + 7, S);
    });
    if (pl.pair)
        return pl.bn == 256 ? launch_i8_pair<I8PairCfg<256, 5>, OUT>(a, p, stream, d, bit)
                            : launch_i8_pair<I8PairCfg<128, 7>, OUT>(a, p, stream, d, bit + 1);
    const bool shared = i8_shared(pl.bn, 1LL * ((p.N + 127) / 128) * ((p.M + pl.bn - 1) / pl.bn) * pl.split, p.num_kblk,
                                  pl.split, d->num_sms);
    switch (pl.bn) {
        case 16:
            return shared ? launch_i8_split<I8ShortSplit16, OUT>(a, p, pl.split, stream, d, bit + 3)
                          : launch_i8_split<Split16, OUT>(a, p, pl.split, stream, d, bit + 2);
        case 32:
            return shared ? launch_i8_split<I8ShortSplit32, OUT>(a, p, pl.split, stream, d, bit + 5)
                          : launch_i8_split<Split32, OUT>(a, p, pl.split, stream, d, bit + 4);
        case 64: return launch_i8_split<Split64, OUT>(a, p, pl.split, stream, d, bit + 6);
        default: return launch_i8_split<Split128, OUT>(a, p, pl.split, stream, d, bit + 7);
    }
}

int check_pointwise_i8(const int8_t *q, const float *q_scale, const int8_t *Wq, const float *w_scale, const float *bias,
                       const void *Y, int M, int Cin, int Cout, int ldq, int ldw, int dtype) {
    if (!q || !q_scale || !Wq || !w_scale || !Y) return CONV_ERR_INVALID_ARG;
    if (M < 1 || Cin < 1 || Cout < 1 || (dtype != CONV_BF16 && dtype != CONV_F32)) return CONV_ERR_INVALID_ARG;
    if (ldq < Cin || ldw < Cin) return CONV_ERR_INVALID_ARG;
    if (Cin > kI8MaxReduce || M > kI8MaxRows || Cout > kI8MaxRows) return CONV_ERR_UNSUPPORTED;
    if (int rc = check_i8_rows(q, Cin, ldq)) return rc;
    if (int rc = check_i8_rows(Wq, Cin, ldw)) return rc;
    if (!aligned(q_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4) || !aligned(Y, i8_elem(dtype)))
        return CONV_ERR_MISALIGNED;
    const long long ny = 1LL * M * Cout * i8_elem(dtype);
    if (overlaps(Y, ny, q, i8_extent(M, Cin, ldq)) || overlaps(Y, ny, Wq, i8_extent(Cout, Cin, ldw)) ||
        overlaps(Y, ny, q_scale, 4LL * M) || overlaps(Y, ny, w_scale, 4LL * Cout) || (bias && overlaps(Y, ny, bias, 4LL * Cout)))
        return CONV_ERR_INVALID_ARG;
    return CONV_OK;
}

int launch_pointwise_i8(const int8_t *q, const float *q_scale, const int8_t *Wq, const float *w_scale, const float *bias,
                        void *Y, int M, int Cin, int Cout, int ldq, int ldw, int dtype, cudaStream_t stream,
                        DeviceState *d) {
    const I8Operands a{q, Wq, Cin, ldq, ldw};
    I8GemmParams p{};
    p.q_scale = q_scale;
    p.w_scale = w_scale;
    p.bias = bias;
    p.Y = Y;
    p.M = M;
    p.N = Cout;
    return dtype == CONV_F32 ? run_i8_product<float>(a, p, stream, d) : run_i8_product<__nv_bfloat16>(a, p, stream, d);
}

}  // namespace
}  // namespace convb200

extern "C" {

// Rows on 32-byte sectors: a tensor copy of rows that start inside one takes up to twice as long (301
// x 4999 x 5003: 22.9 us with a pitch of 5008, 15.0 with 5024, 14.0 with 5120).
int conv_i8_row_pitch(int C) { return C < 1 || C > kInt32Max - 31 ? 0 : (C + 31) / 32 * 32; }

int rmsnorm_i8_fwd(const void *x, const void *residual, const float *weight, void *h, int8_t *q, float *scale, int M,
                   int C, int ldq, float eps, int dtype, cudaStream_t stream) {
    if (!x || !weight || !q || !scale || (residual != nullptr) != (h != nullptr)) return CONV_ERR_INVALID_ARG;
    if (M < 1 || C < 1 || !(eps >= 0x1p-126f) || !(eps <= 3.402823466e+38f) || (dtype != CONV_BF16 && dtype != CONV_F32))
        return CONV_ERR_INVALID_ARG;
    const int e = i8_elem(dtype);
    if (int rc = check_i8_rows(q, C, ldq)) return rc;
    if (C > kI8MaxCols) return CONV_ERR_UNSUPPORTED;
    if (!aligned(x, e) || !aligned(residual, e) || !aligned(h, e) || !aligned(weight, 4) || !aligned(scale, 4))
        return CONV_ERR_MISALIGNED;
    const long long nx = 1LL * M * C * e, nq = i8_extent(M, C, ldq), ns = 4LL * M, nw = 4LL * C;
    // h may be the residual or x itself: a thread reads an element before it writes it
    if ((h && ((h != x && overlaps(h, nx, x, nx)) || (h != residual && overlaps(h, nx, residual, nx)) ||
               overlaps(h, nx, weight, nw) || overlaps(h, nx, q, nq) || overlaps(h, nx, scale, ns) ||
               overlaps(q, nq, residual, nx) || overlaps(scale, ns, residual, nx))) ||
        overlaps(q, nq, x, nx) || overlaps(q, nq, weight, nw) || overlaps(q, nq, scale, ns) || overlaps(scale, ns, x, nx) ||
        overlaps(scale, ns, weight, nw))
        return CONV_ERR_INVALID_ARG;
    DeviceState *d = nullptr;
    if (int rc = device_state(&d)) return rc;
    if (int rc = check_device_ptrs(stream, {x, residual, weight, h, q, scale})) return rc;
    const I8RowsParams p{x, residual, weight, h, q, scale, M, C, ldq, eps};
    return residual ? run_i8_rows<kI8NormResidual>(p, dtype, stream, d) : run_i8_rows<kI8Norm>(p, dtype, stream, d);
}

int quant_rows_i8_fwd(const void *x, int8_t *q, float *scale, int M, int C, int ldq, int glu, int dtype,
                      cudaStream_t stream) {
    if (!x || !q || !scale) return CONV_ERR_INVALID_ARG;
    if (M < 1 || C < 1 || (glu != 0 && glu != 1) || (dtype != CONV_BF16 && dtype != CONV_F32)) return CONV_ERR_INVALID_ARG;
    const int e = i8_elem(dtype);
    if (int rc = check_i8_rows(q, C, ldq)) return rc;
    if (C > kI8MaxCols) return CONV_ERR_UNSUPPORTED;
    if (!aligned(x, e) || !aligned(scale, 4)) return CONV_ERR_MISALIGNED;
    const long long nx = 1LL * M * C * e * (glu ? 2 : 1), nq = i8_extent(M, C, ldq), ns = 4LL * M;
    if (overlaps(q, nq, x, nx) || overlaps(q, nq, scale, ns) || overlaps(scale, ns, x, nx)) return CONV_ERR_INVALID_ARG;
    DeviceState *d = nullptr;
    if (int rc = device_state(&d)) return rc;
    if (int rc = check_device_ptrs(stream, {x, q, scale})) return rc;
    const I8RowsParams p{x, nullptr, nullptr, nullptr, q, scale, M, C, ldq, 0.0f};
    return glu ? run_i8_rows<kI8Glu>(p, dtype, stream, d) : run_i8_rows<kI8Plain>(p, dtype, stream, d);
}

int quant_filter_i8_fwd(const void *F, int8_t *Wq, float *scale, int Cin, int Cout, int ldw, int dtype,
                        cudaStream_t stream) {
    if (!F || !Wq || !scale) return CONV_ERR_INVALID_ARG;
    if (Cin < 1 || Cout < 1 || (dtype != CONV_BF16 && dtype != CONV_F32)) return CONV_ERR_INVALID_ARG;
    if (Cin > kI8MaxReduce || Cout > kI8MaxRows) return CONV_ERR_UNSUPPORTED;
    const int e = i8_elem(dtype);
    if (int rc = check_i8_rows(Wq, Cin, ldw)) return rc;
    if (!aligned(F, e) || !aligned(scale, 4)) return CONV_ERR_MISALIGNED;
    const long long nf = 1LL * Cin * Cout * e, nq = i8_extent(Cout, Cin, ldw), ns = 4LL * Cout;
    if (overlaps(Wq, nq, F, nf) || overlaps(Wq, nq, scale, ns) || overlaps(scale, ns, F, nf)) return CONV_ERR_INVALID_ARG;
    DeviceState *d = nullptr;
    if (int rc = device_state(&d)) return rc;
    if (int rc = check_device_ptrs(stream, {F, Wq, scale})) return rc;
    I8FilterParams p{};
    p.F = F;
    p.q = Wq;
    p.scale = scale;
    p.Cin = Cin;
    p.Cout = Cout;
    p.ldq = ldw;
    return dtype == CONV_F32 ? run_i8_filter<float>(p, stream, d) : run_i8_filter<__nv_bfloat16>(p, stream, d);
}

int dequant_rows_i8_fwd(const int8_t *q, const float *scale, void *y, int M, int C, int ldq, int dtype,
                        cudaStream_t stream) {
    if (!q || !scale || !y) return CONV_ERR_INVALID_ARG;
    if (M < 1 || C < 1 || (dtype != CONV_BF16 && dtype != CONV_F32)) return CONV_ERR_INVALID_ARG;
    const int e = i8_elem(dtype);
    if (int rc = check_i8_rows(q, C, ldq)) return rc;
    if (C > kI8MaxCols) return CONV_ERR_UNSUPPORTED;
    if (!aligned(y, e) || !aligned(scale, 4)) return CONV_ERR_MISALIGNED;
    const long long ny = 1LL * M * C * e;
    if (overlaps(y, ny, q, i8_extent(M, C, ldq)) || overlaps(y, ny, scale, 4LL * M)) return CONV_ERR_INVALID_ARG;
    DeviceState *d = nullptr;
    if (int rc = device_state(&d)) return rc;
    if (int rc = check_device_ptrs(stream, {q, scale, y})) return rc;
    I8DequantParams p{q, scale, y, M, C, ldq, 0};
    const bool vec = (1LL * C * e) % 16 == 0 && aligned(y, 16);
    const int seg = vec ? 4 * 32 * (16 / e) : 512;   // values a warp takes
    const int segs = (C + seg - 1) / seg;
    while (p.wpr_shift < 3 && (1 << p.wpr_shift) < segs) ++p.wpr_shift;
    const long long blocks = (1LL * M + (8 >> p.wpr_shift) - 1) >> (3 - p.wpr_shift);
    const long long seg_blocks = (segs + (1 << p.wpr_shift) - 1) >> p.wpr_shift;
    if (blocks > kInt32Max || seg_blocks > 65535) return CONV_ERR_UNSUPPORTED;   // neither within the limits above
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(seg_blocks));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaError_t rc;
    if (dtype == CONV_F32)
        rc = vec ? launch_k(cfg, i8_dequant_kernel<float, true>, p, d->status)
                 : launch_k(cfg, i8_dequant_kernel<float, false>, p, d->status);
    else
        rc = vec ? launch_k(cfg, i8_dequant_kernel<__nv_bfloat16, true>, p, d->status)
                 : launch_k(cfg, i8_dequant_kernel<__nv_bfloat16, false>, p, d->status);
    return launched(rc, "i8_dequant_kernel");
}

int pointwise_i8_fwd(const int8_t *q, const float *q_scale, const int8_t *Wq, const float *w_scale, const float *bias,
                     void *Y, int M, int Cin, int Cout, int ldq, int ldw, int dtype, cudaStream_t stream) {
    if (int rc = check_pointwise_i8(q, q_scale, Wq, w_scale, bias, Y, M, Cin, Cout, ldq, ldw, dtype)) return rc;
    DeviceState *d = nullptr;
    if (int rc = device_state(&d)) return rc;
    if (int rc = check_device_ptrs(stream, {q, q_scale, Wq, w_scale, bias, Y})) return rc;
    return launch_pointwise_i8(q, q_scale, Wq, w_scale, bias, Y, M, Cin, Cout, ldq, ldw, dtype, stream, d);
}

size_t conv2d_nhwc_i8_workspace(int N, int H, int W, int Cin) {
    if (N < 1 || H < 1 || W < 1 || Cin < 1 || Cin > kI8MaxReduce || 1LL * N * H > kI8MaxRows || 1LL * N * H * W > kI8MaxRows)
        return 0;
    return 1ull * N * H * W * (conv_i8_row_pitch(Cin) + 4);
}

int conv2d_nhwc_fwd_i8(const void *X, const float *norm, float eps, const int8_t *Wq, const float *w_scale,
                       const float *bias, void *Y, void *workspace, size_t workspace_bytes, int N, int H, int W, int Cin,
                       int Cout, int ldw, cudaStream_t stream) {
    if (!X || !Wq || !w_scale || !Y || !workspace) return CONV_ERR_INVALID_ARG;
    if (N < 1 || H < 1 || W < 1 || Cin < 1 || Cout < 1 || ldw < Cin) return CONV_ERR_INVALID_ARG;
    if (norm && (!(eps >= 0x1p-126f) || !(eps <= 3.402823466e+38f))) return CONV_ERR_INVALID_ARG;
    const size_t full = conv2d_nhwc_i8_workspace(N, H, W, Cin);
    if (full == 0) return CONV_ERR_UNSUPPORTED;
    const int ld16 = (Cin + 15) / 16 * 16;
    const size_t least = 1ull * N * H * W * (ld16 + 4);
    if (workspace_bytes < least) return CONV_ERR_INVALID_ARG;
    if (!aligned(workspace, 16) || !aligned(X, 2) || !aligned(norm, 4)) return CONV_ERR_MISALIGNED;
    const int M = N * H * W, ldq = workspace_bytes >= full ? conv_i8_row_pitch(Cin) : ld16;
    int8_t *q = static_cast<int8_t *>(workspace);
    float *q_scale = reinterpret_cast<float *>(q + 1LL * M * ldq);
    if (int rc = check_pointwise_i8(q, q_scale, Wq, w_scale, bias, Y, M, Cin, Cout, ldq, ldw, CONV_BF16)) return rc;
    const long long nx = 2LL * M * Cin, ny = 2LL * M * Cout, nws = 1LL * M * (ldq + 4);
    if (overlaps(Y, ny, X, nx) || (norm && overlaps(Y, ny, norm, 4LL * Cin)) || overlaps(workspace, nws, X, nx) ||
        overlaps(workspace, nws, Wq, i8_extent(Cout, Cin, ldw)) || overlaps(workspace, nws, w_scale, 4LL * Cout) ||
        (bias && overlaps(workspace, nws, bias, 4LL * Cout)) || (norm && overlaps(workspace, nws, norm, 4LL * Cin)))
        return CONV_ERR_INVALID_ARG;
    DeviceState *d = nullptr;
    if (int rc = device_state(&d)) return rc;
    if (int rc = check_device_ptrs(stream, {X, norm, Wq, w_scale, bias, Y, workspace})) return rc;
    const I8RowsParams p{X, nullptr, norm, nullptr, q, q_scale, M, Cin, ldq, eps};
    if (int rc = norm ? run_i8_rows<kI8Norm>(p, CONV_BF16, stream, d) : run_i8_rows<kI8Plain>(p, CONV_BF16, stream, d))
        return rc;
    return launch_pointwise_i8(q, q_scale, Wq, w_scale, bias, Y, M, Cin, Cout, ldq, ldw, CONV_BF16, stream, d);
}

}  // extern "C"
