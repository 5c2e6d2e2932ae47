// The 8-bit entry points: argument checks, kernel choice, tensor maps, launches. Included at the
// end of capi.cu, whose helpers (device state, launch_k, pointer checks) it uses.
#pragma once

namespace convb200 {
namespace {

constexpr int kI8MaxReduce = 131071;   // (131071 + 1) * 128 * 128 = 2^31: the int32 sums are exact below

int i8_elem(int dtype) { return dtype == CONV_F32 ? 4 : 2; }

// Bytes from the first to past the last value of `rows` rows of C bytes, ld apart.
long long i8_extent(long long rows, int C, int ld) { return (rows - 1) * ld + C; }

int check_i8_rows(const void *q, int C, int ld) {
    if (ld < C) return CONV_ERR_INVALID_ARG;
    if (ld % 16 != 0 || !aligned(q, 16)) return CONV_ERR_MISALIGNED;
    return CONV_OK;
}

// ---- rows ------------------------------------------------------------------------------
template <typename T, int MODE, int NV, bool VEC, bool GROUP_WARP, bool STREAM>
int launch_i8_rows(const I8RowsParams &p, int threads, cudaStream_t stream, DeviceState *d) {
    const long long per = GROUP_WARP ? threads / 32 : 1, blocks = (p.M + per - 1) / per;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = stream;
    return launched(launch_k(cfg, i8_rows_kernel<T, MODE, NV, VEC, GROUP_WARP, STREAM>, p, d->status), "i8_rows_kernel");
}

template <typename T, int MODE>
int run_i8_rows(const I8RowsParams &p, cudaStream_t stream, DeviceState *d) {
    const int C = p.C;
    const bool vec = C % 8 == 0 && aligned(p.x, 16) && (!p.residual || aligned(p.residual, 16)) &&
                     (!p.h || aligned(p.h, 16)) && (!p.weight || aligned(p.weight, 16));
    auto block = [&](int nv) {   // threads of a block that holds a row, nv groups of eight a thread
        const int t = ((C + 8 * nv - 1) / (8 * nv) + 31) / 32 * 32;
        return t < 512 ? t : 512;
    };
    if (vec) {
        if (C <= 512) return launch_i8_rows<T, MODE, 2, true, true, false>(p, 256, stream, d);
        if (C <= 1024) return launch_i8_rows<T, MODE, 4, true, true, false>(p, 256, stream, d);
        if (C <= 8192) return launch_i8_rows<T, MODE, 2, true, false, false>(p, block(2), stream, d);
        if (C <= 16384) return launch_i8_rows<T, MODE, 4, true, false, false>(p, block(4), stream, d);
        return launch_i8_rows<T, MODE, 4, true, false, true>(p, 512, stream, d);
    }
    if (C <= 1024) return launch_i8_rows<T, MODE, 4, false, true, false>(p, 256, stream, d);
    if (C <= 16384) return launch_i8_rows<T, MODE, 4, false, false, false>(p, block(4), stream, d);
    return launch_i8_rows<T, MODE, 4, false, false, true>(p, 512, stream, d);
}

template <int MODE>
int run_i8_rows(const I8RowsParams &p, int dtype, cudaStream_t stream, DeviceState *d) {
    return dtype == CONV_F32 ? run_i8_rows<float, MODE>(p, stream, d) : run_i8_rows<__nv_bfloat16, MODE>(p, stream, d);
}

// ---- product -----------------------------------------------------------------------------
// A matrix of 8-bit rows: boxes of 128 values x `box_rows` rows, 128-byte swizzle.
int i8_map(CUtensorMap *m, const int8_t *q, int rows, int C, int ld, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)C, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return g_encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t *>(q), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
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
    if (int rc = i8_map(&tmW, a.Wq, p.N, a.Cin, a.ldw, 128)) return rc;
    if (int rc = i8_map(&tmQ, a.q, p.M, a.Cin, a.ldq, Cfg::BN)) return rc;
    p.n_tiles = (p.N + 127) / 128;
    p.m_tiles = (p.M + Cfg::BN - 1) / Cfg::BN;
    p.split = split;
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

template <typename OUT>
int launch_i8_pair(const I8Operands &a, I8GemmParams p, cudaStream_t stream, DeviceState *d, unsigned bit) {
    using Cfg = I8PairCfg;
    auto kern = i8_pair_kernel<OUT>;
    if (int rc = ensure_smem_attr(d, bit, kern, Cfg::SMEM)) return rc;
    CUtensorMap tmQ, tmW;
    if (int rc = i8_map(&tmQ, a.q, p.M, a.Cin, a.ldq, 128)) return rc;
    if (int rc = i8_map(&tmW, a.Wq, p.N, a.Cin, a.ldw, 128)) return rc;
    p.m_tiles = (p.M + 255) / 256;
    p.n_tiles = (p.N + 255) / 256;
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
    return launched(launch_k(cfg, kern, tmQ, tmW, p, d->status), "i8_pair_kernel");
}

// The kernel for a product: bn = 0 for the pair kernel, else the split kernel's token columns, and
// its split of the reduction.
struct I8Plan {
    int bn, split;
};

I8Plan plan_i8(int M, int N, int num_kblk, int num_sms) {
    I8Plan pl{0, 1};
    if (M <= 512) {
        pl.bn = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
        const long long tiles = 1LL * ((N + 127) / 128) * ((M + pl.bn - 1) / pl.bn);
        while (pl.split < 8 && tiles * pl.split * 2 <= num_sms && pl.split * 4 <= num_kblk) pl.split *= 2;
    }
    // CONV_B200_I8 (tests): "pair", or "split,BN,S"
    if (const char *f = env("CONV_B200_I8")) {
        int bn = 0, s = 0;
        if (std::strcmp(f, "pair") == 0) pl = I8Plan{0, 1};
        else if (std::sscanf(f, "split,%d,%d", &bn, &s) == 2 && (bn == 16 || bn == 32 || bn == 64 || bn == 128) &&
                 (s == 1 || s == 2 || s == 4 || s == 8) && s <= num_kblk)
            pl = I8Plan{bn, s};
    }
    return pl;
}

template <typename OUT>
int run_i8_product(const I8Operands &a, I8GemmParams p, cudaStream_t stream, DeviceState *d) {
    p.num_kblk = (a.Cin + 127) / 128;
    p.vec = aligned(p.Y, 16) && (1LL * p.N * sizeof(OUT)) % 16 == 0;
    const I8Plan pl = plan_i8(p.M, p.N, p.num_kblk, d->num_sms);
    constexpr unsigned bit = sizeof(OUT) == 4 ? 116 : 112;
    switch (pl.bn) {
        case 16: return launch_i8_split<I8SplitCfg<16, 5>, OUT>(a, p, pl.split, stream, d, bit);
        case 32: return launch_i8_split<I8SplitCfg<32, 4>, OUT>(a, p, pl.split, stream, d, bit + 1);
        case 64: return launch_i8_split<I8SplitCfg<64, 3>, OUT>(a, p, pl.split, stream, d, bit + 2);
        case 128: return launch_i8_split<I8SplitCfg<128, 4>, OUT>(a, p, pl.split, stream, d, bit + 3);
        default: return launch_i8_pair<OUT>(a, p, stream, d, sizeof(OUT) == 4 ? 121 : 120);
    }
}

int check_pointwise_i8(const int8_t *q, const float *q_scale, const int8_t *Wq, const float *w_scale, const float *bias,
                       const void *Y, int M, int Cin, int Cout, int ldq, int ldw, int dtype) {
    if (!q || !q_scale || !Wq || !w_scale || !Y) return CONV_ERR_INVALID_ARG;
    if (M < 1 || Cin < 1 || Cout < 1 || (dtype != CONV_BF16 && dtype != CONV_F32)) return CONV_ERR_INVALID_ARG;
    if (ldq < Cin || ldw < Cin) return CONV_ERR_INVALID_ARG;
    if (Cin > kI8MaxReduce) return CONV_ERR_UNSUPPORTED;
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

int conv_i8_row_pitch(int C) { return C < 1 || C > kInt32Max - 15 ? 0 : (C + 15) / 16 * 16; }

int rmsnorm_i8_fwd(const void *x, const void *residual, const float *weight, void *h, int8_t *q, float *scale, int M,
                   int C, int ldq, float eps, int dtype, cudaStream_t stream) {
    if (!x || !weight || !q || !scale || (residual != nullptr) != (h != nullptr)) return CONV_ERR_INVALID_ARG;
    if (M < 1 || C < 1 || !(eps >= 0x1p-126f) || !(eps <= 3.402823466e+38f) || (dtype != CONV_BF16 && dtype != CONV_F32))
        return CONV_ERR_INVALID_ARG;
    const int e = i8_elem(dtype);
    if (int rc = check_i8_rows(q, C, ldq)) return rc;
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
    if (Cin > kI8MaxReduce) return CONV_ERR_UNSUPPORTED;
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
    // a tile of rows per CTA until the cluster has eight, then more tiles each
    const int tiles = (Cin + kI8FilterRows - 1) / kI8FilterRows;
    int S = 1;
    while (S < 8 && S < tiles) S *= 2;
    p.slab = (tiles + S - 1) / S * kI8FilterRows;
    const long long ctas = 1LL * ((Cout + kI8FilterCols - 1) / kI8FilterCols) * S;
    if (ctas > kInt32Max) return CONV_ERR_UNSUPPORTED;
    const bool vec = Cout % 8 == 0 && aligned(F, 16);
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
    cfg.stream = stream;
    cudaError_t rc;
    if (dtype == CONV_F32)
        rc = vec ? launch_k(cfg, i8_filter_kernel<float, true>, p, d->status)
                 : launch_k(cfg, i8_filter_kernel<float, false>, p, d->status);
    else
        rc = vec ? launch_k(cfg, i8_filter_kernel<__nv_bfloat16, true>, p, d->status)
                 : launch_k(cfg, i8_filter_kernel<__nv_bfloat16, false>, p, d->status);
    return launched(rc, "i8_filter_kernel");
}

int dequant_rows_i8_fwd(const int8_t *q, const float *scale, void *y, int M, int C, int ldq, int dtype,
                        cudaStream_t stream) {
    if (!q || !scale || !y) return CONV_ERR_INVALID_ARG;
    if (M < 1 || C < 1 || (dtype != CONV_BF16 && dtype != CONV_F32)) return CONV_ERR_INVALID_ARG;
    const int e = i8_elem(dtype);
    if (int rc = check_i8_rows(q, C, ldq)) return rc;
    if (!aligned(y, e) || !aligned(scale, 4)) return CONV_ERR_MISALIGNED;
    const long long ny = 1LL * M * C * e;
    if (overlaps(y, ny, q, i8_extent(M, C, ldq)) || overlaps(y, ny, scale, 4LL * M)) return CONV_ERR_INVALID_ARG;
    DeviceState *d = nullptr;
    if (int rc = device_state(&d)) return rc;
    if (int rc = check_device_ptrs(stream, {q, scale, y})) return rc;
    I8DequantParams p{q, scale, y, M, C, ldq, (C + 511) / 512};
    const long long blocks = (1LL * M * p.segs + 7) / 8;
    if (blocks > kInt32Max) return CONV_ERR_UNSUPPORTED;
    const bool vec = C % 16 == 0 && aligned(y, 16);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
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
    if (N < 1 || H < 1 || W < 1 || Cin < 1 || Cin > kI8MaxReduce || 1LL * N * H * W > kInt32Max || 1LL * N * H > kInt32Max)
        return 0;
    return 1ull * N * H * W * (conv_i8_row_pitch(Cin) + 4);
}

int conv2d_nhwc_fwd_i8(const void *X, const float *norm, float eps, const int8_t *Wq, const float *w_scale,
                       const float *bias, void *Y, void *workspace, size_t workspace_bytes, int N, int H, int W, int Cin,
                       int Cout, int ldw, cudaStream_t stream) {
    if (!X || !Wq || !w_scale || !Y || !workspace) return CONV_ERR_INVALID_ARG;
    if (N < 1 || H < 1 || W < 1 || Cin < 1 || Cout < 1 || ldw < Cin) return CONV_ERR_INVALID_ARG;
    if (norm && (!(eps >= 0x1p-126f) || !(eps <= 3.402823466e+38f))) return CONV_ERR_INVALID_ARG;
    const size_t need = conv2d_nhwc_i8_workspace(N, H, W, Cin);
    if (need == 0) return CONV_ERR_UNSUPPORTED;
    if (workspace_bytes < need) return CONV_ERR_INVALID_ARG;
    if (!aligned(workspace, 16) || !aligned(X, 2) || !aligned(norm, 4)) return CONV_ERR_MISALIGNED;
    const int M = N * H * W, ldq = conv_i8_row_pitch(Cin);
    int8_t *q = static_cast<int8_t *>(workspace);
    float *q_scale = reinterpret_cast<float *>(q + 1LL * M * ldq);
    if (int rc = check_pointwise_i8(q, q_scale, Wq, w_scale, bias, Y, M, Cin, Cout, ldq, ldw, CONV_BF16)) return rc;
    const long long nx = 2LL * M * Cin, ny = 2LL * M * Cout, nws = static_cast<long long>(need);
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
