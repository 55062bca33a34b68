// Entry points of the block-scaled FP8 operators (quantisation, gate, linear
// layer); specified in include/pgf8.h.  Included by pgf8_api.cu after its
// helpers.
#pragma once

#include "gemm_block.cuh"
#include "gemm_block_pair.cuh"
#include "quantize_blocks.cuh"

namespace pgf8 {

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Bytes of an element, 0 for an unknown type.
static int dtype_bytes(int dt)
{
    return dt == PGF8_F32 ? 4 : (dt == PGF8_F16 || dt == PGF8_BF16) ? 2 : 0;
}

// Calls f with a null pointer of the element type.
template <class F> static pgf8_status by_dtype(int dt, F f)
{
    if (dt == PGF8_F32)
        return f(static_cast<const float *>(nullptr));
    if (dt == PGF8_F16)
        return f(static_cast<const __half *>(nullptr));
    return f(static_cast<const __nv_bfloat16 *>(nullptr));
}

static pgf8_status check_block_quant(const void *x, int xdt, int64_t batch, int64_t rows, int64_t cols, int64_t ldx,
                                     int64_t ldb, int block_rows, const uint8_t *q, const float *scales)
{
    if (batch < 0 || rows < 0 || cols < 16 || cols > (1ll << 30) || ldx < cols || ldx > (1ll << 40) ||
        rows > (1ll << 31) - 1 || batch > (1ll << 31) - 1 || (block_rows != 1 && block_rows != 128))
        return PGF8_ERR_INVALID_ARG;
    if (batch == 0 || rows == 0)
        return PGF8_OK;
    if (batch > 1 && (ldb < 0 || ldb > (1ll << 50)))
        return PGF8_ERR_INVALID_ARG;
    if (!x || !q || !scales)
        return PGF8_ERR_INVALID_ARG;
    const int eb = dtype_bytes(xdt);
    if (eb == 0)
        return PGF8_ERR_UNSUPPORTED;
    if (cols % 16 != 0 || (ldx * eb) % 16 != 0 || (batch > 1 && (ldb * eb) % 16 != 0) || !aligned16(x) ||
        !aligned16(q) || !aligned4(scales))
        return PGF8_ERR_ALIGNMENT;
    // one launch: the grid's x extent holds every CTA (8 threads a row group, a CTA a tile)
    const int64_t cb = ceil_div(cols, 128);
    const double ctas = block_rows == 1 ? static_cast<double>(batch) * rows * cb / 32
                                        : static_cast<double>(batch) * ceil_div(rows, 128) * cb;
    if (ctas > 2147483000.0)
        return PGF8_ERR_UNSUPPORTED;
    return PGF8_OK;
}

// 1 x 128 groups of rows (arguments checked, rows > 0).
static pgf8_status row_blocks_launch(const void *x, int xdt, int64_t rows, int64_t cols, int64_t ldx, uint8_t *q,
                                     float *scales, cudaStream_t cs, int pdl)
{
    const int64_t groups = ceil_div(cols, 128);
    const uint64_t total = static_cast<uint64_t>(rows) * static_cast<uint64_t>(groups);
    const unsigned grid = static_cast<unsigned>((total + 31) / 32);
    return by_dtype(xdt, [&](auto *t) {
        using T = std::remove_cv_t<std::remove_pointer_t<decltype(t)>>;
        return launch_quant(quantize_row_blocks_kernel<T>, grid, cs, pdl, static_cast<const T *>(x), total,
                            static_cast<uint32_t>(groups), cols, ldx, q, scales);
    });
}

// ------------------------------------------------------------------ linear
struct BlockLaunch {
    const uint8_t *aq, *wq;
    const float *sa, *sw;
    void *y;
    int ydt;
    int64_t M, N, K;
    int prefetch_w;
    cudaStream_t stream;
    const void *x = nullptr;   // in-kernel quantisation: the activations, row stride ldx
    int64_t ldx = 0;
};

// ------------------------------------------------------------------ kernel choice
// How many clusters of each size the current device holds at once, for one
// kernel at one amount of shared memory (a cluster's CTAs share a GPC, so
// this is less than the CTAs that fit divided by the size: 16 clusters of 8
// CTAs at one to an SM do not all run at once on a B200, and a grid that
// counts on it takes two rounds).  For kernels that allocate tensor memory the
// occupancy query answers for one CTA to an SM; where two fit (per_sm), a
// cluster takes half as many SMs (measured: 32 clusters of 8 and 80 of 3 run in
// one round, 96 of 3 and 64 of 6 do not).  Set up once per device.
constexpr int kMaxCluster = 8;

struct ClusterFit {
    PerDeviceSetup setup;
    int fit[kSetupDevices + 1][kMaxCluster + 1];
};

template <typename... Args>
static cudaError_t cluster_fit(ClusterFit &c, void (*kernel)(Args...), int threads, int attr_smem, int smem,
                               int per_sm, const int *&fit)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    int *row = c.fit[dev >= 0 && dev < kSetupDevices ? dev : kSetupDevices];
    e = setup_once_per_device(c.setup, [=](int, int *) {
        cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, attr_smem);
        if (err == cudaSuccess)
            err = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                       cudaSharedmemCarveoutMaxShared);
        for (int s = 1; s <= kMaxCluster && err == cudaSuccess; ++s) {
            cudaLaunchConfig_t q;
            std::memset(&q, 0, sizeof(q));
            q.gridDim = dim3(1, 1, static_cast<unsigned>(s));
            q.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
            q.dynamicSmemBytes = static_cast<size_t>(smem);
            cudaLaunchAttribute qa[2];
            qa[0].id = cudaLaunchAttributeClusterDimension;
            qa[0].val.clusterDim.x = qa[0].val.clusterDim.y = 1;
            qa[0].val.clusterDim.z = static_cast<unsigned>(s);
            q.attrs = qa;
            q.numAttrs = 1;
            int n = 0;
            err = cudaOccupancyMaxActiveClusters(&n, kernel, &q);
            row[s] = n > 0 ? n : 1;
        }
        if (per_sm >= 2)
            for (int s = kMaxCluster; s >= 1; --s)
                row[s] = s % 2 == 0 ? row[s / 2] : 2 * row[s];
        return err;
    });
    fit = row;
    return e;
}

// Estimated time in us, measured on a B200 (fixed part about 4 us for every
// kernel, so that it cancels), and the K-split that gives it.
struct BlockPlan {
    double us;
    int splits;
};

// A weight-streaming kernel over `tiles` weight tiles of `kblocks` k-blocks,
// `kb_us` a k-block for one SM: the longest of its rounds' k-blocks one after
// another, of the SMs' total work, and of the weights at HBM speed; 0.7 us for
// the exchange of a split sum, 2 us for each further round, and a quarter of a
// CTA's own k-blocks, by which they end apart.  One token (us at splits of 1, 2,
// 3, 4, 6, 8): 4096 x 4096 12.7, 8.9, 8.0, 7.4, 7.6, 6.3; 12288 x 4096 13.9, 12.9,
// 16.3, 15.4, 18.5, 17.8; 8192 x 28672 72.5, 41.7, 39.9, 38.4, 44.0, 41.5.
static BlockPlan stream_plan(int64_t tiles, int64_t kblocks, double kb_us, double weight_bytes, const int *fit)
{
    static const int kSizes[] = {1, 2, 3, 4, 6, 8};
    BlockPlan best = {1e30, 1};
    const int sms = num_sms();
    for (int s : kSizes) {
        if (s > 1 && kblocks < 2 * s)
            break;
        const double rounds = static_cast<double>(ceil_div(tiles, fit[s]));
        const double own = static_cast<double>(ceil_div(kblocks, s)) * kb_us;
        double us = std::fmax(rounds * own, static_cast<double>(tiles) * kblocks * kb_us / sms);
        us = std::fmax(us, weight_bytes / 6.2e6) + 0.25 * own + 2.0 * (rounds - 1.0) + (s > 1 ? 0.7 : 0.0);
        if (us < best.us)
            best = {us, s};
    }
    return best;
}

static BlockParams block_params(const BlockLaunch &L)
{
    BlockParams p;
    p.M = static_cast<int>(L.M);
    p.N = static_cast<int>(L.N);
    p.K = static_cast<int>(L.K);
    p.kblocks = static_cast<int>(ceil_div(L.K, 128));
    p.prefetch_w = L.prefetch_w;
    p.sa = L.sa;
    p.sw = L.sw;
    p.y = L.y;
    p.ydt = L.ydt;
    p.x = L.x;
    p.ldx = L.ldx;
    return p;
}

template <class C> static bool block_maps(const BlockLaunch &L, CUtensorMap &tmX, CUtensorMap &tmW)
{
    return make_map(&tmX, L.aq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, L.M, L.K, 128, C::kRowsX,
                    CU_TENSOR_MAP_SWIZZLE_128B) &&
           make_map(&tmW, L.wq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, L.N, L.K, 128, C::kRowsW,
                    CU_TENSOR_MAP_SWIZZLE_128B);
}

template <class C> static cudaError_t block_fit(const int *&fit)
{
    static ClusterFit c;
    return cluster_fit(c, gemm_block_kernel<C>, C::kThreads, C::kSmemBytes, C::kSmemBytes, C::CTAS, fit);
}

// kb_us: see stream_plan.
template <class C> static BlockPlan plan_block(const BlockLaunch &L, double kb_us)
{
    const int *fit = nullptr;
    if (block_fit<C>(fit) != cudaSuccess)
        return {1e29, 1};
    const int64_t nt = ceil_div(L.N, 128), mt = ceil_div(L.M, C::BN);
    if (mt > 65535)   // the grid's y extent
        return {1e30, 1};
    return stream_plan(nt * mt, ceil_div(L.K, 128), kb_us, static_cast<double>(L.N) * L.K, fit);
}

template <class C> static pgf8_status launch_block(const BlockLaunch &L, int splits)
{
    const int *fit = nullptr;
    cudaError_t e = block_fit<C>(fit);
    if (e != cudaSuccess)
        return cuda_fail(e);
    CUtensorMap tmX, tmW;
    if constexpr (C::XQ != 0) {
        std::memset(&tmX, 0, sizeof(tmX));   // not used
        if (!make_map(&tmW, L.wq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, L.N, L.K, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B))
            return PGF8_ERR_UNSUPPORTED;
    } else if (!block_maps<C>(L, tmX, tmW)) {
        return PGF8_ERR_UNSUPPORTED;
    }
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(L.N, 128)), static_cast<unsigned>(ceil_div(L.M, C::BN)),
                       static_cast<unsigned>(splits));
    cfg.blockDim = dim3(C::kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = L.stream;
    cudaLaunchAttribute attrs[2];
    fill_attrs(cfg, attrs, splits, C::XQ == 0);   // in-kernel quantisation: an ordinary launch
    e = cudaLaunchKernelEx(&cfg, gemm_block_kernel<C>, tmX, tmW, block_params(L));
    return e == cudaSuccess ? PGF8_OK : cuda_fail(e);
}

// SM pairs: clusters of two CTAs, as many as the GPU holds at once.
template <class C> static pgf8_status launch_block_pair(const BlockLaunch &L)
{
    static PerDeviceSetup setup;
    int pairs_fit = 1;
    const cudaError_t err = setup_once_per_device(setup, [](int, int *v) {
        cudaError_t e = cudaFuncSetAttribute(gemm_block_pair_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             C::kSmemBytes);
        if (e != cudaSuccess)
            return e;
        cudaLaunchConfig_t q;
        std::memset(&q, 0, sizeof(q));
        q.gridDim = dim3(2 * num_sms(), 1, 1);
        q.blockDim = dim3(C::kThreads, 1, 1);
        q.dynamicSmemBytes = C::kSmemBytes;
        cudaLaunchAttribute qa[2];
        fill_attrs(q, qa, 1, 0, 2);
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, gemm_block_pair_kernel<C>, &q);
        *v = n > 0 ? n : 1;
        return e;
    }, &pairs_fit);
    if (err != cudaSuccess)
        return cuda_fail(err);
    CUtensorMap tmX, tmW;
    if (!block_maps<C>(L, tmX, tmW))
        return PGF8_ERR_UNSUPPORTED;
    const int64_t tiles = ceil_div(L.M, 256) * ceil_div(L.N, C::BN);
    if (tiles > 2147483647)
        return PGF8_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>(2 * (tiles < pairs_fit ? tiles : pairs_fit)), 1, 1);
    cfg.blockDim = dim3(C::kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = L.stream;
    cudaLaunchAttribute attrs[2];
    fill_attrs(cfg, attrs, 1, 1, 2);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, gemm_block_pair_kernel<C>, tmX, tmW, block_params(L));
    return e == cudaSuccess ? PGF8_OK : cuda_fail(e);
}

// Up to 64 tokens the weight-row kernel with the narrowest token tile; beyond,
// the shortest of four estimates.  The times a k-block (us) were fitted to
// measurements over N, K from 512 to 16384 and 48 to 2048 tokens: weight rows
// with 128 or 64 tokens to a tile 0.56 and 0.31, a round of SM-pair tiles 0.325
// (128 wide) and 0.48 (256 wide).  For example 4096 x 11008, 160 tokens:
// 28.3, 30.8, 31.8 and 44.7 us; 512 tokens: 49.0, 52.5, 32.9, 45.5; 12288 x
// 4096, 160 tokens: 40.8, 22.4, 26.1, 20.9.
static pgf8_status block_linear_launch(const BlockLaunch &L)
{
    using B16 = BlockCfg<16, 6, 4>;
    using B32 = BlockCfg<32, 5, 4>;
    using B64 = BlockCfg<64, 4, 4>;
    using B128 = BlockCfg<128, 6, 4>;
    if (L.M <= 16)
        return launch_block<B16>(L, plan_block<B16>(L, 0.25).splits);
    if (L.M <= 32)
        return launch_block<B32>(L, plan_block<B32>(L, 0.27).splits);
    const BlockPlan p64 = plan_block<B64>(L, 0.31);
    if (L.M <= 64)
        return launch_block<B64>(L, p64.splits);
    const BlockPlan p128 = plan_block<B128>(L, 0.56);
    const int64_t pairs = num_sms() / 2, mt = ceil_div(L.M, 256), kb = ceil_div(L.K, 128);
    const double wide = static_cast<double>(ceil_div(mt * ceil_div(L.N, 256), pairs)) * kb * 0.48;
    const double narrow = static_cast<double>(ceil_div(mt * ceil_div(L.N, 128), pairs)) * kb * 0.325;
    if (std::fmin(wide, narrow) < std::fmin(p64.us, p128.us))
        return narrow < wide ? launch_block_pair<BlockPairCfg<128, 7>>(L) : launch_block_pair<BlockPairCfg<256, 5>>(L);
    return p64.us < p128.us ? launch_block<B64>(L, p64.splits) : launch_block<B128>(L, p128.splits);
}

// At most this many tokens are quantised in the GEMM itself (without
// PGF8_FLAG_OVERLAP_PREVIOUS: in a chain the quantisation kernel of a layer hides
// its GEMM's first weight loads behind the layer before).
constexpr int kBlockFusedTokens = 4;

// The layer from unquantised activations in one launch; the same codes, scales
// and sums as in two.  False where a CTA's k-blocks would not fit its shared
// memory, where y lies over x, and beyond 32 (token, k-block) groups a CTA, two
// for each eight of its epilogue threads: the weights wait for them.  Us on the
// GPU in one launch / two, by groups a CTA (N x K, bf16):
//   up to 32:  4096 x 4096 7.4 / 8.1 (1 token), 7.8 / 8.5 (4);
//              1024 x 8192 7.4 / 8.2, 7.8 / 8.2; 4096 x 11008 11.2 / 12.8 (1), 12.2 /
//              13.3 (2); 12288 x 4096 12.8 / 13.6, 13.6 / 14.0; 8192 x 8192 14.5 / 15.8,
//              15.4 / 15.9
//   33 to 44:  4096 x 11008 12.8 / 13.5 (3), 13.0 / 13.5 (4)
//   48 to 64:  12288 x 4096 14.3 / 14.1 (3), 15.0 / 14.2 (4); 8192 x 8192 16.3 / 16.0, 16.9
//              / 16.0
static bool block_fused_launch(const BlockLaunch &L, int xdt, pgf8_status &st)
{
    using B = BlockCfg<16, 6, 4>;
    const int splits = plan_block<B>(L, 0.25).splits;
    const int64_t own = ceil_div(ceil_div(L.K, 128), splits);
    if (L.M > kBlockFusedTokens || own > B::kSlots || L.M * own > 32)
        return false;
    // every CTA reads x, some of them after others have written their part of y
    const uintptr_t x = reinterpret_cast<uintptr_t>(L.x), y = reinterpret_cast<uintptr_t>(L.y);
    if (x < y + static_cast<uintptr_t>(L.M * L.N * dtype_bytes(L.ydt)) &&
        y < x + static_cast<uintptr_t>(((L.M - 1) * L.ldx + L.K) * dtype_bytes(xdt)))
        return false;
    st = xdt == PGF8_F32   ? launch_block<BlockCfg<16, 4, 4, 1>>(L, splits)
         : xdt == PGF8_F16 ? launch_block<BlockCfg<16, 4, 4, 2>>(L, splits)
                           : launch_block<BlockCfg<16, 4, 4, 3>>(L, splits);
    return true;
}

// Shapes, types and pointers of a block-scaled linear layer, activations aside.
static pgf8_status check_block_linear(int64_t M, int64_t K, const uint8_t *wq, const float *sw, int64_t N,
                                      const void *y, int ydt)
{
    if (M < 0 || N < 16 || K < 16 || M > (1ll << 23) || N > (1ll << 30) || K > (1ll << 30))
        return PGF8_ERR_INVALID_ARG;
    if (K % 16 != 0 || N % 16 != 0)
        return PGF8_ERR_ALIGNMENT;
    if (M == 0)
        return PGF8_OK;
    if (!wq || !sw || !y)
        return PGF8_ERR_INVALID_ARG;
    if (dtype_bytes(ydt) == 0)
        return PGF8_ERR_UNSUPPORTED;
    if (!aligned16(wq) || !aligned16(y) || !aligned4(sw))
        return PGF8_ERR_ALIGNMENT;
    return PGF8_OK;
}

static size_t block_scales_offset(int64_t M, int64_t K)
{
    return round_up(static_cast<size_t>(M) * static_cast<size_t>(K), 256);
}

} // namespace pgf8

using namespace pgf8;

extern "C" {

pgf8_status pgf8_fp8_quantize_blocks(const void *x, pgf8_dtype xdt, int64_t batch, int64_t rows, int64_t cols,
                                     int64_t ldx, int64_t ldb, int32_t block_rows, uint8_t *q, float *scales,
                                     int32_t flags, void *stream)
{
    pgf8_status st = check_block_quant(x, xdt, batch, rows, cols, ldx, ldb, block_rows, q, scales);
    if (st != PGF8_OK)
        return st;
    if (batch == 0 || rows == 0)
        return PGF8_OK;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const int pdl = (flags & PGF8_FLAG_OVERLAP_PREVIOUS) ? 1 : 0;
    if (block_rows == 1) {
        if (batch > 1) {
            // the matrices' rows as one list: they have to follow one another
            if (ldb != rows * ldx)
                return PGF8_ERR_UNSUPPORTED;
            rows *= batch;
        }
        return row_blocks_launch(x, xdt, rows, cols, ldx, q, scales, cs, pdl);
    }
    const uint32_t rb = static_cast<uint32_t>(ceil_div(rows, 128)), cb = static_cast<uint32_t>(ceil_div(cols, 128));
    const unsigned grid = static_cast<unsigned>(batch * rb * cb);
    return by_dtype(xdt, [&](auto *t) {
        using T = std::remove_cv_t<std::remove_pointer_t<decltype(t)>>;
        return launch_quant(quantize_tiles_kernel<T>, grid, cs, pdl, static_cast<const T *>(x), rows, cols, ldx, ldb,
                            rb, cb, q, scales);
    });
}

pgf8_status pgf8_fp8_silu_mul_quantize_blocks(const void *gu, pgf8_dtype gdt, int64_t rows, int64_t inter,
                                              int64_t ldg, uint8_t *q, float *scales, int32_t flags, void *stream)
{
    if (inter < 0 || inter > (1ll << 30) || ldg < 2 * inter)
        return PGF8_ERR_INVALID_ARG;
    pgf8_status st = check_block_quant(gu, gdt, 1, rows, inter, ldg, 0, 1, q, scales);
    if (st != PGF8_OK)
        return st;
    if (rows == 0)
        return PGF8_OK;
    const int64_t groups = ceil_div(inter, 128);
    const uint64_t total = static_cast<uint64_t>(rows) * static_cast<uint64_t>(groups);
    const unsigned grid = static_cast<unsigned>((total + 31) / 32);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const int pdl = (flags & PGF8_FLAG_OVERLAP_PREVIOUS) ? 1 : 0;
    return by_dtype(gdt, [&](auto *t) {
        using T = std::remove_cv_t<std::remove_pointer_t<decltype(t)>>;
        return launch_quant(silu_mul_row_blocks_kernel<T>, grid, cs, pdl, static_cast<const T *>(gu), total,
                            static_cast<uint32_t>(groups), inter, ldg, q, scales);
    });
}

pgf8_status pgf8_fp8_block_linear(const uint8_t *aq, const float *sa, int64_t M, int64_t K, const uint8_t *wq,
                                  const float *sw, int64_t N, void *y, pgf8_dtype ydt, int32_t flags, void *stream)
{
    pgf8_status st = check_block_linear(M, K, wq, sw, N, y, ydt);
    if (st != PGF8_OK || M == 0)
        return st;
    if (!aq || !sa)
        return PGF8_ERR_INVALID_ARG;
    if (!aligned16(aq) || !aligned4(sa))
        return PGF8_ERR_ALIGNMENT;
    BlockLaunch L = {aq, wq, sa, sw, y, ydt, M, N, K, (flags & PGF8_FLAG_OVERLAP_PREVIOUS) ? 1 : 0,
                     static_cast<cudaStream_t>(stream)};
    return block_linear_launch(L);
}

size_t pgf8_fp8_block_linear_dynamic_scales_offset(int64_t M, int64_t K)
{
    return M < 0 || K < 0 ? 0 : block_scales_offset(M, K);
}

size_t pgf8_fp8_block_linear_dynamic_workspace_size(int64_t M, int64_t K)
{
    if (M <= 0 || K <= 0)
        return 0;
    return block_scales_offset(M, K) + round_up(static_cast<size_t>(M) * ceil_div(K, 128) * 4, 256);
}

pgf8_status pgf8_fp8_block_linear_dynamic(const void *x, pgf8_dtype xdt, int64_t M, int64_t K, int64_t ldx,
                                          const uint8_t *wq, const float *sw, int64_t N, void *y, pgf8_dtype ydt,
                                          void *workspace, size_t workspace_bytes, int32_t flags, void *stream)
{
    pgf8_status st = check_block_linear(M, K, wq, sw, N, y, ydt);
    if (st != PGF8_OK || M == 0)
        return st;
    if (!workspace || workspace_bytes < pgf8_fp8_block_linear_dynamic_workspace_size(M, K))
        return PGF8_ERR_INVALID_ARG;
    if (!aligned16(workspace))
        return PGF8_ERR_ALIGNMENT;
    uint8_t *aq = static_cast<uint8_t *>(workspace);
    float *sa = reinterpret_cast<float *>(aq + block_scales_offset(M, K));
    st = check_block_quant(x, xdt, 1, M, K, ldx, 0, 1, aq, sa);
    if (st != PGF8_OK)
        return st;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    // weights may be read early: the quantisation writes only aq / sa, and the
    // one-launch form follows everything before it
    BlockLaunch L = {aq, wq, sa, sw, y, ydt, M, N, K, 1, cs, x, ldx};
    if (!(flags & PGF8_FLAG_OVERLAP_PREVIOUS) && M <= kBlockFusedTokens && block_fused_launch(L, xdt, st))
        return st;
    st = row_blocks_launch(x, xdt, M, K, ldx, aq, sa, cs, (flags & PGF8_FLAG_OVERLAP_PREVIOUS) ? 1 : 0);
    if (st != PGF8_OK)
        return st;
    return block_linear_launch(L);
}

} // extern "C"
