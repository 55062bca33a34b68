// Entry points of the mixture-of-experts layer; specified in include/pgf8.h.
// Included by pgf8_api.cu after block_api.cuh.
#pragma once

#include "moe.cuh"

namespace pgf8 {

// Regions of the workspace, each 256-byte aligned.
struct MoeWorkspace {
    size_t xq, sx, hq, sh, active, experts, tok, weight, bytes;
    MoeWorkspace(int64_t T, int64_t H, int64_t F, int64_t E, int64_t K)
    {
        size_t at = 0;
        auto take = [&at](size_t n) {
            const size_t here = at;
            at += round_up(n, 256);
            return here;
        };
        const int64_t rows = T * K, most = E < rows ? E : rows;
        xq = take(T * H);
        sx = take(T * ceil_div(H, 128) * 4);
        hq = take(rows * F);
        sh = take(rows * ceil_div(F, 128) * 4);
        active = take(4);
        experts = take(most * sizeof(int4));
        tok = take(rows * 4);
        weight = take(rows * 4);
        bytes = at;
    }
};

// given: ids and weights are given, of which any number may lie outside the experts.
static pgf8_status check_moe_sizes(int64_t T, int64_t H, int64_t F, int64_t E, int64_t K, bool given)
{
    if (T < 0 || H < 16 || F < 16 || E < 1 || K < 1 || (K > E && !given))
        return PGF8_ERR_INVALID_ARG;
    if (T > kMoeMaxTokens || E > kMoeMaxExperts || K > kMoeMaxTopK || H > (1 << 20) || F > (1 << 20) ||
        2 * E * F > 2147483647ll - 128 || E * H > 2147483647ll - 128)
        return PGF8_ERR_UNSUPPORTED;
    if (H % 16 != 0 || F % 16 != 0)
        return PGF8_ERR_ALIGNMENT;
    return PGF8_OK;
}

static pgf8_status check_moe(const pgf8_fp8_moe_layer &a)
{
    pgf8_status st = check_moe_sizes(a.tokens, a.hidden, a.inter, a.experts, a.top_k, !a.logits);
    if (st != PGF8_OK)
        return st;
    if (a.score != kMoeSoftmax && a.score != kMoeSigmoid)
        return PGF8_ERR_INVALID_ARG;
    if (dtype_bytes(a.xdt) == 0 || dtype_bytes(a.ydt) == 0)
        return PGF8_ERR_UNSUPPORTED;
    if (a.tokens == 0)
        return PGF8_OK;
    if (!a.x || !a.w13 || !a.s13 || !a.w2 || !a.s2 || !a.y || !a.workspace || a.ldx < a.hidden ||
        a.ldx > (1ll << 40))
        return PGF8_ERR_INVALID_ARG;
    if (a.logits) {
        if (dtype_bytes(a.ldt) == 0)
            return PGF8_ERR_UNSUPPORTED;
        if (a.ldl < a.experts || a.ldl > (1ll << 40) || !std::isfinite(a.factor))
            return PGF8_ERR_INVALID_ARG;
        if ((reinterpret_cast<uintptr_t>(a.logits) % dtype_bytes(a.ldt)) != 0)
            return PGF8_ERR_ALIGNMENT;
    } else if (!a.ids || !a.weights) {
        return PGF8_ERR_INVALID_ARG;
    }
    if (a.workspace_bytes < MoeWorkspace(a.tokens, a.hidden, a.inter, a.experts, a.top_k).bytes)
        return PGF8_ERR_INVALID_ARG;
    if ((a.ldx * dtype_bytes(a.xdt)) % 16 != 0 || !aligned16(a.x) || !aligned16(a.w13) || !aligned16(a.w2) ||
        !aligned16(a.y) || !aligned16(a.workspace) || !aligned4(a.s13) || !aligned4(a.s2) || !aligned4(a.ids) ||
        !aligned4(a.weights))
        return PGF8_ERR_ALIGNMENT;
    return PGF8_OK;
}

// Launches a kernel of clusters along z with programmatic stream serialization.
template <typename... Args>
static pgf8_status launch_moe(void (*kernel)(Args...), dim3 grid, int threads, int smem, cudaStream_t cs, Args... args)
{
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = cs;
    cudaLaunchAttribute attrs[2];
    fill_attrs(cfg, attrs, static_cast<int>(grid.z), 1);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e == cudaSuccess ? PGF8_OK : cuda_fail(e);
}

// kb_us: see stream_plan (two weight tiles a k-block here).  Us of the layer with
// one of the two kernels' splits set and the other's as chosen:
//                                        gate+up 1    2    3    4    6   takes
//   one token, 64 experts of 2048 x 1408     22.9 21.0 21.4 21.9 26.2    4
//   13 tokens, 8 experts of 4096 x 7184       119  126  122  130  146    1
//   30 tokens, 64 experts of 2048 x 1408      105  104  117  126  157    1
//   64 tokens, 128 experts of 2048 x 768      139  163  206  235  310    1
//                                        down    1    2    3    4    6    8   takes
//   one token                                39.9 30.5 25.6 24.0 22.3 21.7    8
//   13 tokens                                 230  160  142  130  119  118    8
//   30 tokens                                 331  202  155  136  117  106    8
//   64 tokens (16 clusters of 8 do not fit)   389  237  188  164  139  170    6
template <class C>
static pgf8_status launch_moe_up(const CUtensorMap &tmX, const CUtensorMap &tmW, const MoeUpParams &p, int most,
                                 double kb_us, cudaStream_t cs)
{
    static ClusterFit c;
    const int *fit = nullptr;
    const cudaError_t e = cluster_fit(c, moe_gate_up_kernel<C>, C::kThreads, C::kSmemBytes, C::kSmemBytes, C::CTAS, fit);
    if (e != cudaSuccess)
        return cuda_fail(e);
    const int64_t tiles = static_cast<int64_t>(most) * p.fblocks;
    const int splits = stream_plan(tiles, p.hblocks, kb_us, 32768.0 * tiles * p.hblocks, fit).splits;
    return launch_moe(moe_gate_up_kernel<C>,
                      dim3(static_cast<unsigned>(p.fblocks), static_cast<unsigned>(most),
                           static_cast<unsigned>(splits)),
                      C::kThreads, C::kSmemBytes, cs, tmX, tmW, p);
}

template <class C>
static pgf8_status launch_moe_down(const CUtensorMap &tmH, const CUtensorMap &tmW, const MoeDownParams &p,
                                   double kb_us, cudaStream_t cs)
{
    constexpr int kMost = C::kSmemBytes + kMoeMaxExperts * 16 + C::BN * kMoeMaxTopK * 8;
    constexpr int kHalf = kMost < 113 * 1024 ? kMost : 113 * 1024;   // two CTAs on an SM
    static_assert(kMost <= 227 * 1024, "shared memory");
    const int smem = C::kSmemBytes + p.max_active * 16 + p.pairs * 8;
    static ClusterFit two, one;
    const int *fit = nullptr;
    const bool half = smem <= kHalf;
    const cudaError_t e = half ? cluster_fit(two, moe_down_kernel<C>, C::kThreads, kMost, kHalf, 2, fit)
                               : cluster_fit(one, moe_down_kernel<C>, C::kThreads, kMost, kMost, 1, fit);
    if (e != cudaSuccess)
        return cuda_fail(e);
    const int64_t hb = (p.H + 127) / 128, units = static_cast<int64_t>(p.max_active) * p.fblocks;
    const int splits = stream_plan(hb, units, kb_us, 16384.0 * hb * units, fit).splits;
    return launch_moe(moe_down_kernel<C>, dim3(static_cast<unsigned>(hb), 1, static_cast<unsigned>(splits)),
                      C::kThreads, smem, cs, tmH, tmW, p);
}

} // namespace pgf8

extern "C" {

size_t pgf8_fp8_moe_workspace_size(int64_t tokens, int64_t hidden, int64_t inter, int64_t experts, int64_t top_k)
{
    if (tokens == 0 || check_moe_sizes(tokens, hidden, inter, experts, top_k, false) != PGF8_OK)
        return 0;
    return MoeWorkspace(tokens, hidden, inter, experts, top_k).bytes;
}

pgf8_status pgf8_fp8_moe(const pgf8_fp8_moe_layer *layer, int32_t flags, void *stream)
{
    if (!layer)
        return PGF8_ERR_INVALID_ARG;
    const pgf8_fp8_moe_layer &a = *layer;
    pgf8_status st = check_moe(a);
    if (st != PGF8_OK || a.tokens == 0)
        return st;
    const MoeWorkspace ws(a.tokens, a.hidden, a.inter, a.experts, a.top_k);
    uint8_t *base = static_cast<uint8_t *>(a.workspace);
    auto f32 = [base](size_t off) { return reinterpret_cast<float *>(base + off); };
    auto i32 = [base](size_t off) { return reinterpret_cast<int *>(base + off); };
    const MoePlan plan = {i32(ws.active), reinterpret_cast<int4 *>(base + ws.experts), i32(ws.tok), f32(ws.weight)};
    const int T = static_cast<int>(a.tokens), H = static_cast<int>(a.hidden), F = static_cast<int>(a.inter);
    const int E = static_cast<int>(a.experts), K = static_cast<int>(a.top_k);
    const int hblocks = (H + 127) / 128, fblocks = (F + 127) / 128;
    const int pairs = T * K, most = E < pairs ? E : pairs;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const int bn = T <= 16 ? 16 : T <= 32 ? 32 : 64;

    CUtensorMap tmX, tmW13, tmH, tmW2;
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    if (!make_map(&tmX, base + ws.xq, u8, 1, T, H, 128, bn, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&tmW13, a.w13, u8, 1, static_cast<uint64_t>(E) * 2 * F, H, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&tmH, base + ws.hq, u8, 1, pairs, F, 128, 16, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&tmW2, a.w2, u8, 1, static_cast<uint64_t>(E) * H, F, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B))
        return PGF8_ERR_UNSUPPORTED;

    MoeRouteParams r;
    r.x = a.x;
    r.ldx = a.ldx;
    r.T = T;
    r.H = H;
    r.hblocks = hblocks;
    r.xq = base + ws.xq;
    r.sx = f32(ws.sx);
    r.logits = a.logits;
    r.ldt = a.ldt;
    r.ldl = a.ldl;
    r.E = E;
    r.K = K;
    r.score = a.score;
    r.renorm = a.renormalise != 0;
    r.factor = a.factor;
    r.ids = a.ids;
    r.weights = a.weights;
    r.plan = plan;
    // eight tokens to a routing CTA, the CTAs of one cluster; whole clusters of 32-group CTAs for x
    int route = 1;
    while (a.logits && route * (kMoePlanThreads / 32) < T)
        route *= 2;
    r.route_ctas = route;
    const int64_t quant = ceil_div(static_cast<int64_t>(T) * hblocks, kMoePlanThreads / 8);
    const unsigned grid = static_cast<unsigned>(route + ceil_div(quant, route) * route);
    st = by_dtype(a.xdt, [&](auto *x) {
        using X = std::remove_cv_t<std::remove_pointer_t<decltype(x)>>;
        cudaLaunchConfig_t cfg;
        std::memset(&cfg, 0, sizeof(cfg));
        cfg.gridDim = dim3(grid, 1, 1);
        cfg.blockDim = dim3(kMoePlanThreads, 1, 1);
        cfg.stream = cs;
        cudaLaunchAttribute attrs[2];
        fill_attrs(cfg, attrs, 1, (flags & PGF8_FLAG_OVERLAP_PREVIOUS) ? 1 : 0, route);
        const cudaError_t e = cudaLaunchKernelEx(&cfg, moe_plan_kernel<X>, r);
        return e == cudaSuccess ? PGF8_OK : cuda_fail(e);
    });
    if (st != PGF8_OK)
        return st;

    const MoeUpParams up = {T, F, hblocks, fblocks, f32(ws.sx), a.s13, base + ws.hq, f32(ws.sh), plan};
    if (bn == 16)
        st = launch_moe_up<MoeUpCfg<16, 3, 4, 2>>(tmX, tmW13, up, most, 0.40, cs);
    else if (bn == 32)
        st = launch_moe_up<MoeUpCfg<32, 3, 4, 2>>(tmX, tmW13, up, most, 0.45, cs);
    else   // one CTA to an SM: two have 96 registers a thread and two stages (64 tokens of 128 experts: 185 us, 139)
        st = launch_moe_up<MoeUpCfg<64, 5, 2, 1>>(tmX, tmW13, up, most, 0.60, cs);
    if (st != PGF8_OK)
        return st;

    const MoeDownParams down = {T, H, fblocks, most, pairs, f32(ws.sh), a.s2, a.y, a.ydt, plan};
    if (bn == 16)
        return launch_moe_down<MoeDownCfg<16, 5, 4>>(tmH, tmW2, down, 0.28, cs);
    if (bn == 32)
        return launch_moe_down<MoeDownCfg<32, 4, 4>>(tmH, tmW2, down, 0.30, cs);
    return launch_moe_down<MoeDownCfg<64, 6, 4>>(tmH, tmW2, down, 0.37, cs);
}

} // extern "C"
