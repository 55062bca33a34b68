// A mixture-of-experts layer for a few tokens (T <= 64), E4M3 weights with
// 128 x 128 block scales, in three launches:
//   moe_plan_kernel     routing (top-k of the logits) by a cluster of up to eight
//                       CTAs, whose first then lists the chosen experts' tokens;
//                       the other CTAs quantise x per 1 x 128 group
//   moe_gate_up_kernel  for every chosen expert and 128 hidden features:
//                       g = xq W1, u = xq W3, h = silu(g) u in binary32, E4M3
//                       codes of h with one scale per 1 x 128 group
//   moe_down_kernel     y[t] = sum over the chosen experts of w[t, e] hq W2[e]
//
// A few tokens touch nearly as many experts as they choose, so the layer is
// a stream of the chosen experts' weights (3 H F bytes each) and everything
// else has to hide behind it.  Both products keep the weights as the 128-row
// MMA operand and the tokens as the narrow one, accumulate one k-block at a
// time in tensor memory and add it with its scales in registers, as
// gemm_block.cuh does, and split their sums over a thread-block cluster,
// joined in rank order (deterministic, no atomics on sums).
//   gate+up: x's codes are the same for every expert, so the token operand is
//     all T tokens whatever the expert's own tokens are: one contiguous tile
//     instead of a gather; the MMA has time for the unused columns.
//   down: an expert's tokens are consecutive rows of the hidden codes
//     (sorted by expert, then token), only those are loaded; the experts'
//     products run one after another through the same CTA, so the sum over
//     experts is taken in shared memory in expert order and needs no
//     combining launch.
#pragma once

#include "gemm_block.cuh"
#include "quantize_blocks.cuh"

namespace pgf8 {

constexpr int kMoeMaxTokens = 64;     // one 64-bit mask of tokens per expert
constexpr int kMoeMaxExperts = 512;   // 16 logits a lane
constexpr int kMoeMaxTopK = 16;
constexpr int kMoePlanThreads = 256;  // of each CTA: eight tokens to route, or 32 groups to quantise

enum : int { kMoeSoftmax = 0, kMoeSigmoid = 1 };

// What the plan kernel leaves for the other two.
struct MoePlan {
    int *active;      // [1] number of chosen experts
    int4 *experts;    // [min(E, T k)] (expert, first row, rows, 0) in expert order
    int *tok;         // [T k] token of each row of the hidden codes
    float *weight;    // [T k] its weight
};

struct MoeRouteParams {
    const void *x;         // [T, H], row stride ldx
    int64_t ldx;
    int T, H, hblocks;     // hblocks = ceil(H / 128)
    uint8_t *xq;           // [T, H]
    float *sx;             // [T, hblocks]
    const void *logits;    // [T, E], row stride ldl; null: ids / weights are given
    int ldt;               // pgf8_dtype of logits
    int64_t ldl;
    int E, K;              // K choices a token
    int score, renorm;
    float factor;
    int *ids;              // [T, K]; written with logits (may then be null), read without
    float *weights;        // [T, K]
    int route_ctas;        // CTAs of a cluster: 1, 2, 4 or 8
    MoePlan plan;
};

// Largest logits first: an order-preserving 32-bit key of v (-0 as +0, which are ties).
__device__ __forceinline__ uint32_t logit_key(float v)
{
    const uint32_t u = __float_as_uint(v + 0.0f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float key_logit(uint32_t key)
{
    return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}

// Sigmoids of a token that has chosen a logit below kFarLogit (lane j: choice j,
// the largest first).  There 1 + e^-f overflows sooner than e^f / (1 + e^f)
// vanishes, and the shares of such sigmoids are ordinary numbers although the
// sigmoids may all be below the smallest one: with renorm they are taken
// relative to the largest, which goes out with the division by their sum.
// Not inlined: rare, and inlined it takes the plan kernel from 64 to 76
// registers a thread.
constexpr float kFarLogit = -64.0f;

__device__ __noinline__ float far_sigmoid(bool chosen, float f, int renorm)
{
    const float largest = __shfl_sync(0xffffffffu, f, 0);
    const float unit = renorm && largest < 0.0f ? largest : 0.0f;
    if (!chosen)
        return 0.0f;
    return f > 0.0f ? __fdiv_rn(1.0f, 1.0f + expf(-f)) : __fdiv_rn(expf(f - unit), 1.0f + expf(f));
}

__device__ __forceinline__ void st_shared_cluster_u32(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// One warp routes one token: the K largest logits (ties to the lowest index;
// NaN and -inf are never chosen: id -1, weight 0), their softmax over all E or
// their sigmoids, divided by their sum if asked, times factor.  PER logits a
// lane (E <= 32 PER).  Each choice is two warp reductions in hardware: the
// largest key, then the lowest index that has it.  The choices go to sid / sw
// in the shared memory of the cluster's first CTA.
template <int PER>
__device__ __forceinline__ void route_token(const MoeRouteParams &p, int t, uint32_t sid, uint32_t sw)
{
    const int lane = threadIdx.x & 31;
    const float ninf = -INFINITY;
    const int64_t row = static_cast<int64_t>(t) * p.ldl;
    float v[PER];
    uint32_t key[PER];   // 0 for a logit that cannot be chosen
    float top = ninf;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        float f = ninf;
        if (e < p.E) {
            if (p.ldt == 0)
                f = static_cast<const float *>(p.logits)[row + e];
            else if (p.ldt == 1)
                f = __half2float(static_cast<const __half *>(p.logits)[row + e]);
            else
                f = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.logits)[row + e]);
        }
        v[i] = f != f ? ninf : f;
        key[i] = v[i] > ninf ? logit_key(v[i]) : 0u;
        top = fmaxf(top, v[i]);
    }
    float sum = 0.0f;
    if (p.score == kMoeSoftmax) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
        for (int i = 0; i < PER; ++i)
            sum += v[i] > ninf ? expf(v[i] - top) : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    uint32_t my_key = 0u;   // lane j keeps choice j
    int my_id = -1;
    for (int j = 0; j < p.K; ++j) {
        uint32_t best = 0u;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] > best) {
                best = key[i];
                at = lane + 32 * i;
            }
        const uint32_t most = __reduce_max_sync(0xffffffffu, best);
        if (most == 0u)
            break;   // nothing left to choose (the same in every lane)
        const int id = static_cast<int>(
            __reduce_min_sync(0xffffffffu, best == most ? static_cast<unsigned>(at) : 0x7FFFFFFFu));
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (id == lane + 32 * i)
                key[i] = 0u;
        if (lane == j) {
            my_key = most;
            my_id = id;
        }
    }
    float mine = 0.0f;
    if (my_id >= 0) {
        const float f = key_logit(my_key);
        mine = p.score == kMoeSoftmax ? __fdiv_rn(expf(f - top), sum) : __fdiv_rn(1.0f, 1.0f + expf(-f));
    }
    if (p.score != kMoeSoftmax && __any_sync(0xffffffffu, my_id >= 0 && key_logit(my_key) < kFarLogit))
        mine = far_sigmoid(my_id >= 0, key_logit(my_key), p.renorm);
    if (p.renorm) {
        float all = mine;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            all += __shfl_xor_sync(0xffffffffu, all, o);
        mine = all != 0.0f ? __fdiv_rn(mine, all) : 0.0f;
    }
    mine = my_id >= 0 ? mine * p.factor : 0.0f;
    if (lane < p.K) {
        const int at = t * p.K + lane;
        st_shared_cluster_u32(sid + at * 4, static_cast<uint32_t>(my_id));
        st_shared_cluster_u32(sw + at * 4, __float_as_uint(mine));
        if (p.ids)
            p.ids[at] = my_id;
        if (p.weights)
            p.weights[at] = mine;
    }
}

// Inclusive sum over the CTA's kMoePlanThreads threads (red: one int a warp).
__device__ __forceinline__ int plan_scan(int v, int *red)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o)
            v += u;
    }
    if (lane == 31)
        red[warp] = v;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int w = 0; w < kMoePlanThreads / 32; ++w)
        before += w < warp ? red[w] : 0;
    return v + before;
}

// Cluster 0 routes (eight tokens to a CTA) and its first CTA plans; the other
// clusters' CTAs quantise x, 32 groups each.
template <typename T> __global__ void __launch_bounds__(kMoePlanThreads) moe_plan_kernel(const MoeRouteParams p)
{
    static_assert(kMoeMaxExperts == 2 * kMoePlanThreads, "two experts a thread");
    const bool routes = static_cast<int>(blockIdx.x) < p.route_ctas;
    if (routes && p.route_ctas > 1)
        cluster_arrive_relaxed();   // this CTA runs: the others may write to its shared memory
    grid_launch_dependents();
    grid_dependency_wait();
    const int tid = threadIdx.x;
    if (!routes) {
        const int g = (static_cast<int>(blockIdx.x) - p.route_ctas) * (kMoePlanThreads / 8) + (tid >> 3);
        const int row = g / p.hblocks, grp = g - row * p.hblocks;
        const int c = grp * 128 + (tid & 7) * 16;
        const bool live = row < p.T && c < p.H;
        Vec16<T> v;
        if (live)
            v.load(static_cast<const T *>(p.x) + static_cast<int64_t>(row) * p.ldx + c);
        const GroupScale g8(v.v, live);
        if (!live)
            return;
        *reinterpret_cast<uint4 *>(p.xq + static_cast<int64_t>(row) * p.H + c) = g8.encode(v.v);
        if ((tid & 7) == 0)
            p.sx[row * p.hblocks + grp] = g8.d.s;
        return;
    }

    __shared__ int sid[kMoeMaxTokens * kMoeMaxTopK];
    __shared__ float sw[kMoeMaxTokens * kMoeMaxTopK];
    __shared__ unsigned mask[kMoeMaxExperts][2];   // tokens of each expert
    __shared__ int first[kMoeMaxExperts];          // its first row
    __shared__ int red[kMoePlanThreads / 32];
    const int pairs = p.T * p.K;
    for (int e = tid; e < kMoeMaxExperts; e += kMoePlanThreads)
        mask[e][0] = mask[e][1] = 0u;
    if (p.route_ctas > 1)
        cluster_wait_acquire();
    if (p.logits) {
        const int t = static_cast<int>(blockIdx.x) * (kMoePlanThreads / 32) + (tid >> 5);
        if (t < p.T) {
            const uint32_t id0 = map_shared_rank(smem_u32(sid), 0), w0 = map_shared_rank(smem_u32(sw), 0);
            if (p.E <= 64)
                route_token<2>(p, t, id0, w0);
            else if (p.E <= 128)
                route_token<4>(p, t, id0, w0);
            else if (p.E <= 256)
                route_token<8>(p, t, id0, w0);
            else
                route_token<16>(p, t, id0, w0);
        }
        __syncwarp();
        if (p.route_ctas > 1) {
            cluster_sync_all();
            if (blockIdx.x > 0)
                return;
        }
    } else {
        for (int i = tid; i < pairs; i += kMoePlanThreads) {
            sid[i] = p.ids[i];
            sw[i] = p.weights[i];
        }
    }
    __syncthreads();
    auto expert = [&](int i) {   // of pair i, -1 for a slot that is left out
        const int e = sid[i];
        return e >= 0 && e < p.E ? e : -1;
    };
    for (int i = tid; i < pairs; i += kMoePlanThreads) {
        const int e = expert(i), t = i / p.K;
        if (e >= 0)
            atomicOr(&mask[e][t >> 5], 1u << (t & 31));
    }
    __syncthreads();
    const int e0 = 2 * tid;
    const int rows0 = __popc(mask[e0][0]) + __popc(mask[e0][1]);
    const int rows1 = __popc(mask[e0 + 1][0]) + __popc(mask[e0 + 1][1]);
    // both sums in one scan: rows (at most 1024) above the count of experts (at most 512)
    const int mine = ((rows0 + rows1) << 16) | ((rows0 > 0) + (rows1 > 0));
    const int both = plan_scan(mine, red), before = both - mine;
    first[e0] = before >> 16;
    first[e0 + 1] = (before >> 16) + rows0;
    int n = before & 0xFFFF;
    if (rows0 > 0)
        p.plan.experts[n++] = make_int4(e0, first[e0], rows0, 0);
    if (rows1 > 0)
        p.plan.experts[n] = make_int4(e0 + 1, first[e0 + 1], rows1, 0);
    if (tid == kMoePlanThreads - 1)
        *p.plan.active = both & 0xFFFF;
    __syncthreads();
    for (int i = tid; i < pairs; i += kMoePlanThreads) {
        const int e = expert(i);
        if (e < 0)
            continue;
        // a token that names an expert twice is one row with both weights
        const int t = i / p.K;
        float w = 0.0f;
        bool again = false;
        for (int j = t * p.K; j < (t + 1) * p.K; ++j)
            if (sid[j] == e) {
                again = again || j < i;
                w += sw[j];
            }
        if (!again) {
            const unsigned lo = t < 32 ? (1u << t) - 1u : 0xFFFFFFFFu;
            const unsigned hi = t < 32 ? 0u : (1u << (t - 32)) - 1u;
            const int row = first[e] + __popc(mask[e][0] & lo) + __popc(mask[e][1] & hi);
            p.plan.tok[row] = t;
            p.plan.weight[row] = w;
        }
    }
}

// ------------------------------------------------------------------ gate + up
template <int BN_, int STAGES_, int NBUF_, int CTAS_> struct MoeUpCfg {
    static constexpr int BN = BN_;
    static constexpr int STAGES = STAGES_;
    static constexpr int CTAS = CTAS_;                 // per SM
    static constexpr int NBUF = NBUF_;                 // buffers of 2 BN columns (gate, up)
    static constexpr int COLS = BN < 32 ? BN : 32;     // tokens of an epilogue thread
    static constexpr int kEpi = 128 * (BN / COLS);     // epilogue threads
    static constexpr int kThreads = 64 + kEpi;
    static constexpr int kTileA = 128 * 128;
    static constexpr int kStage = 2 * kTileA + BN * 128;
    static constexpr int kTmemCols = NBUF * 2 * BN;
    static constexpr int kRingBytes = STAGES * kStage; // reused for the partial tiles [2][BN][128] f32
    static constexpr int kChunk = BN == 32 ? 4 : 8;    // k-blocks of scales staged at a time
    static constexpr int kScalePitch = BN + 4;
    static constexpr int kScaleOffset = kRingBytes;
    static constexpr int kScaleBytes = 2 * 2 * kChunk * kScalePitch * 4;
    static constexpr int kCtlOffset = kScaleOffset + kScaleBytes;
    static constexpr int kSmemBytes = kCtlOffset + 512 + 1024;
    static_assert(BN == 16 || BN == 32 || BN == 64, "token tile");
    static_assert(STAGES <= 8 && NBUF <= 8, "barriers");
    static_assert((kTmemCols & (kTmemCols - 1)) == 0 && kTmemCols >= 32 && kTmemCols <= 256, "tensor memory");
    static_assert(kRingBytes >= 2 * BN * 128 * 4, "partial tiles");
    static_assert(kSmemBytes <= 227 * 1024 && CTAS * (kSmemBytes + 1024) <= 228 * 1024, "shared memory");
};

struct MoeUpParams {
    int T, F, hblocks, fblocks;
    const float *sx;     // [T, hblocks]
    const float *s13;    // [E, 2, fblocks, hblocks]
    uint8_t *hq;         // [T k, F]
    float *sh;           // [T k, fblocks]
    MoePlan plan;
};

// Grid (fblocks, min(E, T k), splits): cluster of `splits` CTAs along z for
// 128 hidden features of one chosen expert, each a range of k-blocks of H.
template <class C>
__global__ void __launch_bounds__(C::kThreads, C::CTAS)
    moe_gate_up_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                       const MoeUpParams p)
{
    constexpr int BN = C::BN, STAGES = C::STAGES, NBUF = C::NBUF;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *sc = reinterpret_cast<float *>(smem + C::kScaleOffset);
    BlockCtl *ctl = reinterpret_cast<BlockCtl *>(smem + C::kCtlOffset);
    volatile int *abort_flag = &ctl->abort;

    const int warp = warp_index();
    const int lane = threadIdx.x & 31;
    const int f0 = static_cast<int>(blockIdx.x) * 128;
    const int splits = static_cast<int>(gridDim.z);
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.hblocks) * blockIdx.z / splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.hblocks) * (blockIdx.z + 1) / splits);

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int b = 0; b < NBUF; ++b) {
            mbar_init(&ctl->acc_full[b], 1);
            mbar_init(&ctl->acc_empty[b], C::kEpi / 32);
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&ctl->tmem_base, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;

    // The plan comes from the kernel before.  Dependents (the down kernel) may
    // start once every CTA of this grid is past its wait: the plan is complete
    // then, and they read it, and weights, before this grid has finished.
    grid_dependency_wait();
    grid_launch_dependents();
    if (static_cast<int>(blockIdx.y) >= __ldcg(p.plan.active)) {
        // the whole cluster; nothing of it is in flight
        if (warp == 1)
            tmem_dealloc(tmem, C::kTmemCols);
        return;
    }
    const int4 ex = __ldcg(p.plan.experts + blockIdx.y);

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            const uint64_t pol_w = policy_evict_first();
            const uint64_t pol_x = policy_evict_last();
            const int row = ex.x * 2 * p.F + f0;
            int s = 0, issued = 0;
            uint32_t ph = 1;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!wait_step(&ctl->empty[s], ph, abort_flag))
                    break;
                uint8_t *st = smem + s * C::kStage;
                mbar_arrive_expect_tx(&ctl->full[s], C::kStage);
                tma_load_2d_hint(st, &tmW, &ctl->full[s], kb * 128, row, pol_w);
                tma_load_2d_hint(st + C::kTileA, &tmW, &ctl->full[s], kb * 128, row + p.F, pol_w);
                tma_load_2d_hint(st + 2 * C::kTileA, &tmX, &ctl->full[s], kb * 128, 0, pol_x);
                ++issued;
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (*abort_flag) {
                for (int j = 0; j < STAGES && j < issued; ++j)
                    wait_drain(&ctl->full[j], static_cast<uint32_t>((issued - 1 - j) / STAGES) & 1u);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        {
            constexpr uint32_t idesc = make_idesc(128, BN, 0, 0);
            int s = 0, b = 0;
            uint32_t ph = 0, bph = 1;
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb) {
                ok = wait_step(&ctl->acc_empty[b], bph, abort_flag) && wait_step(&ctl->full[s], ph, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t a_addr = smem_u32(smem + s * C::kStage);
                const uint32_t x_addr = a_addr + 2 * C::kTileA;
                if (elect_one()) {
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma_f8f6f4(tmem + (b * 2 + half) * BN, sdesc_sw128(a_addr + half * C::kTileA + k * 32),
                                        sdesc_sw128(x_addr + k * 32), idesc, k > 0 ? 1u : 0u);
                    umma_commit(&ctl->empty[s]);
                    umma_commit(&ctl->acc_full[b]);
                }
                __syncwarp();
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
                if (++b == NBUF) {
                    b = 0;
                    bph ^= 1u;
                }
            }
            if (!ok && elect_one()) {
                umma_commit(&ctl->drain);
                wait_drain(&ctl->drain, 0);
            }
        }
        __syncwarp();
    }

    constexpr int COLS = C::COLS, EPI = C::kEpi;
    float accg[COLS], accu[COLS];
    const int qd = warp & 3;
    const int r = qd * 32 + lane;
    const int col0 = ((warp - 2) >> 2) * COLS;   // this warp's tokens
    if (warp >= 2) {
        // ------------------------------------------------------------ scales and accumulation
#pragma unroll
        for (int j = 0; j < COLS; ++j)
            accg[j] = accu[j] = 0.0f;
        const uint32_t t_row = tmem + (static_cast<uint32_t>(qd * 32) << 16) + static_cast<uint32_t>(col0);
        const int et = static_cast<int>(threadIdx.x) - 64;
        // as in gemm_block.cuh: loaded a chunk ahead, multiplied when stored
        constexpr int CH = C::kChunk, PER = BN * CH / EPI;
        float pre[PER], wg = 0.0f, wu = 0.0f;
        const float *swg = p.s13 + (static_cast<int64_t>(ex.x) * 2 * p.fblocks + blockIdx.x) * p.hblocks;
        const float *swu = swg + static_cast<int64_t>(p.fblocks) * p.hblocks;
        auto fetch = [&](int kb) {
            const int k = kb + (et & (CH - 1));
            wg = k < kb1 ? __ldg(swg + k) : 0.0f;
            wu = k < kb1 ? __ldg(swu + k) : 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int t = (et + EPI * i) / CH;
                pre[i] = (k < kb1 && t < p.T) ? __ldcg(p.sx + t * p.hblocks + k) : 0.0f;
            }
        };
        fetch(kb0);
        int b = 0;
        uint32_t bph = 0;
        bool ok = true;
        for (int i = 0; i < kb1 - kb0; ++i) {
            float *bufg = sc + ((i / CH) & 1) * 2 * CH * C::kScalePitch;
            float *bufu = bufg + CH * C::kScalePitch;
            if (i % CH == 0) {
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const int at = (et & (CH - 1)) * C::kScalePitch + ((et + EPI * j) / CH);
                    bufg[at] = pre[j] * wg;
                    bufu[at] = pre[j] * wu;
                }
                if (i + CH < kb1 - kb0)
                    fetch(kb0 + i + CH);
                bar_sync_epilogue<EPI>();
            }
            ok = ok && wait_step(&ctl->acc_full[b], bph, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
                tc_fence_after();
                const int at = (i % CH) * C::kScalePitch + col0;
                add_scaled<COLS>(t_row + b * 2 * BN, bufg + at, accg);
                add_scaled<COLS>(t_row + b * 2 * BN + BN, bufu + at, accu);
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&ctl->acc_empty[b]);
            }
            if (++b == NBUF) {
                b = 0;
                bph ^= 1u;
            }
        }
    }
    __syncwarp();

    // ---------------------------------------------------------------- partial tiles, gate, codes
    float *part = reinterpret_cast<float *>(smem);
    tc_fence_before();
    __syncthreads();   // the ring is idle
    if (warp >= 2) {
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
            part[(col0 + c) * 128 + r] = accg[c];
            part[(BN + col0 + c) * 128 + r] = accu[c];
        }
    }
    if (splits > 1)
        cluster_sync_all();
    else
        __syncthreads();
    if (warp >= 2) {
        // one warp to a row of hidden codes, four features a lane
        const uint32_t base = smem_u32(part) + lane * 16;
        const int f = f0 + lane * 4;
        for (int i = static_cast<int>(blockIdx.z) + splits * (warp - 2); i < ex.z; i += EPI / 32 * splits) {
            const int row = ex.y + i;
            const uint32_t off = base + __ldcg(p.plan.tok + row) * 512;
            // the partials in rank order, four ranks in flight at a time
            float4 g = make_float4(0.0f, 0.0f, 0.0f, 0.0f), u = g;
#pragma unroll
            for (int z0 = 0; z0 < 8; z0 += 4) {
                if (z0 >= splits)
                    break;
                float4 tg[4], tu[4];
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    if (z0 + z < splits) {
                        const uint32_t a = splits > 1 ? map_shared_rank(off, static_cast<uint32_t>(z0 + z)) : off;
                        tg[z] = ld_shared_cluster_v4_relaxed(a);
                        tu[z] = ld_shared_cluster_v4_relaxed(a + BN * 512);
                    }
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    if (z0 + z < splits) {
                        g = make_float4(g.x + tg[z].x, g.y + tg[z].y, g.z + tg[z].z, g.w + tg[z].w);
                        u = make_float4(u.x + tu[z].x, u.y + tu[z].y, u.z + tu[z].z, u.w + tu[z].w);
                    }
            }
            const bool live = f < p.F;   // F % 16 == 0: a lane's four features exist together
            float h[4] = {silu_mul(g.x, u.x), silu_mul(g.y, u.y), silu_mul(g.z, u.z), silu_mul(g.w, u.w)};
            float a = 0.0f;
            if (live)
                a = fmaxf(fmaxf(fabsf(h[0]), fabsf(h[1])), fmaxf(fabsf(h[2]), fabsf(h[3])));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
            const float s = block_scale(a);
            if (live)
                *reinterpret_cast<uint32_t *>(p.hq + static_cast<int64_t>(row) * p.F + f) =
                    static_cast<uint32_t>(cvt_e4m3x2(__fdiv_rn(h[0], s), __fdiv_rn(h[1], s))) |
                    (static_cast<uint32_t>(cvt_e4m3x2(__fdiv_rn(h[2], s), __fdiv_rn(h[3], s))) << 16);
            if (lane == 0)
                p.sh[row * p.fblocks + blockIdx.x] = s;
        }
    }
    if (splits > 1)
        cluster_sync_all();   // no CTA leaves while its partial may still be read
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// ------------------------------------------------------------------ down
template <int BN_, int STAGES_, int NBUF_> struct MoeDownCfg {
    static constexpr int BN = BN_;
    static constexpr int STAGES = STAGES_;
    static constexpr int NBUF = NBUF_;
    static constexpr int kThreads = 192;
    static constexpr int kTileA = 128 * 128;
    static constexpr int kStage = kTileA + BN * 128;
    static constexpr int kTmemCols = NBUF * BN < 32 ? 32 : NBUF * BN;
    static constexpr int kRingBytes = STAGES * kStage;
    static constexpr int kSumOffset = kRingBytes;        // [BN + 1][128] f32: the output tile, by token
    static constexpr int kScalePitch = BN + 4;
    static constexpr int kScaleOffset = kSumOffset + (BN + 1) * 512;
    static constexpr int kScaleBytes = 2 * kScaleChunk * kScalePitch * 4;
    static constexpr int kCtlOffset = kScaleOffset + kScaleBytes;
    static constexpr int kPlanOffset = kCtlOffset + 512; // experts (int4), tokens, weights: sized at launch
    static constexpr int kSmemBytes = kPlanOffset + 1024;
    static_assert(BN == 16 || BN == 32 || BN == 64, "token tile");
    static_assert(STAGES <= 8 && NBUF <= 8, "barriers");
    static_assert((kTmemCols & (kTmemCols - 1)) == 0 && kTmemCols <= 256, "tensor memory");
};

struct MoeDownParams {
    int T, H, fblocks;
    int max_active, pairs;   // sizes of the plan's lists
    const float *sh;         // [T k, fblocks]
    const float *s2;         // [E, ceil(H / 128), fblocks]
    void *y;                 // [T, H]
    int ydt;
    MoePlan plan;
};

// Grid (ceil(H / 128), 1, splits): a cluster of `splits` CTAs along z for 128
// output features; the (expert, k-block of F) units of all chosen experts, in
// that order, are dealt to its CTAs in equal contiguous ranges.
template <class C>
__global__ void __launch_bounds__(C::kThreads)
    moe_down_kernel(const __grid_constant__ CUtensorMap tmH, const __grid_constant__ CUtensorMap tmW,
                    const MoeDownParams p)
{
    constexpr int BN = C::BN, STAGES = C::STAGES, NBUF = C::NBUF;
    grid_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *sum = reinterpret_cast<float *>(smem + C::kSumOffset);
    float *sc = reinterpret_cast<float *>(smem + C::kScaleOffset);
    BlockCtl *ctl = reinterpret_cast<BlockCtl *>(smem + C::kCtlOffset);
    int4 *experts = reinterpret_cast<int4 *>(smem + C::kPlanOffset);
    int *tok = reinterpret_cast<int *>(experts + p.max_active);
    float *weight = reinterpret_cast<float *>(tok + p.pairs);
    volatile int *abort_flag = &ctl->abort;

    const int warp = warp_index();
    const int lane = threadIdx.x & 31;
    const int splits = static_cast<int>(gridDim.z);

    // The plan was complete before this grid could start (the gate+up kernel
    // lets it start only after its own wait for the plan).
    const int active = __ldcg(p.plan.active);
    for (int i = threadIdx.x; i < active; i += C::kThreads)
        experts[i] = __ldcg(p.plan.experts + i);
    for (int i = threadIdx.x; i < p.pairs; i += C::kThreads) {
        tok[i] = __ldcg(p.plan.tok + i);   // entries behind the last row are not used
        weight[i] = __ldcg(p.plan.weight + i);
    }
    const int units = active * p.fblocks;
    const int u0 = static_cast<int>(static_cast<int64_t>(units) * blockIdx.z / splits);
    const int u1 = static_cast<int>(static_cast<int64_t>(units) * (blockIdx.z + 1) / splits);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int b = 0; b < NBUF; ++b) {
            mbar_init(&ctl->acc_full[b], 1);
            mbar_init(&ctl->acc_empty[b], 4);
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&ctl->tmem_base, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    auto tokens16 = [](int rows) { return (rows + 15) & ~15; };   // the MMA's N

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            const uint64_t pol_w = policy_evict_first();
            const uint64_t pol_h = policy_evict_last();
            auto load_w = [&](int s, int a, int kb) {
                mbar_arrive_expect_tx(&ctl->full[s],
                                      static_cast<uint32_t>(C::kTileA + tokens16(experts[a].z) * 128));
                tma_load_2d_hint(smem + s * C::kStage, &tmW, &ctl->full[s], kb * 128,
                                 experts[a].x * p.H + static_cast<int>(blockIdx.x) * 128, pol_w);
            };
            auto load_h = [&](int s, int a, int kb) {
                for (int c = 0; c < experts[a].z; c += 16)
                    tma_load_2d_hint(smem + s * C::kStage + C::kTileA + c * 128, &tmH, &ctl->full[s], kb * 128,
                                     experts[a].y + c, pol_h);
            };
            // the first ring pass: weights at once, hidden codes when the gate+up kernel has finished
            const int first = u1 - u0 < STAGES ? u1 - u0 : STAGES;
            for (int i = 0; i < first; ++i)
                load_w(i, (u0 + i) / p.fblocks, (u0 + i) % p.fblocks);
            grid_dependency_wait();
            for (int i = 0; i < first; ++i)
                load_h(i, (u0 + i) / p.fblocks, (u0 + i) % p.fblocks);
            int s = 0, issued = first;
            uint32_t ph = 0;
            int a = (u0 + first) / p.fblocks, kb = (u0 + first) % p.fblocks;
            for (int u = u0 + first; u < u1; ++u) {
                if (!wait_step(&ctl->empty[s], ph, abort_flag))
                    break;
                load_w(s, a, kb);
                load_h(s, a, kb);
                ++issued;
                if (++kb == p.fblocks) {
                    kb = 0;
                    ++a;
                }
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (*abort_flag) {
                for (int j = 0; j < STAGES && j < issued; ++j)
                    wait_drain(&ctl->full[j], static_cast<uint32_t>((issued - 1 - j) / STAGES) & 1u);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        grid_dependency_wait();
        {
            int s = 0, b = 0;
            uint32_t ph = 0, bph = 1;
            bool ok = true;
            int a = u0 / p.fblocks, kb = u0 % p.fblocks;
            for (int u = u0; u < u1; ++u) {
                ok = wait_step(&ctl->acc_empty[b], bph, abort_flag) && wait_step(&ctl->full[s], ph, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t idesc = make_idesc(128, tokens16(experts[a].z), 0, 0);
                const uint32_t a_addr = smem_u32(smem + s * C::kStage);
                const uint32_t h_addr = a_addr + C::kTileA;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_f8f6f4(tmem + b * BN, sdesc_sw128(a_addr + k * 32), sdesc_sw128(h_addr + k * 32), idesc,
                                    k > 0 ? 1u : 0u);
                    umma_commit(&ctl->empty[s]);
                    umma_commit(&ctl->acc_full[b]);
                }
                __syncwarp();
                if (++kb == p.fblocks) {
                    kb = 0;
                    ++a;
                }
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
                if (++b == NBUF) {
                    b = 0;
                    bph ^= 1u;
                }
            }
            if (!ok && elect_one()) {
                umma_commit(&ctl->drain);
                wait_drain(&ctl->drain, 0);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ scales, accumulation, sum over experts
        const int qd = warp & 3;
        const int r = qd * 32 + lane;   // this thread alone touches column r of `sum`
        for (int c = 0; c < BN; ++c)
            sum[c * 128 + r] = 0.0f;
        float acc[BN];
#pragma unroll
        for (int j = 0; j < BN; ++j)
            acc[j] = 0.0f;
        grid_dependency_wait();         // the scales of the hidden codes
        const uint32_t t_row = tmem + (static_cast<uint32_t>(qd * 32) << 16);
        const int et = static_cast<int>(threadIdx.x) - 64;
        constexpr int PER = BN * kScaleChunk / 128;
        float pre[PER], wgt = 0.0f;
        int pre_row = 0, pre_rows = 0;
        // sh[row, kb], s2[e, feature block, kb] and the rows' weights of 8 units from u:
        // thread et's values are the expert's rows (et + 128 i) / 8 at unit u + et % 8
        auto fetch = [&](int u) {
            u += et & 7;
            const bool in = u < u1;
            const int a = in ? u / p.fblocks : 0;
            const int k = in ? u - a * p.fblocks : 0;
            const int4 ex = in ? experts[a] : make_int4(0, 0, 0, 0);
            wgt = in ? __ldg(p.s2 + (static_cast<int64_t>(ex.x) * gridDim.x + blockIdx.x) * p.fblocks + k) : 0.0f;
            pre_row = ex.y;
            pre_rows = ex.z;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int c = (et + 128 * i) >> 3;
                pre[i] = c < ex.z ? __ldcg(p.sh + (ex.y + c) * p.fblocks + k) : 0.0f;
            }
        };
        fetch(u0);
        int b = 0;
        uint32_t bph = 0;
        bool ok = true;
        int a = u0 / p.fblocks, kb = u0 % p.fblocks;
        for (int i = 0; i < u1 - u0; ++i) {
            float *buf = sc + ((i / kScaleChunk) & 1) * kScaleChunk * C::kScalePitch;
            if (i % kScaleChunk == 0) {
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const int c = (et + 128 * j) >> 3;
                    buf[(et & 7) * C::kScalePitch + c] = c < pre_rows ? pre[j] * wgt * weight[pre_row + c] : 0.0f;
                }
                if (i + kScaleChunk < u1 - u0)
                    fetch(u0 + i + kScaleChunk);
                bar_sync_epilogue<128>();
            }
            ok = ok && wait_step(&ctl->acc_full[b], bph, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            const int rows = experts[a].z;
            if (ok) {
                tc_fence_after();
                const float *s = buf + (i % kScaleChunk) * C::kScalePitch;
#pragma unroll
                for (int c0 = 0; c0 < BN; c0 += 16) {
                    if (c0 < rows) {
                        uint32_t v[16];
                        tmem_ld_32x32b_x16(t_row + b * BN + c0, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 t = *reinterpret_cast<const float4 *>(s + c0 + j);
                            acc[c0 + j] = fmaf(__uint_as_float(v[j]), t.x, acc[c0 + j]);
                            acc[c0 + j + 1] = fmaf(__uint_as_float(v[j + 1]), t.y, acc[c0 + j + 1]);
                            acc[c0 + j + 2] = fmaf(__uint_as_float(v[j + 2]), t.z, acc[c0 + j + 2]);
                            acc[c0 + j + 3] = fmaf(__uint_as_float(v[j + 3]), t.w, acc[c0 + j + 3]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&ctl->acc_empty[b]);
            }
            if (kb + 1 == p.fblocks || i + 1 == u1 - u0) {
                // the expert's (or the range's) last unit: to the output tile, by token.
                // Rows of one expert are different tokens, so 16 of them are read
                // together; columns behind the last row go to a spare row of the tile.
                const int row0 = experts[a].y;
#pragma unroll
                for (int c0 = 0; c0 < BN; c0 += 16) {
                    if (c0 < rows) {
                        const int mine = c0 + (lane & 15) < rows ? tok[row0 + c0 + (lane & 15)] : BN;
                        float *o[16];
                        float v[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            o[j] = sum + __shfl_sync(0xffffffffu, mine, j) * 128 + r;
                            v[j] = *o[j];
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            *o[j] = v[j] + acc[c0 + j];
                            acc[c0 + j] = 0.0f;
                        }
                    }
                }
            }
            if (++kb == p.fblocks) {
                kb = 0;
                ++a;
            }
            if (++b == NBUF) {
                b = 0;
                bph ^= 1u;
            }
        }
    }
    __syncwarp();

    // ---------------------------------------------------------------- output
    tc_fence_before();
    if (splits > 1)
        cluster_sync_all();
    else
        __syncthreads();
    if (warp >= 2) {
        const int n4 = static_cast<int>(blockIdx.x) * 128 + lane * 4;
        const uint32_t base = smem_u32(sum) + lane * 16;
        for (int t = static_cast<int>(blockIdx.z) + splits * (warp - 2); n4 < p.H && t < p.T; t += 4 * splits) {
            float4 q[8];
#pragma unroll
            for (int z = 0; z < 8; ++z)
                if (z < splits) {
                    const uint32_t off = base + t * 512;
                    q[z] = ld_shared_cluster_v4_relaxed(
                        splits > 1 ? map_shared_rank(off, static_cast<uint32_t>(z)) : off);
                }
            float4 v = q[0];
#pragma unroll
            for (int z = 1; z < 8; ++z)
                if (z < splits)
                    v = make_float4(v.x + q[z].x, v.y + q[z].y, v.z + q[z].z, v.w + q[z].w);
            store_out4(p.y, static_cast<int64_t>(t) * p.H + n4, v, p.ydt);
        }
    }
    if (splits > 1)
        cluster_sync_all();   // no CTA leaves while its sums may still be read
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

} // namespace pgf8
