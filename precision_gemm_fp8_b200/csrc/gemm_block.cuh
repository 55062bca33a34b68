// FP8 linear layer with block scales, weights as the 128-row MMA operand:
//   y[m, n] = sum_b sa[m, b] sw[n / 128, b] sum_{k in block b} a[m, k] w[n, k]
// with blocks of 128 along K (E4M3 codes, scales f32).
//
// The scales vary along K, so the tensor core cannot add the blocks up
// itself: tcgen05 accumulates one k-block (4 MMAs of 32 bytes of K) in tensor
// memory in binary32, and the epilogue warps add it, times its scale, to the
// output tile that they hold in registers, while the MMAs of the next
// k-blocks fill the other accumulator buffers.  Per k-block and tile that is
// one multiply-add an output; each is rounded once to binary32 (sums stay
// in binary32 until the final rounding to the output type).
//
// For few tokens the layer is bound by the weight stream (N K bytes at HBM
// speed), so the K range of a weight tile is split over a thread-block
// cluster until the grid fills the GPU; the CTAs' partial tiles are added in
// rank order through distributed shared memory (no workspace, the same
// result in every run).
//
//   warp 0      TMA producer: STAGES-deep ring of (weight tile, token tile)
//   warp 1      tensor-memory allocation, MMA issue (one thread)
//   warps 2...  scales, accumulation over k-blocks, output: four warps for
//               every 32 tokens, a thread holding one weight row's sums for
//               them (16 at BN = 16).  With one warp a lane quadrant for 128
//               tokens a k-block took about 1000 cycles of one warp's time
//               against the MMA's 256, and the layer was bound by it.
// Waits are bounded as in gemm.cuh; after a wait that gave up the epilogue
// warps keep walking their loop without touching tensor memory, so that
// their barriers stay matched.
#pragma once

#include "gemm.cuh"
#include "packed_ptx.cuh"
#include "quantize_blocks.cuh"

#include <cstddef>

namespace pgf8 {

constexpr int kScaleChunk = 8;   // k-blocks of token scales staged in shared memory at a time

// XQ: 0, the activations arrive as codes; 1 / 2 / 3, f32 / f16 / bf16 activations
// that each CTA quantises itself for its range of K, into shared memory, while
// its first weight tiles are in flight.  For the few tokens for which that is
// less work than another launch.
template <int BN_, int STAGES_, int NBUF_, int XQ_ = 0> struct BlockCfg {
    static constexpr int BN = BN_;
    static constexpr int STAGES = STAGES_;
    static constexpr int NBUF = NBUF_;   // accumulator buffers of BN columns
    static constexpr int CTAS = BN == 128 ? 1 : 2;   // to an SM
    static constexpr int KIND = kE4M3;
    static constexpr int XQ = XQ_;
    static constexpr int kSlots = 20;    // XQ: most k-blocks of a CTA
    static constexpr int COLS = BN < 32 ? BN : 32;       // tokens of an epilogue thread
    static constexpr int kEpi = 128 * (BN / COLS);       // epilogue threads
    static constexpr int kThreads = 64 + kEpi;
    static constexpr int kTileA = 128 * 128;
    static constexpr int kStage = kTileA + (XQ ? 0 : BN * 128);
    static constexpr int kRowsW = 128;
    static constexpr int kRowsX = BN;
    static constexpr int kTmemCols = NBUF * BN < 32 ? 32 : NBUF * BN;
    static constexpr int kRingBytes = STAGES * kStage;   // reused for the partial tile [BN][128] f32
    static constexpr int kCodesOffset = kRingBytes;      // XQ: [kSlots][BN][128] codes
    static constexpr int kScalePitch = BN + 4;           // floats; the 8 k-blocks' writes then hit distinct banks
    static constexpr int kScaleOffset = kCodesOffset + (XQ ? kSlots * BN * 128 : 0);
    static constexpr int kScaleBytes = (XQ ? kSlots : 2 * kScaleChunk) * kScalePitch * 4;
    static constexpr int kCtlOffset = kScaleOffset + kScaleBytes;
    static constexpr int kSmemBytes = kCtlOffset + 512 + 1024;
    static_assert(BN == 16 || BN == 32 || BN == 64 || BN == 128, "token tile");
    static_assert(STAGES <= 8 && NBUF <= 8, "barriers");
    static_assert((kTmemCols & (kTmemCols - 1)) == 0 && kTmemCols <= 512, "tensor memory");
    static_assert(kRingBytes >= BN * 128 * 4, "partial tile");
    static_assert(kSmemBytes <= 227 * 1024 && CTAS * (kSmemBytes + 1024) <= 228 * 1024, "shared memory");
    static_assert(CTAS * kTmemCols <= 512, "tensor memory of an SM");
    static_assert(XQ == 0 || BN == 16, "in-kernel quantisation: the narrowest token tile");
};

// Bounded wait for a barrier that another role of the kernel completes within
// a k-block's time, on every k-block.  The first polls read no clock: the
// timer takes longer to read than such a wait lasts, and the read would sit
// between two roles that hand a buffer to one another.  Then as wait_bounded.
__device__ __forceinline__ bool wait_step(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity))
            return true;
    return wait_bounded(bar, parity, abort);
}

// The same by 32-bit shared-memory addresses, for loops short of registers.
__device__ __forceinline__ bool mbar_try_wait_at(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool wait_step_at(uint32_t bar, uint32_t parity, volatile int *abort)
{
    if (mbar_try_wait_at(bar, parity))
        return true;
    return wait_step(static_cast<uint64_t *>(__cvta_shared_to_generic(bar)), parity, abort);
}

__device__ __forceinline__ void mbar_arrive_at(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

struct BlockCtl {
    uint64_t full[8];
    uint64_t empty[8];
    uint64_t acc_full[8];
    uint64_t acc_empty[8];
    uint64_t drain;
    uint64_t codes;          // XQ: this CTA's activation codes are in shared memory
    uint32_t tmem_base;
    int abort;
};

struct BlockParams {
    int M, N, K, kblocks;
    int prefetch_w;      // 1: weight tiles may be loaded before the grid dependency resolves
    const float *sa;     // [M, kblocks]
    const float *sw;     // [ceil(N / 128), kblocks]
    void *y;             // [M, N]
    int ydt;             // pgf8_dtype
    const void *x;       // XQ: [M, K], row stride ldx elements
    int64_t ldx;
};

// v rounded once to the output type.
__device__ __forceinline__ void store_out(void *y, int64_t i, float v, int dt)
{
    if (dt == 2)
        static_cast<__nv_bfloat16 *>(y)[i] = __float2bfloat16_rn(v);
    else if (dt == 1)
        static_cast<__half *>(y)[i] = __float2half_rn(v);
    else
        static_cast<float *>(y)[i] = v;
}

// Four consecutive outputs (the address is a multiple of four elements).
__device__ __forceinline__ void store_out4(void *y, int64_t i, float4 v, int dt)
{
    if (dt == 2) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(y) + i) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else if (dt == 1) {
        const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
        *reinterpret_cast<uint2 *>(static_cast<__half *>(y) + i) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(y) + i) = v;
    }
}

// Two outputs of a 16-bit type in one word.
__device__ __forceinline__ uint32_t pack_out2(float2 v, int dt)
{
    if (dt == 2) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y);
        return *reinterpret_cast<const uint32_t *>(&a);
    }
    const __half2 a = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&a);
}

// Adds COLS accumulator columns of this thread's row (tensor memory at taddr)
// times their scales (shared memory, 16-byte aligned) to acc.
template <int COLS>
__device__ __forceinline__ void add_scaled(uint32_t taddr, const float *sc, float (&acc)[COLS])
{
#pragma unroll
    for (int c0 = 0; c0 < COLS; c0 += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(taddr + c0, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const float4 t = *reinterpret_cast<const float4 *>(sc + c0 + j);
            fma_pair(acc[c0 + j], acc[c0 + j + 1], v[j], v[j + 1], t.x, t.y);
            fma_pair(acc[c0 + j + 2], acc[c0 + j + 3], v[j + 2], v[j + 3], t.z, t.w);
        }
    }
}

// Named barrier 1 over the N epilogue threads.
template <int N> __device__ __forceinline__ void bar_sync_epilogue()
{
    asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}

template <class C>
__global__ void __launch_bounds__(C::kThreads)
    gemm_block_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                      const BlockParams p)
{
    constexpr int BN = C::BN, STAGES = C::STAGES, NBUF = C::NBUF;
    grid_launch_dependents();

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *sc = reinterpret_cast<float *>(smem + C::kScaleOffset);
    BlockCtl *ctl = reinterpret_cast<BlockCtl *>(smem + C::kCtlOffset);
    volatile int *abort_flag = &ctl->abort;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int n0 = static_cast<int>(blockIdx.x) * 128;
    const int m0 = static_cast<int>(blockIdx.y) * BN;
    const int splits = static_cast<int>(gridDim.z);   // the cluster along z
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.kblocks) * blockIdx.z / splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.kblocks) * (blockIdx.z + 1) / splits);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int b = 0; b < NBUF; ++b) {
            mbar_init(&ctl->acc_full[b], 1);
            mbar_init(&ctl->acc_empty[b], C::kEpi / 32);
        }
        mbar_init(&ctl->drain, 1);
        mbar_init(&ctl->codes, C::kEpi / 32);
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

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            const uint64_t pol_w = policy_evict_first();
            const uint64_t pol_x = policy_evict_last();
            if (!p.prefetch_w)
                grid_dependency_wait();
            // the first ring pass: weights at once, token tiles after the dependency
            const int first = kb1 - kb0 < STAGES ? kb1 - kb0 : STAGES;
            for (int i = 0; i < first; ++i) {
                mbar_arrive_expect_tx(&ctl->full[i], C::kStage);
                tma_load_2d_hint(smem + i * C::kStage, &tmW, &ctl->full[i], (kb0 + i) * 128, n0, pol_w);
            }
            if (p.prefetch_w)
                grid_dependency_wait();
            if constexpr (C::XQ == 0)
                for (int i = 0; i < first; ++i)
                    tma_load_2d_hint(smem + i * C::kStage + C::kTileA, &tmX, &ctl->full[i], (kb0 + i) * 128, m0,
                                     pol_x);
            int s = 0;
            uint32_t ph = 0;
            int issued = first;
            for (int kb = kb0 + first; kb < kb1; ++kb) {
                if (!wait_step(&ctl->empty[s], ph, abort_flag))
                    break;
                uint8_t *st = smem + s * C::kStage;
                mbar_arrive_expect_tx(&ctl->full[s], C::kStage);
                tma_load_2d_hint(st, &tmW, &ctl->full[s], kb * 128, n0, pol_w);
                if constexpr (C::XQ == 0)
                    tma_load_2d_hint(st + C::kTileA, &tmX, &ctl->full[s], kb * 128, m0, pol_x);
                ++issued;
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (*abort_flag) {
                // the last load into each used stage lands (bounded) before the CTA may exit
                for (int j = 0; j < STAGES && j < issued; ++j)
                    wait_drain(&ctl->full[j], static_cast<uint32_t>((issued - 1 - j) / STAGES) & 1u);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        grid_dependency_wait();
        {
            constexpr uint32_t idesc = make_idesc(128, BN, 0, 0);
            int s = 0, b = 0;
            uint32_t ph = 0, bph = 1;
            bool ok = true;
            if constexpr (C::XQ != 0)
                ok = __all_sync(0xffffffffu, wait_step(&ctl->codes, 0, abort_flag));
            for (int kb = kb0; ok && kb < kb1; ++kb) {
                ok = wait_step(&ctl->acc_empty[b], bph, abort_flag) && wait_step(&ctl->full[s], ph, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t a_addr = smem_u32(smem + s * C::kStage);
                const uint32_t b_addr =
                    C::XQ ? smem_u32(smem + C::kCodesOffset) + (kb - kb0) * (BN * 128) : a_addr + C::kTileA;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_f8f6f4(tmem + b * BN, sdesc_sw128(a_addr + k * 32), sdesc_sw128(b_addr + k * 32), idesc,
                                    k > 0 ? 1u : 0u);
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
    float acc[COLS];
    const int qd = warp & 3;
    const int r = qd * 32 + lane;
    const int col0 = ((warp - 2) >> 2) * COLS;   // this warp's tokens of the tile
    if (warp >= 2) {
        // ------------------------------------------------------------ scales and accumulation
        grid_dependency_wait();   // the token scales come from the kernel before
#pragma unroll
        for (int j = 0; j < COLS; ++j)
            acc[j] = 0.0f;
        const uint32_t t_row = tmem + (static_cast<uint32_t>(qd * 32) << 16) + static_cast<uint32_t>(col0);
        const int et = static_cast<int>(threadIdx.x) - 64;
        // sa[m, kb] and sw[n0 / 128, kb] of 8 k-blocks from kb: thread et's values are
        // tokens (et + EPI i) / 8 at k-block kb + et % 8 (32 contiguous bytes a token),
        // loaded a chunk ahead and multiplied when they are stored: a product taken
        // where they are loaded would wait for the loads
        constexpr int PER = BN * kScaleChunk / EPI;
        float pre[PER], wgt = 0.0f;
        const float *swr = p.sw + static_cast<int64_t>(blockIdx.x) * p.kblocks;
        auto fetch = [&](int kb) {
            const int k = kb + (et & 7);
            wgt = k < kb1 ? __ldg(swr + k) : 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int m = m0 + ((et + EPI * i) >> 3);
                pre[i] = (k < kb1 && m < p.M) ? p.sa[static_cast<int64_t>(m) * p.kblocks + k] : 0.0f;
            }
        };
        if constexpr (C::XQ != 0) {
            // codes and scales of this CTA's k-blocks: 8 threads a group as in the
            // quantisation kernel, rows of 128 codes in the MMA's swizzled layout
            // (rows behind the last token hold anything: their columns are not
            // written out)
            using T = std::conditional_t<C::XQ == 1, float, std::conditional_t<C::XQ == 2, __half, __nv_bfloat16>>;
            const int total = (kb1 - kb0) * p.M * 8;
            for (int base = 0; base < total; base += EPI) {
                const int i = base + et;
                const int chunk = i & 7, g = i >> 3;
                const int kb = g / p.M, m = g - kb * p.M;
                const int k = (kb0 + kb) * 128 + chunk * 16;
                const bool live = i < total && k < p.K;
                Vec16<T> v;
                if (live)
                    v.load(static_cast<const T *>(p.x) + static_cast<int64_t>(m) * p.ldx + k);
                const GroupScale g8(v.v, live);
                if (i < total) {
                    *reinterpret_cast<uint4 *>(smem + C::kCodesOffset + kb * (BN * 128) + m * 128 +
                                               ((chunk ^ (m & 7)) << 4)) =
                        live ? g8.encode(v.v) : make_uint4(0u, 0u, 0u, 0u);
                    if (chunk == 0)
                        sc[kb * C::kScalePitch + m] = g8.d.s * __ldg(swr + kb0 + kb);
                }
            }
            fence_proxy_async_smem();   // each writer, before the MMA (async proxy) reads
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&ctl->codes);
            bar_sync_epilogue<EPI>();   // the scales
        } else {
            fetch(kb0);
        }
        int b = 0;
        uint32_t bph = 0;
        bool ok = true;
        for (int i = 0; i < kb1 - kb0; ++i) {
            float *buf = sc + ((i / kScaleChunk) & 1) * kScaleChunk * C::kScalePitch;
            if (C::XQ == 0 && i % kScaleChunk == 0) {
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    buf[(et & 7) * C::kScalePitch + ((et + EPI * j) >> 3)] = pre[j] * wgt;
                if (i + kScaleChunk < kb1 - kb0)
                    fetch(kb0 + i + kScaleChunk);
                bar_sync_epilogue<EPI>();
            }
            ok = ok && wait_step(&ctl->acc_full[b], bph, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
                tc_fence_after();
                add_scaled<COLS>(t_row + b * BN,
                                 (C::XQ ? sc + i * C::kScalePitch : buf + (i % kScaleChunk) * C::kScalePitch) + col0,
                                 acc);
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

    // ---------------------------------------------------------------- output
    const int n = n0 + r;
    if (splits == 1) {
        if (warp >= 2 && n < p.N) {
#pragma unroll
            for (int c = 0; c < COLS; ++c) {
                const int m = m0 + col0 + c;
                if (m < p.M)
                    store_out(p.y, static_cast<int64_t>(m) * p.N + n, acc[c], p.ydt);
            }
        }
        tc_fence_before();
        __syncthreads();
    } else {
        // partial tile [BN][128] over the idle ring; CTA z of the cluster finishes
        // tokens z, z + splits, ... : the partials in rank order
        float *part = reinterpret_cast<float *>(smem);
        const int cols = p.M - m0 < BN ? p.M - m0 : BN;
        tc_fence_before();
        __syncthreads();
        if (warp >= 2) {
#pragma unroll
            for (int c = 0; c < COLS; ++c)
                part[(col0 + c) * 128 + r] = acc[c];
        }
        cluster_sync_all();
        if (warp >= 2) {
            // four weight rows a thread, so that a column's partials are in
            // flight together and go out as one store
            const int n4 = n0 + lane * 4;
            const uint32_t base = smem_u32(part) + lane * 16;
            for (int c = static_cast<int>(blockIdx.z) + splits * (warp - 2); n4 < p.N && c < cols;
                 c += EPI / 32 * splits) {
                float4 t[8];
#pragma unroll
                for (int z = 0; z < 8; ++z)
                    if (z < splits)
                        t[z] = ld_shared_cluster_v4_relaxed(map_shared_rank(base + c * 512, static_cast<uint32_t>(z)));
                float4 v = t[0];
#pragma unroll
                for (int z = 1; z < 8; ++z)
                    if (z < splits)
                        v = make_float4(v.x + t[z].x, v.y + t[z].y, v.z + t[z].z, v.w + t[z].w);
                store_out4(p.y, static_cast<int64_t>(m0 + c) * p.N + n4, v, p.ydt);
            }
        }
        cluster_sync_all();   // no CTA leaves while its partial may still be read
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

} // namespace pgf8
