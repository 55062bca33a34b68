// FP8 linear layer with block scales for many tokens: 256 x BN output tiles
// on SM pairs (tcgen05 cta_group::2), tokens as the MMA's rows.
//
// As in gemm_block.cuh, tensor memory holds one k-block of 128 at a time
// (two buffers of 256 columns, or four of 128) and the epilogue warps add it,
// times its scale, to the tile in their registers.  With the tokens as rows
// an accumulator lane is one token and 128 columns are one weight block, so a
// thread's scale is one number per k-block, sa[m, b] sw[n / 128, b].
//
// Sixteen warps share a CTA's 128 x BN slice (128 lanes x four column
// quarters), four to a scheduler.  What a k-block costs a warp beside its
// multiply-adds is latency - the barrier, the scale, tensor-memory loads that
// compete with the MMAs - and eight warps with twice the columns each were
// bound by it: about 1100 cycles a k-block against the MMA's 512.  Two more
// warps write the k-blocks' scales to a ring in shared memory: loaded by the
// epilogue warps themselves, a row stride apart for every lane, they took more
// of the load unit's time than the tile's multiply-adds took of theirs.  The
// additions are packed multiply-adds, two outputs to an instruction: with four
// warps to a scheduler its issue slots are the next limit (297 us against 277
// at 4096 x 8192 x 9472).
//
// Operand ring, barriers and their two-CTA signalling as in gemm_2sm.cuh: both
// CTAs' loads complete on the even CTA's full barrier, its one MMA thread
// drives both SMs and frees ring stages and publishes accumulators in both
// CTAs by multicast commits.  Waits are bounded; an epilogue warp that gave up
// leaves its loop (no barrier inside it).
#pragma once

#include "gemm_2sm.cuh"
#include "gemm_block.cuh"

namespace pgf8 {

template <int BN_, int STAGES_> struct BlockPairCfg {
    static constexpr int BN = BN_;
    static constexpr int STAGES = STAGES_;
    static constexpr int NBUF = 512 / BN;
    static constexpr int kThreads = 640;               // producer, MMA, two scale warps, 16 epilogue warps
    static constexpr int kTileA = 128 * 128;           // this CTA's 128 tokens
    static constexpr int kTileB = (BN / 2) * 128;      // this CTA's half of the weight rows
    static constexpr int kStage = kTileA + kTileB;
    static constexpr int kRowsX = 128;
    static constexpr int kRowsW = BN / 2;
    static constexpr int kBlocks = BN / 128;           // weight blocks across the tile
    static constexpr int kScaleSlots = 8;              // k-blocks of scales, [kBlocks][128] f32 each
    static constexpr int kOutOffset = STAGES * kStage; // 2 KB for each epilogue warp
    static constexpr int kScaleOffset = kOutOffset + 16 * 2048;
    static constexpr int kCtlOffset = kScaleOffset + kScaleSlots * kBlocks * 512;
    static constexpr int kSmemBytes = kCtlOffset + 512 + 1024;
    static_assert(BN == 128 || BN == 256, "tile width");
    static_assert(STAGES <= 8 && NBUF <= 4, "barriers");
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

// Arrive on the barrier at the same offset in CTA 0 of the cluster.  Scope and
// order are the defaults (release, CTA): what the arrival hands over is tensor
// memory whose loads have completed (tcgen05.wait::ld), no shared or global
// data.  With .release.cluster the odd CTA's eight arrivals per k-block each
// waited for a cluster-wide fence, 1.5 thousand cycles a k-block.
__device__ __forceinline__ void mbar_arrive_cta0(uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .b32 ra;\n\t"
        "mapa.shared::cluster.u32 ra, %0, 0;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [ra];\n\t}\n" ::"r"(bar)
        : "memory");
}

struct BlockPairCtl {
    uint64_t full[8];
    uint64_t empty[8];
    uint64_t acc_full[4];
    uint64_t acc_empty[4];
    uint64_t scale_full[8];
    uint64_t scale_empty[8];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
    gemm_block_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                           const BlockParams p)
{
    constexpr int BN = C::BN, STAGES = C::STAGES, NBUF = C::NBUF;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    BlockPairCtl *ctl = reinterpret_cast<BlockPairCtl *>(smem + C::kCtlOffset);
    volatile int *abort_flag = &ctl->abort;

    const int warp = warp_index();
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool lead = (rank == 0);
    const int pair = static_cast<int>(blockIdx.x >> 1);
    const int npairs = static_cast<int>(gridDim.x >> 1);
    const int m_tiles = (p.M + 255) / 256;
    const int total = m_tiles * ((p.N + BN - 1) / BN);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int b = 0; b < NBUF; ++b) {
            mbar_init(&ctl->acc_full[b], 1);
            mbar_init(&ctl->acc_empty[b], 32);   // 16 epilogue warps in each CTA
        }
        for (int s = 0; s < C::kScaleSlots; ++s) {
            mbar_init(&ctl->scale_full[s], 2);   // the scale warps
            mbar_init(&ctl->scale_empty[s], 16);
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
    }
    if (warp == 1) {
        tmem_alloc_pair(&ctl->tmem_base, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                 // both CTAs' barriers exist before any remote arrive
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    grid_dependency_wait();
    grid_launch_dependents();

    // Registers move from the first four warps to the sixteen that hold the
    // sums: 128 x 56 + 512 x 104 of the launch's 640 x 96.
    float *const scales = reinterpret_cast<float *>(smem + C::kScaleOffset);
    if (warp >= 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        // ------------------------------------------------------------ accumulation and output (both CTAs)
        constexpr int COLS = BN / 4;              // columns of this thread
        const int qd = warp & 3;
        const int quarter = (warp - 4) >> 2;
        const uint32_t t_row = tmem + (static_cast<uint32_t>(qd * 32) << 16) + static_cast<uint32_t>(quarter * COLS);
        const uint32_t my_scale = smem_u32(scales + (quarter * COLS / 128) * 128 + qd * 32 + lane);
        const uint32_t bars = smem_u32(ctl);
        uint32_t it = 0;                          // k-blocks so far: buffers, slots and phases follow from it
        bool ok = true;
        for (int t = pair; t < total; t += npairs) {
            float acc[COLS];
#pragma unroll
            for (int j = 0; j < COLS; ++j)
                acc[j] = 0.0f;
            for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
                const uint32_t b = it % C::NBUF, slot = it % C::kScaleSlots;
                ok = wait_step_at(bars + offsetof(BlockPairCtl, scale_full) + slot * 8, (it / C::kScaleSlots) & 1,
                                  abort_flag);
                const float f = ld_shared_f32(my_scale + slot * C::kBlocks * 512);
                ok = ok && wait_step_at(bars + offsetof(BlockPairCtl, acc_full) + b * 8, (it / C::NBUF) & 1,
                                        abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < COLS; c += 16) {
                    uint32_t v[16];
                    tmem_ld_32x32b_x16(t_row + b * BN + c, v);
                    tmem_ld_wait();
                    if (c + 16 == COLS) {
                        // everything is in registers: the buffer and the scale are free
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive_cta0(bars + offsetof(BlockPairCtl, acc_empty) + b * 8);
                            mbar_arrive_at(bars + offsetof(BlockPairCtl, scale_empty) + slot * 8);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 16; i += 2)
                        fma_pair(acc[c + i], acc[c + i + 1], v[i], v[i + 1], f, f);
                }
            }
            if (!ok)
                break;
            const int m_warp = (t % m_tiles) * 256 + static_cast<int>(rank) * 128 + qd * 32;
            const int n0 = (t / m_tiles) * BN + quarter * COLS;
            // Output through this warp's 2 KB of shared memory, so that a store
            // covers 64 contiguous bytes of a row: 32 rows x 64 bytes at a time,
            // 16-byte chunks swizzled by the row.
            uint4 *stage = reinterpret_cast<uint4 *>(smem + C::kOutOffset) + (warp - 4) * 128;
            const int eb = p.ydt == 0 ? 4 : 2;
            auto flush = [&](int n) {   // columns n .. n + 64 / eb - 1
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = i * 8 + (lane >> 2), ch = lane & 3;
                    const uint4 o = stage[row * 4 + (ch ^ ((row >> 1) & 3))];
                    if (m_warp + row < p.M && n + ch * (16 / eb) < p.N)   // N % 16 == 0
                        *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.y) +
                                                   (static_cast<int64_t>(m_warp + row) * p.N + n + ch * (16 / eb)) *
                                                       eb) = o;
                }
                __syncwarp();
            };
            if (p.ydt == 0) {
#pragma unroll
                for (int c = 0; c < COLS; c += 16) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float *o = acc + c + 4 * i;
                        stage[lane * 4 + (i ^ ((lane >> 1) & 3))] =
                            make_uint4(__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]),
                                       __float_as_uint(o[3]));
                    }
                    flush(n0 + c);
                }
            } else {
#pragma unroll
                for (int c = 0; c < COLS; c += 32) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t o[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            o[q] = pack_out2(make_float2(acc[c + 8 * i + 2 * q], acc[c + 8 * i + 2 * q + 1]), p.ydt);
                        stage[lane * 4 + (i ^ ((lane >> 1) & 3))] = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                    flush(n0 + c);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0) {
            // ------------------------------------------------------------ producers (both CTAs)
            if (lane == 0) {
                const uint64_t pol = policy_evict_last();
                int s = 0, issued = 0;
                uint32_t ph = 1;
                bool ok = true;
                for (int t = pair; ok && t < total; t += npairs) {
                    const int row_x = (t % m_tiles) * 256 + static_cast<int>(rank) * 128;
                    const int row_w = (t / m_tiles) * BN + static_cast<int>(rank) * (BN / 2);
                    for (int kb = 0; kb < p.kblocks; ++kb) {
                        if (!wait_step(&ctl->empty[s], ph, abort_flag)) {
                            ok = false;
                            break;
                        }
                        uint8_t *st = smem + s * C::kStage;
                        if (lead)
                            mbar_arrive_expect_tx(&ctl->full[s], 2 * C::kStage);
                        tma_load_2d_pair(st, &tmX, &ctl->full[s], kb * 128, row_x, pol);
                        tma_load_2d_pair(st + C::kTileA, &tmW, &ctl->full[s], kb * 128, row_w, pol);
                        issued = issued < STAGES ? issued + 1 : issued;
                        if (++s == STAGES) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                }
                if (*abort_flag && lead) {
                    // stage j was last loaded in the ring pass before this one, or in this one below s
                    for (int j = 0; j < issued; ++j)
                        wait_drain(&ctl->full[j], j < s ? ph ^ 1u : ph);
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer (even CTA)
            if (lead) {
                constexpr uint32_t idesc = make_idesc(256, BN, 0, 0);
                int s = 0, b = 0;
                uint32_t ph = 0, bph = 1;
                bool ok = true;
                for (int t = pair; ok && t < total; t += npairs) {
                    for (int kb = 0; kb < p.kblocks; ++kb) {
                        ok = wait_step(&ctl->acc_empty[b], bph, abort_flag) &&
                             wait_step(&ctl->full[s], ph, abort_flag);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok)
                            break;
                        tc_fence_after();
                        const uint32_t a_addr = smem_u32(smem + s * C::kStage);
                        const uint32_t b_addr = a_addr + C::kTileA;
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                umma_f8f6f4_pair(tmem + b * BN, sdesc_sw128(a_addr + k * 32),
                                                 sdesc_sw128(b_addr + k * 32), idesc, k > 0 ? 1u : 0u);
                            umma_commit_pair_both(&ctl->empty[s]);
                            umma_commit_pair_both(&ctl->acc_full[b]);
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
                }
                if (!ok && elect_one()) {
                    umma_commit_pair(&ctl->drain);
                    wait_drain(&ctl->drain, 0);
                }
            }
            __syncwarp();
        } else {
            // ------------------------------------------------------------ scales (both CTAs): two rows a thread
            const int row = (warp - 2) * 32 + lane;
            const bool vec = (p.kblocks & 3) == 0 && (reinterpret_cast<uintptr_t>(p.sa) & 15) == 0;
            int slot = 0;
            uint32_t sph = 1;
            bool ok = true;
            for (int t = pair; ok && t < total; t += npairs) {
                const int m = (t % m_tiles) * 256 + static_cast<int>(rank) * 128 + row;
                const int nb = (t / m_tiles) * C::kBlocks;
                const int nblocks = (p.N + 127) / 128;
                // rows behind the last token and blocks behind the last channel are read
                // from the first: their outputs are not written
                const float *sa0 = p.sa + static_cast<int64_t>(m < p.M ? m : 0) * p.kblocks;
                const float *sa1 = p.sa + static_cast<int64_t>(m + 64 < p.M ? m + 64 : 0) * p.kblocks;
                const float *sw0 = p.sw + static_cast<int64_t>(nb) * p.kblocks;
                const float *sw1 = p.sw + static_cast<int64_t>(nb + 1 < nblocks ? nb + 1 : 0) * p.kblocks;
                for (int kb0 = 0; ok && kb0 < p.kblocks; kb0 += 4) {
                    float a0[4], a1[4], w0[4], w1[4];
                    if (vec) {
                        const float4 x = __ldg(reinterpret_cast<const float4 *>(sa0 + kb0));
                        const float4 y = __ldg(reinterpret_cast<const float4 *>(sa1 + kb0));
                        a0[0] = x.x, a0[1] = x.y, a0[2] = x.z, a0[3] = x.w;
                        a1[0] = y.x, a1[1] = y.y, a1[2] = y.z, a1[3] = y.w;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int k = kb0 + j < p.kblocks ? kb0 + j : p.kblocks - 1;
                        if (!vec) {
                            a0[j] = __ldg(sa0 + k);
                            a1[j] = __ldg(sa1 + k);
                        }
                        w0[j] = __ldg(sw0 + k);
                        w1[j] = C::kBlocks > 1 ? __ldg(sw1 + k) : 0.0f;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (kb0 + j >= p.kblocks)
                            break;
                        ok = wait_step(&ctl->scale_empty[slot], sph, abort_flag);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok)
                            break;
                        float *s = scales + slot * C::kBlocks * 128 + row;
                        s[0] = a0[j] * w0[j];
                        s[64] = a1[j] * w0[j];
                        if (C::kBlocks > 1) {
                            s[128] = a0[j] * w1[j];
                            s[192] = a1[j] * w1[j];
                        }
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(&ctl->scale_full[slot]);
                        if (++slot == C::kScaleSlots) {
                            slot = 0;
                            sph ^= 1u;
                        }
                    }
                }
            }
        }
    }

    // ---------------------------------------------------------------- teardown
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                 // no CTA leaves while its partner may still signal it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

} // namespace pgf8
