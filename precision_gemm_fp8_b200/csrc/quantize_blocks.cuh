// E4M3 quantisation with block scales: one scale per 1 x 128 group of a row
// (activations) or per 128 x 128 block (weights), and the SiLU gate fused
// with the former.  Per block: amax = max |x|, s = fl32(amax / 448) (1 when
// that is 0), code = E4M3(fl32(x / s)), nearest-even, saturating - the rule
// of the per-row quantisation ("7B on an RTX 4060 with FP8" §2.2, §6.1) on
// smaller blocks, so that one outlier costs resolution in its own block only.
// Codes and scales are bit-exact with respect to that definition.
//
// All three are one pass over memory: n values of size b move n (b + 1)
// bytes (the gate: n (2 b + 1)) plus 4 bytes a block, a handful of
// operations a value: bound by HBM, or by the launch for a few rows.
#pragma once

#include "quantize.cuh"

namespace pgf8 {

// Scale of a block from its amax.
__device__ __forceinline__ float block_scale(float amax)
{
    const float s = __fdiv_rn(amax, 448.0f);
    return s == 0.0f ? 1.0f : s;
}

// Largest |v| of the 16 values (NaN ignored), then over the 8 lanes of the
// aligned lane group that share one 1 x 128 group.
__device__ __forceinline__ float amax16(const float (&v)[16])
{
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        a = fmaxf(a, fabsf(v[i]));
    return a;
}

__device__ __forceinline__ float group_max8(float a)
{
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    return a;
}

// Row and group index of 1 x 128 group `g` in rows of `groups` groups.
__device__ __forceinline__ void split_group(uint64_t g, uint32_t groups, uint64_t total, uint64_t &row, uint32_t &grp)
{
    if (total <= 0xFFFFFFFFull) {   // uniform over the grid: the 32-bit division is several times cheaper
        const uint32_t g32 = static_cast<uint32_t>(g);
        row = g32 / groups;
        grp = g32 - static_cast<uint32_t>(row) * groups;
    } else {
        row = g / groups;
        grp = static_cast<uint32_t>(g - row * groups);
    }
}

// 8 threads per 1 x 128 group, 16 values each (64 or 32 contiguous bytes a
// thread): the group's amax takes three shuffles and no barrier, and a
// ragged last group simply leaves lanes idle (cols % 16 == 0).
template <typename T>
__global__ void __launch_bounds__(kQuantThreads)
    quantize_row_blocks_kernel(const T *__restrict__ x, uint64_t total, uint32_t groups, int64_t cols, int64_t ldx,
                               uint8_t *__restrict__ q, float *__restrict__ scales)
{
    grid_launch_dependents();
    grid_dependency_wait();
    const uint64_t g = static_cast<uint64_t>(blockIdx.x) * (kQuantThreads / 8) + (threadIdx.x >> 3);
    uint64_t row = 0;
    uint32_t grp = 0;
    split_group(g < total ? g : 0, groups, total, row, grp);
    const int64_t c = static_cast<int64_t>(grp) * 128 + (threadIdx.x & 7) * 16;
    const bool live = g < total && c < cols;
    Vec16<T> v;
    float a = 0.0f;
    if (live) {
        v.load(x + static_cast<int64_t>(row) * ldx + c);
        a = amax16(v.v);
    }
    a = group_max8(a);   // every lane of the warp takes part
    if (!live)
        return;
    const float s = block_scale(a);
    *reinterpret_cast<uint4 *>(q + static_cast<int64_t>(row) * cols + c) = encode16(v.v, RowDivisor(s));
    if ((threadIdx.x & 7) == 0)
        scales[row * groups + grp] = s;
}

// The same for h = silu(gate) * up of gu [rows, 2 inter] (gate = columns
// [0, inter), up = [inter, 2 inter)); h stays in registers, binary32.
template <typename T>
__global__ void __launch_bounds__(kQuantThreads)
    silu_mul_row_blocks_kernel(const T *__restrict__ gu, uint64_t total, uint32_t groups, int64_t inter, int64_t ldg,
                               uint8_t *__restrict__ q, float *__restrict__ scales)
{
    grid_launch_dependents();
    grid_dependency_wait();
    const uint64_t g = static_cast<uint64_t>(blockIdx.x) * (kQuantThreads / 8) + (threadIdx.x >> 3);
    uint64_t row = 0;
    uint32_t grp = 0;
    split_group(g < total ? g : 0, groups, total, row, grp);
    const int64_t c = static_cast<int64_t>(grp) * 128 + (threadIdx.x & 7) * 16;
    const bool live = g < total && c < inter;
    float h[16];
    float a = 0.0f;
    if (live) {
        Vec16<T> gate, up;
        const T *p = gu + static_cast<int64_t>(row) * ldg + c;
        gate.load(p);
        up.load(p + inter);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            h[i] = silu_mul(gate.v[i], up.v[i]);
        a = amax16(h);
    }
    a = group_max8(a);
    if (!live)
        return;
    const float s = block_scale(a);
    *reinterpret_cast<uint4 *>(q + static_cast<int64_t>(row) * inter + c) = encode16(h, RowDivisor(s));
    if ((threadIdx.x & 7) == 0)
        scales[row * groups + grp] = s;
}

// One CTA per 128 x 128 block of a batch of matrices [rows, cols] (row
// stride ldx, matrix stride ldb): 256 threads hold 4 x 16 values each, 8
// threads to a row, between the amax and the conversion.
template <typename T>
__global__ void __launch_bounds__(kQuantThreads)
    quantize_tiles_kernel(const T *__restrict__ x, int64_t rows, int64_t cols, int64_t ldx, int64_t ldb,
                          uint32_t row_blocks, uint32_t col_blocks, uint8_t *__restrict__ q,
                          float *__restrict__ scales)
{
    __shared__ float red[kQuantThreads / 32];
    grid_launch_dependents();
    grid_dependency_wait();
    const uint32_t cb = blockIdx.x % col_blocks;
    const uint32_t rest = blockIdx.x / col_blocks;
    const uint32_t rb = rest % row_blocks;
    const uint32_t b = rest / row_blocks;
    const int64_t c = static_cast<int64_t>(cb) * 128 + (threadIdx.x & 7) * 16;
    const int64_t r0 = static_cast<int64_t>(rb) * 128 + (threadIdx.x >> 3);
    const T *xb = x + static_cast<int64_t>(b) * ldb + c;
    Vec16<T> v[4];
    float a = 0.0f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t r = r0 + 32 * u;
        if (r < rows && c < cols) {
            v[u].load(xb + r * ldx);
            a = fmaxf(a, amax16(v[u].v));
        }
    }
    a = block_max(a, red);
    const float s = block_scale(a);
    const RowDivisor d(s);
    uint8_t *qb = q + (static_cast<int64_t>(b) * rows) * cols + c;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t r = r0 + 32 * u;
        if (r < rows && c < cols)
            *reinterpret_cast<uint4 *>(qb + r * cols) = encode16(v[u].v, d);
    }
    if (threadIdx.x == 0)
        scales[blockIdx.x] = s;
}

} // namespace pgf8
