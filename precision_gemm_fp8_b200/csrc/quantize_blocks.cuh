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

#include <type_traits>

#include "packed_ptx.cuh"
#include "quantize.cuh"

namespace pgf8 {

// Scale of a block from its amax.
__device__ __forceinline__ float block_scale(float amax)
{
    const float s = __fdiv_rn(amax, 448.0f);
    return s == 0.0f ? 1.0f : s;
}

// Largest |v| of the 16 values, NaN if one of them is NaN (propagated, so that
// one comparison tells whether a whole block is finite).
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float amax16_nan(const float (&v)[16])
{
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        a = max_nan(a, fabsf(v[i]));
    return a;
}

// The same, NaN ignored.
__device__ __forceinline__ float amax16(const float (&v)[16])
{
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        a = fmaxf(a, fabsf(v[i]));
    return a;
}

// Over the 8 lanes of the aligned lane group that share one 1 x 128 group.
__device__ __forceinline__ float group_max8(float a)
{
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    return a;
}

__device__ __forceinline__ float group_max8_nan(float a)
{
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
        a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
    return a;
}

// 16 codes of finite values in a block of scale s, within the range that the
// division's steps need (RowDivisor: Markstein's sequence, the same steps here
// on two values at a time).  5 instructions a value where the checked form
// takes 11: with those the quantisation of 16-bit weights was bound by its
// arithmetic (with this and one reading of the values 91 us against 162 for 64 x
// 1408 x 2048 bf16, 5.9 TB/s).
__device__ __forceinline__ uint4 encode16_finite(const float (&v)[16], const RowDivisor &d)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t half[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float x0 = v[4 * i + 2 * h], x1 = v[4 * i + 2 * h + 1];
            float q0, q1;
            asm("{\n\t.reg .b64 a, y, n, q, r;\n\t"
                "mov.b64 a, {%2, %3};\n\t"
                "mov.b64 y, {%4, %4};\n\t"
                "mov.b64 n, {%5, %5};\n\t"
                "mul.rn.f32x2 q, a, y;\n\t"
                "fma.rn.f32x2 r, n, q, a;\n\t"
                "fma.rn.f32x2 q, r, y, q;\n\t"
                "fma.rn.f32x2 r, n, q, a;\n\t"
                "fma.rn.f32x2 q, r, y, q;\n\t"
                "mov.b64 {%0, %1}, q;\n\t}\n"
                : "=f"(q0), "=f"(q1)
                : "f"(fabsf(x0)), "f"(fabsf(x1)), "f"(d.y), "f"(-d.s));
            half[h] = cvt_e4m3x2(copysignf(q0, x0), copysignf(q1, x1));
        }
        w[i] = half[0] | (half[1] << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A block's scale and whether its values take the short conversion, from the
// NaN-propagating amax of the group; `again` gives the amax with NaN ignored
// (a warp-wide step: every lane of the warp calls this).
struct GroupScale {
    RowDivisor d;
    bool finite;
    __device__ __forceinline__ GroupScale(const float (&v)[16], bool live)
    {
        float a = group_max8_nan(live ? amax16_nan(v) : 0.0f);
        finite = a <= 3.402823466e38f;
        if (__any_sync(0xffffffffu, !finite)) {
            const float b = group_max8(live ? amax16(v) : 0.0f);
            a = finite ? a : b;
        }
        d = RowDivisor(block_scale(a));
    }
    __device__ __forceinline__ uint4 encode(const float (&v)[16]) const
    {
        return finite && d.fast ? encode16_finite(v, d) : encode16(v, d);
    }
};

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
    if (live)
        v.load(x + static_cast<int64_t>(row) * ldx + c);
    const GroupScale g8(v.v, live);   // every lane of the warp takes part
    if (!live)
        return;
    *reinterpret_cast<uint4 *>(q + static_cast<int64_t>(row) * cols + c) = g8.encode(v.v);
    if ((threadIdx.x & 7) == 0)
        scales[row * groups + grp] = g8.d.s;
}

// g / (1 + e^-g) * u: the quotient from the hardware reciprocal (within one
// unit in the last place) and one remainder step, which gives the correctly
// rounded quotient but for the rarest operands, for fewer instructions than
// the division.  Without the step one value in some thousands next to a border
// of E4M3 took the other code.  The remainder is taken as d q - g, which is +0
// where it vanishes, so that the step leaves the sign of a zero alone.  Where g
// or the denominator is infinite there is no remainder (NaN), and q is the
// quotient already: infinite for g = +inf, a zero with the sign of g below
// -88.7, NaN for g = -inf.
__device__ __forceinline__ float gate_mul(float g, float u)
{
    const float d = 1.0f + expf(-g);
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d));
    const float q = g * r;
    const float c = fmaf(-fmaf(d, q, -g), r, q);
    return (c == c ? c : q) * u;
}

// The same for h = silu(gate) * up of gu [rows, 2 inter] (gate = columns
// [0, inter), up = [inter, 2 inter)); h stays in registers, binary32.  Bound by
// the issue slots as much as by HBM, so the CTAs on an SM count: five with 48
// registers a thread for f32 (1021 x 11024: 19.0 us on the GPU, 20.0 with four),
// six with 40 for the 16-bit types (17.0 us, 17.4 with five).
template <typename T>
__global__ void __launch_bounds__(kQuantThreads, sizeof(T) == 4 ? 5 : 6)
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
    if (live) {
        Vec16<T> gate, up;
        const T *p = gu + static_cast<int64_t>(row) * ldg + c;
        gate.load(p);
        up.load(p + inter);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            h[i] = gate_mul(gate.v[i], up.v[i]);
    }
    const GroupScale g8(h, live);
    if (!live)
        return;
    *reinterpret_cast<uint4 *>(q + static_cast<int64_t>(row) * inter + c) = g8.encode(h);
    if ((threadIdx.x & 7) == 0)
        scales[row * groups + grp] = g8.d.s;
}

// 16 values as they stand in memory: half the registers of their binary32
// form for the 16-bit types.
template <typename T> struct Raw16 {
    static constexpr int W = sizeof(T);   // 16-byte words
    uint4 w[W];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < W; ++i)
            w[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    }
    // The same words, but not known to the compiler to be.
    __device__ __forceinline__ void opaque()
    {
#pragma unroll
        for (int i = 0; i < W; ++i)
            asm volatile("" : "+r"(w[i].x), "+r"(w[i].y), "+r"(w[i].z), "+r"(w[i].w));
    }
    __device__ __forceinline__ void to_float(float (&v)[16]) const
    {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const uint32_t t[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 4) {
                    v[4 * i + j] = __uint_as_float(t[j]);
                } else if constexpr (std::is_same_v<T, __half>) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&t[j]));   // exact
                    v[8 * i + 2 * j] = f.x;
                    v[8 * i + 2 * j + 1] = f.y;
                } else {
                    v[8 * i + 2 * j] = __uint_as_float(t[j] << 16);
                    v[8 * i + 2 * j + 1] = __uint_as_float(t[j] & 0xFFFF0000u);
                }
            }
        }
    }
};

// One CTA per 128 x 128 block of a batch of matrices [rows, cols] (row
// stride ldx, matrix stride ldb): 256 threads hold 4 x 16 values each, 8
// threads to a row, between the amax and the conversion.  A CTA loads, then
// computes, then stores, so what fills the memory system is the number of CTAs
// on an SM: the values wait in their own type, which leaves room for four
// CTAs (16-bit) or two, and blocks that need the checked conversion (NaN,
// infinities, scales at the ends of the range) read their values again.
template <typename T>
__global__ void __launch_bounds__(kQuantThreads, sizeof(T) == 2 ? 4 : 2)
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
    // rows of this thread inside the matrix: r0, r0 + 32, ... (none behind the last column)
    const int mine = c < cols && r0 < rows ? static_cast<int>((rows - 1 - r0) / 32 < 3 ? (rows - 1 - r0) / 32 + 1 : 4) : 0;
    const T *xb = x + static_cast<int64_t>(b) * ldb + r0 * ldx + c;
    uint8_t *qb = q + (static_cast<int64_t>(b) * rows + r0) * cols + c;
    Raw16<T> v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        if (u < mine)
            v[u].load(xb + 32 * u * ldx);
        else
            v[u] = Raw16<T>{};
    }
    float a = 0.0f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        float f[16];
        v[u].to_float(f);
        a = max_nan(a, amax16_nan(f));
    }
    const bool finite = !__syncthreads_or(!(a <= 3.402823466e38f));
    // the widened values are made again for the conversion: kept across the
    // reduction they would take twice the registers and be spilled
#pragma unroll
    for (int u = 0; u < 4; ++u)
        v[u].opaque();
    if (!finite) {
        a = 0.0f;   // NaN ignored
#pragma unroll 1
        for (int u = 0; u < mine; ++u) {
            Vec16<T> w;
            w.load(xb + 32 * u * ldx);
            a = fmaxf(a, amax16(w.v));
        }
    }
    const RowDivisor d(block_scale(block_max(a, red)));
    if (finite && d.fast) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (u < mine) {
                float f[16];
                v[u].to_float(f);
                *reinterpret_cast<uint4 *>(qb + 32 * u * cols) = encode16_finite(f, d);
            }
        }
    } else {
#pragma unroll 1
        for (int u = 0; u < mine; ++u) {
            Vec16<T> w;
            w.load(xb + 32 * u * ldx);
            *reinterpret_cast<uint4 *>(qb + 32 * u * cols) = encode16(w.v, d);
        }
    }
    if (threadIdx.x == 0)
        scales[blockIdx.x] = d.s;
}

} // namespace pgf8
