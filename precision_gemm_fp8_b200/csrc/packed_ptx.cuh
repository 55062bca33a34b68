// Inline-PTX wrappers of the block-scaled kernels beside those of
// sm100_ptx.cuh; each is one PTX instruction (or a fixed short sequence) as
// documented in the PTX ISA for sm_100a.
#pragma once

#include "sm100_ptx.cuh"

namespace pgf8 {

// a = x s + a and b = y t + b in one instruction, each rounded once (x, y: the
// bits of binary32 values).  The pairs are bound inside the statement, so that
// the compiler keeps plain registers around it.
__device__ __forceinline__ void fma_pair(float &a, float &b, uint32_t x, uint32_t y, float s, float t)
{
    asm("{\n\t.reg .b64 v, f, d;\n\t"
        "mov.b64 v, {%2, %3};\n\t"
        "mov.b64 f, {%4, %5};\n\t"
        "mov.b64 d, {%0, %1};\n\t"
        "fma.rn.f32x2 d, v, f, d;\n\t"
        "mov.b64 {%0, %1}, d;\n\t}\n"
        : "+f"(a), "+f"(b)
        : "r"(x), "r"(y), "f"(s), "f"(t));
}

// The warp's index in its CTA, the same in every lane for the compiler too: the
// branches of the warp roles are then uniform.
__device__ __forceinline__ int warp_index()
{
    return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
}

// True in one lane of the (converged) warp.  The whole warp runs an MMA
// issuer's loop and this picks the lane that issues: with the loop inside a
// one-lane branch instead, the compiler cannot keep descriptors and barrier
// addresses in uniform registers, and a k-block's four MMAs and two commits
// took about 380 cycles to issue.
__device__ __forceinline__ bool elect_one()
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok));
    return ok != 0;
}

} // namespace pgf8
