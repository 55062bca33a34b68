// Inline-PTX wrappers of the block-scaled kernels beside those of
// sm100_ptx.cuh; each is one PTX instruction (or a fixed short sequence) as
// documented in the PTX ISA for sm_100a.
#pragma once

#include "sm100_ptx.cuh"

namespace pgf8 {

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
