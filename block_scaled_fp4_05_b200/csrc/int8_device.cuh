// Device arithmetic shared by the INT8 products: the scaled result of an
// integer sum and its rounding to 16 bits.  One definition, so that every
// kernel gives the same bits.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace fp4 {
namespace i8 {

// The token's scale first, so that the sum leaves the integer range before the
// channel's scale and bias are applied.
__device__ __forceinline__ float scaled(int sum, float sa, float sb, float bias)
{
    return __fmaf_rn(__fmul_rn(__int2float_rn(sum), sa), sb, bias);
}

// Two results as FP16 (HALF) or BF16, round to nearest even, lo in the low half.
template <bool HALF>
__device__ __forceinline__ uint32_t pack16(float lo, float hi)
{
    uint32_t r;
    if constexpr (HALF)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace i8
}  // namespace fp4
