#pragma once

namespace kvattn {
namespace {

// 2^x (ex2.approx.ftz: a few ulp, far below the rounding to bf16 or f16 that a weight
// goes through on the tensor cores); 2^-inf = 0.
__device__ __forceinline__ float fast_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace
}  // namespace kvattn
