// Elementary functions of the block's kernels (internal).
#pragma once

#include <hip/hip_runtime.h>

namespace blr {

// exp(v) to about 1e-7, and zero below -87.4, where it would be subnormal: the
// product with log2(e) is kept to twice its length, whose tail enters as 1 +
// tail ln 2.
__device__ __forceinline__ float exp_of(float v) {
    const float L = 1.44269504088896340736f;
    const float t = v * L, tail = fmaf(v, L, -t) + v * 1.92596299112661746887e-8f;
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, tail * 0.69314718055994530942f, e);
}
// 1 / v, v >= 1, with one Newton step.
__device__ __forceinline__ float inverse(float v) {
    const float r = __builtin_amdgcn_rcpf(v);
    return fmaf(fmaf(-v, r, 1.0f), r, r);
}
}  // namespace blr
