// Rows kept in 8 bits (internal): 32 consecutive values share the step
// 2^(b - 133), b a byte, and are held as whole numbers of steps, |q| <= 127.
// b is the least for which the largest of them rounds to 127 or less; b = 255
// says that one of them was not finite, and all 32 stand for NaN. A step is a
// power of two, so that q 2^(b - 133) is exact in f32 and bf16 (8 significant
// bits suffice) and no order of operations changes it.
#pragma once

#include "blr_vec.h"

namespace blr {

// Eight elements of a row as they lie in memory.
template <typename T>
struct Raw8 {
    typename Vec<T>::v v[8 / Vec<T>::n];
};
template <typename T>
__device__ __forceinline__ Raw8<T> raw8(const T *p) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < 8 / Vec<T>::n; ++i) r.v[i] = reinterpret_cast<const typename Vec<T>::v *>(p)[i];
    return r;
}
template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T> &r, float *o) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (float)r.v[i / Vec<T>::n][i % Vec<T>::n];
}
// One rounding to nearest even.
template <typename T>
__device__ __forceinline__ Raw8<T> narrow8(const float *v) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i / Vec<T>::n][i % Vec<T>::n] = (T)v[i];
    return r;
}
template <typename T>
__device__ __forceinline__ void put8(T *p, const Raw8<T> &r) {
#pragma unroll
    for (int i = 0; i < 8 / Vec<T>::n; ++i) reinterpret_cast<typename Vec<T>::v *>(p)[i] = r.v[i];
}

// The widest step a type's values get: f16's largest would otherwise round up
// to 65536, which f16 does not hold, and f32's have no wider one. The values
// above 127 steps are cut off there.
template <typename T>
inline constexpr int KEEP_MAX = 254;
template <>
inline constexpr int KEEP_MAX<_Float16> = 142;

// Largest |v| as bits (so that a NaN is the largest of all) of the 8 values.
__device__ __forceinline__ uint32_t top8(const float *v) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu);
    return m;
}
// Its maximum over four neighbouring lanes.
__device__ __forceinline__ uint32_t top_of_quad(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xf, 0xf, true));  // lane ^ 1
    return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xf, 0xf, true));  // lane ^ 2
}
// The block's exponent byte.
__device__ __forceinline__ int keep_exponent(uint32_t top, int most) {
    if (top >= 0x7f800000u) return 255;
    const int b = (int)(top >> 23);
    return b < most && rintf(ldexpf(__builtin_bit_cast(float, top), 133 - b)) > 127.0f ? b + 1 : b;
}
// Eight whole numbers of steps as bytes. Adding 3 * 2^22 rounds to a whole
// number (to nearest even) and leaves it, in two's complement, in the low bits.
__device__ __forceinline__ uint2 keep8(const float *v, int b) {
    uint32_t k[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float s = b == 255 ? 0.0f : ldexpf(v[i], 133 - b);
        k[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_fmed3f(s, -127.0f, 127.0f) + 12582912.0f);
    }
    auto four = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
        return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0c0c0400u), __builtin_amdgcn_perm(b, a, 0x0c0c0400u),
                                     0x05040100u);
    };
    return make_uint2(four(k[0], k[1], k[2], k[3]), four(k[4], k[5], k[6], k[7]));
}
// The values of eight of them: the step itself is a float (a subnormal one for
// b < 7), and its products are exact.
__device__ __forceinline__ void kept8(uint2 q, int b, float *o) {
    const float step = b == 255 ? __builtin_nanf("") : ldexpf(1.0f, b - 133);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (float)(int8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3))) * step;
}

}  // namespace blr
