// Rows of f32, f16 or bf16 as 16-byte vectors of f32 values (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace blr {

typedef float vf4 __attribute__((ext_vector_type(4)));
typedef _Float16 vh4 __attribute__((ext_vector_type(4)));
typedef _Float16 vh8 __attribute__((ext_vector_type(8)));
typedef __bf16 vb4 __attribute__((ext_vector_type(4)));
typedef __bf16 vb8 __attribute__((ext_vector_type(8)));

template <typename T>
struct Vec;  // n elements in 16 bytes (v) and four elements (v4)
template <>
struct Vec<float> {
    static constexpr int n = 4;
    typedef vf4 v;
    typedef vf4 v4;
};
template <>
struct Vec<_Float16> {
    static constexpr int n = 8;
    typedef vh8 v;
    typedef vh4 v4;
};
template <>
struct Vec<__bf16> {
    static constexpr int n = 8;
    typedef vb8 v;
    typedef vb4 v4;
};

// Four consecutive elements as f32, and back (one rounding to nearest even).
template <typename T>
__device__ __forceinline__ vf4 load4(const T *p) {
    return __builtin_convertvector(*reinterpret_cast<const typename Vec<T>::v4 *>(p), vf4);
}
template <typename T>
__device__ __forceinline__ void store4(T *p, vf4 v) {
    *reinterpret_cast<typename Vec<T>::v4 *>(p) = __builtin_convertvector(v, typename Vec<T>::v4);
}

}  // namespace blr
