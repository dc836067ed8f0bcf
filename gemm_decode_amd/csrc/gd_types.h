// gd_types.h -- the element types of the entry points that take a `dtype`:
// vector loads into f32 and stores rounded once (nearest even) from f32.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm_decode.h"

namespace gd {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

template <typename T>
struct Vec4;
template <>
struct Vec4<float> { typedef f32x4 type; };
template <>
struct Vec4<_Float16> { typedef f16x4 type; };
template <>
struct Vec4<__bf16> { typedef bf16x4 type; };

// Four consecutive elements (aligned to four elements) as f32.
template <typename T>
__device__ __forceinline__ f32x4 load4(const T *p) {
    return __builtin_convertvector(*reinterpret_cast<const typename Vec4<T>::type *>(p), f32x4);
}

// Four f32 values rounded to T.
template <typename T>
__device__ __forceinline__ void store4(T *p, f32x4 v) {
    *reinterpret_cast<typename Vec4<T>::type *>(p) = __builtin_convertvector(v, typename Vec4<T>::type);
}

inline bool dtype_ok(int32_t dtype) { return dtype == GD_F32 || dtype == GD_F16 || dtype == GD_BF16; }
inline int64_t dtype_size(int32_t dtype) { return dtype == GD_F32 ? 4 : 2; }

// Calls fn with a value of the dtype's element type.
template <typename F>
inline void dispatch_dtype(int32_t dtype, F fn) {
    if (dtype == GD_F32)
        fn(float{});
    else if (dtype == GD_F16)
        fn(_Float16{});
    else
        fn(__bf16{});
}

}  // namespace gd
