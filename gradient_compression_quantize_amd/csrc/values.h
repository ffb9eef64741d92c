// values.h -- element types of the training operators (gc_dtype): loads to
// and stores from fp32, one value or a 16-byte vector at a time.
#pragma once

#include "gcq_internal.h"

namespace gcq {
namespace {

using bf16_t = __bf16;
using f16_t = _Float16;

// Values in 16 bytes.
template <typename T>
constexpr int kVec = 16 / int(sizeof(T));

template <typename T, int N>
using vec_of = T __attribute__((ext_vector_type(N)));

// fp32 values of one 16-byte vector.
template <typename T>
using vec_f32 = vec_of<float, kVec<T>>;

template <typename T>
__device__ __forceinline__ vec_f32<T> load_vec(const T* p)
{
    return __builtin_convertvector(*reinterpret_cast<const vec_of<T, kVec<T>>*>(p), vec_f32<T>);
}

// Each value rounds once, to nearest even.
template <typename T>
__device__ __forceinline__ void store_vec(T* p, vec_f32<T> v)
{
    *reinterpret_cast<vec_of<T, kVec<T>>*>(p) = __builtin_convertvector(v, vec_of<T, kVec<T>>);
}

// Bytes of one value, 0 for an unknown type.
inline size_t dtype_bytes(int dtype)
{
    return dtype == GC_F32 ? 4 : dtype == GC_BF16 || dtype == GC_F16 ? 2 : 0;
}

inline bool aligned_to(const void* p, size_t bytes)
{
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// Calls f with a value of the element type as its argument.
template <typename F>
inline int with_dtype(int dtype, F f)
{
    switch (dtype) {
    case GC_F32:
        return f(float());
    case GC_BF16:
        return f(bf16_t());
    default:
        return f(f16_t());
    }
}

}  // namespace
}  // namespace gcq
