// vs_types.h -- element types and short vectors of the table operators
// (group.hip, rows.hip, q4.hip).
//
// Arithmetic is fp32 throughout: values are widened on load (exactly) and
// rounded once, to nearest even, when they are stored.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace vs {

enum DType : int { kF32 = 0, kF16 = 1, kBF16 = 2 };

inline int dtype_bytes(int t) { return t == kF32 ? 4 : 2; }

template <typename T>
__device__ __forceinline__ float widen(T x) { return (float)x; }
template <typename T>
__device__ __forceinline__ T narrow(float x) { return (T)x; }

// N elements, accessed 16 bytes at a time at most: longer ones (the scales of
// a block, a row of fp32 partial sums) claim no more alignment than that, which
// is what callers' arrays are asked for.
template <typename T, int N>
struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Vec {
    T v[N];
};

// Accesses that pass the caches by (each value is used once): what they move
// would push out what others still need.
template <int BYTES>
struct RawBits;
template <>
struct RawBits<2> { typedef uint16_t type; };
template <>
struct RawBits<4> { typedef uint32_t type; };
template <>
struct RawBits<8> { typedef __attribute__((ext_vector_type(2))) uint32_t type; };
template <>
struct RawBits<16> { typedef __attribute__((ext_vector_type(4))) uint32_t type; };

template <typename V>
__device__ __forceinline__ V load_once(const V *p) {
    using R = typename RawBits<sizeof(V)>::type;
    const R r = __builtin_nontemporal_load(reinterpret_cast<const R *>(p));
    V v;
    __builtin_memcpy(&v, &r, sizeof(V));
    return v;
}
template <typename V>
__device__ __forceinline__ void store_once(V *p, const V &v) {
    using R = typename RawBits<sizeof(V)>::type;
    R r;
    __builtin_memcpy(&r, &v, sizeof(V));
    __builtin_nontemporal_store(r, reinterpret_cast<R *>(p));
}

// Elements per vector access: 16 bytes where every row starts on a 16-byte
// boundary (the row size and the matrices' addresses allow it), else the
// largest power of two that does.  `addr` is the or of the addresses.
inline int vec_elems(int64_t d, int esize, uintptr_t addr) {
    const uint64_t bits = (uint64_t)d * (uint64_t)esize | (uint64_t)addr | 16u;
    const int bytes = (int)(bits & (~bits + 1));
    return bytes / esize;
}

}  // namespace vs
