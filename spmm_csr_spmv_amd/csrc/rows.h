// Element types (fp32, bf16, fp16) and 16-byte row accesses of the kernels
// that move or quantise whole rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace spx {

// A row is cut into 16-byte chunks.  Rows need not be 16-byte aligned: the
// accesses carry the element's alignment only (the hardware takes them at any
// address).  Where a whole last chunk does not fit, the row kernels take one that
// ends with the row, and rows or tiles' edges shorter than a chunk go element by element.
struct F32 {
    typedef float T;
    static __device__ __forceinline__ float up(float v) { return v; }
    static __device__ __forceinline__ float down(float v) { return v; }
};
struct Bf16 {
    typedef uint16_t T;
    static __device__ __forceinline__ float up(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ uint16_t down(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
};
struct F16 {
    typedef _Float16 T;
    static __device__ __forceinline__ float up(_Float16 v) { return (float)v; }
    static __device__ __forceinline__ _Float16 down(float v) { return (_Float16)v; }
};

// v rounded to D's type after it was an fp32 number: left to itself the compiler fuses a product and its rounding to fp16
// in some places and not in others, even where contraction is off, and the last bit of a value then depends on where in a
// result it stands.
template <class D>
__device__ __forceinline__ typename D::T round_alone(float v) {
    asm("" : "+v"(v));
    return D::down(v);
}

template <class T>
struct Chunk {
    static constexpr int N = 16 / (int)sizeof(T);
    typedef T V __attribute__((ext_vector_type(N)));
    typedef T U __attribute__((ext_vector_type(N), aligned(sizeof(T))));
};

// A whole chunk; the data is used once (non-temporal).
template <class T>
__device__ __forceinline__ typename Chunk<T>::V chunk_stream(const T* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const typename Chunk<T>::U*>(p));
}
template <class T>
__device__ __forceinline__ void chunk_stream(T* p, typename Chunk<T>::V v) {
    __builtin_nontemporal_store(v, reinterpret_cast<typename Chunk<T>::U*>(p));
}

// The first `len` elements of a chunk, the rest zero.
template <class T>
__device__ __forceinline__ typename Chunk<T>::V chunk_load(const T* p, int64_t len) {
    typename Chunk<T>::V v;
    if (len >= Chunk<T>::N) {
        v = *reinterpret_cast<const typename Chunk<T>::U*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < Chunk<T>::N; ++i) v[i] = i < len ? p[i] : (T)0;
    }
    return v;
}
template <class T>
__device__ __forceinline__ void chunk_store(T* p, int64_t len, typename Chunk<T>::V v) {
    if (len >= Chunk<T>::N) {
        *reinterpret_cast<typename Chunk<T>::U*>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < Chunk<T>::N - 1; ++i)
            if (i < len) p[i] = v[i];
    }
}

}  // namespace spx
