// Checks of arguments that the entry points share.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "spmm_csr_spmv.h"

namespace spx {

constexpr int64_t kI32Max = 2147483647;
constexpr int64_t kI64Max = 9223372036854775807LL;

inline bool bad_dtype(int32_t t) { return t != SP_F32 && t != SP_BF16 && t != SP_F16; }
inline size_t elem(int32_t t) { return t == SP_F32 ? 4 : 2; }
inline bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// rows rows ld apart: the last element's byte offset must fit 63 bits
inline bool too_far(int64_t rows, int64_t ld) { return rows > 0 && ld > (kI64Max >> 4) / rows; }

// whether [a, a + an) and [b, b + bn) share a byte
inline bool share(const void* a, size_t an, const void* b, size_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return an > 0 && bn > 0 && (x <= y ? y - x < an : x - y < bn);
}

inline bool bad_act(int32_t a) { return a != SP_ACT_SILU && a != SP_ACT_GELU_TANH; }

}  // namespace spx
