// extern "C" entry points of the mixture-of-experts operators: argument
// checks, then the launch.  None of them allocates or synchronises.
#include "moe.h"
#include "spmm_csr_spmv.h"

namespace {

constexpr int64_t kI32Max = 2147483647;
constexpr int64_t kI64Max = 9223372036854775807LL;

bool bad_dtype(int32_t t) { return t != SP_F32 && t != SP_BF16 && t != SP_F16; }
size_t elem(int32_t t) { return t == SP_F32 ? 4 : 2; }
bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// rows rows ld apart: the last element's byte offset must fit 63 bits
bool too_far(int64_t rows, int64_t ld) { return rows > 0 && ld > (kI64Max >> 4) / rows; }

// whether [a, a + an) and [b, b + bn) share a byte
bool share(const void* a, size_t an, const void* b, size_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return an > 0 && bn > 0 && (x <= y ? y - x < an : x - y < bn);
}

int rows_args(int64_t T, int32_t slots, int64_t H, int64_t S, int32_t dtype) {
    if (T < 0 || T > kI32Max || slots < 1 || H < 0 || H > kI32Max || S < 0 || S > kI32Max) return SP_ERR_SIZE;
    if (T * slots > kI32Max) return SP_ERR_SIZE;
    if (bad_dtype(dtype)) return SP_ERR_UNSUPPORTED;
    return SP_OK;
}

}  // namespace

extern "C" {

int moe_sort_bufsize(int64_t n, int32_t num_experts, size_t* bytes) {
    if (!bytes) return SP_ERR_NULL;
    if (n < 0 || n > kI32Max) return SP_ERR_SIZE;
    if (num_experts < 1 || num_experts > SP_MOE_MAX_EXPERTS) return SP_ERR_UNSUPPORTED;
    *bytes = spx::moe_sort_work_bytes(n, num_experts);
    return SP_OK;
}

int moe_sort(int64_t n, int32_t num_experts, const int32_t* ids, int32_t* offsets, int32_t* src, int32_t* pos,
             void* work, size_t work_bytes, void* stream) {
    size_t need = 0;
    const int rc = moe_sort_bufsize(n, num_experts, &need);
    if (rc) return rc;
    if (!offsets || (n > 0 && (!ids || !src || !pos))) return SP_ERR_NULL;
    if (misaligned(ids, 4) || misaligned(offsets, 4) || misaligned(src, 4) || misaligned(pos, 4))
        return SP_ERR_UNSUPPORTED;
    if (need > 0 && (!work || work_bytes < need || misaligned(work, 4))) return SP_ERR_WORKSPACE;
    // Counts written over the ids would make the second kernel place slots that the first did not count.
    const size_t ids_bytes = (size_t)n * sizeof(int32_t);
    if (share(work, need, ids, ids_bytes) || share(work, need, src, ids_bytes) || share(work, need, pos, ids_bytes) ||
        share(work, need, offsets, ((size_t)num_experts + 1) * sizeof(int32_t)))
        return SP_ERR_WORKSPACE;
    return spx::moe_sort_device(n, num_experts, ids, offsets, src, pos, work, (hipStream_t)stream);
}

int moe_dispatch(int64_t T, int32_t slots, int64_t H, int64_t S, int32_t dtype, const void* X, int64_t ldx,
                 const int32_t* pos, void* Xs, int64_t lds, void* stream) {
    const int rc = rows_args(T, slots, H, S, dtype);
    if (rc) return rc;
    if (ldx < H || lds < H || too_far(T, ldx) || too_far(S, lds)) return SP_ERR_SIZE;
    if (T == 0 || H == 0 || S == 0) return SP_OK;
    if (!X || !pos || !Xs) return SP_ERR_NULL;
    if (misaligned(X, elem(dtype)) || misaligned(Xs, elem(dtype)) || misaligned(pos, 4)) return SP_ERR_UNSUPPORTED;
    return spx::moe_dispatch_device(T, slots, H, S, dtype, X, ldx, pos, Xs, lds, (hipStream_t)stream);
}

int moe_combine(int64_t T, int32_t slots, int64_t H, int64_t S, int32_t dtype, const void* Ys, int64_t lds,
                const int32_t* pos, const float* weights, void* Y, int64_t ldy, void* stream) {
    const int rc = rows_args(T, slots, H, S, dtype);
    if (rc) return rc;
    if (ldy < H || lds < H || too_far(T, ldy) || too_far(S, lds)) return SP_ERR_SIZE;
    if (T == 0 || H == 0) return SP_OK;
    if ((S > 0 && !Ys) || !pos || !Y) return SP_ERR_NULL;  // weights may be NULL: all ones
    if (misaligned(Ys, elem(dtype)) || misaligned(Y, elem(dtype)) || misaligned(pos, 4) || misaligned(weights, 4))
        return SP_ERR_UNSUPPORTED;
    return spx::moe_combine_device(T, slots, H, S, dtype, Ys, lds, pos, weights, Y, ldy, (hipStream_t)stream);
}

int moe_combine_backward(int64_t T, int32_t slots, int64_t H, int64_t S, int32_t dtype, const void* dY, int64_t ldy,
                         const void* Ys, int64_t lds, const int32_t* pos, const float* weights, void* dYs,
                         int64_t ldd, float* dweights, void* stream) {
    const int rc = rows_args(T, slots, H, S, dtype);
    if (rc) return rc;
    if (ldy < H || lds < H || ldd < H || too_far(T, ldy) || too_far(S, lds) || too_far(S, ldd)) return SP_ERR_SIZE;
    if (T == 0) return SP_OK;
    if ((H > 0 && !dY) || (S > 0 && H > 0 && (!Ys || !dYs)) || !pos || !weights || !dweights) return SP_ERR_NULL;
    if (misaligned(dY, elem(dtype)) || misaligned(Ys, elem(dtype)) || misaligned(dYs, elem(dtype)) ||
        misaligned(pos, 4) || misaligned(weights, 4) || misaligned(dweights, 4))
        return SP_ERR_UNSUPPORTED;
    return spx::moe_combine_backward_device(T, slots, H, S, dtype, dY, ldy, Ys, lds, pos, weights, dYs, ldd, dweights,
                                            (hipStream_t)stream);
}

int quantize_rows_i8(int64_t rows, int64_t K, int32_t dtype, const void* X, int64_t ldx, int8_t* q, int64_t ldq,
                     float* scale, void* stream) {
    if (rows < 0 || rows > kI32Max || K < 0 || K > kI32Max) return SP_ERR_SIZE;
    if (bad_dtype(dtype)) return SP_ERR_UNSUPPORTED;
    if (ldx < K || ldq < K || too_far(rows, ldx) || too_far(rows, ldq)) return SP_ERR_SIZE;
    if (rows == 0) return SP_OK;
    if (!scale || (K > 0 && (!X || !q))) return SP_ERR_NULL;
    if (misaligned(X, elem(dtype)) || misaligned(scale, 4)) return SP_ERR_UNSUPPORTED;
    return spx::quantize_rows_i8_device(rows, K, dtype, X, ldx, q, ldq, scale, (hipStream_t)stream);
}

int moe_gemm_i8(int64_t S, int32_t num_experts, int64_t N, int64_t K, const int8_t* A, int64_t a_rows, int64_t lda,
                const float* a_scale, const int32_t* src, int32_t slots, const int8_t* B, int64_t ldb,
                int64_t strideb, const float* b_scale, const int32_t* offsets, int32_t c_type, void* C, int64_t ldc,
                void* stream) {
    if (S < 0 || S > kI32Max || a_rows < 0 || a_rows > kI32Max || N < 0 || N > kI32Max || K < 0 || slots < 1)
        return SP_ERR_SIZE;
    if (K > SP_I8_MAX_K || num_experts < 1 || num_experts > SP_MOE_MAX_EXPERTS || bad_dtype(c_type))
        return SP_ERR_UNSUPPORTED;
    if (lda < K || ldb < K || ldc < N || too_far(a_rows, lda) || too_far(N, ldb) || too_far(S, ldc)) return SP_ERR_SIZE;
    if (num_experts > 1 && N > 0 && (strideb < 0 || strideb < (N - 1) * ldb + K || too_far(num_experts, strideb)))
        return SP_ERR_SIZE;
    if (S == 0 || N == 0) return SP_OK;
    if (!offsets || !C || !b_scale || (a_rows > 0 && !a_scale) || (K > 0 && (!B || (a_rows > 0 && !A))))
        return SP_ERR_NULL;
    if (misaligned(C, elem(c_type)) || misaligned(a_scale, 4) || misaligned(b_scale, 4) || misaligned(offsets, 4) ||
        misaligned(src, 4))
        return SP_ERR_UNSUPPORTED;
    return spx::gemm_i8_device(S, num_experts, N, K, A, a_rows, lda, a_scale, src, slots, B, ldb, strideb, b_scale,
                               offsets, c_type, C, ldc, (hipStream_t)stream);
}

int gemm_i8(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const float* a_scale, const int8_t* B,
            int64_t ldb, const float* b_scale, int32_t c_type, void* C, int64_t ldc, void* stream) {
    if (M < 0 || M > kI32Max || N < 0 || N > kI32Max || K < 0) return SP_ERR_SIZE;
    if (K > SP_I8_MAX_K || bad_dtype(c_type)) return SP_ERR_UNSUPPORTED;
    if (lda < K || ldb < K || ldc < N || too_far(M, lda) || too_far(N, ldb) || too_far(M, ldc)) return SP_ERR_SIZE;
    if (M == 0 || N == 0) return SP_OK;
    if (!C || !a_scale || !b_scale || (K > 0 && (!A || !B))) return SP_ERR_NULL;
    if (misaligned(C, elem(c_type)) || misaligned(a_scale, 4) || misaligned(b_scale, 4)) return SP_ERR_UNSUPPORTED;
    return spx::gemm_i8_device(M, 1, N, K, A, M, lda, a_scale, nullptr, 1, B, ldb, 0, b_scale, nullptr, c_type, C, ldc,
                               (hipStream_t)stream);
}

}  // extern "C"
