// extern "C" entry points of the norm and of the 16-bit products of experts:
// argument checks, then the launches.  None of them allocates or synchronises.
#include <math.h>

#include "checks.h"
#include "moe.h"
#include "spmm_csr_spmv.h"

using namespace spx;

namespace {

// Steps of 64 rows or of 64 elements are counted in 32 bits, a few behind the last among them.
constexpr int64_t kMostRows = kI32Max - 1023, kMostWidth = (int64_t)1 << 29;

int norm_args(const NormRows& n) {
    if (n.rows < 0 || n.rows > kI32Max || n.H < 0 || n.H > kI32Max) return SP_ERR_SIZE;
    if (bad_dtype(n.dtype) || (n.w_type != n.dtype && n.w_type != SP_F32)) return SP_ERR_UNSUPPORTED;
    if (!(n.eps >= 0.0f) || isinf(n.eps)) return SP_ERR_UNSUPPORTED;
    if (n.ldx < n.H || too_far(n.rows, n.ldx) || (n.R && (n.ldr < n.H || too_far(n.rows, n.ldr)))) return SP_ERR_SIZE;
    if (misaligned(n.X, elem(n.dtype)) || misaligned(n.R, elem(n.dtype)) || misaligned(n.weight, elem(n.w_type)))
        return SP_ERR_UNSUPPORTED;
    return SP_OK;
}

int norm(const NormRows& n, void* sum, int64_t lds, void* Y, int64_t ldy, float* scale, bool codes, hipStream_t s) {
    const int rc = norm_args(n);
    if (rc) return rc;
    if (ldy < n.H || too_far(n.rows, ldy) || (sum && (lds < n.H || too_far(n.rows, lds)))) return SP_ERR_SIZE;
    if (n.rows == 0 || (n.H == 0 && !codes)) return SP_OK;
    if ((codes && !scale) || (n.H > 0 && (!n.X || !Y || (n.R && !sum)))) return SP_ERR_NULL;
    if (misaligned(sum, elem(n.dtype)) || (codes ? misaligned(scale, 4) : misaligned(Y, elem(n.dtype))))
        return SP_ERR_UNSUPPORTED;
    return rms_norm_device(n, sum, lds, Y, ldy, scale, s);
}

// The operands of a product and its gradient.  b_rows: rows of a matrix; a, b: whether A, B are read.
int product_args(const Products& p, int64_t b_rows, bool a, bool b) {
    if (p.S < 0 || p.S > kMostRows || p.a_rows < 0 || p.a_rows > kI32Max || p.N < 0 || p.K < 0 || p.slots < 1)
        return SP_ERR_SIZE;
    if (p.N > kMostWidth || p.K > kMostWidth || p.E < 1 || p.E > SP_MOE_MAX_EXPERTS || (!p.offsets && p.E != 1))
        return SP_ERR_UNSUPPORTED;
    if (p.dtype != SP_BF16 && p.dtype != SP_F16) return SP_ERR_UNSUPPORTED;
    if (a && (p.lda < p.K || too_far(p.a_rows, p.lda))) return SP_ERR_SIZE;
    if (b) {
        if (p.ldb < p.K || too_far(b_rows, p.ldb)) return SP_ERR_SIZE;
        if (p.E > 1 && b_rows > 0 && (p.strideb < (b_rows - 1) * p.ldb + p.K || too_far(p.E, p.strideb)))
            return SP_ERR_SIZE;
    }
    if ((a && misaligned(p.A, 2)) || (b && misaligned(p.B, 2)) || misaligned(p.offsets, 4) || misaligned(p.src, 4))
        return SP_ERR_UNSUPPORTED;
    return SP_OK;
}

int product(const Products& p, int32_t gate, void* pre, int64_t ldp, void* C, int64_t ldc, hipStream_t s) {
    const int rc = product_args(p, gate < 0 ? p.N : 2 * p.N, true, true);
    if (rc) return rc;
    if (ldc < p.N || too_far(p.S, ldc) || (pre && (ldp < 2 * p.N || too_far(p.S, ldp)))) return SP_ERR_SIZE;
    if (p.S == 0 || p.N == 0) return SP_OK;
    if (!C || (p.K > 0 && (!p.B || (p.a_rows > 0 && !p.A)))) return SP_ERR_NULL;
    if (misaligned(C, 2) || misaligned(pre, 2)) return SP_ERR_UNSUPPORTED;
    return moe_gemm_device(p, gate, pre, ldp, C, ldc, s);
}

// Of the gradients' outputs.
int gradient_args(const Products& p, int64_t b_rows, const void* dA, int64_t ldda, const void* dB, int64_t lddb,
                  int64_t stridedb) {
    const int rc = product_args(p, b_rows, dB != nullptr, dA != nullptr);
    if (rc) return rc;
    if (dA && (ldda < p.K || too_far(p.S, ldda))) return SP_ERR_SIZE;
    if (dB) {
        if (lddb < p.K || too_far(b_rows, lddb)) return SP_ERR_SIZE;
        if (p.E > 1 && b_rows > 0 && (stridedb < (b_rows - 1) * lddb + p.K || too_far(p.E, stridedb))) return SP_ERR_SIZE;
    }
    if (misaligned(dA, 2) || misaligned(dB, 2)) return SP_ERR_UNSUPPORTED;
    if (p.S > 0 && p.K > 0 && b_rows > 0 && ((dA && !p.B) || (dB && p.a_rows > 0 && !p.A))) return SP_ERR_NULL;
    return SP_OK;
}

int sizes(int64_t S, int32_t num_experts, int64_t N, int64_t K, int32_t dtype) {
    if (S < 0 || S > kMostRows || N < 0 || K < 0) return SP_ERR_SIZE;
    if (N > kMostWidth || K > kMostWidth || num_experts < 1 || num_experts > SP_MOE_MAX_EXPERTS ||
        (dtype != SP_BF16 && dtype != SP_F16))
        return SP_ERR_UNSUPPORTED;
    return SP_OK;
}

int workspace(const void* work, size_t work_bytes, size_t need) {
    return need > 0 && (!work || work_bytes < need || misaligned(work, 16)) ? SP_ERR_WORKSPACE : SP_OK;
}

}  // namespace

extern "C" {

int rms_norm(int64_t rows, int64_t H, int32_t dtype, const void* X, int64_t ldx, const void* residual, int64_t ldr,
             const void* weight, int32_t w_type, float eps, void* sum, int64_t lds, void* Y, int64_t ldy, void* stream) {
    return norm(NormRows{rows, H, dtype, w_type, X, ldx, residual, ldr, weight, eps}, sum, lds, Y, ldy, nullptr, false,
                (hipStream_t)stream);
}

int rms_norm_i8(int64_t rows, int64_t H, int32_t dtype, const void* X, int64_t ldx, const void* residual, int64_t ldr,
                const void* weight, int32_t w_type, float eps, void* sum, int64_t lds, int8_t* q, int64_t ldq,
                float* scale, void* stream) {
    return norm(NormRows{rows, H, dtype, w_type, X, ldx, residual, ldr, weight, eps}, sum, lds, q, ldq, scale, true,
                (hipStream_t)stream);
}

int rms_norm_backward_bufsize(int64_t rows, int64_t H, int32_t dtype, size_t* bytes) {
    if (!bytes) return SP_ERR_NULL;
    if (rows < 0 || rows > kI32Max || H < 0 || H > kI32Max) return SP_ERR_SIZE;
    if (bad_dtype(dtype)) return SP_ERR_UNSUPPORTED;
    *bytes = rows == 0 || H == 0 ? 0 : rms_norm_backward_bytes(rows, H, dtype);
    return SP_OK;
}

int rms_norm_backward(int64_t rows, int64_t H, int32_t dtype, const void* dY, int64_t lddy, const void* sum, int64_t lds,
                      const void* weight, int32_t w_type, float eps, const void* dsum, int64_t ldd, void* dX,
                      int64_t lddx, float* dweight, void* work, size_t work_bytes, void* stream) {
    const NormRows n{rows, H, dtype, w_type, sum, lds, dsum, ldd, weight, eps};
    int rc = norm_args(n);
    if (rc) return rc;
    if (lddy < H || lddx < H || too_far(rows, lddy) || too_far(rows, lddx)) return SP_ERR_SIZE;
    if (H == 0 || (rows == 0 && !dweight)) return SP_OK;
    if (rows > 0 && (!dY || !sum || !dX)) return SP_ERR_NULL;
    if (misaligned(dY, elem(dtype)) || misaligned(dX, elem(dtype)) || misaligned(dweight, 4)) return SP_ERR_UNSUPPORTED;
    if (dweight && rows > 0) rc = workspace(work, work_bytes, rms_norm_backward_bytes(rows, H, dtype));
    return rc ? rc : rms_norm_backward_device(n, dY, lddy, dX, lddx, dweight, work, (hipStream_t)stream);
}

int moe_gemm(int64_t S, int32_t num_experts, int64_t N, int64_t K, int32_t dtype, const void* A, int64_t a_rows,
             int64_t lda, const int32_t* src, int32_t slots, const void* B, int64_t ldb, int64_t strideb,
             const int32_t* offsets, void* C, int64_t ldc, void* stream) {
    return product(Products{S, num_experts, N, K, dtype, A, a_rows, lda, src, slots, B, ldb, strideb, offsets}, -1, nullptr,
                   0, C, ldc, (hipStream_t)stream);
}

int moe_gated(int64_t S, int32_t num_experts, int64_t N, int64_t K, int32_t dtype, const void* A, int64_t a_rows,
              int64_t lda, const int32_t* src, int32_t slots, const void* B, int64_t ldb, int64_t strideb,
              const int32_t* offsets, int32_t act, void* pre, int64_t ldp, void* C, int64_t ldc, void* stream) {
    if (bad_act(act)) return SP_ERR_UNSUPPORTED;
    return product(Products{S, num_experts, N, K, dtype, A, a_rows, lda, src, slots, B, ldb, strideb, offsets}, act, pre, ldp,
                   C, ldc, (hipStream_t)stream);
}

int moe_gemm_backward_bufsize(int64_t S, int32_t num_experts, int64_t N, int64_t K, int32_t dtype, size_t* bytes) {
    if (!bytes) return SP_ERR_NULL;
    const int rc = sizes(S, num_experts, N, K, dtype);
    if (!rc) *bytes = moe_gemm_backward_bytes(Products{S, num_experts, N, K, dtype});
    return rc;
}

int moe_gemm_backward(int64_t S, int32_t num_experts, int64_t N, int64_t K, int32_t dtype, const void* dC, int64_t ldc,
                      const void* A, int64_t a_rows, int64_t lda, const int32_t* src, int32_t slots, const void* B,
                      int64_t ldb, int64_t strideb, const int32_t* offsets, void* dA, int64_t ldda, void* dB,
                      int64_t lddb, int64_t stridedb, void* work, size_t work_bytes, void* stream) {
    const Products p{S, num_experts, N, K, dtype, A, a_rows, lda, src, slots, B, ldb, strideb, offsets};
    int rc = gradient_args(p, N, dA, ldda, dB, lddb, stridedb);
    if (rc) return rc;
    if (ldc < N || too_far(S, ldc)) return SP_ERR_SIZE;
    if (!dC && S > 0 && N > 0) return SP_ERR_NULL;
    if (misaligned(dC, 2)) return SP_ERR_UNSUPPORTED;
    if (dA || dB) rc = workspace(work, work_bytes, moe_gemm_backward_bytes(p));
    return rc ? rc : moe_gemm_backward_device(p, dC, ldc, dA, ldda, dB, lddb, stridedb, work, (hipStream_t)stream);
}

int moe_gated_backward_bufsize(int64_t S, int32_t num_experts, int64_t N, int64_t K, int32_t dtype, size_t* bytes) {
    if (!bytes) return SP_ERR_NULL;
    const int rc = sizes(S, num_experts, N, K, dtype);
    if (!rc) *bytes = moe_gated_backward_bytes(Products{S, num_experts, N, K, dtype});
    return rc;
}

int moe_gated_backward(int64_t S, int32_t num_experts, int64_t N, int64_t K, int32_t dtype, int32_t act, const void* dH,
                       int64_t ldh, const void* pre, int64_t ldp, const void* A, int64_t a_rows, int64_t lda,
                       const int32_t* src, int32_t slots, const void* B, int64_t ldb, int64_t strideb,
                       const int32_t* offsets, void* dA, int64_t ldda, void* dB, int64_t lddb, int64_t stridedb,
                       void* work, size_t work_bytes, void* stream) {
    if (bad_act(act)) return SP_ERR_UNSUPPORTED;
    const Products p{S, num_experts, N, K, dtype, A, a_rows, lda, src, slots, B, ldb, strideb, offsets};
    int rc = gradient_args(p, 2 * N, dA, ldda, dB, lddb, stridedb);
    if (rc) return rc;
    if (ldh < N || too_far(S, ldh) || ldp < 2 * N || too_far(S, ldp)) return SP_ERR_SIZE;
    if ((!dH || !pre) && S > 0 && N > 0) return SP_ERR_NULL;
    if (misaligned(dH, 2) || misaligned(pre, 2)) return SP_ERR_UNSUPPORTED;
    if (!dA && !dB) return SP_OK;
    rc = workspace(work, work_bytes, moe_gated_backward_bytes(p));
    return rc ? rc : moe_gated_backward_device(p, act, dH, ldh, pre, ldp, dA, ldda, dB, lddb, stridedb, work,
                                               (hipStream_t)stream);
}

}  // extern "C"
