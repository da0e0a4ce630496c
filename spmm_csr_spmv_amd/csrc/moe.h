// Declarations of the mixture-of-experts operators and the norm, shared by their entry
// points (moe_api.cpp, layer_api.cpp) and kernels.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "spmm_csr_spmv.h"

namespace spx {

// Mixture of experts (moe.hip), int8 rows (quant.hip) and products (gemm_i8.hip).
size_t moe_sort_work_bytes(int64_t n, int32_t E);
int moe_sort_device(int64_t n, int32_t E, const int32_t* ids, int32_t* offsets, int32_t* src, int32_t* pos,
                    void* work, hipStream_t s);
int moe_dispatch_device(int64_t T, int32_t slots, int64_t H, int64_t S, int32_t dtype, const void* X, int64_t ldx,
                        const int32_t* pos, void* Xs, int64_t lds, hipStream_t s);
int moe_combine_device(int64_t T, int32_t slots, int64_t H, int64_t S, int32_t dtype, const void* Ys, int64_t lds,
                       const int32_t* pos, const float* weights, void* Y, int64_t ldy, hipStream_t s);
int moe_combine_backward_device(int64_t T, int32_t slots, int64_t H, int64_t S, int32_t dtype, const void* dY,
                                int64_t ldy, const void* Ys, int64_t lds, const int32_t* pos, const float* weights,
                                void* dYs, int64_t ldd, float* dweights, hipStream_t s);
int quantize_rows_i8_device(int64_t rows, int64_t K, int32_t dtype, const void* X, int64_t ldx, int8_t* q, int64_t ldq,
                            float* scale, hipStream_t s);
int gemm_i8_device(int64_t S, int32_t E, int64_t N, int64_t K, const int8_t* A, int64_t a_rows, int64_t lda,
                   const float* a_scale, const int32_t* src, int32_t slots, const int8_t* B, int64_t ldb,
                   int64_t strideb, const float* b_scale, const int32_t* offsets, int32_t gate, int32_t c_type, void* C,
                   int64_t ldc, hipStream_t s);  // gate: an activation (B then has 2 N rows a matrix), or -1

// Operands of the 16-bit products (gemm_16.hip); distances in elements.
struct Products {
    int64_t S;  // sorted rows
    int32_t E;
    int64_t N, K;  // columns of C (gated: B has 2 N rows a matrix), length of the sums
    int32_t dtype;
    const void* A;
    int64_t a_rows, lda;
    const int32_t* src;
    int32_t slots;
    const void* B;
    int64_t ldb, strideb;
    const int32_t* offsets;
};
int moe_gemm_device(const Products& p, int32_t gate, void* pre, int64_t ldp, void* C, int64_t ldc, hipStream_t s);
size_t moe_gemm_backward_bytes(const Products& p);
int moe_gemm_backward_device(const Products& p, const void* dC, int64_t ldc, void* dA, int64_t ldda, void* dB,
                             int64_t lddb, int64_t stridedb, void* work, hipStream_t s);
size_t moe_gated_backward_bytes(const Products& p);
int moe_gated_backward_device(const Products& p, int32_t act, const void* dH, int64_t ldh, const void* pre, int64_t ldp,
                              void* dA, int64_t ldda, void* dB, int64_t lddb, int64_t stridedb, void* work,
                              hipStream_t s);

// Rows of the norm (norm.hip).
struct NormRows {
    int64_t rows, H;
    int32_t dtype, w_type;
    const void* X;  // backward: the stored sum
    int64_t ldx;
    const void* R;  // the residual, backward: the sum's own gradient; or NULL
    int64_t ldr;
    const void* weight;  // or NULL
    float eps;
};
// scale: int8 codes in Y; or NULL
int rms_norm_device(const NormRows& n, void* sum, int64_t lds, void* Y, int64_t ldy, float* scale, hipStream_t s);
size_t rms_norm_backward_bytes(int64_t rows, int64_t H, int32_t dtype);
int rms_norm_backward_device(const NormRows& n, const void* dY, int64_t lddy, void* dX, int64_t lddx, float* dweight,
                             void* work, hipStream_t s);

}  // namespace spx
