// Rows quantised to int8 with one scale each:
//   a = max |x|,  scale = a / 127,  q = rint(127 x / a)  (ties to even, |q| <= 127)
// so that q * scale differs from x by at most half a step, a / 254.  A row
// whose scale would be a denormal (a < 2^-119) becomes zeros with scale 0; a
// row that holds an Inf or a NaN gets scale NaN and q = 0, so that every
// product with it is NaN.
//
// The quotient is a true division of the exact 127 x (16-bit inputs): a value
// halfway between two codes (x = a / 2 gives 63.5) then rounds to even on any
// machine, which a product with a rounded 127 / a would not.  Above 2^120 both
// are scaled down by 2^8 first, or 127 x would overflow.
#include <algorithm>

#include "device_common.h"
#include "rows.h"

namespace spx {

namespace {

constexpr uint32_t kInfBits = 0x7f800000u;
constexpr uint32_t kTinyBits = (127u - 119u) << 23;  // 2^-119
constexpr uint32_t kHugeBits = (127u + 120u) << 23;  // 2^120

template <int XOR>
__device__ __forceinline__ uint32_t swz_max(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_ds_swizzle((int)v, (XOR << 10) | 0x1f));
}

template <class D>
__global__ __launch_bounds__(256) void quantize_rows_kernel(int64_t rows, int64_t K,
                                                            const typename D::T* __restrict__ X, int64_t ldx,
                                                            int8_t* __restrict__ q, int64_t ldq,
                                                            float* __restrict__ scale) {
    typedef typename D::T T;
    constexpr int N = Chunk<T>::N;
    __shared__ uint32_t part[4];
    const int tid = threadIdx.x;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T* x = X + r * ldx;
        // magnitudes compare as integers; Inf and NaN are the largest
        uint32_t m = 0;
        for (int64_t c = tid; c * N < K; c += 256) {
            const auto v = chunk_load(x + c * N, K - c * N);
#pragma unroll
            for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(D::up(v[i])) & 0x7fffffffu);
        }
        m = swz_max<1>(m), m = swz_max<2>(m), m = swz_max<4>(m), m = swz_max<8>(m), m = swz_max<16>(m);
        m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
        __syncthreads();  // part[] of the previous row has been read
        if ((tid & 63) == 0) part[tid >> 6] = m;
        __syncthreads();
        m = max(max(part[0], part[1]), max(part[2], part[3]));
        const bool live = m >= kTinyBits && m < kInfBits;
        const float f = m >= kHugeBits ? 0x1p-8f : 1.0f;
        const float a = live ? __uint_as_float(m) * f : 1.0f;
        if (tid == 0) scale[r] = m >= kInfBits ? __builtin_nanf("") : live ? __uint_as_float(m) / 127.0f : 0.0f;
        for (int64_t c = tid; c * N < K; c += 256) {
            const auto v = chunk_load(x + c * N, K - c * N);
            int8_t o[N];
#pragma unroll
            for (int i = 0; i < N; ++i)
                o[i] = live ? (int8_t)(int)rintf(127.0f * (D::up(v[i]) * f) / a) : (int8_t)0;
            int8_t* d = q + r * ldq + c * N;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (c * N + i < K) d[i] = o[i];
        }
    }
}

}  // namespace

int quantize_rows_i8_device(int64_t rows, int64_t K, int32_t dtype, const void* X, int64_t ldx, int8_t* q, int64_t ldq,
                            float* scale, hipStream_t s) {
    const dim3 grid((unsigned)std::min<int64_t>(rows, 1 << 20)), block(256);
    if (dtype == SP_F32)
        hipLaunchKernelGGL((quantize_rows_kernel<F32>), grid, block, 0, s, rows, K, (const float*)X, ldx, q, ldq, scale);
    else if (dtype == SP_BF16)
        hipLaunchKernelGGL((quantize_rows_kernel<Bf16>), grid, block, 0, s, rows, K, (const uint16_t*)X, ldx, q, ldq,
                           scale);
    else
        hipLaunchKernelGGL((quantize_rows_kernel<F16>), grid, block, 0, s, rows, K, (const _Float16*)X, ldx, q, ldq,
                           scale);
    return hipGetLastError() == hipSuccess ? SP_OK : SP_ERR_HIP;
}

}  // namespace spx
