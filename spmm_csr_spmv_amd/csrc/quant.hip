// Rows quantised to int8 with one scale each:
//   a = max |x|,  scale = a / 127,  q = rint(127 x / a)  (ties to even, |q| <= 127)
// so that q * scale differs from x by at most half a step, a / 254.  A row
// whose scale would be a denormal (a < 2^-119) becomes zeros with scale 0; a
// row that holds an Inf or a NaN gets scale NaN and q = 0, so that every
// product with it is NaN.
//
// 127 x is exact (16-bit inputs; rounded to 24 bits for fp32) and the quotient
// is that of a true division, so that a value halfway between two codes
// (x = a / 2 gives 63.5) rounds to even on any machine.  A division an element
// takes more time than the memory, so it is left to the rare chunk that needs
// it: 127 x times a rounded 1 / a is off by at most 127 * 3 * 2^-24, which
// rounds to the same code unless it lies within that of a half.
// Above 2^120 both are scaled down by 2^8 first, or 127 x would overflow.
#include <algorithm>

#include "device_common.h"
#include "moe.h"
#include "rows.h"

namespace spx {

namespace {

constexpr uint32_t kInfBits = 0x7f800000u;
constexpr uint32_t kTinyBits = (127u - 119u) << 23;  // 2^-119
constexpr uint32_t kHugeBits = (127u + 120u) << 23;  // 2^120

template <int S>
struct Bits {
    typedef uint32_t T;
};
template <>
struct Bits<2> {
    typedef uint16_t T;
};

template <int XOR>
__device__ __forceinline__ uint32_t swz_max(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_ds_swizzle((int)v, (XOR << 10) | 0x1f));
}

// TPR lanes share a row, 256 / TPR rows a workgroup.  Up to kHeld chunks a lane
// stay in registers between the maximum and the codes; longer rows are read
// again (from L2).  A last chunk that would pass the row's end starts earlier
// and repeats codes of the one before; rows shorter than a chunk (SHORT) go
// element by element.  Instructions are what bounds it for 16-bit inputs: row
// pointers are scalar (TPR >= 64) and offsets in a row 32-bit.  32768 x 4096
// bf16: 88 us, 4.6 TB/s (106 with the next row loaded ahead); 8192 x 4096 fp32:
// 26 us, 6.5 TB/s.
constexpr int kHeld = 4;

template <class D, int TPR, bool SHORT>
__global__ __launch_bounds__(256) void quantize_rows_kernel(int64_t rows, int32_t K,
                                                            const typename D::T* __restrict__ X, int64_t ldx,
                                                            int8_t* __restrict__ q, int64_t ldq,
                                                            float* __restrict__ scale) {
    typedef typename D::T T;
    typedef typename Chunk<T>::V V;
    constexpr int N = Chunk<T>::N;
    // magnitudes compare as integers; Inf and NaN are the largest
    typedef typename Bits<sizeof(T)>::T B;
    typedef B BV __attribute__((ext_vector_type(N)));
    typedef uint32_t QU __attribute__((ext_vector_type(N / 4), aligned(1)));
    __shared__ uint32_t part[4];
    const int lane = threadIdx.x % TPR;
    const uint32_t chunks = ((uint32_t)K + N - 1) / N, end = SHORT ? 0 : K - N;
    const auto start = [&](uint32_t c) { return min(c * N, end); };
    const int sub = threadIdx.x / TPR;
    for (int64_t r = (int64_t)blockIdx.x * (256 / TPR) + (TPR >= 64 ? __builtin_amdgcn_readfirstlane(sub) : sub);
         r < rows; r += (int64_t)gridDim.x * (256 / TPR)) {
        const T* x = X + r * ldx;
        int8_t* d = q + r * ldq;
        V held[kHeld];
        BV all = (BV)(B)0;
        const auto load = [&](uint32_t c) { return chunk_load(x + start(c), SHORT ? K : N); };
        const auto grow = [&](const V& v) {
            all = __builtin_elementwise_max(all, __builtin_bit_cast(BV, v) & (BV)(B)((B)~(B)0 >> 1));
        };
#pragma unroll
        for (uint32_t h = 0; h < kHeld; ++h)
            if (h * TPR < chunks) held[h] = lane + h * TPR < chunks ? load(lane + h * TPR) : V(0);
#pragma unroll
        for (uint32_t h = 0; h < kHeld; ++h)
            if (h * TPR < chunks) grow(held[h]);
        for (uint32_t c = lane + kHeld * TPR; c < chunks; c += TPR) grow(load(c));
        B most = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) most = max(most, all[i]);
        uint32_t m = __float_as_uint(D::up(__builtin_bit_cast(T, most)));
        m = swz_max<1>(m), m = swz_max<2>(m), m = swz_max<4>(m), m = swz_max<8>(m);
        if (TPR >= 64) {
            m = swz_max<16>(m);
            m = max((uint32_t)__builtin_amdgcn_readlane((int)m, 0), (uint32_t)__builtin_amdgcn_readlane((int)m, 32));
        }
        if (TPR == 256) {
            __syncthreads();  // part[] of the previous row has been read
            if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
            __syncthreads();
            m = max(max(part[0], part[1]), max(part[2], part[3]));
        }
        const bool live = m >= kTinyBits && m < kInfBits;
        const float f = m >= kHugeBits ? 0x1p-8f : 1.0f, f127 = 127.0f * f;  // a power of two: exact
        const float a = live ? __uint_as_float(m) * f : 1.0f, inv = 1.0f / a;
        const uint32_t keep = live ? ~0u : 0u;
        if (lane == 0) scale[r] = m >= kInfBits ? __builtin_nanf("") : live ? __uint_as_float(m) / 127.0f : 0.0f;
        const auto store = [&](uint32_t c, const V& v) {
            // adding 1.5 * 2^23 rounds to an integer, ties to even, and leaves it in the low bits
            constexpr float kMagic = 12582912.0f;
            uint32_t n[N];
            float off = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float x127 = D::up(v[i]) * f127, y = fmaf(x127, inv, kMagic);
                off = fmaxf(off, fabsf(fmaf(x127, inv, -(y - kMagic))));
                n[i] = __float_as_uint(y);
            }
            if (__any(off > 0.4999f)) {
#pragma unroll
                for (int i = 0; i < N; ++i) n[i] = __float_as_uint(D::up(v[i]) * f127 / a + kMagic);
            }
            QU o;
#pragma unroll
            for (int i = 0; i < N; i += 4) {  // the low bytes of four words
                const uint32_t lo = __builtin_amdgcn_perm(n[i + 1], n[i], 0x0c0c0400u);
                const uint32_t hi = __builtin_amdgcn_perm(n[i + 3], n[i + 2], 0x04000c0cu);
                o[i / 4] = (lo | hi) & keep;
            }
            if (SHORT) {
                for (int i = 0; i < K; ++i) d[i] = (int8_t)(o[i / 4] >> (8 * (i % 4)));
            } else {
                *reinterpret_cast<QU*>(d + start(c)) = o;
            }
        };
#pragma unroll
        for (uint32_t h = 0; h < kHeld; ++h)
            if (lane + h * TPR < chunks) store(lane + h * TPR, held[h]);
        for (uint32_t c = lane + kHeld * TPR; c < chunks; c += TPR) store(c, load(c));
    }
}

template <class D>
int quantize_t(int64_t rows, int64_t K, const void* X, int64_t ldx, int8_t* q, int64_t ldq, float* scale,
               hipStream_t s) {
    constexpr int N = Chunk<typename D::T>::N;
    const auto go = [&](auto kernel, int per) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<int64_t>((rows + per - 1) / per, 1 << 20)), dim3(256), 0, s,
                           rows, (int32_t)K, (const typename D::T*)X, ldx, q, ldq, scale);
    };
    // the fewest lanes whose registers hold the row
    if (K < N)
        go(quantize_rows_kernel<D, 16, true>, 16);
    else if (K <= 16 * N * kHeld)
        go(quantize_rows_kernel<D, 16, false>, 16);
    else if (K <= 64 * N * kHeld)
        go(quantize_rows_kernel<D, 64, false>, 4);
    else
        go(quantize_rows_kernel<D, 256, false>, 1);
    return hipGetLastError() == hipSuccess ? SP_OK : SP_ERR_HIP;
}

}  // namespace

int quantize_rows_i8_device(int64_t rows, int64_t K, int32_t dtype, const void* X, int64_t ldx, int8_t* q, int64_t ldq,
                            float* scale, hipStream_t s) {
    if (dtype == SP_F32) return quantize_t<F32>(rows, K, X, ldx, q, ldq, scale, s);
    if (dtype == SP_BF16) return quantize_t<Bf16>(rows, K, X, ldx, q, ldq, scale, s);
    return quantize_t<F16>(rows, K, X, ldx, q, ldq, scale, s);
}

}  // namespace spx
