// Products in 8-bit integers with a scale per row of A (token) and per row of
// B (output channel), over one matrix B or over one per expert:
//   C[p, n] = a_scale[r] b_scale[e, n] sum_k A[r, k] B[e, n, k]
// where p runs over the rows sorted by expert, e is the expert whose range
// offsets[e] .. offsets[e + 1] holds p, and r is p, or the token src[p] / slots.
// The sums are int32 and exact (K <= 131071: K 128^2 < 2^31), so the split of
// K over instructions, waves and workgroups never changes a result; the float
// of a sum is multiplied by a_scale, then by b_scale, and rounded once to C's type.
#include <algorithm>

#include "device_common.h"
#include "rows.h"

namespace spx {

namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
typedef int32_t i32x4_u __attribute__((ext_vector_type(4), aligned(1)));

struct GemmArgs {
    int64_t S, N, K;          // rows of C, columns of C, length of the sums
    const int8_t* A;
    int64_t a_rows, lda;
    const float* a_scale;
    const int32_t* src;       // or NULL: row p of C reads row p of A
    int32_t slots;
    const int8_t* B;          // [E][N][K], rows ldb apart, experts strideb apart
    int64_t ldb, strideb;
    const float* b_scale;     // [E][N]
    const int32_t* offsets;   // or NULL: one matrix, rows 0 .. S
    int32_t E;
    void* C;
    int64_t ldc;
    int64_t m_tiles, n_tiles; // m_tiles is an upper bound when offsets are given
};

// Row tile number `tile` of the launch: expert e, rows [lo, hi) of its range,
// at most BM of them.  Every wave of a workgroup finds it by itself: the
// experts' tile counts, 64 at a time, a prefix sum over the lanes, and the
// first lane past `tile`.  false: there are fewer tiles than that.  Offsets
// outside [0, S] are clamped, a descending pair is an empty expert.
template <int BM>
__device__ __forceinline__ bool find_tile(const GemmArgs& g, int64_t tile, int lane, int& e, int64_t& lo, int64_t& hi) {
    if (!g.offsets) {
        e = 0;
        lo = tile * BM;
        hi = min(lo + BM, g.S);
        return lo < g.S;
    }
    int before = 0;
    for (int e0 = 0; e0 < g.E; e0 += 64) {
        int a = 0, b = 0;
        if (e0 + lane < g.E) {
            a = (int)min(max((int64_t)g.offsets[e0 + lane], (int64_t)0), g.S);
            b = max(a, (int)min(max((int64_t)g.offsets[e0 + lane + 1], (int64_t)0), g.S));
        }
        const int mine = (b - a + (BM - 1)) / BM;
        int sum = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int u = __shfl_up(sum, d, 64);
            if (lane >= d) sum += u;
        }
        const uint64_t past = __ballot(before + sum > tile);
        if (past) {
            const int l = __builtin_ctzll(past);
            e = e0 + l;
            const int first = before + __builtin_amdgcn_readlane(sum, l) - __builtin_amdgcn_readlane(mine, l);
            lo = (int64_t)__builtin_amdgcn_readlane(a, l) + (tile - first) * BM;
            hi = min(lo + BM, (int64_t)__builtin_amdgcn_readlane(b, l));
            return true;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
}

// Row of A that row p of C reads, or -1.
__device__ __forceinline__ int64_t a_row(const GemmArgs& g, int64_t p) {
    if (!g.src) return p < g.a_rows ? p : -1;
    const int f = g.src[p];
    const int r = f / g.slots;
    return f >= 0 && r < g.a_rows ? r : -1;
}

// Bytes [k, k + 16) of a row of K bytes, zero from K on; p need not be aligned.
__device__ __forceinline__ i32x4 load16(const int8_t* row, int64_t k, int64_t K) {
    i32x4 v = {0, 0, 0, 0};
    if (k + 16 <= K) {
        v = *reinterpret_cast<const i32x4_u*>(row + k);
    } else if (k < K) {
        union {
            i32x4 v;
            int8_t b[16];
        } u = {v};
        for (int i = 0; i < 16; ++i)
            if (k + i < K) u.b[i] = row[k + i];
        v = u.v;
    }
    return v;
}

template <class D>
__device__ __forceinline__ typename D::T scaled(int sum, float sa, float sb) {
    return D::down((float)sum * sa * sb);
}

// Any size, alignment and stride: 64 x 64 tile, four waves of 32 x 32, K in
// steps of 64 bytes through registers and LDS.
template <class D>
__global__ __launch_bounds__(256) void gemm_i8_plain(GemmArgs g) {
    constexpr int BM = 64, BN = 64, BK = 64, LD = BK + 16;
    __shared__ __attribute__((aligned(16))) int8_t la[BM * LD], lb[BN * LD];
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63;
    const int row = tid >> 2, chunk = tid & 3;  // what this thread stages
    const int wm = 32 * (w >> 1), wn = 32 * (w & 1);
    const int64_t tiles = g.m_tiles * g.n_tiles;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        int e;
        int64_t lo, hi;
        if (!find_tile<BM>(g, t / g.n_tiles, l, e, lo, hi)) continue;
        const int64_t n0 = t % g.n_tiles * BN;
        const int64_t ar = lo + row < hi ? a_row(g, lo + row) : -1;
        const int8_t* pa = g.A + max(ar, (int64_t)0) * g.lda;
        const int8_t* pb = g.B + e * g.strideb + (n0 + row) * g.ldb;
        const bool bok = n0 + row < g.N;
        i32x16 acc;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0;
        for (int64_t k0 = 0; k0 < g.K; k0 += BK) {
            const int64_t k = k0 + 16 * chunk;
            const i32x4 va = load16(pa, k, ar >= 0 ? g.K : 0), vb = load16(pb, k, bok ? g.K : 0);
            __syncthreads();
            *reinterpret_cast<i32x4*>(la + row * LD + 16 * chunk) = va;
            *reinterpret_cast<i32x4*>(lb + row * LD + 16 * chunk) = vb;
            __syncthreads();
#pragma unroll
            for (int ks = 0; ks < BK; ks += 32) {
                const i32x4 a = *reinterpret_cast<const i32x4*>(la + (wm + (l & 31)) * LD + ks + 16 * (l >> 5));
                const i32x4 b = *reinterpret_cast<const i32x4*>(lb + (wn + (l & 31)) * LD + ks + 16 * (l >> 5));
                acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, acc, 0, 0, 0);
            }
        }
        // D layout of the 32 x 32 MFMA: lane l, register r -> row 8 (r/4) + 4 (l/32) + r%4, column l%32
        const int64_t n = n0 + wn + (l & 31);
        if (n < g.N) {
            const float sb = g.b_scale[e * g.N + n];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int64_t p = lo + wm + 8 * (r >> 2) + 4 * (l >> 5) + (r & 3);
                if (p >= hi) continue;
                const int64_t ra = a_row(g, p);
                if (ra >= 0) ((typename D::T*)g.C)[p * g.ldc + n] = scaled<D>(acc[r], g.a_scale[ra], sb);
            }
        }
    }
}

template <class D>
int gemm_t(GemmArgs g, hipStream_t s) {
    constexpr int64_t BM = 64, BN = 64;
    g.m_tiles = g.offsets ? g.S / BM + std::min<int64_t>(g.E, g.S) : (g.S + BM - 1) / BM;
    g.n_tiles = (g.N + BN - 1) / BN;
    const int64_t grid = std::min<int64_t>(g.m_tiles * g.n_tiles, 1 << 22);
    hipLaunchKernelGGL((gemm_i8_plain<D>), dim3((unsigned)grid), dim3(256), 0, s, g);
    return hipGetLastError() == hipSuccess ? SP_OK : SP_ERR_HIP;
}

}  // namespace

int gemm_i8_device(int64_t S, int32_t E, int64_t N, int64_t K, const int8_t* A, int64_t a_rows, int64_t lda,
                   const float* a_scale, const int32_t* src, int32_t slots, const int8_t* B, int64_t ldb,
                   int64_t strideb, const float* b_scale, const int32_t* offsets, int32_t c_type, void* C, int64_t ldc,
                   hipStream_t s) {
    GemmArgs g{S, N, K, A, a_rows, lda, a_scale, src, slots, B, ldb, strideb, b_scale, offsets, E, C, ldc, 0, 0};
    if (c_type == SP_F32) return gemm_t<F32>(g, s);
    if (c_type == SP_BF16) return gemm_t<Bf16>(g, s);
    return gemm_t<F16>(g, s);
}

}  // namespace spx
