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
    uint32_t m_tiles, n_tiles; // m_tiles is an upper bound when offsets are given; the product fits 31 bits
};

// Tile i of the rows [a, b): as many tiles as BM asks for, of equal height in units of 64 rows.
template <int BM>
__device__ __forceinline__ void cut(int a, int b, int i, int64_t& lo, int64_t& hi) {
    const uint32_t rows = b - a, tiles = (rows + (BM - 1)) / BM;
    const uint32_t units = (rows + 63) / 64;  // 32-bit divisions: a 64-bit one takes hundreds of instructions
    const int64_t height = BM <= 64 ? BM : (units + tiles - 1) / max(tiles, 1u) * 64;
    lo = a + i * height;
    hi = min(lo + height, (int64_t)b);
}

// Row tile number `tile` of the launch: expert e, rows [lo, hi) of its range,
// at most BM of them.  Every wave of a workgroup finds it by itself: the
// experts' tile counts, 64 at a time, a prefix sum over the lanes, and the
// first lane past `tile`.  false: there are fewer tiles than that.  Offsets
// outside [0, S] are clamped, a descending pair is an empty expert.
template <int BM>
__device__ __forceinline__ bool find_tile(const GemmArgs& g, int tile, int lane, int& e, int64_t& lo, int64_t& hi) {
    if (!g.offsets) {
        e = 0;
        cut<BM>(0, (int)g.S, tile, lo, hi);
        return (int64_t)tile * BM < g.S;
    }
    int before = 0;
    for (int e0 = 0; e0 < g.E; e0 += 64) {
        int a = 0, b = 0;
        if (e0 + lane < g.E) {
            a = min(max(g.offsets[e0 + lane], 0), (int)g.S);
            b = max(a, min(max(g.offsets[e0 + lane + 1], 0), (int)g.S));
        }
        const int mine = (int)(((uint32_t)(b - a) + (BM - 1)) / BM);
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
            cut<BM>(__builtin_amdgcn_readlane(a, l), __builtin_amdgcn_readlane(b, l), tile - first, lo, hi);
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
    const uint32_t tiles = g.m_tiles * g.n_tiles;
    for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        int e;
        int64_t lo, hi;
        if (!find_tile<BM>(g, (int)(t / g.n_tiles), l, e, lo, hi)) continue;
        const int64_t n0 = (int64_t)(t % g.n_tiles) * BN;
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

// ---------------------------------------------------------------------------
// Large products: tiles of up to 256 rows x 256 columns, eight waves.
//
// K advances in steps of 128 bytes, double-buffered in LDS: while the matrix
// cores work on one step, global_load_lds brings the next (16 bytes per lane
// straight into LDS; 8 lanes read a whole 128-byte line of a row).  Chunk c of
// a row lies at c ^ (row / 2 % 8): a 16-byte operand read serves 16 lanes, 256
// bytes, at a time, and 16 rows at one c then lie in 16 different places of
// 256 bytes (with row % 8 rows r and r + 8 met in one place: half of all LDS
// cycles were conflicts).
//
// Wave (wm, wn) owns columns 64 wn .. 64 wn + 63 and every second 32-row
// block: rows 32 (2 i + wm), i < F.  F = 1 .. 4 is the tile's height in units
// of 64 rows: a short tile (an expert's last) runs fewer MFMAs and loads fewer
// rows, instead of multiplying rows nobody stores.  An expert's rows are cut
// into tiles of equal height rather than full ones and a rest.
//
// B is the first MFMA operand, so that a lane's four consecutive sums lie in
// one row of C; the sums go through LDS once more to be stored as whole lines.
constexpr int kBig = 256;             // rows and columns of a tile
constexpr int kBigK = 128;            // bytes of K a step
constexpr int kBigRow = 64 + 4;       // LDS words per row of a wave's sums

typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ int big_swizzle(int row) { return (row >> 1) & 7; }

// One wave's share of a step's copies: F blocks of 64 rows of A, then 4 of B;
// copies [from, to) of the F + 4.
template <int F, int FROM, int TO>
__device__ __forceinline__ void big_copy(int8_t* la, int8_t* lb, const int8_t* const (&pa)[4],
                                         const int8_t* const (&pb)[4], int64_t k, int w) {
#pragma unroll
    for (int j = FROM; j < TO; ++j) {
        const int8_t* src = (j < F ? pa[j & 3] : pb[(j - F) & 3]) + k;
        int8_t* dst = (j < F ? la + j * 8192 : lb + (j - F) * 8192) + w * 1024;
        __builtin_amdgcn_global_load_lds((const void*)src, (lds_void*)dst, 16, 0, 0);
    }
}

// MFMA operands of 32 bytes of K: piece ks of a step.
template <int F>
struct BigOps {
    i32x4 a[F], b[2];
    __device__ __forceinline__ void read(const int8_t* la, const int8_t* lb, int ks, int wm, int wn, int l) {
        const int r = l & 31, c = ((2 * ks + (l >> 5)) ^ big_swizzle(r)) << 4;
#pragma unroll
        for (int u = 0; u < 2; ++u) b[u] = *reinterpret_cast<const i32x4*>(lb + (64 * wn + 32 * u + r) * kBigK + c);
#pragma unroll
        for (int i = 0; i < F; ++i) a[i] = *reinterpret_cast<const i32x4*>(la + (32 * (2 * i + wm) + r) * kBigK + c);
    }
    __device__ __forceinline__ void multiply(i32x16 (&acc)[F][2], int i0 = 0, int i1 = F) const {
#pragma unroll
        for (int i = 0; i < F; ++i)
            if (i >= i0 && i < i1)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    acc[i][u] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b[u], a[i], acc[i][u], 0, 0, 0);
    }
    // The same with copies [FROM, FROM + F) .. of a later step between the MFMAs.
    template <int FROM, int TO>
    __device__ __forceinline__ void multiply_and_copy(i32x16 (&acc)[F][2], int8_t* la, int8_t* lb,
                                                      const int8_t* const (&pa)[4], const int8_t* const (&pb)[4],
                                                      int64_t k, int w) const {
        constexpr int N = TO - FROM;
        big_copy<F, FROM, FROM + (N * 1 + F - 1) / F>(la, lb, pa, pb, k, w);
        multiply(acc, 0, 1);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (F > 1) {
            big_copy<F, FROM + (N * 1 + F - 1) / F, FROM + (N * 2 + F - 1) / F>(la, lb, pa, pb, k, w);
            multiply(acc, 1, 2);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (F > 2) {
            big_copy<F, FROM + (N * 2 + F - 1) / F, FROM + (N * 3 + F - 1) / F>(la, lb, pa, pb, k, w);
            multiply(acc, 2, 3);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (F > 3) {
            big_copy<F, FROM + (N * 3 + F - 1) / F, FROM + (N * 4 + F - 1) / F>(la, lb, pa, pb, k, w);
            multiply(acc, 3, 4);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
};

// Waits for the operand reads in flight.  Placed before the next reads are
// issued: left to the compiler, the wait comes after them and takes them in.
__device__ __forceinline__ void big_operands_here() {
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt 0, the others untouched
    __builtin_amdgcn_sched_barrier(0);
}

// Zeroes the bytes from K on in the last step's rows of A (what B holds there is then multiplied by zero).
template <int F>
__device__ __forceinline__ void big_mask(int8_t* la, int left, int tid) {
    for (int i = tid; i < F * 64 * 8; i += 512) {
        const int row = i >> 3, k = ((i & 7) ^ big_swizzle(row)) << 4;
        if (k + 16 <= left) continue;
        i32x4* at = reinterpret_cast<i32x4*>(la + i * 16);
        i32x4 v = *at;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int keep = left - (k + 4 * d);  // bytes of this word
            v[d] = keep >= 4 ? v[d] : keep <= 0 ? 0 : v[d] & ((1 << (8 * keep)) - 1);
        }
        *at = v;
    }
}

template <class D, int F>
__device__ __forceinline__ void big_tile(const GemmArgs& g, int e, int64_t lo, int64_t hi, int64_t n0, int8_t* a0,
                                         int8_t* b0, int8_t* a1, int8_t* b1, int32_t* lrow, float* lscale, int tid, int w,
                                         int l) {
    typedef typename D::T T;
    const int wm = w & 1, wn = w >> 1;
    // the rows this lane copies: 64 j + 8 w + l / 8, chunk (l % 8) ^ big_swizzle(row)
    const int crow = 8 * w + (l >> 3), chunk = ((l & 7) ^ big_swizzle(crow)) << 4;
    const int8_t *pa[4], *pb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t p = lo + 64 * j + crow;
        const int64_t r = j < F && p < hi ? a_row(g, p) : -1;
        pa[j] = g.A + max(r, (int64_t)0) * g.lda;  // a row that is not there copies row 0; its sums are not stored
        if (j < F && (l & 7) == 0) {
            lrow[64 * j + crow] = (int32_t)r;
            lscale[64 * j + crow] = g.a_scale[max(r, (int64_t)0)];
        }
        pb[j] = g.B + e * g.strideb + min(n0 + 64 * j + crow, g.N - 1) * g.ldb;
    }
    if (tid < kBig) lscale[kBig + tid] = g.b_scale[e * g.N + min(n0 + tid, g.N - 1)];
    const int64_t last = (g.K - 1) & ~(int64_t)15;  // chunks behind it are read from there and masked
    const int steps = (int)((g.K + kBigK - 1) / kBigK);
    const int left = (int)(g.K - (int64_t)(steps - 1) * kBigK);

    i32x16 acc[F][2];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][u][r] = 0;

    // The operands of piece ks + 1 are read while the MFMAs of piece ks run.  The
    // barrier that ends a step stands before its last piece's MFMAs, when all of
    // the step's operands are in registers: the copies of step s + 2 and the
    // first operand reads of step s + 1 are then issued under those MFMAs.
    BigOps<F> x0, x1;
    constexpr int kCopies = F + 4, kHalf = kCopies / 2;
    big_copy<F, 0, kCopies>(a0, b0, pa, pb, min((int64_t)chunk, last), w);
    __syncthreads();
    if (steps == 1 && left < kBigK) {
        big_mask<F>(a0, left, tid);
        __syncthreads();
    }
    big_copy<F, 0, kHalf>(a1, b1, pa, pb, min((int64_t)kBigK + chunk, last), w);
    x0.read(a0, b0, 0, wm, wn, l);
#define SPX_STEP(s, la, lb, na, nb)                                                                             \
    {                                                                                                            \
        big_operands_here();                                                                                     \
        x1.read(la, lb, 1, wm, wn, l);                                                                           \
        __builtin_amdgcn_sched_barrier(0);                                                                       \
        x0.template multiply_and_copy<kHalf, kCopies>(acc, na, nb, pa, pb,                                       \
                                             min((int64_t)((s) + 1) * kBigK + chunk, last), w);                  \
        __builtin_amdgcn_sched_barrier(0);                                                                       \
        big_operands_here();                                                                                     \
        x0.read(la, lb, 2, wm, wn, l);                                                                           \
        __builtin_amdgcn_sched_barrier(0);                                                                       \
        x1.multiply(acc);                                                                                        \
        __builtin_amdgcn_sched_barrier(0);                                                                       \
        big_operands_here();                                                                                     \
        x1.read(la, lb, 3, wm, wn, l);                                                                           \
        __builtin_amdgcn_sched_barrier(0);                                                                       \
        x0.multiply(acc);                                                                                        \
        __builtin_amdgcn_sched_barrier(0);                                                                       \
        __syncthreads();                                                                                         \
        if ((s) + 2 == steps && left < kBigK) {                                                                  \
            big_mask<F>(na, left, tid);                                                                          \
            __syncthreads();                                                                                     \
        }                                                                                                        \
        x0.read(na, nb, 0, wm, wn, l);                                                                           \
        __builtin_amdgcn_sched_barrier(0);                                                                       \
        x1.template multiply_and_copy<0, kHalf>(acc, la, lb, pa, pb,                                             \
                                       min((int64_t)((s) + 2) * kBigK + chunk, last), w);                        \
        __builtin_amdgcn_sched_barrier(0);                                                                       \
    }
    int s = 0;
    for (; s + 2 <= steps; s += 2) {
        SPX_STEP(s, a0, b0, a1, b1);
        SPX_STEP(s + 1, a1, b1, a0, b0);
    }
    if (s < steps) SPX_STEP(s, a0, b0, a1, b1);
    __syncthreads();  // the copies behind the last step have landed too
#undef SPX_STEP

    // Sums of one 32-row block at a time through this wave's part of LDS
    // (8.5 KB each, three to a buffer), then 8 consecutive columns a
    // lane, 8 rows an instruction.  D layout of the 32 x 32 MFMA: lane l,
    // register r -> first operand's row 8 (r/4) + 4 (l/32) + r%4 (a column of
    // C), second operand's row l%32 (a row of C).
    int32_t* mine = reinterpret_cast<int32_t*>(w < 3 ? b0 : w < 6 ? b1 : a0) + (w % 3) * (32 * kBigRow);
    const int64_t n = n0 + 64 * wn + 8 * (l & 7);
    float sb[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sb[i] = lscale[kBig + 64 * wn + 8 * (l & 7) + i];
#pragma unroll
    for (int i = 0; i < F; ++i) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const i32x4 v = {acc[i][u][4 * q], acc[i][u][4 * q + 1], acc[i][u][4 * q + 2], acc[i][u][4 * q + 3]};
                *reinterpret_cast<i32x4*>(mine + (l & 31) * kBigRow + 32 * u + 8 * q + 4 * (l >> 5)) = v;
            }
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {  // rolled: straight-line code here is fetched once and costs more than it saves
            const int row = 8 * q + (l >> 3), tr = 32 * (2 * i + wm) + row;
            const i32x4 v0 = *reinterpret_cast<const i32x4*>(mine + row * kBigRow + 8 * (l & 7));
            const i32x4 v1 = *reinterpret_cast<const i32x4*>(mine + row * kBigRow + 8 * (l & 7) + 4);
            const int r = lrow[tr];
            if (r < 0 || n >= g.N) continue;
            const float sa = lscale[tr];
            T* c = (T*)g.C + (lo + tr) * g.ldc + n;
            constexpr int N = Chunk<T>::N;
            typename Chunk<T>::V o[8 / N];
#pragma unroll
            for (int x = 0; x < 8; ++x) o[x / N][x % N] = scaled<D>(x < 4 ? v0[x & 3] : v1[x & 3], sa, sb[x]);
#pragma unroll
            for (int x = 0; x < 8 / N; ++x)
                if (n + x * N < g.N) chunk_store(c + x * N, g.N - n - x * N, o[x]);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <class D>
__global__ __launch_bounds__(512) void gemm_i8_big(GemmArgs g) {
    __shared__ __attribute__((aligned(1024))) int8_t a0[kBig * kBigK], a1[kBig * kBigK], b0[kBig * kBigK], b1[kBig * kBigK];
    __shared__ int32_t lrow[kBig];       // row of A of every row of the tile, or -1
    __shared__ float lscale[2 * kBig];   // scales of the tile's rows, then of its columns
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    // neighbouring tiles on one XCD, four row tiles to a column tile
    const int v = xcd_contiguous((int)blockIdx.x, 0, (int)gridDim.x);
    const uint32_t group = 4 * g.n_tiles, first = v / group * 4, in = v % group;
    const uint32_t high = min(g.m_tiles - first, 4u);
    const int64_t nt = in / high;
    int e;
    int64_t lo, hi;
    if (!find_tile<kBig>(g, (int)(first + in % high), l, e, lo, hi)) return;
    switch ((hi - lo + 63) >> 6) {
        case 1: big_tile<D, 1>(g, e, lo, hi, nt * kBig, a0, b0, a1, b1, lrow, lscale, tid, w, l); break;
        case 2: big_tile<D, 2>(g, e, lo, hi, nt * kBig, a0, b0, a1, b1, lrow, lscale, tid, w, l); break;
        case 3: big_tile<D, 3>(g, e, lo, hi, nt * kBig, a0, b0, a1, b1, lrow, lscale, tid, w, l); break;
        default: big_tile<D, 4>(g, e, lo, hi, nt * kBig, a0, b0, a1, b1, lrow, lscale, tid, w, l); break;
    }
}

bool aligned16(const GemmArgs& g) {
    return ((uintptr_t)g.A | (uintptr_t)g.B | (uintptr_t)g.lda | (uintptr_t)g.ldb | (uintptr_t)(g.E > 1 ? g.strideb : 0)) % 16 == 0;
}

// Tile counts of the launch; false if there are 2^31 or more.
bool set_tiles(GemmArgs& g, int64_t bm, int64_t bn) {
    const int64_t m = g.offsets ? g.S / bm + std::min<int64_t>(g.E, g.S) : (g.S + bm - 1) / bm, n = (g.N + bn - 1) / bn;
    g.m_tiles = (uint32_t)m;
    g.n_tiles = (uint32_t)n;
    return m * n < (int64_t)1 << 31;
}

template <class D>
int launch_big(GemmArgs g, hipStream_t s) {
    set_tiles(g, kBig, kBig);
    hipLaunchKernelGGL((gemm_i8_big<D>), dim3((unsigned)(g.m_tiles * g.n_tiles)), dim3(512), 0, s, g);
    return hipGetLastError() == hipSuccess ? SP_OK : SP_ERR_HIP;
}

template <class D>
int gemm_t(GemmArgs g, hipStream_t s) {
    constexpr int64_t BM = 64, BN = 64;
    const int64_t groups = g.offsets ? std::min<int64_t>(g.E, g.S) : 1;
    if (g.K > 0 && g.a_rows > 0 && aligned16(g) && g.S >= 32 * groups && set_tiles(g, kBig, kBig) &&
        g.m_tiles * g.n_tiles < 1 << 22)
        return launch_big<D>(g, s);
    if (!set_tiles(g, BM, BN)) return SP_ERR_SIZE;
    const uint32_t grid = std::min<uint32_t>(g.m_tiles * g.n_tiles, 1 << 22);
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
