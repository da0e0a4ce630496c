// Products in 8-bit integers with a scale per row of A (token) and per row of
// B (output channel), over one matrix B or over one per expert:
//   C[p, n] = a_scale[r] b_scale[e, n] sum_k A[r, k] B[e, n, k]
// where p runs over the rows sorted by expert, e is the expert whose range
// offsets[e] .. offsets[e + 1] holds p, and r is p, or the token src[p] / slots.
// The sums are int32 and exact (K <= 131071: K 128^2 < 2^31), so the split of
// K over instructions and waves never changes a result; the float of a sum is
// multiplied by a_scale, then by b_scale, and rounded once to C's type.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "moe.h"
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

// The rows of an expert make as many tiles as BM asks for, of equal height in
// units of 64 rows (the last may be lower).  32-bit divisions: a 64-bit one
// takes hundreds of instructions.
template <int BM>
__device__ __forceinline__ uint32_t row_tiles_of(uint32_t rows) {
    return (rows + (BM - 1)) / BM;
}

// Tile i of the rows [a, b).
template <int BM>
__device__ __forceinline__ void cut(int a, int b, int i, int64_t& lo, int64_t& hi) {
    const uint32_t rows = b - a, tiles = max(row_tiles_of<BM>(rows), 1u), units = (rows + 63) / 64;
    const int64_t height = BM <= 64 ? BM : (units + tiles - 1) / tiles * 64;
    lo = a + i * height;
    hi = min(lo + height, (int64_t)b);
}

// Rows [a, b) of expert e.  Offsets outside [0, S] are clamped, a descending
// pair is an empty expert.
__device__ __forceinline__ void expert_rows(const GemmArgs& g, int e, int& a, int& b) {
    a = b = 0;
    if (e < g.E) {
        a = min(max(g.offsets[e], 0), (int)g.S);
        b = max(a, min(max(g.offsets[e + 1], 0), (int)g.S));
    }
}

// Inclusive prefix sum over the 64 lanes: shifts by 1, 2, 4, 8 within rows of
// 16 lanes, then the last lane of row 0 and 2 to the next row, and lane 31 to the upper half.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t lanes_from(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
    v += lanes_from<0x111, 0xf>(v);
    v += lanes_from<0x112, 0xf>(v);
    v += lanes_from<0x114, 0xf>(v);
    v += lanes_from<0x118, 0xf>(v);
    v += lanes_from<0x142, 0xa>(v);
    v += lanes_from<0x143, 0xc>(v);
    return v;
}

// Row tiles that the experts' rows make (the launch has room for more: it
// does not know the offsets).  Every wave counts for itself, 64 experts at a time.
// Offsets whose ranges overlap can make more than the launch has room for, and more
// than 32 bits count: the bound keeps the loop of gemm_i8_staged below 2^31.
template <int BM>
__device__ __forceinline__ uint32_t count_tiles(const GemmArgs& g, int lane) {
    if (!g.offsets) return g.m_tiles;
    uint32_t n = 0;
    for (int e0 = 0; e0 < g.E; e0 += 64) {
        int a, b;
        expert_rows(g, e0 + lane, a, b);
        n += __builtin_amdgcn_readlane(wave_scan(row_tiles_of<BM>(b - a)), 63);
    }
    return min(n, g.m_tiles);
}

// Row tile number `tile` of the launch: expert e and rows [lo, hi) of its
// range, found by every wave of a workgroup for itself: the experts' tile
// counts, a prefix sum over the lanes, and the first lane past `tile`.
// false: there are fewer tiles than that.
template <int BM>
__device__ __forceinline__ bool find_tile(const GemmArgs& g, uint32_t tile, int lane, int& e, int64_t& lo,
                                          int64_t& hi) {
    if (!g.offsets) {
        e = 0;
        cut<BM>(0, (int)g.S, (int)tile, lo, hi);
        return (int64_t)tile * BM < g.S;
    }
    uint32_t before = 0;
    for (int e0 = 0; e0 < g.E; e0 += 64) {
        int a, b;
        expert_rows(g, e0 + lane, a, b);
        const uint32_t mine = row_tiles_of<BM>(b - a), sum = wave_scan(mine);
        const uint64_t past = __ballot(before + sum > tile);
        if (past) {
            const int l = __builtin_ctzll(past);
            e = e0 + l;
            const uint32_t first = before + __builtin_amdgcn_readlane(sum, l) - __builtin_amdgcn_readlane(mine, l);
            cut<BM>(__builtin_amdgcn_readlane(a, l), __builtin_amdgcn_readlane(b, l), (int)(tile - first), lo, hi);
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

// Rows that start anywhere (K >= 16): 16 bytes at min(k, K - 16), so that nothing
// outside the row is read.  The last piece of a row that K cuts then begins
// with bytes that the piece before holds too; low_mask zeroes them on A's
// side (word d of the four, for a piece wanted at k), B's are multiplied by zero.
__device__ __forceinline__ i32x4 load_any(const int8_t* row, int64_t k, int64_t K) {
    return *reinterpret_cast<const i32x4_u*>(row + min(k, K - 16));
}
// For rows that nothing else reads: non-temporal.
__device__ __forceinline__ i32x4 load_any_once(const int8_t* row, int64_t k, int64_t K) {
    return __builtin_nontemporal_load(reinterpret_cast<const i32x4_u*>(row + min(k, K - 16)));
}
__device__ __forceinline__ int32_t low_mask(int64_t k, int64_t K, int d) {
    const int64_t drop = k - (K - 16) - 4 * d;
    return drop <= 0 ? -1 : drop >= 4 ? 0 : (int32_t)(0xffffffffu << (8 * (int)drop));
}

// The bytes of a row shorter than 16 from k on, zeros behind them.
__device__ __forceinline__ i32x4 load_short(const int8_t* row, int64_t k, int64_t K) {
    i32x4 v = {0, 0, 0, 0};
    for (int i = 0; i < 16; ++i)
        if (k + i < K) v[i >> 2] |= (int32_t)((uint32_t)(uint8_t)row[k + i] << (8 * (i & 3)));
    return v;
}

// A sum is below 2^31, so times a scale above 2^96 it can pass fp32's range where
// the result does not (rows whose largest value is near the type's).  Such a scale
// goes in times 2^-32 and the result is multiplied by 2^32, both exact.  That path
// (FAR) is taken where a tile, or the rows of a wave, hold such a scale: the last
// factor on every product made 8192 x 8192 x 4096 take 248 us, without 240, so 240.
__device__ __forceinline__ bool far_scale(float sa) { return fabsf(sa) > 0x1p96f; }
template <class D, bool FAR>
__device__ __forceinline__ typename D::T scaled(int sum, float sa, float sb) {
    // The product is an fp32 number before it is rounded to C's type: left to itself
    // the compiler fuses the two for fp16 in some tiles and not in others, and the
    // last bit then depends on where in C a value stands.
#pragma clang fp contract(off)
    if (FAR && far_scale(sa)) return D::down((float)sum * (sa * 0x1p-32f) * sb * 0x1p32f);
    return D::down((float)sum * sa * sb);
}

// ---------------------------------------------------------------------------
// Many rows: tiles of up to 64 WN rows x 64 WN columns by 2 WN waves, WN = 4
// (256 x 256, one workgroup a CU) or 2 (128 x 128, two).
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
// block: rows 32 (2 i + wm), i < F.  F = 1 .. WN is the tile's height in units
// of 64 rows: a short tile (an expert's last) runs fewer MFMAs and loads fewer
// rows, instead of multiplying rows nobody stores.  An expert's rows are cut
// into tiles of equal height rather than full ones and a rest.
//
// B is the first MFMA operand, so that a lane's four consecutive sums lie in
// one row of C; the sums go through LDS once more to be stored as whole lines.
//
// 8192 x 8192 x 8192 (WN = 4) takes 461 us, 2.39 POP/s (443 to 468 on several
// cards); the MFMAs fill 65 % of the cycles and the chip runs at 1.7 GHz under them
// (one tile alone: 71 % at 2.4 GHz), so that power bounds it.  LDS operand reads
// take 27 % of them, without conflicts.
constexpr int kBigK = 128;            // bytes of K a step
constexpr int kBigRow = 64 + 4;       // LDS words per row of a wave's sums

typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ int big_swizzle(int row) { return (row >> 1) & 7; }

// Copy instructions a wave issues for a step: 16 WN rows each over the workgroup.
template <int WN, int F>
struct BigShape {
    static constexpr int kRows = 16 * WN;            // rows that one instruction of every wave covers
    static constexpr int kA = 64 * F / kRows;        // for the rows of A
    static constexpr int kB = 64 * WN / kRows;       // for the rows of B
    static constexpr int kCopies = kA + kB;
};

// Copies [FROM, TO) of the step's, in the order A, B.  ONCE: no other tile reads these rows of B.
template <int WN, int F, bool ONCE, int FROM, int TO>
__device__ __forceinline__ void big_copy(int8_t* la, int8_t* lb, const int8_t* const (&pa)[4],
                                         const int8_t* const (&pb)[4], int64_t k, int w) {
    using S = BigShape<WN, F>;
#pragma unroll
    for (int j = FROM; j < TO; ++j) {
        const int8_t* src = (j < S::kA ? pa[j & 3] : pb[(j - S::kA) & 3]) + k;
        int8_t* dst = (j < S::kA ? la + j * S::kRows * kBigK : lb + (j - S::kA) * S::kRows * kBigK) + w * 1024;
        if (ONCE && j >= S::kA)
            __builtin_amdgcn_global_load_lds((const void*)src, (lds_void*)dst, 16, 0, 2);  // non-temporal
        else
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
    // The same with copies [FROM, TO) of a later step spread between the MFMAs:
    // a wave that issues them in one go waits for the memory pipeline to take them.
    template <int WN, bool ONCE, int FROM, int TO, int I = 0>
    __device__ __forceinline__ void multiply_and_copy(i32x16 (&acc)[F][2], int8_t* la, int8_t* lb,
                                                      const int8_t* const (&pa)[4], const int8_t* const (&pb)[4],
                                                      int64_t k, int w) const {
        constexpr int N = TO - FROM;
        big_copy<WN, F, ONCE, FROM + (N * I + F - 1) / F, FROM + (N * (I + 1) + F - 1) / F>(la, lb, pa, pb, k, w);
        multiply(acc, I, I + 1);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (I + 1 < F) multiply_and_copy<WN, ONCE, FROM, TO, I + 1>(acc, la, lb, pa, pb, k, w);
    }
};

// Waits for the operand reads in flight.  Placed before the next reads are
// issued: left to the compiler, the wait comes after them and takes them in.
__device__ __forceinline__ void big_operands_here() {
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt 0, the others untouched
    __builtin_amdgcn_sched_barrier(0);
}

// Zeroes the bytes from K on in the last step's rows of A (what B holds there is then multiplied by zero).
template <int WN, int F>
__device__ __forceinline__ void big_mask(int8_t* la, int left, int tid) {
    for (int i = tid; i < F * 64 * 8; i += 128 * WN) {
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

// The buffers of a step: ST of them, each an array of its own, so that the
// compiler can tell the copies into one from the operand reads of another.
template <int ST>
struct BigBuffers {
    int8_t *a[ST], *b[ST];
};

// s_waitcnt that leaves at most n vector-memory operations outstanding and
// waits for all LDS operations (vmcnt in bits 3:0 and 15:14, expcnt 6:4,
// lgkmcnt 11:8), then the barrier.
template <int N>
__device__ __forceinline__ void big_barrier() {
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
    asm volatile("s_barrier" ::: "memory");
}

// Where a lane's copies read: rows kRows j + 8 w + l / 8 of the tile, chunk
// (l % 8) ^ big_swizzle(row); the tile's rows of A and scales go to LDS, and behind
// the rows a word of each wave that says whether it met a far scale.
template <int WN, int F>
struct BigRows {
    const int8_t *a[4], *b[4];
    int chunk;
    __device__ __forceinline__ BigRows(const GemmArgs& g, int e, int64_t lo, int64_t hi, int64_t n0, int32_t* lrow,
                                       float* lscale, int tid, int w, int l) {
        using S = BigShape<WN, F>;
        const int crow = 8 * w + (l >> 3);
        chunk = ((l & 7) ^ big_swizzle(crow)) << 4;
        bool far = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = S::kRows * j + crow;
            const int64_t p = lo + row;
            const int64_t r = j < S::kA && p < hi ? a_row(g, p) : -1;
            a[j] = g.A + max(r, (int64_t)0) * g.lda;  // a row that is not there copies row 0; its sums are not stored
            if (j < S::kA && (l & 7) == 0) {
                lrow[row] = (int32_t)r;
                const float sa = g.a_scale[max(r, (int64_t)0)];
                lscale[row] = sa;
                far |= far_scale(sa);
            }
            b[j] = g.B + e * g.strideb + min(n0 + row, g.N - 1) * g.ldb;
        }
        lrow[64 * WN + w] = __any(far);
        if (tid < 64 * WN) lscale[64 * WN + tid] = g.b_scale[e * g.N + min(n0 + tid, g.N - 1)];
    }
};

// The tile's sums scaled and stored; l0 .. l3 are LDS buffers of 64 WN x kBigK
// bytes that nothing uses any more.
template <class D, int WN, int F>
__device__ __forceinline__ void big_out(const GemmArgs& g, const i32x16 (&acc)[F][2], int8_t* l0, int8_t* l1, int8_t* l2,
                                        int8_t* l3, const int32_t* lrow, const float* lscale, int64_t lo, int64_t n0,
                                        int w, int l) {
    typedef typename D::T T;
    const int wm = w & 1, wn = w >> 1;
    // Sums of one 32-row block at a time through this wave's part of LDS, then 8
    // consecutive columns a lane, 8 rows an instruction.  D layout of the 32 x 32
    // MFMA: lane l, register r -> first operand's row 8 (r/4) + 4 (l/32) + r%4 (a
    // column of C), second operand's row l%32 (a row of C).
    constexpr int kSums = 32 * kBigRow, kPer = 64 * WN * kBigK / (4 * kSums);  // waves to a buffer
    static_assert(4 * kPer >= 2 * WN, "the waves' sums fit the four buffers");
    int8_t* const buffer = w / kPer == 0 ? l0 : w / kPer == 1 ? l1 : w / kPer == 2 ? l2 : l3;
    int32_t* mine = reinterpret_cast<int32_t*>(buffer) + (w % kPer) * kSums;
    constexpr int N = Chunk<T>::N;
    const int64_t n = n0 + 64 * wn + 8 * (l & 7);
    const bool far = __any(lrow[64 * WN + (l & (2 * WN - 1))]);  // whether any row of the tile has a far scale
    const bool inside = n0 + 64 * WN <= g.N && !far;  // the whole tile's columns, and ordinary scales
    float sb[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sb[i] = lscale[64 * WN + 64 * wn + 8 * (l & 7) + i];
    // one 32-row block; `whole` (a compile-time constant) where all is inside
    const auto block = [&](int i, auto whole) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const i32x4 v = {acc[i][u][4 * q], acc[i][u][4 * q + 1], acc[i][u][4 * q + 2], acc[i][u][4 * q + 3]};
                *reinterpret_cast<i32x4*>(mine + (l & 31) * kBigRow + 32 * u + 8 * q + 4 * (l >> 5)) = v;
            }
        __builtin_amdgcn_wave_barrier();
        const auto row_out = [&](float sa, i32x4 v0, i32x4 v1, int64_t tr) {
            T* c = (T*)g.C + (lo + tr) * g.ldc + n;
            typename Chunk<T>::V o[8 / N];
#pragma unroll
            for (int x = 0; x < 8; ++x) o[x / N][x % N] = scaled<D, !whole.value>(x < 4 ? v0[x & 3] : v1[x & 3], sa, sb[x]);
#pragma unroll
            for (int x = 0; x < 8 / N; ++x) {
                if (whole.value)
                    *reinterpret_cast<typename Chunk<T>::U*>(c + x * N) = o[x];
                else if (n + x * N < g.N)
                    chunk_store(c + x * N, g.N - n - x * N, o[x]);
            }
        };
        const int32_t* at = mine + (l >> 3) * kBigRow + 8 * (l & 7);
        const int tr0 = 32 * (2 * i + wm) + (l >> 3);
        if (whole.value) {
            i32x4 v[4][2];
            int r[4];
            float sa[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[q][0] = *reinterpret_cast<const i32x4*>(at + 8 * q * kBigRow);
                v[q][1] = *reinterpret_cast<const i32x4*>(at + 8 * q * kBigRow + 4);
                r[q] = lrow[tr0 + 8 * q];
                sa[q] = lscale[tr0 + 8 * q];
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (r[q] >= 0) row_out(sa[q], v[q][0], v[q][1], tr0 + 8 * q);
        } else {
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                const i32x4 v0 = *reinterpret_cast<const i32x4*>(at + 8 * q * kBigRow);
                const i32x4 v1 = *reinterpret_cast<const i32x4*>(at + 8 * q * kBigRow + 4);
                const int r = lrow[tr0 + 8 * q];
                if (r >= 0) row_out(lscale[tr0 + 8 * q], v0, v1, tr0 + 8 * q);
            }
        }
        __builtin_amdgcn_wave_barrier();
    };
    if (inside) {
#pragma unroll
        for (int i = 0; i < F; ++i) block(i, std::true_type());
    } else {
#pragma unroll
        for (int i = 0; i < F; ++i) block(i, std::false_type());
    }
}

template <class D, int WN, int ST, bool ONCE, int F>
__device__ __forceinline__ void big_tile(const GemmArgs& g, int e, int64_t lo, int64_t hi, int64_t n0,
                                         const BigBuffers<ST>& m, int32_t* lrow, float* lscale, int tid, int w, int l) {
    using S = BigShape<WN, F>;
    const int wm = w & 1, wn = w >> 1;
    const BigRows<WN, F> rows(g, e, lo, hi, n0, lrow, lscale, tid, w, l);
    const auto& pa = rows.a;
    const auto& pb = rows.b;
    const int chunk = rows.chunk;
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
    // the step's operands are in registers: its buffer then takes the copies of
    // step s + ST, half of them under those MFMAs and half under the next
    // piece's.  Before the barrier a wave waits for its own copies of step s + 1;
    // those of ST - 2 later steps stay in flight.  Copies behind the last step
    // read its last chunk again, which keeps the counts the same.
    BigOps<F> x0, x1;
    constexpr int kCopies = S::kCopies, kHalf = kCopies / 2;
#define SPX_AT(s) min((int64_t)(s) * kBigK + chunk, last)
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) big_copy<WN, F, ONCE, 0, kCopies>(m.a[i], m.b[i], pa, pb, SPX_AT(i), w);
    big_copy<WN, F, ONCE, 0, kHalf>(m.a[ST - 1], m.b[ST - 1], pa, pb, SPX_AT(ST - 1), w);
    big_barrier<(ST - 2) * kCopies + kHalf>();
    if (steps == 1 && left < kBigK) {
        big_mask<WN, F>(m.a[0], left, tid);
        big_barrier<(ST - 2) * kCopies + kHalf>();
    }
    x0.read(m.a[0], m.b[0], 0, wm, wn, l);
#define SPX_STEP(s, I)                                                                                   \
    {                                                                                                     \
        constexpr int kNext = ((I) + 1) % ST, kBack = ((I) + ST - 1) % ST;                                \
        big_operands_here();                                                                              \
        x1.read(m.a[I], m.b[I], 1, wm, wn, l);                                                            \
        __builtin_amdgcn_sched_barrier(0);                                                                \
        x0.template multiply_and_copy<WN, ONCE, kHalf, kCopies>(acc, m.a[kBack], m.b[kBack], pa, pb,      \
                                                                SPX_AT((s) + ST - 1), w);                       \
        big_operands_here();                                                                              \
        x0.read(m.a[I], m.b[I], 2, wm, wn, l);                                                            \
        __builtin_amdgcn_sched_barrier(0);                                                                \
        x1.multiply(acc);                                                                                 \
        big_operands_here();                                                                              \
        x1.read(m.a[I], m.b[I], 3, wm, wn, l);                                                            \
        __builtin_amdgcn_sched_barrier(0);                                                                \
        x0.multiply(acc);                                                                                 \
        __builtin_amdgcn_sched_barrier(0);                                                                \
        big_barrier<(ST - 2) * kCopies>();                                                                \
        if ((s) + 2 == steps && left < kBigK) {                                                           \
            big_mask<WN, F>(m.a[kNext], left, tid);                                                       \
            big_barrier<(ST - 2) * kCopies>();                                                            \
        }                                                                                                 \
        x0.read(m.a[kNext], m.b[kNext], 0, wm, wn, l);                                                    \
        __builtin_amdgcn_sched_barrier(0);                                                                \
        x1.template multiply_and_copy<WN, ONCE, 0, kHalf>(acc, m.a[I], m.b[I], pa, pb, SPX_AT((s) + ST), w); \
    }
    int s = 0;
    for (; s + ST <= steps; s += ST) {
        SPX_STEP(s, 0);
        SPX_STEP(s + 1, 1);
        if constexpr (ST == 4) {
            SPX_STEP(s + 2, 2);
            SPX_STEP(s + 3, 3);
        }
    }
    if (s < steps) {
        SPX_STEP(s, 0);
        if constexpr (ST == 4) {
            if (s + 1 < steps) {
                SPX_STEP(s + 1, 1);
                if (s + 2 < steps) SPX_STEP(s + 2, 2);
            }
        }
    }
#undef SPX_STEP
#undef SPX_AT
    big_barrier<0>();  // the copies behind the last step have landed too: the sums take their LDS

    big_out<D, WN, F>(g, acc, m.b[0], m.b[1], m.a[0], m.a[1], lrow, lscale, lo, n0, w, l);
}

// Tile number t of the m_tiles x n_tiles that there are.  Four row tiles to a
// column tile follow each other.  It is the tiles that there are, not those that
// the launch has room for, that are dealt out to the XCDs.
//
// One matrix: neighbours run on one XCD and share rows of A and of B in its L2.
// Experts: tiles go to the XCDs RUN at a time in turn: experts with many rows,
// bound by the matrix cores, and with few, bound by memory, are then under way
// on all of them.  Against runs of neighbours, and one and eight at a time (us;
// uneven loads are log-normal with sigma 0.7): 8192 rows of 64 uneven experts,
// 4096 x 2048 192, 179, 186; 16384 of 128, 2048 x 1536 141, 131, 132; 512 of 8
// even ones, 4096 x 14336 133, 119, 132; in 256 x 256 tiles 8192 of 8 541, 524,
// 515; 32768 of 64, 4096 x 2048 340, 338, 336.  The tallest tiles first gained
// nothing on that.  RUN = 0, neighbours, where a row tile has few column tiles
// and all matrices fit the caches: 40000 of 16, 512 x 300 26, 29, 29.
template <int WN, int RUN>
__device__ __forceinline__ bool big_place(const GemmArgs& g, uint32_t m_tiles, uint32_t t, int lane, int& e,
                                          int64_t& lo, int64_t& hi, int64_t& n0) {
    const uint32_t all = m_tiles * g.n_tiles;
    constexpr uint32_t kRound = RUN > 0 ? RUN * kXcds : 1;
    uint32_t v = t;
    if (RUN == 0 || !g.offsets)
        v = (uint32_t)xcd_contiguous((int)t, 0, (int)all);
    else if (t < all / kRound * kRound)
        v = t / kRound * kRound + t % kXcds * RUN + t / kXcds % RUN;
    const uint32_t group = 4 * g.n_tiles, first = v / group * 4, in = v % group;
    const uint32_t high = min(m_tiles - first, 4u);
    n0 = (int64_t)(in / high) * (64 * WN);
    return find_tile<64 * WN>(g, first + in % high, lane, e, lo, hi);
}

template <class D, int WN, int ST, bool ONCE>
__global__ __launch_bounds__(128 * WN, WN * ST <= 4 ? 2 : 1) void gemm_i8_big(GemmArgs g) {
    constexpr int kBytes = 64 * WN * kBigK;
    __shared__ __attribute__((aligned(1024))) int8_t a0[kBytes], a1[kBytes], b0[kBytes], b1[kBytes];
    __shared__ int32_t lrow[64 * WN + 2 * WN];  // row of A of every row of the tile, or -1; words of the waves
    __shared__ float lscale[2 * 64 * WN];   // scales of the tile's rows, then of its columns
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    int e;
    int64_t lo, hi, n0;
    const uint32_t m_tiles = count_tiles<64 * WN>(g, l);
    if (blockIdx.x >= m_tiles * g.n_tiles) return;
    if (!big_place<WN, ST == 4 ? 1 : WN == 4 ? 8 : 0>(g, m_tiles, blockIdx.x, l, e, lo, hi, n0)) return;
    const int blocks = (int)((hi - lo + 63) >> 6);
    if constexpr (ST == 4) {
        __shared__ __attribute__((aligned(1024))) int8_t a2[kBytes], a3[kBytes], b2[kBytes], b3[kBytes];
        const BigBuffers<4> m = {{a0, a1, a2, a3}, {b0, b1, b2, b3}};
        if (blocks == 1) return big_tile<D, WN, ST, ONCE, 1>(g, e, lo, hi, n0, m, lrow, lscale, tid, w, l);
        big_tile<D, WN, ST, ONCE, 2>(g, e, lo, hi, n0, m, lrow, lscale, tid, w, l);
    } else {
        const BigBuffers<2> m = {{a0, a1}, {b0, b1}};
        if (blocks == 1) return big_tile<D, WN, ST, ONCE, 1>(g, e, lo, hi, n0, m, lrow, lscale, tid, w, l);
        if constexpr (WN == 4) {
            if (blocks == 3) return big_tile<D, WN, ST, ONCE, 3>(g, e, lo, hi, n0, m, lrow, lscale, tid, w, l);
            if (blocks == 4) return big_tile<D, WN, ST, ONCE, 4>(g, e, lo, hi, n0, m, lrow, lscale, tid, w, l);
        }
        big_tile<D, WN, ST, ONCE, 2>(g, e, lo, hi, n0, m, lrow, lscale, tid, w, l);
    }
}

// ---------------------------------------------------------------------------
// Rows of any alignment and length: the 128 x 128 tiles, with the copies
// through registers (global_load_lds wants aligned pieces): the next step's
// loads are in flight while this one is multiplied, and go to the other LDS
// buffer after it.  8192 x 8192 x 4095 takes 474 us, 1.16 POP/s, bound by the
// unaligned loads (with aligned rows, copied straight to LDS, these tiles take
// 313).  A workgroup goes on to the next tile where there are more
// than the launch has workgroups.
template <class D, int F>
__device__ __forceinline__ void staged_tile(const GemmArgs& g, int e, int64_t lo, int64_t hi, int64_t n0,
                                            const BigBuffers<2>& m, int32_t* lrow, float* lscale, int tid, int w, int l) {
    using S = BigShape<2, F>;
    const int wm = w & 1, wn = w >> 1;
    const BigRows<2, F> rows(g, e, lo, hi, n0, lrow, lscale, tid, w, l);
    const int steps = (int)((g.K + kBigK - 1) / kBigK);
    i32x4 v[S::kCopies];
    const auto load = [&](int s) {
        const int64_t k = (int64_t)s * kBigK + rows.chunk;
        if (g.K >= 16) {
#pragma unroll
            for (int j = 0; j < S::kCopies; ++j) v[j] = load_any(j < S::kA ? rows.a[j & 3] : rows.b[(j - S::kA) & 3], k, g.K);
        } else {
#pragma unroll
            for (int j = 0; j < S::kCopies; ++j)
                v[j] = load_short(j < S::kA ? rows.a[j & 3] : rows.b[(j - S::kA) & 3], k, g.K);
        }
    };
    const auto store = [&](int s) {
        const int64_t k = (int64_t)s * kBigK + rows.chunk;
        if (s == steps - 1 && g.K >= 16) {
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int32_t keep = low_mask(k, g.K, d);
#pragma unroll
                for (int j = 0; j < S::kA; ++j) v[j][d] &= keep;
            }
        }
        int8_t* la = (s & 1 ? m.a[1] : m.a[0]) + w * 1024 + l * 16;
        int8_t* lb = (s & 1 ? m.b[1] : m.b[0]) + w * 1024 + l * 16;
#pragma unroll
        for (int j = 0; j < S::kCopies; ++j)
            *reinterpret_cast<i32x4*>(j < S::kA ? la + j * S::kRows * kBigK : lb + (j - S::kA) * S::kRows * kBigK) = v[j];
    };

    i32x16 acc[F][2];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][u][r] = 0;
    if (steps > 0) {
        load(0);
        store(0);
    }
    __syncthreads();
    for (int s = 0; s < steps; ++s) {
        const int8_t* la = s & 1 ? m.a[1] : m.a[0];
        const int8_t* lb = s & 1 ? m.b[1] : m.b[0];
        if (s + 1 < steps) load(s + 1);
        BigOps<F> x0, x1;
        x0.read(la, lb, 0, wm, wn, l);
#pragma unroll
        for (int ks = 0; ks < 4; ks += 2) {
            x1.read(la, lb, ks + 1, wm, wn, l);
            x0.multiply(acc);
            if (ks == 0) x0.read(la, lb, 2, wm, wn, l);
            x1.multiply(acc);
        }
        if (s + 1 < steps) store(s + 1);
        __syncthreads();
    }
    big_out<D, 2, F>(g, acc, m.b[0], m.b[1], m.a[0], m.a[1], lrow, lscale, lo, n0, w, l);
}

template <class D>
__global__ __launch_bounds__(256, 2) void gemm_i8_staged(GemmArgs g) {
    constexpr int kBytes = 128 * kBigK;
    __shared__ __attribute__((aligned(1024))) int8_t a0[kBytes], a1[kBytes], b0[kBytes], b1[kBytes];
    __shared__ int32_t lrow[128 + 4];
    __shared__ float lscale[2 * 128];
    const BigBuffers<2> m = {{a0, a1}, {b0, b1}};
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    const uint32_t m_tiles = count_tiles<128>(g, l), total = m_tiles * g.n_tiles;
    for (uint32_t t = blockIdx.x; t < total; t += gridDim.x) {
        int e;
        int64_t lo, hi, n0;
        if (!big_place<2, 8>(g, m_tiles, t, l, e, lo, hi, n0)) continue;
        __syncthreads();  // the tile before has been stored
        if (hi - lo <= 64)
            staged_tile<D, 1>(g, e, lo, hi, n0, m, lrow, lscale, tid, w, l);
        else
            staged_tile<D, 2>(g, e, lo, hi, n0, m, lrow, lscale, tid, w, l);
    }
}

// ---------------------------------------------------------------------------
// Few rows: tiles of 16 R rows x 16 C columns, W waves that share the tile and
// split K; rows of any alignment, K >= 16.
//
// With few rows the time is that of reading B once.  Each wave takes 128 bytes
// of every row in turn, eight lanes a row, and has its next 128 in flight while
// it puts these together to MFMA operands, through LDS that no other wave
// uses: nothing waits for another wave before the int32 sums meet, exact in
// any order.  32 tokens x 8 of 64 experts, 4096 x 2048 (R = 1, C = 2, W = 4):
// 72 us where 50 experts get a token (419 MB, 5.8 TB/s), 85 where 63 do (6.2; reads
// alone reach 7.1), with ONCE, non-temporal loads of B where one row tile reads it
// (81 and 97 without).  Operands loaded as the MFMA wants them, sixteen rows of 64
// bytes an instruction, took a sixth longer (and half as long again non-temporal,
// which fetched each line twice), 64 x 4096 x 4096 so 12.1 against 9.4, and with
// unaligned rows three times as long.
template <int R, int C, bool ONCE>
struct ThinOps {
    static constexpr int kA = 2 * R, kB = 2 * C;
    static constexpr int kLds = 16 * (R + C) * kBigK;
    i32x4 v[kA + kB];
    // load j of this lane: row 8 j + l / 8 of A's, then of B's, 16 bytes at k + 16 (l % 8)
    __device__ __forceinline__ void read(const int8_t* const (&pa)[kA], const int8_t* const (&pb)[kB], int64_t k,
                                         int64_t K) {
#pragma unroll
        for (int j = 0; j < kB; ++j) v[kA + j] = ONCE ? load_any_once(pb[j], k, K) : load_any(pb[j], k, K);
#pragma unroll
        for (int j = 0; j < kA; ++j) v[j] = load_any(pa[j], k, K);
    }
    __device__ __forceinline__ void mask(int64_t k, int64_t K) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int32_t m = low_mask(k, K, d);
#pragma unroll
            for (int j = 0; j < kA; ++j) v[j][d] &= m;
        }
    }
    // The lanes of a wave read what others of them wrote.  A wave's LDS operations
    // are done in the order of its instructions, so no wait is needed, only that
    // the compiler keeps that order: the barriers emit nothing.
    __device__ __forceinline__ void multiply(i32x4 (&acc)[R][C], int8_t* lds, int l) const {
        __builtin_amdgcn_wave_barrier();  // the operands of the 128 bytes before have been read
#pragma unroll
        for (int j = 0; j < kA + kB; ++j) {
            const int r = 8 * j + (l >> 3);
            *reinterpret_cast<i32x4*>(lds + r * kBigK + (((l & 7) ^ big_swizzle(r)) << 4)) = v[j];
        }
        __builtin_amdgcn_wave_barrier();
        i32x4 x[2][R + C];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < R + C; ++j) {
                const int r = 16 * j + (l & 15);
                x[h][j] = *reinterpret_cast<const i32x4*>(lds + r * kBigK + (((4 * h + (l >> 4)) ^ big_swizzle(r)) << 4));
            }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < C; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[h][R + j], x[h][i], acc[i][j], 0, 0, 0);
    }
};

template <class D, int R, int C, int W, bool ONCE>
__global__ __launch_bounds__(64 * W) void gemm_i8_thin(GemmArgs g) {
    typedef typename D::T T;
    typedef ThinOps<R, C, ONCE> Ops;
    constexpr int BM = 16 * R, BN = 16 * C, LD = BN + 4;
    constexpr int kSums = BM * LD * 4, kWave = Ops::kLds > kSums ? Ops::kLds : kSums;
    __shared__ __attribute__((aligned(1024))) int8_t lds[W * kWave];
    int32_t* part = reinterpret_cast<int32_t*>(lds);
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    // the row tiles of one column tile follow each other: those of one expert meet its rows of B in one L2
    const uint32_t v = xcd_contiguous((int)blockIdx.x, 0, (int)gridDim.x);
    int e;
    int64_t lo, hi;
    if (!find_tile<BM>(g, v % g.m_tiles, l, e, lo, hi)) return;
    const int64_t n0 = (int64_t)(v / g.m_tiles) * BN;
    const int8_t *pa[Ops::kA], *pb[Ops::kB];
#pragma unroll
    for (int i = 0; i < Ops::kA; ++i) {
        const int64_t p = lo + 8 * i + (l >> 3);
        pa[i] = g.A + max(p < hi ? a_row(g, p) : -1, (int64_t)0) * g.lda;
    }
#pragma unroll
    for (int j = 0; j < Ops::kB; ++j) pb[j] = g.B + e * g.strideb + min(n0 + 8 * j + (l >> 3), g.N - 1) * g.ldb;

    i32x4 acc[R][C];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < C; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    const int lk = 16 * (l & 7);
    int8_t* const mine = lds + w * Ops::kLds;
    Ops x, y;
    int64_t k = 128 * w;
    x.read(pa, pb, k + lk, g.K);
    for (; k < g.K; k += 256 * W) {
        y.read(pa, pb, k + 128 * W + lk, g.K);
        if (k + 128 > g.K) x.mask(k + lk, g.K);
        x.multiply(acc, mine, l);
        if (k + 128 * W >= g.K) break;
        x.read(pa, pb, k + 256 * W + lk, g.K);
        if (k + 128 * W + 128 > g.K) y.mask(k + 128 * W + lk, g.K);
        y.multiply(acc, mine, l);
    }
    __syncthreads();  // the sums take the same LDS
    // D layout of the 16 x 16 MFMA: lane l, register r -> first operand's row 4 (l/16) + r (a column of C),
    // second operand's row l%16 (a row of C)
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < C; ++j)
            *reinterpret_cast<i32x4*>(part + (w * BM + 16 * i + (l & 15)) * LD + 16 * j + 4 * (l >> 4)) = acc[i][j];
    __syncthreads();
    for (int x4 = tid; x4 < BM * BN / 4; x4 += 64 * W) {
        const int row = x4 / (BN / 4), col = x4 % (BN / 4) * 4;
        const int64_t p = lo + row, n = n0 + col;
        if (p >= hi || n >= g.N) continue;
        const int64_t ra = a_row(g, p);
        if (ra < 0) continue;
        i32x4 sum = {0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < W; ++u) sum += *reinterpret_cast<const i32x4*>(part + (u * BM + row) * LD + col);
        const float sa = g.a_scale[ra];
        const float* sb = g.b_scale + e * g.N + n;
        T* c = (T*)g.C + p * g.ldc + n;
        typedef T V4 __attribute__((ext_vector_type(4), aligned(sizeof(T))));
        const auto out = [&](auto far) {
            if (n + 4 <= g.N) {
                V4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = scaled<D, far.value>(sum[i], sa, sb[i]);
                *reinterpret_cast<V4*>(c) = o;
            } else {
                for (int i = 0; i < 3; ++i)
                    if (n + i < g.N) c[i] = scaled<D, far.value>(sum[i], sa, sb[i]);
            }
        };
        if (__any(far_scale(sa)))
            out(std::true_type());
        else
            out(std::false_type());
    }
}

// ---------------------------------------------------------------- launch
bool aligned16(const GemmArgs& g) {
    return ((uintptr_t)g.A | (uintptr_t)g.B | (uintptr_t)g.lda | (uintptr_t)g.ldb |
            (uintptr_t)(g.E > 1 ? g.strideb : 0)) % 16 == 0;
}

// Tile counts of a launch with bm x bn tiles (an upper bound on the row tiles
// when the offsets are on the device).
int64_t row_tiles(const GemmArgs& g, int64_t bm) {
    return g.offsets ? g.S / bm + std::min<int64_t>(g.E, g.S) : (g.S + bm - 1) / bm;
}
int64_t tiles(const GemmArgs& g, int64_t bm, int64_t bn) { return row_tiles(g, bm) * ((g.N + bn - 1) / bn); }

// Workgroups of a launch: all kernels but gemm_i8_staged take one tile each and
// are not launched with more; that one goes on to the next.
constexpr int64_t kMostTiles = 1 << 22;

template <class K>
int launch(K kernel, GemmArgs g, int64_t bm, int64_t bn, int threads, hipStream_t s) {
    const int64_t n = tiles(g, bm, bn);
    if (n >= (int64_t)1 << 31) return SP_ERR_SIZE;
    g.m_tiles = (uint32_t)row_tiles(g, bm);
    g.n_tiles = (uint32_t)((g.N + bn - 1) / bn);
    hipLaunchKernelGGL(kernel, dim3((unsigned)std::min(n, kMostTiles)), dim3(threads), 0, s, g);
    return hipGetLastError() == hipSuccess ? SP_OK : SP_ERR_HIP;
}

template <class D, int R, int C, int W>
int launch_thin(bool once, const GemmArgs& g, hipStream_t s) {
    return once ? launch(gemm_i8_thin<D, R, C, W, true>, g, 16 * R, 16 * C, 64 * W, s)
                : launch(gemm_i8_thin<D, R, C, W, false>, g, 16 * R, 16 * C, 64 * W, s);
}

// Which kernel.  Times are medians in us, M x N x K, or tokens x choices, experts,
// K, N, of calls that follow each other in a graph, on normally distributed codes,
// with 1 GB of weights in turn, so that they come from memory.  Routing is uneven
// (scores favour experts with a standard deviation of 0.7, the scores' own being
// 1) unless it says even (no favour): uneven routing leaves some experts unused
// where there are few tokens, and makes the tiles of the others higher.
template <class D>
int gemm_t(GemmArgs g, hipStream_t s) {
    if (g.a_rows == 0) return SP_OK;  // no row of C has a row of A
    const int64_t groups = g.offsets ? std::min<int64_t>(g.E, g.S) : 1;
    const int64_t mid = tiles(g, 128, 128);
    const bool any = !aligned16(g);
    if (g.K < 16 || mid > kMostTiles) return launch(gemm_i8_staged<D>, g, 128, 128, 256, s);
    const bool few = tiles(g, 16, 32) <= kMostTiles;
    const bool matrix = few && groups == 1, experts = few && groups > 1 && !any;
    const bool deep = g.K > 2048;
    // Up to 32 rows a matrix: B's rows are (nearly all) read by one row tile,
    // and non-temporal.  32 x 8, 64, 4096, 2048 72 against 81 otherwise; 160 x 8
    // (20 rows) 114, 119; 512 x 8 (64 rows) 144, 129; 64 x 2048 x 2048 5.5, 5.0.
    // Not where unaligned pieces share lines: 96 x 8, 64, 4095, 2048 181, 152.
    const bool once = !any && g.S <= 32 * groups;
    // Few tiles: the smallest ones, or most CUs stay idle.  A step up where 128
    // or 256 tiles are reached: 1 x 4096 x 4096 16x16 5.8, 16x32 7.4;
    // 8 x 8192 x 4096 16x16 9.7, 16x32 9.4; 32 x 4096 x 4096 16x32 8.4,
    // 32x32 9.2; 64 x 4096 x 4096 16x32 10.3, 32x32 9.4, 32x64 11.7;
    // 128 x 4096 x 4096 32x32 12.4, 32x64 11.5, 128x128 23.4;
    // 300 x 4096 x 1024 32x32 9.6, 32x64 13.9, 128x128 9.2.
    //
    // Few rows a matrix take them in any number.  One matrix: 16 rows 16x32
    // (16 x 14336 x 4096 14.7, 32x64 15.3, 128x128 19.9), 32 rows 32x64
    // (32 x 14336 x 4096 15.9, 32x32 16.5, 128x128 21.2).  Experts: up to 8 rows
    // on the average, where some have more, 16x32 (32 x 8, 64, 4096, 2048 72,
    // 32x32 77, 128x128 102; 64 x 8 91, 92, 113), up to 16 rows 32x32 (128 x 8
    // 104, 16x32 117, 128x128 115; 160 x 8 (20 rows) 116, 136, 114, but even 106,
    // 145, 121).  Shorter sums do not pay their four waves as long: 96 x 8, 128,
    // 2048, 2048 (6 rows) 16x32 83, 128x128 88; 128 x 8 (8 rows) 92, 91, but even
    // 98, 106; 17 x 28672 x 2048 32x64 16.5, 128x128 14.2.
    if (tiles(g, 16, 32) <= 128) return launch_thin<D, 1, 1, 8>(once, g, s);
    if (tiles(g, 16, 32) <= 256 || (matrix && g.S <= 16) || (experts && g.S <= (deep ? 8 : 6) * groups))
        return launch_thin<D, 1, 2, 4>(once, g, s);
    if (tiles(g, 32, 32) <= 256 || (experts && g.S <= 16 * groups && deep))
        return launch_thin<D, 2, 2, 4>(once, g, s);
    // Unaligned rows, whose 128 x 128 tiles are slower, up to 512 tiles:
    // 256 x 4096 x 4097 32, 128x128 54; 1024 x 1024 x 1023 13.1, 15.1.
    if (tiles(g, 32, 64) <= (any ? 512 : 256) || (matrix && g.S <= 32 && deep))
        return launch_thin<D, 2, 4, 4>(once, g, s);
    // 8192 x 8192 x 4095 474, with aligned rows 250; 32 x 8, 64, 4095, 2048 119
    // (thin tiles 107), 96 x 8 134 (152), 24 x 8, 128, 1023, 2047 52 (55).
    if (any) return launch(gemm_i8_staged<D>, g, 128, 128, 256, s);
    // One 128 x 128 tile a CU at most, or tiles that mostly wait for memory: four
    // steps in LDS.  1024 x 4096 x 4096 24 against 35 with two steps and two
    // workgroups a CU, and 55 with 256 x 256 tiles; 512 x 8, 64, 4096, 2048 (64
    // rows) 129, 162, 159; 1024 x 8 (128 rows) 159, 199, 182; 1024 x 2, 8, 4096,
    // 14336 (256 rows) 222, 228, 187; 512 x 2 (128 rows) 151, 163, 170, but even
    // 165, 163, 138; shorter sums 512 x 8, 128, 2048, 1536 (32 rows) 90, 93, 94;
    // 2048 x 8 (128 rows) 144, 144, 130.
    if (once) return launch(gemm_i8_big<D, 2, 4, true>, g, 128, 128, 256, s);
    if (mid <= 256 || (few && g.S <= (deep ? 128 : 64) * groups))
        return launch(gemm_i8_big<D, 2, 4, false>, g, 128, 128, 256, s);
    // Up to two 128 x 128 tiles a CU: 2048 x 4096 x 4096 43, with four steps 47,
    // with 256 x 256 tiles 57.  Also where 256-wide tiles would be empty for a
    // fifth: 20000 x 2, 16, 512, 300 25, with 256 x 256 33.
    const int64_t wide = (g.N + 255) / 256 * 256, narrow = (g.N + 127) / 128 * 128;
    if (mid <= 512 || (few && 5 * wide >= 6 * narrow))
        return launch(gemm_i8_big<D, 2, 2, false>, g, 128, 128, 256, s);
    // 8192 x 8192 x 4096 250 against 313 with 128 x 128 tiles; 4096 x 4096 x 4096
    // 68, 82; 4096 x 8, 64, 4096, 2048 (512 rows) 341, even 335 against 415.
    return launch(gemm_i8_big<D, 4, 2, false>, g, 256, 256, 512, s);
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
