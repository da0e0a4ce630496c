// Tiles of products over rows that are sorted by expert, shared by the 8-bit
// (gemm_i8.hip) and 16-bit products (gemm_16.hip):
//   C[p, n] = sum_k A[r, k] B[e, n, k]
// where p runs over the sorted rows, e is the expert whose range offsets[e] ..
// offsets[e + 1] holds p, and r is p, or the token src[p] / slots.  A gated product
// has matrices of 2 N rows, gate rows before up rows, and gives
//   C[p, n] = a(sum_k A[r, k] B[e, n, k]) sum_k A[r, k] B[e, N + n, k]
// Lengths and distances of operand rows are in bytes here, whatever their type:
// 16 bytes of K are an MFMA operand of a lane in 8 and in 16 bits.
#pragma once

#include <algorithm>
#include <type_traits>

#include "act.h"
#include "device_common.h"
#include "moe.h"
#include "rows.h"

namespace spx {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int32_t i32x4_u __attribute__((ext_vector_type(4), aligned(1)));

// What the operands hold: the sums' type and the MFMAs, first operand times second.
// The 32-wide one takes 32 bytes of K (lane l: row l % 32, bytes 16 (l / 32)), the
// 16-wide one 64 (row l % 16, bytes 16 (l / 16)).
struct KindI8 {
    static constexpr bool kFloat = false;
    typedef int32_t S;
    typedef i32x4 S4;
    typedef i32x16 S16;
    static __device__ __forceinline__ S16 mfma32(i32x4 a, i32x4 b, S16 c) {
        return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ S4 mfma16(i32x4 a, i32x4 b, S4 c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
    }
};
struct KindBf16 {
    static constexpr bool kFloat = true;
    typedef __bf16 V __attribute__((ext_vector_type(8)));
    typedef float S;
    typedef f32x4 S4;
    typedef f32x16 S16;
    static __device__ __forceinline__ S16 mfma32(i32x4 a, i32x4 b, S16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ S4 mfma16(i32x4 a, i32x4 b, S4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b), c, 0, 0, 0);
    }
};
struct KindF16 {
    static constexpr bool kFloat = true;
    typedef _Float16 V __attribute__((ext_vector_type(8)));
    typedef float S;
    typedef f32x4 S4;
    typedef f32x16 S16;
    static __device__ __forceinline__ S16 mfma32(i32x4 a, i32x4 b, S16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ S4 mfma16(i32x4 a, i32x4 b, S4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b), c, 0, 0, 0);
    }
};

struct GemmArgs {
    int64_t S, N, K;          // rows of C, columns of C, bytes of a row of A (and of B, where its rows are columns of C)
    const int8_t* A;
    int64_t a_rows, lda;
    const float* a_scale;     // int8 only, as b_scale
    const int32_t* src;       // or NULL: row p of C reads row p of A
    int32_t slots;
    const int8_t* B;          // [E][rows], rows ldb apart, experts strideb apart
    int64_t ldb, strideb;
    const float* b_scale;     // [E][rows]
    const int32_t* offsets;   // or NULL: one matrix, rows 0 .. S
    int32_t E;
    void* C;
    int64_t ldc;
    void* pre;                // gated: what the activation and the product take (S x 2 N), or NULL
    int64_t ldp;
    int32_t act;
    uint32_t m_tiles, n_tiles; // m_tiles is an upper bound when offsets are given; the product fits 31 bits
    float* part;              // the sums of a part of K each: [splits][S][N], or NULL
    int32_t splits;
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
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int E, int64_t S, int e, int& a, int& b) {
    a = b = 0;
    if (e < E) {
        a = min(max(offsets[e], 0), (int)S);
        b = max(a, min(max(offsets[e + 1], 0), (int)S));
    }
}
__device__ __forceinline__ void expert_rows(const GemmArgs& g, int e, int& a, int& b) {
    expert_rows(g.offsets, g.E, g.S, e, a, b);
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
// than 32 bits count: the bound keeps the loop of gemm_staged below 2^31.
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
#pragma clang fp contract(off)
    if (FAR && far_scale(sa)) return round_alone<D>((float)sum * (sa * 0x1p-32f) * sb * 0x1p32f);
    return round_alone<D>((float)sum * sa * sb);
}

// The bytes of v from byte n (0 .. 16) on, zeros behind them.
__device__ __forceinline__ i32x4 shift_down(i32x4 v, int n) {
    typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
    u64x2 x = __builtin_bit_cast(u64x2, v);
    if (n >= 8) x = u64x2{x[1], 0};
    const int bits = 8 * (n >= 8 ? n - 8 : n);
    const uint64_t carry = bits ? x[1] << (64 - bits & 63) : 0;
    x = bits >= 64 ? u64x2{0, 0} : u64x2{x[0] >> bits | carry, x[1] >> bits};
    return __builtin_bit_cast(i32x4, x);
}

// Column i of a tile's rows of B: row of B's matrix.  Gated: blocks of 32 gate rows and the 32 up rows of the
// same columns of C in turn.
template <bool GATED>
__device__ __forceinline__ int64_t b_row(const GemmArgs& g, int64_t n0, int i) {
    if (!GATED) return min(n0 + i, g.N - 1);
    return ((i >> 5) & 1) * g.N + min(n0 + (i >> 6) * 32 + (i & 31), g.N - 1);
}

// ---------------------------------------------------------------------------
// Many rows: tiles of up to 64 CB rows x 64 CB columns by W waves, CB = 4
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
// Operands whose rows are steps of the sum (gradients; 16 bits only) are
// transposed on their way to the matrix cores: LDS holds 64 rows of 64 CB columns,
// and ds_read_b64_tr_b16 gives a lane four rows of one column.  Their blocks of 32
// columns (64 bytes) lie at block ^ (row % 4), so that the four rows that half a
// wave reads at once lie in different banks.
//
// Wave (wm, wn) owns columns 32 U wn .. 32 U (wn + 1) - 1 and every second 32-row
// block: rows 32 (2 i + wm), i < F.  F = 1 .. CB is the tile's height in units
// of 64 rows: a short tile (an expert's last) runs fewer MFMAs and loads fewer
// rows, instead of multiplying rows nobody stores.  An expert's rows are cut
// into tiles of equal height rather than full ones and a rest.
//
// B is the first MFMA operand, so that a lane's four consecutive sums lie in
// one row of C; the sums go through LDS once more to be stored as whole lines.
// In a gated product 64 of a wave's columns are 32 of the gate and the same 32 of the
// other projection: both meet in its own part of LDS.
constexpr int kBigK = 128;            // bytes of K a step
constexpr int kBigRow = 64 + 4;       // LDS words per row of a wave's sums

typedef __attribute__((address_space(3))) void lds_void;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) const int8_t lds_int8;

__device__ __forceinline__ int big_swizzle(int row) { return (row >> 1) & 7; }

// What global_load_lds reads for rows that are not there.
static __device__ __attribute__((aligned(16))) int8_t big_zeros[16];

// A tile's shape: 64 CB columns, W waves, U 32-column blocks a wave.
template <int CB_, int W_>
struct Tile {
    static constexpr int CB = CB_, W = W_, U = 4 * CB / W, kSize = 64 * CB, kThreads = 64 * W;
    static constexpr int kCopied = kSize / (8 * W);  // copies of a wave for as many rows as the tile has columns
};
typedef Tile<2, 4> Tile128;
typedef Tile<4, 8> Tile256;

// Copy instructions a wave issues for a step: 1024 W bytes each over the workgroup.
template <class X, int F>
struct BigShape {
    static constexpr int kRows = 8 * X::W;           // rows of K-contiguous operands that one instruction of every wave covers
    static constexpr int kA = 64 * F / kRows;        // for the rows of A
    static constexpr int kB = X::kSize / kRows;      // for the rows of B
    static constexpr int kCopies = kA + kB;
};

// Where a lane's copy j of a step reads a K-contiguous operand.
template <class X>
struct BigDirect {
    static constexpr bool kGather = false;
    const int8_t* p[X::kCopied];
    int64_t chunk, last, K;  // chunks behind the last are read from there and masked
    __device__ __forceinline__ void fetch(int) {}
    __device__ __forceinline__ const int8_t* at(int j, int step) const {
        return p[j % X::kCopied] + min((int64_t)step * kBigK + chunk, last);
    }
    // Rows of any alignment, K >= 16 (SHORT: of any length): load(), and then finish() what it gave.  The last piece of
    // a row that K cuts begins with bytes that the piece before holds: zeroed, or with ALONE, where the other operand does not
    // begin with the same, moved to where they belong.
    template <bool SHORT>
    __device__ __forceinline__ i32x4 load(int j, int step) const {
        const int64_t k = (int64_t)step * kBigK + chunk;
        return SHORT && K < 16 ? load_short(p[j % X::kCopied], k, K) : load_any(p[j % X::kCopied], k, K);
    }
    template <bool SHORT, bool ALONE>
    __device__ __forceinline__ i32x4 finish(i32x4 v, int step, bool last_step) const {
        if (!last_step || (SHORT && K < 16)) return v;
        const int64_t k = (int64_t)step * kBigK + chunk;
        if (ALONE) return shift_down(v, (int)min(max(k - (K - 16), (int64_t)0), (int64_t)16));
#pragma unroll
        for (int d = 0; d < 4; ++d) v[d] &= low_mask(k, K, d);
        return v;
    }
    __device__ __forceinline__ bool is_short() const { return K < 16; }
};

// n / d for 0 <= n < 2^31 as (n * m) >> 32 >> s with m = floor(2^(32 + s) / d) + 1 and 2^s < d <= 2^(s + 1):
// m d exceeds 2^(32 + s) by at most d <= 2^(s + 1), so that the product exceeds n / d by less than (n / 2^31) / d < 1 / d.
// d = 1: (2 n * 2^31) >> 32.
struct FastDiv {
    uint32_t m, s, one;
    static FastDiv by(int32_t d) {
        FastDiv f{1u << 31, 0, 1};
        if (d == 1) return f;
        f.one = 0;
        while ((2ll << f.s) < d) ++f.s;
        f.m = (uint32_t)(((1ull << (32 + f.s)) / (uint32_t)d) + 1);
        return f;
    }
    __device__ __forceinline__ int32_t operator()(int32_t n) const { return (int32_t)(__umulhi((uint32_t)n << one, m) >> s); }
};

// Where a lane's copy j of a step reads an operand whose rows are steps of the sum.  GATHER: row i of the sum is the
// row of slot src[i]; the sources of a step are read ahead of its copies (fetch), with scalar loads, which do not queue
// behind the copies in flight.
template <class X, bool GATHER>
struct BigTransposed {
    static constexpr bool kGather = GATHER;
    static constexpr int kWave = 8 / X::CB, kAll = X::W * kWave;  // rows of one copy of a wave, of all waves
    const int8_t* base;          // the lane's chunk in its row of copy 0 (GATHER: in row 0)
    const int8_t* zeros;         // read for rows that are not there
    int64_t ld;
    int rows, row0;              // rows of the sum; the lane's row of copy 0
    int cols;                    // load: elements from the lane's chunk to the row's end, 8 at most
    bool inside, narrow;         // load: all the tile's chunks are whole; rows shorter than a chunk
    int w;                       // GATHER only, as what follows
    const int32_t* src;          // the rows' slots (readable where there are no rows too)
    FastDiv slots;
    uint32_t sources;            // slots of the rows that there are, 2^31 at most
    int32_t f[GATHER ? X::kCopied : 1][kWave];  // sources of the step fetched last
    mutable const int8_t* found[GATHER ? X::kCopied : 1];  // where copy j reads, left by find() for at()
    // first: row 0; width: the rows' elements; n0: the tile's first column; STAGED: for load(), else for at()
    template <bool STAGED>
    __device__ __forceinline__ void place(const int8_t* first, int64_t ld_, int rows_, int64_t n0, int64_t width, int w_,
                                          int l) {
        constexpr int kChunks = 8 * X::CB;
        w = w_;
        row0 = w * kWave + l / kChunks;
        const int chunk = (l % kChunks) ^ (4 * (row0 & 3));
        cols = (int)max(min(width - n0 - chunk * 8, (int64_t)8), (int64_t)0);
        inside = n0 + X::kSize <= width;
        narrow = width < 8;
        const int64_t at = 2 * n0 + 16 * chunk;
        base = first + (STAGED ? at : min(at, (2 * width - 1) & ~(int64_t)15)) + (GATHER ? 0 : row0 * ld_);
        zeros = big_zeros;
        ld = ld_;
        rows = rows_;
    }
    __device__ __forceinline__ void fetch(int step) {
        if constexpr (GATHER) {
            const __attribute__((address_space(4))) int32_t* s = (const __attribute__((address_space(4))) int32_t*)src;
#pragma unroll
            for (int j = 0; j < X::kCopied; ++j)
#pragma unroll
                for (int i = 0; i < kWave; ++i) {
                    const int at = step * 64 + kAll * j + w * kWave + i;
                    f[j][i] = s[max(min(at, rows - 1), 0)];
                }
        }
    }
    // The lane's chunk of its row of copy j, or `none` where there is no such row.  Distances from row to row are the same
    // for all lanes, and so is whether all rows of a copy are there.
    __device__ __forceinline__ const int8_t* row(int j, int step, const int8_t* none) const {
        const int u = step * 64 + kAll * j;
        if constexpr (!GATHER) {
            const int8_t* p = base + (int64_t)u * ld;
            return u + row0 < rows ? p : none;
        } else {
            const int mine = row0 - w * kWave;
            const int8_t* p = none;
#pragma unroll
            for (int i = 0; i < kWave; ++i) {
                const int at = u + w * kWave + i, t = slots(f[j][i] & 0x7fffffff);
                // the same for all lanes
                const bool there = (uint32_t)f[j][i] < sources && at < rows;
                const int8_t* q = reinterpret_cast<const int8_t*>(reinterpret_cast<uintptr_t>(base) + (uint64_t)(uint32_t)t * (uint64_t)ld);
                p = mine == i && there ? q : p;
            }
            return p;
        }
    }
    // Whether the lane's row of copy j of the step fetched last has a source: a mask of lanes, made by scalar instructions.
    __device__ __forceinline__ bool sourced(int j) const {
        constexpr uint64_t kRow = ~0ull >> (64 - 64 / kWave);  // the lanes of a row
        uint64_t lanes = 0;
#pragma unroll
        for (int i = 0; i < kWave; ++i) lanes |= (uint32_t)f[j][i] < sources ? kRow << (i * (64 / kWave)) : 0;
        return __builtin_amdgcn_inverse_ballot_w64(lanes);
    }
    // Finds where copy j reads, and says whether the lane's row is there.
    __device__ __forceinline__ bool find(int j, int step) const {
        found[j] = row(j, step, zeros);
        return found[j] != zeros;
    }
    __device__ __forceinline__ const int8_t* at(int j, int step) const { return GATHER ? found[j] : row(j, step, zeros); }
    // A chunk that the row's end cuts is loaded with the elements before it and moved down; rows shorter than a chunk
    // (SHORT) go element by element.  there: false for a row that counts as zeros.
    template <bool SHORT>
    __device__ __forceinline__ i32x4 load(int j, int step, bool there = true) const {
        if (SHORT && narrow) {
            const int8_t* p = there ? row(j, step, nullptr) : nullptr;
            i32x4 v = {0, 0, 0, 0};
            for (int i = 0; i < 7; ++i)
                if (p && i < cols) v[i >> 1] |= (int32_t)((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1)));
            return v;
        }
        const int8_t* p = there ? row(j, step, zeros) : zeros;
        return *reinterpret_cast<const i32x4_u*>(cols == 0 ? zeros : p == zeros ? p : p + (2 * cols - 16));
    }
    template <bool SHORT, bool>
    __device__ __forceinline__ i32x4 finish(i32x4 v, int, bool) const {
        return inside || (SHORT && narrow) ? v : shift_down(v, 16 - 2 * cols);
    }
    __device__ __forceinline__ bool is_short() const { return narrow; }
};

// The same of rows that go with another operand's rows, and count as zeros where those have no source.  A step's copies of
// these come after its fetch, and before its copies of the other's, whose places they find (once for both: a test of each
// source on its own cost a tenth of a short sum's time, 777 x 3 of 7 experts, 1112 x 512 bf16 20.0 us against 18.5).
template <class X>
struct BigPartner {
    BigTransposed<X, false> mine;
    const BigTransposed<X, true>& other;
    __device__ __forceinline__ const int8_t* at(int j, int step) const {
        const int8_t* p = mine.at(j, step);
        return other.find(j, step) ? p : mine.zeros;
    }
    template <bool SHORT>
    __device__ __forceinline__ i32x4 load(int j, int step) const {
        return mine.template load<SHORT>(j, step, other.sourced(j));
    }
    template <bool SHORT, bool ALONE>
    __device__ __forceinline__ i32x4 finish(i32x4 v, int step, bool last) const {
        return mine.template finish<SHORT, ALONE>(v, step, last);
    }
    __device__ __forceinline__ bool is_short() const { return mine.is_short(); }
};

// Copies [FROM, TO) of the step's, in the order A, B.  ONCE: no other tile reads these rows of B.
template <class X, int F, bool ONCE, int FROM, int TO, class SA, class SB>
__device__ __forceinline__ void big_copy(int8_t* la, int8_t* lb, const SA& sa, const SB& sb, int step, int w) {
    using S = BigShape<X, F>;
#pragma unroll
    for (int j = FROM; j < TO; ++j) {
        const int8_t* src = j < S::kA ? sa.at(j, step) : sb.at(j - S::kA, step);
        int8_t* dst = (j < S::kA ? la + j * S::kRows * kBigK : lb + (j - S::kA) * S::kRows * kBigK) + w * 1024;
        if (ONCE && j >= S::kA)
            __builtin_amdgcn_global_load_lds((const void*)src, (lds_void*)dst, 16, 0, 2);  // non-temporal
        else
            __builtin_amdgcn_global_load_lds((const void*)src, (lds_void*)dst, 16, 0, 0);
    }
}

// An MFMA operand of 32 rows (block) and 32 bytes of K: piece ks of a step.
template <class X, bool T>
__device__ __forceinline__ i32x4 big_operand(const int8_t* lds, int block, int ks, int l) {
    if constexpr (!T) {
        const int r = l & 31;
        return *reinterpret_cast<const i32x4*>(lds + (32 * block + r) * kBigK + (((2 * ks + (l >> 5)) ^ big_swizzle(r)) << 4));
    } else {
        // lanes 16 q + 4 i + c name row i, columns 4 c .. 4 c + 3 of their 16; lane 16 q + i gets column i of the four rows
        int at = (8 * (l >> 5) + ((l >> 2) & 3)) * (2 * X::kSize) + ((block ^ ((l >> 2) & 3)) << 6) + 32 * ((l >> 4) & 1) +
                 8 * (l & 3);
        // One number for the compiler: an address few steps from the buffer's tells it which buffer is read.  Built from the
        // terms above it loses track, and makes the read wait for the copies into all buffers.
        asm("" : "+v"(at));
        lds_int8* const from = (lds_int8*)lds + at;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(from + 16 * ks * (2 * X::kSize)));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(from + (16 * ks + 4) * (2 * X::kSize)));
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        return __builtin_bit_cast(i32x4, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
}

// MFMA operands of 32 bytes of K.  TA, TB: rows of A, of B are steps of the sum.
template <class Kind, class X, int F, bool TA, bool TB>
struct BigOps {
    typedef typename Kind::S16 S16;
    i32x4 a[F], b[X::U];
    __device__ __forceinline__ void read(const int8_t* la, const int8_t* lb, int ks, int wm, int wn, int l) {
#pragma unroll
        for (int u = 0; u < X::U; ++u) b[u] = big_operand<X, TB>(lb, X::U * wn + u, ks, l);
#pragma unroll
        for (int i = 0; i < F; ++i) a[i] = big_operand<X, TA>(la, 2 * i + wm, ks, l);
    }
    __device__ __forceinline__ void multiply(S16 (&acc)[F][X::U], int i0 = 0, int i1 = F) const {
#pragma unroll
        for (int i = 0; i < F; ++i)
            if (i >= i0 && i < i1)
#pragma unroll
                for (int u = 0; u < X::U; ++u) acc[i][u] = Kind::mfma32(b[u], a[i], acc[i][u]);
    }
    // The same with copies [FROM, TO) of a later step spread between the MFMAs:
    // a wave that issues them in one go waits for the memory pipeline to take them.
    template <bool ONCE, int FROM, int TO, int I = 0, class SA, class SB>
    __device__ __forceinline__ void multiply_and_copy(S16 (&acc)[F][X::U], int8_t* la, int8_t* lb, const SA& sa, const SB& sb,
                                                      int step, int w) const {
        constexpr int N = TO - FROM;
        big_copy<X, F, ONCE, FROM + (N * I + F - 1) / F, FROM + (N * (I + 1) + F - 1) / F>(la, lb, sa, sb, step, w);
        multiply(acc, I, I + 1);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (I + 1 < F) multiply_and_copy<ONCE, FROM, TO, I + 1>(acc, la, lb, sa, sb, step, w);
    }
};

// Waits for the operand reads in flight.  Placed before the next reads are
// issued: left to the compiler, the wait comes after them and takes them in.
__device__ __forceinline__ void big_operands_here() {
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt 0, the others untouched
    __builtin_amdgcn_sched_barrier(0);
}

// Zeroes the bytes from K on in the last step's `rows` rows of a K-contiguous operand.
__device__ __forceinline__ void big_mask(int8_t* lds, int rows, int left, int tid, int threads) {
    for (int i = tid; i < rows * 8; i += threads) {
        const int row = i >> 3, k = ((i & 7) ^ big_swizzle(row)) << 4;
        if (k + 16 <= left) continue;
        i32x4* at = reinterpret_cast<i32x4*>(lds + i * 16);
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

template <class S16, int F, int U>
__device__ __forceinline__ void big_clear(S16 (&acc)[F][U]) {
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][u][r] = 0;
}

// The sums of a tile over `steps` steps, copies straight to LDS.  left: bytes of the last step that a
// K-contiguous operand has.  In 8 bits only A's are masked, what B holds there is then multiplied by zero;
// in floating point that could be an Inf or a NaN, and both are.
//
// The operands of piece ks + 1 are read while the MFMAs of piece ks run.  The
// barrier that ends a step stands before its last piece's MFMAs, when all of
// the step's operands are in registers: its buffer then takes the copies of
// step s + ST, half of them under those MFMAs and half under the next
// piece's.  Before the barrier a wave waits for its own copies of step s + 1;
// those of ST - 2 later steps stay in flight.  Copies behind the last step
// read its last chunk again (or zeros), which keeps the counts the same.
template <class Kind, class X, int ST, int F, bool TA, bool TB, bool ONCE, class SA, class SB>
__device__ __forceinline__ void big_sums(typename Kind::S16 (&acc)[F][X::U], const BigBuffers<ST>& m, const SA& sa, SB& sb,
                                         int steps, int left, int tid, int w, int l) {
    using S = BigShape<X, F>;
    const int wm = w & 1, wn = w >> 1;
    big_clear(acc);
    const auto mask = [&](int8_t* la, int8_t* lb) {
        if (!TA) big_mask(la, 64 * F, left, tid, X::kThreads);
        if (Kind::kFloat && !TB) big_mask(lb, X::kSize, left, tid, X::kThreads);
    };
    BigOps<Kind, X, F, TA, TB> x0, x1;
    constexpr int kCopies = S::kCopies, kHalf = kCopies / 2;
    if constexpr (SB::kGather) {
        SB last = sb;
        last.fetch(ST - 1);  // with the first step's: one wait for both
        sb.fetch(0);
        big_copy<X, F, ONCE, 0, kCopies>(m.a[0], m.b[0], sa, sb, 0, w);
        sb = last;
        static_assert(ST == 2, "sources are fetched for two steps");
    } else {
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) big_copy<X, F, ONCE, 0, kCopies>(m.a[i], m.b[i], sa, sb, i, w);
    }
    big_copy<X, F, ONCE, 0, kHalf>(m.a[ST - 1], m.b[ST - 1], sa, sb, ST - 1, w);
    big_barrier<(ST - 2) * kCopies + kHalf>();
    if (steps == 1 && left < kBigK) {
        mask(m.a[0], m.b[0]);
        big_barrier<(ST - 2) * kCopies + kHalf>();
    }
    x0.read(m.a[0], m.b[0], 0, wm, wn, l);
#define SPX_STEP(s, I)                                                                                    \
    {                                                                                                     \
        constexpr int kNext = ((I) + 1) % ST, kBack = ((I) + ST - 1) % ST;                                \
        big_operands_here();                                                                              \
        x1.read(m.a[I], m.b[I], 1, wm, wn, l);                                                            \
        __builtin_amdgcn_sched_barrier(0);                                                                \
        x0.template multiply_and_copy<ONCE, kHalf, kCopies>(acc, m.a[kBack], m.b[kBack], sa, sb, (s) + ST - 1, w); \
        sb.fetch((s) + ST);                                                                               \
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
            mask(m.a[kNext], m.b[kNext]);                                                                 \
            big_barrier<(ST - 2) * kCopies>();                                                            \
        }                                                                                                 \
        x0.read(m.a[kNext], m.b[kNext], 0, wm, wn, l);                                                    \
        __builtin_amdgcn_sched_barrier(0);                                                                \
        x1.template multiply_and_copy<ONCE, 0, kHalf>(acc, m.a[I], m.b[I], sa, sb, (s) + ST, w);          \
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
    big_barrier<0>();  // the copies behind the last step have landed too: the sums take their LDS
}

// The same for rows of any alignment and length, with the copies through registers
// (global_load_lds wants aligned pieces): the loads of the next steps are in flight while a step is multiplied, after
// which the oldest go to the other LDS buffer.  Two steps ahead in 16 bits, where a step alone takes a quarter of a load's
// latency (dA of 1024 x 1000 x 1001 bf16 23 us, one ahead 47; three would not fit the registers); one in 8 bits
// (8192 x 8192 x 4095 474, two ahead 485).
template <class Kind, int F, bool TA, bool TB, bool SHORT, class SA, class SB>
__device__ __forceinline__ void staged_loop(typename Kind::S16 (&acc)[F][2], const BigBuffers<2>& m, const SA& sa, SB& sb,
                                            int steps, int w, int l) {
    using S = BigShape<Tile128, F>;
    constexpr int D = SHORT || !Kind::kFloat ? 1 : 2;
    const int wm = w & 1, wn = w >> 1;
    i32x4 v[D][S::kCopies];
    const auto load = [&](i32x4 (&x)[S::kCopies], int s) {
        sb.fetch(s);
#pragma unroll
        for (int j = 0; j < S::kCopies; ++j)
            x[j] = j < S::kA ? sa.template load<SHORT>(j, s) : sb.template load<SHORT>(j - S::kA, s);
    };
    const auto store = [&](const i32x4 (&x)[S::kCopies], int s) {
        int8_t* la = (s & 1 ? m.a[1] : m.a[0]) + w * 1024 + l * 16;
        int8_t* lb = (s & 1 ? m.b[1] : m.b[0]) + w * 1024 + l * 16;
        const bool last = s == steps - 1;
#pragma unroll
        for (int j = 0; j < S::kCopies; ++j) {
            if (j < S::kA)
                *reinterpret_cast<i32x4*>(la + j * S::kRows * kBigK) = sa.template finish<SHORT, TB>(x[j], s, last);
            else
                *reinterpret_cast<i32x4*>(lb + (j - S::kA) * S::kRows * kBigK) =
                    sb.template finish<SHORT, TA>(x[j], s, Kind::kFloat && last);
        }
    };
    big_clear(acc);
    // steps behind the last are not loaded; set i holds steps i, i + D, ..
#pragma unroll
    for (int i = 0; i < D; ++i)
        if (i < steps) load(v[i], i);
    if (steps > 0) store(v[0], 0);
    __syncthreads();
    for (int s0 = 0; s0 < steps; s0 += D) {
#pragma unroll
        for (int i = 0; i < D; ++i) {
            const int s = s0 + i;
            if (s >= steps) break;
            if (s + D < steps) load(v[i], s + D);
            const int8_t* la = s & 1 ? m.a[1] : m.a[0];
            const int8_t* lb = s & 1 ? m.b[1] : m.b[0];
            BigOps<Kind, Tile128, F, TA, TB> x0, x1;
            x0.read(la, lb, 0, wm, wn, l);
#pragma unroll
            for (int ks = 0; ks < 4; ks += 2) {
                x1.read(la, lb, ks + 1, wm, wn, l);
                x0.multiply(acc);
                if (ks == 0) x0.read(la, lb, 2, wm, wn, l);
                x1.multiply(acc);
            }
            if (s + 1 < steps) store(v[(i + 1) % D], s + 1);
            __syncthreads();
        }
    }
}
template <class Kind, int F, bool TA, bool TB, class SA, class SB>
__device__ __forceinline__ void staged_sums(typename Kind::S16 (&acc)[F][2], const BigBuffers<2>& m, const SA& sa, SB& sb,
                                            int steps, int w, int l) {
    if (sa.is_short() || sb.is_short())
        staged_loop<Kind, F, TA, TB, true>(acc, m, sa, sb, steps, w, l);
    else
        staged_loop<Kind, F, TA, TB, false>(acc, m, sa, sb, steps, w, l);
}

// Where the copies of K-contiguous operands read: rows kRows j + 8 w + l / 8 of the tile, chunk
// (l % 8) ^ big_swizzle(row); the tile's rows of A (and scales) go to LDS, and behind
// the rows a word of each wave that says whether it met a far scale.
template <class Kind, class X, int F>
__device__ __forceinline__ void big_rows(const GemmArgs& g, int64_t lo, int64_t hi, int32_t* lrow, float* lscale,
                                         BigDirect<X>& a, int w, int l) {
    using S = BigShape<X, F>;
    const int crow = 8 * w + (l >> 3);
    a.chunk = ((l & 7) ^ big_swizzle(crow)) << 4;
    a.last = (g.K - 1) & ~(int64_t)15;
    a.K = g.K;
    bool far = false;
#pragma unroll
    for (int j = 0; j < X::kCopied; ++j) {
        const int row = S::kRows * j + crow;
        const int64_t p = lo + row;
        const int64_t r = j < S::kA && p < hi ? a_row(g, p) : -1;
        a.p[j] = g.A + max(r, (int64_t)0) * g.lda;  // a row that is not there copies row 0; its sums are not stored
        if (j < S::kA && (l & 7) == 0) {
            lrow[row] = (int32_t)r;
            if constexpr (!Kind::kFloat) {
                const float sa = g.a_scale[max(r, (int64_t)0)];
                lscale[row] = sa;
                far |= far_scale(sa);
            }
        }
    }
    if (!Kind::kFloat) lrow[X::kSize + w] = __any(far);
}
template <class Kind, class X, bool GATED>
__device__ __forceinline__ void big_columns(const GemmArgs& g, int e, int64_t n0, float* lscale, BigDirect<X>& b, int tid,
                                            int w, int l) {
    const int crow = 8 * w + (l >> 3);
    b.chunk = ((l & 7) ^ big_swizzle(crow)) << 4;
    b.last = (g.K - 1) & ~(int64_t)15;
    b.K = g.K;
#pragma unroll
    for (int j = 0; j < X::kCopied; ++j) b.p[j] = g.B + e * g.strideb + b_row<GATED>(g, n0, 8 * X::W * j + crow) * g.ldb;
    if constexpr (!Kind::kFloat) {
        for (int i = tid; i < X::kSize; i += X::kThreads)
            lscale[X::kSize + i] = g.b_scale[e * (GATED ? 2 * g.N : g.N) + b_row<GATED>(g, n0, i)];
    }
}

// Where a tile's sums go: rows lo .. of C (those whose lrow is not negative), columns n0 .. below N.
struct BigOut {
    void* C;
    int64_t ldc, N, lo, n0;
    void* pre;
    int64_t ldp;
    int act;
};
__device__ __forceinline__ BigOut big_out_of(const GemmArgs& g, int64_t lo, int64_t n0) {
    return BigOut{g.C, g.ldc, g.N, lo, n0, g.pre, g.ldp, g.act};
}

// The tile's sums scaled and stored; l0 .. l3 are LDS buffers of X::kSize x kBigK
// bytes that nothing uses any more.
template <class Kind, class D, class X, int F, bool GATED>
__device__ __forceinline__ void big_out(const BigOut& g, const typename Kind::S16 (&acc)[F][X::U], int8_t* l0, int8_t* l1,
                                        int8_t* l2, int8_t* l3, const int32_t* lrow, const float* lscale, int w, int l) {
    typedef typename D::T T;
    typedef typename Kind::S S;
    typedef typename Kind::S4 S4;
    const int wm = w & 1, wn = w >> 1;
    // Sums of one 32-row block at a time through this wave's part of LDS, then 8
    // consecutive columns a lane, 8 rows an instruction (gated: 8 columns of each
    // projection, 16 rows).  D layout of the 32 x 32 MFMA: lane l, register r ->
    // first operand's row 8 (r/4) + 4 (l/32) + r%4 (a column of C), second operand's
    // row l%32 (a row of C).
    constexpr int kSums = 32 * kBigRow, kPer = X::kSize * kBigK / (4 * kSums);  // waves to a buffer
    static_assert(4 * kPer >= X::W, "the waves' sums fit the four buffers");
    int8_t* const buffer = w / kPer == 0 ? l0 : w / kPer == 1 ? l1 : w / kPer == 2 ? l2 : l3;
    S* mine = reinterpret_cast<S*>(buffer) + (w % kPer) * kSums;
    constexpr int N = Chunk<T>::N;
    constexpr int kLanes = GATED ? 4 : 8, kRows = 64 / kLanes, kWide = GATED ? 32 : 64;  // lanes a row, rows an instruction
    const int64_t n1 = g.n0 + kWide * (X::U / 2) * wn + 8 * (l % kLanes);
    bool far = false;  // whether any row of the tile has a far scale
    if constexpr (!Kind::kFloat) far = __any(lrow[X::kSize + (l & (X::W - 1))]);
    const bool inside = g.n0 + kWide * X::CB <= g.N && !far;  // the whole tile's columns, and ordinary scales
    // 32 rows and 64 of the wave's columns; `whole` (a compile-time constant) where all is inside
    const auto block = [&](int i, int y, auto whole) {
        const int64_t n = n1 + kWide * y;
        float sb[GATED ? 16 : 8];
        if constexpr (!Kind::kFloat)
#pragma unroll
            for (int x = 0; x < (GATED ? 16 : 8); ++x)
                sb[x] = lscale[X::kSize + 32 * X::U * wn + 64 * y + 8 * (l % kLanes) + (x < 8 ? x : 32 + x - 8)];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const auto& s = acc[i][2 * y + u];
                const S4 v = {s[4 * q], s[4 * q + 1], s[4 * q + 2], s[4 * q + 3]};
                *reinterpret_cast<S4*>(mine + (l & 31) * kBigRow + 32 * u + 8 * q + 4 * (l >> 5)) = v;
            }
        __builtin_amdgcn_wave_barrier();
        const auto put = [&](T* c, const T (&o)[8]) {
#pragma unroll
            for (int x = 0; x < 8 / N; ++x) {
                typename Chunk<T>::V v;
#pragma unroll
                for (int y = 0; y < N; ++y) v[y] = o[x * N + y];
                if (whole.value)
                    *reinterpret_cast<typename Chunk<T>::U*>(c + x * N) = v;
                else if (n + x * N < g.N)
                    chunk_store(c + x * N, g.N - n - x * N, v);
            }
        };
        // v: 8 sums (gated: 8 of the gate, 8 of the other projection)
        const auto row_out = [&](float sa, const S4 (&v)[GATED ? 4 : 2], int64_t tr) {
            T o[8];
            if constexpr (!GATED) {
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    if constexpr (Kind::kFloat)
                        o[x] = D::down(v[x / 4][x % 4]);
                    else
                        o[x] = scaled<D, !whole.value>(v[x / 4][x % 4], sa, sb[x]);
                }
            } else {
                float a[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    if constexpr (Kind::kFloat)
                        a[x] = v[x / 4][x % 4];
                    else
                        a[x] = scaled<F32, !whole.value>(v[x / 4][x % 4], sa, sb[x]);
                }
                if (Kind::kFloat && g.pre) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int x = 0; x < 8; ++x) o[x] = D::down(a[8 * h + x]);
                        put((T*)g.pre + (g.lo + tr) * g.ldp + h * g.N + n, o);
                    }
                }
#pragma unroll
                for (int x = 0; x < 8; ++x) o[x] = round_alone<D>(gated(a[x], a[8 + x], g.act));
            }
            put((T*)g.C + (g.lo + tr) * g.ldc + n, o);
        };
        const S* at = mine + (l / kLanes) * kBigRow + 8 * (l % kLanes);
        const int tr0 = 32 * (2 * i + wm) + l / kLanes;
        const auto sums = [&](int q, S4 (&v)[GATED ? 4 : 2]) {
#pragma unroll
            for (int x = 0; x < (GATED ? 4 : 2); ++x)
                v[x] = *reinterpret_cast<const S4*>(at + kRows * q * kBigRow + 4 * (x & 1) + 32 * (x >> 1));
        };
        constexpr int kQ = 32 / kRows;
        if (whole.value) {
            S4 v[kQ][GATED ? 4 : 2];
            int r[kQ];
            float sa[kQ];
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
                sums(q, v[q]);
                r[q] = lrow[tr0 + kRows * q];
                sa[q] = Kind::kFloat ? 1.0f : lscale[tr0 + kRows * q];
            }
#pragma unroll
            for (int q = 0; q < kQ; ++q)
                if (r[q] >= 0) row_out(sa[q], v[q], tr0 + kRows * q);
        } else {
#pragma unroll 1
            for (int q = 0; q < kQ; ++q) {
                S4 v[GATED ? 4 : 2];
                sums(q, v);
                const int r = lrow[tr0 + kRows * q];
                if (r >= 0) row_out(Kind::kFloat ? 1.0f : lscale[tr0 + kRows * q], v, tr0 + kRows * q);
            }
        }
        __builtin_amdgcn_wave_barrier();
    };
    if (inside) {
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int y = 0; y < X::U / 2; ++y) block(i, y, std::true_type());
    } else {
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int y = 0; y < X::U / 2; ++y) block(i, y, std::false_type());
    }
}

// The steps of part `split` of a sum whose B's rows are steps: C is then the part's sums.  No part is empty.
__device__ __forceinline__ GemmArgs part_of(GemmArgs g, int split) {
    const int64_t steps = (g.K + kBigK - 1) / kBigK, each = (steps + g.splits - 1) / g.splits, from = split * each;
    g.A += from * kBigK;
    g.B += from * (kBigK / 2) * g.ldb;
    g.K = min(g.K - from * kBigK, each * kBigK);
    g.C = g.part + split * g.S * g.N;
    g.ldc = g.N;
    return g;
}

// One tile of rows by expert.  TB: B's rows are the steps of the sum (g.K / 2 of them, g.N elements each).
template <class Kind, class D, class X, int ST, bool ONCE, bool GATED, bool TB, int F>
__device__ __forceinline__ void big_tile(const GemmArgs& g, int e, int64_t lo, int64_t hi, int64_t n0,
                                         const BigBuffers<ST>& m, int32_t* lrow, float* lscale, int tid, int w, int l) {
    BigDirect<X> sa;
    big_rows<Kind, X, F>(g, lo, hi, lrow, lscale, sa, w, l);
    typename Kind::S16 acc[F][X::U];
    const int steps = (int)((g.K + kBigK - 1) / kBigK);
    const int left = (int)(g.K - (int64_t)(steps - 1) * kBigK);
    if constexpr (TB) {
        BigTransposed<X, false> sb;
        sb.template place<false>(g.B + e * g.strideb, g.ldb, (int)(g.K / 2), n0, g.N, w, l);
        big_sums<Kind, X, ST, F, false, true, ONCE>(acc, m, sa, sb, steps, left, tid, w, l);
    } else {
        BigDirect<X> sb;
        big_columns<Kind, X, GATED>(g, e, n0, lscale, sb, tid, w, l);
        big_sums<Kind, X, ST, F, false, false, ONCE>(acc, m, sa, sb, steps, left, tid, w, l);
    }
    big_out<Kind, D, X, F, GATED>(big_out_of(g, lo, n0), acc, m.b[0], m.b[1], m.a[0], m.a[1], lrow, lscale, w, l);
}

// Tile number t of the m_tiles x n_tiles that there are.  Four row tiles to a
// column tile follow each other.  It is the tiles that there are, not those that
// the launch has room for, that are dealt out to the XCDs.
//
// One matrix: neighbours run on one XCD and share rows of A and of B in its L2.
// Experts: tiles go to the XCDs RUN at a time in turn: experts with many rows,
// bound by the matrix cores, and with few, bound by memory, are then under way
// on all of them.  Against runs of neighbours, and one and eight at a time (us, int8;
// uneven loads are log-normal with sigma 0.7): 8192 rows of 64 uneven experts,
// 4096 x 2048 192, 179, 186; 16384 of 128, 2048 x 1536 141, 131, 132; 512 of 8
// even ones, 4096 x 14336 133, 119, 132; in 256 x 256 tiles 8192 of 8 541, 524,
// 515; 32768 of 64, 4096 x 2048 340, 338, 336.  The tallest tiles first gained
// nothing on that.  RUN = 0, neighbours, where a row tile has few column tiles
// and all matrices fit the caches: 40000 of 16, 512 x 300 26, 29, 29.
template <class X, int RUN, bool GATED>
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
    n0 = (int64_t)(in / high) * (GATED ? X::kSize / 2 : X::kSize);
    return find_tile<X::kSize>(g, first + in % high, lane, e, lo, hi);
}

template <class Kind, class D, class X, int ST, bool ONCE, bool GATED, bool TB, bool PART = false>
__global__ __launch_bounds__(X::kThreads, X::W == 8 || X::CB * ST <= 4 ? 2 : 1) void gemm_big(GemmArgs args) {
    const GemmArgs g = PART ? part_of(args, blockIdx.y) : args;
    constexpr int kBytes = X::kSize * kBigK;
    __shared__ __attribute__((aligned(1024))) int8_t a0[kBytes], a1[kBytes], b0[kBytes], b1[kBytes];
    __shared__ int32_t lrow[X::kSize + X::W];  // row of A of every row of the tile, or -1; words of the waves
    __shared__ float lscale[Kind::kFloat ? 1 : 2 * X::kSize];   // scales of the tile's rows, then of its columns
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    int e;
    int64_t lo, hi, n0;
    const uint32_t m_tiles = count_tiles<X::kSize>(g, l);
    if (blockIdx.x >= m_tiles * g.n_tiles) return;
    if (!big_place<X, ST == 4 ? 1 : X::CB == 4 ? 8 : 0, GATED>(g, m_tiles, blockIdx.x, l, e, lo, hi, n0)) return;
    const int blocks = (int)((hi - lo + 63) >> 6);
#define SPX_TILE(F) big_tile<Kind, D, X, ST, ONCE, GATED, TB, F>(g, e, lo, hi, n0, m, lrow, lscale, tid, w, l)
    if constexpr (ST == 4) {
        __shared__ __attribute__((aligned(1024))) int8_t a2[kBytes], a3[kBytes], b2[kBytes], b3[kBytes];
        const BigBuffers<4> m = {{a0, a1, a2, a3}, {b0, b1, b2, b3}};
        if (blocks == 1) return SPX_TILE(1);
        SPX_TILE(2);
    } else {
        const BigBuffers<2> m = {{a0, a1}, {b0, b1}};
        if (blocks == 1) return SPX_TILE(1);
        if constexpr (X::CB == 4) {
            if (blocks == 3) return SPX_TILE(3);
            if (blocks == 4) return SPX_TILE(4);
        }
        SPX_TILE(2);
    }
#undef SPX_TILE
}

// ---------------------------------------------------------------------------
// Rows of any alignment and length: the 128 x 128 tiles, with the copies
// through registers.  A workgroup goes on to the next tile where there are more
// than the launch has workgroups.
template <class Kind, class D, bool GATED, bool TB, int F>
__device__ __forceinline__ void staged_tile(const GemmArgs& g, int e, int64_t lo, int64_t hi, int64_t n0,
                                            const BigBuffers<2>& m, int32_t* lrow, float* lscale, int tid, int w, int l) {
    BigDirect<Tile128> sa;
    big_rows<Kind, Tile128, F>(g, lo, hi, lrow, lscale, sa, w, l);
    typename Kind::S16 acc[F][2];
    const int steps = (int)((g.K + kBigK - 1) / kBigK);
    if constexpr (TB) {
        BigTransposed<Tile128, false> sb;
        sb.template place<true>(g.B + e * g.strideb, g.ldb, (int)(g.K / 2), n0, g.N, w, l);
        staged_sums<Kind, F, false, true>(acc, m, sa, sb, steps, w, l);
    } else {
        BigDirect<Tile128> sb;
        big_columns<Kind, Tile128, GATED>(g, e, n0, lscale, sb, tid, w, l);
        staged_sums<Kind, F, false, false>(acc, m, sa, sb, steps, w, l);
    }
    big_out<Kind, D, Tile128, F, GATED>(big_out_of(g, lo, n0), acc, m.b[0], m.b[1], m.a[0], m.a[1], lrow, lscale, w, l);
}

template <class Kind, class D, bool GATED, bool TB, bool PART = false>
__global__ __launch_bounds__(256, 2) void gemm_staged(GemmArgs args) {
    const GemmArgs g = PART ? part_of(args, blockIdx.y) : args;
    constexpr int kBytes = 128 * kBigK;
    __shared__ __attribute__((aligned(1024))) int8_t a0[kBytes], a1[kBytes], b0[kBytes], b1[kBytes];
    __shared__ int32_t lrow[128 + 4];
    __shared__ float lscale[Kind::kFloat ? 1 : 2 * 128];
    const BigBuffers<2> m = {{a0, a1}, {b0, b1}};
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    const uint32_t m_tiles = count_tiles<128>(g, l), total = m_tiles * g.n_tiles;
    for (uint32_t t = blockIdx.x; t < total; t += gridDim.x) {
        int e;
        int64_t lo, hi, n0;
        if (!big_place<Tile128, 8, GATED>(g, m_tiles, t, l, e, lo, hi, n0)) continue;
        __syncthreads();  // the tile before has been stored
        if (hi - lo <= 64)
            staged_tile<Kind, D, GATED, TB, 1>(g, e, lo, hi, n0, m, lrow, lscale, tid, w, l);
        else
            staged_tile<Kind, D, GATED, TB, 2>(g, e, lo, hi, n0, m, lrow, lscale, tid, w, l);
    }
}

// ---------------------------------------------------------------------------
// Few rows: tiles of 16 R rows x 16 C columns (gated: 8 C of each projection), W waves that share the tile and
// split K; rows of any alignment, K >= 16.
//
// With few rows the time is that of reading B once.  Each wave takes 128 bytes
// of every row in turn, eight lanes a row, and has its next 128 in flight while
// it puts these together to MFMA operands, through LDS that no other wave
// uses: nothing waits for another wave before the sums meet (int32 ones are exact
// in any order, fp32 ones are added in the waves' order).  int8, 32 tokens x 8 of 64 experts, 4096 x 2048
// (R = 1, C = 2, W = 4):
// 72 us where 50 experts get a token (419 MB, 5.8 TB/s), 85 where 63 do (6.2; reads
// alone reach 7.1), with ONCE, non-temporal loads of B where one row tile reads it
// (81 and 97 without).  Operands loaded as the MFMA wants them, sixteen rows of 64
// bytes an instruction, took a sixth longer (and half as long again non-temporal,
// which fetched each line twice), 64 x 4096 x 4096 so 12.1 against 9.4, and with
// unaligned rows three times as long.
template <class Kind, int R, int C, bool ONCE>
struct ThinOps {
    typedef typename Kind::S4 S4;
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
    // In floating point B's too: what its zeroed partner would be multiplied with may be an Inf or a NaN.
    __device__ __forceinline__ void mask(int64_t k, int64_t K) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int32_t m = low_mask(k, K, d);
#pragma unroll
            for (int j = 0; j < (Kind::kFloat ? kA + kB : kA); ++j) v[j][d] &= m;
        }
    }
    // The lanes of a wave read what others of them wrote.  A wave's LDS operations
    // are done in the order of its instructions, so no wait is needed, only that
    // the compiler keeps that order: the barriers emit nothing.
    __device__ __forceinline__ void multiply(S4 (&acc)[R][C], int8_t* lds, int l) const {
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
                for (int j = 0; j < C; ++j) acc[i][j] = Kind::mfma16(x[h][R + j], x[h][i], acc[i][j]);
    }
};

template <class Kind, class D, int R, int C, int W, bool ONCE, bool GATED>
__global__ __launch_bounds__(64 * W) void gemm_thin(GemmArgs g) {
    static_assert(!GATED || C % 2 == 0, "half the columns are the gate's");
    typedef typename D::T T;
    typedef typename Kind::S S;
    typedef typename Kind::S4 S4;
    typedef ThinOps<Kind, R, C, ONCE> Ops;
    constexpr int BM = 16 * R, BN = 16 * C, LD = BN + 4, kWide = GATED ? BN / 2 : BN;  // kWide columns of C
    constexpr int kSums = BM * LD * 4, kWave = Ops::kLds > kSums ? Ops::kLds : kSums;
    __shared__ __attribute__((aligned(1024))) int8_t lds[W * kWave];
    S* part = reinterpret_cast<S*>(lds);
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    // the row tiles of one column tile follow each other: those of one expert meet its rows of B in one L2
    const uint32_t v = xcd_contiguous((int)blockIdx.x, 0, (int)gridDim.x);
    int e;
    int64_t lo, hi;
    if (!find_tile<BM>(g, v % g.m_tiles, l, e, lo, hi)) return;
    const int64_t n0 = (int64_t)(v / g.m_tiles) * kWide;
    const int8_t *pa[Ops::kA], *pb[Ops::kB];
#pragma unroll
    for (int i = 0; i < Ops::kA; ++i) {
        const int64_t p = lo + 8 * i + (l >> 3);
        pa[i] = g.A + max(p < hi ? a_row(g, p) : -1, (int64_t)0) * g.lda;
    }
#pragma unroll
    for (int j = 0; j < Ops::kB; ++j) {
        const int i = 8 * j + (l >> 3), col = i % kWide;  // gated: row i - kWide of the other projection
        pb[j] = g.B + e * g.strideb + (min(n0 + col, g.N - 1) + (i >= kWide ? g.N : 0)) * g.ldb;
    }

    S4 acc[R][C];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < C; ++j) acc[i][j] = S4{0, 0, 0, 0};
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
            *reinterpret_cast<S4*>(part + (w * BM + 16 * i + (l & 15)) * LD + 16 * j + 4 * (l >> 4)) = acc[i][j];
    __syncthreads();
    for (int x4 = tid; x4 < BM * kWide / 4; x4 += 64 * W) {
        const int row = x4 / (kWide / 4), col = x4 % (kWide / 4) * 4;
        const int64_t p = lo + row, n = n0 + col;
        if (p >= hi || n >= g.N) continue;
        const int64_t ra = a_row(g, p);
        if (ra < 0) continue;
        S4 sum[GATED ? 2 : 1];
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); ++h) {
            sum[h] = *reinterpret_cast<const S4*>(part + row * LD + col + h * kWide);
#pragma unroll
            for (int u = 1; u < W; ++u) sum[h] += *reinterpret_cast<const S4*>(part + (u * BM + row) * LD + col + h * kWide);
        }
        float sa = 1.0f;
        const float* sb = nullptr;
        if constexpr (!Kind::kFloat) {
            sa = g.a_scale[ra];
            sb = g.b_scale + e * (GATED ? 2 * g.N : g.N) + n;
        }
        typedef T V4 __attribute__((ext_vector_type(4), aligned(sizeof(T))));
        const auto store = [&](T* c, const T (&o)[4]) {
            if (n + 4 <= g.N) {
                *reinterpret_cast<V4*>(c) = V4{o[0], o[1], o[2], o[3]};
            } else {
                for (int i = 0; i < 3; ++i)
                    if (n + i < g.N) c[i] = o[i];
            }
        };
        const auto out = [&](auto far) {
            T o[4];
            T* c = (T*)g.C + p * g.ldc + n;
            if constexpr (!GATED) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (Kind::kFloat)
                        o[i] = D::down(sum[0][i]);
                    else
                        o[i] = scaled<D, far.value>(sum[0][i], sa, sb[min((int64_t)i, g.N - 1 - n)]);
                }
            } else {
                float a[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (Kind::kFloat)
                            a[h][i] = sum[h][i];
                        else
                            a[h][i] = scaled<F32, far.value>(sum[h][i], sa, sb[h * g.N + min((int64_t)i, g.N - 1 - n)]);
                    }
                if (Kind::kFloat && g.pre)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[i] = D::down(a[h][i]);
                        store((T*)g.pre + p * g.ldp + h * g.N + n, o);
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = round_alone<D>(gated(a[0][i], a[1][i], g.act));
            }
            store(c, o);
        };
        if (!Kind::kFloat && __any(far_scale(sa)))
            out(std::true_type());
        else
            out(std::false_type());
    }
}

// ---------------------------------------------------------------------------
// Few rows, B's rows the steps of the sum (16 bits): tiles of 16 R rows x 64 columns, four waves that share the tile
// and split the steps; rows of any alignment.  A wave takes 64 rows of B in turn, the tile's 128 bytes of each, with its
// next 64 in flight, and transposes them on the way from its own part of LDS to the matrix cores: LDS holds 64 rows of 64
// columns, block c of 16 columns of row r at c ^ (r / 2 % 2 + 2 (r / 8 % 2)), so that the eight rows that half a wave reads
// at once lie in different banks.
template <class Kind, int R, bool ONCE>
struct ThinRows {
    typedef typename Kind::S4 S4;
    static constexpr int kA = 2 * R, kLds = 64 * 128 + 16 * R * kBigK;
    i32x4 a[kA], b[8];
    static __device__ __forceinline__ int place(int r) { return ((r >> 1) & 1) | ((r >> 2) & 2); }
    // Steps s .. s + 63 of `rows`; pa: rows of A, pb: the lane's chunk of B's first row; zeros behind the last step.
    // cols: the lane's elements inside B's rows (8: all); whole: of every lane.
    __device__ __forceinline__ void read(const int8_t* const (&pa)[kA], const int8_t* pb, int64_t ldb, int64_t s,
                                         int64_t rows, int cols, bool whole, bool narrow, const int8_t* zeros, int l) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t r = s + 8 * j + (l >> 3);
            const int8_t* p = r < rows ? pb + r * ldb : zeros;
            if (whole) {
                b[j] = ONCE ? __builtin_nontemporal_load(reinterpret_cast<const i32x4_u*>(p)) : *reinterpret_cast<const i32x4_u*>(p);
            } else if (narrow) {
                b[j] = i32x4{0, 0, 0, 0};
                for (int i = 0; i < 7; ++i)
                    if (r < rows && i < cols)
                        b[j][i >> 1] |= (int32_t)((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1)));
            } else {
                p = r < rows && cols > 0 ? p + 2 * cols - 16 : zeros;
                b[j] = shift_down(*reinterpret_cast<const i32x4_u*>(p), 16 - 2 * cols);
            }
        }
        const int64_t k = 2 * s + 16 * (l & 7), K = 2 * rows;
#pragma unroll
        for (int j = 0; j < kA; ++j) a[j] = K < 16 ? load_short(pa[j], k, K) : load_any(pa[j], k, K);
        if (s + 64 > rows && K >= 16)
#pragma unroll
            for (int j = 0; j < kA; ++j) a[j] = shift_down(a[j], (int)min(max(k - (K - 16), (int64_t)0), (int64_t)16));
    }
    // No wait for other waves: as ThinOps::multiply.
    __device__ __forceinline__ void multiply(S4 (&acc)[R][4], int8_t* lds, int l) const {
        int8_t* const la = lds + 64 * 128;
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = 8 * j + (l >> 3);
            *reinterpret_cast<i32x4*>(lds + r * 128 + ((((l & 7) >> 1) ^ place(r)) << 5) + ((l & 1) << 4)) = b[j];
        }
#pragma unroll
        for (int j = 0; j < kA; ++j) {
            const int r = 8 * j + (l >> 3);
            *reinterpret_cast<i32x4*>(la + r * kBigK + (((l & 7) ^ big_swizzle(r)) << 4)) = a[j];
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            i32x4 x[4], y[R];
            const int r = 32 * h + 8 * (l >> 4) + ((l >> 2) & 3);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int8_t* p = lds + r * 128 + 8 * (l & 3);
                const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + ((c ^ place(r)) << 5)));
                const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * 128 + ((c ^ place(r + 4)) << 5)));
                typedef short s16x8 __attribute__((ext_vector_type(8)));
                x[c] = __builtin_bit_cast(i32x4, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int q = 16 * i + (l & 15);
                y[i] = *reinterpret_cast<const i32x4*>(la + q * kBigK + (((4 * h + (l >> 4)) ^ big_swizzle(q)) << 4));
            }
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[i][c] = Kind::mfma16(x[c], y[i], acc[i][c]);
        }
    }
};

template <class Kind, class D, int R, bool ONCE, bool PART>
__global__ __launch_bounds__(256, 2) void gemm_thin_rows(GemmArgs args) {
    typedef typename D::T T;
    typedef typename Kind::S4 S4;
    typedef ThinRows<Kind, R, ONCE> Ops;
    constexpr int BM = 16 * R, W = 4, LD = 64 + 4, kSums = BM * LD * 4, kWave = Ops::kLds > kSums ? Ops::kLds : kSums;
    const GemmArgs g = PART ? part_of(args, blockIdx.y) : args;
    __shared__ __attribute__((aligned(1024))) int8_t lds[W * kWave];
    float* part = reinterpret_cast<float*>(lds);
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    // the row tiles of one column tile follow each other, as in gemm_thin
    const uint32_t v = xcd_contiguous((int)blockIdx.x, 0, (int)gridDim.x);
    int e;
    int64_t lo, hi;
    if (!find_tile<BM>(g, v % g.m_tiles, l, e, lo, hi)) return;
    const int64_t n0 = (int64_t)(v / g.m_tiles) * 64, rows = g.K / 2;
    const int8_t* pa[Ops::kA];
#pragma unroll
    for (int i = 0; i < Ops::kA; ++i) {
        const int64_t p = lo + 8 * i + (l >> 3);
        pa[i] = g.A + max(p < hi ? a_row(g, p) : -1, (int64_t)0) * g.lda;
    }
    const int8_t* pb = g.B + e * g.strideb + 2 * n0 + 16 * (l & 7);
    const int cols = (int)max(min(g.N - n0 - 8 * (l & 7), (int64_t)8), (int64_t)0);
    const bool whole = n0 + 64 <= g.N, narrow = g.N < 8;
    S4 acc[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][c] = S4{0, 0, 0, 0};
    int8_t* const mine = lds + w * Ops::kLds;
    Ops x, y;
    int64_t s = 64 * w;
    if (s < rows) x.read(pa, pb, g.ldb, s, rows, cols, whole, narrow, big_zeros, l);
    for (; s < rows; s += 128 * W) {
        const bool more = s + 64 * W < rows;
        if (more) y.read(pa, pb, g.ldb, s + 64 * W, rows, cols, whole, narrow, big_zeros, l);
        x.multiply(acc, mine, l);
        if (!more) break;
        if (s + 128 * W < rows) x.read(pa, pb, g.ldb, s + 128 * W, rows, cols, whole, narrow, big_zeros, l);
        y.multiply(acc, mine, l);
    }
    __syncthreads();  // the sums take the same LDS
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            *reinterpret_cast<S4*>(part + (w * BM + 16 * i + (l & 15)) * LD + 16 * c + 4 * (l >> 4)) = acc[i][c];
    __syncthreads();
    for (int x4 = tid; x4 < BM * 16; x4 += 64 * W) {
        const int row = x4 / 16, col = x4 % 16 * 4;
        const int64_t p = lo + row, n = n0 + col;
        if (p >= hi || n >= g.N) continue;
        S4 sum = *reinterpret_cast<const S4*>(part + row * LD + col);
#pragma unroll
        for (int u = 1; u < W; ++u) sum += *reinterpret_cast<const S4*>(part + (u * BM + row) * LD + col);
        T* c = (T*)g.C + p * g.ldc + n;
        typedef T V4 __attribute__((ext_vector_type(4), aligned(sizeof(T))));
        if (n + 4 <= g.N)
            *reinterpret_cast<V4*>(c) = V4{D::down(sum[0]), D::down(sum[1]), D::down(sum[2]), D::down(sum[3])};
        else
            for (int i = 0; i < 3; ++i)
                if (n + i < g.N) c[i] = D::down(sum[i]);
    }
}

// ---------------------------------------------------------------- launch
// go(kind, type)
template <class Go>
inline int by_type(int32_t dtype, Go go) {
    return dtype == SP_BF16 ? go(KindBf16(), Bf16()) : go(KindF16(), F16());
}

inline bool aligned16(const GemmArgs& g) {
    return ((uintptr_t)g.A | (uintptr_t)g.B | (uintptr_t)g.lda | (uintptr_t)g.ldb |
            (uintptr_t)(g.E > 1 ? g.strideb : 0)) % 16 == 0;
}

// Tile counts of a launch with bm x bn tiles (an upper bound on the row tiles
// when the offsets are on the device).
inline int64_t row_tiles(const GemmArgs& g, int64_t bm) {
    return g.offsets ? g.S / bm + std::min<int64_t>(g.E, g.S) : (g.S + bm - 1) / bm;
}
inline int64_t tiles(const GemmArgs& g, int64_t bm, int64_t bn) { return row_tiles(g, bm) * ((g.N + bn - 1) / bn); }

// Workgroups of a launch: all kernels but gemm_staged take one tile each and
// are not launched with more; that one goes on to the next.
constexpr int64_t kMostTiles = 1 << 22;

template <class K>
int gemm_launch(K kernel, GemmArgs g, int64_t bm, int64_t bn, int threads, hipStream_t s) {
    const int64_t n = tiles(g, bm, bn);
    if (n >= (int64_t)1 << 31) return SP_ERR_SIZE;
    g.m_tiles = (uint32_t)row_tiles(g, bm);
    g.n_tiles = (uint32_t)((g.N + bn - 1) / bn);
    hipLaunchKernelGGL(kernel, dim3((unsigned)std::min(n, kMostTiles), (unsigned)std::max(g.splits, 1)), dim3(threads), 0,
                       s, g);
    return hipGetLastError() == hipSuccess ? SP_OK : SP_ERR_HIP;
}

}  // namespace spx
