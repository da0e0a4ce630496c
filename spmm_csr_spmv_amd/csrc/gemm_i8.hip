// Products in 8-bit integers with a scale per row of A (token) and per row of
// B (output channel), over one matrix B or over one per expert:
//   C[p, n] = a_scale[r] b_scale[e, n] sum_k A[r, k] B[e, n, k]
// where p runs over the rows sorted by expert, e is the expert whose range
// offsets[e] .. offsets[e + 1] holds p, and r is p, or the token src[p] / slots; and the
// gated products a(g) u of two such sums, whose matrices have 2 N rows.
// The sums are int32 and exact (K <= 131071: K 128^2 < 2^31), so the split of
// K over instructions and waves never changes a result; the float of a sum is
// multiplied by a_scale, then by b_scale, and rounded once to C's type (gated: g and u
// are fp32 numbers, and what is made of them is rounded).
//
// The tiles are those of gemm_tiles.h.  8192 x 8192 x 8192 (256 x 256 tiles) takes 461 us,
// 2.39 POP/s (443 to 468 on several cards); the MFMAs fill 65 % of the cycles and the chip
// runs at 1.7 GHz under them (one tile alone: 71 % at 2.4 GHz), so that power bounds it.  LDS
// operand reads take 27 % of them, without conflicts.  Unaligned rows: 8192 x 8192 x 4095 takes
// 474 us, 1.16 POP/s, bound by the unaligned loads (with aligned rows, copied straight to LDS,
// these tiles take 313).
#include "gemm_tiles.h"

namespace spx {

namespace {

template <class D, int R, int C, int W, bool GATED>
int launch_thin(bool once, const GemmArgs& g, hipStream_t s) {
    constexpr int kWide = GATED ? 8 * C : 16 * C;
    return once ? gemm_launch(gemm_thin<KindI8, D, R, C, W, true, GATED>, g, 16 * R, kWide, 64 * W, s)
                : gemm_launch(gemm_thin<KindI8, D, R, C, W, false, GATED>, g, 16 * R, kWide, 64 * W, s);
}

// Which kernel.  Times are medians in us, M x N x K, or tokens x choices, experts,
// K, N, of calls that follow each other in a graph, on normally distributed codes,
// with 1 GB of weights in turn, so that they come from memory.  Routing is uneven
// (scores favour experts with a standard deviation of 0.7, the scores' own being
// 1) unless it says even (no favour): uneven routing leaves some experts unused
// where there are few tokens, and makes the tiles of the others higher.
template <class D, bool GATED>
int gemm_t(GemmArgs g, hipStream_t s) {
    // bn rows of B a tile
    const auto tiles = [&](int64_t bm, int64_t bn) { return spx::tiles(g, bm, GATED ? bn / 2 : bn); };
    const auto launch = [&](auto kernel, int64_t bm, int64_t bn, int threads) {
        return gemm_launch(kernel, g, bm, GATED ? bn / 2 : bn, threads, s);
    };
    if (g.a_rows == 0) return SP_OK;  // no row of C has a row of A
    const int64_t groups = g.offsets ? std::min<int64_t>(g.E, g.S) : 1;
    const int64_t mid = tiles(128, 128);
    const bool any = !aligned16(g);
    if (g.K < 16 || mid > kMostTiles) return launch(gemm_staged<KindI8, D, GATED, false>, 128, 128, 256);
    const bool few = tiles(16, 32) <= kMostTiles;
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
    if (tiles(16, 32) <= 128) return launch_thin<D, 1, GATED ? 2 : 1, 8, GATED>(once, g, s);
    if (tiles(16, 32) <= 256 || (matrix && g.S <= 16) || (experts && g.S <= (deep ? 8 : 6) * groups))
        return launch_thin<D, 1, 2, 4, GATED>(once, g, s);
    if (tiles(32, 32) <= 256 || (experts && g.S <= 16 * groups && deep))
        return launch_thin<D, 2, 2, 4, GATED>(once, g, s);
    // Unaligned rows, whose 128 x 128 tiles are slower, up to 512 tiles:
    // 256 x 4096 x 4097 32, 128x128 54; 1024 x 1024 x 1023 13.1, 15.1.
    if (tiles(32, 64) <= (any ? 512 : 256) || (matrix && g.S <= 32 && deep))
        return launch_thin<D, 2, 4, 4, GATED>(once, g, s);
    // 8192 x 8192 x 4095 474, with aligned rows 250; 32 x 8, 64, 4095, 2048 119
    // (thin tiles 107), 96 x 8 134 (152), 24 x 8, 128, 1023, 2047 52 (55).
    if (any) return launch(gemm_staged<KindI8, D, GATED, false>, 128, 128, 256);
    // One 128 x 128 tile a CU at most, or tiles that mostly wait for memory: four
    // steps in LDS.  1024 x 4096 x 4096 24 against 35 with two steps and two
    // workgroups a CU, and 55 with 256 x 256 tiles; 512 x 8, 64, 4096, 2048 (64
    // rows) 129, 162, 159; 1024 x 8 (128 rows) 159, 199, 182; 1024 x 2, 8, 4096,
    // 14336 (256 rows) 222, 228, 187; 512 x 2 (128 rows) 151, 163, 170, but even
    // 165, 163, 138; shorter sums 512 x 8, 128, 2048, 1536 (32 rows) 90, 93, 94;
    // 2048 x 8 (128 rows) 144, 144, 130.
    if (once) return launch(gemm_big<KindI8, D, Tile128, 4, true, GATED, false>, 128, 128, 256);
    if (mid <= 256 || (few && g.S <= (deep ? 128 : 64) * groups))
        return launch(gemm_big<KindI8, D, Tile128, 4, false, GATED, false>, 128, 128, 256);
    // Up to two 128 x 128 tiles a CU: 2048 x 4096 x 4096 43, with four steps 47,
    // with 256 x 256 tiles 57.  Also where 256-wide tiles would be empty for a
    // fifth: 20000 x 2, 16, 512, 300 25, with 256 x 256 33.
    const int64_t cols = GATED ? 2 * g.N : g.N, wide = (cols + 255) / 256 * 256, narrow = (cols + 127) / 128 * 128;
    if (mid <= 512 || (few && 5 * wide >= 6 * narrow))
        return launch(gemm_big<KindI8, D, Tile128, 2, false, GATED, false>, 128, 128, 256);
    // 8192 x 8192 x 4096 250 against 313 with 128 x 128 tiles; 4096 x 4096 x 4096
    // 68, 82; 4096 x 8, 64, 4096, 2048 (512 rows) 341, even 335 against 415.
    return launch(gemm_big<KindI8, D, Tile256, 2, false, GATED, false>, 256, 256, 512);
}

}  // namespace

int gemm_i8_device(int64_t S, int32_t E, int64_t N, int64_t K, const int8_t* A, int64_t a_rows, int64_t lda,
                   const float* a_scale, const int32_t* src, int32_t slots, const int8_t* B, int64_t ldb,
                   int64_t strideb, const float* b_scale, const int32_t* offsets, int32_t gate, int32_t c_type, void* C,
                   int64_t ldc, hipStream_t s) {
    GemmArgs g{S, N, K, A, a_rows, lda, a_scale, src, slots, B, ldb, strideb, b_scale, offsets, E, C, ldc};
    const auto go = [&](auto d) {
        typedef decltype(d) D;
        if (gate < 0) return gemm_t<D, false>(g, s);
        g.act = gate;
        return gemm_t<D, true>(g, s);
    };
    if (c_type == SP_F32) return go(F32());
    if (c_type == SP_BF16) return go(Bf16());
    return go(F16());
}

}  // namespace spx
