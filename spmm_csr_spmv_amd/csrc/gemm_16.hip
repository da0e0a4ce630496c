// Products of 16-bit rows (bf16, fp16; fp32 sums) sorted by expert, over one matrix or one per expert:
//   C = A B_e^T           rows of expert e; gated: a(A G_e^T) (A U_e^T) with B_e = [G_e; U_e]
// in the tiles of gemm_tiles.h.  8192 x 8192 x 8192 bf16 takes 840 us, 1.31 PFLOP/s (8192 x 8192 x 4096 420 to 452 on
// several cards; the library's 680 and 367, so that power alone is not what bounds it): the MFMAs fill 65 % of the cycles at
// 1.6 to 1.8 GHz, and the clock falls as they fill more (79 % at 1.72 GHz where copies read the caches only); LDS operand
// reads take 27 %.  A gated product of as many columns takes 4 % more.  A tile's end, in which its CU multiplies nothing,
// takes about 4 us: 8192 x 8192 x 2048, four tiles a CU of 32 steps each, 227 (the library's 189); 32 even experts of 1024
// rows, 2048 x 2048 274, 2816 x 2048 381 (about 0.27 a tile, whole rounds of 256 or not).
#include "gemm_tiles.h"

namespace spx {

namespace {

template <class Kind, class D, int R, int C, int W, bool GATED>
int launch_thin(bool once, const GemmArgs& g, hipStream_t s) {
    constexpr int kWide = GATED ? 8 * C : 16 * C;
    return once ? gemm_launch(gemm_thin<Kind, D, R, C, W, true, GATED>, g, 16 * R, kWide, 64 * W, s)
                : gemm_launch(gemm_thin<Kind, D, R, C, W, false, GATED>, g, 16 * R, kWide, 64 * W, s);
}

// Which kernel.  Times are medians in us, M x N x K, or tokens x choices, experts, N, K, bf16, of calls that follow each
// other in a graph, with 1 GB of weights in turn, so that they come from memory (256 MB stay in the caches in part, and
// favour other tiles).  The tiles and the order of the tests are those of the int8 products, whose bytes a row are the
// same; the limits are of 16-bit rows.
template <class Kind, class D, bool GATED>
int gemm16_t(const GemmArgs& g, hipStream_t s) {
    // bn rows of B a tile
    const auto tiles = [&](int64_t bm, int64_t bn) { return spx::tiles(g, bm, GATED ? bn / 2 : bn); };
    const auto launch = [&](auto kernel, int64_t bm, int64_t bn, int threads) {
        return gemm_launch(kernel, g, bm, GATED ? bn / 2 : bn, threads, s);
    };
    const int64_t groups = g.offsets ? std::min<int64_t>(g.E, g.S) : 1;
    const int64_t mid = tiles(128, 128);
    const bool any = !aligned16(g);
    if (g.K < 16 || mid > kMostTiles) return launch(gemm_staged<Kind, D, GATED, false>, 128, 128, 256);
    const bool few = tiles(16, 32) <= kMostTiles;
    const bool matrix = few && groups == 1, experts = few && groups > 1 && !any;
    const bool deep = g.K >= 2048;
    const bool once = !any && g.S <= 32 * groups;
    // Few tiles: 1 x 4096 x 4096 16x16 7.7, 16x32 10.8; 16 x 4096 x 1024 4.5, 5.1; 32 x 4096 x 4096 16x32 11.0, 16x16 12.9,
    // 32x32 13.0; 64 x 4096 x 4096 32x32 13.2, 16x32 15.7, 32x64 17.5, 128x128 31; 128 x 4096 x 4096 32x64 16.9, 32x32 19.2,
    // 128x128 40.  Few rows of one matrix in any number: 16 x 14336 x 4096 16x32 22.2, 16x16 25.4, 128x128 30; 32 x 14336 x
    // 4096 32x64 22.6, 32x32 25.0, 16x32 33.8, 128x128 32.  Experts of few rows: 16 x 8, 64, 2048, 2048 16x32 53, 32x32 56, 128x128
    // 79; 64 x 8 82, 80, 106; 128 x 8 (16 rows) 32x32 104, 16x32 113, 128x128 113; 128 x 8, 128, 1024, 1024 (8 rows) 16x32 46,
    // 32x32 48, 128x128 52.
    //
    // Gated, of as many gate columns as N says (the tiles' columns are then half gate): 1 x 2048 x 4096 16x16 10.3, 16x32
    // 11.5; 16 x 2048 x 4096 12.0, 12.3; 64 x 2048 x 4096 32x32 14.3, 16x32 17.1, 32x64 18.4; 128 x 2048 x 4096 32x64 17.5,
    // 32x32 20.6, 128x128 41; 16 x 7168 x 4096 16x32 24.7, 32x64 23.8, 128x128 32; 32 x 7168 x 4096 32x64 24.6, 32x32 28.2,
    // 128x128 34; 256 x 2048 x 4096 (512 of 32x64) 128x128 40, 32x64 31.  Experts, 64, 1024, 2048: 64 x 8 16x32 98, 32x32 96,
    // 128x128 114; 128 x 8 32x32 123, 128x128 125; 512 x 8 128x128 139, 32x32 189.  Without pre-activations; they add up to 3 %.
    //
    // Rows off 16 bytes, whose 128 x 128 tiles are slower, up to 512 tiles of 32x64: 256 x 4096 x 4095 45, 128x128 91;
    // 1024 x 1024 x 1023 14.8, 21.5; from 1024 on no longer: 512 x 4096 x 4095 86, 88; 1024 x 2048 x 2047 44, 38.  Experts of
    // such rows: 128 x 8, 64, 1023, 1025 128x128 40, 32x32 48; 64 x 8 36, 16x32 38; but 16 x 8, 64, 2047, 2049 105, 16x32 81.
    if (tiles(16, 32) <= 128) return launch_thin<Kind, D, 1, GATED ? 2 : 1, 8, GATED>(once, g, s);
    if (tiles(16, 32) <= 256 || (matrix && g.S <= 16) || (experts && g.S <= (deep ? 8 : 6) * groups))
        return launch_thin<Kind, D, 1, 2, 4, GATED>(once, g, s);
    if (tiles(32, 32) <= 256 || (experts && g.S <= 16 * groups && deep))
        return launch_thin<Kind, D, 2, 2, 4, GATED>(once, g, s);
    if (tiles(32, 64) <= (any ? 512 : 256) || (matrix && g.S <= 32 && deep))
        return launch_thin<Kind, D, 2, 4, 4, GATED>(once, g, s);
    if (any) return launch(gemm_staged<Kind, D, GATED, false>, 128, 128, 256);
    // One 128 x 128 tile a CU at most, or tiles that mostly wait for memory: four steps in LDS.  512 x 4096 x 4096 38, two
    // steps 60, 256x256 98; 1024 x 4096 x 4096 40, 59, 96; 512 x 8, 64, 2048, 2048 (64 rows) 127, 153, 168; 1024 x 8 (128
    // rows) 157, 186, 179; 512 x 2, 8, 4096, 4096 (128 rows) 84, 91, 107.
    if (mid <= 256 || (few && g.S <= (deep ? 128 : 64) * groups))
        return launch(gemm_big<Kind, D, Tile128, 4, false, GATED, false>, 128, 128, 256);
    // Up to two 128 x 128 tiles a CU: 512 x 14336 x 4096 77, four steps 82, 256x256 101.
    const int64_t cols = GATED ? 2 * g.N : g.N, wide = (cols + 255) / 256 * 256, narrow = (cols + 127) / 128 * 128;
    if (mid <= 512 || (few && 5 * wide >= 6 * narrow))
        return launch(gemm_big<Kind, D, Tile128, 2, false, GATED, false>, 128, 128, 256);
    // 1024 x 14336 x 4096 113, 128x128 140; 8192 x 8192 x 4096 452, 559; 8192 x 4, 32, 2048, 1408 217, 260; gated 1024 x
    // 7168 x 4096 115, 128x128 144 (512 rows 106, 76).
    return launch(gemm_big<Kind, D, Tile256, 2, false, GATED, false>, 256, 256, Tile256::kThreads);
}

}  // namespace

int moe_gemm_device(const Products& p, int32_t gate, void* pre, int64_t ldp, void* C, int64_t ldc, hipStream_t s) {
    if (p.a_rows == 0) return SP_OK;  // no row of C has a row of A
    GemmArgs g{p.S, p.N, 2 * p.K, (const int8_t*)p.A, p.a_rows, 2 * p.lda, nullptr, p.src, p.slots, (const int8_t*)p.B,
               2 * p.ldb, 2 * p.strideb, nullptr, p.offsets, p.E, C, ldc, pre, ldp, gate};
    return by_type(p.dtype, [&](auto k, auto d) {
        return gate < 0 ? gemm16_t<decltype(k), decltype(d), false>(g, s)
                        : gemm16_t<decltype(k), decltype(d), true>(g, s);
    });
}

}  // namespace spx
