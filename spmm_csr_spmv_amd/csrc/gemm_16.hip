// Products of 16-bit rows (bf16, fp16; fp32 sums) sorted by expert, over one matrix or one per expert:
//   C = A B_e^T           rows of expert e; gated: a(A G_e^T) (A U_e^T) with B_e = [G_e; U_e]
// in the tiles of gemm_tiles.h.  8192 x 8192 x 8192 bf16 takes 840 us, 1.31 PFLOP/s (8192 x 8192 x 4096 420; the library's
// 680 and 367): the MFMAs fill 65 % of the cycles at 1.8 GHz, and the clock falls as they fill more (79 % at 1.72 GHz where
// copies read the caches only), so that power bounds it.  A gated product of as many columns takes 4 % more.
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
// other in a graph, with at least 256 MB of weights in turn.  The tiles and the order of the tests are those of the int8
// products, whose bytes a row are the same; the limits are of 16-bit rows.
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
    // A matrix whose 128 x 128 tiles nearly fill the chip: 16 x 14336 x 4096 21.4, 16x32 25.0; 32 x 14336 x 4096 21.4, 32x64
    // 28.7; not one row (21.9, 16x32 20.9), and not 32 tiles (16 x 4096 x 4096 21.8, 16x16 9.6).
    if (matrix && !any && g.S >= 8 && g.S <= 128 && mid >= 88 && mid <= 256)
        return launch(gemm_big<Kind, D, Tile128, 4, false, GATED, false>, 128, 128, 256);
    // Few tiles: 1 x 4096 x 4096 16x16 7.9, 16x32 11.0; 16 x 4096 x 1024 4.7, 5.3; 32 x 4096 x 4096 16x32 11.4, 16x16 13.3,
    // 32x32 13.4; 64 x 4096 x 4096 32x32 11.7, 16x32 13.7, 32x64 15.9, 128x128 24; 128 x 4096 x 4096 32x64 16.4, 32x32 16.9,
    // 128x128 34.  Experts of few rows: 16 x 8, 64, 2048, 2048 16x32 55, 32x32 58, 128x128 68; 64 x 8 94, 91, 112; 128 x 8
    // (16 rows) 32x32 113, 16x32 125, 128x128 120; 128 x 8, 128, 1024, 1024 (8 rows) 16x32 51, 32x32 51, 128x128 55.
    if (tiles(16, 32) <= 128) return launch_thin<Kind, D, 1, GATED ? 2 : 1, 8, GATED>(once, g, s);
    if (tiles(16, 32) <= 256 || (matrix && g.S <= 16) || (experts && g.S <= (deep ? 8 : 6) * groups))
        return launch_thin<Kind, D, 1, 2, 4, GATED>(once, g, s);
    if (tiles(32, 32) <= 256 || (experts && g.S <= 16 * groups && deep))
        return launch_thin<Kind, D, 2, 2, 4, GATED>(once, g, s);
    if (tiles(32, 64) <= (any ? 512 : 256) || (matrix && g.S <= 32 && deep))
        return launch_thin<Kind, D, 2, 4, 4, GATED>(once, g, s);
    if (any) return launch(gemm_staged<Kind, D, GATED, false>, 128, 128, 256);
    // One 128 x 128 tile a CU at most, or tiles that mostly wait for memory: four steps in LDS.  512 x 4096 x 4096 35, two
    // steps 51, 256x256 87; 1024 x 4096 x 4096 39, 58, 89; 512 x 8, 64, 2048, 2048 (64 rows) 135, 165, 182; 1024 x 8 (128
    // rows) 163, 191, 188; 512 x 2, 8, 4096, 4096 (128 rows) 85, 97, 109.
    if (mid <= 256 || (few && g.S <= (deep ? 128 : 64) * groups))
        return launch(gemm_big<Kind, D, Tile128, 4, false, GATED, false>, 128, 128, 256);
    // Up to two 128 x 128 tiles a CU: 512 x 14336 x 4096 68, four steps 71, 256x256 82.
    const int64_t cols = GATED ? 2 * g.N : g.N, wide = (cols + 255) / 256 * 256, narrow = (cols + 127) / 128 * 128;
    if (mid <= 512 || (few && 5 * wide >= 6 * narrow))
        return launch(gemm_big<Kind, D, Tile128, 2, false, GATED, false>, 128, 128, 256);
    // 1024 x 14336 x 4096 114, 128x128 136; 8192 x 8192 x 4096 428.
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
