// Products of 16-bit rows (bf16, fp16; fp32 sums) sorted by expert, over one matrix or one per expert:
//   C = A B_e^T           rows of expert e; gated: a(A G_e^T) (A U_e^T) with B_e = [G_e; U_e]
// in the tiles of gemm_tiles.h.
#include "gemm_tiles.h"

namespace spx {

namespace {

template <class Kind, class D, int R, int C, int W, bool GATED>
int launch_thin(bool once, const GemmArgs& g, hipStream_t s) {
    constexpr int kWide = GATED ? 8 * C : 16 * C;
    return once ? gemm_launch(gemm_thin<Kind, D, R, C, W, true, GATED>, g, 16 * R, kWide, 64 * W, s)
                : gemm_launch(gemm_thin<Kind, D, R, C, W, false, GATED>, g, 16 * R, kWide, 64 * W, s);
}

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
    const bool deep = g.K > 2048;
    const bool once = !any && g.S <= 32 * groups;
    if (tiles(16, 32) <= 128) return launch_thin<Kind, D, 1, GATED ? 2 : 1, 8, GATED>(once, g, s);
    if (tiles(16, 32) <= 256 || (matrix && g.S <= 16) || (experts && g.S <= (deep ? 8 : 6) * groups))
        return launch_thin<Kind, D, 1, 2, 4, GATED>(once, g, s);
    if (tiles(32, 32) <= 256 || (experts && g.S <= 16 * groups && deep))
        return launch_thin<Kind, D, 2, 2, 4, GATED>(once, g, s);
    if (tiles(32, 64) <= (any ? 512 : 256) || (matrix && g.S <= 32 && deep))
        return launch_thin<Kind, D, 2, 4, 4, GATED>(once, g, s);
    if (any) return launch(gemm_staged<Kind, D, GATED, false>, 128, 128, 256);
    if (mid <= 256 || (few && g.S <= (deep ? 128 : 64) * groups))
        return launch(gemm_big<Kind, D, Tile128, 4, false, GATED, false>, 128, 128, 256);
    const int64_t cols = GATED ? 2 * g.N : g.N, wide = (cols + 255) / 256 * 256, narrow = (cols + 127) / 128 * 128;
    if (mid <= 512 || (few && 5 * wide >= 6 * narrow))
        return launch(gemm_big<Kind, D, Tile128, 2, false, GATED, false>, 128, 128, 256);
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
