// The gradients of the 16-bit products of experts (gemm_16.hip):
//   dA = dC B_e           the tiles of the products, B's rows the steps of the sum
//   dB_e = dC^T A         over the expert's rows: both operands' rows are steps of the sum
// The gated product's gradient is that of a product with 2 N columns, whose dC
// a kernel of its own forms from dH and the kept pre-activations.
#include "gemm_tiles.h"

namespace spx {

namespace {

// ---------------------------------------------------------------- dB
struct GradArgs {
    int64_t S, M, N;          // rows; rows and columns of a matrix of dB
    const int8_t* P;          // dC, S x M, rows ldp bytes apart
    int64_t ldp;
    const int8_t* Q;          // A, rows of N, ldq bytes apart
    int64_t q_rows, ldq;
    const int32_t* src;       // or NULL: row p goes with row p of A
    FastDiv slots;
    uint32_t sources;         // slots of A's rows, 2^31 at most
    const int32_t* offsets;   // or NULL: one matrix, rows 0 .. S
    int32_t E;
    void* C;                  // dB, rows ldc and experts stridec elements apart
    int64_t ldc, stridec;
    float* part;              // splits > 1: [splits][E][M][N]
    int32_t splits;           // of an expert's rows
    uint32_t m_tiles, n_tiles;
};

// Square tiles of dB, steps of 64 rows.  Where an expert has many rows and the tiles are few, its rows
// are split and the parts' fp32 sums (PART) added afterwards in the order of the splits.
// Bound as the products are: 4096 rows, 8192 x 8192 bf16 in 420 to 440 us, 1.28 PFLOP/s (the library 480); 8192 x 4 of 32
// experts, 2816 x 2048 405 to 430 (128 x 128 tiles 509), with sources 440 to 465, of rows off 16 bytes 1060.  512 x 8 of 64
// experts, 1024 x 1024, one step a tile: 45 with sources.
template <class Kind, class D, class X, bool STAGED, bool PART, bool GATHER>
__device__ __forceinline__ void rows_sum_tile(const GradArgs& g, uint32_t t, uint32_t total, const BigBuffers<2>& m,
                                              int32_t* lrow, int tid, int w, int l) {
    // eight tiles in a row, which share a tile's columns of A, on one XCD
    const uint32_t v = t < total / 64 * 64 ? t / 64 * 64 + t % 8 * 8 + t / 8 % 8 : t;
    const uint32_t per = g.m_tiles * g.n_tiles, part = v / per, in = v % per;
    const int e = (int)(part / g.splits), split = (int)(part % g.splits);
    const int64_t m0 = (int64_t)(in % g.m_tiles) * (X::kSize), n0 = (int64_t)(in / g.m_tiles) * (X::kSize);
    int a = 0, b = (int)g.S;
    if (g.offsets) expert_rows(g.offsets, g.E, g.S, e, a, b);
    a = __builtin_amdgcn_readfirstlane(a);
    b = __builtin_amdgcn_readfirstlane(b);
    const int each = (int)(((uint32_t)(b - a) + g.splits * 64u - 1) / (g.splits * 64u)) * 64;
    const int from = (int)min((int64_t)a + (int64_t)split * each, (int64_t)b);
    int rows = min(each, b - from);
    // A row of dC whose row of A is not there counts as zeros too: what it holds may be an Inf or a NaN.
    if (!GATHER) rows = (int)max(min((int64_t)rows, g.q_rows - from), (int64_t)0);
    for (int i = tid; i < X::kSize; i += X::kThreads) lrow[i] = m0 + i < g.M ? 0 : -1;
    BigTransposed<X, false> sa;
    BigTransposed<X, GATHER> sb;
    sa.template place<STAGED>(g.P + from * g.ldp, g.ldp, rows, m0, g.M, w, l);
    if constexpr (GATHER) {
        sb.template place<STAGED>(g.Q, g.ldq, rows, n0, g.N, w, l);
        sb.src = rows > 0 ? g.src + from : reinterpret_cast<const int32_t*>(big_zeros);
        sb.slots = g.slots;
        sb.sources = g.sources;
    } else {
        sb.template place<STAGED>(g.Q + from * g.ldq, g.ldq, rows, n0, g.N, w, l);
    }
    constexpr int F = X::CB;
    typename Kind::S16 acc[F][X::U];
    const int steps = (rows + 63) >> 6;
    static_assert(BigShape<X, F>::kA == BigShape<X, F>::kB, "a step's copies of dC come after the fetch of its sources");
    const auto sums = [&](const auto& p) {
        if constexpr (STAGED)
            staged_sums<Kind, F, true, true>(acc, m, p, sb, steps, w, l);
        else
            big_sums<Kind, X, 2, F, true, true, false>(acc, m, p, sb, steps, kBigK, tid, w, l);
    };
    if constexpr (GATHER)
        sums(BigPartner<X>{sa, sb});
    else
        sums(sa);
    BigOut o{(typename D::T*)g.C + e * g.stridec, g.ldc, g.N, m0, n0, nullptr, 0, 0};
    if (PART) o.C = g.part + ((int64_t)split * g.E + e) * g.M * g.N, o.ldc = g.N;
    const float* none = nullptr;
    big_out<Kind, std::conditional_t<PART, F32, D>, X, F, false>(o, acc, m.b[0], m.b[1], m.a[0], m.a[1], lrow, none, w, l);
}

template <class Kind, class D, class X, bool STAGED, bool PART, bool GATHER>
__global__ __launch_bounds__(X::kThreads, X::W == 8 || X::CB == 2 ? 2 : 1) void gemm_rows_sum(GradArgs g) {
    constexpr int kBytes = X::kSize * kBigK;
    __shared__ __attribute__((aligned(1024))) int8_t a0[kBytes], a1[kBytes], b0[kBytes], b1[kBytes];
    __shared__ int32_t lrow[X::kSize];
    const BigBuffers<2> m = {{a0, a1}, {b0, b1}};
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    const uint32_t total = g.m_tiles * g.n_tiles * (uint32_t)g.splits * (uint32_t)g.E;
    if constexpr (!STAGED) {  // as many workgroups as tiles
        rows_sum_tile<Kind, D, X, STAGED, PART, GATHER>(g, blockIdx.x, total, m, lrow, tid, w, l);
    } else {
        for (uint32_t t = blockIdx.x; t < total; t += gridDim.x) {
            if (t != blockIdx.x) __syncthreads();  // the tile before has been stored
            rows_sum_tile<Kind, D, X, STAGED, PART, GATHER>(g, t, total, m, lrow, tid, w, l);
        }
    }
}

// The parts' sums, in their order, rounded: rows of N, row i going to row i % M of matrix i / M.  With offsets (dA; one
// matrix) only the rows that some expert has.  A workgroup does 1024 columns of a row.
struct PartArgs {
    const float* part;  // [splits][rows][N]
    int32_t splits;
    int64_t rows, N, M;
    void* C;
    int64_t ldc, stridec;
    const int32_t* offsets;
    int32_t E;
};
template <class D>
__global__ __launch_bounds__(256) void add_parts_kernel(PartArgs g) {
    typedef float F4 __attribute__((ext_vector_type(4)));
    typedef float F4U __attribute__((ext_vector_type(4), aligned(4)));
    typedef typename D::T T;
    typedef T V4 __attribute__((ext_vector_type(4), aligned(sizeof(T))));
    const int64_t n = (int64_t)blockIdx.y * 1024 + 4 * threadIdx.x;
    for (int64_t row = blockIdx.x; row < g.rows; row += gridDim.x) {
        if (g.offsets) {
            int mine = 0;
            for (int e = threadIdx.x; e < g.E; e += 256) {
                int a, b;
                expert_rows(g.offsets, g.E, g.rows, e, a, b);
                mine |= a <= row && row < b;
            }
            if (!__syncthreads_or(mine)) continue;
        }
        T* to = (T*)g.C + row / g.M * g.stridec + row % g.M * g.ldc + n;
        const float* from = g.part + row * g.N + n;
        const int64_t next = g.rows * g.N;
        if (n + 4 <= g.N) {
            F4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
            int s = 0;
            for (; s + 4 <= g.splits; s += 4) {
                F4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const F4U*>(from + (s + i) * next);
#pragma unroll
                for (int i = 0; i < 4; ++i) sum += v[i];
            }
            for (; s < g.splits; ++s) sum += *reinterpret_cast<const F4U*>(from + s * next);
            *reinterpret_cast<V4*>(to) = V4{D::down(sum[0]), D::down(sum[1]), D::down(sum[2]), D::down(sum[3])};
        } else {
            for (int i = 0; i < 3 && n + i < g.N; ++i) {
                float sum = 0.0f;
                for (int s = 0; s < g.splits; ++s) sum += from[s * next + i];
                to[i] = D::down(sum);
            }
        }
    }
}
template <class D>
int add_parts(const PartArgs& g, hipStream_t s) {
    const int64_t y = (g.N + 1023) / 1024;
    if (y > 65535) return SP_ERR_SIZE;
    hipLaunchKernelGGL((add_parts_kernel<D>), dim3((unsigned)std::min<int64_t>(g.rows, 1 << 20), (unsigned)y), dim3(256), 0, s, g);
    return hipGetLastError() == hipSuccess ? SP_OK : SP_ERR_HIP;
}

// Rows of these lengths, laid out without gaps, are not aligned.  (The workspace's size goes by the lengths alone.)
bool odd(int64_t M, int64_t N) { return M % 8 || N % 8; }

// Into how many parts to cut the sums of `steps` steps of a product's tiles, and whether 256 x 256 tiles are better than
// 128 x 128 ones: the least of an estimate in us.  A step (64 of the sum) of 128 x 128 tiles takes `one` where there is one
// on a CU (dA's, of rows from memory, 0.4 to 0.65 measured; dB's 0.65), 1.1 where there are two; of 256 x 256 ones 1.8; of 128 x 128 ones of unaligned rows 1.05 and 1.6.  All of it takes
// `memory` at least.  Parts are `outputs` fp32 numbers each, written and read at 4 TB/s, and a launch.
// dB (bf16, us): of 32768 rows, 1024 x 1024 in parts 106, whole 324; of 512 rows, 1024 x 4096 whole 10, in 4 parts 36; of
// 2048 x 8 of 64 experts, 2816 x 2048 in 256 x 256 tiles 358, in 128 x 128 ones 433.
struct Cut {
    bool wide;
    int splits;
};
Cut best_cut(int64_t narrow_tiles, int64_t wide_tiles, int64_t steps, double one, double memory, double outputs,
             bool wide_parts, bool unaligned) {
    Cut best{false, 1};
    double least = 1e300;
    for (int w = 0; w < (unaligned ? 1 : 2); ++w)
        for (const int n : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
            if (n > 1 && (2 * n > steps || (w && !wide_parts))) break;
            const int64_t each = (steps + n - 1) / n, parts = n == 1 ? 1 : (steps + each - 1) / each;  // none is empty
            const int64_t tiles = (w ? wide_tiles : narrow_tiles) * parts;
            const double step = w              ? 1.8 * ((tiles + 255) / 256)
                                : tiles <= 256 ? (unaligned ? 1.05 : one)
                                               : (unaligned ? 1.6 : 1.1) * ((tiles + 511) / 512);
            const double us = std::max(step * each, memory) + (parts > 1 ? 4.0 + 2e-6 * parts * outputs : 0.0);
            if (us < least) least = us, best = Cut{w != 0, (int)parts};
        }
    return best;
}

// ---------------------------------------------------------------- the gate's gradient
// dpre[p] = [dg du] of the rows up to the last that some expert has (offsets need not ascend), rows ldd elements apart;
// rounded to the operands' type, which the matrix cores want.  Memory bounds it: 32768 x 1408 bf16 in 75 to 84 us, 5.4 to 6.1 TB/s.
template <class D>
__global__ __launch_bounds__(256) void gate_backward_kernel(int64_t S, int64_t N, int32_t E, const int32_t* offsets, int act,
                                                            const typename D::T* __restrict__ dH, int64_t ldh,
                                                            const typename D::T* __restrict__ pre, int64_t ldp,
                                                            typename D::T* __restrict__ out, int64_t ldd) {
    typedef typename D::T T;
    constexpr int C = Chunk<T>::N;
    __shared__ int most;
    if (threadIdx.x == 0) most = 0;
    __syncthreads();
    for (int e = threadIdx.x; offsets && e < E; e += 256) atomicMax(&most, offsets[e + 1]);  // the order does not matter
    __syncthreads();
    const int64_t rows = offsets ? min((int64_t)most, S) : S, chunks = (N + C - 1) / C;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * chunks; i += (int64_t)gridDim.x * 256) {
        const int64_t p = i / chunks, c = i % chunks * C, left = N - c;
        const auto dh = chunk_load(dH + p * ldh + c, left), g = chunk_load(pre + p * ldp + c, left),
                   u = chunk_load(pre + p * ldp + N + c, left);
        typename Chunk<T>::V dg, du;
#pragma unroll
        for (int x = 0; x < C; ++x) {
            float a, b;
            gated_backward(D::up(dh[x]), D::up(g[x]), D::up(u[x]), act, a, b);
            dg[x] = round_alone<D>(a);
            du[x] = round_alone<D>(b);
        }
        chunk_store(out + p * ldd + c, left, dg);
        chunk_store(out + p * ldd + N + c, left, du);
    }
}

// ---------------------------------------------------------------- launch
// dA = dC B, M rows of B a sum.  One matrix of up to 2^23 numbers and up to 32 rows: tiles of 16 or 32 rows, whose sums are
// cut into as many parts as give 512 workgroups; else 128 x 128 or 256 x 256 ones, in parts where best_cut says so, four
// steps in LDS where there is a tile a CU.  bf16, weights from memory, us (rows, M, columns): 16 x 4096 x 1024 thin 8.8,
// 128 x 128 tiles in 8 parts 11.1; 16 x 3840 x 2048 11.1, 11.7; from there on alike, and thin ones lose with more rows: 16 x
// 14336 x 4096 29.1, 29.2 (4.0 TB/s of weights; whole 92), 32 x 28672 x 4096 53.6, 49.2; 64 x 4096 x 14336 in 2 parts 31,
// whole 41; two tiles a CU 1536 x 6528 x 1536 in 3 parts 52 (with four steps 58), whole 58, 1536 x 16384 x 1536 103 (112),
// 137.  Experts' weights take their time whatever the tiles, so that parts and thin tiles only cost: 128 x 8 of 64
// experts, 2816 x 2048 whole 134 (5.5 TB/s of weights), in 2 parts 156, thin 165; 64 x 2 of 8, 4096 x 4096 49, 58, 67; rows
// off 16 bytes (128 x 8 of 64, 2815 x 2047) 150, 168, 334.  4096 x 8192 x 8192 in 256 x 256 tiles 435, 1.26 PFLOP/s (the
// library 417).
struct RowPlan {
    int high;    // rows of a thin tile (16 R), or 0
    bool wide;
    int splits;
};
RowPlan row_plan(int64_t S, int32_t E, int64_t M, int64_t N) {
    const int64_t groups = std::max<int64_t>(std::min<int64_t>(E, S), 1), rows = S / groups;
    const int high = groups > 1 || M * N > (1 << 23) ? 0 : rows <= 16 ? 16 : rows <= 32 ? 32 : 0;
    const int64_t steps = (M + 63) / 64;
    const auto tiles = [&](int64_t bm, int64_t bn) {
        return std::max<int64_t>((groups > 1 ? S / bm + groups : (S + bm - 1) / bm) * ((N + bn - 1) / bn), 1);
    };
    if (high && tiles(high, 64) <= kMostTiles / 2) {
        const int64_t want = std::min<int64_t>({512 / tiles(high, 64), steps / 4, 32});  // a step for each of four waves
        const int64_t each = (steps + want - 1) / std::max<int64_t>(want, 1);
        return RowPlan{high, false, want < 2 ? 1 : (int)((steps + each - 1) / each)};  // none is empty
    }
    // an expert's last tile is half as high as the others on the average, and takes half their time
    const auto even = [&](int64_t b) { return tiles(b, b) - (groups > 1 ? groups / 2 * ((N + b - 1) / b) : 0); };
    const double memory = 2.0 * groups * M * N / 5.5e6;  // B at 5.5 TB/s
    const Cut c = best_cut(even(128), even(256), steps, 0.55, memory, (double)S * N, false, odd(M, N));
    return RowPlan{0, c.wide, c.splits};
}

template <class Kind, class D>
int row_gradient_t(const GemmArgs& g, const RowPlan& plan, hipStream_t s) {
    const auto launch = [&](auto kernel, int64_t bm, int64_t bn, int threads) { return gemm_launch(kernel, g, bm, bn, threads, s); };
    const int64_t groups = g.offsets ? std::min<int64_t>(g.E, g.S) : 1;
    const bool any = !aligned16(g), once = !any && g.S <= 32 * groups;
    const int64_t mid = tiles(g, 128, 128);
    const auto thin = [&](auto part) {
        constexpr bool P = decltype(part)::value;
        typedef std::conditional_t<P, F32, D> O;
        return plan.high == 16 ? (once ? launch(gemm_thin_rows<Kind, O, 1, true, P>, 16, 64, 256)
                                  : launch(gemm_thin_rows<Kind, O, 1, false, P>, 16, 64, 256))
                          : (once ? launch(gemm_thin_rows<Kind, O, 2, true, P>, 32, 64, 256)
                                  : launch(gemm_thin_rows<Kind, O, 2, false, P>, 32, 64, 256));
    };
    if (g.splits > 1) {
        const int rc = plan.high ? thin(std::true_type())
                       : any ? launch(gemm_staged<Kind, F32, false, true, true>, 128, 128, 256)
                       : mid * g.splits <= 256
                           ? launch(gemm_big<Kind, F32, Tile128, 4, false, false, true, true>, 128, 128, 256)
                           : launch(gemm_big<Kind, F32, Tile128, 2, false, false, true, true>, 128, 128, 256);
        if (rc) return rc;
        return add_parts<D>(PartArgs{g.part, g.splits, g.S, g.N, g.S, g.C, g.ldc, 0, g.offsets, g.E}, s);
    }
    if (plan.high) return thin(std::false_type());
    if (any || g.K < 16 || mid > kMostTiles) return launch(gemm_staged<Kind, D, false, true>, 128, 128, 256);
    if (plan.wide) return launch(gemm_big<Kind, D, Tile256, 2, false, false, true>, 256, 256, Tile256::kThreads);
    if (mid <= 256 || g.S <= 128 * groups) return launch(gemm_big<Kind, D, Tile128, 4, false, false, true>, 128, 128, 256);
    return launch(gemm_big<Kind, D, Tile128, 2, false, false, true>, 128, 128, 256);
}

// dB: the parts of an expert's rows, of 64 rows a step on the average.
Cut grad_cut(int64_t S, int32_t E, int64_t M, int64_t N) {
    const auto tiles = [&](int64_t b) { return (M + b - 1) / b * ((N + b - 1) / b) * E; };
    return best_cut(tiles(128), tiles(256), (S / E + 63) / 64, 0.65, 0.0, (double)E * M * N, true, odd(M, N));
}

template <class Kind, class D>
int rows_sum_t(GradArgs g, hipStream_t s) {
    const bool any = ((uintptr_t)g.P | (uintptr_t)g.Q | (uintptr_t)g.ldp | (uintptr_t)g.ldq) % 16 != 0;
    const auto launch = [&](auto kernel, int64_t size, int threads) {
        g.m_tiles = (uint32_t)((g.M + size - 1) / size);
        g.n_tiles = (uint32_t)((g.N + size - 1) / size);
        const int64_t n = (int64_t)g.m_tiles * g.n_tiles * g.splits * g.E;
        if (n >= (int64_t)1 << 31) return SP_ERR_SIZE;
        hipLaunchKernelGGL(kernel, dim3((unsigned)std::min(n, kMostTiles)), dim3(threads), 0, s, g);
        return hipGetLastError() == hipSuccess ? SP_OK : SP_ERR_HIP;
    };
    const int64_t mid = (g.M + 127) / 128 * ((g.N + 127) / 128) * g.E * g.splits;
    const bool wide = grad_cut(g.S, g.E, g.M, g.N).wide;
    const auto go = [&](auto part, auto gather) {
        constexpr bool P = decltype(part)::value, G = decltype(gather)::value;
        return any || mid > kMostTiles ? launch(gemm_rows_sum<Kind, D, Tile128, true, P, G>, 128, 256)
               : wide                  ? launch(gemm_rows_sum<Kind, D, Tile256, false, P, G>, 256, Tile256::kThreads)
                                       : launch(gemm_rows_sum<Kind, D, Tile128, false, P, G>, 128, 256);
    };
    const std::true_type yes{};
    const std::false_type no{};
    const int rc = g.splits > 1 ? (g.src ? go(yes, yes) : go(yes, no)) : (g.src ? go(no, yes) : go(no, no));
    if (rc || g.splits <= 1) return rc;
    return add_parts<D>(PartArgs{g.part, g.splits, g.E * g.M, g.N, g.M, g.C, g.ldc, g.stridec, nullptr, 0}, s);
}

int64_t pre_stride(int64_t N) { return (2 * N + 63) / 64 * 64; }  // rows on 128-byte lines

// Workspace of product_backward, whose two products use it one after the other.
size_t parts_bytes(const Products& p, int64_t M) {
    const int rows = row_plan(p.S, p.E, M, p.K).splits, sums = grad_cut(p.S, p.E, M, p.K).splits;
    const size_t a = rows > 1 ? (size_t)rows * p.S * p.K : 0, b = sums > 1 ? (size_t)sums * p.E * M * p.K : 0;
    return std::max(a, b) * sizeof(float);
}

// dA and dB (either may be NULL) from dC, S x M.
int product_backward(const Products& p, int64_t M, const void* dC, int64_t ldc, void* dA, int64_t ldda, void* dB,
                     int64_t lddb, int64_t stridedb, float* part, hipStream_t s) {
    if (dA && p.S > 0 && p.K > 0) {
        GemmArgs g{p.S, p.K, 2 * M, (const int8_t*)dC, p.S, 2 * ldc, nullptr, nullptr, 1, (const int8_t*)p.B, 2 * p.ldb,
                   2 * p.strideb, nullptr, p.offsets, p.E, dA, ldda};
        const RowPlan plan = row_plan(p.S, p.E, M, p.K);
        g.part = part;
        g.splits = plan.splits;
        const int rc = by_type(p.dtype, [&](auto k, auto d) { return row_gradient_t<decltype(k), decltype(d)>(g, plan, s); });
        if (rc) return rc;
    }
    if (dB && M > 0 && p.K > 0) {
        GradArgs g{p.S, M, p.K, (const int8_t*)dC, 2 * ldc, (const int8_t*)p.A, p.a_rows, 2 * p.lda, p.src,
                   FastDiv::by(p.slots), (uint32_t)std::min<int64_t>(p.a_rows * p.slots, (int64_t)1 << 31), p.offsets, p.E,
                   dB, lddb, stridedb, part, grad_cut(p.S, p.E, M, p.K).splits};
        return by_type(p.dtype, [&](auto k, auto d) { return rows_sum_t<decltype(k), decltype(d)>(g, s); });
    }
    return SP_OK;
}

}  // namespace

size_t moe_gemm_backward_bytes(const Products& p) { return parts_bytes(p, p.N); }

int moe_gemm_backward_device(const Products& p, const void* dC, int64_t ldc, void* dA, int64_t ldda, void* dB,
                             int64_t lddb, int64_t stridedb, void* work, hipStream_t s) {
    return product_backward(p, p.N, dC, ldc, dA, ldda, dB, lddb, stridedb, (float*)work, s);
}

size_t moe_gated_backward_bytes(const Products& p) {
    return parts_bytes(p, 2 * p.N) + (size_t)p.S * pre_stride(p.N) * 2;
}

int moe_gated_backward_device(const Products& p, int32_t act, const void* dH, int64_t ldh, const void* pre, int64_t ldp,
                              void* dA, int64_t ldda, void* dB, int64_t lddb, int64_t stridedb, void* work,
                              hipStream_t s) {
    const int64_t ldd = pre_stride(p.N);
    void* dpre = work;
    float* part = (float*)((char*)work + (size_t)p.S * ldd * 2);
    if (p.S > 0 && p.N > 0) {
        const int64_t chunks = p.S * ((p.N + 7) / 8);
        const unsigned grid = (unsigned)std::min<int64_t>((chunks + 255) / 256, 1 << 14);  // each reads the offsets
        by_type(p.dtype, [&](auto, auto d) {
            typedef decltype(d) D;
            typedef typename D::T T;
            hipLaunchKernelGGL((gate_backward_kernel<D>), dim3(grid), dim3(256), 0, s, p.S, p.N, p.E, p.offsets, act,
                               (const T*)dH, ldh, (const T*)pre, ldp, (T*)dpre, ldd);
            return 0;
        });
        if (hipGetLastError() != hipSuccess) return SP_ERR_HIP;
    }
    return product_backward(p, 2 * p.N, dpre, ldd, dA, ldda, dB, lddb, stridedb, part, s);
}

}  // namespace spx
