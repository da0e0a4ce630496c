// Tokens sorted by expert and back: the counting sort, the rows moved into
// sorted order, the weighted sum back, and the gradient of that sum.
//
// With n = T * slots slots, slot f = t * slots + j of token t, and ids[f] its
// expert, the sort is the COO -> CSR step of this library with expert ids as
// rows (count, prefix sum, stable placement), and the row movements are
// products with the n-entry sparse matrix it describes:
//   dispatch          Xs = P X         P[pos[f], f / slots] = 1
//   combine           Y  = W Ys        W[f / slots, pos[f]] = weights[f]
//   combine backward  dYs = W^T dY,    dweights = the products dY Ys^T
//                     sampled at W's entries
// Every kernel works from the token's side (pos), so a token's row is read or
// written once however many experts it goes to.  Sums are held in fp32, in
// slot order; nothing is added with atomics.
#include <algorithm>

#include "device_common.h"
#include "moe.h"
#include "rows.h"

namespace spx {

namespace {

// ---------------------------------------------------------------- counting sort
constexpr int kSortThreads = 1024;   // 512 above kSortWideE experts, whose counts would not fit 64 KB of LDS
constexpr int kSortWideE = 512;
constexpr int kSortOneBlock = 4096;  // up to this many slots one workgroup does everything (6.9 us; two kernels 8.4)

// The floor is bytes that take a microsecond; what the sort takes is its chain
// of dependent steps: 3.8 us for one token's 8 slots, 3.0 (counts) + 10.4
// (placement) for 524288 slots over 128 experts.
//
// Workgroups of the two-kernel path: 1024 slots each up to 128 of them (16384
// slots 8.6 us, 9.5 with 4096 each), then up to 256 (524288 slots 12.9 us with
// 128, 13.5 with 256).  Every workgroup of the second kernel reads all counts,
// so that kSortHist bounds them.
constexpr int kSortHist = 1 << 17;

int sort_blocks(int64_t n, int32_t E) {
    if (n <= kSortOneBlock) return 1;
    const int64_t nb = std::min<int64_t>((n + 1023) / 1024, std::max<int64_t>(128, std::min<int64_t>(256, n / 4096)));
    return (int)std::min<int64_t>(nb, kSortHist / E);  // at least 128
}

__global__ __launch_bounds__(kSortThreads) void moe_count_kernel(const int32_t* __restrict__ ids, int64_t n, int E,
                                                                 int64_t per_block, int32_t* __restrict__ hist) {
    extern __shared__ int32_t lds[];
    for (int e = threadIdx.x; e < E; e += kSortThreads) lds[e] = 0;
    __syncthreads();
    const int64_t b = blockIdx.x * per_block, end = min(b + per_block, n);
#pragma unroll 4
    for (int64_t f = b + threadIdx.x; f < end; f += kSortThreads) {
        const int id = ids[f];
        if ((unsigned)id < (unsigned)E) atomicAdd(&lds[id], 1);  // integers: the order does not matter
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kSortThreads) hist[(int64_t)blockIdx.x * E + e] = lds[e];
}

// Slots f, f + 64, .. (up to end), loaded together; -1 behind the end.
constexpr int kSortBatch = 4;
__device__ __forceinline__ void load_ids(const int32_t* __restrict__ ids, int64_t f, int64_t end,
                                         int (&id)[kSortBatch]) {
#pragma unroll
    for (int b = 0; b < kSortBatch; ++b) id[b] = ids[min(f + 64 * b, end - 1)];
#pragma unroll
    for (int b = 0; b < kSortBatch; ++b)
        if (f + 64 * b >= end) id[b] = -1;
}

// Inclusive prefix sum over the 64 lanes.
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(v, d, 64);
        if (lane >= d) v += u;
    }
    return v;
}

// Places the slots of workgroup b's range.  LDS: cnt[waves][E] (counts of each
// wave's own range, then the place of its next slot of each expert), start[E]
// (the expert's first place), tot and before [groups][E2].
// Wave w owns one contiguous piece of the range and takes it 64 slots at a
// time in order; inside a step the lanes with the same id are found by one
// ballot per id bit, and a slot's place is the wave's running place plus the
// number of equal ids in lower lanes.  So places ascend with the slot index.
__global__ __launch_bounds__(kSortThreads) void moe_place_kernel(const int32_t* __restrict__ ids, int64_t n, int E,
                                                                 int E2, int id_bits, int64_t per_block,
                                                                 const int32_t* __restrict__ hist,
                                                                 int32_t* __restrict__ offsets,
                                                                 int32_t* __restrict__ src,
                                                                 int32_t* __restrict__ pos) {
    extern __shared__ int32_t lds[];
    const int tid = threadIdx.x, nth = blockDim.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6), nw = nth >> 6;
    int32_t* cnt = lds;             // [nw][E]
    int32_t* start = cnt + nw * E;  // [E + 1]
    int32_t* tot = start + E + 1;   // [groups][E2], hist only
    const int nb = gridDim.x;
    for (int i = tid; i < nw * E; i += nth) cnt[i] = 0;
    __syncthreads();

    const int64_t b = blockIdx.x * per_block, end = min(b + per_block, n);
    const int64_t per_wave = (per_block + 64 * nw - 1) / (64 * nw) * 64;
    const int64_t wb = min(b + w * per_wave, end), we = min(wb + per_wave, end);
    int32_t* mine = cnt + w * E;
    for (int64_t f0 = wb; f0 < we; f0 += 64 * kSortBatch) {
        int id[kSortBatch];
        load_ids(ids, f0 + lane, we, id);
#pragma unroll
        for (int b = 0; b < kSortBatch; ++b)
            if ((unsigned)id[b] < (unsigned)E) atomicAdd(&mine[id[b]], 1);
    }
    // slots of each expert in all workgroups and in the earlier ones
    const int groups = hist ? max(1, nth / E2) : 0;
    int32_t* before = tot + groups * E2;
    for (int i = tid; i < groups * E2; i += nth) {
        const int g = i / E2, e = i % E2;
        int all = 0, early = 0;
        if (e < E)
#pragma unroll 8
            for (int r = g; r < nb; r += groups) {
                const int v = hist[(int64_t)r * E + e];
                all += v;
                early += r < (int)blockIdx.x ? v : 0;
            }
        tot[i] = all;
        before[i] = early;
    }
    __syncthreads();
    // start[e] := slots of expert e (all workgroups)
    for (int e = tid; e < E; e += nth) {
        int s = 0;
        if (hist) {
            for (int g = 0; g < groups; ++g) s += tot[g * E2 + e];
        } else {
#pragma unroll
            for (int v = 0; v < kSortThreads / 64; ++v) s += v < nw ? cnt[v * E + e] : 0;
        }
        start[e] = s;
    }
    __syncthreads();
    if (w == 0) {  // exclusive prefix sum over the experts
        int carry = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int v = e0 + lane < E ? start[e0 + lane] : 0;
            const int s = wave_scan(v, lane);
            if (e0 + lane < E) start[e0 + lane] = carry + s - v;
            carry += __shfl(s, 63, 64);
        }
        if (lane == 0) start[E] = carry;
    }
    __syncthreads();
    // cnt[v][e] := place of the first slot of expert e in wave v's piece
    for (int e = tid; e < E; e += nth) {
        int p = start[e];
        if (hist)
            for (int g = 0; g < groups; ++g) p += before[g * E2 + e];
        int c[kSortThreads / 64];  // all loads first
#pragma unroll
        for (int v = 0; v < kSortThreads / 64; ++v) c[v] = v < nw ? cnt[v * E + e] : 0;
#pragma unroll
        for (int v = 0; v < kSortThreads / 64; ++v) {
            if (v < nw) cnt[v * E + e] = p;
            p += c[v];
        }
    }
    if (blockIdx.x == 0)
        for (int e = tid; e <= E; e += nth) offsets[e] = start[e];
    __syncthreads();

    for (int64_t f0 = wb; f0 < we; f0 += 64 * kSortBatch) {
        int ids4[kSortBatch];
        load_ids(ids, f0 + lane, we, ids4);
#pragma unroll
        for (int b = 0; b < kSortBatch; ++b) {
            const int64_t f = f0 + 64 * b + lane;
            const int id = ids4[b];
            const bool live = (unsigned)id < (unsigned)E;
            uint64_t same = __ballot(live);
            if (same == 0) {  // nothing routed in this step (or behind the end)
                if (f < we) pos[f] = -1;
                continue;
            }
            for (int k = 0; k < id_bits; ++k) {
                const uint64_t m = __ballot((id >> k) & 1);
                same &= ((id >> k) & 1) ? m : ~m;
            }
            const int rank = __popcll(same & ((1ull << lane) - 1));
            const int p = mine[live ? id : 0] + rank;
            __builtin_amdgcn_wave_barrier();  // the wave's lanes have all read it
            if (live) {
                if (rank == 0) mine[id] = p + __popcll(same);
                src[p] = (int32_t)f;
                pos[f] = p;
            } else if (f < we) {
                pos[f] = -1;
            }
            __builtin_amdgcn_wave_barrier();
        }
    }
    // the places behind the last routed slot
    for (int64_t p = start[E] + (int64_t)blockIdx.x * nth + tid; p < n; p += (int64_t)nb * nth) src[p] = -1;
}

// ---------------------------------------------------------------- rows
// TPR lanes share a token, 256 / TPR tokens a workgroup.  A token's slots are
// taken U at a time: their places first, then the U rows' chunks, all in
// flight together.  A slot routed nowhere is made to read the first row (there
// is one, or no row is live) and its bits are zeroed, so that the loads need
// no branch; its weight counts as zero.
//
// Memory bounds all three: 16384 x 4 rows of 4096 bf16 dispatched in 124 us
// (5.4 TB/s, four fifths writes), combined in 112 (6.0), their gradients formed
// in 226 (5.3); a copy reaches 5.6 TB/s.
//
// A row's last chunk starts at H - N where a whole one does not fit: it then
// repeats elements of the chunk before it, which are written twice with the
// same value (and counted once in the products of the gradient).  Only rows
// shorter than one chunk (kShort) go element by element.
//
// Where every row starts on a 128-byte line the loads are non-temporal (kStream; each
// byte is read once: combine of 16384 x 8 rows of 2048 fp16 98 us, 115
// without), and with 256 lanes a token the stores too (kStreamBoth; dispatch of 16384 x 4
// rows of 4096 bf16 123 us, 129 without; rows of 1024 by 64 lanes 66, 63
// without).  Rows that start inside a line share lines with their neighbours,
// which only the caches put together: dispatch of 30000 x 6 rows of 333 fp16
// 41 us non-temporal, 25 without.
struct RowArgs {
    int64_t T, H, S, ld_tok, ld_row;
    int32_t slots;
    bool lines;  // every row starts on a 128-byte line
};
enum Access { kShort, kCached, kStream, kStreamBoth };

template <int TPR>
__device__ __forceinline__ int64_t first_token() {
    const int sub = threadIdx.x / TPR;
    // a wave's lanes share the token: its places and weights are then scalar loads
    return (int64_t)blockIdx.x * (256 / TPR) + (TPR >= 64 ? __builtin_amdgcn_readfirstlane(sub) : sub);
}

// Places of slots [j0, j0 + U) of token t, -1 where there is none.
template <int U>
__device__ __forceinline__ void places(const RowArgs& a, const int32_t* __restrict__ pos, int64_t t, int j0,
                                       int (&q)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int p = pos[t * a.slots + min(j0 + u, a.slots - 1)];
        q[u] = j0 + u < a.slots && (unsigned)p < (unsigned)a.S ? p : -1;
    }
}

template <class D, Access A>
__device__ __forceinline__ typename Chunk<typename D::T>::V row_load(const RowArgs& a, const typename D::T* p) {
    if (A == kShort) return chunk_load(p, a.H);
    return A == kCached ? chunk_load(p, Chunk<typename D::T>::N) : chunk_stream(p);
}
template <class D, Access A>
__device__ __forceinline__ void row_store(const RowArgs& a, typename D::T* p, typename Chunk<typename D::T>::V v) {
    if (A == kStreamBoth)
        chunk_stream(p, v);
    else
        chunk_store(p, A == kShort ? a.H : Chunk<typename D::T>::N, v);
}

// The chunk at element k of the rows of U slots, zeros for a slot routed nowhere.
template <class D, int U, Access A>
__device__ __forceinline__ void slot_rows(const RowArgs& a, const typename D::T* __restrict__ Ys, int64_t ld, int64_t k,
                                          const int (&q)[U], typename Chunk<typename D::T>::V (&y)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) y[u] = row_load<D, A>(a, Ys + max(q[u], 0) * ld + k);
#pragma unroll
    for (int u = 0; u < U; ++u) y[u] = q[u] >= 0 ? y[u] : typename Chunk<typename D::T>::V(0);
}

template <class D, int TPR, Access A>
__global__ __launch_bounds__(256) void moe_dispatch_kernel(RowArgs a, const typename D::T* __restrict__ X,
                                                           const int32_t* __restrict__ pos,
                                                           typename D::T* __restrict__ Xs) {
    constexpr int N = Chunk<typename D::T>::N, U = 4;
    const int64_t step = (int64_t)gridDim.y * TPR;
    for (int64_t t = first_token<TPR>(); t < a.T; t += (int64_t)gridDim.x * (256 / TPR))
        for (int64_t c = (int64_t)blockIdx.y * TPR + threadIdx.x % TPR; c * N < a.H; c += step) {
            const int64_t k = A == kShort ? 0 : min(c * N, a.H - N);
            const auto v = row_load<D, A>(a, X + t * a.ld_tok + k);
            for (int j0 = 0; j0 < a.slots; j0 += U) {
                int q[U];
                places<U>(a, pos, t, j0, q);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (q[u] >= 0) row_store<D, A>(a, Xs + q[u] * a.ld_row + k, v);
            }
        }
}

// weights NULL: all ones (a product with 1 is exact).
template <class D, int TPR, int U, Access A>
__global__ __launch_bounds__(256) void moe_combine_kernel(RowArgs a, const typename D::T* __restrict__ Ys,
                                                          const int32_t* __restrict__ pos,
                                                          const float* __restrict__ weights,
                                                          typename D::T* __restrict__ Y) {
    typedef typename D::T T;
    constexpr int N = Chunk<T>::N;
    const int64_t step = (int64_t)gridDim.y * TPR;
    for (int64_t t = first_token<TPR>(); t < a.T; t += (int64_t)gridDim.x * (256 / TPR))
        for (int64_t c = (int64_t)blockIdx.y * TPR + threadIdx.x % TPR; c * N < a.H; c += step) {
            const int64_t k = A == kShort ? 0 : min(c * N, a.H - N);
            float acc[N];
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = 0.0f;
            for (int j0 = 0; j0 < a.slots; j0 += U) {
                int q[U];
                float w[U];
                typename Chunk<T>::V y[U];
                places<U>(a, pos, t, j0, q);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float v = weights ? weights[t * a.slots + min(j0 + u, a.slots - 1)] : 1.0f;
                    w[u] = q[u] >= 0 ? v : 0.0f;
                }
                slot_rows<D, U, A>(a, Ys, a.ld_row, k, q, y);
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < N; ++i) acc[i] = fmaf(w[u], D::up(y[u][i]), acc[i]);
            }
            typename Chunk<T>::V o;
#pragma unroll
            for (int i = 0; i < N; ++i) o[i] = D::down(acc[i]);
            row_store<D, A>(a, Y + t * a.ld_tok + k, o);
        }
}

// TPR lanes form the products of a token's dY with U of its rows at a time and
// add them across the lanes in a fixed order.
template <class D, int TPR, int U, Access A>
__global__ __launch_bounds__(256) void moe_combine_backward_kernel(RowArgs a, const typename D::T* __restrict__ dY,
                                                                   const typename D::T* __restrict__ Ys, int64_t ld_ys,
                                                                   const int32_t* __restrict__ pos,
                                                                   const float* __restrict__ weights,
                                                                   typename D::T* __restrict__ dYs,
                                                                   float* __restrict__ dweights) {
    typedef typename D::T T;
    constexpr int N = Chunk<T>::N;
    __shared__ float part[4][U];
    const int lane = threadIdx.x % TPR;
    for (int64_t t = first_token<TPR>(); t < a.T; t += (int64_t)gridDim.x * (256 / TPR))
        for (int j0 = 0; j0 < a.slots; j0 += U) {
            int q[U];
            float w[U], dot[U];
            places<U>(a, pos, t, j0, q);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                w[u] = weights[t * a.slots + min(j0 + u, a.slots - 1)];
                dot[u] = 0.0f;
            }
            for (int64_t c = lane; c * N < a.H; c += TPR) {
                const int64_t k = A == kShort ? 0 : min(c * N, a.H - N);
                const auto g = row_load<D, A>(a, dY + t * a.ld_tok + k);
                typename Chunk<T>::V y[U];
                slot_rows<D, U, A>(a, Ys, ld_ys, k, q, y);
                float f[N];
#pragma unroll
                for (int i = 0; i < N; ++i) f[i] = D::up(g[i]);
                // what the chunk before holds already counts as zero in the products, on both sides (0 * Inf is NaN)
                const int again = (int)(c * N - k);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    typename Chunk<T>::V o;
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const float d = fmaf(f[i], D::up(y[u][i]), dot[u]);
                        dot[u] = i >= again ? d : dot[u];
                        o[i] = D::down(w[u] * f[i]);
                    }
                    if (q[u] >= 0) row_store<D, A>(a, dYs + q[u] * a.ld_row + k, o);
                }
            }
            if (TPR == 256) __syncthreads();  // part[] of the slots before has been read
#pragma unroll
            for (int u = 0; u < U; ++u) {
                dot[u] = group_sum(dot[u], TPR < 64 ? TPR : 64);
                if (TPR == 256 && (threadIdx.x & 63) == 0) part[threadIdx.x >> 6][u] = dot[u];
            }
            if (TPR == 256) __syncthreads();
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (lane == u && j0 + u < a.slots) {
                    const float d = TPR == 256 ? (part[0][u] + part[1][u]) + (part[2][u] + part[3][u]) : dot[u];
                    dweights[t * a.slots + j0 + u] = q[u] >= 0 ? d : 0.0f;
                }
        }
}

constexpr int64_t kMaxGrid = 1 << 20;  // larger problems take several rounds of the grid

// Lanes per token: 16, 64 or 256, so that none takes more than `each` chunks
// where 256 suffice for that.  The row movements take one (grid.y cuts longer
// rows); the gradient two, to spread its reduction over more of the row
// (65536 x 2 rows of 1024 bf16 104 us with a wave per token, 126 with four;
// 16384 x 4 rows of 4096 239 with one, 222 with four).
template <class D>
int lanes(int64_t H, int each) {
    const int64_t chunks = (H + Chunk<typename D::T>::N - 1) / Chunk<typename D::T>::N;
    return chunks <= 16 * each ? 16 : chunks <= 64 * each ? 64 : 256;
}

// Tokens in x; with few of them rows are cut over y (16 x 8 rows of 4096 bf16
// combined in 3.5 us, uncut 4.4).  Many tokens fill the chip by themselves,
// and a workgroup then takes whole rows (dispatch of 16384 x 4 rows of 4096
// 123 us, cut 132).
template <class D>
dim3 rows_grid(const RowArgs& a, int tpr) {
    const int64_t rpb = 256 / tpr, per = (int64_t)Chunk<typename D::T>::N * tpr;
    return dim3((unsigned)std::min<int64_t>((a.T + rpb - 1) / rpb, kMaxGrid),
                (unsigned)(a.T >= 2048 ? 1 : std::min<int64_t>((a.H + per - 1) / per, 1024)));
}

bool on_lines(const void* p, int64_t ld, int32_t dtype) {
    return ((uintptr_t)p | (uintptr_t)(ld * (dtype == SP_F32 ? 4 : 2))) % 128 == 0;
}

// go(shape) with the lanes and the kind of access as compile-time constants
template <int L, Access A>
struct Shape {
    static constexpr int lanes = L;
    static constexpr Access access = A;
};
template <class D, class Go>
void by_shape(int lanes, const RowArgs& a, Go go) {
    if (a.H < Chunk<typename D::T>::N)
        go(Shape<16, kShort>{});
    else if (lanes == 16)
        go(Shape<16, kCached>{});
    else if (lanes == 64)
        a.lines ? go(Shape<64, kStream>{}) : go(Shape<64, kCached>{});
    else
        a.lines ? go(Shape<256, kStreamBoth>{}) : go(Shape<256, kCached>{});
}

template <class D>
hipError_t dispatch_t(const RowArgs& a, const void* X, const int32_t* pos, void* Xs, hipStream_t s) {
    by_shape<D>(lanes<D>(a.H, 1), a, [&](auto c) {
        typedef decltype(c) C;
        hipLaunchKernelGGL((moe_dispatch_kernel<D, C::lanes, C::access>), rows_grid<D>(a, C::lanes), dim3(256), 0, s, a,
                           (const typename D::T*)X, pos, (typename D::T*)Xs);
    });
    return hipGetLastError();
}

template <class D, int U>
hipError_t combine_u(const RowArgs& a, const void* Ys, const int32_t* pos, const float* weights, void* Y,
                     hipStream_t s) {
    by_shape<D>(lanes<D>(a.H, 1), a, [&](auto c) {
        typedef decltype(c) C;
        hipLaunchKernelGGL((moe_combine_kernel<D, C::lanes, U, C::access>), rows_grid<D>(a, C::lanes), dim3(256), 0, s,
                           a, (const typename D::T*)Ys, pos, weights, (typename D::T*)Y);
    });
    return hipGetLastError();
}

template <class D>
hipError_t combine_t(const RowArgs& a, const void* Ys, const int32_t* pos, const float* weights, void* Y,
                     hipStream_t s) {
    return a.slots <= 2   ? combine_u<D, 2>(a, Ys, pos, weights, Y, s)
           : a.slots <= 4 ? combine_u<D, 4>(a, Ys, pos, weights, Y, s)
                          : combine_u<D, 8>(a, Ys, pos, weights, Y, s);
}

template <class D, int U>
hipError_t combine_backward_u(const RowArgs& a, const void* dY, const void* Ys, int64_t ld_ys, const int32_t* pos,
                              const float* weights, void* dYs, float* dweights, hipStream_t s) {
    by_shape<D>(lanes<D>(a.H, 2), a, [&](auto c) {
        typedef decltype(c) C;
        const int64_t rpb = 256 / C::lanes;
        hipLaunchKernelGGL((moe_combine_backward_kernel<D, C::lanes, U, C::access>),
                           dim3((unsigned)std::min<int64_t>((a.T + rpb - 1) / rpb, kMaxGrid)), dim3(256), 0, s, a,
                           (const typename D::T*)dY, (const typename D::T*)Ys, ld_ys, pos, weights, (typename D::T*)dYs,
                           dweights);
    });
    return hipGetLastError();
}

template <class D>
hipError_t combine_backward_t(const RowArgs& a, const void* dY, const void* Ys, int64_t ld_ys, const int32_t* pos,
                              const float* weights, void* dYs, float* dweights, hipStream_t s) {
    return a.slots <= 2   ? combine_backward_u<D, 2>(a, dY, Ys, ld_ys, pos, weights, dYs, dweights, s)
           : a.slots <= 4 ? combine_backward_u<D, 4>(a, dY, Ys, ld_ys, pos, weights, dYs, dweights, s)
                          : combine_backward_u<D, 8>(a, dY, Ys, ld_ys, pos, weights, dYs, dweights, s);
}

int status(hipError_t e) { return e == hipSuccess ? SP_OK : SP_ERR_HIP; }

}  // namespace

size_t moe_sort_work_bytes(int64_t n, int32_t E) {
    const int nb = sort_blocks(n, E);
    return nb > 1 ? (size_t)nb * E * sizeof(int32_t) : 0;
}

int moe_sort_device(int64_t n, int32_t E, const int32_t* ids, int32_t* offsets, int32_t* src, int32_t* pos,
                    void* work, hipStream_t s) {
    const int nb = sort_blocks(n, E);
    int bits = 1;
    while ((1 << bits) < E) ++bits;
    int32_t* hist = nb > 1 ? (int32_t*)work : nullptr;
    const int64_t per_block = nb > 1 ? (n + nb - 1) / nb : n;
    if (hist) {
        hipLaunchKernelGGL(moe_count_kernel, dim3(nb), dim3(kSortThreads), E * sizeof(int32_t), s, ids, n, E, per_block,
                           hist);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return SP_ERR_HIP;
    }
    const int most = E > kSortWideE ? kSortThreads / 2 : kSortThreads;
    const int threads = (int)std::min<int64_t>(most, std::max<int64_t>(64, (n + 63) / 64 * 64));
    int E2 = 64;
    while (E2 < E) E2 *= 2;
    const int groups = hist ? std::max(1, threads / E2) : 0;
    const size_t lds = ((size_t)(threads / 64) * E + E + 1 + 2 * (size_t)groups * E2) * sizeof(int32_t);
    hipLaunchKernelGGL(moe_place_kernel, dim3(nb), dim3(threads), lds, s, ids, n, E, E2, bits, per_block, hist, offsets,
                       src, pos);
    return status(hipGetLastError());
}

int moe_dispatch_device(int64_t T, int32_t slots, int64_t H, int64_t S, int32_t dtype, const void* X, int64_t ldx,
                        const int32_t* pos, void* Xs, int64_t lds, hipStream_t s) {
    const RowArgs a{T, H, S, ldx, lds, slots, on_lines(X, ldx, dtype) && on_lines(Xs, lds, dtype)};
    if (dtype == SP_F32) return status(dispatch_t<F32>(a, X, pos, Xs, s));
    if (dtype == SP_BF16) return status(dispatch_t<Bf16>(a, X, pos, Xs, s));
    return status(dispatch_t<F16>(a, X, pos, Xs, s));
}

int moe_combine_device(int64_t T, int32_t slots, int64_t H, int64_t S, int32_t dtype, const void* Ys, int64_t lds,
                       const int32_t* pos, const float* weights, void* Y, int64_t ldy, hipStream_t s) {
    const RowArgs a{T, H, S, ldy, lds, slots, on_lines(Y, ldy, dtype) && on_lines(Ys, lds, dtype)};
    if (S == 0) Ys = Y;  // no slot is live: what is read in their place is thrown away
    if (dtype == SP_F32) return status(combine_t<F32>(a, Ys, pos, weights, Y, s));
    if (dtype == SP_BF16) return status(combine_t<Bf16>(a, Ys, pos, weights, Y, s));
    return status(combine_t<F16>(a, Ys, pos, weights, Y, s));
}

int moe_combine_backward_device(int64_t T, int32_t slots, int64_t H, int64_t S, int32_t dtype, const void* dY,
                                int64_t ldy, const void* Ys, int64_t lds, const int32_t* pos, const float* weights,
                                void* dYs, int64_t ldd, float* dweights, hipStream_t s) {
    const RowArgs a{T, H, S, ldy, ldd, slots,
                    on_lines(dY, ldy, dtype) && on_lines(Ys, lds, dtype) && on_lines(dYs, ldd, dtype)};
    if (S == 0) Ys = dY;  // as in moe_combine_device
    if (dtype == SP_F32) return status(combine_backward_t<F32>(a, dY, Ys, lds, pos, weights, dYs, dweights, s));
    if (dtype == SP_BF16) return status(combine_backward_t<Bf16>(a, dY, Ys, lds, pos, weights, dYs, dweights, s));
    return status(combine_backward_t<F16>(a, dY, Ys, lds, pos, weights, dYs, dweights, s));
}

}  // namespace spx
