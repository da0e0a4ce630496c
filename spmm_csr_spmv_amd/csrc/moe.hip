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
#include "rows.h"

namespace spx {

namespace {

// ---------------------------------------------------------------- counting sort
constexpr int kSortThreads = 1024;   // 512 above kSortWideE experts, whose counts would not fit 64 KB of LDS
constexpr int kSortWideE = 512;
constexpr int kSortChunk = 4096;     // slots per workgroup, at least (more when the grid is at its cap)
constexpr int kSortOneBlock = 8192;  // up to this many slots one workgroup does everything

// Workgroups of the two-kernel path.  Every workgroup of the second kernel
// reads all counts, so their number is bounded by kSortHist.
constexpr int kSortMaxBlocks = 256;
constexpr int kSortHist = 1 << 16;

int sort_blocks(int64_t n, int32_t E) {
    if (n <= kSortOneBlock) return 1;
    int64_t nb = (n + kSortChunk - 1) / kSortChunk;
    const int64_t cap = std::max<int64_t>(8, std::min<int64_t>(kSortMaxBlocks, kSortHist / E));
    return (int)std::min(nb, cap);
}

__global__ __launch_bounds__(kSortThreads) void moe_count_kernel(const int32_t* __restrict__ ids, int64_t n, int E,
                                                                 int64_t per_block, int32_t* __restrict__ hist) {
    extern __shared__ int32_t lds[];
    for (int e = threadIdx.x; e < E; e += kSortThreads) lds[e] = 0;
    __syncthreads();
    const int64_t b = blockIdx.x * per_block, end = min(b + per_block, n);
    for (int64_t f = b + threadIdx.x; f < end; f += kSortThreads) {
        const int id = ids[f];
        if ((unsigned)id < (unsigned)E) atomicAdd(&lds[id], 1);  // integers: the order does not matter
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kSortThreads) hist[(int64_t)blockIdx.x * E + e] = lds[e];
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
    for (int64_t f = wb + lane; f < we; f += 64) {
        const int id = ids[f];
        if ((unsigned)id < (unsigned)E) atomicAdd(&mine[id], 1);
    }
    // slots of each expert in all workgroups and in the earlier ones
    const int groups = hist ? max(1, nth / E2) : 0;
    int32_t* before = tot + groups * E2;
    for (int i = tid; i < groups * E2; i += nth) {
        const int g = i / E2, e = i % E2;
        int all = 0, early = 0;
        if (e < E)
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
        if (hist)
            for (int g = 0; g < groups; ++g) s += tot[g * E2 + e];
        else
            for (int v = 0; v < nw; ++v) s += cnt[v * E + e];
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
        for (int v = 0; v < nw; ++v) {
            const int c = cnt[v * E + e];
            cnt[v * E + e] = p;
            p += c;
        }
    }
    if (blockIdx.x == 0)
        for (int e = tid; e <= E; e += nth) offsets[e] = start[e];
    __syncthreads();

    for (int64_t f0 = wb; f0 < we; f0 += 64) {
        const int64_t f = f0 + lane;
        const int id = f < we ? ids[f] : -1;
        const bool live = (unsigned)id < (unsigned)E;
        uint64_t same = __ballot(live);
        for (int k = 0; k < id_bits; ++k) {
            const uint64_t m = __ballot((id >> k) & 1);
            same &= ((id >> k) & 1) ? m : ~m;
        }
        if (live) {
            const int rank = __popcll(same & ((1ull << lane) - 1));
            const int p = mine[id] + rank;
            if (rank == 0) mine[id] = p + __popcll(same);  // the wave's lanes have all read it
            src[p] = (int32_t)f;
            pos[f] = p;
        } else if (f < we) {
            pos[f] = -1;
        }
        __builtin_amdgcn_wave_barrier();
    }
    // the places behind the last routed slot
    for (int64_t p = start[E] + (int64_t)blockIdx.x * nth + tid; p < n; p += (int64_t)nb * nth) src[p] = -1;
}

// ---------------------------------------------------------------- rows
// A workgroup of 256 threads takes 256 / tpr tokens; tpr lanes (a power of
// two) share a token's row, and blockIdx.y cuts the row when tpr lanes of one
// chunk do not cover it.
struct RowArgs {
    int64_t T, H, S, ld_tok, ld_row;
    int32_t slots;
    int32_t tpr_log;
};

template <class D>
__global__ __launch_bounds__(256) void moe_dispatch_kernel(RowArgs a, const typename D::T* __restrict__ X,
                                                           const int32_t* __restrict__ pos,
                                                           typename D::T* __restrict__ Xs) {
    typedef typename D::T T;
    constexpr int N = Chunk<T>::N;
    const int rpb = 256 >> a.tpr_log, sub = threadIdx.x >> a.tpr_log, lane = threadIdx.x & ((1 << a.tpr_log) - 1);
    const int64_t step = (int64_t)gridDim.y << a.tpr_log;
    for (int64_t t = (int64_t)blockIdx.x * rpb + sub; t < a.T; t += (int64_t)gridDim.x * rpb) {
        const int32_t* p = pos + t * a.slots;
        for (int64_t c = ((int64_t)blockIdx.y << a.tpr_log) + lane; c * N < a.H; c += step) {
            const auto v = chunk_load(X + t * a.ld_tok + c * N, a.H - c * N);
            for (int j = 0; j < a.slots; ++j) {
                const int q = p[j];
                if (q >= 0 && q < a.S) chunk_store(Xs + q * a.ld_row + c * N, a.H - c * N, v);
            }
        }
    }
}

template <class D, bool W>
__global__ __launch_bounds__(256) void moe_combine_kernel(RowArgs a, const typename D::T* __restrict__ Ys,
                                                          const int32_t* __restrict__ pos,
                                                          const float* __restrict__ weights,
                                                          typename D::T* __restrict__ Y) {
    typedef typename D::T T;
    constexpr int N = Chunk<T>::N;
    const int rpb = 256 >> a.tpr_log, sub = threadIdx.x >> a.tpr_log, lane = threadIdx.x & ((1 << a.tpr_log) - 1);
    const int64_t step = (int64_t)gridDim.y << a.tpr_log;
    for (int64_t t = (int64_t)blockIdx.x * rpb + sub; t < a.T; t += (int64_t)gridDim.x * rpb) {
        const int32_t* p = pos + t * a.slots;
        const float* w = weights + t * a.slots;
        for (int64_t c = ((int64_t)blockIdx.y << a.tpr_log) + lane; c * N < a.H; c += step) {
            float acc[N];
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = 0.0f;
            for (int j = 0; j < a.slots; ++j) {
                const int q = p[j];
                if (q < 0 || q >= a.S) continue;
                const auto v = chunk_load(Ys + q * a.ld_row + c * N, a.H - c * N);
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] = W ? fmaf(w[j], D::up(v[i]), acc[i]) : acc[i] + D::up(v[i]);
            }
            typename Chunk<T>::V o;
#pragma unroll
            for (int i = 0; i < N; ++i) o[i] = D::down(acc[i]);
            chunk_store(Y + t * a.ld_tok + c * N, a.H - c * N, o);
        }
    }
}

// One workgroup per token: the token's dY row times each of its expert rows.
template <class D>
__global__ __launch_bounds__(256) void moe_combine_backward_kernel(RowArgs a, const typename D::T* __restrict__ dY,
                                                                   const typename D::T* __restrict__ Ys, int64_t ld_ys,
                                                                   const int32_t* __restrict__ pos,
                                                                   const float* __restrict__ weights,
                                                                   typename D::T* __restrict__ dYs,
                                                                   float* __restrict__ dweights) {
    typedef typename D::T T;
    constexpr int N = Chunk<T>::N;
    __shared__ float part[4];
    const int tid = threadIdx.x;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        for (int j = 0; j < a.slots; ++j) {
            const int q = pos[t * a.slots + j];
            const bool live = q >= 0 && q < a.S;
            float dot = 0.0f;
            if (live) {
                const float w = weights[t * a.slots + j];
                for (int64_t c = tid; c * N < a.H; c += 256) {
                    const auto g = chunk_load(dY + t * a.ld_tok + c * N, a.H - c * N);
                    const auto y = chunk_load(Ys + q * ld_ys + c * N, a.H - c * N);
                    typename Chunk<T>::V o;
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        dot = fmaf(D::up(g[i]), D::up(y[i]), dot);
                        o[i] = D::down(w * D::up(g[i]));
                    }
                    chunk_store(dYs + q * a.ld_row + c * N, a.H - c * N, o);
                }
            }
            dot = wave_sum(dot);
            if ((tid & 63) == 0) part[tid >> 6] = dot;
            __syncthreads();
            if (tid == 0) dweights[t * a.slots + j] = live ? (part[0] + part[1]) + (part[2] + part[3]) : 0.0f;
            __syncthreads();
        }
    }
}

// Lanes per token: the power of two that covers the row with one chunk a lane, 8 to 256.
int lanes_log(int64_t H, int elems) {
    const int64_t chunks = (H + elems - 1) / elems;
    int l = 3;
    while (l < 8 && ((int64_t)1 << l) < chunks) ++l;
    return l;
}

constexpr int64_t kMaxGrid = 1 << 20;  // larger problems take several rounds of the grid

template <class D>
dim3 rows_grid(const RowArgs& a) {
    constexpr int N = Chunk<typename D::T>::N;
    const int64_t rpb = 256 >> a.tpr_log;
    const int64_t per = (int64_t)N << a.tpr_log;
    return dim3((unsigned)std::min<int64_t>((a.T + rpb - 1) / rpb, kMaxGrid),
                (unsigned)std::min<int64_t>((a.H + per - 1) / per, 1024));
}

template <class D>
hipError_t dispatch_t(RowArgs a, const void* X, const int32_t* pos, void* Xs, hipStream_t s) {
    a.tpr_log = lanes_log(a.H, Chunk<typename D::T>::N);
    hipLaunchKernelGGL((moe_dispatch_kernel<D>), rows_grid<D>(a), dim3(256), 0, s, a, (const typename D::T*)X, pos,
                       (typename D::T*)Xs);
    return hipGetLastError();
}

template <class D>
hipError_t combine_t(RowArgs a, const void* Ys, const int32_t* pos, const float* weights, void* Y, hipStream_t s) {
    a.tpr_log = lanes_log(a.H, Chunk<typename D::T>::N);
    auto kernel = weights ? moe_combine_kernel<D, true> : moe_combine_kernel<D, false>;
    hipLaunchKernelGGL(kernel, rows_grid<D>(a), dim3(256), 0, s, a, (const typename D::T*)Ys, pos, weights,
                       (typename D::T*)Y);
    return hipGetLastError();
}

template <class D>
hipError_t combine_backward_t(RowArgs a, const void* dY, const void* Ys, int64_t ld_ys, const int32_t* pos,
                              const float* weights, void* dYs, float* dweights, hipStream_t s) {
    hipLaunchKernelGGL((moe_combine_backward_kernel<D>), dim3((unsigned)std::min(a.T, kMaxGrid)), dim3(256), 0, s, a,
                       (const typename D::T*)dY, (const typename D::T*)Ys, ld_ys, pos, weights, (typename D::T*)dYs,
                       dweights);
    return hipGetLastError();
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
    const RowArgs a{T, H, S, ldx, lds, slots, 0};
    if (dtype == SP_F32) return status(dispatch_t<F32>(a, X, pos, Xs, s));
    if (dtype == SP_BF16) return status(dispatch_t<Bf16>(a, X, pos, Xs, s));
    return status(dispatch_t<F16>(a, X, pos, Xs, s));
}

int moe_combine_device(int64_t T, int32_t slots, int64_t H, int64_t S, int32_t dtype, const void* Ys, int64_t lds,
                       const int32_t* pos, const float* weights, void* Y, int64_t ldy, hipStream_t s) {
    const RowArgs a{T, H, S, ldy, lds, slots, 0};
    if (dtype == SP_F32) return status(combine_t<F32>(a, Ys, pos, weights, Y, s));
    if (dtype == SP_BF16) return status(combine_t<Bf16>(a, Ys, pos, weights, Y, s));
    return status(combine_t<F16>(a, Ys, pos, weights, Y, s));
}

int moe_combine_backward_device(int64_t T, int32_t slots, int64_t H, int64_t S, int32_t dtype, const void* dY,
                                int64_t ldy, const void* Ys, int64_t lds, const int32_t* pos, const float* weights,
                                void* dYs, int64_t ldd, float* dweights, hipStream_t s) {
    const RowArgs a{T, H, S, ldy, ldd, slots, 0};
    if (dtype == SP_F32) return status(combine_backward_t<F32>(a, dY, Ys, lds, pos, weights, dYs, dweights, s));
    if (dtype == SP_BF16) return status(combine_backward_t<Bf16>(a, dY, Ys, lds, pos, weights, dYs, dweights, s));
    return status(combine_backward_t<F16>(a, dY, Ys, lds, pos, weights, dYs, dweights, s));
}

}  // namespace spx
