// Root-mean-square norm of rows, with the residual's addition before it:
//   s = x + r (rounded to the rows' type; s = x without r)
//   i = 1 / sqrt(mean s^2 + eps),  y = s i w
// y in the rows' type, or as int8 codes with a scale per row as the 8-bit products read them
// (a = max |y|, scale = a / 127, q = rint(127 y / a)); and its gradient, with n = s i and dn = dy w:
//   ds = i (dn - n mean(dn n)) + dsum,  dw = sum over rows of dy n
// The norm is that of the stored sum s, so that the gradient, which has only s, is this function's.
//
// A row's lanes hold it in registers between the sums and the results, so that each
// byte is read and written once; longer rows are read again (from L2).  Sums are fp32, added
// across lanes in a fixed order.  Squares beyond fp32's range: a row whose sum of squares is
// not below 2^120 (or, with an eps near zero, not above 2^-60) is summed again scaled by 2^-96 (2^92).
//
// Memory bounds all of it from some thousand rows on: 16384 x 4096 bf16 with a residual in 92 us (5.8 TB/s, half of
// it writes), without 46, into int8 with a residual 78 (6.0), the gradient with the sum's own 92; rows that share lines with
// their neighbours take longer (48613 x 1091 fp32 with a residual 166, 5.1 TB/s).  One row of 4096 takes 3.2 us.  What rows
// out of range need (sums formed again, codes of s i w, a mean of dy w n) stands in branches that others pass by: at most 2 %.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "moe.h"
#include "rows.h"

namespace spx {

namespace {

constexpr float kTiny = 0x1p-119f;  // rows whose largest magnitude is below it have the scale 0
constexpr int kHeld = 2;            // chunks of a row that a lane holds

struct NormArgs {
    int64_t rows, H;
    const void* X;            // backward: s
    int64_t ldx;
    const void* R;            // or NULL; backward: dsum
    int64_t ldr;
    const void* weight;       // or NULL: ones
    float eps;
    void* sum;                // or NULL
    int64_t lds;
    void* Y;                  // rows, or int8 codes; backward: ds
    int64_t ldy;
    float* scale;             // int8 codes only
    const void* dY;           // backward only, as what follows
    int64_t lddy;
    float* part;              // [parts][part_stride(H)]: sums of dy n over some rows each, or NULL
    float* rstd;              // or NULL: i of every row
};

__host__ __device__ constexpr int64_t part_stride(int64_t n) { return (n + 3) / 4 * 4; }

// The TPR lanes that share a row reduce one or two values at a time, in a fixed order, every lane getting both results.
// Two places in LDS take turns, so that one barrier a call suffices.
template <int TPR>
struct Across {
    static constexpr int kWaves = TPR / 64 > 0 ? TPR / 64 : 1;
    float (*part)[2][kWaves];  // [2]
    int turn;
    template <class F>
    static __device__ __forceinline__ float wave(float v, F f) {
        v = f(v, swz_xor<1>(v));
        v = f(v, swz_xor<2>(v));
        v = f(v, swz_xor<4>(v));
        v = f(v, swz_xor<8>(v));
        if (TPR >= 64) {
            v = f(v, swz_xor<16>(v));
            v = f(__int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0)),
                  __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 32)));
        }
        return v;
    }
    template <class F>
    static __device__ __forceinline__ float waves(const float* v, F f) {
        float w[kWaves];
#pragma unroll
        for (int i = 0; i < kWaves; ++i) w[i] = v[i];
#pragma unroll
        for (int d = 1; d < kWaves; d *= 2)
#pragma unroll
            for (int i = 0; i < kWaves; i += 2 * d) w[i] = f(w[i], w[i + d]);
        return w[0];
    }
    template <class F, class G>
    __device__ __forceinline__ void operator()(float& a, float& b, F f, G g) {
        a = wave(a, f);
        b = wave(b, g);
        if (kWaves > 1) {
            auto& p = part[turn];
            turn ^= 1;
            if ((threadIdx.x & 63) == 0) p[0][threadIdx.x >> 6] = a, p[1][threadIdx.x >> 6] = b;
            __syncthreads();
            a = waves(p[0], f);
            b = waves(p[1], g);
        }
    }
    // One value.
    template <class F>
    __device__ __forceinline__ void operator()(float& a, F f) {
        a = wave(a, f);
        if (kWaves > 1) {
            auto& p = part[turn];
            turn ^= 1;
            if ((threadIdx.x & 63) == 0) p[0][threadIdx.x >> 6] = a;
            __syncthreads();
            a = waves(p[0], f);
        }
    }
};
struct Add {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
// A NaN stays one.
struct Most {
    __device__ __forceinline__ float operator()(float a, float b) const { return a >= b || a != a ? a : b; }
};

// The factor that brings a row's sum of squares into range; 1 where it is there.  2^-60 becomes 2^124, and a row whose
// largest value is 2^-126 2^-68.
__device__ __forceinline__ float range_factor(float ss, float eps) {
    return !(ss < 0x1p120f) ? 0x1p-96f : ss < 0x1p-60f && eps < 0x1p-100f ? 0x1p92f : 1.0f;
}
// i / f for a sum of squares of values that were multiplied by f.
__device__ __forceinline__ float inverse_rms(float ss, float H, float eps, float f) {
    return 1.0f / sqrtf(ss / fmaxf(H, 1.0f) + eps * f * f);
}

// v rounded to D's type; to fp16 on its own, as the compiler fuses a product with the rounding of some of a lane's values
// only (to fp32 and bf16 it cannot).
template <class D>
__device__ __forceinline__ typename D::T rounded(float v) {
    if constexpr (std::is_same<D, F16>::value) return round_alone<D>(v);
    return D::down(v);
}

// N weights from column k on, len of them inside the row.
template <class W, int N>
__device__ __forceinline__ void weights_at(const void* weight, int64_t k, int64_t len, float (&w)[N]) {
    if (!weight) {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = 1.0f;
        return;
    }
    const typename W::T* p = (const typename W::T*)weight + k;
    if (len >= N) {
        typedef typename W::T V __attribute__((ext_vector_type(N), aligned(sizeof(typename W::T))));
        const V v = *reinterpret_cast<const V*>(p);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = W::up(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = i < len ? W::up(p[i]) : 0.0f;
    }
}

// Threads of a workgroup, and rows that it takes at a time.
template <int TPR>
constexpr int kThreads = TPR > 256 ? TPR : 256;
template <int TPR>
constexpr int kRows = kThreads<TPR> / TPR;

template <int TPR>
__device__ __forceinline__ int64_t first_row() {
    const int sub = threadIdx.x / TPR;
    return (int64_t)blockIdx.x * kRows<TPR> + (TPR >= 64 ? __builtin_amdgcn_readfirstlane(sub) : sub);
}

// A chunk of a row, len elements of which are inside.  LINES: whole, and rows lie on 128-byte lines, of which no other
// row has a part: non-temporal.
template <class T, bool LINES>
__device__ __forceinline__ typename Chunk<T>::V norm_load(const T* p, int64_t len) {
    return LINES ? chunk_stream(p) : chunk_load(p, len);
}
template <class T, bool LINES>
__device__ __forceinline__ void norm_store(T* p, int64_t len, typename Chunk<T>::V v) {
    if (LINES)
        chunk_stream(p, v);
    else
        chunk_store(p, len, v);
}

// A workgroup goes over its rows with the next one's loads in flight, and keeps the weights of its columns.
template <class D, class W, int TPR, bool LINES, bool I8>
__global__ __launch_bounds__(kThreads<TPR>) void rms_norm_kernel(NormArgs g) {
    typedef typename D::T T;
    typedef typename Chunk<T>::V V;
    constexpr int N = Chunk<T>::N;
    __shared__ float part[2][2][Across<TPR>::kWaves];
    Across<TPR> across{part, 0};
    const int lane = threadIdx.x % TPR;
    const int64_t chunks = (g.H + N - 1) / N, step = (int64_t)gridDim.x * kRows<TPR>;
    float w[kHeld][N];
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
        if (lane + h * TPR < chunks) weights_at<W, N>(g.weight, (lane + h * TPR) * N, g.H - (lane + h * TPR) * N, w[h]);
    const auto load = [&](const void* p, int64_t ld, int64_t row, int64_t c) {
        return norm_load<T, LINES>((const T*)p + row * ld + c * N, g.H - c * N);
    };
    struct Held {
        V x[kHeld], r[kHeld];
    };
    const auto hold = [&](Held& b, int64_t row) {
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
            if (lane + h * TPR < chunks) {
                b.x[h] = load(g.X, g.ldx, row, lane + h * TPR);
                if (g.R) b.r[h] = load(g.R, g.ldr, row, lane + h * TPR);
            }
    };
    int64_t row = first_row<TPR>();
    Held next;
    if (row < g.rows) hold(next, row);
    for (; row < g.rows; row += step) {
        const Held now = next;
        if (row + step < g.rows) hold(next, row + step);
        T* sum = g.sum ? (T*)g.sum + row * g.lds : nullptr;
        const T* stored = sum ? sum : (const T*)g.X + row * g.ldx;
        float held[kHeld][N];  // s, for codes s w
        float ss = 0.0f, most = 0.0f;
        const auto sums = [&](const float (&s)[N], const float (&t)[N]) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                ss = fmaf(s[i], s[i], ss);
                if (I8) most = Most()(fabsf(t[i]), most);
            }
        };
        const auto reduce = [&] {
            if constexpr (I8)
                across(ss, most, Add(), Most());
            else
                across(ss, Add());
        };
        // s of chunk c, formed and stored; u: its weights; t: s, for codes s w
        const auto first = [&](int64_t c, V v, V q, const float (&u)[N], float (&t)[N]) {
            const int64_t k = c * N, len = g.H - k;
            if (g.R) {
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] = rounded<D>(D::up(v[i]) + D::up(q[i]));
            }
            if (sum) norm_store<T, LINES>(sum + k, len, v);
            float s[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                s[i] = D::up(v[i]);
                t[i] = I8 ? s[i] * u[i] : s[i];
            }
            sums(s, t);
        };
        // s f and s f w of chunk c, from the stored sum
        const auto again = [&](int64_t c, float f, float (&s)[N], float (&t)[N]) {
            const int64_t k = c * N, len = g.H - k;
            const V v = chunk_load(stored + k, len);
            weights_at<W, N>(g.weight, k, len, t);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                s[i] = D::up(v[i]) * f;
                t[i] *= s[i];
            }
        };
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
            if (lane + h * TPR < chunks) first(lane + h * TPR, now.x[h], now.r[h], w[h], held[h]);
        for (int64_t c = lane + kHeld * TPR; c < chunks; c += TPR) {
            float u[N], t[N];
            const V v = load(g.X, g.ldx, row, c);
            if (I8) weights_at<W, N>(g.weight, c * N, g.H - c * N, u);
            first(c, v, g.R ? load(g.R, g.ldr, row, c) : v, u, t);
        }
        reduce();
        const float f = range_factor(ss, g.eps);
        if (f != 1.0f) {  // rare: the same for all lanes of the row
            ss = 0.0f;
            for (int64_t c = lane; c < chunks; c += TPR) {
                float s[N], t[N];
                again(c, f, s, t);
#pragma unroll
                for (int i = 0; i < N; ++i) ss = fmaf(s[i], s[i], ss);
            }
            across(ss, Add());
            most = __builtin_nanf("");
        }
        const float unit = inverse_rms(ss, (float)g.H, g.eps, f), inv = unit * f;
        float before = I8 ? 1.0f : inv, top = 1.0f, by = 1.0f, down = 1.0f;
        bool whole = true, live = false;  // whole: what is held is what the results are made of
        if constexpr (I8) {
            // The codes are those of s w, as the row's i cancels, or of s i w where s w may be out of range: beyond it, or
            // so far below that its bits or its reciprocal are lost though the scale is not 0 (s w is off by 2^-150 then).
            float a = most * unit;
            const uint32_t low = __float_as_uint(0x1p-100f), high = __float_as_uint(0x1p120f);
            if (__float_as_uint(most) - low >= high - low && !((most + 0x1p-149f) * unit < 0.5f * kTiny)) {  // rare as well
                most = 0.0f;
                for (int64_t c = lane; c < chunks; c += TPR) {
                    float s[N], t[N];
                    again(c, inv, s, t);
#pragma unroll
                    for (int i = 0; i < N; ++i) most = Most()(fabsf(t[i]), most);
                }
                across(most, Most());
                a = most;
                down = most < 0x1p120f ? 1.0f : 0x1p-8f;  // 127 times a value stays in range
                most *= down;
                before = inv;
                whole = false;
            }
            live = a >= kTiny && a < __builtin_inff();
            top = live ? most : 1.0f;
            by = 1.0f / top;
            if (lane == 0) g.scale[row] = live ? a / 127.0f : a < kTiny ? 0.0f : __builtin_nanf("");
        }
        // chunk c of the result: t, or its codes
        const auto out = [&](int64_t c, const float (&t)[N]) {
            const int64_t k = c * N, len = g.H - k;
            if constexpr (!I8) {
                V o;
#pragma unroll
                for (int i = 0; i < N; ++i) o[i] = rounded<D>(t[i]);
                norm_store<T, LINES>((T*)g.Y + row * g.ldy + k, len, o);
            } else {
                // adding 1.5 * 2^23 rounds to an integer, ties to even, and leaves it in the low bits;
                // the product with a rounded 1 / top is off by less than 1e-4 of a code: near a half divide
                constexpr float kMagic = 12582912.0f;
                uint32_t n[N];
                float off = 0.0f;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float t127 = t[i] * 127.0f, y = fmaf(t127, by, kMagic);
                    off = fmaxf(off, fabsf(fmaf(t127, by, -(y - kMagic))));
                    n[i] = __float_as_uint(y);
                }
                if (__any(off > 0.4999f)) {
#pragma unroll
                    for (int i = 0; i < N; ++i) n[i] = __float_as_uint(t[i] * 127.0f / top + kMagic);
                }
                typedef uint32_t QU __attribute__((ext_vector_type(N / 4), aligned(1)));
                QU o;
#pragma unroll
                for (int i = 0; i < N; i += 4)
                    o[i / 4] = live ? (n[i] & 255u) | (n[i + 1] & 255u) << 8 | (n[i + 2] & 255u) << 16 | n[i + 3] << 24 : 0u;
                int8_t* q = (int8_t*)g.Y + row * g.ldy + k;
                if (len >= N) {
                    *reinterpret_cast<QU*>(q) = o;
                } else {
#pragma unroll
                    for (int i = 0; i < N - 1; ++i)
                        if (i < len) q[i] = (int8_t)(o[i / 4] >> (8 * (i % 4)));
                }
            }
        };
        // 1 / rms comes before the weight: s w may be out of range where s i w is not
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
            if (whole && lane + h * TPR < chunks) {
                if constexpr (!I8)
#pragma unroll
                    for (int i = 0; i < N; ++i) held[h][i] = held[h][i] * inv * w[h][i];
                out(lane + h * TPR, held[h]);
            }
        for (int64_t c = lane + (whole ? kHeld * TPR : 0); c < chunks; c += TPR) {
            float s[N], t[N];
            again(c, before, s, t);
            if (I8 && !whole)
#pragma unroll
                for (int i = 0; i < N; ++i) t[i] *= down;
            out(c, t);
        }
    }
}

// The gradient.  Rows of up to kHeld chunks a lane are held (PARTS): the next row's loads are in flight while a row is
// worked on, and a lane adds up its columns' dy n over the rows of its workgroup, whose sums go to
// part[blockIdx.x].  Longer rows are read again and leave i in rstd.
template <class D, class W, int TPR, bool LINES, bool PARTS>
__global__ __launch_bounds__(kThreads<TPR>, 3) void rms_norm_backward_kernel(NormArgs g) {
    typedef typename D::T T;
    typedef typename Chunk<T>::V V;
    constexpr int N = Chunk<T>::N, R = kRows<TPR>;
    __shared__ float part[2][2][Across<TPR>::kWaves];
    Across<TPR> across{part, 0};
    const int lane = threadIdx.x % TPR;
    const int64_t chunks = (g.H + N - 1) / N, step = (int64_t)gridDim.x * R;
    float acc[PARTS ? kHeld : 1][N], w[PARTS ? kHeld : 1][N];
#pragma unroll
    for (int h = 0; h < (PARTS ? kHeld : 1); ++h)
#pragma unroll
        for (int i = 0; i < N; ++i) acc[h][i] = w[h][i] = 0.0f;
    const auto weights = [&](int64_t c, float (&v)[N]) { weights_at<W, N>(g.weight, c * N, g.H - c * N, v); };
    if (PARTS)
#pragma unroll
        for (int h = 0; h < (PARTS ? kHeld : 1); ++h)
            if (lane + h * TPR < chunks) weights(lane + h * TPR, w[h]);
    const auto at = [&](const void* p, int64_t ld, int64_t row, int64_t c) { return (const T*)p + row * ld + c * N; };
    const auto load = [&](const T* p, int64_t c) { return norm_load<T, LINES>(p, g.H - c * N); };
    struct Held {
        V x[kHeld], y[kHeld], d[kHeld];
    };
    const auto hold = [&](Held& b, int64_t row) {
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            const int64_t c = lane + h * TPR;
            if (c < chunks) {
                b.x[h] = load(at(g.X, g.ldx, row, c), c);
                b.y[h] = load(at(g.dY, g.lddy, row, c), c);
                if (g.R) b.d[h] = load(at(g.R, g.ldr, row, c), c);
            }
        }
    };
    int64_t row = first_row<TPR>();
    Held next;
    if (PARTS && row < g.rows) hold(next, row);
    for (; row < g.rows; row += step) {
        const Held now = next;
        if (PARTS && row + step < g.rows) hold(next, row + step);
        float ss = 0.0f, dot = 0.0f;  // of (s f)^2 and of dn s f
        const auto sums = [&](const V& vx, const V& vy, const float (&u)[N], float f) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float s = D::up(vx[i]) * f;
                ss = fmaf(s, s, ss);
                dot = fmaf(D::up(vy[i]) * u[i], s, dot);
            }
        };
        const auto rest = [&](float f) {
            for (int64_t c = lane; c < chunks; c += TPR) {
                float u[N];
                weights(c, u);
                sums(chunk_load(at(g.X, g.ldx, row, c), g.H - c * N), chunk_load(at(g.dY, g.lddy, row, c), g.H - c * N), u, f);
            }
        };
        if (PARTS) {
#pragma unroll
            for (int h = 0; h < (PARTS ? kHeld : 1); ++h)
                if (lane + h * TPR < chunks) sums(now.x[h], now.y[h], w[h], 1.0f);
        } else {
            rest(1.0f);
        }
        across(ss, dot, Add(), Add());
        const float f = range_factor(ss, g.eps);
        const bool ranged = f == 1.0f && fabsf(dot) < 0x1p120f;
        if (!ranged) {  // rare: dn s may be out of range where dn n is not
            if (f != 1.0f) {
                ss = 0.0f;
                rest(f);
                across(ss, Add());
            }
            const float all = ss;
            dot = 0.0f;
            rest(inverse_rms(ss, (float)g.H, g.eps, f) * f);
            across(dot, Add());
            ss = all;
        }
        const float unit = inverse_rms(ss, (float)g.H, g.eps, f), inv = unit * f;
        const float mean = dot * (ranged ? unit : 1.0f) / (float)g.H;  // of dn n
        if (!PARTS && g.rstd && lane == 0) g.rstd[row] = inv;
        const auto out = [&](int64_t c, const V& vx, const V& vy, const V& vd, const float (&u)[N], float (&sum)[N]) {
            V o;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float n = D::up(vx[i]) * inv, dy = D::up(vy[i]);
                float v = inv * fmaf(-n, mean, dy * u[i]);
                if (g.R) v += D::up(vd[i]);
                o[i] = rounded<D>(v);
                sum[i] = fmaf(dy, n, sum[i]);
            }
            norm_store<T, LINES>((T*)g.Y + row * g.ldy + c * N, g.H - c * N, o);
        };
        if (PARTS) {
#pragma unroll
            for (int h = 0; h < (PARTS ? kHeld : 1); ++h)
                if (lane + h * TPR < chunks) out(lane + h * TPR, now.x[h], now.y[h], now.d[h], w[h], acc[h]);
        } else {
            for (int64_t c = lane; c < chunks; c += TPR) {
                const int64_t len = g.H - c * N;
                const V vx = chunk_load(at(g.X, g.ldx, row, c), len), vy = chunk_load(at(g.dY, g.lddy, row, c), len);
                weights(c, w[0]);
                out(c, vx, vy, g.R ? chunk_load(at(g.R, g.ldr, row, c), len) : vx, w[0], acc[0]);
            }
        }
    }
    if constexpr (PARTS) {
        if (!g.part) return;
        typedef float F4 __attribute__((ext_vector_type(4)));
        F4* to = reinterpret_cast<F4*>(g.part + (int64_t)blockIdx.x * part_stride(g.H));
        const int64_t quads = part_stride(g.H) / 4;
        if constexpr (R == 1) {
#pragma unroll
            for (int h = 0; h < kHeld; ++h)
#pragma unroll
                for (int i = 0; i < N; i += 4) {
                    const int64_t q = (int64_t)(lane + h * TPR) * (N / 4) + i / 4;
                    if (q < quads) to[q] = F4{acc[h][i], acc[h][i + 1], acc[h][i + 2], acc[h][i + 3]};
                }
        } else {
            // what the workgroup's R rows at a time came to, added in their order
            constexpr int kQuads = TPR * kHeld * N / 4;
            __shared__ F4 all[R][kQuads];
#pragma unroll
            for (int h = 0; h < kHeld; ++h)
#pragma unroll
                for (int i = 0; i < N; i += 4)
                    all[threadIdx.x / TPR][(lane + h * TPR) * (N / 4) + i / 4] = F4{acc[h][i], acc[h][i + 1], acc[h][i + 2], acc[h][i + 3]};
            __syncthreads();
            for (int q = threadIdx.x; q < quads; q += kThreads<TPR>) {
                F4 v = all[0][q];
                for (int j = 1; j < R; ++j) v += all[j][q];
                to[q] = v;
            }
        }
    }
}

// part[blockIdx.y] = the sums over a range of rows of dy s i, i from rstd; a thread a column.
template <class D>
__global__ __launch_bounds__(256) void norm_columns_kernel(NormArgs g, int64_t each) {
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= g.H) return;
    const int64_t from = blockIdx.y * each, to = min(from + each, g.rows);
    const typename D::T *x = (const typename D::T*)g.X + k, *y = (const typename D::T*)g.dY + k;
    float v = 0.0f;
#pragma unroll 4
    for (int64_t r = from; r < to; ++r) v = fmaf(D::up(y[r * g.lddy]), D::up(x[r * g.ldx]) * g.rstd[r], v);
    g.part[blockIdx.y * part_stride(g.H) + k] = v;
}

// dweight = the parts' sum: 16 columns a workgroup, 64 threads to four of them, each every 64th part, added in order.
__global__ __launch_bounds__(256) void norm_parts_kernel(const float* __restrict__ part, int64_t parts, int64_t H,
                                                         float* __restrict__ dweight) {
    typedef float F4 __attribute__((ext_vector_type(4)));
    __shared__ F4 all[64][4];
    const int c = threadIdx.x & 3, r = threadIdx.x >> 2;
    const int64_t k = (int64_t)blockIdx.x * 16 + 4 * c, ld = part_stride(H);
    F4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (k < H)
#pragma unroll 8
        for (int64_t p = r; p < parts; p += 64) v += *reinterpret_cast<const F4*>(part + p * ld + k);
    all[r][c] = v;
    __syncthreads();
    if (threadIdx.x >= 16) return;
    const float* f = reinterpret_cast<const float*>(all) + threadIdx.x;
    float sum = 0.0f;
#pragma unroll 16
    for (int j = 0; j < 64; ++j) sum += f[16 * j];
    const int64_t at = (int64_t)blockIdx.x * 16 + threadIdx.x;
    if (at < H) dweight[at] = sum;
}

// ---------------------------------------------------------------- launch
int status(hipError_t e) { return e == hipSuccess ? SP_OK : SP_ERR_HIP; }
int chunk_of(int32_t dtype) { return dtype == SP_F32 ? 4 : 8; }
// Lanes a row: the fewest whose registers hold it, up to 1024; the gradient's, which hold more, up to 512.  us with 16, 64,
// 256, 512 and 1024, bf16: 65536 x 128 9.8, 21, 70, 129, 274; 32768 x 1024 28, 24, 45, 75, 142; 16384 x 2048 32, 31, 26, 42, 75;
// 8192 x 8192 71, 71, 56, 44, 64; 4096 x 16384 125, 68, 60, 57, 46; one row of 4096 18, 5.5, 3.2, 3.2, 3.3.  A row that is a
// little longer than what some lanes hold leaves the next ones half idle: 65536 x 264 16, 23; 4096 x 8200 27 with 512, 33 with 1024.
// The gradient: 32768 x 1024 39 with 64, 91 with 256; 16384 x 4096 76 with 256, 111 with 512.
constexpr int kMostForward = 1024, kMostBackward = 512;
int norm_lanes(int64_t H, int32_t dtype, int most) {
    const int64_t chunks = (H + chunk_of(dtype) - 1) / chunk_of(dtype);
    for (const int lanes : {16, 64, 256, 512})
        if (chunks <= lanes * kHeld) return lanes;
    return most;
}
// Whether the gradient's lanes hold a row.  Longer ones, above 8192 in 16 bits and 4096 in fp32, are read twice by their
// workgroup, the second time from the caches in part, and dweight's sums read both operands once more, a thread a column: 4096 x 16384 bf16 152 us,
// without dweight 100 (1.6 times the time of one read of each and one write at 5.6 TB/s, 72); 8192 x 8192 fp32 298, 191 (144).
// Held rows read again so: 8192 x 8192 bf16 144 us instead of 91, without dweight 90 instead of 76; 8192 x 4096 fp32 136 instead of 72.
bool held(int64_t H, int32_t dtype) { return (H + chunk_of(dtype) - 1) / chunk_of(dtype) <= kMostBackward * kHeld; }
// Whether rows are whole lines that no other row shares.
bool on_lines(const void* p, int64_t ld, int64_t H, int32_t dtype) {
    const int64_t size = dtype == SP_F32 ? 4 : 2;
    return ((uintptr_t)p | (uintptr_t)(ld * size) | (uintptr_t)(H * size)) % 128 == 0;
}

// Workgroups; more rows take several rounds (us with 1024 and 4096: 16384 x 4096 bf16 without a residual 46.1, 46.1,
// int8 with one 78, 80; 3000 x 16384 37.6, 46.6, int8 71, 82; 48613 x 1091 fp32 with a residual 166, 179).  Whole lines of
// four streams, two of them written, want more: 16384 x 4096 bf16 with a residual 95, 92; 65536 x 512 46.5, 45.6.
constexpr int64_t kMostGroups = 1024, kMostFour = 4096;

// Workgroups of the gradient, and so parts of dweight, which have to be written and read; rows that share lines
// with their neighbours want more of them (us with 512 and 1024: 16384 x 4096 bf16 92, 108, 65536 x 512 48, 60; 48613 x 1091
// fp32 254, 172).  lines: whether they do not; the workspace has room for either.
int64_t backward_groups(int64_t rows, int64_t H, int32_t dtype, bool lines) {
    const int lanes = norm_lanes(H, dtype, kMostBackward), per = std::max(256, lanes) / lanes;
    return std::min<int64_t>((rows + per - 1) / per, lines || rows < 4096 ? 512 : 1024);
}
// Rows a part of norm_columns_kernel.
int64_t column_rows(int64_t rows) { return std::max<int64_t>(16, (rows + 255) / 256); }

template <int L>
struct Lanes {
    static constexpr int value = L;
};
// go(type, weight's type, lanes, on lines)
template <int MOST, class Go>
int norm_by(int32_t dtype, int32_t w_type, int64_t H, bool lines, Go go) {
    const auto lanes = [&](auto d, auto w) {
        const int n = norm_lanes(H, dtype, MOST);
        const auto with = [&](auto l) { return lines ? go(d, w, l, std::true_type()) : go(d, w, l, std::false_type()); };
        return n == 16    ? go(d, w, Lanes<16>(), std::false_type())
               : n == 64  ? with(Lanes<64>())
               : n == 256 ? with(Lanes<256>())
               : n == 512 ? with(Lanes<512>())
                          : with(Lanes<MOST>());
    };
    if (dtype == SP_F32) return lanes(F32(), F32());
    if (dtype == SP_BF16) return w_type == SP_F32 ? lanes(Bf16(), F32()) : lanes(Bf16(), Bf16());
    return w_type == SP_F32 ? lanes(F16(), F32()) : lanes(F16(), F16());
}

}  // namespace

int rms_norm_device(const NormRows& n, void* sum, int64_t lds, void* Y, int64_t ldy, float* scale, hipStream_t s) {
    NormArgs g{};
    g.rows = n.rows, g.H = n.H, g.X = n.X, g.ldx = n.ldx, g.R = n.R, g.ldr = n.ldr, g.weight = n.weight, g.eps = n.eps;
    g.sum = sum, g.lds = lds, g.Y = Y, g.ldy = ldy, g.scale = scale;
    const bool lines = on_lines(n.X, n.ldx, n.H, n.dtype) && on_lines(n.R, n.R ? n.ldr : 0, n.H, n.dtype) &&
                       on_lines(sum, sum ? lds : 0, n.H, n.dtype) && (scale || on_lines(Y, ldy, n.H, n.dtype));
    return norm_by<kMostForward>(n.dtype, n.w_type, n.H, lines, [&](auto d, auto w, auto l, auto on) {
        typedef decltype(d) D;
        typedef decltype(w) W;
        constexpr int L = decltype(l)::value;
        constexpr bool kLines = decltype(on)::value;
        const dim3 grid((unsigned)std::min<int64_t>((g.rows + kRows<L> - 1) / kRows<L>, kLines && n.R && !scale ? kMostFour : kMostGroups));
        if (scale)
            hipLaunchKernelGGL((rms_norm_kernel<D, W, L, kLines, true>), grid, dim3(kThreads<L>), 0, s, g);
        else
            hipLaunchKernelGGL((rms_norm_kernel<D, W, L, kLines, false>), grid, dim3(kThreads<L>), 0, s, g);
        return status(hipGetLastError());
    });
}

size_t rms_norm_backward_bytes(int64_t rows, int64_t H, int32_t dtype) {
    if (held(H, dtype)) return (size_t)backward_groups(rows, H, dtype, false) * part_stride(H) * sizeof(float);
    const int64_t each = column_rows(rows);
    return ((size_t)part_stride(rows) + (size_t)((rows + each - 1) / each) * part_stride(H)) * sizeof(float);
}

int rms_norm_backward_device(const NormRows& n, const void* dY, int64_t lddy, void* dX, int64_t lddx, float* dweight,
                             void* work, hipStream_t s) {
    NormArgs g{};
    g.rows = n.rows, g.H = n.H, g.X = n.X, g.ldx = n.ldx, g.R = n.R, g.ldr = n.ldr, g.weight = n.weight, g.eps = n.eps;
    g.dY = dY, g.lddy = lddy, g.Y = dX, g.ldy = lddx;
    const bool whole = held(n.H, n.dtype);
    const bool lines = whole && on_lines(n.X, n.ldx, n.H, n.dtype) && on_lines(n.R, n.R ? n.ldr : 0, n.H, n.dtype) &&
                       on_lines(dY, lddy, n.H, n.dtype) && on_lines(dX, lddx, n.H, n.dtype);
    const int64_t each = column_rows(n.rows);
    const int64_t parts = n.rows == 0 ? 0 : whole ? backward_groups(n.rows, n.H, n.dtype, lines) : (n.rows + each - 1) / each;
    float* const part = (float*)work + (whole ? 0 : part_stride(n.rows));
    if (dweight) {
        g.part = part;
        if (!whole) g.rstd = (float*)work;
    }
    if (n.rows > 0) {
        const int rc = norm_by<kMostBackward>(n.dtype, n.w_type, n.H, lines, [&](auto d, auto w, auto l, auto on) {
            typedef decltype(d) D;
            typedef decltype(w) W;
            constexpr int L = decltype(l)::value;
            constexpr bool kLines = decltype(on)::value;
            if (whole) {
                hipLaunchKernelGGL((rms_norm_backward_kernel<D, W, L, kLines, true>), dim3((unsigned)parts), dim3(kThreads<L>), 0,
                                   s, g);
            } else if constexpr (L == kMostBackward && !kLines) {
                hipLaunchKernelGGL((rms_norm_backward_kernel<D, W, L, false, false>),
                                   dim3((unsigned)std::min<int64_t>(g.rows, kMostGroups)), dim3(kThreads<L>), 0, s, g);
                const int rc = status(hipGetLastError());
                if (rc || !g.rstd) return rc;
                hipLaunchKernelGGL((norm_columns_kernel<D>), dim3((unsigned)((g.H + 255) / 256), (unsigned)parts), dim3(256), 0, s,
                                   g, each);
            }
            return status(hipGetLastError());
        });
        if (rc) return rc;
    }
    if (!dweight) return SP_OK;
    hipLaunchKernelGGL(norm_parts_kernel, dim3((unsigned)((n.H + 15) / 16)), dim3(256), 0, s, part, parts, n.H, dweight);
    return status(hipGetLastError());
}

}  // namespace spx
