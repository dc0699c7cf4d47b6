// gdn_norm.hip -- layer norm and RMS norm over rows, forward and backward.
//
// Forward, per row of D values: xh = (x - mean) rstd with rstd = 1 /
// sqrt(var + eps) (RMS: mean = 0, rstd = 1 / sqrt(mean(x^2) + eps)), y = xh
// weight + bias.  The row stays in registers, so the variance is summed from
// the differences to the mean, and x is read once.
// Backward, with q = dy weight: dx = rstd (q - mean(q) - xh mean(q xh)) (RMS:
// without mean(q)) + d_residual, dweight = sum over rows of dy xh, dbias = sum
// of dy.  A work-group keeps its columns' sums of all its rows in registers
// and leaves them once; a second kernel adds the work-groups' sums in order.
// Everything is in 32 bits between the loads and the stores.
// Bound: HBM, and the launch where there are few rows (1 x 2048: 3.1 us).
#include "gdn_device.hpp"
#include "gdn_kernels.hpp"

namespace gdn {

namespace {

// W adjacent elements as they lie in memory, element aligned
template <bool BF16, int W>
struct Run {
    static constexpr int kWords = BF16 ? W / 2 : W;
    typedef uint32_t V __attribute__((ext_vector_type(kWords), aligned(BF16 ? 2 : 4)));
    V v;
    __device__ __forceinline__ void load(const void* p, int64_t at) {
        v = *reinterpret_cast<const V*>(static_cast<const uint8_t*>(p) + at * (BF16 ? 2 : 4));
    }
    __device__ __forceinline__ void load_once(const void* p, int64_t at) {
        v = __builtin_nontemporal_load(reinterpret_cast<const V*>(static_cast<const uint8_t*>(p) + at * (BF16 ? 2 : 4)));
    }
    __device__ __forceinline__ float get(int e) const {
        if constexpr (BF16) return __uint_as_float(e % 2 ? v[e / 2] & 0xFFFF0000u : v[e / 2] << 16);
        else return __uint_as_float(v[e]);
    }
    __device__ __forceinline__ static void store(void* p, int64_t at, const float* f) {
        V o;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (BF16) {
                const f32x2 t = {f[2 * i], f[2 * i + 1]};
                o[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(t, bf16x2));
            } else {
                o[i] = __float_as_uint(f[i]);
            }
        }
        __builtin_nontemporal_store(o, reinterpret_cast<V*>(static_cast<uint8_t*>(p) + at * (BF16 ? 2 : 4)));
    }
};

template <bool BF16>
__device__ __forceinline__ float load_one(const void* p, int64_t at) {
    if constexpr (BF16) return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[at]);
    else return static_cast<const float*>(p)[at];
}
template <bool BF16>
__device__ __forceinline__ void store_one(void* p, int64_t at, float f) {
    if constexpr (BF16) static_cast<uint16_t*>(p)[at] = f32_to_bf16_bits(f);
    else static_cast<float*>(p)[at] = f;
}

// Columns of a thread: NV runs of W, T threads to a row.  Run j begins at
// column W (t + T j), but never past D - W: the last runs of a row whose D is
// no multiple of their columns begin earlier and repeat columns that another
// thread (or run) has too.  Those count once: fresh() tells.  So no load has a
// condition, and both threads store them, with the same bits: in these kernels no
// product is joined with a sum but by fmaf (left to the compiler that differs
// from run to run, and the bits with it; stored by one thread only, 300000 x 100
// in bf16 backward takes 48 us instead of 44).  (D >= W; where NV > 1 more than half of a row's runs are needed,
// so the first half of a thread's are whole.)
template <int W, int T, int NV>
struct Columns {
    int at[NV], from[NV];                     // first column; the first that counts here (at + W: none)
    __device__ __forceinline__ void init(int t, int64_t D) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = static_cast<int64_t>(W) * (t + T * j);
            at[j] = static_cast<int>(c + W <= D ? c : D - W);
            from[j] = static_cast<int>(c < D ? c : D);
        }
    }
    __device__ __forceinline__ bool fresh(int j, int e) const { return (NV > 1 && j < NV / 2) || at[j] + e >= from[j]; }
    __device__ __forceinline__ bool any(int j, int64_t D) const { return (NV > 1 && j < NV / 2) || from[j] < D; }

    // A value of p for each column (NULL: `none`), and one to each that counts
    // here, four at a time (16 x 8192 in bf16, backward: one by one 17 us, so 8;
    // 32768 x 4096, forward and backward: 279 and 265).
    __device__ __forceinline__ void load(const float* p, float none, float* v) const {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int g = 0; g < W / 4; ++g) {
                Run<false, 4> q;
                if (p) q.load(p, at[j] + 4 * g);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[W * j + 4 * g + e] = p ? q.get(e) : none;
            }
    }
    __device__ __forceinline__ void store(float* p, const float* v) const {
        typedef float V __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if ((NV > 1 && j < NV / 2) || from[j] == at[j]) {
#pragma unroll
                for (int g = 0; g < W / 4; ++g)
                    *reinterpret_cast<V*>(p + at[j] + 4 * g) = V{v[W * j + 4 * g], v[W * j + 4 * g + 1], v[W * j + 4 * g + 2], v[W * j + 4 * g + 3]};
            } else {
#pragma unroll
                for (int e = 0; e < W; ++e)
                    if (fresh(j, e)) p[at[j] + e] = v[W * j + e];
            }
        }
    }
};

// Sums of N values over the T threads of a row, in every one of them.  red:
// one of two places in LDS, in turn (a wave that is a sum ahead writes the
// other one).
template <int T, int N>
__device__ __forceinline__ void row_sums(float* s, float* red, int t) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (T <= 16) {
            s[i] = group_sum<T>(s[i]);
        } else if constexpr (T == 32) {
            s[i] = group_sum<16>(s[i]);
            s[i] += __shfl_xor(s[i], 16, kWave);
        } else {
            s[i] = wave_sum(s[i]);
        }
    }
    if constexpr (T > kWave) {
        constexpr int kW = T / kWave;
        if (t % kWave == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) red[i * kW + t / kWave] = s[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            s[i] = red[i * kW];
#pragma unroll
            for (int w = 1; w < kW; ++w) s[i] += red[i * kW + w];
        }
    }
}

constexpr int rows_of(int T) { return T < 256 ? 256 / T : 1; }   // rows that a work-group holds at a time

// The rows all at once: one block of them a work-group (more only where the
// grid would be past what a launch holds).  4096 x 2048 in fp32 to bf16: 9.4 us
// with the call (the kernel 8.4, 6.0 TB/s), 12.3 with work-groups that stay.
// MASK: D is not W T NV.
template <bool XB, bool YB, bool MASK, int T, int NV>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_row_kernel(NormParams p) {
#pragma clang fp contract(off)
    constexpr int W = XB && YB ? 8 : 4, R = rows_of(T);
    __shared__ float red[2][T > kWave ? T / kWave : 1];
    const int t = threadIdx.x % T;
    Columns<W, T, NV> cols;
    cols.init(t, p.D);
    const float per = 1.f / static_cast<float>(p.D);
    int turn = 0;
    for (int64_t m0 = static_cast<int64_t>(blockIdx.x) * R; m0 < p.M; m0 += static_cast<int64_t>(gridDim.x) * R) {
        int64_t m = m0 + threadIdx.x / T;
        const bool real = R == 1 || m < p.M;
        if (!real) m = p.M - 1;
        Run<XB, W> x[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) x[j].load_once(p.x, m * p.xs + cols.at[j]);
        float s[1] = {0.f}, mean = 0.f;
        if (p.center) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < W; ++e) s[0] += !MASK || cols.fresh(j, e) ? x[j].get(e) : 0.f;
            row_sums<T, 1>(s, red[turn], t);
            turn ^= 1;
            mean = s[0] / static_cast<float>(p.D);   // (a constant row has differences of 0)
            s[0] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float d = !MASK || cols.fresh(j, e) ? x[j].get(e) - mean : 0.f;
                s[0] = fmaf(d, d, s[0]);
            }
        row_sums<T, 1>(s, red[turn], t);
        turn ^= 1;
        const float rstd = 1.f / sqrtf(fmaf(s[0], per, p.eps));
        if (!real) continue;
        if (t == 0 && p.stats) {
            p.stats[m] = mean;
            p.stats[p.M + m] = rstd;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (MASK && !cols.any(j, p.D)) continue;
            float f[W];
#pragma unroll
            for (int e = 0; e < W; ++e) f[e] = (x[j].get(e) - mean) * rstd;
#pragma unroll
            for (int g = 0; g < W / 4; ++g) {
                if (p.weight) {
                    Run<false, 4> w;
                    w.load(p.weight, cols.at[j] + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[4 * g + e] *= w.get(e);
                }
                if (p.bias) {
                    Run<false, 4> b;
                    b.load(p.bias, cols.at[j] + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[4 * g + e] += b.get(e);
                }
            }
            Run<YB, W>::store(p.y, m * p.ys + cols.at[j], f);
        }
    }
}

// Many long rows: a work-group takes every gridDim-th block of them and keeps
// its columns' weights in registers (read again for each row they are several
// times the row's own bytes), the next row on its way while one is summed.
// 32768 x 4096 in bf16: 89 to 123 us (4.4 to 6.0 TB/s), 131 with a wave a row.
template <bool XB, bool YB, bool MASK, int T, int NV>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_forward_kernel(NormParams p) {
#pragma clang fp contract(off)
    constexpr int W = XB && YB ? 8 : 4, R = rows_of(T), C = W * NV;
    __shared__ float red[2][R][T > kWave ? T / kWave : 1];
    const int t = threadIdx.x % T, r = threadIdx.x / T;
    Columns<W, T, NV> cols;
    cols.init(t, p.D);
    float w[C], b[C];
    cols.load(p.weight, 1.f, w);
    cols.load(p.bias, 0.f, b);
    const float per = 1.f / static_cast<float>(p.D);
    int turn = 0;
    // (rows past the end read the last one)
    auto row_at = [&](int64_t m0) { return m0 + r < p.M ? m0 + r : p.M - 1; };
    Run<XB, W> x[NV], next[NV];
    int64_t m0 = static_cast<int64_t>(blockIdx.x) * R;
#pragma unroll
    for (int j = 0; j < NV; ++j) next[j].load_once(p.x, row_at(m0) * p.xs + cols.at[j]);
    for (; m0 < p.M; m0 += static_cast<int64_t>(gridDim.x) * R) {
        const int64_t m = row_at(m0), m1 = row_at(m0 + static_cast<int64_t>(gridDim.x) * R);
        const bool real = R == 1 || m0 + r < p.M;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            x[j] = next[j];
            next[j].load_once(p.x, m1 * p.xs + cols.at[j]);
        }
        float s[1] = {0.f}, mean = 0.f;
        if (p.center) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < W; ++e) s[0] += !MASK || cols.fresh(j, e) ? x[j].get(e) : 0.f;
            row_sums<T, 1>(s, red[turn][r], t);
            turn ^= 1;
            mean = s[0] / static_cast<float>(p.D);   // (a constant row has differences of 0)
            s[0] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float d = !MASK || cols.fresh(j, e) ? x[j].get(e) - mean : 0.f;
                s[0] = fmaf(d, d, s[0]);
            }
        row_sums<T, 1>(s, red[turn][r], t);
        turn ^= 1;
        const float rstd = 1.f / sqrtf(fmaf(s[0], per, p.eps));
        if (!real) continue;
        if (t == 0 && p.stats) {
            p.stats[m] = mean;
            p.stats[p.M + m] = rstd;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (MASK && !cols.any(j, p.D)) continue;
            float f[W];
#pragma unroll
            for (int e = 0; e < W; ++e) f[e] = fmaf((x[j].get(e) - mean) * rstd, w[W * j + e], b[W * j + e]);
            Run<YB, W>::store(p.y, m * p.ys + cols.at[j], f);
        }
    }
}

// Rows of fewer than eight values: a thread to a row (2^20 x 7 in
// fp32: 23 us with the call, 1690 with a work-group a row).
constexpr int kNarrow = 7, kNarrowThreads = 256;

// x[c], or 0 past the row's end (whose loads are not done)
template <bool BF16>
__device__ __forceinline__ void load_narrow(const void* p, int64_t at, int D, float* x) {
#pragma unroll
    for (int c = 0; c < kNarrow; ++c) x[c] = c < D ? load_one<BF16>(p, at + c) : 0.f;
}

template <bool XB, bool YB>
__global__ __launch_bounds__(kNarrowThreads) void norm_narrow_kernel(NormParams p) {
    const int D = static_cast<int>(p.D);
    const float per = 1.f / static_cast<float>(p.D);
    for (int64_t m = static_cast<int64_t>(blockIdx.x) * kNarrowThreads + threadIdx.x; m < p.M;
         m += static_cast<int64_t>(gridDim.x) * kNarrowThreads) {
        float x[kNarrow], mean = 0.f, s = 0.f;
        load_narrow<XB>(p.x, m * p.xs, D, x);
        if (p.center) {
#pragma unroll
            for (int c = 0; c < kNarrow; ++c) s += x[c];
            mean = s / static_cast<float>(p.D);      // (a constant row has differences of 0)
            s = 0.f;
        }
#pragma unroll
        for (int c = 0; c < kNarrow; ++c) {
            const float d = c < D ? x[c] - mean : 0.f;
            s = fmaf(d, d, s);
        }
        const float rstd = 1.f / sqrtf(fmaf(s, per, p.eps));
        if (p.stats) {
            p.stats[m] = mean;
            p.stats[p.M + m] = rstd;
        }
#pragma unroll
        for (int c = 0; c < kNarrow; ++c) {
            if (c >= D) break;
            float f = (x[c] - mean) * rstd;
            if (p.weight) f *= p.weight[c];
            if (p.bias) f += p.bias[c];
            store_one<YB>(p.y, m * p.ys + c, f);
        }
    }
}

// Rows that no work-group can hold: read again for each step (from the L2).
constexpr int kLongThreads = 512;

template <bool XB, bool YB>
__global__ __launch_bounds__(kLongThreads) void norm_forward_long_kernel(NormParams p) {
    __shared__ float red[2][kLongThreads / kWave];
    const int t = threadIdx.x;
    const float per = 1.f / static_cast<float>(p.D);
    int turn = 0;
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        float s[1] = {0.f}, mean = 0.f;
        if (p.center) {
            for (int64_t c = t; c < p.D; c += kLongThreads) s[0] += load_one<XB>(p.x, m * p.xs + c);
            row_sums<kLongThreads, 1>(s, red[turn], t);
            turn ^= 1;
            mean = s[0] / static_cast<float>(p.D);   // (a constant row has differences of 0)
            s[0] = 0.f;
        }
        for (int64_t c = t; c < p.D; c += kLongThreads) {
            const float d = load_one<XB>(p.x, m * p.xs + c) - mean;
            s[0] = fmaf(d, d, s[0]);
        }
        row_sums<kLongThreads, 1>(s, red[turn], t);
        turn ^= 1;
        const float rstd = 1.f / sqrtf(fmaf(s[0], per, p.eps));
        if (t == 0 && p.stats) {
            p.stats[m] = mean;
            p.stats[p.M + m] = rstd;
        }
        for (int64_t c = t; c < p.D; c += kLongThreads) {
            float f = (load_one<XB>(p.x, m * p.xs + c) - mean) * rstd;
            if (p.weight) f *= p.weight[c];
            if (p.bias) f += p.bias[c];
            store_one<YB>(p.y, m * p.ys + c, f);
        }
    }
}

// ---- backward ------------------------------------------------------------------
// A work-group takes every gridDim-th block of rows, the next one on its way
// while one is summed.  part: [work-group][2][D] sums of dy xh and of dy.
// Bound: HBM (32768 x 4096 in bf16 with d_residual 170 to 180 us, 6.0 to 6.3 TB/s;
// in fp32 to bf16 222 us, 6.0 TB/s).
template <bool XB, bool YB, bool MASK, int T, int NV>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_backward_kernel(NormParams p) {
#pragma clang fp contract(off)
    constexpr int W = XB && YB ? 8 : 4, R = rows_of(T), C = W * NV;
    constexpr int kW = T > kWave ? T / kWave : 1;
    __shared__ float red[2][R][2 * kW];
    const int t = threadIdx.x % T, r = threadIdx.x / T;
    Columns<W, T, NV> cols;
    cols.init(t, p.D);
    float w[C], dw[C], db[C];
    cols.load(p.weight, 1.f, w);
#pragma unroll
    for (int i = 0; i < C; ++i) dw[i] = db[i] = 0.f;
    const float per = 1.f / static_cast<float>(p.D);
    const bool params = p.part != nullptr;
    int turn = 0;
    // (rows past the end read the last one)
    auto row_at = [&](int64_t m0) { return m0 + r < p.M ? m0 + r : p.M - 1; };
    Run<XB, W> x[NV], skip[NV], next_x[NV], next_skip[NV];
    Run<YB, W> dy[NV], next_dy[NV];
    float next_mean = 0.f, next_rstd;
    auto fetch = [&](int64_t m) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            next_x[j].load_once(p.x, m * p.xs + cols.at[j]);
            next_dy[j].load_once(p.dy, m * p.dys + cols.at[j]);
        }
        if (p.d_residual) {
#pragma unroll
            for (int j = 0; j < NV; ++j) next_skip[j].load_once(p.d_residual, m * p.drs + cols.at[j]);
        }
        if (p.center) next_mean = p.stats_in[m];
        next_rstd = p.stats_in[p.M + m];
    };
    constexpr bool kAhead = T <= 512;         // (1024 threads' registers are full without the next row)
    int64_t m0 = static_cast<int64_t>(blockIdx.x) * R;
    if constexpr (kAhead) fetch(row_at(m0));
    for (; m0 < p.M; m0 += static_cast<int64_t>(gridDim.x) * R) {
        const int64_t m = row_at(m0);
        const bool real = R == 1 || m0 + r < p.M;
        if constexpr (!kAhead) fetch(m);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            x[j] = next_x[j];
            dy[j] = next_dy[j];
            skip[j] = next_skip[j];
        }
        const float mean = next_mean, rstd = next_rstd;
        if constexpr (kAhead) fetch(row_at(m0 + static_cast<int64_t>(gridDim.x) * R));
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const bool count = !MASK || cols.fresh(j, e);
                const float d = count ? dy[j].get(e) : 0.f, xh = (x[j].get(e) - mean) * rstd, q = d * w[W * j + e];
                s[0] += q;
                s[1] = fmaf(q, count ? xh : 0.f, s[1]);
                if (params && real) {
                    dw[W * j + e] = fmaf(d, count ? xh : 0.f, dw[W * j + e]);
                    db[W * j + e] += d;
                }
            }
        if (!p.dx) continue;
        row_sums<T, 2>(s, red[turn][r], t);
        turn ^= 1;
        if (!real) continue;
        const float a = p.center ? s[0] * per : 0.f, b = s[1] * per;
        if constexpr (!kAhead) {
            // (the inputs are unpacked again, not kept as floats meanwhile)
#pragma unroll
            for (int j = 0; j < NV; ++j) asm volatile("" : "+v"(x[j].v), "+v"(dy[j].v));
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (MASK && !cols.any(j, p.D)) continue;
            float f[W];
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float xh = (x[j].get(e) - mean) * rstd, q = dy[j].get(e) * w[W * j + e];
                const float t = fmaf(-xh, b, q - a);
                f[e] = p.d_residual ? fmaf(rstd, t, skip[j].get(e)) : rstd * t;
            }
            Run<XB, W>::store(p.dx, m * p.dxs + cols.at[j], f);
        }
    }
    if (!params) return;
    // one work-group's sums are the gradients themselves
    const bool only = gridDim.x == 1;
    float* const ow = only ? p.dweight : p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
    float* const ob = only ? p.dbias : ow + p.D;
    if constexpr (R > 1) {                    // the rows' sums, added in order
        __shared__ float all[R - 1][2 * C][T];
        if (r > 0) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                all[r - 1][i][t] = dw[i];
                all[r - 1][C + i][t] = db[i];
            }
        }
        __syncthreads();
        if (r > 0) return;
#pragma unroll 1
        for (int k = 0; k < R - 1; ++k)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                dw[i] += all[k][i][t];
                db[i] += all[k][C + i][t];
            }
    }
    if (ow) cols.store(ow, dw);
    if (ob) cols.store(ob, db);
}

// A thread to a row: its sums of all its rows, then the work-group's.  (2^20 x 7
// in fp32 with both sums: 30 us with the call; as rows of more than 16384 go, by
// at most 64 work-groups, 6040, and the sums of a thread lost 2586 halves of a
// last bit of 2^20 equal values.)
template <bool XB, bool YB>
__global__ __launch_bounds__(kNarrowThreads) void norm_backward_narrow_kernel(NormParams p) {
    const int D = static_cast<int>(p.D);
    const float per = 1.f / static_cast<float>(p.D);
    float w[kNarrow], sums[2 * kNarrow];
#pragma unroll
    for (int c = 0; c < kNarrow; ++c) {
        w[c] = c >= D ? 0.f : p.weight ? p.weight[c] : 1.f;
        sums[c] = sums[kNarrow + c] = 0.f;
    }
    for (int64_t m = static_cast<int64_t>(blockIdx.x) * kNarrowThreads + threadIdx.x; m < p.M;
         m += static_cast<int64_t>(gridDim.x) * kNarrowThreads) {
        const float mean = p.center ? p.stats_in[m] : 0.f, rstd = p.stats_in[p.M + m];
        float xh[kNarrow], dy[kNarrow], a = 0.f, b = 0.f;
        load_narrow<XB>(p.x, m * p.xs, D, xh);
        load_narrow<YB>(p.dy, m * p.dys, D, dy);
#pragma unroll
        for (int c = 0; c < kNarrow; ++c) {
            xh[c] = c < D ? (xh[c] - mean) * rstd : 0.f;
            const float q = dy[c] * w[c];
            a += q;
            b = fmaf(q, xh[c], b);
            sums[c] = fmaf(dy[c], xh[c], sums[c]);
            sums[kNarrow + c] += dy[c];
        }
        if (!p.dx) continue;
        a = p.center ? a * per : 0.f;
        b *= per;
#pragma unroll
        for (int c = 0; c < kNarrow; ++c) {
            if (c >= D) break;
            float f = rstd * (dy[c] * w[c] - a - xh[c] * b);
            if (p.d_residual) f += load_one<XB>(p.d_residual, m * p.drs + c);
            store_one<XB>(p.dx, m * p.dxs + c, f);
        }
    }
    if (!p.part) return;
    __shared__ float red[2 * kNarrow * (kNarrowThreads / kWave)];
    row_sums<kNarrowThreads, 2 * kNarrow>(sums, red, threadIdx.x);
    // one work-group's sums are the gradients themselves
    const bool only = gridDim.x == 1;
    float* const ow = only ? p.dweight : p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
    float* const ob = only ? p.dbias : ow + p.D;
    if (threadIdx.x > 0) return;
#pragma unroll
    for (int c = 0; c < kNarrow; ++c) {
        if (ow && c < D) ow[c] = sums[c];
        if (ob && c < D) ob[c] = sums[kNarrow + c];
    }
}

template <bool XB, bool YB>
__global__ __launch_bounds__(kLongThreads) void norm_backward_long_kernel(NormParams p) {
    __shared__ float red[2][2 * kLongThreads / kWave];
    const int t = threadIdx.x;
    const float per = 1.f / static_cast<float>(p.D);
    int turn = 0;
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        const float mean = p.center ? p.stats_in[m] : 0.f, rstd = p.stats_in[p.M + m];
        float s[2] = {0.f, 0.f};
        for (int64_t c = t; c < p.D; c += kLongThreads) {
            const float q = load_one<YB>(p.dy, m * p.dys + c) * (p.weight ? p.weight[c] : 1.f);
            s[0] += q;
            s[1] = fmaf(q, (load_one<XB>(p.x, m * p.xs + c) - mean) * rstd, s[1]);
        }
        row_sums<kLongThreads, 2>(s, red[turn], t);
        turn ^= 1;
        const float a = p.center ? s[0] * per : 0.f, b = s[1] * per;
        for (int64_t c = t; c < p.D; c += kLongThreads) {
            const float q = load_one<YB>(p.dy, m * p.dys + c) * (p.weight ? p.weight[c] : 1.f);
            const float xh = (load_one<XB>(p.x, m * p.xs + c) - mean) * rstd;
            float f = rstd * (q - a - xh * b);
            if (p.d_residual) f += load_one<XB>(p.d_residual, m * p.drs + c);
            store_one<XB>(p.dx, m * p.dxs + c, f);
        }
    }
}

// The parameters' sums of the same rows: a column a thread, blockIdx.y taking
// every gridDim.y-th row.
template <bool XB, bool YB>
__global__ __launch_bounds__(256) void norm_params_long_kernel(NormParams p) {
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (c >= p.D) return;
    float dw = 0.f, db = 0.f;
    for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
        const float mean = p.center ? p.stats_in[m] : 0.f, rstd = p.stats_in[p.M + m];
        const float d = load_one<YB>(p.dy, m * p.dys + c);
        dw = fmaf(d, (load_one<XB>(p.x, m * p.xs + c) - mean) * rstd, dw);
        db += d;
    }
    const bool only = gridDim.y == 1;
    float* const ow = only ? p.dweight : p.part + static_cast<int64_t>(blockIdx.y) * 2 * p.D;
    float* const ob = only ? p.dbias : ow + p.D;
    if (ow) ow[c] = dw;
    if (ob) ob[c] = db;
}

// dweight and dbias from the work-groups' sums, in their order: 32 columns a
// work-group, each by 32 threads.
__global__ __launch_bounds__(1024) void norm_sum_kernel(NormParams p, int blocks) {
    __shared__ float t[32][33];
    const int col = threadIdx.x % 32, sl = threadIdx.x / 32;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + col;
    float s = 0.f;
    if (c < 2 * p.D) {
#pragma unroll 8
        for (int64_t i = sl; i < blocks; i += 32) s += p.part[i * 2 * p.D + c];
    }
    t[sl][col] = s;
    __syncthreads();
    if (sl == 0 && c < 2 * p.D) {
#pragma unroll
        for (int k = 1; k < 32; ++k) s += t[k][col];
        if (c < p.D) {
            if (p.dweight) p.dweight[c] = s;
        } else if (p.dbias) {
            p.dbias[c - p.D] = s;
        }
    }
}

// (a launch of 2^32 work-items or more runs a part of them without an error)
dim3 grid_of_rows(int64_t n) { return dim3(static_cast<unsigned>(n < (1 << 21) ? n : 1 << 21)); }

constexpr int64_t kLongRow = 16384;

template <bool XB, bool YB, int T, int NV>
hipError_t rows_t(const NormParams& p, hipStream_t s) {
    constexpr int W = XB && YB ? 8 : 4, R = rows_of(T);
    if (p.D == W * T * NV)
        hipLaunchKernelGGL((norm_row_kernel<XB, YB, false, T, NV>), grid_of_rows((p.M + R - 1) / R), dim3(T < 256 ? 256 : T), 0, s, p);
    else
        hipLaunchKernelGGL((norm_row_kernel<XB, YB, true, T, NV>), grid_of_rows((p.M + R - 1) / R), dim3(T < 256 ? 256 : T), 0, s, p);
    return hipGetLastError();
}

template <bool XB, bool YB, int T, int NV>
hipError_t forward_t(const NormParams& p, hipStream_t s) {
    constexpr int W = XB && YB ? 8 : 4, R = rows_of(T);
    const int64_t blocks = (p.M + R - 1) / R, fill = 2 * compute_units();
    const dim3 grid(static_cast<unsigned>(blocks < fill ? blocks : fill));
    if (p.D == W * T * NV) hipLaunchKernelGGL((norm_forward_kernel<XB, YB, false, T, NV>), grid, dim3(T < 256 ? 256 : T), 0, s, p);
    else hipLaunchKernelGGL((norm_forward_kernel<XB, YB, true, T, NV>), grid, dim3(T < 256 ? 256 : T), 0, s, p);
    return hipGetLastError();
}

// Threads of a row and runs of a thread: a wave to a row as long as its
// registers hold it (eight runs), then work-groups.  Work-groups that stay,
// with 16 columns a thread, from 2^25 values in rows of more than 1024 on
// (8192 x 2048 in bf16: 20 us, all rows at once 17; 8192 x 4096: 31 and 36;
// 32768 x 512: 22 and 17).
template <bool XB, bool YB>
hipError_t forward(const NormParams& p, hipStream_t s) {
    constexpr int W = XB && YB ? 8 : 4, NV = 16 / W;
    if (p.D <= kNarrow) {
        hipLaunchKernelGGL((norm_narrow_kernel<XB, YB>), grid_of_rows((p.M + kNarrowThreads - 1) / kNarrowThreads), dim3(kNarrowThreads), 0, s, p);
        return hipGetLastError();
    }
    if (p.D > kLongRow) {
        hipLaunchKernelGGL((norm_forward_long_kernel<XB, YB>), grid_of_rows(p.M), dim3(kLongThreads), 0, s, p);
        return hipGetLastError();
    }
    if (p.D > 1024 && p.M * p.D >= (int64_t(1) << 25)) {
        if (p.D <= 2048) return forward_t<XB, YB, 128, NV>(p, s);
        if (p.D <= 4096) return forward_t<XB, YB, 256, NV>(p, s);
        if (p.D <= 8192) return forward_t<XB, YB, 512, NV>(p, s);
        return forward_t<XB, YB, 1024, NV>(p, s);
    }
    const int64_t runs = (p.D + W - 1) / W;
    if (runs <= 8) return rows_t<XB, YB, 8, 1>(p, s);
    if (runs <= 16) return rows_t<XB, YB, 16, 1>(p, s);
    if (runs <= 32) return rows_t<XB, YB, 32, 1>(p, s);
    if (runs <= 64) return rows_t<XB, YB, 64, 1>(p, s);
    if (runs <= 128) return rows_t<XB, YB, 64, 2>(p, s);
    if (runs <= 256) return rows_t<XB, YB, 64, 4>(p, s);
    if (runs <= 512) return rows_t<XB, YB, 64, 8>(p, s);
    if (runs <= 1024) return rows_t<XB, YB, 256, 4>(p, s);
    if constexpr (W == 4) {
        if (runs > 2048) return rows_t<XB, YB, 1024, 4>(p, s);
    }
    return rows_t<XB, YB, 256, 8>(p, s);
}

// Work-groups of the backward pass, each of which leaves a sum for each column:
// one for each block of rows up to 64 (100 x 2048 in bf16: 6.6 us from a graph,
// 7.3 with two blocks each), then with two blocks at least (100 x 8192 in fp32:
// 9.5, 10.3 with one each) up to as many a compute unit as are fastest: four up
// to 512 columns (2^25 values in rows of 256 in bf16: 84, 57, 46, 42 and 49 us
// with 1, 2, 3, 4 and 6; of 300 in fp32 156, 102, 87, 87, 91), two up to 1536
// (of 768 in bf16 71, 48, 60, 53, 58) and where 2^24 values fit, up to 2048
// columns or 4096 in bf16 (8192 x 4096 in bf16: 58 and 50, 4096 x 4096: 34 and
// 33; 32768 x 4096 in fp32: 221 and 244).  Rows that are read in steps: up to
// 64, for the parameters' sums.  A few blocks of rows go to one work-group,
// whose sums no second kernel has to add: a launch less, 3 us of the host's, for
// about 1 us more on the device (4 x 8192 in bf16: 7.7 and 6.6 us; 100 x 64: 6.4
// and 7.0; 4 x 16000: 14.6 and 10.6, so two there).
int64_t norm_parts_of(int64_t M, int64_t D, bool both_bf16) {
    const bool in_steps = D > kLongRow;
    const int64_t rows = D > 2048 ? 1 : D > 1024 ? 2 : D > 256 ? 4 : D > 64 ? 8 : D > kNarrow ? 16 : kNarrowThreads;
    const bool two = D <= 1536 || (M * D >= (int64_t(1) << 24) && (D <= 2048 || (both_bf16 && D <= 4096)));
    const int64_t most = in_steps ? 64 : (D <= 512 ? 4 : two ? 2 : 1) * compute_units();
    if (M <= (D > 8192 ? 2 : D > 256 ? 4 : 8) * rows) return 1;
    const int64_t each = (M + rows - 1) / rows, n = each <= 64 ? each : (M + 2 * rows - 1) / (2 * rows);
    return n < most ? n : most;
}

template <bool XB, bool YB, bool MASK, int T, int NV>
hipError_t backward_t(const NormParams& p, hipStream_t s) {
    hipLaunchKernelGGL((norm_backward_kernel<XB, YB, MASK, T, NV>), dim3(static_cast<unsigned>(norm_parts_of(p.M, p.D, XB && YB))),
                       dim3(T < 256 ? 256 : T), 0, s, p);
    return hipGetLastError();
}

template <bool XB, bool YB, int T, int NV>
hipError_t backward_m(const NormParams& p, hipStream_t s) {
    constexpr int W = XB && YB ? 8 : 4;
    return p.D == W * T * NV ? backward_t<XB, YB, false, T, NV>(p, s) : backward_t<XB, YB, true, T, NV>(p, s);
}

template <bool XB, bool YB>
hipError_t backward(const NormParams& p, hipStream_t s) {
    constexpr int W = XB && YB ? 8 : 4, NV = 16 / W;
    if (p.D <= kNarrow) {
        hipLaunchKernelGGL((norm_backward_narrow_kernel<XB, YB>), dim3(static_cast<unsigned>(norm_parts_of(p.M, p.D, XB && YB))),
                           dim3(kNarrowThreads), 0, s, p);
        return hipGetLastError();
    }
    if (p.D > kLongRow) {
        if (p.dx) {
            hipLaunchKernelGGL((norm_backward_long_kernel<XB, YB>), grid_of_rows(p.M), dim3(kLongThreads), 0, s, p);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess || !p.part) return e;
        }
        hipLaunchKernelGGL((norm_params_long_kernel<XB, YB>),
                           dim3(static_cast<unsigned>((p.D + 255) / 256), static_cast<unsigned>(norm_parts_of(p.M, p.D, XB && YB))), dim3(256), 0, s, p);
        return hipGetLastError();
    }
    if (p.D <= 8 * W) return backward_m<XB, YB, 8, 1>(p, s);
    if (p.D <= 16 * W) return backward_m<XB, YB, 16, 1>(p, s);
    if (p.D <= 32 * W) return backward_m<XB, YB, 32, 1>(p, s);
    if (p.D <= 64 * W) return backward_m<XB, YB, 64, 1>(p, s);
    if (W == 4 && p.D <= 512) return backward_m<XB, YB, 64, 2>(p, s);
    if (p.D <= 1024) return backward_m<XB, YB, 64, NV>(p, s);
    if (p.D <= 2048) return backward_m<XB, YB, 128, NV>(p, s);
    if (p.D <= 4096) return backward_m<XB, YB, 256, NV>(p, s);
    if (p.D <= 8192) return backward_m<XB, YB, 512, NV>(p, s);
    return backward_m<XB, YB, 1024, NV>(p, s);
}

}  // namespace

int norm_parts(int64_t M, int64_t D) {
    const int64_t a = norm_parts_of(M, D, false), b = norm_parts_of(M, D, true);
    return static_cast<int>(a > b ? a : b);
}

hipError_t launch_norm(const NormParams& p, bool x_bf16, bool y_bf16, hipStream_t s) {
    if (x_bf16) return y_bf16 ? forward<true, true>(p, s) : forward<true, false>(p, s);
    return y_bf16 ? forward<false, true>(p, s) : forward<false, false>(p, s);
}

hipError_t launch_norm_backward(const NormParams& p, bool x_bf16, bool y_bf16, hipStream_t s) {
    hipError_t e;
    if (x_bf16) e = y_bf16 ? backward<true, true>(p, s) : backward<true, false>(p, s);
    else e = y_bf16 ? backward<false, true>(p, s) : backward<false, false>(p, s);
    if (e != hipSuccess || !p.part || norm_parts_of(p.M, p.D, x_bf16 && y_bf16) == 1) return e;
    hipLaunchKernelGGL(norm_sum_kernel, dim3(static_cast<unsigned>((2 * p.D + 31) / 32)), dim3(1024), 0, s, p,
                       static_cast<int>(norm_parts_of(p.M, p.D, x_bf16 && y_bf16)));
    return hipGetLastError();
}

}  // namespace gdn
