// gdn_loss.hip -- the softmax cross entropy of a linear layer's outputs over a
// vocabulary, and its gradients, without keeping the logits.
//
// With l = x w^T + bias, lse = log sum_v exp(l_v), e the label smoothing and c
// the weight of the squared normaliser, per row with target t:
//   loss = (1 - e) (lse - l_t) + e (lse - mean_v l_v) + c lse^2
//   dl_v = g ((1 + 2 c lse) exp(l_v - lse) - (1 - e) [v = t] - e / V)
//   dx = dl w,  dw = dl^T x,  dbias = sum over the rows of dl
//
// Forward: the tiles of the product x w^T leave, for each of their rows, the
// largest of their logits and the sum of the exponentials of the others' (all)
// distances to it; a second kernel joins a row's tiles.  Nothing of the size
// rows x vocabulary is written.  Up to 16 rows it is a stream over w, bound by
// HBM.
// Backward: for a piece of the vocabulary at a time the tiles of the product
// are computed once more and leave dl in bf16, the operand type of the two
// products that follow: dx, in 32 bits from piece to piece, and the piece's
// rows of dw.  Rows without a target add nothing: a large call first brings the
// others together, and all that follows is as long as there are of those (the
// host does not know how many: tiles past them end at once); in a small one dw
// is formed from a copy of x in which they are zero, so that an infinity or NaN
// in them does not reach it as 0 times that.
// dl is rounded to bf16 once, as dp is in the linear layer's backward pass
// (dbias sums it in 32 bits before that), and not by itself but over (1 - e)
// times the largest |g|, by which the outputs are multiplied in 32 bits: with
// one g for all rows the target's entry is then next to -1 and rounds as any
// other value.  (Times g it would be next to -g in every row, all of them off
// by the same up to 2^-8 of themselves: 4096 x 248320 x 2048 with g = 1/3686:
// dw 3.4e-3 off in its norm, of which 1.7e-3 are its own rounding.)  A g that
// is not finite is no factor of the outputs, whose zeros it would make NaN, but
// of its own rows of dl: rows without a target stay zero.
// Statistics are in base two: 2^(l log2 e - top), one multiply-add and one
// v_exp_f32 a logit.
#include <cmath>

#include "gdn_tiles.hpp"

namespace gdn {

namespace {

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int64_t target_of(const LossRows& r, int64_t m) {
    return r.targets64 ? static_cast<const int64_t*>(r.targets)[m] : static_cast<const int32_t*>(r.targets)[m];
}

// over the four lanes that share a row of a tile's 16 x 16 accumulators
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor(x, 16, kWave));
    return fmaxf(x, __shfl_xor(x, 32, kWave));
}
__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor(x, 16, kWave);
    return x + __shfl_xor(x, 32, kWave);
}

// A set of logits: the largest times log2 e, and the sum of 2^(l log2 e - top).
// None: top = -inf, sum = 0.
struct Part {
    float top, sum;
};
__device__ __forceinline__ Part join(Part a, Part b) {
    const float top = fmaxf(a.top, b.top);
    // (an empty part's -inf less -inf counts as nothing; NaN stays NaN through the sums)
    const float ea = a.top == top ? 1.f : __builtin_amdgcn_exp2f(a.top - top);
    const float eb = b.top == top ? 1.f : __builtin_amdgcn_exp2f(b.top - top);
    return Part{top, fmaf(a.sum, ea, b.sum * eb)};
}

// the piece of the product that a launch covers
struct LossProduct : GemmProduct {
    LossRows rows;
    int64_t v0;                               // the vocabulary's index of column 0
    const float* bias;                        // of column 0, or NULL
    // forward
    Part* part;                               // [column tiles][M]
    float* totals;                            // [column tiles][M] sums of the logits, or NULL
    // backward
    GemmProduct out;                          // dl: rows, columns (padded with zeros), address and stride
    float* columns;                           // [row tiles][V] sums of dl, or NULL
    int64_t columns_ld;
    const int32_t* count;                     // device: how many of the M rows there are; NULL: all
    uint16_t* clean;                          // [M][K]: receives x, zeros where a row has no target, or NULL
};

// row of a wave's accumulators acc[i][.] in lane l16
template <typename S>
__device__ __forceinline__ int64_t row_of(int64_t m0, int wave, int i, int l16) {
    return m0 + wave / S::NWN * S::kWaveStep + i / S::kStripTiles * S::kHalfStep + 16 * (i % S::kStripTiles) + l16;
}

// acc += bias, and -inf for columns past the vocabulary (they hold the last column's product again)
template <typename S>
__device__ __forceinline__ void finish_logits(const LossProduct& p, f32x4 (&acc)[S::TM][S::TN], int64_t n0, int wave, int lane) {
    const bool cut = n0 + S::BN > p.N;
    if (!p.bias && !cut) return;
    const int64_t first = n0 + wave % S::NWN * S::WN + 4 * (lane / 16);
#pragma unroll
    for (int j = 0; j < S::TN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t n = first + 16 * j + e;
            const float b = p.bias && n < p.N ? p.bias[n] : 0.f;
#pragma unroll
            for (int i = 0; i < S::TM; ++i) acc[i][j][e] = n < p.N ? acc[i][j][e] + b : -__builtin_inff();
        }
}

// Which of a lane's columns first + 16 j + e (0 .. WN - 1) is row m's target; -1: none
template <typename S>
__device__ __forceinline__ int column_of(const LossProduct& p, int64_t target, int64_t first) {
    const int64_t at = target - p.v0 - first;
    return at >= 0 && at < S::WN && at % 16 < 4 ? static_cast<int>(at) : -1;
}

// What an epilogue reads of its rows is requested before the last slices are
// multiplied, all rows at once (1537 x 50001 x 1000, forward and backward: 751
// us row by row, 745 so).

// ---- forward -------------------------------------------------------------------
// Bound: the matrix cores at the card's power (4096 x 248320 x 2048: 2.99 to
// 3.07 ms, 1360 to 1390 TFLOP/s, where an 8192^3 product of the vendor's library
// reaches 1380 to 1460; a loop of nothing but these instructions on random
// operands in registers does 2100, and of their 32 x 32 x 16 form 1870).
// A tile's rows to their parts: each lane its 4 TN logits of a row, the four
// lanes that share the row, then the waves that do, through LDS.
template <typename S>
struct RowParts {
    int64_t m0, n0;
    __device__ __forceinline__ void init(const LossProduct&, int64_t m, int64_t n, int, int) {
        m0 = m;
        n0 = n;
    }
    __device__ __forceinline__ void fetch(const LossProduct&, int) {}
    __device__ __forceinline__ void run(const LossProduct& p, f32x4 (&acc)[S::TM][S::TN], uint8_t* shared, int wave, int lane) {
        Part* const red = reinterpret_cast<Part*>(shared);                         // [NWN][BM]
        float* const tot = reinterpret_cast<float*>(shared + S::NWN * S::BM * sizeof(Part));
        const int l16 = lane % 16, lq = lane / 16, wn = wave % S::NWN;
        const int64_t first = n0 + wn * S::WN + 4 * lq;
        finish_logits<S>(p, acc, n0, wave, lane);
#pragma unroll
        for (int i = 0; i < S::TM; ++i) {
            const int64_t m = row_of<S>(m0, wave, i, l16);
            float top = acc[i][0][0];
#pragma unroll
            for (int j = 0; j < S::TN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, acc[i][j][e]);
            top = quad_max(top) * kLog2e;
            const float base = top == -__builtin_inff() ? 0.f : top;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < S::TN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) sum += __builtin_amdgcn_exp2f(fmaf(acc[i][j][e], kLog2e, -base));
            sum = quad_sum(sum);
            const int r = static_cast<int>(m - m0);
            if (lq == 0) red[wn * S::BM + r] = Part{top, sum};
            if (p.totals) {
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < S::TN; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s += first + 16 * j + e < p.N ? acc[i][j][e] : 0.f;
                s = quad_sum(s);
                if (lq == 0) tot[wn * S::BM + r] = s;
            }
        }
        __syncthreads();
        for (int r = threadIdx.x; r < S::BM; r += S::kThreads) {
            if (m0 + r >= p.M) continue;
            Part a = red[r];
#pragma unroll
            for (int w = 1; w < S::NWN; ++w) a = join(a, red[w * S::BM + r]);
            const int64_t at = n0 / S::BN * p.M + m0 + r;
            p.part[at] = a;
            if (p.totals) {
                float s = tot[r];
#pragma unroll
                for (int w = 1; w < S::NWN; ++w) s += tot[w * S::BM + r];
                p.totals[at] = s;
            }
        }
    }
};

template <typename S>
__global__ __launch_bounds__(S::kThreads, S::kPerSimd) void loss_forward_kernel(LossProduct p) {
    __shared__ __align__(1024) uint8_t shared[S::kBytes];
    gemm_tile<true, true, RowParts<S>, S>(p, blockIdx.x, shared);
}

// Up to 16 rows: a wave takes 16 columns at a time, over the whole of K, and
// keeps its rows' parts from one to the next.  Per 64-wide step of K the lanes
// of a row read two runs of 64 bytes of their weight row and of their row of x,
// kFewDepth steps ahead.  Bound: HBM (1 x 248320 x 2048: 193 us, 5.3 TB/s).
constexpr int kFewWaves = 4, kFewDepth = 4;

__global__ __launch_bounds__(kFewWaves * kWave, 4) void loss_few_kernel(LossProduct p) {
    __shared__ Part red[kFewWaves][16];
    __shared__ float tot[kFewWaves][16];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
    const int l16 = lane % 16, lq = lane / 16;
    const int64_t groups = (p.N + 15) / 16, all = static_cast<int64_t>(gridDim.x) * kFewWaves;
    const int64_t m = l16 < p.M ? l16 : p.M - 1;                                   // (rows past the end are never stored)
    const uint16_t* const arow = static_cast<const uint16_t*>(p.A) + m * p.lda;
    const int steps = static_cast<int>((p.K + 63) / 64);
    Part mine{-__builtin_inff(), 0.f};
    float total = 0.f;
    for (int64_t g = static_cast<int64_t>(blockIdx.x) * kFewWaves + wave; g < groups; g += all) {
        const int64_t n0 = 16 * g;
        const uint16_t* const brow = static_cast<const uint16_t*>(p.B) + (n0 + l16 < p.N ? n0 + l16 : p.N - 1) * p.ldb;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        u32x4 bf[kFewDepth][2], af[kFewDepth][2];
        auto load = [&](int st, int slot) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t k = 64 * static_cast<int64_t>(st) + 32 * h + 8 * lq;
                bf[slot][h] = *reinterpret_cast<const u32x4*>(k < p.K ? brow + k : zero_chunk);
                af[slot][h] = *reinterpret_cast<const u32x4*>(k < p.K ? arow + k : zero_chunk);
            }
        };
#pragma unroll
        for (int d = 0; d < kFewDepth; ++d) load(d, d);
        for (int st = 0; st < steps; st += kFewDepth) {
#pragma unroll
            for (int d = 0; d < kFewDepth; ++d) {
                acc = mfma(bf[d][0], af[d][0], acc);
                acc = mfma(bf[d][1], af[d][1], acc);
                if (st + kFewDepth < steps) load(st + kFewDepth + d, d);
            }
        }
        // this lane: row l16, columns n0 + 4 lq ..
        Part a{-__builtin_inff(), 0.f};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t n = n0 + 4 * lq + e;
            if (n >= p.N) { acc[e] = -__builtin_inff(); continue; }
            if (p.bias) acc[e] += p.bias[n];
            total += acc[e];
        }
        a.top = fmaxf(fmaxf(acc[0], acc[1]), fmaxf(acc[2], acc[3])) * kLog2e;
        const float base = a.top == -__builtin_inff() ? 0.f : a.top;
#pragma unroll
        for (int e = 0; e < 4; ++e) a.sum += __builtin_amdgcn_exp2f(fmaf(acc[e], kLog2e, -base));
        mine = join(mine, a);
    }
#pragma unroll
    for (int x = 16; x < kWave; x *= 2) {
        const Part o{__shfl_xor(mine.top, x, kWave), __shfl_xor(mine.sum, x, kWave)};
        mine = join(mine, o);
        total += __shfl_xor(total, x, kWave);
    }
    if (lane < 16) {
        red[wave][lane] = mine;
        tot[wave][lane] = total;
    }
    __syncthreads();
    const int r = threadIdx.x;
    if (r >= p.M) return;
    Part a = red[0][r];
    float s = tot[0][r];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) {
        a = join(a, red[w][r]);
        s += tot[w][r];
    }
    p.part[blockIdx.x * p.M + r] = a;
    if (p.totals) p.totals[blockIdx.x * p.M + r] = s;
}

// A row's parts to its lse and loss: 16 rows a work-group, 64 threads each,
// whose parts are joined in their order.  The target's logit is computed here,
// from its row of w (looked for among a tile's logits it takes 1 us of a tile:
// 4096 x 65536 x 64 148 instead of 124 us).
constexpr int kJoinRows = 16, kJoinSlices = 64;

__global__ __launch_bounds__(kJoinRows * kJoinSlices) void loss_join_kernel(LossProduct p, int64_t tiles, float* loss, float* lse) {
    __shared__ Part red[kJoinSlices][kJoinRows];
    __shared__ float tot[kJoinSlices][kJoinRows], dot[kJoinSlices][kJoinRows];
    const int r = threadIdx.x % kJoinRows, sl = threadIdx.x / kJoinRows;
    const int64_t m = static_cast<int64_t>(blockIdx.x) * kJoinRows + r;
    Part a{-__builtin_inff(), 0.f};
    float total = 0.f;
    if (m < p.M) {
#pragma unroll 4
        for (int64_t t = sl; t < tiles; t += kJoinSlices) a = join(a, p.part[t * p.M + m]);
        if (p.totals) {
#pragma unroll 4
            for (int64_t t = sl; t < tiles; t += kJoinSlices) total += p.totals[t * p.M + m];
        }
    }
    float hot = 0.f;
    int64_t t = -1;
    bool there = false;
    if (m < p.M) {
        t = target_of(p.rows, m);
        there = t != p.rows.ignore && t >= 0 && t < p.rows.V;
    }
    if (there && loss) {
        const uint16_t* const x = static_cast<const uint16_t*>(p.A) + m * p.lda;
        const uint16_t* const w = static_cast<const uint16_t*>(p.B) + t * p.ldb;
#pragma unroll 4
        for (int64_t k = 8 * sl; k < p.K; k += 8 * kJoinSlices) {
            const u32x4 q = *reinterpret_cast<const u32x4*>(x + k), v = *reinterpret_cast<const u32x4*>(w + k);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                hot = fmaf(__uint_as_float(q[e] << 16), __uint_as_float(v[e] << 16), hot);
                hot = fmaf(__uint_as_float(q[e] & 0xFFFF0000u), __uint_as_float(v[e] & 0xFFFF0000u), hot);
            }
        }
        if (sl == 0 && p.bias) hot += p.bias[t];
    }
    red[sl][r] = a;
    tot[sl][r] = total;
    dot[sl][r] = hot;
    for (int half = kJoinSlices / 2; half > 0; half /= 2) {
        __syncthreads();
        if (sl < half) {
            red[sl][r] = join(red[sl][r], red[sl + half][r]);
            tot[sl][r] += tot[sl + half][r];
            dot[sl][r] += dot[sl + half][r];
        }
    }
    if (sl > 0 || m >= p.M) return;
    a = red[0][r];
    const float l = (a.top + __builtin_amdgcn_logf(a.sum)) * kLn2;                  // (v_log_f32: base two)
    if (lse) lse[m] = l;
    float out = 0.f;
    if (there) {
        // No logit and no mean of logits is above lse, but its own sum's rounding
        // may put it there (a row that is sure of its target).
        const auto above = [](float a, float b) { const float d = a - b; return d < 0.f ? 0.f : d; };
        const float e = p.rows.smooth;
        out = (1.f - e) * above(l, dot[0][r]) + p.rows.z * l * l;
        if (e > 0.f) out += e * above(l, tot[0][r] / static_cast<float>(p.rows.V));
    } else if (t != p.rows.ignore) {
        out = __builtin_nanf("");
        if (p.rows.status) __hip_atomic_fetch_or(p.rows.status, GDN_STATUS_BAD_INDEX, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (loss) loss[m] = out;
}

// ---- backward ------------------------------------------------------------------
// Bound: the matrix cores (4096 x 248320 x 2048 of whose rows 3686 count: the 13
// pieces of 19200 columns take 281 us for dl, 1030 TFLOP/s, and 446 us for the
// two products, 1300).  dl's tiles fill 4.4 rounds of the compute units; where
// all launches come out even (4096 x 245760 x 2048 in 15 pieces) the pass is 3%
// faster, since a compute unit without a tile leaves its power to the others.
// A tile's logits to dl, in place, and on as the linear layer's outputs go: as
// bf16 through LDS in whole rows.
template <typename S>
struct Gradient {
    int64_t m0, n0, first;
    int wave, l16, at[S::TM];
    float g[S::TM], lse[S::TM];
    uint32_t counts = 0, odd = 0;             // a bit for each row; of those: dloss is not finite (g: 1)
    Store<S, true, true> store;
    __device__ __forceinline__ void init(const LossProduct& p, int64_t m, int64_t n, int w, int lane) {
        m0 = m;
        n0 = n;
        wave = w;
        l16 = lane % 16;
        first = n0 + wave % S::NWN * S::WN + 4 * (lane / 16);
        store.init(p.out, m, n, wave, lane);
    }
    __device__ __forceinline__ void fetch(const LossProduct& p, int) {
        int64_t t[S::TM];
#pragma unroll
        for (int i = 0; i < S::TM; ++i) {
            int64_t m = row_of<S>(m0, wave, i, l16);
            m = m < p.M ? m : p.M - 1;
            t[i] = target_of(p.rows, m);
            lse[i] = p.rows.lse[m];
            g[i] = p.rows.dloss[p.rows.dloss_one ? 0 : m];
        }
        const float scale = p.rows.dloss_one ? 1.f : *p.rows.scale;
#pragma unroll
        for (int i = 0; i < S::TM; ++i) {
            counts |= row_of<S>(m0, wave, i, l16) < p.M && t[i] != p.rows.ignore && t[i] >= 0 && t[i] < p.rows.V ? 1u << i : 0u;
            at[i] = column_of<S>(p, t[i], first);
            odd |= is_finite(g[i]) ? 0u : counts & 1u << i;
            g[i] = p.rows.dloss_one || !is_finite(g[i]) ? 1.f : g[i] / scale;
        }
    }
    __device__ __forceinline__ void run(const LossProduct& p, f32x4 (&acc)[S::TM][S::TN], uint8_t* shared, int wave, int lane) {
        const int lq = lane / 16, wn = wave % S::NWN;
        finish_logits<S>(p, acc, n0, wave, lane);
        const float smooth = p.rows.smooth, over = 1.f / (1.f - smooth), even = smooth / static_cast<float>(p.rows.V);
#pragma unroll
        for (int i = 0; i < S::TM; ++i) {
            const bool real = (counts >> i & 1u) != 0;
            const float g1 = g[i] * over, c = g1 * fmaf(2.f * p.rows.z, lse[i], 1.f), base = lse[i] * kLog2e, rest = g1 * even;
#pragma unroll
            for (int j = 0; j < S::TN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float d = fmaf(c, __builtin_amdgcn_exp2f(fmaf(acc[i][j][e], kLog2e, -base)), -rest);
                    acc[i][j][e] = real ? d : 0.f;
                }
            if (real && at[i] >= 0) {                // (few lanes: the target is one of V)
#pragma unroll
                for (int j = 0; j < S::TN; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (at[i] == 16 * j + e) acc[i][j][e] -= g[i];
            }
            if (odd >> i & 1u) {
                const float d = p.rows.dloss[p.rows.dloss_one ? 0 : row_of<S>(m0, wave, i, l16)];
#pragma unroll
                for (int j = 0; j < S::TN; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][e] *= d;
            }
        }
        if (n0 + S::BN > p.N) {                      // columns past the end
#pragma unroll
            for (int j = 0; j < S::TN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (first + 16 * j + e >= p.N) {
#pragma unroll
                        for (int i = 0; i < S::TM; ++i) acc[i][j][e] = 0.f;
                    }
        }
        if (p.columns) {
            float* const red = reinterpret_cast<float*>(shared);                   // [NWM][BN]
#pragma unroll
            for (int j = 0; j < S::TN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float s = acc[0][j][e];
#pragma unroll
                    for (int i = 1; i < S::TM; ++i) s += acc[i][j][e];
                    s = group_sum<16>(s);
                    if (l16 == 0) red[wave / S::NWN * S::BN + wn * S::WN + 16 * j + 4 * lq + e] = s;
                }
            __syncthreads();
            for (int n = threadIdx.x; n < S::BN; n += S::kThreads) {
                float s = red[n];
#pragma unroll
                for (int w = 1; w < S::NWM; ++w) s += red[w * S::BN + n];
                if (n0 + n < p.N) p.columns[m0 / S::BM * p.columns_ld + p.v0 + n0 + n] = s;
            }
            __syncthreads();
        }
        store.run(p.out, acc, shared, wave, lane);
    }
};

// The work-groups after the tiles' write p.clean: up to kCleanGroups, a thread 8
// values kCleanEach times at once (4096 x 2000 x 2048, forward and backward: 141
// us without, 152 us with 1024 work-groups and once, 146 us so).
constexpr int kCleanGroups = 256, kCleanEach = 8;

__host__ __device__ inline int clean_groups(int64_t M, int64_t K, int threads) {
    const int64_t n = (M * (K / 8) + threads - 1) / threads;
    return static_cast<int>(n < kCleanGroups ? n : kCleanGroups);
}

template <typename S>
__global__ __launch_bounds__(S::kThreads, S::kPerSimd) void loss_gradient_kernel(LossProduct p) {
    __shared__ __align__(1024) uint8_t shared[S::kBytes];
    if (p.count) p.M = p.out.M = *p.count;
    const int64_t past = static_cast<int64_t>(blockIdx.x) - ((p.M + S::BM - 1) / S::BM) * ((p.N + S::BN - 1) / S::BN);
    if (past >= 0) {
        if (!p.clean) return;
        const uint32_t per = static_cast<uint32_t>(p.K / 8), all = static_cast<uint32_t>(p.M) * per;
        const uint32_t step = clean_groups(p.M, p.K, S::kThreads) * S::kThreads;
        for (uint32_t i = static_cast<uint32_t>(past) * S::kThreads + threadIdx.x; i < all; i += kCleanEach * step) {
            u32x4 q[kCleanEach];
#pragma unroll
            for (int u = 0; u < kCleanEach; ++u) {
                const uint32_t at = i + u * step < all ? i + u * step : i, m = at / per, k = at % per * 8;
                const int64_t t = target_of(p.rows, m);
                const bool real = t != p.rows.ignore && t >= 0 && t < p.rows.V;
                q[u] = *reinterpret_cast<const u32x4*>(real ? static_cast<const uint16_t*>(p.A) + m * p.lda + k : zero_chunk);
            }
#pragma unroll
            for (int u = 0; u < kCleanEach; ++u)
                if (i + u * step < all) *reinterpret_cast<u32x4*>(p.clean + 8 * static_cast<int64_t>(i + u * step)) = q[u];
        }
        return;
    }
    gemm_tile<true, true, Gradient<S>, S>(p, blockIdx.x, shared);
}

// The rows that count, in their order: place[m] among them or -1, and how many.
constexpr int kListThreads = 1024, kListEach = 8;

__global__ __launch_bounds__(kListThreads) void loss_list_kernel(LossRows r, int64_t M, int32_t* place, int32_t* count) {
    __shared__ int32_t waves[kListThreads / kWave];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    int32_t before = 0;
    for (int64_t m0 = 0; m0 < M; m0 += kListThreads * kListEach) {
        const int64_t first = m0 + static_cast<int64_t>(threadIdx.x) * kListEach;
        uint32_t mine = 0;
#pragma unroll
        for (int e = 0; e < kListEach; ++e) {
            const int64_t m = first + e, t = target_of(r, m < M ? m : M - 1);
            mine |= m < M && t != r.ignore && t >= 0 && t < r.V ? 1u << e : 0u;
        }
        const int32_t own = __builtin_popcount(mine);
        int32_t upto = own;                                   // of the wave's lanes up to this one
#pragma unroll
        for (int x = 1; x < kWave; x *= 2) {
            const int32_t v = __shfl_up(upto, x, kWave);
            upto += lane >= x ? v : 0;
        }
        if (lane == kWave - 1) waves[wave] = upto;
        __syncthreads();
        int32_t at = before + upto - own;
#pragma unroll
        for (int w = 0; w < kListThreads / kWave; ++w) {
            at += w < wave ? waves[w] : 0;
            before += waves[w];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kListEach; ++e) {
            if (first + e < M) place[first + e] = mine >> e & 1u ? at : -1;
            at += static_cast<int32_t>(mine >> e & 1u);
        }
    }
    if (threadIdx.x == 0) *count = before;
}

// What the backward pass reads of those rows, together; a wave a row.
struct LossList {
    const int32_t* place;                     // [M]
    uint16_t* x;                              // [count][K]
    int32_t* targets;
    float *lse, *dloss;                       // dloss: not written where there is one for all
};

__global__ __launch_bounds__(256) void loss_gather_kernel(LossRows r, LossList l, const uint16_t* x, int64_t ldx, int64_t M, int64_t K) {
    const int lane = threadIdx.x % kWave;
    for (int64_t m = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / kWave; m < M; m += static_cast<int64_t>(gridDim.x) * 4) {
        const int64_t at = l.place[m];
        if (at < 0) continue;
        for (int64_t k = 8 * lane; k < K; k += 8 * kWave)
            *reinterpret_cast<u32x4*>(l.x + at * K + k) = *reinterpret_cast<const u32x4*>(x + m * ldx + k);
        if (lane == 0) {
            l.targets[at] = static_cast<int32_t>(target_of(r, m));
            l.lse[at] = r.lse[m];
            if (!r.dloss_one) l.dloss[at] = r.dloss[m];
        }
    }
}

// The largest finite |g| of the rows that count (0: none).
__global__ __launch_bounds__(1024) void loss_scale_kernel(LossRows r, int64_t M, float* out) {
    __shared__ float red[1024 / kWave];
    float top = 0.f;
    for (int64_t m = threadIdx.x; m < M; m += 1024) {
        const int64_t t = target_of(r, m);
        const float g = fabsf(r.dloss[m]);
        if (t != r.ignore && t >= 0 && t < r.V && g < __builtin_inff()) top = fmaxf(top, g);
    }
#pragma unroll
    for (int x = 1; x < kWave; x *= 2) top = fmaxf(top, __shfl_xor(top, x, kWave));
    if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = top;
    __syncthreads();
    if (threadIdx.x > 0) return;
#pragma unroll
    for (int w = 1; w < 1024 / kWave; ++w) top = fmaxf(top, red[w]);
    *out = top > 0.f ? top : 1.f;
}

// dx and dw of a piece in one launch.  dx: its reduction, the piece's columns,
// is cut into `parts`, each with sums of its own ([parts][M][K] in 32 bits),
// to which a piece adds.  The tiles with the longer reductions come first.
// DIRECT: one piece, one part: dx is what the product gives.
__host__ __device__ inline int64_t loss_share(int64_t n, int parts) {
    return ((n + 127) / 128 + parts - 1) / parts * 128;
}

template <typename S, bool DIRECT>
__global__ __launch_bounds__(S::kThreads, S::kPerSimd) void loss_products_kernel(GemmProduct dx, ScaledProduct dw, int parts, int tx, int tw,
                                                                                        const int32_t* count) {
    __shared__ __align__(1024) uint8_t shared[S::kBytes];
    if (count) {
        dx.M = dw.K = *count;
        if (tx > 0) tx = static_cast<int>((dx.M + S::BM - 1) / S::BM * ((dx.N + S::BN - 1) / S::BN)) * parts;
        if (static_cast<int>(blockIdx.x) >= tx + tw) return;
    }
    const int64_t share = loss_share(dx.K, parts);
    const bool dw_leads = dw.K > share;
    const int b = blockIdx.x, first = dw_leads ? tw : tx;
    const int tile = b < first ? b : b - first;
    if ((b < first) == dw_leads) {
        gemm_tile<false, false, Store<S, true, false, ScaledProduct>, S>(dw, tile, shared);
        return;
    }
    if constexpr (DIRECT) {
        ScaledProduct p;
        static_cast<GemmProduct&>(p) = dx;
        p.scale = dw.scale;
        p.factor = dw.factor;
        gemm_tile<true, false, Store<S, true, false, ScaledProduct>, S>(p, tile, shared);
        return;
    }
    const int per = tx / parts, part = tile / per;
    const int64_t k0 = share * part;
    GemmProduct p = dx;
    p.K = dx.K - k0 < share ? (dx.K > k0 ? dx.K - k0 : 0) : share;
    if (p.K > 0) {
        p.A = static_cast<const uint16_t*>(dx.A) + k0;
        p.B = static_cast<const uint16_t*>(dx.B) + k0 * dx.ldb;
    }
    float* const sums = static_cast<float*>(dx.ep.y) + part * dx.M * dx.N;
    p.ep.y = sums;
    if (p.ep.residual) p.ep.residual = sums;
    gemm_tile<true, false, Store<S, false>, S>(p, tile % per, shared);
}

// dx from its parts' sums, four columns a thread, and dbias from the row
// tiles' sums, a column a thread.
struct LossFinish {
    const float* sums;                        // [parts][rows][K]
    int parts;
    int64_t M, K, V;
    const int32_t *place, *count;             // NULL: the rows are all M
    uint16_t* dx;
    int64_t lddx, dx_blocks;
    const float* columns;                     // [row tiles][V]
    int tile_rows;
    float* dbias;
    const float* scale;
    float factor;
};

__global__ __launch_bounds__(256) void loss_finish_kernel(LossFinish f) {
    const float by = finite_or_one(*f.scale) * f.factor;
    const int64_t rows = f.count ? *f.count : f.M;
    if (static_cast<int64_t>(blockIdx.x) < f.dx_blocks) {
        const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, per = f.K / 4, m = i / per, k = i % per * 4;
        if (m >= f.M) return;
        const int64_t at = f.place ? f.place[m] : m;
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
        if (at >= 0) {
            s = *reinterpret_cast<const f32x4*>(f.sums + at * f.K + k);
            for (int a = 1; a < f.parts; ++a) s += *reinterpret_cast<const f32x4*>(f.sums + (a * rows + at) * f.K + k);
            s *= by;
        }
        const float v[4] = {s[0], s[1], s[2], s[3]};
        store_n<4>(f.dx, true, m * f.lddx + k, 4, v);
        return;
    }
    const int64_t v = (blockIdx.x - f.dx_blocks) * 256 + threadIdx.x, tiles = (rows + f.tile_rows - 1) / f.tile_rows;
    if (v >= f.V) return;
    float s = 0.f;
#pragma unroll 8
    for (int64_t r = 0; r < tiles; ++r) s += f.columns[r * f.V + v];
    f.dbias[v] = s * by;
}

template <typename S>
hipError_t forward_t(const LossProduct& p, hipStream_t s) {
    hipLaunchKernelGGL((loss_forward_kernel<S>), dim3(static_cast<unsigned>(tiles<S>(p))), dim3(S::kThreads), 0, s, p);
    return hipGetLastError();
}

template <typename S>
hipError_t gradient_t(const LossProduct& p, hipStream_t s) {
    const int64_t n = tiles<S>(p) + (p.clean ? clean_groups(p.M, p.K, S::kThreads) : 0);
    hipLaunchKernelGGL((loss_gradient_kernel<S>), dim3(static_cast<unsigned>(n)), dim3(S::kThreads), 0, s, p);
    return hipGetLastError();
}

template <typename S>
hipError_t products_t(const GemmProduct& dx, const ScaledProduct& dw, int parts, bool direct, const int32_t* count, hipStream_t s) {
    const int64_t tx = dx.ep.y ? tiles<S>(dx) * parts : 0, tw = dw.ep.y ? tiles<S>(dw) : 0;
    const dim3 grid(static_cast<unsigned>(tx + tw)), block(S::kThreads);
    const int nx = static_cast<int>(tx), nw = static_cast<int>(tw);
    if (direct) hipLaunchKernelGGL((loss_products_kernel<S, true>), grid, block, 0, s, dx, dw, parts, nx, nw, count);
    else hipLaunchKernelGGL((loss_products_kernel<S, false>), grid, block, 0, s, dx, dw, parts, nx, nw, count);
    return hipGetLastError();
}

#define GDN_LOSS_TILES(T, CALL)        \
    switch (T) {                       \
        case kLarge: return CALL(Large);   \
        case kWide: return CALL(Wide);     \
        case kMedium: return CALL(Medium); \
        default: return CALL(Small);       \
    }

hipError_t forward(const LossProduct& p, Tiles t, hipStream_t s) {
#define GDN_CALL(S) forward_t<S>(p, s)
    GDN_LOSS_TILES(t, GDN_CALL)
#undef GDN_CALL
}
hipError_t gradient(const LossProduct& p, Tiles t, hipStream_t s) {
#define GDN_CALL(S) gradient_t<S>(p, s)
    GDN_LOSS_TILES(t, GDN_CALL)
#undef GDN_CALL
}
hipError_t products(const GemmProduct& dx, const ScaledProduct& dw, Tiles t, int parts, bool direct, const int32_t* count, hipStream_t s) {
#define GDN_CALL(S) products_t<S>(dx, dw, parts, direct, count, s)
    GDN_LOSS_TILES(t, GDN_CALL)
#undef GDN_CALL
}

int tile_rows(Tiles t) { return t == kLarge || t == kWide ? 256 : t == kMedium ? 128 : 64; }
int tile_cols(Tiles t) { return t == kLarge ? 256 : t == kWide || t == kMedium ? 128 : 64; }

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Times of tiles in us, by which tiles, parts and pieces are chosen: a tile of
// reduction 2048 when the card is full of them (`full`: tiles that share a
// compute unit divided by how many do) and when it has a compute unit to itself
// (`alone`; faster for the large ones, which do not meet the card's power then),
// and what a tile takes beside its reduction, with each epilogue.  Fitted to, in the order 256 x
// 256, 256 x 128, 128 x 128, 64 x 64 (rows x vocabulary x K):
//   forward   4096 x 248320 x 2048: 2965, 3612, 3691, 8226 us;  1537 x 50001 x 1000: 173, 190, 184, 399;
//             200 x 5000 x 4096: 76, 48, 37, 34;  8192 x 20000 x 512: 164, 199, 191, 292
//   dl alone  the same: 3451, 4195, 4284, 8871;  204, 243, 228, 412;  79, 49, 38, 34;  252, 274, 241, 342
//   backward with the best parts: 9262, 10457, 10640, 19558;  504, 579, 575, 840;  71, 67, 63, 70;  700, 552, 559, 857
struct TileTimes {
    double full, alone, forward, gradient, product;
};
constexpr TileTimes kTimes[4] = {{42, 35, 7, 10, 6}, {25, 22, 5, 6.5, 6}, {13, 17, 2.5, 3, 3}, {7.5, 15, 1.5, 1.5, 1.5}};
constexpr double kBytesPerUs = 4.5e6;

// n tiles of one kind: the large ones have a compute unit each and go in rounds
double tiles_us(Tiles t, int64_t n, double reduction, double other) {
    const int cus = compute_units();
    const double r = reduction / 2048, rounds = t == kLarge || t == kWide ? static_cast<double>(up(n, cus)) : static_cast<double>(n) / cus;
    const double full = rounds * (r * kTimes[t].full + other), alone = r * kTimes[t].alone + other;
    return full > alone ? full : alone;
}

// tiles of x w^T
Tiles tiles_for(int64_t M, int64_t N, int64_t K, double TileTimes::*other, double* us) {
    Tiles best = kLarge;
    *us = 1e30;
    for (Tiles t : {kLarge, kWide, kMedium, kSmall}) {
        const double e = tiles_us(t, up(M, tile_rows(t)) * up(N, tile_cols(t)), static_cast<double>(K), kTimes[t].*other);
        if (e < *us) { *us = e; best = t; }
    }
    return best;
}

// work-groups of the kernel for few rows: four of them fill a compute unit
int64_t few_groups(int64_t V) {
    const int64_t n = ((V + 15) / 16 + kFewWaves - 1) / kFewWaves, most = 4 * compute_units();
    return n < most ? n : most;
}

// How the backward pass runs.
struct Plan {
    int64_t piece;                            // columns of the vocabulary at a time
    Tiles gradient, products;
    int parts;                                // of dx's reduction
    bool gather;                              // the rows that count are brought together first
};

// When the last of a launch's tiles ends: n0 of t0 us first, then n1 of t1, each
// taken by the next free of `units`.
double makespan(int64_t n0, double t0, int64_t n1, double t1, int64_t units) {
    const int64_t q = n0 / units, r = n0 % units;             // r units have one more of the first kind
    const double early = static_cast<double>(q) * t0, late = early + (r > 0 ? t0 : 0.0);
    if (n1 == 0) return late;
    const double even = (static_cast<double>(n0) * t0 + static_cast<double>(n1) * t1) / static_cast<double>(units);
    const double least = even > late ? even : late;
    double end = 1e30;
    for (double from : {early, late}) {
        int64_t i = static_cast<int64_t>(std::ceil((least - from) / t1 - 1e-9));
        for (;; ++i) {                                        // (two steps at the most: a unit idles for less than t1)
            const double t = from + static_cast<double>(i) * t1;
            if ((units - r) * static_cast<int64_t>((t - early) / t1 + 1e-9) + r * static_cast<int64_t>((t - late) / t1 + 1e-9) >= n1) {
                if (t < end) end = t;
                break;
            }
        }
    }
    return end;
}

// The best tiles, and parts of dx's reduction, for the products of a piece.  A
// launch has dx's and dw's tiles, the ones of the longer reduction first.
double plan_products(int64_t M, int64_t piece, int64_t K, bool one, Plan* b) {
    const int cus = compute_units();
    double least = 1e30;
    // w in, dw out
    const double memory = 4.0 * static_cast<double>(piece) * K / kBytesPerUs;
    for (int parts = 1; parts <= 32 && (parts == 1 || (piece / parts >= 256 && up(M, 64) * up(K, 64) <= 4096)); parts *= 2) {
        // the parts' sums: out, and in again; one piece without parts has none, and no kernel that adds them
        const double sums = one && parts == 1 ? 0.0 : 8.0 * M * K * parts / kBytesPerUs + (one ? 4.0 : 0.0);
        for (Tiles t : {kLarge, kWide, kMedium, kSmall}) {
            const TileTimes& c = kTimes[t];
            const int64_t tx = up(M, tile_rows(t)) * up(K, tile_cols(t)) * parts, tw = up(piece, tile_rows(t)) * up(K, tile_cols(t));
            const double lx = static_cast<double>(up(piece, parts)) / 2048, lw = static_cast<double>(M) / 2048;
            const double x = lx * c.full + c.product, w = lw * c.full + c.product;
            double us = (lx > lw ? lx : lw) * c.alone + c.product;
            const double full = t == kMedium || t == kSmall ? (static_cast<double>(tx) * x + static_cast<double>(tw) * w) / cus
                                : lx >= lw ? makespan(tx, x, tw, w, cus) : makespan(tw, w, tx, x, cus);
            us = us > full ? us : full;
            us = (us > memory ? us : memory) + sums;
            if (us < least) { least = us; b->products = t; b->parts = parts; }
        }
    }
    return least;
}

// Pieces of up to 160 MiB of dl, which stay in the last-level cache from the
// launch that writes them to the one that reads them twice (2048 x 128000 x
// 1024, forward and backward: 1.93 ms in pieces of 125 MiB, 1.98 in ones of
// 250; 4096 x 248320 x 2048: 12.6 to 13.3 ms at 8 to 24 pieces, in no order).
// Of up to 8192 columns they hold 256 MiB, as dx's sums go out and in with each
// piece (16384 x 128000 x 1024: 13.8 ms, 15.0 in pieces of 4096 columns), and
// they have no fewer than 4096.
constexpr int64_t kPieceBytes = int64_t(160) << 20, kWidePieceBytes = int64_t(256) << 20, kWidePiece = 8192, kLeastPiece = 4096;

Plan plan_of(int64_t M, int64_t V, int64_t K) {
    Plan best{};
    double least = 1e30;
    const int64_t rows = 2 * (M > 0 ? M : 1);
    int64_t most = kWidePieceBytes / rows / 256 * 256;
    if (most > kWidePiece) most = kWidePiece;
    if (most < kPieceBytes / rows / 256 * 256) most = kPieceBytes / rows / 256 * 256;
    if (most < kLeastPiece) most = kLeastPiece;
    int64_t before = 0;
    // (one piece of at most 32 MiB: it is launched fewer times than any other)
    const int tries = 2 * M * V <= (int64_t(32) << 20) ? 1 : 5;
    for (int64_t pieces = up(V, most), tried = 0; tried < tries; pieces += 1 + pieces / 4, ++tried) {
        Plan b{};
        b.piece = up(up(V, pieces), 256) * 256;
        if (b.piece > V) b.piece = V;
        if (b.piece == before || (tried > 0 && b.piece < kLeastPiece)) break;
        before = b.piece;
        double dl;
        b.gradient = tiles_for(M, b.piece, K, &TileTimes::gradient, &dl);
        const double us = (dl + plan_products(M, b.piece, K, b.piece == V, &b) + 8) * static_cast<double>(V) / static_cast<double>(b.piece);   // 8: two launches
        if (us < least) { least = us; best = b; }
    }
    // (two more launches, 15 us: of a call that takes 20 times that)
    best.gather = least >= 300 && M >= 512;
    return best;
}

}  // namespace

// Parts of the forward pass: tiles (or work-groups) across the vocabulary
static int64_t forward_parts(int64_t M, int64_t V, int64_t K, Tiles* t) {
    if (M <= kLinearStreamRows) return few_groups(V);
    double us;
    *t = tiles_for(M, V, K, &TileTimes::forward, &us);
    return (V + tile_cols(*t) - 1) / tile_cols(*t);
}

static int64_t round_256(int64_t n) { return (n + 255) / 256 * 256; }

int64_t loss_workspace(int64_t M, int64_t V, int64_t K) {
    Tiles t;
    return round_256(8 * forward_parts(M, V, K, &t) * M) + round_256(4 * forward_parts(M, V, K, &t) * M);
}

hipError_t launch_loss(const LossCall& c, void* ws, hipStream_t s) {
    Tiles t = kLarge;
    const int64_t parts = forward_parts(c.M, c.V, c.K, &t);
    LossProduct p{};
    p.A = c.x; p.B = c.w;
    p.lda = c.ldx; p.ldb = c.ldw;
    p.M = c.M; p.N = c.V; p.K = c.K;
    p.rows = c.rows;
    p.bias = c.bias;
    uint8_t* const base = static_cast<uint8_t*>(ws);
    p.part = reinterpret_cast<Part*>(base);
    if (c.rows.smooth > 0.f) p.totals = reinterpret_cast<float*>(base + round_256(8 * parts * c.M));
    hipError_t e;
    if (c.M <= kLinearStreamRows) {
        hipLaunchKernelGGL(loss_few_kernel, dim3(static_cast<unsigned>(parts)), dim3(kFewWaves * kWave), 0, s, p);
        e = hipGetLastError();
    } else {
        e = forward(p, t, s);
    }
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(loss_join_kernel, dim3(static_cast<unsigned>((c.M + kJoinRows - 1) / kJoinRows)), dim3(kJoinRows * kJoinSlices), 0, s,
                       p, parts, c.loss, c.lse);
    return hipGetLastError();
}

struct BackwardWs {
    int64_t ld, off_sums, off_columns, off_scale, off_place, off_rows, off_x, total;
};

// dl of a piece, dx's sums, and the row tiles' sums for dbias
static bool is_direct(int64_t V, const Plan& b) { return b.piece >= V && b.parts == 1 && !b.gather; }

static BackwardWs backward_ws(int64_t M, int64_t V, int64_t K, const Plan& b) {
    BackwardWs w;
    w.ld = (b.piece + 63) / 64 * 64;
    w.off_sums = round_256(2 * M * w.ld);
    w.off_columns = w.off_sums + (is_direct(V, b) ? 0 : round_256(4 * b.parts * M * K));
    w.off_scale = w.off_columns + round_256(4 * ((M + tile_rows(b.gradient) - 1) / tile_rows(b.gradient)) * V);
    w.off_place = w.off_scale + 256;          // the rows that count: their places, and their number before them
    w.off_rows = w.off_place + (b.gather ? round_256(4 * M) : 0);
    w.off_x = w.off_rows + (b.gather ? 3 * round_256(4 * M) : 0);
    w.total = w.off_x + round_256(2 * M * K);
    return w;
}

int64_t loss_backward_workspace(int64_t M, int64_t V, int64_t K) { return backward_ws(M, V, K, plan_of(M, V, K)).total; }

hipError_t launch_loss_backward(const LossCall& c, void* ws, hipStream_t s) {
    if (c.M == 0) {                           // sums over no rows
        GemmProduct none{};
        ScaledProduct pw{};
        pw.B = c.x; pw.lda = pw.ldb = 8;
        pw.M = c.V; pw.N = c.K;
        pw.ep.bf16 = 1;
        pw.ep.y = c.dw; pw.ep.ldy = c.lddw;
        const hipError_t e = c.dw ? products(none, pw, kSmall, 1, false, nullptr, s) : hipSuccess;
        return e != hipSuccess ? e : launch_fill_zero(c.dbias, c.V, s);
    }
    const Plan b = plan_of(c.M, c.V, c.K);
    const BackwardWs w = backward_ws(c.M, c.V, c.K, b);
    uint8_t* const base = static_cast<uint8_t*>(ws);
    uint16_t* const dl = reinterpret_cast<uint16_t*>(base);
    float* const sums = reinterpret_cast<float*>(base + w.off_sums);
    float* const columns = reinterpret_cast<float*>(base + w.off_columns);
    const bool direct = is_direct(c.V, b);
    LossRows rows = c.rows;
    const float* scale = rows.dloss;
    if (!rows.dloss_one) {
        float* const top = reinterpret_cast<float*>(base + w.off_scale);
        hipLaunchKernelGGL(loss_scale_kernel, dim3(1), dim3(1024), 0, s, rows, c.M, top);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        scale = top;
    }
    rows.scale = scale;
    const void* x = c.x;
    int64_t ldx = c.ldx;
    const int32_t *place = nullptr, *count = nullptr;
    if (b.gather) {
        int32_t* const list = reinterpret_cast<int32_t*>(base + w.off_place);
        int32_t* const n = reinterpret_cast<int32_t*>(base + w.off_scale + 128);
        uint8_t* const kept = base + w.off_rows;
        const int64_t each = round_256(4 * c.M);
        LossList l{list, reinterpret_cast<uint16_t*>(base + w.off_x), reinterpret_cast<int32_t*>(kept),
                   reinterpret_cast<float*>(kept + each), reinterpret_cast<float*>(kept + 2 * each)};
        hipLaunchKernelGGL(loss_list_kernel, dim3(1), dim3(kListThreads), 0, s, rows, c.M, list, n);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int64_t groups = (c.M + 3) / 4;
        hipLaunchKernelGGL(loss_gather_kernel, dim3(static_cast<unsigned>(groups < (1 << 20) ? groups : 1 << 20)), dim3(256), 0, s, rows, l,
                           static_cast<const uint16_t*>(c.x), c.ldx, c.M, c.K);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        place = list;
        count = n;
        x = l.x;
        ldx = c.K;
        rows.targets = l.targets;
        rows.targets64 = 0;
        rows.ignore = -1;
        rows.lse = l.lse;
        if (!rows.dloss_one) rows.dloss = l.dloss;
    }
    uint16_t* const clean = c.dw && !b.gather ? reinterpret_cast<uint16_t*>(base + w.off_x) : nullptr;
    for (int64_t v0 = 0; v0 < c.V; v0 += b.piece) {
        const int64_t n = c.V - v0 < b.piece ? c.V - v0 : b.piece;
        LossProduct p{};
        p.A = x; p.lda = ldx;
        p.count = count;
        p.B = static_cast<const uint16_t*>(c.w) + v0 * c.ldw; p.ldb = c.ldw;
        p.M = c.M; p.N = n; p.K = c.K;
        p.rows = rows;
        p.v0 = v0;
        p.bias = c.bias ? c.bias + v0 : nullptr;
        p.out.M = c.M; p.out.N = (n + 7) / 8 * 8;
        p.out.ep.y = dl; p.out.ep.ldy = w.ld; p.out.ep.bf16 = 1;
        p.columns = c.dbias ? columns : nullptr;
        p.columns_ld = c.V;
        p.clean = v0 == 0 ? clean : nullptr;
        hipError_t e = gradient(p, b.gradient, s);
        if (e != hipSuccess) return e;
        if (!c.dx && !c.dw) continue;
        GemmProduct px{};
        ScaledProduct pw{};
        pw.scale = scale;
        pw.factor = 1.f - c.rows.smooth;
        px.A = dl; px.lda = w.ld;
        px.B = p.B; px.ldb = c.ldw;
        px.M = c.M; px.N = c.K; px.K = n;
        if (direct) {
            px.ep.y = c.dx; px.ep.ldy = c.lddx; px.ep.bf16 = 1;
        } else {
            px.ep.y = c.dx ? sums : nullptr; px.ep.ldy = c.K;
            px.ep.residual = v0 > 0 ? sums : nullptr; px.ep.ldr = c.K;
        }
        pw.A = dl; pw.lda = w.ld;
        pw.B = clean ? clean : x; pw.ldb = clean ? c.K : ldx;
        pw.M = n; pw.N = c.K; pw.K = c.M;
        pw.ep.bf16 = 1;
        pw.ep.y = c.dw ? static_cast<uint16_t*>(c.dw) + v0 * c.lddw : nullptr; pw.ep.ldy = c.lddw;
        e = products(px, pw, b.products, b.parts, direct, p.count, s);
        if (e != hipSuccess) return e;
    }
    const int64_t dx_blocks = c.dx && !direct ? (c.M * (c.K / 4) + 255) / 256 : 0, bias_blocks = c.dbias ? (c.V + 255) / 256 : 0;
    if (dx_blocks + bias_blocks == 0) return hipSuccess;
    const LossFinish f{sums, b.parts, c.M, c.K, c.V, place, count, static_cast<uint16_t*>(c.dx), c.lddx, dx_blocks, columns,
                       tile_rows(b.gradient), c.dbias, scale, 1.f - c.rows.smooth};
    hipLaunchKernelGGL(loss_finish_kernel, dim3(static_cast<unsigned>(dx_blocks + bias_blocks)), dim3(256), 0, s, f);
    return hipGetLastError();
}

}  // namespace gdn
