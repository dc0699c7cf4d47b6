// gdn_linear.hip -- the linear layer with its epilogue in the product's
// kernel, y = act(x w^T + bias) + residual, and its backward pass.
//
// Forward: y[m][n] = sum_k x[m][k] w[n][k].  Backward, with p the
// pre-activation: dp = dy act'(p), dbias[n] = sum_m dp, dx = dp w
// (dx[m][k] = sum_n dp[m][n] w[n][k]), dw = dp^T x (dw[n][k] = sum_m dp[m][n]
// x[m][k]).  All three products run on one tiled kernel: an operand is a
// matrix whose rows are either the output's rows with the reduction
// contiguous (x and w forward, dp for dx), or the reduction's rows with the
// output's rows contiguous (w for dx, dp and x for dw).  The second kind is
// transposed on the way from LDS to the matrix cores (ds_read_b64_tr_b16),
// so nothing is ever transposed in memory.
//
// Few rows: the product is a stream over w, and bound by HBM.  Up to 16 rows
// each work-group takes 16 columns with K split over its waves; up to 256 rows
// K is split over work-groups of 64 columns, whose sums a second kernel adds.
#include <cmath>

#include "gdn_tiles.hpp"

namespace gdn {

namespace {

template <typename S>
__global__ __launch_bounds__(S::kThreads, S::kPerSimd) void linear_forward_kernel(GemmProduct p) {
    __shared__ __align__(1024) uint8_t shared[S::kBytes];
    gemm_tile<true, true, Store<S, false>, S>(p, blockIdx.x, shared);
}

// dbias from the row blocks' column sums, each column's blocks in a fixed
// order: 64 columns a work-group.  The backward products' launches have these
// work-groups too, after their tiles (a launch of its own takes 5 us).
constexpr int kSumCols = 64;

struct ColumnSums {
    const float* part;                        // [blocks][N]
    int64_t blocks, N;
    float* out;                               // NULL: none
};

template <int THREADS>
__device__ __forceinline__ void column_sums(const ColumnSums& c, int block, float* t) {
    constexpr int kSlices = THREADS / kSumCols;
    const int col = threadIdx.x % kSumCols, sl = threadIdx.x / kSumCols;
    const int64_t n = static_cast<int64_t>(block) * kSumCols + col;
    float s = 0.f;
    if (n < c.N) {
#pragma unroll 8
        for (int64_t i = sl; i < c.blocks; i += kSlices) s += c.part[i * c.N + n];
    }
    t[threadIdx.x] = s;
    __syncthreads();
    if (sl == 0 && n < c.N) {
#pragma unroll
        for (int k = 1; k < kSlices; ++k) s += t[k * kSumCols + col];
        c.out[n] = s;
    }
}

static int64_t sum_blocks(const ColumnSums& c) { return c.out ? (c.N + kSumCols - 1) / kSumCols : 0; }

// dx and dw in one launch: each alone often has fewer tiles than the card has
// compute units.  The product with the longer reduction takes the first
// work-groups, so that its tiles are not the last ones running.
// tx, tw: tiles (or tiles in parts) of dx and dw.
__device__ __forceinline__ bool is_dx(int tx, int tw, bool dw_leads, int* tile) {
    const int b = blockIdx.x, first = dw_leads ? tw : tx;
    *tile = b < first ? b : b - first;
    return (b < first) != dw_leads;
}

template <typename S>
__global__ __launch_bounds__(S::kThreads, S::kPerSimd) void linear_backward_kernel(GemmProduct dx, GemmProduct dw, int tx, int tw,
                                                                                          ColumnSums sums) {
    __shared__ __align__(1024) uint8_t shared[S::kBytes];
    int tile;
    if (static_cast<int>(blockIdx.x) >= tx + tw) {
        column_sums<S::kThreads>(sums, blockIdx.x - (tx + tw), reinterpret_cast<float*>(shared));
        return;
    }
    if (is_dx(tx, tw, dw.K > dx.K, &tile)) gemm_tile<true, false, Store<S, true>, S>(dx, tile, shared);
    else gemm_tile<false, false, Store<S, true>, S>(dw, tile, shared);
}

// ---- the reduction in parts ------------------------------------------------------
// Products with fewer tiles than compute units, and enough of a reduction:
// part s of `parts` takes an equal share of it (in rounds of 128) and leaves
// its sums in 32 bits; a second kernel adds the parts in order and finishes.
__host__ __device__ inline int64_t part_share(int64_t K, int parts) {
    return ((K + 127) / 128 + parts - 1) / parts * 128;
}

template <bool AK, bool BK>
__device__ __forceinline__ void gemm_part(const GemmProduct& whole, int block, float* sums, int parts, uint8_t* shared) {
    const int tiles = static_cast<int>(((whole.M + 63) / 64) * ((whole.N + 63) / 64));
    const int part = block / tiles;
    const int64_t share = part_share(whole.K, parts), k0 = share * part;
    GemmProduct p = whole;
    p.K = whole.K - k0 < share ? (whole.K > k0 ? whole.K - k0 : 0) : share;
    if (p.K > 0) {
        p.A = static_cast<const uint16_t*>(whole.A) + (AK ? k0 : k0 * whole.lda);
        p.B = static_cast<const uint16_t*>(whole.B) + (BK ? k0 : k0 * whole.ldb);
    }
    p.ep.y = sums + part * whole.M * whole.N;
    p.ep.ldy = whole.N;
    p.ep.bf16 = 0;
    gemm_tile<AK, BK, Store<Small, true>, Small>(p, block % tiles, shared);
}

__global__ __launch_bounds__(Small::kThreads, Small::kPerSimd) void linear_part_kernel(GemmProduct p, float* sums, int parts) {
    __shared__ __align__(1024) uint8_t shared[Small::kBytes];
    gemm_part<true, true>(p, blockIdx.x, sums, parts, shared);
}

// dx and dw in parts
__global__ __launch_bounds__(Small::kThreads, Small::kPerSimd) void linear_backward_part_kernel(
        GemmProduct dx, GemmProduct dw, float* sx, float* sw, int px, int pw, int tx, int tw, ColumnSums sums) {
    __shared__ __align__(1024) uint8_t shared[Small::kBytes];
    int tile;
    if (static_cast<int>(blockIdx.x) >= tx + tw) {
        column_sums<Small::kThreads>(sums, blockIdx.x - (tx + tw), reinterpret_cast<float*>(shared));
        return;
    }
    if (is_dx(tx, tw, part_share(dw.K, pw) > part_share(dx.K, px), &tile)) gemm_part<true, false>(dx, tile, sx, px, shared);
    else gemm_part<false, false>(dw, tile, sw, pw, shared);
}

// four columns a thread
__device__ __forceinline__ void join(const GemmProduct& p, const float* sums, int parts, int64_t i) {
    const int64_t per = (p.N + 3) / 4, m = i / per, n = (i % per) * 4;
    if (m >= p.M) return;
    const int nv = p.N - n < 4 ? static_cast<int>(p.N - n) : 4;
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    const int64_t step = p.M * p.N, at = m * p.N + n;
    int s = 0;
    for (; s + 4 <= parts; s += 4) {
        float t[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) load_n<4>(sums, false, (s + u) * step + at, nv, t[u]);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] += t[u][e];
    }
    for (; s < parts; ++s) {
        float t[4];
        load_n<4>(sums, false, s * step + at, nv, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] += t[e];
    }
    finish_n<4>(p.ep, m, n, nv, f);
}

constexpr int kJoinThreads = 256;

__global__ __launch_bounds__(kJoinThreads) void linear_join_kernel(GemmProduct p, const float* sums, int parts) {
    join(p, sums, parts, static_cast<int64_t>(blockIdx.x) * kJoinThreads + threadIdx.x);
}

__global__ __launch_bounds__(kJoinThreads) void linear_backward_join_kernel(GemmProduct dx, GemmProduct dw, const float* sx,
                                                                           const float* sw, int px, int pw, int first) {
    const int b = blockIdx.x;
    if (b < first) join(dx, sx, px, static_cast<int64_t>(b) * kJoinThreads + threadIdx.x);
    else join(dw, sw, pw, static_cast<int64_t>(b - first) * kJoinThreads + threadIdx.x);
}

// ---- few rows --------------------------------------------------------------------
// Up to 16 rows; bound by HBM: 1 x 12352 x 2048 takes 12.7 us, 4.0 TB/s of
// weights.  (More rows would read all of x through each compute unit's L1 for
// every 16 columns: 64 x 2048 x 4096 took 23 us so, and 13 in parts.)  A
// work-group owns 16 rows of w (16 columns of y) and splits K over its waves;
// per 64-wide step of K the lanes of a row read two runs of 64 bytes of their
// weight row and of their row of x, DEPTH steps ahead.  Steps past a
// wave's share and k past K read zeros.  The waves' partial tiles are summed
// in LDS in wave order.
constexpr int kFewStep = 64, kFewWaves = 8;

template <int DEPTH>
__global__ __launch_bounds__(kFewWaves * kWave, 2) void linear_few_kernel(GemmProduct p) {
    __shared__ f32x4 part[kFewWaves][kWave];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
    const int l16 = lane % 16, lq = lane / 16;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
    const int steps = static_cast<int>((p.K + kFewStep - 1) / kFewStep);
    const int s0 = static_cast<int>(static_cast<int64_t>(steps) * wave / kFewWaves);
    const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (wave + 1) / kFewWaves);
    const int64_t end = static_cast<int64_t>(s1) * kFewStep < p.K ? static_cast<int64_t>(s1) * kFewStep : p.K;
    // rows past the end: never stored
    const uint16_t* brow = static_cast<const uint16_t*>(p.B) + (n0 + l16 < p.N ? n0 + l16 : p.N - 1) * p.ldb;
    const uint16_t* arow = static_cast<const uint16_t*>(p.A) + (l16 < p.M ? l16 : p.M - 1) * p.lda;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    u32x4 bf[DEPTH][2], af[DEPTH][2];
    auto load = [&](int st, int slot) {
        const int64_t k0 = static_cast<int64_t>(st) * kFewStep + lq * 8;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t k = k0 + 32 * h;
            bf[slot][h] = *reinterpret_cast<const u32x4*>(k < end ? brow + k : zero_chunk);
            af[slot][h] = *reinterpret_cast<const u32x4*>(k < end ? arow + k : zero_chunk);
        }
    };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(s0 + d, d);
    for (int st = s0; st < s1; st += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            acc = mfma(bf[d][0], af[d][0], acc);
            acc = mfma(bf[d][1], af[d][1], acc);
            if (st + DEPTH < s1) load(st + DEPTH + d, d);
        }
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave != 0) return;
    f32x4 s = part[0][lane];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) s += part[w][lane];
    const int64_t m = l16, n = n0 + 4 * lq;
    if (m >= p.M || n >= p.N) return;
    const int nv = p.N - n < 4 ? static_cast<int>(p.N - n) : 4;
    float f[4] = {s[0], s[1], s[2], s[3]};
    finish_n<4>(p.ep, m, n, nv, f);
}

// ---- dp = dy act'(p) and its column sums -------------------------------------------
// Bound: HBM (dy and p in, dp out: 4096 x 4096 in bf16 25 us, 4.0 TB/s).  A work-group covers 32 rows x 256
// columns: 32 lanes of eight columns, every eighth row, the four rows' loads
// in flight together.  dp is rounded to bf16, the products' operand type: what
// it had beyond that would need a second product (dp as the sum of two bf16
// values), twice the work of dx and dw.  Rounded, their error against 64 bits is
// 2.3e-3 of their norm (4096 x 4096 x 2048, tanh gelu), where their own rounding
// makes 1.7e-3.  The sums are of the values before that.
constexpr int kDpRows = 32, kDpCols = 256, kDpBatch = 4;

// ROWS, COLS: all rows of the block, all eight columns of the lane exist.
// (dy's type and the columns are settled outside, so that the batch's loads
// stand together: a branch around each waits for each, 9.2 us instead of 6.8
// at 1537 x 1000.)
template <bool BF16, bool ROWS, bool COLS>
__device__ __forceinline__ void dp_rows(const LinearDp& p, int64_t m0, int64_t n, int nv, int g, float* s) {
#pragma unroll
    for (int i0 = 0; i0 < kDpRows / 8; i0 += kDpBatch) {
        float d[kDpBatch][8], q[kDpBatch][8];
        int64_t row[kDpBatch];                    // rows past the end read the last one
#pragma unroll
        for (int u = 0; u < kDpBatch; ++u) {
            const int64_t m = m0 + g + 8 * (i0 + u);
            row[u] = ROWS || m < p.M ? m : p.M - 1;
            load_n<8>(p.dy, BF16, row[u] * p.ldy + n, COLS ? 8 : nv, d[u]);
        }
        if (p.act != kActNone) {
#pragma unroll
            for (int u = 0; u < kDpBatch; ++u) {
                load_n<8>(p.preact, true, row[u] * p.ldp + n, COLS ? 8 : nv, q[u]);
            }
            switch (p.act) {
#define GDN_SLOPE_CASE(ACT)                                                               \
    case ACT:                                                                             \
        _Pragma("unroll") for (int u = 0; u < kDpBatch; ++u)                              \
            _Pragma("unroll") for (int e = 0; e < 8; ++e) d[u][e] *= slope(q[u][e], ACT); \
        break;
                GDN_SLOPE_CASE(kActRelu)
                GDN_SLOPE_CASE(kActGelu)
                GDN_SLOPE_CASE(kActGeluTanh)
                GDN_SLOPE_CASE(kActSilu)
#undef GDN_SLOPE_CASE
                default: break;
            }
        }
#pragma unroll
        for (int u = 0; u < kDpBatch; ++u) {
            const int64_t m = m0 + g + 8 * (i0 + u);
            if (!ROWS && m >= p.M) break;
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += d[u][e];              // (columns past the end: zeros)
            if (p.dp && (COLS || n < p.ldd)) {
                const u32x4 h = {pack_bf16(d[u][0], d[u][1]), pack_bf16(d[u][2], d[u][3]), pack_bf16(d[u][4], d[u][5]),
                                 pack_bf16(d[u][6], d[u][7])};
                *reinterpret_cast<u32x4*>(p.dp + m * p.ldd + n) = h;   // (the workspace's rows: whole 16-byte runs)
            }
        }
    }
}

template <bool BF16>
__global__ __launch_bounds__(256) void linear_dp_kernel(LinearDp p) {
    __shared__ float sums[8][kDpCols];
    const int lane = threadIdx.x % 32, g = threadIdx.x / 32;
    const int64_t block = blockIdx.x / p.cols, col0 = static_cast<int64_t>(blockIdx.x % p.cols) * kDpCols;
    const int64_t m0 = block * kDpRows, n = col0 + 8 * lane;
    const int64_t left = p.N - n;
    const int nv = left < 0 ? 0 : (left < 8 ? static_cast<int>(left) : 8);
    float s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = 0.f;
    if (nv == 8 && m0 + kDpRows <= p.M) dp_rows<BF16, true, true>(p, m0, n, nv, g, s);
    else if (nv == 8) dp_rows<BF16, false, true>(p, m0, n, nv, g, s);
    else if (nv > 0) dp_rows<BF16, false, false>(p, m0, n, nv, g, s);
    if (!p.part) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[g][8 * lane + e] = s[e];
    __syncthreads();
    const int64_t c = col0 + threadIdx.x;
    if (c < p.N) {
        float t = sums[0][threadIdx.x];
#pragma unroll
        for (int k = 1; k < 8; ++k) t += sums[k][threadIdx.x];
        p.part[block * p.N + c] = t;
    }
}

__global__ __launch_bounds__(1024) void linear_sum_kernel(ColumnSums c) {
    __shared__ float t[1024];
    column_sums<1024>(c, blockIdx.x, t);
}

template <typename S>
hipError_t forward_t(const GemmProduct& p, hipStream_t s) {
    hipLaunchKernelGGL((linear_forward_kernel<S>), dim3(static_cast<unsigned>(tiles<S>(p))), dim3(S::kThreads), 0, s, p);
    return hipGetLastError();
}

template <typename S>
hipError_t backward_t(const GemmProduct& dx, const GemmProduct& dw, const ColumnSums& sums, hipStream_t s) {
    const int64_t t1 = dx.ep.y ? tiles<S>(dx) : 0, t2 = dw.ep.y ? tiles<S>(dw) : 0;
    hipLaunchKernelGGL((linear_backward_kernel<S>), dim3(static_cast<unsigned>(t1 + t2 + sum_blocks(sums))), dim3(S::kThreads), 0,
                       s, dx, dw, static_cast<int>(t1), static_cast<int>(t2), sums);
    return hipGetLastError();
}

}  // namespace

static hipError_t forward(const GemmProduct& p, Tiles t, hipStream_t s) {
    switch (t) {
        case kLarge: return forward_t<Large>(p, s);
        case kWide: return forward_t<Wide>(p, s);
        case kMedium: return forward_t<Medium>(p, s);
        default: return forward_t<Small>(p, s);
    }
}

// Columns n0 .. n0 + n - 1 of a product
static GemmProduct columns(const GemmProduct& p, int64_t n0, int64_t n) {
    GemmProduct c = p;
    const size_t es = p.ep.bf16 ? 2 : 4;
    c.N = n;
    c.B = static_cast<const uint16_t*>(p.B) + n0 * p.ldb;
    if (c.ep.bias) c.ep.bias += n0;
    if (c.ep.preact) c.ep.preact += n0;
    if (c.ep.residual) c.ep.residual = static_cast<const uint8_t*>(p.ep.residual) + n0 * es;
    c.ep.y = static_cast<uint8_t*>(p.ep.y) + n0 * es;
    return c;
}

// Parts of the reduction of 17 to 64 rows: as many as there are compute units
// for each tile of 64 columns, of 256 at least.  64 x 2048 x 4096: 17.0 us with
// 16 parts, 13.2 with 8, 14.6 with 4; 64 x 12352 x 2048: 20.3 with 1, 22.6 with 2.
// Of 65 to 256 rows: the same for four tiles of rows, of 1024 at least (128 x
// 1024 x 8192: 53 us in one part, 21 in four).  The number is one for all the
// rows of a range, so that a row's sum does not depend on how many there are.
int linear_parts(int64_t M, int64_t N, int64_t K) {
    if (M <= kLinearStreamRows || M > kLinearSomeRows || N <= 0) return 1;
    const bool few = M <= kLinearFewRows;
    const int64_t want = compute_units() / ((few ? 1 : 4) * ((N + 63) / 64)), most = K / (few ? 256 : 1024);
    const int64_t n = want < most ? want : most;
    return n < 1 ? 1 : static_cast<int>(n > 64 ? 64 : n);
}

// Tiles of more than kLinearFewRows rows.  A last column of tiles that is
// nearly empty can cost a whole round of them (12352 = 48 x 256 + 64 columns
// at 4096 rows: 784 tiles, four rounds instead of three; with gelu, bias and
// residual 210 us): then the rest goes by itself in smaller tiles (184 us).  A
// column's sum runs in the same order either way.  (The times compared are
// those of K = 2048 whatever K is: with a short one the second launch can cost
// more than the round, 2048 x 8264 x 64 23 us.)
struct ForwardPlan {
    int64_t columns;                              // of `tiles`; N or what is left over goes in `rest`
    Tiles tiles, rest;
};

static ForwardPlan forward_plan(const GemmProduct& p) {
    const int cus = compute_units();
    const Choice whole = choose(p, cus);
    const int64_t rest = p.N % 256, main = p.N - rest;
    if (rest > 0 && main > 0) {
        GemmProduct m = p, r = p;
        m.N = main;
        r.N = rest;
        const Choice cm = choose(m, cus), cr = choose(r, cus);
        if (cm.us + cr.us + 3.0 < whole.us) return {main, cm.tiles, cr.tiles};   // 3: the second launch
    }
    return {p.N, whole.tiles, whole.tiles};
}

static void tile_size(Tiles t, int32_t* rows, int32_t* cols) {
    *rows = t == kLarge ? Large::BM : t == kWide ? Wide::BM : t == kMedium ? Medium::BM : Small::BM;
    *cols = t == kLarge ? Large::BN : t == kWide ? Wide::BN : t == kMedium ? Medium::BN : Small::BN;
}

void linear_tiles(int64_t M, int64_t N, int64_t K, int32_t* rows, int32_t* cols) {
    GemmProduct p{};
    p.M = M; p.N = N; p.K = K;
    if (M <= kLinearStreamRows) *rows = *cols = 16;
    else tile_size(linear_parts(M, N, K) > 1 || M <= kLinearFewRows ? kSmall : forward_plan(p).tiles, rows, cols);
}

static int64_t join_blocks(const GemmProduct& p) { return (p.M * ((p.N + 3) / 4) + kJoinThreads - 1) / kJoinThreads; }

hipError_t launch_linear(const GemmProduct& given, float* sums, hipStream_t s) {
    if (given.M <= 0 || given.N <= 0) return hipSuccess;
    GemmProduct p = given;
    if (p.ep.act == kActGelu && p.ep.bf16) p.ep.act = kActGeluBf16;
    if (p.M <= kLinearStreamRows) {
        hipLaunchKernelGGL((linear_few_kernel<4>), dim3(static_cast<unsigned>((p.N + 15) / 16)), dim3(kFewWaves * kWave), 0, s, p);
        return hipGetLastError();
    }
    const int parts = linear_parts(p.M, p.N, p.K);
    if (parts > 1) {
        hipLaunchKernelGGL(linear_part_kernel, dim3(static_cast<unsigned>(tiles<Small>(p) * parts)), dim3(Small::kThreads), 0, s, p,
                           sums, parts);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(linear_join_kernel, dim3(static_cast<unsigned>(join_blocks(p))), dim3(kJoinThreads), 0, s, p, sums, parts);
        return hipGetLastError();
    }
    if (p.M <= kLinearFewRows) return forward_t<Small>(p, s);
    const ForwardPlan plan = forward_plan(p);
    if (plan.columns == p.N) return forward(p, plan.tiles, s);
    const hipError_t e = forward(columns(p, 0, plan.columns), plan.tiles, s);
    return e != hipSuccess ? e : forward(columns(p, plan.columns, p.N - plan.columns), plan.rest, s);
}

int64_t linear_dp_blocks(int64_t M) { return (M + kDpRows - 1) / kDpRows; }

// How the backward products run, by the sizes alone (so that either has the
// same bits with and without the other): dx (reduction N) and dw (reduction M) share
// a launch, so their tiles' times are weighed by their reductions: the work
// over the compute units in rounds of the shorter reduction, and no less than
// one tile of the longer one takes by itself.  Reductions may be cut into parts, which costs the sums' way through
// memory and a launch.  Measured, in the order 256 x 256, 256 x 128, 128 x
// 128, 64 x 64, and the best number of parts' time:
//    700 x 8192 x  256: 126,  91,  65,  38 us, 24 in parts of 2048
//   8192 x  512 x  512: 126,  84,  62,  44 us, 33 in parts of 2048
//   4096 x 1000 x  512:  67,  45,  33,  27 us, 29 in parts of 2048
//   1537 x 1000 x 2048:  39,  26,  24,  29 us, 43 in parts of 1024
//   2048 x 2048 x 2048:  42,  32,  36,  54 us, 77 in parts of 1024
//   8192 x 2048 x 2048: 146, 118, 131, 227 us, 245 in parts of 2048
//   4096 x 4096 x 2048:  97, 125, 127, 221 us, 243 in parts of 2048
struct BackwardPlan {
    Tiles tiles;
    int px, pw;                                   // parts of dx's and dw's reductions (1, 1: no sums)
};

static BackwardPlan backward_plan(int64_t M, int64_t N, int64_t K) {
    const int cus = compute_units();
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    auto us = [&](int bm, int bn, double each, double alone, int px, int pw) {
        const int64_t tx = up(M, bm) * up(K, bn) * px, tw = up(N, bm) * up(K, bn) * pw;
        const double lx = static_cast<double>(up(N, px)), lw = static_cast<double>(up(M, pw));
        const double least = lx < lw ? lx : lw, most = lx < lw ? lw : lx;
        // (large outputs have tiles enough; a launch holds 2^32 work-items)
        if (least <= 0 || (px * pw > 1 && tx + tw > (int64_t(1) << 21))) return px * pw > 1 ? 1e30 : 0.0;
        const double work = std::ceil((tx * lx + tw * lw) / (cus * least)) * least * each;
        return (work > most * alone ? work : most * alone) / 2048;
    };
    BackwardPlan best{kLarge, 1, 1};
    double least = us(256, 256, kLargeUs, kLargeUs, 1, 1);
    auto offer = [&](double t, BackwardPlan p) {
        if (t < least) { least = t; best = p; }
    };
    offer(us(256, 128, kWideUs, kWideUs, 1, 1), {kWide, 1, 1});
    offer(us(128, 128, kMediumUs, kMediumAlone, 1, 1), {kMedium, 1, 1});
    offer(us(64, 64, kSmallUs, kSmallAlone, 1, 1), {kSmall, 1, 1});
    for (int len = 256; len <= (1 << 20); len *= 2) {
        const int px = N > len ? static_cast<int>(up(N, len)) : 1, pw = M > len ? static_cast<int>(up(M, len)) : 1;
        if (px == 1 && pw == 1) break;
        if (px > 64 || pw > 64) continue;         // (the sums are joined one after the other)
        const double sums = 8.0 * static_cast<double>(K) * (static_cast<double>(px) * M + static_cast<double>(pw) * N);
        offer(us(64, 64, kSmallUs, kSmallAlone, px, pw) + 5 + sums / 3e6, {kSmall, px, pw});
    }
    return best;
}

// (the sums' places: no sums where no reduction is cut)
void linear_backward_parts(int64_t M, int64_t N, int64_t K, int* dx, int* dw) {
    const BackwardPlan b = backward_plan(M, N, K);
    *dx = b.px;
    *dw = b.pw;
}

void linear_backward_tiles(int64_t M, int64_t N, int64_t K, int32_t* rows, int32_t* cols) {
    tile_size(backward_plan(M, N, K).tiles, rows, cols);
}

hipError_t launch_linear_backward(const LinearDp& dp, const GemmProduct& dx, const GemmProduct& dw, float* dbias, float* sums_dx,
                                  float* sums_dw, hipStream_t s) {
    if (dp.dp || dp.part) {
        LinearDp d = dp;
        d.cols = static_cast<int>(((dp.dp ? dp.ldd : dp.N) + kDpCols - 1) / kDpCols);
        const int64_t grid = d.cols * linear_dp_blocks(dp.M);
        if (d.dy_bf16) hipLaunchKernelGGL(linear_dp_kernel<true>, dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, d);
        else hipLaunchKernelGGL(linear_dp_kernel<false>, dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, d);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    ColumnSums sums{dp.part, linear_dp_blocks(dp.M), dp.N, dbias};
    const bool products = dx.ep.y || dw.ep.y;
    const BackwardPlan plan = backward_plan(dp.M, dp.N, dx.N);
    const int px = plan.px, pw = plan.pw;
    // (a large tile has a compute unit to itself: the sums would wait for its end)
    if (dbias && (!products || plan.tiles == kLarge || plan.tiles == kWide)) {
        hipLaunchKernelGGL(linear_sum_kernel, dim3(static_cast<unsigned>(sum_blocks(sums))), dim3(1024), 0, s, sums);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        sums.out = nullptr;
    }
    if (!products) return hipSuccess;
    if (px > 1 || pw > 1) {
        const int64_t t1 = dx.ep.y ? tiles<Small>(dx) * px : 0, t2 = dw.ep.y ? tiles<Small>(dw) * pw : 0;
        hipLaunchKernelGGL(linear_backward_part_kernel, dim3(static_cast<unsigned>(t1 + t2 + sum_blocks(sums))),
                           dim3(Small::kThreads), 0, s, dx, dw, sums_dx, sums_dw, px, pw, static_cast<int>(t1),
                           static_cast<int>(t2), sums);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int64_t b1 = dx.ep.y ? join_blocks(dx) : 0, b2 = dw.ep.y ? join_blocks(dw) : 0;
        hipLaunchKernelGGL(linear_backward_join_kernel, dim3(static_cast<unsigned>(b1 + b2)), dim3(kJoinThreads), 0, s, dx, dw,
                           sums_dx, sums_dw, px, pw, static_cast<int>(b1));
        return hipGetLastError();
    }
    switch (plan.tiles) {
        case kLarge: return backward_t<Large>(dx, dw, sums, s);
        case kWide: return backward_t<Wide>(dx, dw, sums, s);
        case kMedium: return backward_t<Medium>(dx, dw, sums, s);
        default: return backward_t<Small>(dx, dw, sums, s);
    }
}

}  // namespace gdn
