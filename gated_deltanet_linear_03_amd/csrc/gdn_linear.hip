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
// Few rows (M <= 64): the product is a stream over w, and bound by HBM; the
// few-row kernel reads each weight once in 256-byte runs with K split over
// the waves of a work-group.
#include "gdn_device.hpp"
#include "gdn_kernels.hpp"

namespace gdn {

namespace {

__device__ __align__(16) const uint16_t zero_chunk[8] = {};   // what lanes past the reduction's end read

// ---- activations -------------------------------------------------------------
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float sigmoid_fast(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// e^(y^2) erfc(y) for y >= 0 as a polynomial in t = 1 / (1 + 0.33 y)
// (degree 8 without a constant term, least squares on the relative error over
// y in [0, 9.5], where it is below 1e-7; beyond, e^(-y^2) is 0 in 32 bits):
// the left tail of gelu keeps its relative precision.
__device__ __forceinline__ float erfcx_poly(float y) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.33f, y, 1.0f));
    float p = -1.359293708e-01f;
    p = fmaf(p, t, 4.626906779e-01f);
    p = fmaf(p, t, -3.554432462e-01f);
    p = fmaf(p, t, 4.125456214e-01f);
    p = fmaf(p, t, 4.500852111e-02f);
    p = fmaf(p, t, 2.019244518e-01f);
    p = fmaf(p, t, 1.828371481e-01f);
    p = fmaf(p, t, 1.863661150e-01f);
    return p * t;
}

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kTanhC = 0.79788456080286536f;      // sqrt(2 / pi)
constexpr float kTanhD = 0.044715f;

// half of erfc(|p| / sqrt(2)), and e^(-p^2 / 2)
__device__ __forceinline__ float half_erfc(float p, float* e) {
    *e = __builtin_amdgcn_exp2f(p * p * (-0.5f * kLog2e));
    return 0.5f * erfcx_poly(fabsf(p) * kSqrtHalf) * *e;
}

__device__ __forceinline__ float activate(float p, int act) {
    switch (act) {
        case kActRelu: return p < 0.f ? 0.f : p;      // NaN stays NaN
        case kActGelu: {
            float e;
            const float c = half_erfc(p, &e);
            return p * (p > 0.f ? 1.f - c : c);
        }
        case kActGeluTanh: return p * sigmoid_fast(2.f * kTanhC * fmaf(kTanhD * p * p, p, p));
        case kActSilu: return p * sigmoid_fast(p);
        default: return p;
    }
}

__device__ __forceinline__ float slope(float p, int act) {
    // far out the slopes are 0 or 1 to the bit: what multiplies their
    // vanishing parts stays finite
    const float pc = fminf(fmaxf(p, -128.f), 128.f);
    switch (act) {
        case kActRelu: return p != p ? p : (p > 0.f ? 1.f : 0.f);
        case kActGelu: {
            float e;
            const float c = half_erfc(p, &e);
            return (p > 0.f ? 1.f - c : c) + pc * e * 0.3989422804014327f;   // 1 / sqrt(2 pi)
        }
        case kActGeluTanh: {
            const float q = sigmoid_fast(2.f * kTanhC * fmaf(kTanhD * p * p, p, p));
            const float d = 2.f * kTanhC * fmaf(3.f * kTanhD * pc, pc, 1.f);
            return q + pc * q * (1.f - q) * d;
        }
        case kActSilu: {
            const float q = sigmoid_fast(p);
            return q * fmaf(pc, 1.f - q, 1.f);
        }
        default: return 1.f;
    }
}

// ---- output elements -----------------------------------------------------------
struct __attribute__((packed, aligned(2))) Half4 { uint32_t lo, hi; };
struct __attribute__((packed, aligned(4))) Float4 { float e[4]; };

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// up to four adjacent elements, element aligned only
__device__ __forceinline__ void load4(const void* p, bool bf16, int64_t at, int nv, float* f) {
    if (bf16) {
        const uint16_t* q = static_cast<const uint16_t*>(p) + at;
        if (nv == 4) {
            const Half4 h = *reinterpret_cast<const Half4*>(q);
            f[0] = __uint_as_float(h.lo << 16);
            f[1] = __uint_as_float(h.lo & 0xFFFF0000u);
            f[2] = __uint_as_float(h.hi << 16);
            f[3] = __uint_as_float(h.hi & 0xFFFF0000u);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = e < nv ? bf16_bits_to_f32(q[e]) : 0.f;
        }
    } else {
        const float* q = static_cast<const float*>(p) + at;
        if (nv == 4) {
            const Float4 h = *reinterpret_cast<const Float4*>(q);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = h.e[e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = e < nv ? q[e] : 0.f;
        }
    }
}

__device__ __forceinline__ void store4(void* p, bool bf16, int64_t at, int nv, const float* f) {
    if (bf16) {
        uint16_t* q = static_cast<uint16_t*>(p) + at;
        if (nv == 4) {
            Half4 h;
            h.lo = pack_bf16(f[0], f[1]);
            h.hi = pack_bf16(f[2], f[3]);
            *reinterpret_cast<Half4*>(q) = h;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < nv) q[e] = f32_to_bf16_bits(f[e]);
        }
    } else {
        float* q = static_cast<float*>(p) + at;
        if (nv == 4) {
            Float4 h;
#pragma unroll
            for (int e = 0; e < 4; ++e) h.e[e] = f[e];
            *reinterpret_cast<Float4*>(q) = h;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < nv) q[e] = f[e];
        }
    }
}

// y = act(sum + bias) + residual for up to four adjacent columns of one row;
// preact receives sum + bias
__device__ __forceinline__ void finish4(const GemmEpilogue& ep, int64_t m, int64_t n, int nv, float* f) {
    if (ep.bias) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < nv) f[e] += ep.bias[n + e];
    }
    if (ep.preact) store4(ep.preact, true, m * ep.ldp + n, nv, f);
    if (ep.act != kActNone) {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = activate(f[e], ep.act);
    }
    if (ep.residual) {
        float r[4];
        load4(ep.residual, ep.bf16, m * ep.ldr + n, nv, r);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] += r[e];
    }
    store4(ep.y, ep.bf16, m * ep.ldy + n, nv, f);
}

// ---- the tiled kernel ------------------------------------------------------------
constexpr int kThreads = 512, kWaves = kThreads / kWave;
constexpr int kTK = 64;                       // reduction per LDS stage
constexpr int kWGM = 2, kWGN = 4;             // waves over the tile

using LdsPtr = __attribute__((address_space(3))) void*;

// One operand's tile of R output rows x 64 of the reduction, in an LDS stage
// of R * 64 bf16 that is filled by global_load_lds (a wave's 64 lanes x 16
// bytes land in a row of 1 KiB; which 16 bytes a lane fetches is free, and
// that is where the bank swizzle is done).
//   KC (reduction contiguous): rows of 64 = eight 16-byte chunks, chunk c of
//     row r at c ^ (r % 8); a fragment is one ds_read_b128.
//   else (output rows contiguous): 64 rows of R, each as 32-byte pairs, pair
//     q of reduction row k at q ^ f(k), f = k % 4 + 4 ((k / 8) % 4) (as many
//     bits as there are pairs); a fragment is two ds_read_b64_tr_b16, whose
//     16 lanes read four rows x 32 bytes and get a column each.
template <bool KC, int R>
struct Operand {
    static constexpr int kLoads = R / 64;     // per wave and stage
    static constexpr int kPairs = R / 16;
    const uint16_t* src[kLoads];
    int k[kLoads];                            // this lane's first reduction index within a stage
    int64_t step;

    __device__ __forceinline__ static int pair_swizzle(int kr) { return ((kr & 3) | (((kr >> 3) & 3) << 2)) & (kPairs - 1); }

    // rows: of the output; row0: the tile's first
    __device__ __forceinline__ void init(const uint16_t* p, int64_t ld, int64_t row0, int64_t rows, int wave, int lane) {
        step = KC ? kTK : kTK * ld;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const int j = wave + u * kWaves;
            if constexpr (KC) {
                const int r = 8 * j + lane / 8;
                k[u] = 8 * ((lane & 7) ^ (lane / 8));
                const int64_t g = row0 + r < rows ? row0 + r : rows - 1;   // rows past the end: never stored
                src[u] = p + g * ld + k[u];
            } else {
                constexpr int kChunks = R / 8;
                k[u] = j * (kWave / kChunks) + lane / kChunks;
                const int c = (lane % kChunks) ^ (pair_swizzle(k[u]) << 1);
                const int64_t g = row0 + 8 * c < rows ? row0 + 8 * c : 0;   // (ld covers whole chunks)
                src[u] = p + k[u] * ld + g;
            }
        }
    }

    __device__ __forceinline__ void issue(uint16_t* lds, int wave, int64_t left) {
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const int j = wave + u * kWaves;
            const uint16_t* s = left >= kTK || k[u] < left ? src[u] : zero_chunk;
            __builtin_amdgcn_global_load_lds(s, (LdsPtr)(lds + j * 512), 16, 0, 0);
            src[u] += step;
        }
    }

    // fragment of output rows r0 .. r0 + 15 (r0 a multiple of 16), reduction 32 ks ..
    __device__ __forceinline__ static u32x4 frag(const uint16_t* lds, int r0, int ks, int l16, int lq) {
        if constexpr (KC) {
            return *reinterpret_cast<const u32x4*>(lds + (r0 + l16) * kTK + 8 * ((4 * ks + lq) ^ (l16 & 7)));
        } else {
            const int kr = 32 * ks + 8 * lq + l16 / 4;
            const uint16_t* at = lds + kr * R + 16 * ((r0 / 16) ^ pair_swizzle(kr)) + 4 * (l16 % 4);
            union { s16x4 h[2]; u32x4 v; } f;
            f.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at));
            f.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at + 4 * R));
            return f.v;
        }
    }
};

// Tile t of a grid of mt x nt tiles.  Work-groups go round the eight XCDs, so
// XCD x takes the x-th eighth of the tiles, and within it eight tiles of rows
// side by side before the next tile of columns: an XCD's tiles share their
// operands' rows in its L2.
__device__ __forceinline__ void tile_of(int t, int mt, int nt, int* tm, int* tn) {
    const int total = mt * nt, per = total / 8, rest = total % 8;
    const int x = t % 8, i = t / 8;
    t = x * per + (x < rest ? x : rest) + i;
    constexpr int G = 8;
    const int band = t / (G * nt), in = t % (G * nt);
    const int rows = mt - band * G < G ? mt - band * G : G;
    *tm = band * G + in % rows;
    *tn = in / rows;
}

template <bool AK, bool BK, int BM, int BN>
__device__ __forceinline__ void gemm_tile(const GemmProduct& p, int tile, uint16_t* As0, uint16_t* As1, uint16_t* Bs0,
                                          uint16_t* Bs1) {
    constexpr int WM = BM / kWGM, WN = BN / kWGN, TM = WM / 16, TN = WN / 16;
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
    const int l16 = lane % 16, lq = lane / 16;
    const int wm = wave / kWGN, wn = wave % kWGN;
    int tm, tn;
    tile_of(tile, static_cast<int>((p.M + BM - 1) / BM), static_cast<int>((p.N + BN - 1) / BN), &tm, &tn);
    const int64_t m0 = static_cast<int64_t>(tm) * BM, n0 = static_cast<int64_t>(tn) * BN;

    Operand<AK, BM> a;
    Operand<BK, BN> b;
    a.init(static_cast<const uint16_t*>(p.A), p.lda, m0, p.M, wave, lane);
    b.init(static_cast<const uint16_t*>(p.B), p.ldb, n0, p.N, wave, lane);

    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // slice kt from one stage while slice kt + 1 arrives in the other
    auto step = [&](int64_t k0, const uint16_t* as, const uint16_t* bs, uint16_t* an, uint16_t* bn) {
        wait_vm_all();                        // this wave's loads of the slice
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();         // and everyone's; the other stage is free
        asm volatile("" ::: "memory");
        if (k0 + kTK < p.K) {
            a.issue(an, wave, p.K - k0 - kTK);
            b.issue(bn, wave, p.K - k0 - kTK);
        }
#pragma unroll
        for (int ks = 0; ks < kTK / 32; ++ks) {
            u32x4 fb[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j) fb[j] = Operand<BK, BN>::frag(bs, wn * WN + 16 * j, ks, l16, lq);
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const u32x4 fa = Operand<AK, BM>::frag(as, wm * WM + 16 * i, ks, l16, lq);
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = mfma(fb[j], fa, acc[i][j]);
            }
        }
    };
    if (p.K > 0) {
        a.issue(As0, wave, p.K);
        b.issue(Bs0, wave, p.K);
    }
    for (int64_t k0 = 0; k0 < p.K; k0 += 2 * kTK) {
        step(k0, As0, Bs0, As1, Bs1);
        if (k0 + kTK < p.K) step(k0 + kTK, As1, Bs1, As0, Bs0);
    }

    // the weights' fragment is the first operand, so a lane holds row l16 and
    // the four adjacent columns 4 lq .. of each 16 x 16 tile
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int64_t m = m0 + wm * WM + 16 * i + l16;
        if (m >= p.M) continue;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t n = n0 + wn * WN + 16 * j + 4 * lq;
            if (n >= p.N) continue;
            const int nv = p.N - n < 4 ? static_cast<int>(p.N - n) : 4;
            float f[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
            finish4(p.ep, m, n, nv, f);
        }
    }
}

template <int BM, int BN>
struct Stages {
    static constexpr int kA = BM * kTK, kB = BN * kTK;
};

template <int BM, int BN>
__global__ __launch_bounds__(kThreads, 2) void linear_forward_kernel(GemmProduct p) {
    __shared__ __align__(1024) uint16_t As0[BM * kTK], As1[BM * kTK];
    __shared__ __align__(1024) uint16_t Bs0[BN * kTK], Bs1[BN * kTK];
    gemm_tile<true, true, BM, BN>(p, blockIdx.x, As0, As1, Bs0, Bs1);
}

// dx (first `first` work-groups) and dw (the rest) in one launch: each alone
// often has fewer tiles than the card has compute units.
template <int BM, int BN>
__global__ __launch_bounds__(kThreads, 2) void linear_backward_kernel(GemmProduct dx, GemmProduct dw, int first) {
    __shared__ __align__(1024) uint16_t As0[BM * kTK], As1[BM * kTK];
    __shared__ __align__(1024) uint16_t Bs0[BN * kTK], Bs1[BN * kTK];
    if (static_cast<int>(blockIdx.x) < first) gemm_tile<true, false, BM, BN>(dx, blockIdx.x, As0, As1, Bs0, Bs1);
    else gemm_tile<false, false, BM, BN>(dw, blockIdx.x - first, As0, As1, Bs0, Bs1);
}

// ---- few rows --------------------------------------------------------------------
// A work-group owns 16 rows of w (16 columns of y) and splits K over its NWV
// waves; per 128-wide step of K, lane (l16, lq) reads 64 contiguous bytes of
// its weight row and of its row of each 16-row tile of x.  The waves' partial
// tiles are summed in LDS in wave order.
constexpr int kFewRows = 64, kFewStep = 128;

template <int MT, int NWV>
__global__ __launch_bounds__(NWV * kWave) void linear_few_kernel(GemmProduct p) {
    __shared__ f32x4 part[NWV][MT][kWave];
    const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
    const int l16 = lane % 16, lq = lane / 16;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
    const int64_t steps = (p.K + kFewStep - 1) / kFewStep;
    const int64_t s0 = steps * wave / NWV, s1 = steps * (wave + 1) / NWV;
    const bool nok = n0 + l16 < p.N;
    const uint16_t* brow = static_cast<const uint16_t*>(p.B) + (nok ? n0 + l16 : 0) * p.ldb;
    const uint16_t* arow[MT];
    bool mok[MT];
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        mok[t] = 16 * t + l16 < p.M;
        arow[t] = static_cast<const uint16_t*>(p.A) + (mok[t] ? 16 * t + l16 : 0) * p.lda;
        acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll 2
    for (int64_t st = s0; st < s1; ++st) {
        const int64_t kb = st * kFewStep + lq * 32;
        u32x4 bf[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            bf[j] = nok && kb + 8 * j < p.K ? *reinterpret_cast<const u32x4*>(brow + kb + 8 * j) : zero;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            u32x4 af[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                af[j] = mok[t] && kb + 8 * j < p.K ? *reinterpret_cast<const u32x4*>(arow[t] + kb + 8 * j) : zero;
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[t] = mfma(bf[j], af[j], acc[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) part[wave][t][lane] = acc[t];
    __syncthreads();
    for (int t = wave; t < MT; t += NWV) {
        f32x4 s = part[0][t][lane];
        for (int w = 1; w < NWV; ++w) s += part[w][t][lane];
        const int64_t m = 16 * t + l16, n = n0 + 4 * lq;
        if (m >= p.M || n >= p.N) continue;
        const int nv = p.N - n < 4 ? static_cast<int>(p.N - n) : 4;
        float f[4] = {s[0], s[1], s[2], s[3]};
        finish4(p.ep, m, n, nv, f);
    }
}

// ---- dp = dy act'(p) and its column sums -------------------------------------------
// A work-group covers 64 rows x 256 columns: lane l of 64 takes four columns
// of every fourth row; dp is rounded to bf16 (the products' operand type), the
// sums are of the values before that.
constexpr int kDpRows = 64, kDpCols = 256;

__global__ __launch_bounds__(256) void linear_dp_kernel(LinearDp p) {
    __shared__ float sums[4][kDpCols];
    const int lane = threadIdx.x % 64, g = threadIdx.x / 64;
    const int64_t block = blockIdx.x / p.cols, col0 = static_cast<int64_t>(blockIdx.x % p.cols) * kDpCols;
    const int64_t m0 = block * kDpRows, n = col0 + 4 * lane;
    const int64_t left = p.N - n;
    const int nv = left < 0 ? 0 : (left < 4 ? static_cast<int>(left) : 4);
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = g; i < kDpRows; i += 4) {
        const int64_t m = m0 + i;
        if (m >= p.M) break;
        float d[4], q[4];
        load4(p.dy, p.dy_bf16, m * p.ldy + n, nv, d);
        if (p.act != kActNone) {
            load4(p.preact, true, m * p.ldp + n, nv, q);
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = e < nv ? d[e] * slope(q[e], p.act) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += d[e];
        if (p.dp && n < p.ldd) store4(p.dp, true, m * p.ldd + n, 4, d);   // (columns past N: zeros)
    }
    if (!p.part) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[g][4 * lane + e] = s[e];
    __syncthreads();
    const int64_t c = col0 + threadIdx.x;
    if (c < p.N)
        p.part[block * p.N + c] =
            (sums[0][threadIdx.x] + sums[1][threadIdx.x]) + (sums[2][threadIdx.x] + sums[3][threadIdx.x]);
}

constexpr int kSumCols = 64, kSumSlices = 16;

__global__ __launch_bounds__(kSumCols * kSumSlices) void linear_sum_kernel(const float* part, int64_t blocks, int64_t N,
                                                                          float* out) {
    __shared__ float t[kSumSlices][kSumCols];
    const int c = threadIdx.x % kSumCols, sl = threadIdx.x / kSumCols;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * kSumCols + c;
    float s = 0.f;
    if (n < N)
        for (int64_t i = sl; i < blocks; i += kSumSlices) s += part[i * N + n];
    t[sl][c] = s;
    __syncthreads();
    if (sl == 0 && n < N) {
#pragma unroll
        for (int k = 1; k < kSumSlices; ++k) s += t[k][c];
        out[n] = s;
    }
}

template <int BM, int BN>
int64_t tiles(const GemmProduct& p) { return ((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN); }

template <int BM, int BN>
hipError_t forward_t(const GemmProduct& p, hipStream_t s) {
    hipLaunchKernelGGL((linear_forward_kernel<BM, BN>), dim3(static_cast<unsigned>(tiles<BM, BN>(p))), dim3(kThreads), 0, s, p);
    return hipGetLastError();
}

template <int BM, int BN>
hipError_t backward_t(const GemmProduct& dx, const GemmProduct& dw, hipStream_t s) {
    const int64_t t1 = dx.ep.y ? tiles<BM, BN>(dx) : 0, t2 = dw.ep.y ? tiles<BM, BN>(dw) : 0;
    hipLaunchKernelGGL((linear_backward_kernel<BM, BN>), dim3(static_cast<unsigned>(t1 + t2)), dim3(kThreads), 0, s, dx, dw,
                       static_cast<int>(t1));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear(const GemmProduct& p, hipStream_t s) {
    if (p.M <= 0 || p.N <= 0) return hipSuccess;
    const int cus = compute_units();
    if (p.M <= kFewRows) {
        const dim3 grid(static_cast<unsigned>((p.N + 15) / 16));
        switch ((p.M + 15) / 16) {
            case 1: hipLaunchKernelGGL((linear_few_kernel<1, 8>), grid, dim3(8 * kWave), 0, s, p); break;
            case 2: hipLaunchKernelGGL((linear_few_kernel<2, 8>), grid, dim3(8 * kWave), 0, s, p); break;
            case 3: hipLaunchKernelGGL((linear_few_kernel<3, 8>), grid, dim3(8 * kWave), 0, s, p); break;
            default: hipLaunchKernelGGL((linear_few_kernel<4, 8>), grid, dim3(8 * kWave), 0, s, p); break;
        }
        return hipGetLastError();
    }
    if (tiles<256, 256>(p) >= cus) return forward_t<256, 256>(p, s);
    if (tiles<128, 128>(p) >= cus) return forward_t<128, 128>(p, s);
    return forward_t<64, 64>(p, s);
}

int64_t linear_dp_blocks(int64_t M) { return (M + kDpRows - 1) / kDpRows; }

hipError_t launch_linear_backward(const LinearDp& dp, const GemmProduct& dx, const GemmProduct& dw, float* dbias,
                                  hipStream_t s) {
    if (dp.dp || dp.part) {
        LinearDp d = dp;
        d.cols = static_cast<int>(((dp.dp ? dp.ldd : dp.N) + kDpCols - 1) / kDpCols);
        const int64_t grid = d.cols * linear_dp_blocks(dp.M);
        hipLaunchKernelGGL(linear_dp_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, d);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (dbias) {
        hipLaunchKernelGGL(linear_sum_kernel, dim3(static_cast<unsigned>((dp.N + kSumCols - 1) / kSumCols)),
                           dim3(kSumCols * kSumSlices), 0, s, dp.part, linear_dp_blocks(dp.M), dp.N, dbias);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!dx.ep.y && !dw.ep.y) return hipSuccess;
    const int cus = compute_units();
    const int64_t big = (dx.ep.y ? tiles<256, 256>(dx) : 0) + (dw.ep.y ? tiles<256, 256>(dw) : 0);
    const int64_t mid = (dx.ep.y ? tiles<128, 128>(dx) : 0) + (dw.ep.y ? tiles<128, 128>(dw) : 0);
    if (big >= cus) return backward_t<256, 256>(dx, dw, s);
    if (mid >= cus) return backward_t<128, 128>(dx, dw, s);
    return backward_t<64, 64>(dx, dw, s);
}

}  // namespace gdn
