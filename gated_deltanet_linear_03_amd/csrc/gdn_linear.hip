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

// The same, log2 of it as a polynomial of degree 9 in |p| (minimax on [0,
// 13.3]; relative error of the result, rounding included, below 7e-6 for |p| <
// 4, 1e-4 below 6 and 9e-4 up to 12.9, from where on the result, below 2^-126,
// counts as 0): 17 vector operations a value instead of 24.  For outputs in
// bf16, whose rounding is off by up to 2^-8.
__device__ __forceinline__ float half_erfc_bf16(float p) {
    const float x = fabsf(p);
    float q = -1.144341066e-09f;
    q = fmaf(q, x, 1.063108286e-07f);
    q = fmaf(q, x, -3.947418463e-06f);
    q = fmaf(q, x, 8.015496132e-05f);
    q = fmaf(q, x, -1.016277121e-03f);
    q = fmaf(q, x, 8.726238273e-03f);
    q = fmaf(q, x, -5.425874144e-02f);
    q = fmaf(q, x, -4.582666755e-01f);
    q = fmaf(q, x, -1.151299953e+00f);
    q = fmaf(q, x, -9.999933839e-01f);
    return __builtin_amdgcn_exp2f(q);
}

// gelu for an output in bf16 (chosen by the launchers; not part of the ABI)
constexpr int kActGeluBf16 = 5;

__device__ __forceinline__ float activate(float p, int act) {
    switch (act) {
        case kActGeluBf16: {
            const float c = half_erfc_bf16(p);
            return p * (p > 0.f ? 1.f - c : c);
        }
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
typedef uint32_t Run8 __attribute__((ext_vector_type(4), aligned(2)));   // eight bf16, element aligned

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// up to W adjacent elements, element aligned only
template <int W>
__device__ __forceinline__ void load_n(const void* p, bool bf16, int64_t at, int nv, float* f) {
    if (bf16) {
        const uint16_t* q = static_cast<const uint16_t*>(p) + at;
        if (nv == W) {
#pragma unroll
            for (int g = 0; g < W / 4; ++g) {
                const Half4 h = *reinterpret_cast<const Half4*>(q + 4 * g);
                f[4 * g] = __uint_as_float(h.lo << 16);
                f[4 * g + 1] = __uint_as_float(h.lo & 0xFFFF0000u);
                f[4 * g + 2] = __uint_as_float(h.hi << 16);
                f[4 * g + 3] = __uint_as_float(h.hi & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e) f[e] = e < nv ? bf16_bits_to_f32(q[e]) : 0.f;
        }
    } else {
        const float* q = static_cast<const float*>(p) + at;
        if (nv == W) {
#pragma unroll
            for (int g = 0; g < W / 4; ++g) {
                const Float4 h = *reinterpret_cast<const Float4*>(q + 4 * g);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[4 * g + e] = h.e[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e) f[e] = e < nv ? q[e] : 0.f;
        }
    }
}

template <int W>
__device__ __forceinline__ void store_n(void* p, bool bf16, int64_t at, int nv, const float* f) {
    if (bf16) {
        uint16_t* q = static_cast<uint16_t*>(p) + at;
        if (nv == W) {
            if constexpr (W == 8) {
                // (non-temporal: the tiles' outputs and residuals pass the L2 by, which holds operands)
                const Run8 h = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
                __builtin_nontemporal_store(h, reinterpret_cast<Run8*>(q));
            } else {
                *reinterpret_cast<Half4*>(q) = Half4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
            }
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e)
                if (e < nv) q[e] = f32_to_bf16_bits(f[e]);
        }
    } else {
        float* q = static_cast<float*>(p) + at;
        if (nv == W) {
#pragma unroll
            for (int g = 0; g < W / 4; ++g)
                *reinterpret_cast<Float4*>(q + 4 * g) = Float4{{f[4 * g], f[4 * g + 1], f[4 * g + 2], f[4 * g + 3]}};
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e)
                if (e < nv) q[e] = f[e];
        }
    }
}

template <int W>
__device__ __forceinline__ void activate_n(float* f, int act) {
    switch (act) {                                // (uniform: one branch for all the values)
#define GDN_ACT_CASE(ACT)                                                         \
    case ACT:                                                                     \
        _Pragma("unroll") for (int e = 0; e < W; ++e) f[e] = activate(f[e], ACT); \
        break;
        GDN_ACT_CASE(kActRelu)
        GDN_ACT_CASE(kActGelu)
        GDN_ACT_CASE(kActGeluBf16)
        GDN_ACT_CASE(kActGeluTanh)
        GDN_ACT_CASE(kActSilu)
#undef GDN_ACT_CASE
        default: break;
    }
}

// y = act(sum + bias) + residual for up to W adjacent columns of one row;
// preact receives sum + bias
template <int W>
__device__ __forceinline__ void finish_n(const GemmEpilogue& ep, int64_t m, int64_t n, int nv, float* f) {
    if (ep.bias) {
        float c[W];
        load_n<W>(ep.bias, false, n, nv, c);
#pragma unroll
        for (int e = 0; e < W; ++e) f[e] += c[e];
    }
    if (ep.preact) store_n<W>(ep.preact, true, m * ep.ldp + n, nv, f);
    activate_n<W>(f, ep.act);
    if (ep.residual) {
        float r[W];
        load_n<W>(ep.residual, ep.bf16, m * ep.ldr + n, nv, r);
#pragma unroll
        for (int e = 0; e < W; ++e) f[e] += r[e];
    }
    store_n<W>(ep.y, ep.bf16, m * ep.ldy + n, nv, f);
}

// ---- the tiled kernels -----------------------------------------------------------
constexpr int kTK = 32;                       // reduction per LDS stage

using LdsPtr = __attribute__((address_space(3))) void*;

// 16 bytes from each lane's address into LDS at `lds` + 16 * lane, without the
// compiler knowing that it writes LDS.  It takes every ds_read_b64_tr_b16 to
// depend on all such loads in flight and waits for them, which undoes the
// stages (dx of 2048 x 2048 x 2048 in tiles of 128 x 128: 41 us instead of
// 23); here the waits are this code's own.  A load has no register to write,
// reads its addresses when it is issued, and the memory clobber keeps LDS
// accesses on their side of it; the s_nop covers an address register that a
// vector instruction has just written.
__device__ __forceinline__ void load_to_lds(const void* uniform, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(uniform) : "memory", "m0");
}
__device__ __forceinline__ void load_to_lds(const void* p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "memory", "m0");
}

// One operand's tile of R output rows x TK (32 or 64) of the reduction, in an
// LDS stage of R * TK bf16 that is filled by load_to_lds (a wave's 64 lanes x
// 16 bytes land in a row of 1 KiB; which 16 bytes a lane fetches is free, and
// that is where the bank swizzle is done).
//   KC (reduction contiguous): rows of TK = four or eight 16-byte chunks,
//     chunk c of row r at c ^ f(r).  TK 32: f = bit 2 of r + 2 (bit 1 ^ bit 3);
//     TK 64: f = r / 2 % 8; the chunks that 8 or 16 adjacent lanes read lie in
//     different banks.  A fragment is one ds_read_b128.  With TK 64 a row's
//     request is a whole 128-byte line: 4096 x 12288 x 2048 in tiles of 256 x
//     256 takes 177 us with requests of 64 bytes, 155 with these.
//   else (output rows contiguous): TK rows of R, each as 32-byte pairs, pair
//     q of reduction row k at q ^ f(k), f = k % 4 + 4 (k % 32 / 8) (as many
//     bits as there are pairs).  A fragment is two ds_read_b64_tr_b16, whose
//     16 lanes read four rows x 32 bytes and get a column each.
// NW: waves of the work-group; WR: rows of a wave.
template <bool KC, int R, int NW, int WR, int TK>
struct Operand {
    static constexpr int kLoads = R * TK * 2 / 1024 / NW;        // per wave and stage
    static constexpr int kPairs = R / 16;
    static_assert(kLoads >= 1, "a stage is at least one load of each wave");
    // A lane's addresses: a wave-uniform one that moves along the reduction,
    // plus 32-bit byte offsets (strides are of 22 bits).
    const uint8_t* base;
    int64_t step;                             // bytes per stage
    uint32_t off[kLoads];
    int k[kLoads];                            // first reduction index within a stage
    // fragment addresses within a stage, elements (KC: of each half of TK 64)
    int at[KC ? TK / 32 : WR / 16];

    __device__ __forceinline__ static int chunk_swizzle(int r) {
        return TK == 64 ? (r >> 1) & 7 : ((r >> 2) & 1) | ((((r >> 1) ^ (r >> 3)) & 1) << 1);
    }
    __device__ __forceinline__ static int pair_swizzle(int kr) { return ((kr & 3) | (((kr & 31) >> 3) << 2)) & (kPairs - 1); }

    // rows: of the output; row0: the tile's first; w: which of the tile's WR rows are this wave's
    __device__ __forceinline__ void init(const uint16_t* p, int64_t ld, int64_t row0, int64_t rows, int wave, int lane, int w) {
        const int l16 = lane % 16, lq = lane / 16;
        step = 2 * (KC ? TK : TK * ld);
        // rows past the end, up to a whole tile of them, read the last row and are never stored
        if (row0 >= rows) row0 = KC ? rows - 1 : (rows - 1) / 8 * 8;
        base = reinterpret_cast<const uint8_t*>(KC ? p + row0 * ld : p + row0);
        const int left = rows - row0 < R ? static_cast<int>(rows - row0) : R;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const int j = wave + u * NW;
            if constexpr (KC) {
                constexpr int kChunks = TK / 8;
                const int r = kWave / kChunks * j + lane / kChunks;
                k[u] = 8 * ((lane % kChunks) ^ chunk_swizzle(r));
                off[u] = 2 * (static_cast<uint32_t>(r < left ? r : left - 1) * static_cast<uint32_t>(ld) + k[u]);
            } else {
                constexpr int kChunks = R / 8;
                k[u] = j * (kWave / kChunks) + lane / kChunks;
                const int c = 8 * ((lane % kChunks) ^ (pair_swizzle(k[u]) << 1));
                off[u] = 2 * (static_cast<uint32_t>(k[u]) * static_cast<uint32_t>(ld) + (c < left ? c : 0));   // (ld covers whole chunks)
            }
        }
        if constexpr (KC) {
#pragma unroll
            for (int h = 0; h < TK / 32; ++h) at[h] = (w * WR + l16) * TK + 8 * ((4 * h + lq) ^ chunk_swizzle(l16));
        } else {
            const int kr = 8 * lq + l16 / 4;
#pragma unroll
            for (int i = 0; i < WR / 16; ++i) at[i] = kr * R + 16 * ((w * (WR / 16) + i) ^ pair_swizzle(kr)) + 4 * (l16 % 4);
        }
    }

    // the next TK of the reduction into a stage; left: how much of it there
    // still is (FULL: all of TK at least)
    template <bool FULL>
    __device__ __forceinline__ void issue(uint16_t* lds, int wave, int64_t left) {
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const uint32_t to = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((LdsPtr)(lds + (wave + u * NW) * 512)));
            if constexpr (FULL) load_to_lds(base, off[u], to);
            else load_to_lds(k[u] < left ? static_cast<const void*>(base + off[u]) : zero_chunk, to);
        }
        base += step;
    }

    // fragment of the wave's output rows 16 i .. 16 i + 15 and the reduction's 32 h .. 32 h + 31
    __device__ __forceinline__ u32x4 frag(const uint16_t* lds, int i, int h) const {
        if constexpr (KC) {
            return *reinterpret_cast<const u32x4*>(lds + at[h] + 16 * i * TK);
        } else {
            lds += at[i] + 32 * h * R;
            union { s16x4 h[2]; u32x4 v; } f;
            f.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)lds);
            f.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(lds + 4 * R));
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

// s_waitcnt vmcnt(N) lgkmcnt(0) (gfx9 encoding)
template <int N>
__device__ __forceinline__ void wait_vm_lds() {
    __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));
}
// s_waitcnt vmcnt(N)
template <int N>
__device__ __forceinline__ void wait_vm() {
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}

template <bool V>
struct Bool { static constexpr bool value = V; };

__device__ __forceinline__ void wave_barrier() {   // (nothing is scheduled across it, matrix instructions included)
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// A tile of BM x BN for NWM x NWN waves, each with WM x WN of it.
// PER_SIMD: waves that share a SIMD when the compute unit is full.
template <int BM_, int BN_, int NWM_, int NWN_, int STAGES, int PER_SIMD>
struct Shape {
    static constexpr int BM = BM_, BN = BN_, NWM = NWM_, NWN = NWN_, kStages = STAGES, kPerSimd = PER_SIMD;
    static constexpr int kWaves = NWM * NWN, kThreads = kWaves * kWave;
    static constexpr int WM = BM / NWM, WN = BN / NWN, TM = WM / 16, TN = WN / 16;
    static constexpr int kA = BM * kTK, kB = BN * kTK;            // elements of a stage
    // rows of a wave: two runs of WM / 2.  From 128 rows on: one in each half
    // of the tile, which are operands of their own; else one after the other.
    static constexpr bool kHalves = BM >= 128;
    static constexpr int kHalfRows = WM / 2, kHalfStep = kHalves ? BM / 2 : kHalfRows, kWaveStep = kHalves ? kHalfRows : WM;
    // the epilogue's strips: half of each wave's rows, in 32 bits, four columns of padding
    static constexpr int kStripTiles = TM / 2;
    static constexpr int kStripLd = WN + 4, kStrip = 16 * kStripTiles * kStripLd;
    static constexpr int kStageBytes = kStages * (kA + kB) * 2, kStripBytes = kWaves * kStrip * 4;
    static constexpr int kBytes = kStageBytes > kStripBytes ? kStageBytes : kStripBytes;
};

// From the accumulators to the outputs.  The weights' fragment is the first
// operand of a matrix instruction, so a lane holds row l16 and the four
// adjacent columns 4 lq .. of each 16 x 16 tile; through LDS (each wave its
// own strip, half of its rows at a time), so that a row of the wave's columns
// is finished and stored as one run, eight columns a lane.  The residual's
// rows of the first half are requested before the last slices are multiplied,
// those of the second half before the first one is finished.
// PLAIN: nothing but y.
template <typename S, bool PLAIN>
struct Store {
    static constexpr int kRun = S::WN / 8;    // lanes of a row
    static constexpr int kRowsAtOnce = kWave / kRun;
    static constexpr int kRows = 16 * S::kStripTiles, kMine = kRows / kRowsAtOnce;   // rows of a half; of a lane
    static constexpr int kBatch = kMine < 4 ? kMine : 4;
    int64_t m0, n;                            // the wave's first row, the lane's first column
    int first, nv;                            // the lane's first row of a half; its columns
    bool early;                               // the residual can be fetched as bf16 runs
    Run8 res[kMine];

    __device__ __forceinline__ void init(const GemmProduct& p, int64_t m, int64_t n0, int lane) {
        m0 = m;
        first = lane / kRun;
        n = n0 + 8 * (lane % kRun);
        nv = p.N - n < 8 ? (p.N > n ? static_cast<int>(p.N - n) : 0) : 8;
        early = !PLAIN && p.ep.residual && p.ep.bf16 && nv == 8;
    }

    __device__ __forceinline__ void fetch(const GemmProduct& p, int half) {
        if (PLAIN || !early) return;
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
            const int64_t m = m0 + half * S::kHalfStep + first + u * kRowsAtOnce;
            if (m < p.M)
                res[u] = __builtin_nontemporal_load(
                    reinterpret_cast<const Run8*>(static_cast<const uint16_t*>(p.ep.residual) + m * p.ep.ldr + n));
        }
    }

    __device__ __forceinline__ void run(const GemmProduct& p, f32x4 (&acc)[S::TM][S::TN], float* strip, int lane) {
        const int l16 = lane % 16, lq = lane / 16;
        float bias[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) bias[e] = 0.f;
        if (!PLAIN && p.ep.bias && nv > 0) load_n<8>(p.ep.bias, false, n, nv, bias);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int i = 0; i < S::kStripTiles; ++i)
#pragma unroll
                for (int j = 0; j < S::TN; ++j)
                    *reinterpret_cast<f32x4*>(strip + (16 * i + l16) * S::kStripLd + 16 * j + 4 * lq) =
                        acc[half * S::kStripTiles + i][j];
            asm volatile("" ::: "memory");    // one wave: its LDS accesses stay in order
#pragma unroll
            for (int u0 = 0; u0 < kMine; u0 += kBatch) {
                float f[kBatch][8];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const f32x4* q = reinterpret_cast<const f32x4*>(strip + (first + (u0 + u) * kRowsAtOnce) * S::kStripLd +
                                                                    8 * (lane % kRun));
                    const f32x4 q0 = q[0], q1 = q[1];
#pragma unroll
                    for (int e = 0; e < 4; ++e) { f[u][e] = q0[e] + bias[e]; f[u][4 + e] = q1[e] + bias[4 + e]; }
                }
                const int64_t mb = m0 + half * S::kHalfStep + first + u0 * kRowsAtOnce;
                if (!PLAIN && p.ep.preact) {
#pragma unroll
                    for (int u = 0; u < kBatch; ++u) {
                        const int64_t m = mb + u * kRowsAtOnce;
                        if (m < p.M && nv > 0) store_n<8>(p.ep.preact, true, m * p.ep.ldp + n, nv, f[u]);
                    }
                }
                if (!PLAIN) activate_n<8 * kBatch>(&f[0][0], p.ep.act);
                if (PLAIN) {
                } else if (early) {
#pragma unroll
                    for (int u = 0; u < kBatch; ++u)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            f[u][2 * e] += __uint_as_float(res[u0 + u][e] << 16);
                            f[u][2 * e + 1] += __uint_as_float(res[u0 + u][e] & 0xFFFF0000u);
                        }
                } else if (p.ep.residual) {
                    float r[kBatch][8];
#pragma unroll
                    for (int u = 0; u < kBatch; ++u) {
                        const int64_t m = mb + u * kRowsAtOnce;
                        if (m < p.M && nv > 0) load_n<8>(p.ep.residual, p.ep.bf16, m * p.ep.ldr + n, nv, r[u]);
                    }
#pragma unroll
                    for (int u = 0; u < kBatch; ++u)
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[u][e] += r[u][e];
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int64_t m = mb + u * kRowsAtOnce;
                    if (m < p.M && nv > 0) store_n<8>(p.ep.y, p.ep.bf16, m * p.ep.ldy + n, nv, f[u]);
                }
            }
            if (half == 0) fetch(p, 1);
            asm volatile("" ::: "memory");
        }
    }
};

// Large tiles, 256 x 256 for 2 x 4 waves of 128 x 64: one work-group fills a
// compute unit, with two waves on each SIMD.  A stage is 64 of the reduction,
// so that a row's request is a whole line, in three operands: the weights, and
// the tile's upper and lower rows (a wave has as many of either).  It is four
// phases of 16 matrix instructions a wave: the upper rows with the first and
// the second 32 of the reduction, then the lower rows with both (the weights'
// fragments stay in registers); before a phase the wave reads the fragments
// it needs, between two barriers.  The lower four waves run half a phase
// behind the upper four, so while one wave of a SIMD feeds the matrix core the
// other one reads and requests.
// Two stages in LDS: in the fourth phase of stage t the weights and upper rows
// of t + 2 are requested into their places in it, which were last read in the
// second phase, and in the second phase the lower rows of t + 1, into those of
// t - 1, last read in its fourth phase: every wave had those fragments in
// registers before the barrier that the requesting phase began with.  What is
// requested has four phases to land.
// Bound: the matrix cores at the clock that their power leaves (4096 x 12288 x
// 2048: 148 to 155 us by the card, 1330 to 1390 TFLOP/s).  The epilogue of a
// round of tiles does not overlap with the next one's products: with gelu, bias
// and residual 182 to 204 us.
template <bool AK, bool BK, bool PLAIN, typename S>
__device__ __forceinline__ void gemm_large(const GemmProduct& p, int tile, uint8_t* shared) {
    constexpr int K2 = 2 * kTK, TM = S::TM, TN = S::TN, H = TM / 2;
    using OA = Operand<AK, S::BM / 2, S::kWaves, S::kHalfRows, K2>;
    using OB = Operand<BK, S::BN, S::kWaves, S::WN, K2>;
    constexpr int kInFlight = 2 * OA::kLoads + OB::kLoads;
    static_assert(S::kStages == 4, "two stages of 64");
    uint16_t* const us = reinterpret_cast<uint16_t*>(shared);
    uint16_t* const ls = us + 2 * S::kA;
    uint16_t* const bs = ls + 2 * S::kA;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
    const int wm = wave / S::NWN, wn = wave % S::NWN;
    int tm, tn;
    tile_of(tile, static_cast<int>((p.M + S::BM - 1) / S::BM), static_cast<int>((p.N + S::BN - 1) / S::BN), &tm, &tn);
    const int64_t m0 = static_cast<int64_t>(tm) * S::BM, n0 = static_cast<int64_t>(tn) * S::BN;
    OA upper, lower;
    OB b;
    upper.init(static_cast<const uint16_t*>(p.A), p.lda, m0, p.M, wave, lane, wm);
    lower.init(static_cast<const uint16_t*>(p.A), p.lda, m0 + S::BM / 2, p.M, wave, lane, wm);
    b.init(static_cast<const uint16_t*>(p.B), p.ldb, n0, p.N, wave, lane, wn);
    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // an even number of stages: past the reduction's end they read zeros
    const int nk = static_cast<int>((p.K + K2 - 1) / K2 + 1) / 2 * 2;
    const int full = static_cast<int>(p.K / K2);
    Store<S, PLAIN> out;
    out.init(p, m0 + wm * S::kWaveStep, n0 + wn * S::WN, lane);
    auto round = [&](auto whole, int kt) {    // stages kt and kt + 1 (kt even)
        constexpr bool FULL = decltype(whole)::value;
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            u32x4 fa[H], fb[2][TN];
#pragma unroll
            for (int ph = 0; ph < 4; ++ph) {
                const int h = ph % 2, half = ph / 2;
                if (half == 0) {
#pragma unroll
                    for (int j = 0; j < TN; ++j) fb[h][j] = b.frag(bs + st * 2 * S::kB, j, h);
                }
#pragma unroll
                for (int i = 0; i < H; ++i) fa[i] = half == 0 ? upper.frag(us + st * S::kA, i, h) : lower.frag(ls + st * S::kA, i, h);
                if (ph == 1) {
                    lower.template issue<FULL>(ls + (st ^ 1) * S::kA, wave, p.K - static_cast<int64_t>(kt + st + 1) * K2);
                    wait_vm<kInFlight>();     // this stage's lower rows have landed
                }
                if (ph == 3) {
                    const int64_t left = p.K - static_cast<int64_t>(kt + st + 2) * K2;
                    upper.template issue<FULL>(us + st * S::kA, wave, left);
                    b.template issue<FULL>(bs + st * 2 * S::kB, wave, left);
                    wait_vm<kInFlight>();     // the next stage's weights and upper rows have landed
                }
                wave_barrier();
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int i = 0; i < H; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j) acc[half * H + i][j] = mfma(fb[h][j], fa[i], acc[half * H + i][j]);
                __builtin_amdgcn_s_setprio(0);
                wave_barrier();
            }
        }
    };
    if (nk > 0) {
        upper.template issue<false>(us, wave, p.K);
        b.template issue<false>(bs, wave, p.K);
        lower.template issue<false>(ls, wave, p.K);
        upper.template issue<false>(us + S::kA, wave, p.K - K2);
        b.template issue<false>(bs + 2 * S::kB, wave, p.K - K2);
        wait_vm<kInFlight>();                 // the first stage's weights and upper rows
        wave_barrier();
        if (wave >= S::kWaves / 2) wave_barrier();   // half a phase behind
        int kt = 0;
        for (; kt + 4 <= full; kt += 2) round(Bool<true>{}, kt);
        out.fetch(p, 0);
        for (; kt < nk; kt += 2) round(Bool<false>{}, kt);
        if (wave < S::kWaves / 2) wave_barrier();
        wait_vm<0>();                         // the requests past the end
    }
    wave_barrier();                           // the stages become the epilogue's strips
    if (nk == 0) out.fetch(p, 0);
    out.run(p, acc, reinterpret_cast<float*>(shared) + wave * S::kStrip, lane);
}

// Tiles of 128 x 128 for 2 x 2 waves: two work-groups share a compute unit and
// hide each other's latencies.  Operands, stages and the four phases of a
// stage as above; while a wave multiplies one phase from registers it reads
// the next one's fragments into the other set, and two barriers a stage do:
// before the second phase (the upper rows and weights have been read, and the
// lower rows landed) and before the fourth (the other way round).  What is
// requested after a barrier has six phases until it is read.  2048 x 2048 x
// 2048: 23.2 us (24.5 with stages of 32 and requests of 64 bytes); 1500 x 1500
// x 1496: 19.7 us (24.2).
template <bool AK, bool BK, bool PLAIN, typename S>
__device__ __forceinline__ void gemm_medium(const GemmProduct& p, int tile, uint8_t* shared) {
    constexpr int K2 = 2 * kTK, TM = S::TM, TN = S::TN, H = TM / 2;
    using OA = Operand<AK, S::BM / 2, S::kWaves, S::kHalfRows, K2>;
    using OB = Operand<BK, S::BN, S::kWaves, S::WN, K2>;
    constexpr int kInFlight = 2 * OA::kLoads + OB::kLoads;
    static_assert(S::kStages == 4, "two stages of 64");
    uint16_t* const us = reinterpret_cast<uint16_t*>(shared);
    uint16_t* const ls = us + 2 * S::kA;
    uint16_t* const bs = ls + 2 * S::kA;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
    const int wm = wave / S::NWN, wn = wave % S::NWN;
    int tm, tn;
    tile_of(tile, static_cast<int>((p.M + S::BM - 1) / S::BM), static_cast<int>((p.N + S::BN - 1) / S::BN), &tm, &tn);
    const int64_t m0 = static_cast<int64_t>(tm) * S::BM, n0 = static_cast<int64_t>(tn) * S::BN;
    OA upper, lower;
    OB b;
    upper.init(static_cast<const uint16_t*>(p.A), p.lda, m0, p.M, wave, lane, wm);
    lower.init(static_cast<const uint16_t*>(p.A), p.lda, m0 + S::BM / 2, p.M, wave, lane, wm);
    b.init(static_cast<const uint16_t*>(p.B), p.ldb, n0, p.N, wave, lane, wn);
    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int nk = static_cast<int>((p.K + K2 - 1) / K2 + 1) / 2 * 2;
    const int full = static_cast<int>(p.K / K2);
    Store<S, PLAIN> out;
    out.init(p, m0 + wm * S::kWaveStep, n0 + wn * S::WN, lane);
    u32x4 fa[2][H], fb[2][TN];
    auto rows = [&](const OA& o, const uint16_t* stage, int h) {
#pragma unroll
        for (int i = 0; i < H; ++i) fa[h][i] = o.frag(stage, i, h);
    };
    auto weights = [&](const uint16_t* stage, int h) {
#pragma unroll
        for (int j = 0; j < TN; ++j) fb[h][j] = b.frag(stage, j, h);
    };
    auto multiply = [&](int half, int h) {
#pragma unroll
        for (int i = 0; i < H; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[half * H + i][j] = mfma(fb[h][j], fa[h][i], acc[half * H + i][j]);
    };
    auto round = [&](auto whole, int kt) {    // stages kt and kt + 1 (kt even)
        constexpr bool FULL = decltype(whole)::value;
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const int64_t left = p.K - static_cast<int64_t>(kt + st + 2) * K2;
            rows(upper, us + st * S::kA, 1);
            weights(bs + st * 2 * S::kB, 1);
            multiply(0, 0);
            wait_vm_lds<kInFlight>();         // this stage's lower rows have landed, its upper rows and weights are in registers
            wave_barrier();
            upper.template issue<FULL>(us + st * S::kA, wave, left);
            b.template issue<FULL>(bs + st * 2 * S::kB, wave, left);
            rows(lower, ls + st * S::kA, 0);
            multiply(0, 1);
            rows(lower, ls + st * S::kA, 1);
            multiply(1, 0);
            wait_vm_lds<kInFlight>();         // the next stage's upper rows and weights have landed, this one's lower rows are in registers
            wave_barrier();
            lower.template issue<FULL>(ls + st * S::kA, wave, left);
            rows(upper, us + (st ^ 1) * S::kA, 0);
            weights(bs + (st ^ 1) * 2 * S::kB, 0);
            multiply(1, 1);
        }
    };
    if (nk > 0) {
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const int64_t left = p.K - st * K2;
            upper.template issue<false>(us + st * S::kA, wave, left);
            b.template issue<false>(bs + st * 2 * S::kB, wave, left);
            lower.template issue<false>(ls + st * S::kA, wave, left);
        }
        wait_vm<kInFlight + OA::kLoads>();    // the first stage's upper rows and weights
        wave_barrier();
        rows(upper, us, 0);
        weights(bs, 0);
        int kt = 0;
        for (; kt + 4 <= full; kt += 2) round(Bool<true>{}, kt);
        out.fetch(p, 0);
        for (; kt < nk; kt += 2) round(Bool<false>{}, kt);
        wait_vm<0>();                         // the requests past the end
    }
    wave_barrier();                           // the stages become the epilogue's strips
    if (nk == 0) out.fetch(p, 0);
    out.run(p, acc, reinterpret_cast<float*>(shared) + wave * S::kStrip, lane);
}

// Tiles of 64 x 64 for 2 x 2 waves: up to five work-groups share a compute
// unit.  In iteration kt a wave multiplies slice kt
// from registers, reads slice kt + 1's fragments from LDS into the other set
// and requests slice kt + 4 into the stage that slice kt's fragments were
// read from an iteration ago; one barrier an iteration.
template <bool AK, bool BK, bool PLAIN, typename S>
__device__ __forceinline__ void gemm_small(const GemmProduct& p, int tile, uint8_t* shared) {
    using OA = Operand<AK, S::BM, S::kWaves, S::WM, kTK>;
    using OB = Operand<BK, S::BN, S::kWaves, S::WN, kTK>;
    constexpr int TM = S::TM, TN = S::TN;
    constexpr int kPer = OA::kLoads + OB::kLoads, kStages = S::kStages;
    uint16_t* const as = reinterpret_cast<uint16_t*>(shared);
    uint16_t* const bs = as + kStages * S::kA;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
    const int wm = wave / S::NWN, wn = wave % S::NWN;
    int tm, tn;
    tile_of(tile, static_cast<int>((p.M + S::BM - 1) / S::BM), static_cast<int>((p.N + S::BN - 1) / S::BN), &tm, &tn);
    const int64_t m0 = static_cast<int64_t>(tm) * S::BM, n0 = static_cast<int64_t>(tn) * S::BN;
    OA a;
    OB b;
    a.init(static_cast<const uint16_t*>(p.A), p.lda, m0, p.M, wave, lane, wm);
    b.init(static_cast<const uint16_t*>(p.B), p.ldb, n0, p.N, wave, lane, wn);
    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int nk = static_cast<int>((p.K + kTK - 1) / kTK + kStages - 1) / kStages * kStages;
    const int full = static_cast<int>(p.K / kTK);
    Store<S, PLAIN> out;
    out.init(p, m0 + wm * S::kWaveStep, n0 + wn * S::WN, lane);
    u32x4 fa[2][TM], fb[2][TN];
    auto fragments = [&](int stage, int set) {
#pragma unroll
        for (int j = 0; j < TN; ++j) fb[set][j] = b.frag(bs + stage * S::kB, j, 0);
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[set][i] = a.frag(as + stage * S::kA, i, 0);
    };
    auto round = [&](auto whole, int kt) {
        constexpr bool FULL = decltype(whole)::value;
#pragma unroll
        for (int st = 0; st < kStages; ++st) {
            const int64_t left = p.K - static_cast<int64_t>(kt + st + kStages) * kTK;
            wait_vm_lds<2 * kPer>();          // slice kt + 1 has landed, slice kt's fragments are in registers
            wave_barrier();
            a.template issue<FULL>(as + st * S::kA, wave, left);
            b.template issue<FULL>(bs + st * S::kB, wave, left);
            fragments((st + 1) % kStages, (st + 1) % 2);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = mfma(fb[st % 2][j], fa[st % 2][i], acc[i][j]);
        }
    };
    if (nk > 0) {
#pragma unroll
        for (int st = 0; st < kStages; ++st) {
            const int64_t left = p.K - st * kTK;
            a.template issue<false>(as + st * S::kA, wave, left);
            b.template issue<false>(bs + st * S::kB, wave, left);
        }
        wait_vm_lds<3 * kPer>();              // slice 0
        wave_barrier();
        fragments(0, 0);
        int kt = 0;
        for (; kt + 2 * kStages <= full; kt += kStages) round(Bool<true>{}, kt);
        out.fetch(p, 0);
        for (; kt < nk; kt += kStages) round(Bool<false>{}, kt);
        wait_vm_lds<0>();                     // the requests past the end
    }
    wave_barrier();                           // the stages become the epilogue's strips
    if (nk == 0) out.fetch(p, 0);
    out.run(p, acc, reinterpret_cast<float*>(shared) + wave * S::kStrip, lane);
}

using Large = Shape<256, 256, 2, 4, 4, 2>;
using Wide = Shape<256, 128, 4, 2, 4, 2>;
using Medium = Shape<128, 128, 2, 2, 4, 2>;
using Small = Shape<64, 64, 2, 2, 4, 2>;

template <bool AK, bool BK, bool PLAIN, typename S>
__device__ __forceinline__ void gemm_tile(const GemmProduct& p, int tile, uint8_t* shared) {
    if constexpr (S::BM == 256) gemm_large<AK, BK, PLAIN, S>(p, tile, shared);
    else if constexpr (S::BM == 128) gemm_medium<AK, BK, PLAIN, S>(p, tile, shared);
    else gemm_small<AK, BK, PLAIN, S>(p, tile, shared);
}

template <typename S>
__global__ __launch_bounds__(S::kThreads, S::kPerSimd) void linear_forward_kernel(GemmProduct p) {
    __shared__ __align__(1024) uint8_t shared[S::kBytes];
    gemm_tile<true, true, false, S>(p, blockIdx.x, shared);
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
    if (is_dx(tx, tw, dw.K > dx.K, &tile)) gemm_tile<true, false, true, S>(dx, tile, shared);
    else gemm_tile<false, false, true, S>(dw, tile, shared);
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
    gemm_tile<AK, BK, true, Small>(p, block % tiles, shared);
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
int64_t tiles(const GemmProduct& p) { return ((p.M + S::BM - 1) / S::BM) * ((p.N + S::BN - 1) / S::BN); }

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

// Which tiles: the time of one tile on a compute unit at K = 2048, in us, times
// the rounds of tiles over the compute units; tiles that share one take longer
// where they have it to themselves.  Measured, in the order 256 x
// 256, 256 x 128, 128 x 128, 64 x 64:
//   4096 x 12288 x 2048: 148, 173, 231, 341 us
//   4096 x  2048 x 4096:  73,  55,  75, 125 us
//   2048 x  2048 x 2048:  41,  27,  24,  34 us
//   1024 x  2048 x 2048:  40,  26,  23,  18 us
//   1024 x 12352 x 2048:  45,  54,  70,  93 us
constexpr double kLargeUs = 46.0, kWideUs = 27.0, kMediumUs = 18.0, kSmallUs = 8.5;
constexpr double kMediumAlone = 24.0, kSmallAlone = 11.0;
enum Tiles { kLarge, kWide, kMedium, kSmall };

struct Choice {
    Tiles tiles;
    double us;
};

static Choice choose(const GemmProduct& p, int cus) {
    auto us = [&](int64_t n, double each, double alone) {
        const double t = static_cast<double>((n + cus - 1) / cus) * each;
        return t > alone ? t : alone;
    };
    const Choice all[4] = {{kLarge, us(tiles<Large>(p), kLargeUs, kLargeUs)}, {kWide, us(tiles<Wide>(p), kWideUs, kWideUs)},
                           {kMedium, us(tiles<Medium>(p), kMediumUs, kMediumAlone)},
                           {kSmall, us(tiles<Small>(p), kSmallUs, kSmallAlone)}};
    Choice best = all[0];
    for (int i = 1; i < 4; ++i)
        if (all[i].us < best.us) best = all[i];
    return best;
}

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
