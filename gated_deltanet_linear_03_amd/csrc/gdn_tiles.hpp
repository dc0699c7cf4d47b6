// gdn_tiles.hpp -- matrix products in tiles on the matrix cores, for the kernels
// that put an epilogue of their own behind them: the operands' way through
// LDS, the loops over the reduction for four tile sizes, and the linear
// layer's epilogue (bias, activation, residual, pre-activation).
//
// A tile loop is a template over its epilogue `Out`, an object of which each
// thread has:
//   init(p, m0, n0, wave, lane)   the tile's first row and column
//   fetch(p, half)                called before the last slices are multiplied
//                                 (half 0): what the epilogue reads can be requested
//   run(p, acc, shared, wave, lane)   all waves, after the last product; the
//                                 stages' LDS is the epilogue's
#pragma once
#include <type_traits>

#include "gdn_device.hpp"
#include "gdn_kernels.hpp"

namespace gdn {

namespace {   // (each source file that includes this has its own copy)

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

// KEEP: eight bf16 go the ordinary way, for a kernel that reads them next
template <int W, bool KEEP = false>
__device__ __forceinline__ void store_n(void* p, bool bf16, int64_t at, int nv, const float* f) {
    if (bf16) {
        uint16_t* q = static_cast<uint16_t*>(p) + at;
        if (nv == W) {
            if constexpr (W == 8) {
                // (non-temporal: the tiles' outputs and residuals pass the L2 by, which holds operands)
                const Run8 h = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
                if constexpr (KEEP) *reinterpret_cast<Run8*>(q) = h;
                else __builtin_nontemporal_store(h, reinterpret_cast<Run8*>(q));
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
// PLAIN: nothing but y.  KEEP: as in store_n.  P: GemmProduct, or one with a
// factor of its own for the sums (PLAIN).
struct ScaledProduct : GemmProduct {
    const float* scale;                       // device; NULL, or not finite: 1
    float factor;
};

__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) <= 3.402823466e38f; }
__device__ __forceinline__ float finite_or_one(float x) { return is_finite(x) ? x : 1.f; }

template <typename S, bool PLAIN, bool KEEP = false, typename P = GemmProduct>
struct Store {
    static constexpr int kRun = S::WN / 8;    // lanes of a row
    static constexpr int kRowsAtOnce = kWave / kRun;
    static constexpr int kRows = 16 * S::kStripTiles, kMine = kRows / kRowsAtOnce;   // rows of a half; of a lane
    static constexpr int kBatch = kMine < 4 ? kMine : 4;
    int64_t m0, n;                            // the wave's first row, the lane's first column
    int first, nv;                            // the lane's first row of a half; its columns
    bool early;                               // the residual can be fetched as bf16 runs
    Run8 res[kMine];

    __device__ __forceinline__ void init(const P& p, int64_t tile_m, int64_t tile_n, int wave, int lane) {
        m0 = tile_m + wave / S::NWN * S::kWaveStep;
        first = lane / kRun;
        n = tile_n + wave % S::NWN * S::WN + 8 * (lane % kRun);
        nv = p.N - n < 8 ? (p.N > n ? static_cast<int>(p.N - n) : 0) : 8;
        early = !PLAIN && p.ep.residual && p.ep.bf16 && nv == 8;
    }

    __device__ __forceinline__ void fetch(const P& p, int half) {
        if (PLAIN || !early) return;
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
            const int64_t m = m0 + half * S::kHalfStep + first + u * kRowsAtOnce;
            if (m < p.M)
                res[u] = __builtin_nontemporal_load(
                    reinterpret_cast<const Run8*>(static_cast<const uint16_t*>(p.ep.residual) + m * p.ep.ldr + n));
        }
    }

    __device__ __forceinline__ void run(const P& p, f32x4 (&acc)[S::TM][S::TN], uint8_t* shared, int wave, int lane) {
        float* const strip = reinterpret_cast<float*>(shared) + wave * S::kStrip;
        const int l16 = lane % 16, lq = lane / 16;
        float bias[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) bias[e] = 0.f;
        if (!PLAIN && p.ep.bias && nv > 0) load_n<8>(p.ep.bias, false, n, nv, bias);
        constexpr bool kScaled = !std::is_same<P, GemmProduct>::value;
        float scale = 1.f;
        if constexpr (kScaled) scale = p.scale ? finite_or_one(*p.scale) * p.factor : 1.f;
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
                    for (int e = 0; e < 4; ++e) {
                        f[u][e] = kScaled ? q0[e] * scale : q0[e] + bias[e];
                        f[u][4 + e] = kScaled ? q1[e] * scale : q1[e] + bias[4 + e];
                    }
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
                    if (m < p.M && nv > 0) store_n<8, KEEP>(p.ep.y, p.ep.bf16, m * p.ep.ldy + n, nv, f[u]);
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
template <bool AK, bool BK, typename Out, typename S, typename P>
__device__ __forceinline__ void gemm_large(const P& p, int tile, uint8_t* shared) {
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
    Out out;
    out.init(p, m0, n0, wave, lane);
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
    out.run(p, acc, shared, wave, lane);
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
template <bool AK, bool BK, typename Out, typename S, typename P>
__device__ __forceinline__ void gemm_medium(const P& p, int tile, uint8_t* shared) {
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
    Out out;
    out.init(p, m0, n0, wave, lane);
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
    out.run(p, acc, shared, wave, lane);
}

// Tiles of 64 x 64 for 2 x 2 waves: up to five work-groups share a compute
// unit.  In iteration kt a wave multiplies slice kt
// from registers, reads slice kt + 1's fragments from LDS into the other set
// and requests slice kt + 4 into the stage that slice kt's fragments were
// read from an iteration ago; one barrier an iteration.
template <bool AK, bool BK, typename Out, typename S, typename P>
__device__ __forceinline__ void gemm_small(const P& p, int tile, uint8_t* shared) {
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
    Out out;
    out.init(p, m0, n0, wave, lane);
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
    out.run(p, acc, shared, wave, lane);
}

using Large = Shape<256, 256, 2, 4, 4, 2>;
using Wide = Shape<256, 128, 4, 2, 4, 2>;
using Medium = Shape<128, 128, 2, 2, 4, 2>;
using Small = Shape<64, 64, 2, 2, 4, 2>;

template <bool AK, bool BK, typename Out, typename S, typename P>
__device__ __forceinline__ void gemm_tile(const P& p, int tile, uint8_t* shared) {
    if constexpr (S::BM == 256) gemm_large<AK, BK, Out, S>(p, tile, shared);
    else if constexpr (S::BM == 128) gemm_medium<AK, BK, Out, S>(p, tile, shared);
    else gemm_small<AK, BK, Out, S>(p, tile, shared);
}

template <typename S>
int64_t tiles(const GemmProduct& p) { return ((p.M + S::BM - 1) / S::BM) * ((p.N + S::BN - 1) / S::BN); }

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

inline Choice choose(const GemmProduct& p, int cus) {
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

}  // namespace

}  // namespace gdn
