// gdn_adamw.hip -- one AdamW step over many tensors, 48 (states in 8 bits)
// or 64 of them a launch.
//
//   m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g^2
//   p' = p - lr (m' / (1 - b1^k) / (sqrt(v' / (1 - b2^k)) + eps) + decay p)
//
// The states are m and v in 32 bits, or, in 8 bits, m and r = sqrt(v) in e4m3
// with one 32-bit scale for kAdamwBlock elements (the largest magnitude / 448).
// Why r: e4m3 spans a ratio of 2.3e5, which for r is one of 5e10 for v.  Why
// they are rounded up or down at random, by the probability that keeps the
// expected value: a step changes v by a thousandth of itself and e4m3 has
// steps of an eighth to a sixteenth, so rounding to the nearest would leave v
// where it was for ever.  A positive r is never rounded to zero (the next step
// would divide by eps alone).
// Everything between the loads and the stores is in 32 bits, but for what
// decides an 8-bit code: where a value lies between two codes is compared with
// the random bits, and 32 bits would decide a millionth of the elements
// otherwise than the formula does, each of them by a whole step.  So the
// scales come from the largest value in 64 bits, and a block with a value that
// lies nearer to its border than 32 bits can tell (one or two in a hundred)
// takes them from 64 bits: 269.5 M elements take 776 to 818 us, 948 with all of them in
// 64 bits and 745 with none.
//
// Bound: HBM.  Each element is read and written once: 28 bytes with 32-bit
// states, a bf16 gradient and a bf16 copy, 16 with 8-bit states (269.5 M elements:
// 1.27 to 1.30 ms, 5.8 TB/s, and 0.78 to 0.82 ms, 5.4, with the vector units busy
// throughout).  A wave's 64
// lanes take four adjacent elements each, which is a block of the 8-bit
// states, so a block's largest magnitude is one reduction over a wave.
#include <type_traits>

#include "gdn_device.hpp"
#include "gdn_kernels.hpp"

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int kLane = 4;                                    // adjacent elements of a lane
static_assert(kAdamwBlock == kLane * kWave, "a wave is a block of the 8-bit states");
constexpr int kRounds = 4;                                  // blocks that a wave has in flight
constexpr int kChunk = kThreads * kLane * kRounds;          // elements of a work-group
static_assert((kChunk & (kChunk - 1)) == 0, "a chunk does not cross a multiple of 2^32");

// A tensor as the kernel sees it.  A launch's arguments hold as many as 4 KiB do.
struct Tensor {
    int64_t n;
    float* param;
    const void* grad;
    void* copy;
    void *m, *v;
    float weight_decay;
    uint32_t index;                                         // its place in the call, and (top bit) a bf16 gradient
};
struct Scales {
    float *m_scale, *v_scale;
};
struct NoScales {};

template <bool EIGHT>
struct Launch {
    static constexpr int kTensors = EIGHT ? 48 : 64;
    AdamwParams p;
    Tensor t[kTensors];
    typename std::conditional<EIGHT, Scales, NoScales>::type scales[EIGHT ? kTensors : 1];
    uint32_t first[kTensors + 1];                           // work-groups before each tensor's
    int count;
};
static_assert(sizeof(Launch<true>) <= 4096 && sizeof(Launch<false>) <= 4096, "kernel arguments");

struct Target : Tensor, Scales {};

typedef uint32_t U4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t U2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t U1 __attribute__((aligned(1)));

// The finaliser of MurmurHash3 (Austin Appleby, public domain): every bit of
// the word depends on every bit of h.
__device__ __forceinline__ uint32_t mix(uint32_t h) {
    h = (h ^ (h >> 16)) * 0x85EBCA6Bu;
    h = (h ^ (h >> 13)) * 0xC2B2AE35u;
    return h ^ (h >> 16);
}

// Code of y (|y| <= 448 but for a rounding) in e4m3, up or down by 16 random
// bits: they are added below the last of the three mantissa bits that stay.
// Below 2^-6 the format's steps are 2^-9 throughout, which are those of the
// mantissa of y + 2^-6.  near: y is within kNear of its last bits of the
// border.  (In those bits m' y is off by up to 5: m' by 1, the scale's
// reciprocal and the product by up to 2 and 1 at the upper end of a binade, y +
// 2^-6 by 1/2; r's y by up to 8: its square by 2.5 halves, the root by 2, and
// the same.)
constexpr uint32_t kNear = 8;
__device__ __forceinline__ uint32_t e4m3(float y, uint32_t random16, bool* near) {
    const float a = fabsf(y);
    const bool small = a < 0.015625f;
    const uint32_t t = __float_as_uint(small ? a + 0.015625f : a) + (random16 << 4);
    *near = ((t + kNear) & 0xFFFFFu) < 2 * kNear;
    // exponent -6 has the codes 8 .. 15
    uint32_t code = (t >> 20) - ((127 - 6) << 3) + (small ? 0 : 8);
    code = code < 0x7E ? code : 0x7E;
    return __float_as_uint(y) >> 31 << 7 | (y != y ? 0x7F : code);
}
// the same in 64 bits, of whose upper word all that counts is part
__device__ __forceinline__ uint32_t upper_word(double y) {
    return static_cast<uint32_t>(static_cast<uint64_t>(__double_as_longlong(y)) >> 32);
}
__device__ __forceinline__ uint32_t e4m3(double y, uint32_t random16) {
    const double a = fabs(y);
    const bool small = a < 0.015625;
    const uint32_t t = upper_word(small ? a + 0.015625 : a) + (random16 << 1);
    uint32_t code = (t >> 17) - ((1023 - 6) << 3) + (small ? 0 : 8);
    code = code < 0x7E ? code : 0x7E;
    return upper_word(y) >> 31 << 7 | (y != y ? 0x7F : code);
}

// The largest x >= 0 of a wave, in a scalar register: within rows of 16 lanes,
// from row to row, to lane 63 (non-negative floats are ordered like their
// bits; lanes without a neighbour get 0).
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t x) {
    const uint32_t y = __builtin_amdgcn_update_dpp(0, x, CTRL, 0xF, 0xF, true);
    return x > y ? x : y;
}
__device__ __forceinline__ float wave_max(float v) {
    uint32_t x = __float_as_uint(v);
    x = max_dpp<0x111>(x);                                  // row_shr 1, 2, 4, 8
    x = max_dpp<0x112>(x);
    x = max_dpp<0x114>(x);
    x = max_dpp<0x118>(x);
    x = max_dpp<0x142>(x);                                  // row_bcast 15, 31
    x = max_dpp<0x143>(x);
    return __uint_as_float(__builtin_amdgcn_readlane(x, 63));
}

// what a step's elements have in common
struct Step {
    double b1, b2, rest1, rest2;                            // beta and 1 - beta
    float f_b1, f_b2, f_rest1, f_rest2, low_b1, low_rest1;  // in 32 bits, and what is left
    float lr, eps, decay, c1, c2;                           // c1 = lr / (1 - b1^k), c2 = 1 / sqrt(1 - b2^k)
    float grad_scale;
    uint32_t key;                                           // of the random bits, with the index's upper word
};

// Squares below this may lose bits in 32 (gradients below 1e-13 or so): there the
// r of 8-bit states comes from 64 (2^26 elements: 202 us, 197 to 199 without;
// zeros 196 and 184, all of them small 252 and 187).
constexpr float kSmallSquare = 0x1p-96f;

// m' and v' in 64 bits, each operation rounded by itself: beta1 = 0.9 makes m' =
// (9 m + g) / 10, which is a short number every fifth time, and then the ratio
// to the scale can lie on a border to the bit.
__device__ __forceinline__ double new_m(const Step& s, float m0, float g) {
#pragma clang fp contract(off)
    const double a = s.b1 * static_cast<double>(m0), b = s.rest1 * static_cast<double>(g);
    return a + b;
}
// (r0: the old v's root; its square counts in 32 bits where those hold it)
__device__ __forceinline__ double new_v(const Step& s, float r0, float g) {
#pragma clang fp contract(off)
    const float q = r0 * r0;
    const double v0 = q < kSmallSquare ? static_cast<double>(r0) * static_cast<double>(r0) : static_cast<double>(q);
    const double a = s.b2 * v0, b = s.rest2 * static_cast<double>(g) * static_cast<double>(g);
    return a + b;
}
// sqrt(v') to its last bit or next to it: two of Newton's steps from the root in 32 bits
__device__ __forceinline__ double new_r(const Step& s, float r0, float g) {
    const double v1 = new_v(s, r0, g);
    if (v1 < kSmallSquare && v1 > 0.0) return sqrt(v1);
    const float r = __builtin_amdgcn_sqrtf(static_cast<float>(v1));
    if (!(r > 0.f && r < __builtin_inff())) return r;
    const double half = 0.5 * static_cast<double>(__builtin_amdgcn_rcpf(r)), a = r;
    const double b = fma(fma(-a, a, v1), half, a);
    return fma(fma(-b, b, v1), half, b);
}
// the same in 32 bits where v' is below kSmallSquare; zero only for zero
__device__ __forceinline__ float small_r(const Step& s, float r0, float g) {
    const double r = sqrt(new_v(s, r0, g));
    const float f = static_cast<float>(r);
    return r > 0.0 && f == 0.f ? 0x1p-149f : f;
}
// v_sqrt_f32 takes a subnormal number for zero
__device__ __forceinline__ float root(float v) {
    const bool small = v < kSmallSquare;
    return __builtin_amdgcn_sqrtf(small ? v * 0x1p64f : v) * (small ? 0x1p-32f : 1.f);
}

// What a wave's blocks' scales come from, in the lanes 2 i (m) and 2 i + 1 (r)
// of block i: the largest magnitude in 32 bits, and the state's value and the
// gradient behind it.  The scales' 64 bits are then computed once for all of
// them (block by block 269.5 M elements take 813 us where that takes 783).
struct Largest {
    float top, old, grad;

    __device__ __forceinline__ static float of(const float (&x)[kLane], int e, int lane) {
        const float a = x[0], b = x[1], c = x[2], d = x[3];
        const float lo = e & 1 ? b : a, hi = e & 1 ? d : c, v = e & 2 ? hi : lo;
        return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
    }
    __device__ __forceinline__ static float put(float v, int lane, float to) {
        return static_cast<int>(__lane_id()) == lane ? v : to;
    }

    // size: the lane's magnitudes (NaN does not count); x, g: what they come from
    template <bool R>
    __device__ __forceinline__ void offer(const Step& s, int at, const float (&size)[kLane], const float (&x)[kLane], const float (&g)[kLane]) {
        static_assert(kLane == 4, "four values");
        const float t = fmaxf(fmaxf(size[0], size[1]), fmaxf(size[2], fmaxf(size[3], 0.f))), most = wave_max(t);
        // those that 32 bits do not tell from the largest: one as a rule
        const float least = most * (1.f - 0x1p-20f);
        const uint32_t mine = (size[0] >= least ? 1u : 0u) | (size[1] >= least ? 2u : 0u) | (size[2] >= least ? 4u : 0u) | (size[3] >= least ? 8u : 0u);
        uint64_t who = __ballot(t >= least);
        int lane = __builtin_ctzll(who | 1ull << 63);
        uint32_t bits = __builtin_amdgcn_readlane(mine, lane);
        int e = __builtin_ctz(bits | 16u) % kLane;
        float x1 = of(x, e, lane), g1 = of(g, e, lane);
        if ((who & (who - 1)) != 0 || (bits & (bits - 1)) != 0) {
            // One after the other, all that come from the same pair (or, as
            // magnitudes go, from its negative) at once: gradients of one size
            // make ties of whole blocks (2^26 elements of one gradient: value by
            // value 6.78 ms, so 0.24; of random ones 0.20 to 0.21 either way).
            double best = -1.0;
            uint32_t left = mine;
            while (who != 0 && most > 0.f) {
                lane = __builtin_ctzll(who);
                e = __builtin_ctz(__builtin_amdgcn_readlane(left, lane) | 16u) % kLane;
                const float x2 = of(x, e, lane), g2 = of(g, e, lane);
                const double v = R ? new_r(s, x2, g2) : fabs(new_m(s, x2, g2));
                if (v > best) { best = v; x1 = x2; g1 = g2; }
#pragma unroll
                for (int k = 0; k < kLane; ++k) {
                    const bool same = (x[k] == x2 && (R ? fabsf(g[k]) == fabsf(g2) : g[k] == g2)) || (!R && x[k] == -x2 && g[k] == -g2);
                    left &= same ? ~(1u << k) : ~0u;
                }
                // (the one itself in any case: the loop ends after 256 of them at the most)
                left &= static_cast<int>(__lane_id()) == lane ? ~(1u << e) : ~0u;
                who = __ballot(left != 0);
            }
        }
        top = put(most, at, top);
        old = put(x1, at, old);
        grad = put(g1, at, grad);
    }

    // the scale of this lane's block and kind
    __device__ __forceinline__ float scale(const Step& s, int lane) const {
        const double m = fabs(new_m(s, old, grad)), r = new_r(s, old, grad);
        const float v = static_cast<float>((lane % 2 ? r : m) / 448.0);   // (not times 1 / 448: ties)
        // (next to nothing counts as nothing: the ratios stay finite)
        return !(top < __builtin_inff()) ? top : top < 0x1p-100f ? 0.f : v;
    }
};

__device__ __forceinline__ float from_lane(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

template <bool EIGHT, bool GB, bool FULL>
struct Elements {
    float p[kLane], g[kLane], m[kLane], v[kLane];
    float m0[EIGHT ? kLane : 1], r0[EIGHT ? kLane : 1];     // 8 bits: what the states stand for (v: r)
    // 8 bits: codes and scales before the step and after it (the scales are the wave's)
    uint32_t qm, qv, new_qm, new_qv;
    float sm, sv;
    uint32_t border;                                        // bits 0 .. 3: m's elements next to their borders, 4 .. 7: r's
    float ms, vs;

    // (FULL: all four elements exist)
    __device__ __forceinline__ void load(const Target& t, int64_t at, int nv) {
        if constexpr (FULL) {
            const U4 a = __builtin_nontemporal_load(reinterpret_cast<const U4*>(t.param + at));
#pragma unroll
            for (int e = 0; e < kLane; ++e) p[e] = __uint_as_float(a[e]);
            if constexpr (GB) {
                const U2 b = __builtin_nontemporal_load(reinterpret_cast<const U2*>(static_cast<const uint16_t*>(t.grad) + at));
#pragma unroll
                for (int e = 0; e < kLane; ++e) g[e] = __uint_as_float(e % 2 ? b[e / 2] & 0xFFFF0000u : b[e / 2] << 16);
            } else {
                const U4 b = __builtin_nontemporal_load(reinterpret_cast<const U4*>(static_cast<const float*>(t.grad) + at));
#pragma unroll
                for (int e = 0; e < kLane; ++e) g[e] = __uint_as_float(b[e]);
            }
            if constexpr (EIGHT) {
                qm = __builtin_nontemporal_load(reinterpret_cast<const U1*>(static_cast<const uint8_t*>(t.m) + at));
                qv = __builtin_nontemporal_load(reinterpret_cast<const U1*>(static_cast<const uint8_t*>(t.v) + at));
            } else {
                const U4 b = __builtin_nontemporal_load(reinterpret_cast<const U4*>(static_cast<const float*>(t.m) + at));
                const U4 c = __builtin_nontemporal_load(reinterpret_cast<const U4*>(static_cast<const float*>(t.v) + at));
#pragma unroll
                for (int e = 0; e < kLane; ++e) { m[e] = __uint_as_float(b[e]); v[e] = __uint_as_float(c[e]); }
            }
        } else {
            qm = qv = 0;
#pragma unroll
            for (int e = 0; e < kLane; ++e) {
                p[e] = g[e] = m[e] = v[e] = 0.f;
                if (e < nv) {
                    p[e] = t.param[at + e];
                    g[e] = GB ? bf16_bits_to_f32(static_cast<const uint16_t*>(t.grad)[at + e]) : static_cast<const float*>(t.grad)[at + e];
                    if constexpr (EIGHT) {
                        qm |= static_cast<uint32_t>(static_cast<const uint8_t*>(t.m)[at + e]) << (8 * e);
                        qv |= static_cast<uint32_t>(static_cast<const uint8_t*>(t.v)[at + e]) << (8 * e);
                    } else {
                        m[e] = static_cast<const float*>(t.m)[at + e];
                        v[e] = static_cast<const float*>(t.v)[at + e];
                    }
                }
            }
        }
        if constexpr (EIGHT) {
            const int64_t block = __builtin_amdgcn_readfirstlane(static_cast<int>(at / kAdamwBlock));   // (fewer than 2^31: n is below 2^36)
            ms = t.m_scale[block];
            vs = t.v_scale[block];
        }
    }

    __device__ __forceinline__ void decode() {
        const f32x2 m0 = __builtin_amdgcn_cvt_pk_f32_fp8(qm, false), m1 = __builtin_amdgcn_cvt_pk_f32_fp8(qm, true);
        const f32x2 v0 = __builtin_amdgcn_cvt_pk_f32_fp8(qv, false), v1 = __builtin_amdgcn_cvt_pk_f32_fp8(qv, true);
        m[0] = m0[0]; m[1] = m0[1]; m[2] = m1[0]; m[3] = m1[1];
        v[0] = v0[0]; v[1] = v0[1]; v[2] = v1[0]; v[3] = v1[1];
    }

    // p, and m and v (8 bits: r in v) after the step
    __device__ __forceinline__ void update(const Step& s) {
        if constexpr (EIGHT) decode();
        float r[kLane];
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
            g[e] *= s.grad_scale;
            if constexpr (EIGHT) {
                m0[e] = m[e] * ms;
                r0[e] = v[e] * vs;
                // to its last bit also where its terms cancel: with what the
                // product and the factors have lost (a multiply-add rounds the other)
                const float gg = s.f_rest1 * g[e], q = fmaf(s.f_b1, m0[e], gg);
                m[e] = q + fmaf(s.low_b1, m0[e], fmaf(s.low_rest1, g[e], fmaf(s.f_rest1, g[e], -gg)));
                v[e] = fmaf(s.f_b2, r0[e] * r0[e], s.f_rest2 * g[e] * g[e]);
                r[e] = __builtin_amdgcn_sqrtf(v[e]);
            } else {
                m[e] = fmaf(s.f_b1, m[e], s.f_rest1 * g[e]);
                v[e] = fmaf(s.f_b2, v[e], s.f_rest2 * g[e] * g[e]);
                r[e] = root(v[e]);
            }
        }
        if constexpr (EIGHT) {
            static_assert(kLane == 4, "four values");
            if (__any(fminf(fminf(v[0], v[1]), fminf(v[2], v[3])) < kSmallSquare)) {
                uint32_t small = 0;                         // (zeros of zeros are as they are)
#pragma unroll
                for (int e = 0; e < kLane; ++e)
                    small |= v[e] < kSmallSquare && (__float_as_uint(r0[e]) | __float_as_uint(g[e])) << 1 != 0 ? 1u << e : 0u;
                if (__any(small != 0)) {
#pragma unroll
                    for (int e = 0; e < kLane; ++e)
                        if (small >> e & 1u) r[e] = small_r(s, r0[e], g[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < kLane; ++e) v[e] = r[e];
        }
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
            const float step = m[e] * s.c1 * __builtin_amdgcn_rcpf(fmaf(r[e], s.c2, s.eps));
            p[e] -= fmaf(s.lr * s.decay, p[e], step);
        }
    }

    __device__ __forceinline__ static uint32_t random(const Step& s, int64_t at) {
        return mix(s.key + static_cast<uint32_t>(at) * 0x9E3779B1u);
    }

    __device__ __forceinline__ void offer(const Step& s, int block, Largest* l) const {
        // (elements past the end are zeros)
        float size[kLane];
#pragma unroll
        for (int e = 0; e < kLane; ++e) size[e] = fabsf(m[e]);
        l->offer<false>(s, 2 * block, size, m0, g);
        l->offer<true>(s, 2 * block + 1, v, r0, g);
    }

    // the codes of the new states
    __device__ __forceinline__ void encode(const Step& s, int64_t at, float new_sm, float new_sv) {
        sm = new_sm;
        sv = new_sv;
        const float um = sm > 0.f ? __builtin_amdgcn_rcpf(sm) : 0.f, uv = sv > 0.f ? __builtin_amdgcn_rcpf(sv) : 0.f;
        new_qm = new_qv = border = 0;
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
            const uint32_t h = random(s, at + e);
            bool near_m, near_r;
            new_qm |= e4m3(m[e] * um, h & 0xFFFFu, &near_m) << (8 * e);
            const uint32_t r = e4m3(v[e] * uv, h >> 16, &near_r);
            new_qv |= (r == 0 && v[e] > 0.f && sv > 0.f ? 1u : r) << (8 * e);
            border |= (near_m ? 1u << e : 0u) | (near_r ? 16u << e : 0u);
        }
    }

    // Codes next to a border once more, from 64 bits, over those that store()
    // has written (a lane's stores to an address stay in order).  One or two
    // blocks in a hundred have any.
    __device__ __forceinline__ void settle(const Target& t, const Step& s, int64_t at) {
        while (border) {
            const int b = __builtin_ctz(border), e = b % kLane;
            border &= border - 1;
            const bool of_m = b < kLane;
            const float grad = s.grad_scale * (GB ? bf16_bits_to_f32(static_cast<const uint16_t*>(t.grad)[at + e])
                                                  : static_cast<const float*>(t.grad)[at + e]);
            const uint32_t h = random(s, at + e);
            const float old = __builtin_amdgcn_cvt_f32_fp8((of_m ? qm : qv) >> (8 * e), 0) * (of_m ? ms : vs);
            uint32_t code;
            if (of_m) {
                code = e4m3(sm > 0.f ? new_m(s, old, grad) / static_cast<double>(sm) : 0.0, h & 0xFFFFu);
            } else {
                const double r = sqrt(new_v(s, old, grad));
                code = e4m3(sv > 0.f ? r / static_cast<double>(sv) : 0.0, h >> 16);
                if (code == 0 && r > 0.0 && sv > 0.f) code = 1;
            }
            static_cast<uint8_t*>(of_m ? t.m : t.v)[at + e] = static_cast<uint8_t>(code);
        }
    }

    // nv of the elements of each lane
    __device__ __forceinline__ void store_param(const Target& t, int64_t at, int nv) const {
        if constexpr (FULL) {
            const U4 a = {__float_as_uint(p[0]), __float_as_uint(p[1]), __float_as_uint(p[2]), __float_as_uint(p[3])};
            __builtin_nontemporal_store(a, reinterpret_cast<U4*>(t.param + at));
            if (t.copy) {
                const f32x2 lo = {p[0], p[1]}, hi = {p[2], p[3]};
                const U2 c = {__builtin_bit_cast(uint32_t, __builtin_convertvector(lo, bf16x2)),
                              __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, bf16x2))};
                __builtin_nontemporal_store(c, reinterpret_cast<U2*>(static_cast<uint16_t*>(t.copy) + at));
            }
        } else {
#pragma unroll
            for (int e = 0; e < kLane; ++e) {
                if (e >= nv) continue;
                t.param[at + e] = p[e];
                if (t.copy) static_cast<uint16_t*>(t.copy)[at + e] = f32_to_bf16_bits(p[e]);
            }
        }
    }

    __device__ __forceinline__ void store_state(const Target& t, int64_t at, int nv, int lane) const {
        if constexpr (EIGHT) {
            if (lane == 0) {
                t.m_scale[at / kAdamwBlock] = sm;
                t.v_scale[at / kAdamwBlock] = sv;
            }
        }
        if constexpr (FULL) {
            if constexpr (EIGHT) {
                __builtin_nontemporal_store(new_qm, reinterpret_cast<U1*>(static_cast<uint8_t*>(t.m) + at));
                __builtin_nontemporal_store(new_qv, reinterpret_cast<U1*>(static_cast<uint8_t*>(t.v) + at));
            } else {
                const U4 b = {__float_as_uint(m[0]), __float_as_uint(m[1]), __float_as_uint(m[2]), __float_as_uint(m[3])};
                const U4 c = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
                __builtin_nontemporal_store(b, reinterpret_cast<U4*>(static_cast<float*>(t.m) + at));
                __builtin_nontemporal_store(c, reinterpret_cast<U4*>(static_cast<float*>(t.v) + at));
            }
        } else {
#pragma unroll
            for (int e = 0; e < kLane; ++e) {
                if (e >= nv) continue;
                if constexpr (EIGHT) {
                    static_cast<uint8_t*>(t.m)[at + e] = static_cast<uint8_t>(new_qm >> (8 * e));
                    static_cast<uint8_t*>(t.v)[at + e] = static_cast<uint8_t>(new_qv >> (8 * e));
                } else {
                    static_cast<float*>(t.m)[at + e] = m[e];
                    static_cast<float*>(t.v)[at + e] = v[e];
                }
            }
        }
    }
};

template <int I>
struct Int { static constexpr int value = I; };

template <bool EIGHT, bool GB>
__device__ __forceinline__ void chunk(const Target& t, const Step& s, int64_t base) {
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    // a wave's blocks follow one another
    const int64_t at0 = base + static_cast<int64_t>(wave) * kRounds * kAdamwBlock + kLane * lane;
    if (base + kChunk <= t.n) {
        // (indices known to the compiler from the start: the blocks stay in registers)
        static_assert(kRounds == 4, "four blocks");
        auto each = [](auto f) __attribute__((always_inline)) { f(Int<0>{}); f(Int<1>{}); f(Int<2>{}); f(Int<3>{}); };
        Elements<EIGHT, GB, true> x[kRounds];
        Largest l{0.f, 0.f, 0.f};
        each([&](auto i) __attribute__((always_inline)) { x[i.value].load(t, at0 + i.value * kAdamwBlock, kLane); });
        each([&](auto i) __attribute__((always_inline)) {
            auto& b = x[i.value];
            b.update(s);
            b.store_param(t, at0 + i.value * kAdamwBlock, kLane);
            if constexpr (EIGHT) b.offer(s, i.value, &l);
            else b.store_state(t, at0 + i.value * kAdamwBlock, kLane, lane);
        });
        if constexpr (EIGHT) {
            const float scale = l.scale(s, lane);
            each([&](auto i) __attribute__((always_inline)) {
                auto& b = x[i.value];
                b.encode(s, at0 + i.value * kAdamwBlock, from_lane(scale, 2 * i.value), from_lane(scale, 2 * i.value + 1));
                b.store_state(t, at0 + i.value * kAdamwBlock, kLane, lane);
            });
            each([&](auto i) __attribute__((always_inline)) { x[i.value].settle(t, s, at0 + i.value * kAdamwBlock); });
        }
        return;
    }
    for (int i = 0; i < kRounds; ++i) {
        const int64_t at = at0 + i * kAdamwBlock, left = t.n - at;
        if (left + kLane * lane <= 0) return;               // (the whole wave)
        const int nv = left >= kLane ? kLane : left > 0 ? static_cast<int>(left) : 0;
        Elements<EIGHT, GB, false> x;
        x.load(t, at, nv);
        x.update(s);
        x.store_param(t, at, nv);
        if constexpr (EIGHT) {
            Largest l{0.f, 0.f, 0.f};
            x.offer(s, 0, &l);
            const float scale = l.scale(s, lane);
            x.encode(s, at, from_lane(scale, 0), from_lane(scale, 1));
        }
        x.store_state(t, at, nv, lane);
        if constexpr (EIGHT) {
            x.border &= ((1u << nv) - 1) * 0x11u;           // (none of elements past the end)
            x.settle(t, s, at);
        }
    }
}

template <bool EIGHT>
__global__ __launch_bounds__(kThreads, EIGHT ? 4 : 5) void adamw_kernel(Launch<EIGHT> a) {
    const AdamwParams& p = a.p;
    // the gradients' factor decides whether there is a step at all
    const float gs = p.grad_scale ? *p.grad_scale : 1.f;
    if (!(fabsf(gs) <= 3.402823466e38f)) return;
    const uint32_t b = blockIdx.x;
    int i = 0;
    for (int step = 32; step > 0; step /= 2)
        if (i + step < a.count && b >= a.first[i + step]) i += step;
    Target t;
    static_cast<Tensor&>(t) = a.t[i];
    if constexpr (EIGHT) static_cast<Scales&>(t) = a.scales[i];
    Step s;
    int32_t k = p.step_ptr ? *p.step_ptr : p.step;
    k = k < 1 ? 1 : k;
    s.lr = p.lr_ptr ? *p.lr_ptr : p.lr;
    s.b1 = p.beta1;
    s.b2 = p.beta2;
    s.rest1 = p.rest1;
    s.rest2 = p.rest2;
    s.f_b1 = static_cast<float>(p.beta1);
    s.f_b2 = static_cast<float>(p.beta2);
    s.f_rest1 = static_cast<float>(p.rest1);
    s.f_rest2 = static_cast<float>(p.rest2);
    s.low_b1 = static_cast<float>(p.beta1 - s.f_b1);
    s.low_rest1 = static_cast<float>(p.rest1 - s.f_rest1);
    s.eps = p.eps;
    s.decay = t.weight_decay;
    s.grad_scale = gs;
    // 1 - b^k = -expm1(k ln b): no cancellation where b^k is next to one
    s.c1 = s.lr / -expm1f(static_cast<float>(k) * p.log_beta1);
    s.c2 = 1.f / sqrtf(-expm1f(static_cast<float>(k) * p.log_beta2));
    s.key = mix(mix(p.seed + static_cast<uint32_t>(k) * 0x9E3779B1u) + (t.index & 0x7FFFFFFFu) * 0x9E3779B1u);
    const int64_t base = static_cast<int64_t>(b - a.first[i]) * kChunk;
    s.key += mix(static_cast<uint32_t>(static_cast<uint64_t>(base) >> 32));   // (one for all of the chunk)
    if (t.index >> 31) chunk<EIGHT, true>(t, s, base);
    else chunk<EIGHT, false>(t, s, base);
}

}  // namespace

int64_t adamw_chunks(int64_t n) { return (n + kChunk - 1) / kChunk; }

namespace {

template <bool EIGHT>
hipError_t launch(const AdamwParams& p, const gdn_adamw_tensor* tensors, int count, hipStream_t s) {
    for (int i = 0; i < count;) {
        Launch<EIGHT> a;
        a.p = p;
        a.count = 0;
        a.first[0] = 0;
        for (; i < count && a.count < Launch<EIGHT>::kTensors; ++i) {
            const gdn_adamw_tensor& t = tensors[i];
            if (t.n <= 0) continue;
            const int64_t end = a.first[a.count] + adamw_chunks(t.n);
            if (a.count > 0 && end > kAdamwMostChunks) break;
            a.t[a.count] = {t.n, t.param, t.grad, t.copy, t.m, t.v, t.weight_decay,
                            static_cast<uint32_t>(i) | (t.grad_dtype == GDN_DTYPE_BF16 ? 1u << 31 : 0u)};
            if constexpr (EIGHT) a.scales[a.count] = {t.m_scale, t.v_scale};
            a.first[++a.count] = static_cast<uint32_t>(end);
        }
        if (a.count == 0) break;
        hipLaunchKernelGGL(adamw_kernel<EIGHT>, dim3(a.first[a.count]), dim3(kThreads), 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_adamw(const AdamwParams& p, const gdn_adamw_tensor* tensors, int count, bool eight, hipStream_t s) {
    return eight ? launch<true>(p, tensors, count, s) : launch<false>(p, tensors, count, s);
}

}  // namespace gdn
