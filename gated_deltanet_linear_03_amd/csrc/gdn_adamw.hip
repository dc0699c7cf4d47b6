// gdn_adamw.hip -- one AdamW step over many tensors in one launch for every
// kAdamwTensors of them.
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
// would divide by eps alone).  Everything between the loads and the stores is
// in 32 bits.
//
// Bound: HBM.  Each element is read and written once: 28 bytes with 32-bit
// states, a bf16 gradient and a bf16 copy, 16 with 8-bit states.  A wave's 64
// lanes take four adjacent elements each, which is a block of the 8-bit
// states, so a block's largest magnitude is one reduction over a wave.
#include "gdn_device.hpp"
#include "gdn_kernels.hpp"

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int kLane = 4;                                    // adjacent elements of a lane
static_assert(kAdamwBlock == kLane * kWave, "a wave is a block of the 8-bit states");
constexpr int kRounds = 4;                                  // blocks that a wave has in flight
constexpr int kChunk = kThreads * kLane * kRounds;          // elements of a work-group

struct Launch {
    AdamwParams p;
    gdn_adamw_tensor t[kAdamwTensors];
    int64_t first[kAdamwTensors + 1];                       // work-groups before each tensor's
    int32_t index[kAdamwTensors];                           // a tensor's place in the whole call
    int count;
};
static_assert(sizeof(Launch) <= 4096, "kernel arguments");

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
// mantissa of y + 2^-6.
__device__ __forceinline__ uint32_t e4m3(float y, uint32_t random16) {
    const uint32_t bits = __float_as_uint(y), sign = bits >> 31 << 7;
    const float a = fabsf(y);
    const bool small = a < 0.015625f;
    const uint32_t t = __float_as_uint(small ? a + 0.015625f : a) + (random16 << 4);
    // exponent -6 has the codes 8 .. 15
    uint32_t code = (t >> 20) - ((127 - 6) << 3) + (small ? 0 : 8);
    code = code < 0x7E ? code : 0x7E;
    return sign | (y != y ? 0x7F : code);
}

__device__ __forceinline__ float wave_max(float x) {
    x = fmaxf(x, dpp_f32<0xB1>(x));
    x = fmaxf(x, dpp_f32<0x4E>(x));
    x = fmaxf(x, dpp_f32<0x141>(x));
    x = fmaxf(x, dpp_f32<0x140>(x));
    x = fmaxf(x, __shfl_xor(x, 16, kWave));
    return fmaxf(x, __shfl_xor(x, 32, kWave));
}

// what a step's elements have in common
struct Step {
    float lr, b1, b2, rest1, rest2, eps, decay, c1, c2;     // c1 = lr / (1 - b1^k), c2 = 1 / sqrt(1 - b2^k)
    float grad_scale;
    uint32_t key;                                           // of the random bits
};

template <bool EIGHT, bool GB, bool FULL>
struct Elements {
    float p[kLane], g[kLane], m[kLane], v[kLane];
    float ms, vs;

    // (FULL: all four elements exist)
    __device__ __forceinline__ void load(const gdn_adamw_tensor& t, int64_t at, int nv) {
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
                const uint32_t qm = __builtin_nontemporal_load(reinterpret_cast<const U1*>(static_cast<const uint8_t*>(t.m) + at));
                const uint32_t qv = __builtin_nontemporal_load(reinterpret_cast<const U1*>(static_cast<const uint8_t*>(t.v) + at));
                decode(qm, qv);
            } else {
                const U4 b = __builtin_nontemporal_load(reinterpret_cast<const U4*>(static_cast<const float*>(t.m) + at));
                const U4 c = __builtin_nontemporal_load(reinterpret_cast<const U4*>(static_cast<const float*>(t.v) + at));
#pragma unroll
                for (int e = 0; e < kLane; ++e) { m[e] = __uint_as_float(b[e]); v[e] = __uint_as_float(c[e]); }
            }
        } else {
            uint32_t qm = 0, qv = 0;
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
            if constexpr (EIGHT) decode(qm, qv);
        }
        if constexpr (EIGHT) {
            const int64_t block = at / kAdamwBlock;
            ms = nv > 0 ? t.m_scale[block] : 0.f;
            vs = nv > 0 ? t.v_scale[block] : 0.f;
        }
    }

    __device__ __forceinline__ void decode(uint32_t qm, uint32_t qv) {
        const f32x2 m0 = __builtin_amdgcn_cvt_pk_f32_fp8(qm, false), m1 = __builtin_amdgcn_cvt_pk_f32_fp8(qm, true);
        const f32x2 v0 = __builtin_amdgcn_cvt_pk_f32_fp8(qv, false), v1 = __builtin_amdgcn_cvt_pk_f32_fp8(qv, true);
        m[0] = m0[0]; m[1] = m0[1]; m[2] = m1[0]; m[3] = m1[1];
        v[0] = v0[0]; v[1] = v0[1]; v[2] = v1[0]; v[3] = v1[1];
    }

    // p, and m and v (8 bits: r in v) after the step
    __device__ __forceinline__ void update(const Step& s) {
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
            float m0 = m[e], v0 = v[e];
            if constexpr (EIGHT) {
                m0 *= ms;
                v0 *= vs;
                v0 *= v0;
            }
            const float grad = g[e] * s.grad_scale;
            m[e] = fmaf(s.b1, m0, s.rest1 * grad);
            const float v1 = fmaf(s.b2, v0, s.rest2 * grad * grad);
            const float r = __builtin_amdgcn_sqrtf(v1);
            v[e] = EIGHT ? r : v1;
            const float step = m[e] * s.c1 * __builtin_amdgcn_rcpf(fmaf(r, s.c2, s.eps));
            p[e] -= fmaf(s.lr * s.decay, p[e], step);
        }
    }

    // all of a wave's lanes, nv of the elements of each
    __device__ __forceinline__ void store(const gdn_adamw_tensor& t, const Step& s, int64_t at, int nv, int lane) {
        uint32_t qm = 0, qv = 0;
        if constexpr (EIGHT) {
            float tm = 0.f, tv = 0.f;
#pragma unroll
            for (int e = 0; e < kLane; ++e)
                if (FULL || e < nv) { tm = fmaxf(tm, fabsf(m[e])); tv = fmaxf(tv, v[e]); }
            tm = wave_max(tm);
            tv = wave_max(tv);
            // (next to nothing counts as nothing: 448 / 2^-100 is finite)
            const float um = tm < 0x1p-100f ? 0.f : 448.f / tm, uv = tv < 0x1p-100f ? 0.f : 448.f / tv;
            if (lane == 0) {
                t.m_scale[at / kAdamwBlock] = um > 0.f ? tm * (1.f / 448.f) : 0.f;
                t.v_scale[at / kAdamwBlock] = uv > 0.f ? tv * (1.f / 448.f) : 0.f;
            }
            const uint32_t high = mix(static_cast<uint32_t>(static_cast<uint64_t>(at) >> 32));   // (0 for 0)
#pragma unroll
            for (int e = 0; e < kLane; ++e) {
                const uint32_t h = mix(s.key + high + static_cast<uint32_t>(at + e) * 0x9E3779B1u);
                qm |= e4m3(m[e] * um, h & 0xFFFFu) << (8 * e);
                const uint32_t r = e4m3(v[e] * uv, h >> 16);
                qv |= (r == 0 && v[e] > 0.f && uv > 0.f ? 1u : r) << (8 * e);
            }
        }
        if constexpr (FULL) {
            const U4 a = {__float_as_uint(p[0]), __float_as_uint(p[1]), __float_as_uint(p[2]), __float_as_uint(p[3])};
            __builtin_nontemporal_store(a, reinterpret_cast<U4*>(t.param + at));
            if (t.copy) {
                const f32x2 lo = {p[0], p[1]}, hi = {p[2], p[3]};
                const U2 c = {__builtin_bit_cast(uint32_t, __builtin_convertvector(lo, bf16x2)),
                              __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, bf16x2))};
                __builtin_nontemporal_store(c, reinterpret_cast<U2*>(static_cast<uint16_t*>(t.copy) + at));
            }
            if constexpr (EIGHT) {
                __builtin_nontemporal_store(qm, reinterpret_cast<U1*>(static_cast<uint8_t*>(t.m) + at));
                __builtin_nontemporal_store(qv, reinterpret_cast<U1*>(static_cast<uint8_t*>(t.v) + at));
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
                t.param[at + e] = p[e];
                if (t.copy) static_cast<uint16_t*>(t.copy)[at + e] = f32_to_bf16_bits(p[e]);
                if constexpr (EIGHT) {
                    static_cast<uint8_t*>(t.m)[at + e] = static_cast<uint8_t>(qm >> (8 * e));
                    static_cast<uint8_t*>(t.v)[at + e] = static_cast<uint8_t>(qv >> (8 * e));
                } else {
                    static_cast<float*>(t.m)[at + e] = m[e];
                    static_cast<float*>(t.v)[at + e] = v[e];
                }
            }
        }
    }
};

template <bool EIGHT, bool GB>
__device__ __forceinline__ void chunk(const gdn_adamw_tensor& t, const Step& s, int64_t base) {
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    // a wave's blocks follow one another
    const int64_t at0 = base + static_cast<int64_t>(wave) * kRounds * kAdamwBlock + kLane * lane;
    if (base + kChunk <= t.n) {
        Elements<EIGHT, GB, true> x[kRounds];
#pragma unroll
        for (int i = 0; i < kRounds; ++i) x[i].load(t, at0 + i * kAdamwBlock, kLane);
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            x[i].update(s);
            x[i].store(t, s, at0 + i * kAdamwBlock, kLane, lane);
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
        x.store(t, s, at, nv, lane);
    }
}

template <bool EIGHT>
__global__ __launch_bounds__(kThreads) void adamw_kernel(Launch a) {
    const AdamwParams& p = a.p;
    // the gradients' factor decides whether there is a step at all
    const float gs = p.grad_scale ? *p.grad_scale : 1.f;
    if (!(fabsf(gs) <= 3.402823466e38f)) return;
    const int64_t b = blockIdx.x;
    int i = 0;
    for (int step = kAdamwTensors / 2; step > 0; step /= 2)
        if (i + step < a.count && b >= a.first[i + step]) i += step;
    const gdn_adamw_tensor t = a.t[i];
    Step s;
    int32_t k = p.step_ptr ? *p.step_ptr : p.step;
    k = k < 1 ? 1 : k;
    s.lr = p.lr_ptr ? *p.lr_ptr : p.lr;
    s.b1 = p.beta1;
    s.b2 = p.beta2;
    s.rest1 = p.rest1;
    s.rest2 = p.rest2;
    s.eps = p.eps;
    s.decay = t.weight_decay;
    s.grad_scale = gs;
    // 1 - b^k = -expm1(k ln b): no cancellation where b^k is next to one
    s.c1 = s.lr / -expm1f(static_cast<float>(k) * p.log_beta1);
    s.c2 = 1.f / sqrtf(-expm1f(static_cast<float>(k) * p.log_beta2));
    s.key = mix(mix(p.seed + static_cast<uint32_t>(k) * 0x9E3779B1u) + static_cast<uint32_t>(a.index[i]) * 0x9E3779B1u);
    const int64_t base = (b - a.first[i]) * kChunk;
    if (t.grad_dtype == GDN_DTYPE_BF16) chunk<EIGHT, true>(t, s, base);
    else chunk<EIGHT, false>(t, s, base);
}

}  // namespace

int64_t adamw_chunks(int64_t n) { return (n + kChunk - 1) / kChunk; }

hipError_t launch_adamw(const AdamwParams& p, const gdn_adamw_tensor* tensors, int count, bool eight, hipStream_t s) {
    for (int i = 0; i < count;) {
        Launch a;
        a.p = p;
        a.count = 0;
        a.first[0] = 0;
        for (; i < count && a.count < kAdamwTensors; ++i) {
            if (tensors[i].n <= 0) continue;
            const int64_t chunks = adamw_chunks(tensors[i].n);
            if (a.count > 0 && a.first[a.count] + chunks > kAdamwMostChunks) break;
            a.t[a.count] = tensors[i];
            a.index[a.count] = i;
            a.first[a.count + 1] = a.first[a.count] + chunks;
            ++a.count;
        }
        if (a.count == 0) break;
        const dim3 grid(static_cast<unsigned>(a.first[a.count]));
        if (eight) hipLaunchKernelGGL(adamw_kernel<true>, grid, dim3(kThreads), 0, s, a);
        else hipLaunchKernelGGL(adamw_kernel<false>, grid, dim3(kThreads), 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace gdn
