// gdn_recur.hip -- the diagonal gated recurrence: forward over packed
// sequences, backward, and one token per sequence.
//
// Per sequence and channel (fp32 inside, whatever the activations' type):
//   v = a + dt_bias, g = -exp(A_log) softplus(v), alpha = e^g,
//   w = sqrt(1 - alpha^2), beta = sigmoid(b), u = w beta x,
//   h_t = alpha_t h_{t-1} + u_t,   y_t = h_t silu(z_t)   (no z: y_t = h_t)
// and for the gradient, with G_t = dL/dh_t and c_t = alpha_t G_t:
//   G_t = dy_t silu(z_t) + c_{t+1},   c_t = alpha_t c_{t+1} + alpha_t dy_t silu(z_t)
//   dx = G w beta, db = G w x beta (1 - beta), dz = dy h silu'(z),
//   dg = alpha G (h_{t-1} - beta x alpha / w), da = -dg exp(A_log) sigmoid(v).
// Both directions are first-order recurrences of the form s <- A s + H, and
// such steps compose: (A2, H2) after (A1, H1) is (A2 A1, A2 H1 + H2).
//
// Bound: HBM.  The forward pass has to read x, a, b, z and write y (10 bytes
// an element in bf16), the backward pass to read those and dy and to write
// four gradients (18 bytes); the arithmetic is about 80 vector operations an
// element forward.  So every input is read once: a work-group owns a tile of
// rows (tokens) x 64 channels, keeps its decays and inputs in registers,
// composes them into the tile's (A, H), publishes that, takes the state
// before the tile from the tiles before it, and runs its rows from there.
//
// The state before a tile: every tile publishes one 64-bit word per channel,
// first its (A, H), then, once it knows its own start, the state after it.
// A tile looks back over its predecessors' words to the nearest one that
// holds a state and applies the (A, H) words after that in order.  A state
// after a tile is always fma(A, state before it, H), whichever word it was
// taken from, so the bits do not depend on timing, on the batch or on how
// many tiles run at once.  Work-groups draw their tile from a counter per
// channel group when they start, so the tiles a work-group can wait for
// belong to work-groups that already run and publish without waiting for a
// later one: every wait ends.
#include "gdn_device.hpp"
#include "gdn_kernels.hpp"

namespace gdn {

namespace {

constexpr int kRT = 512;                          // threads of a tile work-group
constexpr int kRWaves = kRT / kWave;
constexpr int kCh = kRecurChannels;               // channels of a tile
constexpr int kVC = 4;                            // adjacent channels per lane
constexpr int kChLanes = kCh / kVC;               // 16 lanes side by side
constexpr int kGroups = kRT / kChLanes;           // 32 groups of consecutive rows
constexpr int kGroupsPerWave = kWave / kChLanes;  // 4
constexpr int kFwdRows = kRecurUnit / kGroups;    // rows per lane, forward (8)
constexpr int kBwdTile = kRecurUnit / 2;          // rows of a backward tile
constexpr int kBwdRows = kBwdTile / kGroups;      // rows per lane, backward (4)

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---- words: what a tile publishes per channel ----------------------------
// high half: A (its bits are never negative: A is a product of decays in
// [0, 1], NaN is stored as the positive quiet NaN), kState for a state, or
// kEmpty; low half: H or the state.
constexpr uint32_t kEmpty = 0xFFFFFFFFu, kState = 0xBF800000u;

__device__ __forceinline__ uint64_t pack_word(uint32_t hi, float lo) {
    return (static_cast<uint64_t>(hi) << 32) | __float_as_uint(lo);
}
__device__ __forceinline__ uint64_t step_word(float A, float H) {
    return pack_word(A != A ? 0x7FC00000u : __float_as_uint(A), H);
}
__device__ __forceinline__ void put_word(uint64_t* p, uint64_t w) {
    __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t get_word(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float apply_word(uint64_t w, float s) {
    const uint32_t hi = static_cast<uint32_t>(w >> 32);
    const float lo = __uint_as_float(static_cast<uint32_t>(w));
    return hi == kState ? lo : fmaf(__uint_as_float(hi), s, lo);
}

constexpr int kWindow = 16;                       // words looked at in one go

// The state after the predecessor tile.  Predecessor k (1 = the nearest,
// `depth` = the first tile of the sequence) has its word at w + k * step.
// The first tile of a sequence only ever publishes a state, so the search
// stops there at the latest.  One whole wave, a channel per lane.
__device__ __forceinline__ float look_back(const uint64_t* w, int64_t step, int depth) {
    int far = 0;                                  // predecessors 1 .. far: words seen, no state in some lane
    uint64_t v[kWindow];
    int hit;
    for (;;) {
        const int n = depth - far < kWindow ? depth - far : kWindow;
#pragma unroll
        for (int j = 0; j < kWindow; ++j)
            v[j] = get_word(w + (far + 1 + (j < n ? j : n - 1)) * step);
        hit = -1;
        bool blocked = false;
#pragma unroll
        for (int j = 0; j < kWindow; ++j) {
            if (j < n && hit < 0 && !blocked) {
                const uint32_t hi = static_cast<uint32_t>(v[j] >> 32);
                if (hi == kState) hit = j;
                else if (hi == kEmpty) blocked = true;
            }
        }
        if (__all(hit >= 0)) break;
        if (__any(blocked)) __builtin_amdgcn_s_sleep(1);
        else far += kWindow;
    }
    float s = 0.f;
#pragma unroll
    for (int j = kWindow - 1; j >= 0; --j)
        if (j <= hit) s = apply_word(v[j], s);
    while (far > 0) {                             // nearer windows: multiples of kWindow
#pragma unroll
        for (int j = 0; j < kWindow; ++j) v[j] = get_word(w + (far - j) * step);
#pragma unroll
        for (int j = 0; j < kWindow; ++j) s = apply_word(v[j], s);
        far -= kWindow;
    }
    return s;
}

// ---- four adjacent channels of one row -------------------------------------
template <bool BF16>
struct Quad;
template <>
struct Quad<true> {
    using T = uint16_t;
    uint32_t lo, hi;
    // rows and tensors are element aligned only (packed projections of any width)
    struct __attribute__((packed, aligned(2))) Mem { uint32_t lo, hi; };
    __device__ __forceinline__ static Quad load(const T* p) {
        const Mem m = *reinterpret_cast<const Mem*>(p);
        return Quad{m.lo, m.hi};
    }
    __device__ __forceinline__ static Quad load(const T* p, int nv) {
        uint32_t e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = j < nv ? p[j] : 0u;
        return Quad{e[0] | (e[1] << 16), e[2] | (e[3] << 16)};
    }
    __device__ __forceinline__ float get(int j) const {
        const uint32_t v = j < 2 ? lo : hi;
        return __uint_as_float(j & 1 ? v & 0xFFFF0000u : v << 16);
    }
    __device__ __forceinline__ static void store(T* p, const float* f, int nv) {
        if (nv == 4) {
            const f32x2 a = {f[0], f[1]}, b = {f[2], f[3]};
            Mem m;
            m.lo = __builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf16x2));
            m.hi = __builtin_bit_cast(uint32_t, __builtin_convertvector(b, bf16x2));
            *reinterpret_cast<Mem*>(p) = m;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < nv) p[j] = f32_to_bf16_bits(f[j]);
        }
    }
};
template <>
struct Quad<false> {
    using T = float;
    float e[4];
    struct __attribute__((packed, aligned(4))) Mem { float e[4]; };
    __device__ __forceinline__ static Quad load(const T* p) {
        const Mem m = *reinterpret_cast<const Mem*>(p);
        return Quad{{m.e[0], m.e[1], m.e[2], m.e[3]}};
    }
    __device__ __forceinline__ static Quad load(const T* p, int nv) {
        Quad q;
#pragma unroll
        for (int j = 0; j < 4; ++j) q.e[j] = j < nv ? p[j] : 0.f;
        return q;
    }
    __device__ __forceinline__ float get(int j) const { return e[j]; }
    __device__ __forceinline__ static void store(T* p, const float* f, int nv) {
        if (nv == 4) {
            Mem m;
#pragma unroll
            for (int j = 0; j < 4; ++j) m.e[j] = f[j];
            *reinterpret_cast<Mem*>(p) = m;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < nv) p[j] = f[j];
        }
    }
};

// ---- the gates -------------------------------------------------------------
// log(1 + e) / e on [0, 1], degree 9 (interpolated at the Chebyshev points;
// relative error below 1.3e-8): a polynomial costs less than the hardware
// log and the division that keeps its small values exact.
__device__ __forceinline__ float log1p_unit(float e) {
    float p = -3.176057013e-03f;
    p = fmaf(p, e, 1.954252832e-02f);
    p = fmaf(p, e, -5.637361482e-02f);
    p = fmaf(p, e, 1.054362357e-01f);
    p = fmaf(p, e, -1.526966691e-01f);
    p = fmaf(p, e, 1.966327429e-01f);
    p = fmaf(p, e, -2.495161593e-01f);
    p = fmaf(p, e, 3.332971036e-01f);
    p = fmaf(p, e, -4.999989271e-01f);
    p = fmaf(p, e, 1.0f);
    return p * e;
}

__device__ __forceinline__ float sigmoid_fast(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// rate2 = exp(A_log) log2(e).  g2 = g log2(e) = -rate2 softplus(v); alpha =
// 2^g2; q = 1 - alpha^2 = -expm1(2 g), by its series near 0 (seven terms at
// |2 g| < 0.35: relative error below 2e-8) so that slow channels keep it.
struct Gate {
    float g2, alpha, q;
};
__device__ __forceinline__ Gate gate(float v, float rate2) {
    const float e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(v));
    const float s = fmaxf(v, 0.f) + log1p_unit(e);
    Gate r;
    r.g2 = -rate2 * s;
    r.alpha = __builtin_amdgcn_exp2f(r.g2);
    const float t = r.g2 * (2.f * kLn2);          // 2 g
    float p = 1.f / 5040.f;
    p = fmaf(p, t, 1.f / 720.f);
    p = fmaf(p, t, 1.f / 120.f);
    p = fmaf(p, t, 1.f / 24.f);
    p = fmaf(p, t, 1.f / 6.f);
    p = fmaf(p, t, 0.5f);
    p = fmaf(p, t, 1.f);
    r.q = t > -0.35f ? -t * p : fmaf(-r.alpha, r.alpha, 1.f);
    return r;
}

// ---- where a tile lies -----------------------------------------------------
struct Place {
    int seq;
    int unit;                                     // unit of the sequence (kRecurUnit rows)
    int units;                                    // of the sequence, >= 1 (an empty one has one without rows)
    int64_t row0;                                 // first row of the unit
    int rows;                                     // rows of the unit
};

__device__ __forceinline__ int units_of(int len) { return len > 0 ? (len + kRecurUnit - 1) / kRecurUnit : 1; }

__device__ __forceinline__ Place place_of(int lo, int len, int seq, int unit) {
    Place pl;
    pl.seq = seq;
    pl.unit = unit;
    pl.units = units_of(len);
    pl.row0 = static_cast<int64_t>(lo) + static_cast<int64_t>(unit) * kRecurUnit;
    const int left = len - unit * kRecurUnit;
    pl.rows = left < kRecurUnit ? left : kRecurUnit;
    return pl;
}

struct Lane {
    int wave, lane, cl, rg, nv;                   // cl: lane along the channels; rg: row group of the tile
    int c;                                        // first channel
};
__device__ __forceinline__ Lane lane_of(int c0, int D) {
    Lane l;
    l.wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    l.lane = threadIdx.x % kWave;
    l.cl = l.lane % kChLanes;
    l.rg = threadIdx.x / kChLanes;
    l.c = c0 + l.cl * kVC;
    const int left = D - l.c;
    l.nv = left < 0 ? 0 : (left < kVC ? left : kVC);
    return l;
}

// Inclusive (A, H) over the wave's four row groups up to this lane's, in
// row order (REV: from the last group down to this one).
template <bool REV>
__device__ __forceinline__ void wave_compose(const Lane& l, float* A, float* H) {
    const int g = l.lane / kChLanes, at = REV ? kGroupsPerWave - 1 - g : g;
#pragma unroll
    for (int d = 1; d < kGroupsPerWave; d *= 2) {
        const int from = REV ? l.lane + d * kChLanes : l.lane - d * kChLanes;
#pragma unroll
        for (int j = 0; j < kVC; ++j) {
            const float a = __shfl(A[j], from & (kWave - 1), kWave), h = __shfl(H[j], from & (kWave - 1), kWave);
            if (at >= d) {
                H[j] = fmaf(A[j], h, H[j]);
                A[j] *= a;
            }
        }
    }
}

// This lane's start: `s` through the inclusive (A, H) of the group before
// it in the wave.
template <bool REV>
__device__ __forceinline__ void wave_start(const Lane& l, const float* A, const float* H, float* s) {
    const int g = l.lane / kChLanes, at = REV ? kGroupsPerWave - 1 - g : g;
    const int from = (REV ? l.lane + kChLanes : l.lane - kChLanes) & (kWave - 1);
#pragma unroll
    for (int j = 0; j < kVC; ++j) {
        const float a = __shfl(A[j], from, kWave), h = __shfl(H[j], from, kWave);
        if (at > 0) s[j] = fmaf(a, s[j], h);
    }
}

// ---- forward ---------------------------------------------------------------
struct FwdShared {
    float2 step[kRWaves][kCh];                    // (A, H) of a wave's rows
    float start[kCh];                             // state before the tile
    int tile;
};

template <bool BF16, bool GATE>
struct FwdTile {
    using Q = Quad<BF16>;
    using T = typename Q::T;
    float al[kFwdRows][kVC], u[kFwdRows][kVC];
    Q z[kFwdRows];
    float A[kVC], H[kVC];                         // inclusive over the wave's groups

    // Reads the tile's rows, and composes them up to this lane.  Rows past
    // the unit's end read its last row and act as (A, H) = (1, 0).
    __device__ __forceinline__ void load(const RecurParams& p, const Place& pl, const Lane& l, const float* rate2,
                                         const float* bias, bool whole) {
        const int r0 = l.rg * kFwdRows;
        Q x[kFwdRows], a[kFwdRows], b[kFwdRows];
        auto fetch = [&](auto take) {
#pragma unroll
            for (int i = 0; i < kFwdRows; ++i) {
                const int r = r0 + i < pl.rows ? r0 + i : pl.rows - 1;
                const int64_t row = pl.row0 + r;
                a[i] = take(static_cast<const T*>(p.a) + row * p.as + l.c);
                b[i] = take(static_cast<const T*>(p.b) + row * p.bs + l.c);
                x[i] = take(static_cast<const T*>(p.x) + row * p.xs + l.c);
            }
            if constexpr (GATE) {
#pragma unroll
                for (int i = 0; i < kFwdRows; ++i) {
                    const int r = r0 + i < pl.rows ? r0 + i : pl.rows - 1;
                    z[i] = take(static_cast<const T*>(p.z) + (pl.row0 + r) * p.zs + l.c);
                }
            }
        };
        if (whole) fetch([](const T* q) { return Q::load(q); });
        else fetch([&](const T* q) { return Q::load(q, l.nv); });
#pragma unroll
        for (int j = 0; j < kVC; ++j) { A[j] = 1.f; H[j] = 0.f; }
#pragma unroll
        for (int i = 0; i < kFwdRows; ++i) {
            const bool on = r0 + i < pl.rows;
#pragma unroll
            for (int j = 0; j < kVC; ++j) {
                const Gate g = gate(a[i].get(j) + bias[j], rate2[j]);
                const float v = __builtin_amdgcn_sqrtf(g.q) * sigmoid_fast(b[i].get(j)) * x[i].get(j);
                al[i][j] = on ? g.alpha : 1.f;
                u[i][j] = on ? v : 0.f;
                H[j] = fmaf(al[i][j], H[j], u[i][j]);
                A[j] *= al[i][j];
            }
        }
        wave_compose<false>(l, A, H);
    }

    __device__ __forceinline__ void publish(FwdShared& sh, const Lane& l) {
        if (l.lane / kChLanes == kGroupsPerWave - 1) {
#pragma unroll
            for (int j = 0; j < kVC; ++j) sh.step[l.wave][l.cl * kVC + j] = make_float2(A[j], H[j]);
        }
    }

    // The rows from the state before the tile (sh.start) to the outputs.
    __device__ __forceinline__ void finish(const RecurParams& p, const FwdShared& sh, const Place& pl, const Lane& l,
                                           int64_t unit_index) {
        float s[kVC];
#pragma unroll
        for (int j = 0; j < kVC; ++j) s[j] = sh.start[l.cl * kVC + j];
        for (int w = 0; w < l.wave; ++w) {
#pragma unroll
            for (int j = 0; j < kVC; ++j) {
                const float2 e = sh.step[w][l.cl * kVC + j];
                s[j] = fmaf(e.x, s[j], e.y);
            }
        }
        wave_start<false>(l, A, H, s);
        if (p.saved && l.rg % (kGroups / 2) == 0) {
            float* to = p.saved + (2 * unit_index + l.rg / (kGroups / 2)) * p.D + l.c;
            Quad<false>::store(to, s, l.nv);
        }
        const int r0 = l.rg * kFwdRows;
#pragma unroll
        for (int i = 0; i < kFwdRows; ++i) {
            float o[kVC];
#pragma unroll
            for (int j = 0; j < kVC; ++j) {
                s[j] = fmaf(al[i][j], s[j], u[i][j]);
                o[j] = s[j];
                if constexpr (GATE) {
                    const float zj = z[i].get(j);
                    o[j] *= zj * sigmoid_fast(zj);
                }
            }
            if (r0 + i < pl.rows && l.nv > 0)
                Q::store(static_cast<T*>(p.y) + (pl.row0 + r0 + i) * p.ys + l.c, o, l.nv);
        }
    }
};

__device__ __forceinline__ void load_params(const RecurParams& p, const Lane& l, float* rate2, float* bias) {
#pragma unroll
    for (int j = 0; j < kVC; ++j) {
        rate2[j] = j < l.nv ? expf(p.A_log[l.c + j]) * kLog2e : 0.f;
        bias[j] = j < l.nv ? p.dt_bias[l.c + j] : 0.f;
    }
}

// (A, H) of a whole tile, for channel `lane`
__device__ __forceinline__ float2 tile_step(const float2 (*step)[kCh], int lane, bool rev) {
    float A = 1.f, H = 0.f;
#pragma unroll
    for (int w = 0; w < kRWaves; ++w) {
        const float2 e = step[rev ? kRWaves - 1 - w : w][lane];
        H = fmaf(e.x, H, e.y);
        A *= e.x;
    }
    return make_float2(A, H);
}

// grid: channel groups x the bound on units
template <bool BF16, bool GATE>
__global__ __launch_bounds__(kRT, 2) void recur_forward_kernel(RecurParams p) {
    __shared__ FwdShared sh;
    const int total = p.unit_off[p.N];
    const int cg = blockIdx.x % p.groups;
    if (threadIdx.x == 0)
        sh.tile = static_cast<int>(__hip_atomic_fetch_add(p.tickets + cg, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    const int c0 = cg * kCh;
    const Lane l = lane_of(c0, p.D);
    float rate2[kVC], bias[kVC];
    load_params(p, l, rate2, bias);
    __syncthreads();
    const int tile = __builtin_amdgcn_readfirstlane(sh.tile);
    if (tile >= total) return;                    // total < 0: the call's indices were rejected
    const int seq = p.unit_seq[tile];
    const int lo = p.cu[seq];
    const Place pl = place_of(lo, p.cu[seq + 1] - lo, seq, tile - p.unit_off[seq]);

    FwdTile<BF16, GATE> t;
    if (pl.rows > 0) {
        t.load(p, pl, l, rate2, bias, c0 + kCh <= p.D);
        t.publish(sh, l);
    }
    __syncthreads();
    if (l.wave == 0) {
        const int c = c0 + l.lane;
        const float2 e = pl.rows > 0 ? tile_step(sh.step, l.lane, false) : make_float2(1.f, 0.f);
        uint64_t* w = p.words + static_cast<int64_t>(tile) * p.groups * kCh + c;
        const bool last = pl.unit + 1 == pl.units;
        float s = 0.f;
        if (pl.unit == 0) {
            if (p.h0 && c < p.D) s = p.h0[static_cast<int64_t>(state_slot(p.slots, seq)) * p.D + c];
        } else {
            if (!last) put_word(w, step_word(e.x, e.y));
            s = look_back(w, -static_cast<int64_t>(p.groups) * kCh, pl.unit);
        }
        const float after = fmaf(e.x, s, e.y);
        if (!last) put_word(w, pack_word(kState, after));
        else if (p.hT && c < p.D) p.hT[static_cast<int64_t>(state_slot(p.slots, seq)) * p.D + c] = pl.rows > 0 ? after : s;
        sh.start[l.lane] = s;
    }
    __syncthreads();
    if (pl.rows > 0) t.finish(p, sh, pl, l, tile);
}

// One work-group per (channel group, sequence) walks the sequence's tiles in
// order: no words, no workspace, one launch.  Same bits: the state after a
// tile is the same fma.
template <bool BF16, bool GATE>
__global__ __launch_bounds__(kRT, 2) void recur_walk_kernel(RecurParams p) {
    __shared__ FwdShared sh;
    __shared__ int bad, first_unit;
    if (threadIdx.x == 0) { bad = 0; first_unit = 0; }
    __syncthreads();
    // every work-group checks the indices, so nothing is written on a bad one
    const int seq = blockIdx.x / p.groups;
    int mine = 0, before = 0;
    for (int n = threadIdx.x; n < p.N; n += kRT) {
        const int lo = p.cu[n], hi = p.cu[n + 1];
        if (hi < lo || (n == 0 && lo != 0) || (n + 1 == p.N && hi != p.T)) mine = 1;
        if (p.slots && (p.slots[n] < 0 || p.slots[n] >= p.num_slots)) mine = 1;
        if (n < seq && hi >= lo) before += units_of(hi - lo);
    }
    if (mine) atomicOr(&bad, 1);
    if (p.saved && before) atomicAdd(&first_unit, before);
    __syncthreads();
    if (p.status && blockIdx.x == 0 && threadIdx.x == 0) *p.status = bad ? kStatusBadIndex : 0;
    if (bad) return;
    const int cg = blockIdx.x % p.groups;
    const int c0 = cg * kCh;
    const Lane l = lane_of(c0, p.D);
    float rate2[kVC], bias[kVC];
    load_params(p, l, rate2, bias);
    const int lo = p.cu[seq], len = p.cu[seq + 1] - lo;
    const int c = c0 + l.lane;
    const int64_t at = static_cast<int64_t>(state_slot(p.slots, seq)) * p.D + c;
    if (l.wave == 0) sh.start[l.lane] = p.h0 && c < p.D ? p.h0[at] : 0.f;
    FwdTile<BF16, GATE> t;
    const int units = units_of(len);
    for (int k = 0; k < units && len > 0; ++k) {
        const Place pl = place_of(lo, len, seq, k);
        t.load(p, pl, l, rate2, bias, c0 + kCh <= p.D);
        t.publish(sh, l);
        __syncthreads();
        t.finish(p, sh, pl, l, static_cast<int64_t>(first_unit) + k);
        float after = 0.f;
        if (l.wave == 0) {
            const float2 e = tile_step(sh.step, l.lane, false);
            after = fmaf(e.x, sh.start[l.lane], e.y);
        }
        __syncthreads();
        if (l.wave == 0) sh.start[l.lane] = after;
    }
    if (l.wave == 0 && p.hT && c < p.D) p.hT[at] = sh.start[l.lane];
}

// Block 0 checks the indices and lays out the units (unit_off, unit_seq);
// the others, and block 0 after that, set the words to kEmpty and the
// tickets to 0.
constexpr int kPlanThreads = 1024;

__global__ __launch_bounds__(kPlanThreads) void recur_plan_kernel(RecurParams p) {
    const int tid = threadIdx.x;
    const int64_t nwords = static_cast<int64_t>(p.tiles) * p.groups * kCh;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kPlanThreads;
    uint2* words = reinterpret_cast<uint2*>(p.words);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid; i < nwords; i += stride)
        words[i] = make_uint2(kEmpty, kEmpty);
    if (blockIdx.x != 0) return;
    for (int i = tid; i < p.groups; i += kPlanThreads) p.tickets[i] = 0;
    __shared__ int part[kPlanThreads];
    __shared__ int bad;
    if (tid == 0) bad = 0;
    __syncthreads();
    const int per = (p.N + kPlanThreads - 1) / kPlanThreads;
    const int n0 = tid * per < p.N ? tid * per : p.N, n1 = n0 + per < p.N ? n0 + per : p.N;
    int sum = 0, mine = 0;
    for (int n = n0; n < n1; ++n) {
        const int lo = p.cu[n], hi = p.cu[n + 1];
        if (hi < lo || lo < 0 || hi > p.T || (n == 0 && lo != 0) || (n + 1 == p.N && hi != p.T)) mine = 1;
        else sum += units_of(hi - lo);
        if (p.slots && (p.slots[n] < 0 || p.slots[n] >= p.num_slots)) mine = 1;
    }
    if (mine) atomicOr(&bad, 1);
    part[tid] = sum;
    __syncthreads();
    for (int d = 1; d < kPlanThreads; d *= 2) {   // inclusive sums
        const int v = tid >= d ? part[tid - d] : 0;
        __syncthreads();
        part[tid] += v;
        __syncthreads();
    }
    if (bad) {
        if (tid == 0) p.unit_off[p.N] = -1;
    } else {
        int at = part[tid] - sum;
        for (int n = n0; n < n1; ++n) {
            p.unit_off[n] = at;
            const int k = units_of(p.cu[n + 1] - p.cu[n]);
            for (int i = 0; i < k; ++i) p.unit_seq[at + i] = n;
            at += k;
        }
        if (tid == 0) p.unit_off[p.N] = part[kPlanThreads - 1];
    }
    if (tid == 0 && p.status) *p.status = bad ? kStatusBadIndex : 0;
}

// ---- backward --------------------------------------------------------------
struct BwdShared {
    float2 fwd[kRWaves][kCh], rev[kRWaves][kCh];
    float2 sums[kRWaves][kCh];
    float start[kCh];                             // c past the tile's last row
    int tile;
};

// grid: channel groups x 2 x the bound on units; a tile is half a unit, and
// the tiles of a sequence are taken from its end.  The rows' h are run again
// from the state the forward pass saved at the tile's first row.
template <bool BF16, bool GATE>
__global__ __launch_bounds__(kRT, 2) void recur_backward_kernel(RecurParams p) {
    using Q = Quad<BF16>;
    using T = typename Q::T;
    constexpr int L = kBwdRows;
    __shared__ BwdShared sh;
    const int total = 2 * p.unit_off[p.N];
    const int cg = blockIdx.x % p.groups;
    if (threadIdx.x == 0)
        sh.tile = static_cast<int>(__hip_atomic_fetch_add(p.tickets + cg, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    const int c0 = cg * kCh;
    const Lane l = lane_of(c0, p.D);
    float rate2[kVC], bias[kVC];
    load_params(p, l, rate2, bias);
    __syncthreads();
    const int ticket = __builtin_amdgcn_readfirstlane(sh.tile);
    if (ticket >= total) return;
    const int tile = total - 1 - ticket;
    const int seq = p.unit_seq[tile / 2];
    const int lo = p.cu[seq], len = p.cu[seq + 1] - lo;
    const Place pl = place_of(lo, len, seq, tile / 2 - p.unit_off[seq]);
    const int t0 = (tile % 2) * kBwdTile;         // first row within the unit
    const int left = pl.rows - t0;
    const int rows = left < 0 ? 0 : (left < kBwdTile ? left : kBwdTile);
    const int64_t row0 = pl.row0 + t0;
    const int behind = 2 * pl.units - 1 - (2 * pl.unit + tile % 2);   // tiles of the sequence after this one

    const int r0 = l.rg * L;
    Q x[L], a[L], b[L], z[L], dy[L];
    float al[L][kVC], hp[L][kVC], c[L][kVC];      // alpha, h before the row, alpha dy silu(z)
    float Af[kVC], Hf[kVC], Ar[kVC], Hr[kVC];
    if (rows > 0) {
        auto fetch = [&](auto take) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int64_t row = row0 + (r0 + i < rows ? r0 + i : rows - 1);
                a[i] = take(static_cast<const T*>(p.a) + row * p.as + l.c);
                b[i] = take(static_cast<const T*>(p.b) + row * p.bs + l.c);
                x[i] = take(static_cast<const T*>(p.x) + row * p.xs + l.c);
                dy[i] = take(static_cast<const T*>(p.dy) + row * p.dys + l.c);
                if constexpr (GATE) z[i] = take(static_cast<const T*>(p.z) + row * p.zs + l.c);
            }
        };
        if (c0 + kCh <= p.D) fetch([](const T* q) { return Q::load(q); });
        else fetch([&](const T* q) { return Q::load(q, l.nv); });
#pragma unroll
        for (int j = 0; j < kVC; ++j) { Af[j] = Ar[j] = 1.f; Hf[j] = Hr[j] = 0.f; }
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const bool on = r0 + i < rows;
#pragma unroll
            for (int j = 0; j < kVC; ++j) {
                const Gate g = gate(a[i].get(j) + bias[j], rate2[j]);
                const float u = __builtin_amdgcn_sqrtf(g.q) * sigmoid_fast(b[i].get(j)) * x[i].get(j);
                float e = dy[i].get(j);
                if constexpr (GATE) {
                    const float zj = z[i].get(j);
                    e *= zj * sigmoid_fast(zj);
                }
                al[i][j] = on ? g.alpha : 1.f;
                hp[i][j] = on ? u : 0.f;          // u for now
                c[i][j] = on ? g.alpha * e : 0.f;
                Hf[j] = fmaf(al[i][j], Hf[j], hp[i][j]);
                Af[j] *= al[i][j];
            }
        }
#pragma unroll
        for (int i = L - 1; i >= 0; --i)
#pragma unroll
            for (int j = 0; j < kVC; ++j) {
                Hr[j] = fmaf(al[i][j], Hr[j], c[i][j]);
                Ar[j] *= al[i][j];
            }
        wave_compose<false>(l, Af, Hf);
        wave_compose<true>(l, Ar, Hr);
        if (l.lane / kChLanes == kGroupsPerWave - 1) {
#pragma unroll
            for (int j = 0; j < kVC; ++j) sh.fwd[l.wave][l.cl * kVC + j] = make_float2(Af[j], Hf[j]);
        }
        if (l.lane / kChLanes == 0) {
#pragma unroll
            for (int j = 0; j < kVC; ++j) sh.rev[l.wave][l.cl * kVC + j] = make_float2(Ar[j], Hr[j]);
        }
    }
    __syncthreads();
    if (l.wave == 0) {
        const int ch = c0 + l.lane;
        const float2 e = rows > 0 ? tile_step(sh.rev, l.lane, true) : make_float2(1.f, 0.f);
        uint64_t* w = p.words + static_cast<int64_t>(tile) * p.groups * kCh + ch;
        const bool first = 2 * pl.unit + tile % 2 == 0;
        float s = 0.f;
        if (behind == 0) {
            if (p.dhT && ch < p.D) s = p.dhT[static_cast<int64_t>(seq) * p.D + ch];
        } else {
            if (!first) put_word(w, step_word(e.x, e.y));
            s = look_back(w, static_cast<int64_t>(p.groups) * kCh, behind);
        }
        const float after = fmaf(e.x, s, e.y);
        if (!first) put_word(w, pack_word(kState, after));
        else if (p.dh0 && ch < p.D) p.dh0[static_cast<int64_t>(seq) * p.D + ch] = rows > 0 ? after : s;
        sh.start[l.lane] = s;
    }
    __syncthreads();
    float sa[kVC], sb[kVC];                       // sums of dg g2 and of dg sigmoid(v)
#pragma unroll
    for (int j = 0; j < kVC; ++j) sa[j] = sb[j] = 0.f;
    if (rows > 0) {
        float s[kVC], r[kVC];
        const Quad<false> h = Quad<false>::load(p.saved + static_cast<int64_t>(tile) * p.D + l.c, l.nv);
#pragma unroll
        for (int j = 0; j < kVC; ++j) {
            s[j] = h.get(j);
            r[j] = sh.start[l.cl * kVC + j];
        }
        for (int w = 0; w < l.wave; ++w)
#pragma unroll
            for (int j = 0; j < kVC; ++j) {
                const float2 e = sh.fwd[w][l.cl * kVC + j];
                s[j] = fmaf(e.x, s[j], e.y);
            }
        for (int w = kRWaves - 1; w > l.wave; --w)
#pragma unroll
            for (int j = 0; j < kVC; ++j) {
                const float2 e = sh.rev[w][l.cl * kVC + j];
                r[j] = fmaf(e.x, r[j], e.y);
            }
        wave_start<false>(l, Af, Hf, s);
        wave_start<true>(l, Ar, Hr, r);
#pragma unroll
        for (int i = 0; i < L; ++i)               // hp: from u to the state before the row
#pragma unroll
            for (int j = 0; j < kVC; ++j) {
                const float next = fmaf(al[i][j], s[j], hp[i][j]);
                hp[i][j] = s[j];
                s[j] = next;
            }
#pragma unroll
        for (int i = L - 1; i >= 0; --i) {
            const bool on = r0 + i < rows;
            float dx[kVC], da[kVC], db[kVC], dz[kVC];
#pragma unroll
            for (int j = 0; j < kVC; ++j) {
                const float v = a[i].get(j) + bias[j];
                const Gate g = gate(v, rate2[j]);
                const float w = __builtin_amdgcn_sqrtf(g.q);
                // g -> 0: alpha / w grows as sigmoid(v) falls, their product goes to 0
                const float over = g.q > 0.f ? __builtin_amdgcn_rcpf(w) : 0.f;
                const float beta = sigmoid_fast(b[i].get(j));
                const float xj = x[i].get(j);
                float e = dy[i].get(j);
                if constexpr (GATE) {
                    const float zj = z[i].get(j), q = sigmoid_fast(zj);
                    const float hrow = fmaf(al[i][j], hp[i][j], w * beta * xj);
                    dz[j] = e * hrow * (q * fmaf(zj, 1.f - q, 1.f));
                    e *= zj * q;
                }
                const float G = e + r[j];
                r[j] = fmaf(al[i][j], r[j], c[i][j]);
                const float bx = beta * xj;
                dx[j] = G * w * beta;
                db[j] = G * w * bx * (1.f - beta);
                const float dg = g.alpha * G * (hp[i][j] - bx * g.alpha * over);
                const float ds = dg * sigmoid_fast(v);
                da[j] = -ds * (rate2[j] * kLn2);
                if (on) {
                    sa[j] = fmaf(dg, g.g2, sa[j]);
                    sb[j] += ds;
                }
            }
            if (on && l.nv > 0) {
                const int64_t row = row0 + r0 + i;
                Q::store(static_cast<T*>(p.dx) + row * p.dxs + l.c, dx, l.nv);
                Q::store(static_cast<T*>(p.da) + row * p.das + l.c, da, l.nv);
                Q::store(static_cast<T*>(p.db) + row * p.dbs + l.c, db, l.nv);
                if constexpr (GATE) Q::store(static_cast<T*>(p.dz) + row * p.dzs + l.c, dz, l.nv);
            }
        }
    }
    if (!p.partial) return;
    // the tile's sums over its rows, in a fixed order
#pragma unroll
    for (int j = 0; j < kVC; ++j) {
        sa[j] += __shfl_xor(sa[j], 16, kWave);
        sb[j] += __shfl_xor(sb[j], 16, kWave);
        sa[j] += __shfl_xor(sa[j], 32, kWave);
        sb[j] += __shfl_xor(sb[j], 32, kWave);
    }
    if (l.lane < kChLanes) {
#pragma unroll
        for (int j = 0; j < kVC; ++j) sh.sums[l.wave][l.cl * kVC + j] = make_float2(sa[j], sb[j]);
    }
    __syncthreads();
    if (l.wave == 0) {
        float2 t = sh.sums[0][l.lane];
#pragma unroll
        for (int w = 1; w < kRWaves; ++w) {
            const float2 e = sh.sums[w][l.lane];
            t.x += e.x;
            t.y += e.y;
        }
        p.partial[static_cast<int64_t>(tile) * p.groups * kCh + c0 + l.lane] = t;
    }
}

// dA_log and ddt_bias from the tiles' sums, each channel's tiles in a fixed
// order.  One work-group per channel group: 16 threads a channel.
constexpr int kSumThreads = 1024, kSumSlices = kSumThreads / kCh;

__global__ __launch_bounds__(kSumThreads) void recur_sum_kernel(RecurParams p) {
    const int total = 2 * p.unit_off[p.N];
    if (total < 0) return;
    __shared__ float2 part[kSumSlices][kCh];
    const int ch = threadIdx.x % kCh, sl = threadIdx.x / kCh;
    const int c = blockIdx.x * kCh + ch;
    float2 t = make_float2(0.f, 0.f);
    for (int i = sl; i < total; i += kSumSlices) {
        const float2 e = p.partial[static_cast<int64_t>(i) * p.groups * kCh + c];
        t.x += e.x;
        t.y += e.y;
    }
    part[sl][ch] = t;
    __syncthreads();
    if (sl == 0 && c < p.D) {
#pragma unroll
        for (int s = 1; s < kSumSlices; ++s) {
            t.x += part[s][ch].x;
            t.y += part[s][ch].y;
        }
        if (p.dA_log) p.dA_log[c] = t.x * kLn2;   // g = g2 ln 2
        if (p.ddt_bias) p.ddt_bias[c] = -t.y * expf(p.A_log[c]);
    }
}

// ---- one token per sequence ------------------------------------------------
constexpr int kDecodeThreads = 256;

template <bool BF16, bool GATE>
__global__ __launch_bounds__(kDecodeThreads) void recur_decode_kernel(RecurParams p) {
    using Q = Quad<BF16>;
    using T = typename Q::T;
    const int per = (p.D + kVC - 1) / kVC;        // lanes of a row
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kDecodeThreads + threadIdx.x;
    const int n = static_cast<int>(i / per);
    if (n >= p.N) return;
    const int c = static_cast<int>(i % per) * kVC;
    const int nv = p.D - c < kVC ? p.D - c : kVC;
    const int slot = state_slot(p.slots, n);
    if (p.slots && (slot < 0 || slot >= p.num_slots)) {
        if (p.status && c == 0) __hip_atomic_fetch_or(p.status, kStatusBadIndex, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return;
    }
    auto take = [&](const void* t, int64_t s) {
        const T* q = static_cast<const T*>(t) + n * s + c;
        return nv == kVC ? Q::load(q) : Q::load(q, nv);
    };
    const Q a = take(p.a, p.as), b = take(p.b, p.bs), x = take(p.x, p.xs);
    Q z{};
    if constexpr (GATE) z = take(p.z, p.zs);
    const int64_t at = static_cast<int64_t>(slot) * p.D + c;
    Quad<false> h{};
    if (p.h0) h = nv == kVC ? Quad<false>::load(p.h0 + at) : Quad<false>::load(p.h0 + at, nv);
    float s[kVC], o[kVC];
#pragma unroll
    for (int j = 0; j < kVC; ++j) {
        const float rate2 = j < nv ? expf(p.A_log[c + j]) * kLog2e : 0.f, bias = j < nv ? p.dt_bias[c + j] : 0.f;
        const Gate g = gate(a.get(j) + bias, rate2);
        const float u = __builtin_amdgcn_sqrtf(g.q) * sigmoid_fast(b.get(j)) * x.get(j);
        s[j] = fmaf(g.alpha, h.get(j), u);
        o[j] = s[j];
        if constexpr (GATE) {
            const float zj = z.get(j);
            o[j] *= zj * sigmoid_fast(zj);
        }
    }
    Quad<false>::store(p.hT + at, s, nv);
    Q::store(static_cast<T*>(p.y) + n * p.ys + c, o, nv);
}

__global__ __launch_bounds__(256) void fill_zero_kernel(float* p, int64_t n) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i < n) p[i] = 0.f;
}

}  // namespace

hipError_t launch_fill_zero(float* p, int64_t n, hipStream_t s) {
    if (!p || n <= 0) return hipSuccess;
    hipLaunchKernelGGL(fill_zero_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, s, p, n);
    return hipGetLastError();
}

#define GDN_RECUR_CALL(KERNEL, GRID, BLOCK)                                                  \
    do {                                                                                     \
        const dim3 g_(static_cast<unsigned>(GRID)), b_(BLOCK);                               \
        if (bf16 && p.z) hipLaunchKernelGGL((KERNEL<true, true>), g_, b_, 0, s, p);          \
        else if (bf16) hipLaunchKernelGGL((KERNEL<true, false>), g_, b_, 0, s, p);           \
        else if (p.z) hipLaunchKernelGGL((KERNEL<false, true>), g_, b_, 0, s, p);            \
        else hipLaunchKernelGGL((KERNEL<false, false>), g_, b_, 0, s, p);                    \
    } while (0)

static hipError_t launch_plan(const RecurParams& p, hipStream_t s) {
    const int64_t nwords = static_cast<int64_t>(p.tiles) * p.groups * kCh;
    int64_t blocks = 1 + nwords / (kPlanThreads * 8);
    if (blocks > 1024) blocks = 1024;
    hipLaunchKernelGGL(recur_plan_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kPlanThreads), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_recur_forward(const RecurParams& p, bool bf16, hipStream_t s) {
    if (p.walk) {
        GDN_RECUR_CALL(recur_walk_kernel, static_cast<int64_t>(p.groups) * p.N, kRT);
        return hipGetLastError();
    }
    hipError_t e = launch_plan(p, s);
    if (e != hipSuccess) return e;
    GDN_RECUR_CALL(recur_forward_kernel, static_cast<int64_t>(p.groups) * p.tiles, kRT);
    return hipGetLastError();
}

hipError_t launch_recur_backward(const RecurParams& p, bool bf16, hipStream_t s) {
    hipError_t e = launch_plan(p, s);
    if (e != hipSuccess) return e;
    GDN_RECUR_CALL(recur_backward_kernel, static_cast<int64_t>(p.groups) * p.tiles, kRT);
    e = hipGetLastError();
    if (e != hipSuccess || !p.partial) return e;
    hipLaunchKernelGGL(recur_sum_kernel, dim3(static_cast<unsigned>(p.groups)), dim3(kSumThreads), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_recur_decode(const RecurParams& p, bool bf16, hipStream_t s) {
    const int64_t lanes = static_cast<int64_t>(p.N) * ((p.D + kVC - 1) / kVC);
    GDN_RECUR_CALL(recur_decode_kernel, (lanes + kDecodeThreads - 1) / kDecodeThreads, kDecodeThreads);
    return hipGetLastError();
}

}  // namespace gdn
