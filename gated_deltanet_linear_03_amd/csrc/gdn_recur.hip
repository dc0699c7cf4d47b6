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
// 1 / w grows without end as alpha goes to 1, while sigmoid(v) in da, and g in
// dA_log's dg g, fall with w^2: dg is formed from 1 / w itself, at most 2^63,
// never from 1 / w^2, and where w^2 is below the smallest normal number both w
// and 1 / w count as 0 (what they stand for in a gradient is below 2^-63 of
// its other factors).
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

constexpr int kThreads = 256;                     // of a tile work-group: four waves
constexpr int kWaves = kThreads / kWave;
constexpr int kCh = kRecurChannels;               // channels of a tile
constexpr int kVC = 4;                            // adjacent channels per lane
constexpr int kChLanes = kCh / kVC;               // 16 lanes side by side
constexpr int kGroupsPerWave = kWave / kChLanes;  // 4
constexpr int kGroups = kThreads / kChLanes;      // 16 groups of consecutive rows
constexpr int kFwdRows = kRecurUnit / kGroups;    // rows per lane, forward (8)
constexpr int kBwdTile = kRecurSaved;             // rows of a backward tile
constexpr int kHalves = kRecurUnit / kBwdTile;
constexpr int kBwdRows = kBwdTile / kGroups;      // rows per lane, backward (4)

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// A grid dimension holds fewer than 2^32 work-items, and a launch with more runs
// a part of them without an error: past kGridX work-groups a call goes on in
// the second dimension (the last row of groups may have some with nothing to do).
constexpr int kGridX = 1 << 22;

__device__ __forceinline__ uint32_t group_index() { return blockIdx.y * static_cast<uint32_t>(kGridX) + blockIdx.x; }

dim3 grid_of(int64_t groups) {
    return groups <= kGridX ? dim3(static_cast<unsigned>(groups))
                            : dim3(kGridX, static_cast<unsigned>((groups + kGridX - 1) / kGridX));
}

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

constexpr int kWindow = 4;                        // words looked at in one go (8: 6% slower at 131072 x 2048, whose kernel then takes 136 registers instead of 128)

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

// A row pointer is a wave-uniform address plus a lane's 32-bit byte offset:
// the loads and stores of whole tiles then cost no vector address arithmetic.
template <typename T>
__device__ __forceinline__ const T* lane_ptr(const T* base, uint32_t off) {
    return reinterpret_cast<const T*>(reinterpret_cast<const char*>(base) + off);
}
template <typename T>
__device__ __forceinline__ T* lane_ptr(T* base, uint32_t off) {
    return reinterpret_cast<T*>(reinterpret_cast<char*>(base) + off);
}

// ---- four adjacent channels of one row (ONCE: nothing reads them again soon;
// stores of whole quads are non-temporal too: 131072 x 2048, forward without
// its arithmetic, 587 us with plain accesses, 559 with such stores, 544 with
// both) -------------------------------------
template <bool BF16>
struct Quad;
template <>
struct Quad<true> {
    using T = uint16_t;
    uint32_t lo, hi;
    // rows and tensors are element aligned only (packed projections of any width)
    typedef uint32_t Mem __attribute__((ext_vector_type(2), aligned(2)));
    template <bool ONCE = false>
    __device__ __forceinline__ static Quad load(const T* p) {
        const Mem* q = reinterpret_cast<const Mem*>(p);
        const Mem m = ONCE ? __builtin_nontemporal_load(q) : *q;
        return Quad{m.x, m.y};
    }
    __device__ __forceinline__ static Quad load(const T* p, int nv) {
        uint32_t e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = j < nv ? p[j] : 0u;
        return Quad{e[0] | (e[1] << 16), e[2] | (e[3] << 16)};
    }
    // the value is what it was, but nothing computed from it before is kept for later
    __device__ __forceinline__ void forget() { asm volatile("" : "+v"(lo), "+v"(hi)); }
    __device__ __forceinline__ Quad dropped(int n) const {
        const uint64_t v = n < 4 ? ((static_cast<uint64_t>(hi) << 32) | lo) >> (16 * n) : 0ull;
        return Quad{static_cast<uint32_t>(v), static_cast<uint32_t>(v >> 32)};
    }
    __device__ __forceinline__ float get(int j) const {
        const uint32_t v = j < 2 ? lo : hi;
        return __uint_as_float(j & 1 ? v & 0xFFFF0000u : v << 16);
    }
    __device__ __forceinline__ static void store(T* p, const float* f, int nv) {
        if (nv == 4) {
            const f32x2 a = {f[0], f[1]}, b = {f[2], f[3]};
            const Mem m = {__builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf16x2)),
                           __builtin_bit_cast(uint32_t, __builtin_convertvector(b, bf16x2))};
            __builtin_nontemporal_store(m, reinterpret_cast<Mem*>(p));
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
    typedef float Mem __attribute__((ext_vector_type(4), aligned(4)));
    template <bool ONCE = false>
    __device__ __forceinline__ static Quad load(const T* p) {
        const Mem* q = reinterpret_cast<const Mem*>(p);
        const Mem m = ONCE ? __builtin_nontemporal_load(q) : *q;
        return Quad{{m.x, m.y, m.z, m.w}};
    }
    __device__ __forceinline__ static Quad load(const T* p, int nv) {
        Quad q;
#pragma unroll
        for (int j = 0; j < 4; ++j) q.e[j] = j < nv ? p[j] : 0.f;
        return q;
    }
    __device__ __forceinline__ void forget() { asm volatile("" : "+v"(e[0]), "+v"(e[1]), "+v"(e[2]), "+v"(e[3])); }
    __device__ __forceinline__ Quad dropped(int n) const {
        return n == 0 ? *this : n == 1 ? Quad{{e[1], e[2], e[3], 0.f}} : n == 2 ? Quad{{e[2], e[3], 0.f, 0.f}}
                      : n == 3 ? Quad{{e[3], 0.f, 0.f, 0.f}} : Quad{{0.f, 0.f, 0.f, 0.f}};
    }
    __device__ __forceinline__ float get(int j) const { return e[j]; }
    __device__ __forceinline__ static void store(T* p, const float* f, int nv) {
        if (nv == 4) {
            const Mem m = {f[0], f[1], f[2], f[3]};
            __builtin_nontemporal_store(m, reinterpret_cast<Mem*>(p));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < nv) p[j] = f[j];
        }
    }
};

// ---- the gates -------------------------------------------------------------
// log(1 + e) on [0, 1] as e times a polynomial of degree 8 (log(1 + e) / e
// interpolated at the Chebyshev points; relative error below 1e-7): it costs
// less than the hardware log with the correction that keeps small values
// exact.
__device__ __forceinline__ float log1p_unit_over(float e) {
    float p = 5.126101896e-03f;
    p = fmaf(p, e, -2.907406539e-02f);
    p = fmaf(p, e, 7.751608640e-02f);
    p = fmaf(p, e, -1.360224783e-01f);
    p = fmaf(p, e, 1.907688081e-01f);
    p = fmaf(p, e, -2.483539879e-01f);
    p = fmaf(p, e, 3.331812024e-01f);
    p = fmaf(p, e, -4.999944568e-01f);
    return fmaf(p, e, 9.999999404e-01f);
}

__device__ __forceinline__ float sigmoid_fast(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// nrate2 = -exp(A_log) log2(e).  g2 = g log2(e) = nrate2 softplus(v); alpha =
// 2^g2; q = 1 - alpha^2 = -expm1(2 g), near 0 from expm1(t) / t (degree 4,
// relative error below 3e-8 on [-0.35, 0]) so that slow channels keep it.
struct Gate {
    float e;                                      // e^-|v|
    float g2, alpha, q;
};
__device__ __forceinline__ Gate gate(float v, float nrate2) {
    Gate r;
    r.e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(v));
    r.g2 = nrate2 * fmaf(log1p_unit_over(r.e), r.e, fmaxf(v, 0.f));
    r.alpha = __builtin_amdgcn_exp2f(r.g2);
    const float t = r.g2 * (2.f * kLn2);          // 2 g
    float p = 7.211245596e-03f;
    p = fmaf(p, t, 4.133187234e-02f);
    p = fmaf(p, t, 1.666253060e-01f);
    p = fmaf(p, t, 4.999982119e-01f);
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

// How much of a tile exists: all of it; all rows but not all channels (the
// last group: still one load per four channels, from addresses moved back
// into the row); or fewer rows, with every row's address clamped by itself.
// 9001 rows of 1023 fp32 channels, rows 1023 apart, take 55 us with kEdge and
// 66 us with the clamped form for the last group; 1024 channels take 47.
enum Part { kWhole, kEdge, kSome };
__device__ __forceinline__ Part part_of(bool rows, int c0, int D) {
    return !rows || D < kVC ? kSome : c0 + kCh <= D ? kWhole : kEdge;
}

struct Lane {
    int wave, lane, cl, rg, nv;                   // cl: lane along the channels; rg: row group of the tile
    int c;                                        // first channel
    int lc, drop;                                 // quads of a row that ends inside: read at lc, drop the first elements
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
    l.lc = left < kVC ? D - kVC : l.c;            // (D < kVC: read element by element)
    l.drop = kVC - l.nv;
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
__device__ __forceinline__ void wave_start(const Lane& l, const float* A, const float* H, float* s) {
    const int from = (l.lane - kChLanes) & (kWave - 1);
#pragma unroll
    for (int j = 0; j < kVC; ++j) {
        const float a = __shfl(A[j], from, kWave), h = __shfl(H[j], from, kWave);
        if (l.lane >= kChLanes) s[j] = fmaf(a, s[j], h);
    }
}

// Four channels of a row in a tile that may end inside them: one load for
// any width from kVC up.
template <typename Q>
__device__ __forceinline__ Q load_edge(const typename Q::T* row, const Lane& l, int D) {
    if (D >= kVC) return Q::load(row + l.lc).dropped(l.drop);
    const Q q = Q::load(row + l.c, l.nv);
    __builtin_amdgcn_sched_barrier(0);            // row by row: the elements' registers are not kept for all rows
    return q;
}

// Rows r0 .. r0 + ROWS - 1 of a tile of `rows` rows at `base`; those past the
// end read the last one.
// FAST: one address and offsets of 32 bits.  It takes registers from the whole
// tiles of the kernel that it is compiled into (166 instead of 128): forward
// without saved states, 131072 x 2048 in one sequence 646 us (618 without FAST),
// 60000 x 1024 in 600 sequences 205 us (296).
template <typename Q, int ROWS, bool ONCE, bool FAST>
__device__ __forceinline__ void load_some(Q* to, const typename Q::T* base, int64_t stride, int r0, int rows, const Lane& l, int D) {
    const int at = r0 < rows ? r0 : rows - 1, more = rows - 1 - at;
    if (FAST && D >= kVC) {
        const uint32_t ld = static_cast<uint32_t>(stride), off = static_cast<uint32_t>(at) * ld + l.lc;
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            to[i] = Q::template load<ONCE>(
                lane_ptr(base, (off + __umul24(i < more ? i : more, ld)) * static_cast<uint32_t>(sizeof(typename Q::T))));
#pragma unroll
        for (int i = 0; i < ROWS; ++i) to[i] = to[i].dropped(l.drop);
    } else {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) to[i] = load_edge<Q>(base + (r0 + i < rows ? r0 + i : rows - 1) * stride, l, D);
    }
}

// ---- forward ---------------------------------------------------------------
struct FwdShared {
    float2 step[kWaves][kCh];                  // (A, H) of a wave's rows
    float start[kCh];                             // state before the tile
    int tile;
};

// KEEP: the inputs are read again by a backward pass; FAST: see load_some
template <bool BF16, bool GATE, bool KEEP, bool FAST>
struct FwdTile {
    using Q = Quad<BF16>;
    using T = typename Q::T;
    float al[kFwdRows][kVC], u[kFwdRows][kVC];
    Q z[kFwdRows];
    float A[kVC], H[kVC];                         // inclusive over the wave's groups

    // Reads the tile's rows and composes them up to this lane.  Rows past the
    // unit's end read its last row and act as (A, H) = (1, 0).
    template <Part PART>
    __device__ __forceinline__ void load(const RecurParams& p, const Place& pl, const Lane& l, const float* nrate2,
                                         const float* bias) {
        const int r0 = l.rg * kFwdRows;
        Q x[kFwdRows], a[kFwdRows], b[kFwdRows];
        auto fetch = [&](Q* to, const void* from, int64_t stride) {
            if constexpr (PART != kSome) {
                const T* base = static_cast<const T*>(from) + pl.row0 * stride;
                const uint32_t off = (static_cast<uint32_t>(r0) * static_cast<uint32_t>(stride) + (PART == kEdge ? l.lc : l.c)) * sizeof(T);
#pragma unroll
                for (int i = 0; i < kFwdRows; ++i) to[i] = Q::template load<!KEEP>(lane_ptr(base + i * stride, off));
                if constexpr (PART == kEdge) {
#pragma unroll
                    for (int i = 0; i < kFwdRows; ++i) to[i] = to[i].dropped(l.drop);
                }
            } else {
                load_some<Q, kFwdRows, !KEEP, FAST>(to, static_cast<const T*>(from) + pl.row0 * stride, stride, r0, pl.rows, l, p.D);
            }
        };
        fetch(a, p.a, p.as);
        fetch(b, p.b, p.bs);
        fetch(x, p.x, p.xs);
        if constexpr (GATE) fetch(z, p.z, p.zs);
#pragma unroll
        for (int i = 0; i < kFwdRows; ++i) {
#pragma unroll
            for (int j = 0; j < kVC; ++j) {
                const Gate g = gate(a[i].get(j) + bias[j], nrate2[j]);
                al[i][j] = g.alpha;
                u[i][j] = __builtin_amdgcn_sqrtf(g.q) * sigmoid_fast(b[i].get(j)) * x[i].get(j);
                if constexpr (PART == kSome) {
                    if (r0 + i >= pl.rows) { al[i][j] = 1.f; u[i][j] = 0.f; }
                }
                H[j] = i == 0 ? u[i][j] : fmaf(al[i][j], H[j], u[i][j]);
                A[j] = i == 0 ? al[i][j] : A[j] * al[i][j];
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
    template <Part PART>
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
        wave_start(l, A, H, s);
        constexpr int kPer = kGroups / kHalves;   // row groups between saved states
        if (p.saved && l.rg % kPer == 0)
            Quad<false>::store(p.saved + (kHalves * unit_index + l.rg / kPer) * p.D + l.c, s, l.nv);
        const int r0 = l.rg * kFwdRows;
        T* base = static_cast<T*>(p.y) + pl.row0 * p.ys + (l.c - l.cl * kVC);
        const uint32_t off = (static_cast<uint32_t>(r0) * static_cast<uint32_t>(p.ys) + l.cl * kVC) * sizeof(T);
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
            if constexpr (PART == kWhole) Q::store(lane_ptr(base + i * p.ys, off), o, kVC);
            else if ((PART == kEdge || r0 + i < pl.rows) && l.nv > 0) Q::store(lane_ptr(base + i * p.ys, off), o, l.nv);
        }
    }
};

__device__ __forceinline__ void load_params(const RecurParams& p, const Lane& l, float* nrate2, float* bias) {
#pragma unroll
    for (int j = 0; j < kVC; ++j) {
        nrate2[j] = j < l.nv ? -kLog2e * expf(p.A_log[l.c + j]) : 0.f;
        bias[j] = j < l.nv ? p.dt_bias[l.c + j] : 0.f;
    }
}

// (A, H) of a whole tile, for channel `lane`
__device__ __forceinline__ float2 tile_step(const float2 (*step)[kCh], int lane) {
    float A = 1.f, H = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const float2 e = step[w][lane];
        H = fmaf(e.x, H, e.y);
        A *= e.x;
    }
    return make_float2(A, H);
}

// Where tile `tile` of the units' table lies (tile < total)
__device__ __forceinline__ Place unit_place(const RecurParams& p, int unit) {
    const int seq = p.unit_seq[unit];
    const int lo = p.cu[seq];
    return place_of(lo, p.cu[seq + 1] - lo, seq, unit - p.unit_off[seq]);
}

__device__ __forceinline__ int draw_ticket(const RecurParams& p, int cg) {
    return static_cast<int>(__hip_atomic_fetch_add(p.tickets + cg * kRecurTicketPitch, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}

// grid: channel groups x the bound on units.  131072 x 2048 bf16: 615 us, 4.4
// TB/s of the 4.8 a large copy reaches; 4096 x 2048, one round of work-groups,
// 24 us.  (Work-groups that stay and draw
// tile after tile, with the next ticket drawn early, were slower: they need
// more registers, so fewer run at once.)
template <bool BF16, bool GATE, bool KEEP, bool FAST>
__global__ __launch_bounds__(kThreads, 3) void recur_forward_kernel(RecurParams p) {
    __shared__ FwdShared sh;
    const int total = p.unit_off[p.N];            // < 0: the call's indices were rejected
    const int cg = group_index() % p.groups;
    if (threadIdx.x == 0) sh.tile = draw_ticket(p, cg);
    const int c0 = cg * kCh;
    const Lane l = lane_of(c0, p.D);
    float nrate2[kVC], bias[kVC];
    load_params(p, l, nrate2, bias);
    __syncthreads();
    const int tile = __builtin_amdgcn_readfirstlane(sh.tile);
    if (tile >= total) return;
    const Place pl = unit_place(p, tile);
    FwdTile<BF16, GATE, KEEP, FAST> t;
    const Part part = part_of(pl.rows == kRecurUnit, c0, p.D);
    if (part == kWhole) t.template load<kWhole>(p, pl, l, nrate2, bias);
    else if (part == kEdge) t.template load<kEdge>(p, pl, l, nrate2, bias);
    else if (pl.rows > 0) t.template load<kSome>(p, pl, l, nrate2, bias);
    if (pl.rows > 0) t.publish(sh, l);
    __syncthreads();
    if (l.wave == 0) {
        const int c = c0 + l.lane;
        const float2 e = pl.rows > 0 ? tile_step(sh.step, l.lane) : make_float2(1.f, 0.f);
        uint64_t* w = p.words + static_cast<int64_t>(tile) * p.groups * kCh + c;
        const bool last = pl.unit + 1 == pl.units;
        float s = 0.f;
        if (pl.unit == 0) {
            if (p.h0 && c < p.D) s = p.h0[static_cast<int64_t>(state_slot(p.slots, pl.seq)) * p.D + c];
        } else {
            if (!last) put_word(w, step_word(e.x, e.y));
            s = look_back(w, -static_cast<int64_t>(p.groups) * kCh, pl.unit);
        }
        const float after = fmaf(e.x, s, e.y);
        if (!last) put_word(w, pack_word(kState, after));
        else if (p.hT && c < p.D)
            p.hT[static_cast<int64_t>(state_slot(p.slots, pl.seq)) * p.D + c] = pl.rows > 0 ? after : s;
        sh.start[l.lane] = s;
    }
    __syncthreads();
    if (part == kWhole) t.template finish<kWhole>(p, sh, pl, l, tile);
    else if (pl.rows > 0) t.template finish<kSome>(p, sh, pl, l, tile);
}

// One work-group per (channel group, sequence) walks the sequence's tiles in
// order: no words, no workspace, one launch.  Same bits: the state after a
// tile is the same fma.  Bound by the latency of a tile, one after the other: 8
// sequences of 64 tokens x 2048 14.4 us (the call's host time), one of 512 22.3,
// where tiles that run side by side take 18.7 for 513 tokens.
template <bool BF16, bool GATE, bool KEEP>
__global__ __launch_bounds__(kThreads, 3) void recur_walk_kernel(RecurParams p) {
    __shared__ FwdShared sh;
    __shared__ int bad, first_unit;
    const uint32_t id = group_index();
    const int seq = id / p.groups;
    if (seq >= p.N) return;
    if (threadIdx.x == 0) { bad = 0; first_unit = 0; }
    __syncthreads();
    // every work-group checks the indices, so nothing is written on a bad one
    int mine = 0, before = 0;
    for (int n = threadIdx.x; n < p.N; n += kThreads) {
        const int lo = p.cu[n], hi = p.cu[n + 1];
        if (hi < lo || (n == 0 && lo != 0) || (n + 1 == p.N && hi != p.T)) mine = 1;
        if (p.slots && (p.slots[n] < 0 || p.slots[n] >= p.num_slots)) mine = 1;
        if (n < seq && hi >= lo) before += units_of(hi - lo);
    }
    if (mine) atomicOr(&bad, 1);
    if (p.saved && before) atomicAdd(&first_unit, before);
    __syncthreads();
    if (p.status && id == 0 && threadIdx.x == 0) *p.status = bad ? kStatusBadIndex : 0;
    if (bad) return;
    const int cg = id % p.groups;
    const int c0 = cg * kCh;
    const Lane l = lane_of(c0, p.D);
    float nrate2[kVC], bias[kVC];
    load_params(p, l, nrate2, bias);
    const int lo = p.cu[seq], len = p.cu[seq + 1] - lo;
    const int c = c0 + l.lane;
    const int64_t at = static_cast<int64_t>(state_slot(p.slots, seq)) * p.D + c;
    if (l.wave == 0) sh.start[l.lane] = p.h0 && c < p.D ? p.h0[at] : 0.f;
    FwdTile<BF16, GATE, KEEP, false> t;
    const int units = units_of(len);
    for (int k = 0; k < units && len > 0; ++k) {
        const Place pl = place_of(lo, len, seq, k);
        const bool whole = part_of(pl.rows == kRecurUnit, c0, p.D) == kWhole;
        if (whole) t.template load<kWhole>(p, pl, l, nrate2, bias);
        else t.template load<kSome>(p, pl, l, nrate2, bias);
        t.publish(sh, l);
        __syncthreads();
        if (whole) t.template finish<kWhole>(p, sh, pl, l, static_cast<int64_t>(first_unit) + k);
        else t.template finish<kSome>(p, sh, pl, l, static_cast<int64_t>(first_unit) + k);
        float after = 0.f;
        if (l.wave == 0) {
            const float2 e = tile_step(sh.step, l.lane);
            after = fmaf(e.x, sh.start[l.lane], e.y);
        }
        __syncthreads();
        if (l.wave == 0) sh.start[l.lane] = after;
    }
    if (l.wave == 0 && p.hT && c < p.D) p.hT[at] = sh.start[l.lane];
}

// Block 0 checks the indices, lays out the units (unit_off, unit_seq) and sets
// the tickets to 0; the others set the words to kEmpty.
constexpr int kPlanThreads = 256;

__global__ __launch_bounds__(kPlanThreads) void recur_plan_kernel(RecurParams p) {
    const int tid = threadIdx.x;
    const int64_t nwords = static_cast<int64_t>(p.tiles) * p.groups * kCh;
    if (blockIdx.x != 0) {
        const int64_t stride = static_cast<int64_t>(gridDim.x - 1) * kPlanThreads;
        u32x4* pairs = reinterpret_cast<u32x4*>(p.words);              // (nwords is even)
        for (int64_t i = static_cast<int64_t>(blockIdx.x - 1) * kPlanThreads + tid; i < nwords / 2; i += stride)
            pairs[i] = u32x4{kEmpty, kEmpty, kEmpty, kEmpty};
        return;
    }
    for (int i = tid; i < p.groups; i += kPlanThreads) p.tickets[i * kRecurTicketPitch] = 0;
    __shared__ int part[kPlanThreads / kWave];
    // each thread a run of sequences
    const int per = (p.N + kPlanThreads - 1) / kPlanThreads;
    const int n0 = tid * per < p.N ? tid * per : p.N, n1 = n0 + per < p.N ? n0 + per : p.N;
    int sum = 0, mine = 0;
    for (int n = n0; n < n1; ++n) {
        const int lo = p.cu[n], hi = p.cu[n + 1];
        if (hi < lo || lo < 0 || hi > p.T || (n == 0 && lo != 0) || (n + 1 == p.N && hi != p.T)) mine = 1;
        else sum += units_of(hi - lo);
        if (p.slots && (p.slots[n] < 0 || p.slots[n] >= p.num_slots)) mine = 1;
    }
    int upto = sum;                               // inclusive over the wave, then over the waves
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const int v = __shfl_up(upto, d, kWave);
        if (tid % kWave >= d) upto += v;
    }
    if (tid % kWave == kWave - 1) part[tid / kWave] = upto;
    const bool bad = __syncthreads_or(mine);
    if (tid == 0 && p.status) *p.status = bad ? kStatusBadIndex : 0;
    if (bad) {
        if (tid == 0) p.unit_off[p.N] = -1;
        return;
    }
    int total = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / kWave; ++w) {
        if (w < tid / kWave) upto += part[w];
        total += part[w];
    }
    int at = upto - sum;
    for (int r = 0; r < per; ++r) {               // (as many rounds for every thread of a wave)
        const int n = n0 + r;
        const int k = n < n1 ? units_of(p.cu[n + 1] - p.cu[n]) : 0;
        if (n < n1) p.unit_off[n] = at;
        if (p.N > kPlanThreads) {                 // (few sequences: all threads together, below)
            // a long sequence's units by the whole wave
            for (uint64_t wide = __ballot(k > kWave); wide != 0; wide &= wide - 1) {
                const int from = __ffsll(static_cast<unsigned long long>(wide)) - 1;
                const int first_of = __shfl(at, from, kWave), units = __shfl(k, from, kWave), seq = __shfl(n, from, kWave);
                for (int i = tid % kWave; i < units; i += kWave) p.unit_seq[first_of + i] = seq;
            }
            if (k <= kWave)
                for (int i = 0; i < k; ++i) p.unit_seq[at + i] = n;
        }
        at += k;
    }
    if (tid == 0) p.unit_off[p.N] = total;
    if (p.N > kPlanThreads) return;
    __shared__ int first[kPlanThreads];
    first[tid] = upto - sum;                      // (one sequence a thread)
    __syncthreads();
    for (int i = tid; i < total; i += kPlanThreads) {
        int lo = 0, hi = p.N;                     // the last sequence that begins at or before unit i
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (first[mid] <= i) lo = mid;
            else hi = mid;
        }
        p.unit_seq[i] = lo;
    }
}

// ---- backward --------------------------------------------------------------
struct BwdShared {
    // each row group's (A, H), inclusive over its wave (kept here, not in
    // registers, while the tile waits)
    float2 fwd[kGroups][kCh], rev[kGroups][kCh];
    float2 sums[kWaves][kCh];
    // each lane's own, for the same reason: g log2(e), and da / dg
    f32x4 g2[kBwdRows][kThreads], sg[kBwdRows][kThreads];
    float start[kCh];                             // c past the tile's last row
    float before[kCh];                            // the state before its first row
    int tile;
};

// A lane's rows of a backward tile: what the second half (after the tile's
// start is known) needs of each element.  Registers decide how many
// work-groups share a compute unit, so what comes from z and dy is computed
// again from their packed rows, and what a's gate gives beside alpha waits in
// LDS.
template <bool BF16, bool GATE>
struct BwdTile {
    using Q = Quad<BF16>;
    using T = typename Q::T;
    static constexpr int L = kBwdRows;
    Q dy[L], z[L];
    float al[L][kVC], u[L][kVC];                  // alpha; u, later h before the row
    float wb[L][kVC];                             // w beta
    float xn[L][kVC], xk[L][kVC];                 // x (1 - beta), beta x alpha / w (0 where w is)

    // dy silu(z)
    __device__ __forceinline__ float into_h(int i, int j) const {
        if constexpr (!GATE) return dy[i].get(j);
        const float zj = z[i].get(j);
        return dy[i].get(j) * (zj * sigmoid_fast(zj));
    }

    template <Part PART>
    __device__ __forceinline__ void load(const RecurParams& p, BwdShared& sh, const Lane& l, int64_t row0, int rows,
                                         const float* nrate2, const float* bias) {
        const int r0 = l.rg * L;
        float A[kVC], H[kVC], Ar[kVC], Hr[kVC];
        Q a[L], x[L], b[L];
        auto fetch = [&](Q* to, const void* from, int64_t stride) {
            if constexpr (PART != kSome) {
                const T* base = static_cast<const T*>(from) + row0 * stride;
                const uint32_t off = (static_cast<uint32_t>(r0) * static_cast<uint32_t>(stride) + (PART == kEdge ? l.lc : l.c)) * sizeof(T);
#pragma unroll
                for (int i = 0; i < L; ++i) to[i] = Q::template load<true>(lane_ptr(base + i * stride, off));
                if constexpr (PART == kEdge) {
#pragma unroll
                    for (int i = 0; i < L; ++i) to[i] = to[i].dropped(l.drop);
                }
            } else {
                load_some<Q, L, true, true>(to, static_cast<const T*>(from) + row0 * stride, stride, r0, rows, l, p.D);
            }
        };
        fetch(a, p.a, p.as);
        fetch(b, p.b, p.bs);
        fetch(x, p.x, p.xs);
        fetch(dy, p.dy, p.dys);
        if constexpr (GATE) fetch(z, p.z, p.zs);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            f32x4 g2, sg;
#pragma unroll
            for (int j = 0; j < kVC; ++j) {
                const float v = a[i].get(j) + bias[j], xj = x[i].get(j);
                const Gate g = gate(v, nrate2[j]);
                const float beta = sigmoid_fast(b[i].get(j));
                const float over = g.q >= 0x1p-126f ? __builtin_amdgcn_rsqf(g.q) : 0.f;   // 1 / w
                xn[i][j] = xj * (1.f - beta);
                wb[i][j] = g.q * over * beta;
                xk[i][j] = xj * beta * g.alpha * over;
                al[i][j] = g.alpha;
                u[i][j] = wb[i][j] * xj;
                const float rv = __builtin_amdgcn_rcpf(1.f + g.e);
                g2[j] = g.g2;
                sg[j] = (v < 0.f ? g.e * rv : rv) * (nrate2[j] * kLn2);
                if constexpr (PART == kSome) {
                    if (r0 + i >= rows) { al[i][j] = 1.f; u[i][j] = 0.f; }
                }
                H[j] = i == 0 ? u[i][j] : fmaf(al[i][j], H[j], u[i][j]);
                A[j] = i == 0 ? al[i][j] : A[j] * al[i][j];
            }
            sh.g2[i][threadIdx.x] = g2;
            sh.sg[i][threadIdx.x] = sg;
        }
        // c_t = alpha_t (c_{t+1} + e_t); a row past the end hands c on
#pragma unroll
        for (int j = 0; j < kVC; ++j) {
            Ar[j] = A[j];
            Hr[j] = 0.f;
#pragma unroll
            for (int i = L - 1; i >= 0; --i)
                if (PART != kSome || r0 + i < rows) Hr[j] = al[i][j] * (Hr[j] + into_h(i, j));
        }
        wave_compose<false>(l, A, H);
        wave_compose<true>(l, Ar, Hr);
#pragma unroll
        for (int j = 0; j < kVC; ++j) {
            sh.fwd[l.rg][l.cl * kVC + j] = make_float2(A[j], H[j]);
            sh.rev[l.rg][l.cl * kVC + j] = make_float2(Ar[j], Hr[j]);
        }
    }

    // sa, sb: sums of dg g2 and of da over the lane's rows
    template <Part PART>
    __device__ __forceinline__ void finish(const RecurParams& p, const BwdShared& sh, const Lane& l, int64_t row0, int rows,
                                           float* sa, float* sb) {
        if constexpr (GATE) {
#pragma unroll
            for (int i = 0; i < L; ++i) z[i].forget();
        }
        float s[kVC], r[kVC];
#pragma unroll
        for (int j = 0; j < kVC; ++j) {
            s[j] = sh.before[l.cl * kVC + j];
            r[j] = sh.start[l.cl * kVC + j];
        }
        // through the waves before this one, then through its groups before this lane's
        auto apply = [&](const float2* t, float* v) {
#pragma unroll
            for (int j = 0; j < kVC; ++j) v[j] = fmaf(t[l.cl * kVC + j].x, v[j], t[l.cl * kVC + j].y);
        };
        for (int w = 0; w < l.wave; ++w) apply(sh.fwd[w * kGroupsPerWave + kGroupsPerWave - 1], s);
        for (int w = kWaves - 1; w > l.wave; --w) apply(sh.rev[w * kGroupsPerWave], r);
        if (l.rg % kGroupsPerWave > 0) apply(sh.fwd[l.rg - 1], s);
        if (l.rg % kGroupsPerWave < kGroupsPerWave - 1) apply(sh.rev[l.rg + 1], r);
        const int r0 = l.rg * L;
        // a row's four gradients at (row0 + r0 + i); strides are of 22 bits, so offsets are of 32
        auto put = [&](void* to, int64_t stride, int i, const float* f) {
            T* base = static_cast<T*>(to) + row0 * stride + (l.c - l.cl * kVC);
            const uint32_t off = (static_cast<uint32_t>(r0) * static_cast<uint32_t>(stride) + l.cl * kVC) * sizeof(T);
            if constexpr (PART == kWhole) Q::store(lane_ptr(base + i * stride, off), f, kVC);
            else if (r0 + i < rows && l.nv > 0) Q::store(lane_ptr(base + i * stride, off), f, l.nv);
        };
#pragma unroll
        for (int i = 0; i < L; ++i) {             // u: from u to the state before the row; dz
            float o[kVC];
#pragma unroll
            for (int j = 0; j < kVC; ++j) {
                const float next = fmaf(al[i][j], s[j], u[i][j]);
                u[i][j] = s[j];
                s[j] = next;
                if constexpr (GATE) {
                    const float zj = z[i].get(j), q = sigmoid_fast(zj);
                    o[j] = next * (dy[i].get(j) * (q * fmaf(zj, 1.f - q, 1.f)));
                }
            }
            if constexpr (GATE) put(p.dz, p.dzs, i, o);
        }
#pragma unroll
        for (int i = L - 1; i >= 0; --i) {
            float dx[kVC], da[kVC], db[kVC];
            const f32x4 g2 = sh.g2[i][threadIdx.x], sg = sh.sg[i][threadIdx.x];
#pragma unroll
            for (int j = 0; j < kVC; ++j) {
                const bool on = PART == kWhole || r0 + i < rows;
                const float G = (on ? into_h(i, j) : 0.f) + r[j];
                const float aG = al[i][j] * G;
                r[j] = aG;
                dx[j] = G * wb[i][j];
                db[j] = dx[j] * xn[i][j];
                const float dg = aG * (u[i][j] - xk[i][j]);
                da[j] = dg * sg[j];
                if (on) {
                    sa[j] = fmaf(dg, g2[j], sa[j]);
                    sb[j] += da[j];
                }
            }
            put(p.dx, p.dxs, i, dx);
            put(p.da, p.das, i, da);
            put(p.db, p.dbs, i, db);
        }
    }
};

// grid: channel groups x kHalves x the bound on units; the tiles of a sequence
// are taken from its end.  The rows' h are run again from the state the
// forward pass saved at the tile's first row.
// 32768 x 4096 bf16: 604 to 628 us, 3.9 TB/s.  Three waves a SIMD: with all of the
// gates' values in registers (228, two waves) the training step of that size
// took 1.12 ms, with a's gate computed again 1.00, with it in LDS 0.95.
// Work-groups of 512 threads that keep all of it in 122 registers: 1.18, as
// only two share a compute unit.  (fp32 spills 3 registers, 18 without z: 16384
// x 2048 247 us, without z 204, 4.9 and 4.6 TB/s.)
template <bool BF16, bool GATE>
__global__ __launch_bounds__(kThreads, 3) void recur_backward_kernel(RecurParams p) {
    __shared__ BwdShared sh;
    const int total = kHalves * p.unit_off[p.N];
    const int cg = group_index() % p.groups;
    if (threadIdx.x == 0) sh.tile = draw_ticket(p, cg);
    const int c0 = cg * kCh;
    const Lane l = lane_of(c0, p.D);
    float nrate2[kVC], bias[kVC];
    load_params(p, l, nrate2, bias);
    __syncthreads();
    const int tile = total - 1 - __builtin_amdgcn_readfirstlane(sh.tile);
    if (tile < 0) return;
    const Place pl = unit_place(p, tile / kHalves);
    const int t0 = (tile % kHalves) * kBwdTile;   // first row within the unit
    const int left = pl.rows - t0;
    const int rows = left < 0 ? 0 : (left < kBwdTile ? left : kBwdTile);
    const int64_t row0 = pl.row0 + t0;
    const Part part = part_of(rows == kBwdTile, c0, p.D);
    BwdTile<BF16, GATE> t;
    if (part == kWhole) t.template load<kWhole>(p, sh, l, row0, rows, nrate2, bias);
    else if (part == kEdge) t.template load<kEdge>(p, sh, l, row0, rows, nrate2, bias);
    else if (rows > 0) t.template load<kSome>(p, sh, l, row0, rows, nrate2, bias);
    __syncthreads();
    if (l.wave == 0) {
        const int ch = c0 + l.lane;
        float2 e = make_float2(1.f, 0.f);         // (A, H) of the whole tile
        for (int w = kWaves - 1; w >= 0 && rows > 0; --w) {
            const float2 g = sh.rev[w * kGroupsPerWave][l.lane];
            e.y = fmaf(g.x, e.y, g.y);
            e.x *= g.x;
        }
        uint64_t* w = p.words + static_cast<int64_t>(tile) * p.groups * kCh + ch;
        const bool first = pl.unit == 0 && tile % kHalves == 0;
        const int behind = kHalves * (pl.units - pl.unit) - 1 - tile % kHalves;   // tiles of the sequence after this one
        float s = 0.f;
        if (behind == 0) {
            if (p.dhT && ch < p.D) s = p.dhT[static_cast<int64_t>(pl.seq) * p.D + ch];
        } else {
            if (!first) put_word(w, step_word(e.x, e.y));
            s = look_back(w, static_cast<int64_t>(p.groups) * kCh, behind);
        }
        const float after = fmaf(e.x, s, e.y);
        if (!first) put_word(w, pack_word(kState, after));
        else if (p.dh0 && ch < p.D) p.dh0[static_cast<int64_t>(pl.seq) * p.D + ch] = rows > 0 ? after : s;
        sh.start[l.lane] = s;
    } else if (l.wave == 1) {
        sh.before[l.lane] = c0 + l.lane < p.D ? p.saved[static_cast<int64_t>(tile) * p.D + c0 + l.lane] : 0.f;
    }
    __syncthreads();
    float sa[kVC], sb[kVC];
#pragma unroll
    for (int j = 0; j < kVC; ++j) sa[j] = sb[j] = 0.f;
    if (part == kWhole) t.template finish<kWhole>(p, sh, l, row0, rows, sa, sb);
    else if (rows > 0) t.template finish<kSome>(p, sh, l, row0, rows, sa, sb);
    if (!p.partial) return;
    // the tile's sums over its rows, in a fixed order
#pragma unroll
    for (int j = 0; j < kVC; ++j) {
#pragma unroll
        for (int d = kChLanes; d < kWave; d *= 2) {
            sa[j] += __shfl_xor(sa[j], d, kWave);
            sb[j] += __shfl_xor(sb[j], d, kWave);
        }
    }
    if (l.lane < kChLanes) {
#pragma unroll
        for (int j = 0; j < kVC; ++j) sh.sums[l.wave][l.cl * kVC + j] = make_float2(sa[j], sb[j]);
    }
    __syncthreads();
    if (l.wave == 0) {
        float2 v = sh.sums[0][l.lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) {
            const float2 e = sh.sums[w][l.lane];
            v.x += e.x;
            v.y += e.y;
        }
        p.partial[static_cast<int64_t>(tile) * p.groups * kCh + c0 + l.lane] = v;
    }
}

// dA_log and ddt_bias from the tiles' sums, each channel's tiles in a fixed
// order.  A work-group for 16 channels, 64 threads a channel.
constexpr int kSumThreads = 1024, kSumCh = 16, kSumSlices = kSumThreads / kSumCh;

__global__ __launch_bounds__(kSumThreads) void recur_sum_kernel(RecurParams p) {
    const int total = kHalves * p.unit_off[p.N];
    if (total < 0) return;
    __shared__ float2 part[kSumSlices][kSumCh];
    const int ch = threadIdx.x % kSumCh, sl = threadIdx.x / kSumCh;
    const int c = blockIdx.x * kSumCh + ch;
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
        if (p.ddt_bias) p.ddt_bias[c] = t.y;
    }
}

// ---- one token per sequence ------------------------------------------------
// (bound by the launch: 64 x 4096 takes 4.6 us)
constexpr int kDecodeThreads = 256;

template <bool BF16, bool GATE>
__global__ __launch_bounds__(kDecodeThreads) void recur_decode_kernel(RecurParams p) {
    using Q = Quad<BF16>;
    using T = typename Q::T;
    const int per = (p.D + kVC - 1) / kVC;        // lanes of a row
    const int64_t i = static_cast<int64_t>(group_index()) * kDecodeThreads + threadIdx.x;
    if (i / per >= p.N) return;
    const int n = static_cast<int>(i / per);
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
        const float nrate2 = j < nv ? -kLog2e * expf(p.A_log[c + j]) : 0.f, bias = j < nv ? p.dt_bias[c + j] : 0.f;
        const Gate g = gate(a.get(j) + bias, nrate2);
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

// KERNEL<bf16, gate, ...>
#define GDN_RECUR_CALL(KERNEL, GRID, BLOCK, ...)                                                    \
    do {                                                                                            \
        const dim3 g_ = grid_of(GRID), b_(BLOCK);                                                   \
        if (bf16 && p.z) hipLaunchKernelGGL((KERNEL<true, true __VA_ARGS__>), g_, b_, 0, s, p);     \
        else if (bf16) hipLaunchKernelGGL((KERNEL<true, false __VA_ARGS__>), g_, b_, 0, s, p);      \
        else if (p.z) hipLaunchKernelGGL((KERNEL<false, true __VA_ARGS__>), g_, b_, 0, s, p);       \
        else hipLaunchKernelGGL((KERNEL<false, false __VA_ARGS__>), g_, b_, 0, s, p);               \
    } while (0)

static hipError_t launch_plan(const RecurParams& p, hipStream_t s) {
    const int64_t nwords = static_cast<int64_t>(p.tiles) * p.groups * kCh;
    int64_t blocks = 2 + nwords / (kPlanThreads * 16);
    if (blocks > 2048) blocks = 2048;
    hipLaunchKernelGGL(recur_plan_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kPlanThreads), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_recur_forward(const RecurParams& p, bool bf16, hipStream_t s) {
    if (p.walk) {
        GDN_RECUR_CALL(recur_walk_kernel, static_cast<int64_t>(p.groups) * p.N, kThreads, , true);
        return hipGetLastError();
    }
    hipError_t e = launch_plan(p, s);
    if (e != hipSuccess) return e;
    const int64_t grid = static_cast<int64_t>(p.groups) * p.tiles;
    // Saved states: 132 registers without FAST, so three waves a SIMD either way
    // (32768 x 4096 in 8 whole sequences 319 us with FAST, 320 without; in 8
    // ragged ones 329 and 349; 60000 x 1024 in 600 sequences 213 and 359).  Else
    // sequences of fewer than four units on average: a quarter of the tiles or
    // more is cut (33000 x 1024, 300 tokens each: 114 us with FAST, 118
    // without; 900 tokens each: 104 and 100)
    if (p.saved) GDN_RECUR_CALL(recur_forward_kernel, grid, kThreads, , true, true);
    else if (p.T / p.N < 4 * kRecurUnit) GDN_RECUR_CALL(recur_forward_kernel, grid, kThreads, , false, true);
    else GDN_RECUR_CALL(recur_forward_kernel, grid, kThreads, , false, false);
    return hipGetLastError();
}

hipError_t launch_recur_backward(const RecurParams& p, bool bf16, hipStream_t s) {
    hipError_t e = launch_plan(p, s);
    if (e != hipSuccess) return e;
    GDN_RECUR_CALL(recur_backward_kernel, static_cast<int64_t>(p.groups) * p.tiles, kThreads);
    e = hipGetLastError();
    if (e != hipSuccess || !p.partial) return e;
    hipLaunchKernelGGL(recur_sum_kernel, dim3(static_cast<unsigned>((p.D + kSumCh - 1) / kSumCh)), dim3(kSumThreads), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_recur_decode(const RecurParams& p, bool bf16, hipStream_t s) {
    const int64_t lanes = static_cast<int64_t>(p.N) * ((p.D + kVC - 1) / kVC);
    GDN_RECUR_CALL(recur_decode_kernel, (lanes + kDecodeThreads - 1) / kDecodeThreads, kDecodeThreads);
    return hipGetLastError();
}

}  // namespace gdn
