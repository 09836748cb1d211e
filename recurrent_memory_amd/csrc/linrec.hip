// Gated linear recurrence h_t = exp(g_t) h_{t-1} + beta_t x_t per channel, its
// backward pass and its single-token step.
//
// Method.  A run of tokens acts on the state as one affine map h -> A h + c (A the
// product of its decays, c the state it reaches from zero), and maps of adjacent
// runs join by (A2, c2) after (A1, c1) = (A2 A1, A2 c1 + c2).  The backward pass is
// the same recurrence in reverse: with r the gradient that arrives at h_t from later
// tokens, e_t = r + dO_t and r <- exp(g_t) e_t.
//
// Tiles.  HBM traffic is the bound (4 values per element forward, 7 backward, about
// 10 operations each), so every value is read once: a workgroup holds a tile of 128
// tokens x 64 lanes (one 4-byte word of channels a lane) in registers from its loads
// to its stores.  A wave takes 16 consecutive tokens; the waves join their maps
// through LDS, and the tiles of a sequence through device memory, in one launch: a
// tile publishes its map as soon as it has it, without waiting for anything, then
// collects the maps of the tiles before it.  So that a late tile need not read all of
// them, every 16th tile publishes the state behind it, and a tile reads the last
// such state and at most 15 maps.  Which values are joined in which order depends on
// positions alone, so results do not depend on timing.
//
// Forgetting.  A decay that is zero in fp32 drops the state in front of it, whatever that
// is: 0 times an infinity would be NaN.  So does the map of a run that holds such a token;
// a product of decays that only gets small stops at the smallest normal number instead
// (which moves a state by at most 2^-126 of one before it), so that an infinity stays one.
// A wave takes its 16 tokens without regard to this.  If their product of decays leaves
// the normal numbers in some lane, it reduces them once more with a selection for each; and
// if then a decay was zero and a state or gradient ends not finite (none becomes finite
// again on the way), it takes its outputs again, token by token, in a loop that needs few
// registers (selections in every wave: backward 181 instead of 170 us at B=1 T=32768 D=2048
// bf16; a second form of the unrolled code for the waves with a zero, which spills: 124
// instead of 100 us at B=4 T=4096 D=2048 with a document's border every 512 tokens).
//
// Waiting.  A published word carries its own readiness: the workspace is filled with
// all-ones (a NaN pattern that is never published) before the launch, and readers poll
// the word itself with relaxed device-scope atomics, so no fence or flag is needed.
// The tiles of a column (64 lanes, all tokens) are handed out in their order of action
// by the column's counter: a workgroup waits only for earlier tiles of its column,
// which are held by workgroups that already run, and publishes its own map before it
// waits; by induction over the column every wait ends, whatever else runs on the GPU.
// (One counter for all columns hands out a tile every 20 ns at best, 50 tiles a
// microsecond, which is as much as HBM takes.)
#include <type_traits>

#include "common.h"
#include "kernels.h"
#include "slots.h"

namespace dr {
namespace {

constexpr int kTok = 16;            // tokens of a wave, and tokens per row of `states`
constexpr int kMaxWaves = 8;        // waves of a workgroup: tiles of 128 tokens
constexpr int kSingleWaves = 16;    // sequences of up to 256 tokens are one tile
constexpr int kGroup = 16;          // tiles from one published state to the next
constexpr int kCarryWave = kMaxWaves - 1;   // the last wave collects the state, the others maps,
constexpr int kPer = (kGroup - 1 + kMaxWaves - 2) / (kMaxWaves - 1);   // this many each
constexpr int kStepThreads = 256;
constexpr float kSmallest = 0x1p-126f;
constexpr uint32_t kMaxGrid = 1u << 16;   // workgroups; with more tiles than that, each takes several

// A map applied to a state, and the decays of adjacent runs joined (see Forgetting).
__device__ __forceinline__ float apply(float a, float h, float c) { return a == 0.f ? c : fmaf(a, h, c); }
__device__ __forceinline__ float join(float A, float a) { return A == 0.f || a == 0.f ? 0.f : fmaxf(A * a, kSmallest); }

// Memory accesses of the tiles.  NT: non-temporal, where rows are whole cache lines and
// every line passes once (B=1 T=32768 D=2048 bf16: forward 112 us plain, 106 us
// non-temporal, backward 185 and 169 us; D=2112, where a wave's end falls inside a row,
// B=4 T=4096: forward 67 and 61 us, backward 113 and 102 us); plain where two waves share
// lines, which then may meet in a cache (B=3 T=8000 D=1000 bf16: forward 56 us plain, 60 us
// non-temporal; backward 100 and 118 us; T=4000 D=1001 fp32: 54 and 62, 104 and 129 us).
template <bool NT, typename P>
__device__ __forceinline__ P load_word(const P* p) {
    if constexpr (NT) return __builtin_nontemporal_load(p);
    else return *p;
}
template <bool NT, typename P, typename V>
__device__ __forceinline__ void store_word(P* p, V v) {
    if constexpr (NT) __builtin_nontemporal_store(static_cast<P>(v), p);
    else *p = static_cast<P>(v);
}

// A lane's channels: one fp32, or a word of two bf16.  Where D is odd (Bf16Odd) words
// start on any 2-byte address, and the last lane of a row has a single channel; a lane
// with `lone` set touches only that.
struct Fp32 {
    typedef float T;
    static constexpr int VEC = 1;
    static constexpr bool kOdd = false;
    template <bool NT>
    static __device__ __forceinline__ uint32_t load(const T* p) { return __float_as_uint(load_word<NT>(p)); }
    static __device__ __forceinline__ void unpack(uint32_t r, float* f) { f[0] = __uint_as_float(r); }
    template <bool NT>
    static __device__ __forceinline__ void store(T* p, const float* f, bool) { store_word<NT>(p, f[0]); }
};
struct Bf16Even {
    typedef uint16_t T;
    static constexpr int VEC = 2;
    static constexpr bool kOdd = false;
    template <bool NT>
    static __device__ __forceinline__ uint32_t load(const T* p) {
        return load_word<NT>(reinterpret_cast<const uint32_t*>(p));
    }
    static __device__ __forceinline__ void unpack(uint32_t r, float* f) {
        f[0] = __uint_as_float(r << 16);
        f[1] = __uint_as_float(r & 0xffff0000u);
    }
    static __device__ __forceinline__ uint32_t pack(const float* f) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        const f32x2 v = {f[0], f[1]};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    }
    template <bool NT>
    static __device__ __forceinline__ void store(T* p, const float* f, bool) {
        store_word<NT>(reinterpret_cast<uint32_t*>(p), pack(f));
    }
};
struct Bf16Odd : Bf16Even {
    struct __attribute__((packed, aligned(2))) Word { uint32_t w; };
    static constexpr bool kOdd = true;
    template <bool NT>
    static __device__ __forceinline__ uint32_t load(const T* p) { return reinterpret_cast<const Word*>(p)->w; }
    template <bool NT>
    static __device__ __forceinline__ void store(T* p, const float* f, bool lone) {
        const uint32_t w = pack(f);
        if (lone) *p = static_cast<uint16_t>(w);
        else reinterpret_cast<Word*>(p)->w = w;
    }
};

// How the tiles of a call are numbered, and its workspace.
struct Tiles {
    uint32_t lanes;        // B * row_lanes
    uint32_t row_lanes;    // lanes of a sequence: D / VEC, rounded up
    uint32_t columns;      // lane groups of 64
    uint32_t n;            // tiles: columns * chain
    int chain;             // tiles of a sequence
    uint32_t* ticket;      // a counter per column, kCounter words apart
    uint64_t* maps;        // [chain][B * D] (A, c)
    uint32_t* after;       // [ceil(chain / kGroup)][B * D] state behind every 16th tile
};

constexpr int kCounter = 16;               // 64 bytes: columns do not share a cache line's atomics
constexpr uint64_t kNoMap = ~uint64_t(0);
constexpr uint32_t kNoState = ~uint32_t(0);
constexpr uint32_t kNan = 0x7fc00000u;     // every NaN is published as this one

__device__ __forceinline__ uint32_t published(float f) { return f != f ? kNan : __float_as_uint(f); }

__device__ __forceinline__ void publish_map(uint64_t* at, float A, float c) {
    const uint64_t v = static_cast<uint64_t>(published(A)) << 32 | published(c);
    __hip_atomic_store(at, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The maps of n (1 .. kPer) consecutive tiles, joined, for the lane's channels; waits
// until all of the wave's are published.  at: the first tile's, `stride` words a tile.
template <int VEC>
__device__ __forceinline__ void collect_maps(const uint64_t* at, int64_t stride, int n, int nch,
                                             float2* out) {
    uint64_t m[kPer][VEC];
    bool ready;
    do {
        ready = true;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                m[i][v] = 0;
                if (v < nch && i < n)
                    m[i][v] = __hip_atomic_load(at + i * stride + v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) ready = ready && m[i][v] != kNoMap;
        }
        ready = __all(ready);
        if (!ready) __builtin_amdgcn_s_sleep(1);
    } while (!ready);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        float A = 1.f, c = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (i < n) {
                const float a = __uint_as_float(static_cast<uint32_t>(m[i][v] >> 32));
                c = apply(a, c, __uint_as_float(static_cast<uint32_t>(m[i][v])));
                A = join(A, a);
            }
        }
        out[v] = make_float2(A, c);
    }
}

template <int VEC>
__device__ __forceinline__ void collect_state(const uint32_t* at, int nch, float* out) {
    uint32_t v[VEC];
    bool ready;
    do {
        ready = true;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            v[e] = e < nch ? __hip_atomic_load(at + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
            ready = ready && v[e] != kNoState;
        }
        ready = __all(ready);
        if (!ready) __builtin_amdgcn_s_sleep(1);
    } while (!ready);
#pragma unroll
    for (int e = 0; e < VEC; ++e) out[e] = __uint_as_float(v[e]);
}

// What a tile's waves share.
template <int VEC>
struct Joint {
    float2 wave[kSingleWaves][64 * VEC];  // the waves' maps, in the order they act
    float2 tile[kMaxWaves - 1][64 * VEC]; // maps of the tiles before this one, of its group
    float carry[64 * VEC];                // the state in front of those
    float start[kSingleWaves][64 * VEC];  // what wave_start() gave the waves that may begin again
    uint32_t ticket;
};

// The state in front of a wave's tokens, from the wave maps in LDS.  pos: the wave's
// place in the order of action; q: the tile's place in its sequence's chain; init:
// the initial state (or null), ch: the index in [B, D] of the lane's first channel, nch:
// how many it has.  Called by all waves, after J.wave[pos] is written by each.
template <int VEC>
__device__ __forceinline__ void wave_start(Joint<VEC>& J, const Tiles& ts, int w, int pos, int waves,
                                           int q, const float* init, uint32_t ch, int64_t channels,
                                           int nch, float* h) {
    const int lane = threadIdx.x & 63;
    const int loader = waves > kCarryWave ? kCarryWave : waves - 1;
    // the initial state is read before anything is published: it may be the buffer that
    // the last tile writes the final state to
    if (q == 0 && w == loader) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) J.carry[lane * VEC + v] = init != nullptr && v < nch ? init[ch + v] : 0.f;
    }
    __syncthreads();
    float A[VEC], c[VEC];
    const int j = q % kGroup;
    const bool more = q + 1 < ts.chain;
    if (ts.chain > 1) {
        if (w == kCarryWave && more) {
            // the tile's own map; tile 0 acts from its initial state on, whatever precedes it
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                A[v] = 1.f;
                c[v] = q == 0 ? J.carry[lane * VEC + v] : 0.f;
            }
            for (int k = 0; k < waves; ++k) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float2 m = J.wave[k][lane * VEC + v];
                    c[v] = apply(m.x, c[v], m.y);
                    A[v] = join(A[v], m.x);
                }
            }
            if (q == 0) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) A[v] = 0.f;
            }
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                if (v < nch) publish_map(ts.maps + q * channels + ch + v, A[v], c[v]);
        }
        if (w < kCarryWave && w * kPer < j)
            collect_maps<VEC>(ts.maps + (q - j + w * kPer) * channels + ch, channels, min(j - w * kPer, kPer), nch,
                              &J.tile[w][lane * VEC]);
        if (w == kCarryWave && q > 0) {
            float s[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) s[v] = 0.f;      // first group: tile 0's map says it all
            if (q >= kGroup) collect_state<VEC>(ts.after + (q / kGroup - 1) * channels + ch, nch, s);
#pragma unroll
            for (int v = 0; v < VEC; ++v) J.carry[lane * VEC + v] = s[v];
        }
        __syncthreads();
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = J.carry[lane * VEC + v];
    for (int k = 0; k * kPer < j; ++k) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float2 m = J.tile[k][lane * VEC + v];
            h[v] = apply(m.x, h[v], m.y);
        }
    }
    if (ts.chain > 1 && w == kCarryWave && more && j == kGroup - 1) {
#pragma unroll
        for (int v = 0; v < VEC; ++v)
            if (v < nch)
                __hip_atomic_store(ts.after + (q / kGroup) * channels + ch + v, published(apply(A[v], h[v], c[v])),
                                   __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    for (int k = 0; k < pos; ++k) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float2 m = J.wave[k][lane * VEC + v];
            h[v] = apply(m.x, h[v], m.y);
        }
    }
}

// The turn-th tile of this workgroup: its column, and its place q in the column's order
// of action.  False when there is none.
template <int VEC>
__device__ __forceinline__ bool next_tile(Joint<VEC>& J, const Tiles& ts, uint32_t turn,
                                          uint32_t* column, int* q) {
    const uint32_t k = blockIdx.x + turn * gridDim.x;
    if (k >= ts.n) return false;
    // A different column first in each turn of the columns: workgroups go round the eight
    // XCDs, and with the same columns always on the same XCD, its L2 would see a few
    // residues of the row's addresses only, a few of its channels (B=1 T=32768 D=2048
    // bf16 forward: 125 us so, 106 us with the columns turned).
    *column = (k % ts.columns + k / ts.columns) % ts.columns;
    *q = 0;
    if (turn > 0) __syncthreads();      // the last tile's LDS is no longer read
    if (ts.chain > 1) {
        if (threadIdx.x == 0)
            J.ticket = __hip_atomic_fetch_add(ts.ticket + *column * kCounter, 1u, __ATOMIC_RELAXED,
                                              __HIP_MEMORY_SCOPE_AGENT) + 1u;      // from all-ones
        __syncthreads();
        *q = __builtin_amdgcn_readfirstlane(J.ticket);
    }
    return true;
}

// A wave's part of a tile: its lane's channels and its tokens.
// UNI: D is a multiple of the 64 lanes' channels, so that a wave lies in one sequence
// and its addresses are a scalar row plus the lane.
template <typename W, bool UNI>
struct Place {
    int64_t seq;       // sequence
    uint32_t c;        // first channel in it
    uint32_t ch;       // first channel in [B, D]
    int nch;           // channels: VEC, 1 in the lone lane of an odd row, 0 behind the last
    bool lone;
    __device__ __forceinline__ Place(const Tiles& ts, uint32_t column, int lane, int D) {
        const uint32_t L = column * 64u + lane;
        if constexpr (UNI) {
            const uint32_t L0 = column * 64u;
            seq = L0 / ts.row_lanes;
            c = (L0 % ts.row_lanes + lane) * W::VEC;
        } else {
            seq = L / ts.row_lanes;
            c = L % ts.row_lanes * W::VEC;
        }
        ch = static_cast<uint32_t>(seq) * D + c;
        lone = W::kOdd && c + 1 == static_cast<uint32_t>(D);
        nch = UNI || L < ts.lanes ? (lone ? 1 : W::VEC) : 0;
    }
};

// The words of n (0 .. 16) tokens from element `row` on, rows of D elements; zeros
// beyond them and in lanes without channels (g = 0, x = 0, dO = 0 act as identity).
template <bool NT, typename W, bool UNI>
__device__ __forceinline__ void load_tokens(const void* base, int64_t row, const Place<W, UNI>& at, int D,
                                            int n, uint32_t* r) {
    const typename W::T* p = static_cast<const typename W::T*>(base) + row;
#pragma unroll
    for (int i = 0; i < kTok; ++i) r[i] = 0;
    if (at.nch == 0) return;
    if (W::kOdd && __any(at.lone)) {
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const typename W::T* q = p + static_cast<int64_t>(i) * D + at.c;
            if (i < n) r[i] = at.lone ? static_cast<uint32_t>(*q) : W::template load<NT>(q);
        }
    } else if (n == kTok) {
#pragma unroll
        for (int i = 0; i < kTok; ++i) r[i] = W::template load<NT>(p + static_cast<int64_t>(i) * D + at.c);
    } else {
#pragma unroll
        for (int i = 0; i < kTok; ++i)
            if (i < n) r[i] = W::template load<NT>(p + static_cast<int64_t>(i) * D + at.c);
    }
}

// Makes the compiler take the words as new values, so that what it computed from them
// before (two fp32 decays or products for each word) is computed again, not kept in
// registers.
__device__ __forceinline__ void forget_derived(uint32_t* r) {
#pragma unroll
    for (int i = 0; i < kTok; ++i) asm volatile("" : "+v"(r[i]));
}

// The word of one token, of a lane that has channels.
template <typename W, bool UNI>
__device__ __forceinline__ uint32_t load_token(const void* base, int64_t row, const Place<W, UNI>& at) {
    const typename W::T* q = static_cast<const typename W::T*>(base) + row + at.c;
    if (W::kOdd && at.lone) return static_cast<uint32_t>(*q);
    return W::template load<false>(q);
}

// Whether a token of the wave may forget, from the products of its lanes' decays; after
// join() made these, whether one does.
template <int VEC>
__device__ __forceinline__ bool any_forgets(const float* A) {
    bool normal = true;
#pragma unroll
    for (int v = 0; v < VEC; ++v) normal = normal && A[v] >= kSmallest;
    return __any(!normal);
}
template <int VEC>
__device__ __forceinline__ bool all_finite(const float* f) {
    bool finite = true;
#pragma unroll
    for (int v = 0; v < VEC; ++v) finite = finite && __builtin_isfinite(f[v]);
    return finite;
}

// Six waves a SIMD, three workgroups of eight waves a CU, for words of one channel and
// without a gate, which the compiler misses by a few registers (B=4 T=4096 D=2048 bf16
// without a gate 44.7 us, with five waves 47.2; D=1024 fp32 with one 53.7 us, with five
// 55.0; two registers spilled where rows are not whole waves).  Two channels and a gate take
// a hundred registers, two workgroups.
template <typename W, bool BETA, bool UNI, bool NT>
__global__ __launch_bounds__(kSingleWaves * 64, BETA && W::VEC == 2 ? 1 : 6) void linrec_fwd_kernel(LinrecArgs p, Tiles ts) {
    constexpr int VEC = W::VEC;
    __shared__ Joint<VEC> J;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int64_t channels = static_cast<int64_t>(p.B) * p.D, blocks = (p.T - 1) / kTok + 1;
    for (uint32_t turn = 0;; ++turn) {
        uint32_t column;
        int q;
        if (!next_tile(J, ts, turn, &column, &q)) return;
        const Place<W, UNI> at(ts, column, lane, p.D);
        const int64_t t0 = (static_cast<int64_t>(q) * waves + w) * kTok;
        const int n = static_cast<int>(p.T - t0 >= kTok ? kTok : p.T > t0 ? p.T - t0 : 0);
        const int64_t row = (at.seq * p.T + t0) * p.D;
        uint32_t xr[kTok], gr[kTok], br[kTok];
        load_tokens<NT>(p.x, row, at, p.D, n, xr);
        load_tokens<NT>(p.g, row, at, p.D, n, gr);
        if constexpr (BETA) load_tokens<NT>(p.beta, row, at, p.D, n, br);

        // one token's decay and written value
        auto token = [&](int i, float* a, float* u) {
            float b[VEC];
            W::unpack(xr[i], u);
            W::unpack(gr[i], a);
            if constexpr (BETA) W::unpack(br[i], b);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                a[v] = __expf(a[v]);
                if constexpr (BETA) u[v] *= b[v];
            }
        };
        float A[VEC], h[VEC];
        auto reduce = [&](auto forgets) {
            float a[VEC], u[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) { A[v] = 1.f; h[v] = 0.f; }
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                token(i, a, u);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    h[v] = forgets ? apply(a[v], h[v], u[v]) : fmaf(a[v], h[v], u[v]);
                    A[v] = forgets ? join(A[v], a[v]) : A[v] * a[v];
                }
            }
        };
        reduce(std::false_type());
        bool forgets = any_forgets<VEC>(A);
        if (__builtin_expect(forgets, 0)) {
            forget_derived(gr);
            forget_derived(xr);
            if constexpr (BETA) forget_derived(br);
            reduce(std::true_type());
            forgets = any_forgets<VEC>(A);
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) J.wave[w][lane * VEC + v] = make_float2(A[v], h[v]);
        forget_derived(gr);
        forget_derived(xr);
        if constexpr (BETA) forget_derived(br);
        wave_start<VEC>(J, ts, w, w, waves, q, p.h0, at.ch, channels, at.nch, h);
        if (at.nch > 0 && n > 0) {             // all lanes go on to the next tile's barrier
            if (p.states != nullptr) {
                float* s = p.states + (at.seq * blocks + t0 / kTok) * p.D + at.c;
#pragma unroll
                for (int v = 0; v < VEC; ++v)
                    if (v < at.nch) s[v] = h[v];
            }
            typename W::T* o = static_cast<typename W::T*>(p.o) + row;
            if (forgets) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) J.start[w][lane * VEC + v] = h[v];
            }
            float a[VEC], u[VEC];
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                token(i, a, u);
#pragma unroll
                for (int v = 0; v < VEC; ++v) h[v] = fmaf(a[v], h[v], u[v]);
                if (i < n) W::template store<NT>(o + static_cast<int64_t>(i) * p.D + at.c, h, at.lone);
            }
            if (__builtin_expect(forgets && !all_finite<VEC>(h), 0)) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) h[v] = J.start[w][lane * VEC + v];
#pragma unroll 1
                for (int i = 0; i < n; ++i) {
                    const int64_t el = row + static_cast<int64_t>(i) * p.D;
                    float b[VEC];
                    W::unpack(load_token<W>(p.x, el, at), u);
                    W::unpack(load_token<W>(p.g, el, at), a);
                    if constexpr (BETA) W::unpack(load_token<W>(p.beta, el, at), b);
#pragma unroll
                    for (int v = 0; v < VEC; ++v) {
                        if constexpr (BETA) u[v] *= b[v];
                        h[v] = apply(__expf(a[v]), h[v], u[v]);
                    }
                    W::template store<NT>(static_cast<typename W::T*>(p.o) + el + at.c, h, at.lone);
                }
            }
            // beyond the last token h is carried along unchanged
            if (p.hT != nullptr && t0 + n == p.T) {
#pragma unroll
                for (int v = 0; v < VEC; ++v)
                    if (v < at.nch) p.hT[at.ch + v] = h[v];
            }
        }
    }
}

template <typename W, bool BETA, bool UNI, bool NT>
__global__ __launch_bounds__(kSingleWaves * 64) void linrec_bwd_kernel(LinrecBwdArgs p, Tiles ts) {
    constexpr int VEC = W::VEC;
    __shared__ Joint<VEC> J;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6, pos = waves - 1 - w;
    const int64_t channels = static_cast<int64_t>(p.B) * p.D, blocks = (p.T - 1) / kTok + 1;
    for (uint32_t turn = 0;; ++turn) {
        uint32_t column;
        int q;                                 // from the last tokens to the first
        if (!next_tile(J, ts, turn, &column, &q)) return;
        const Place<W, UNI> at(ts, column, lane, p.D);
        const int64_t t0 = (static_cast<int64_t>(ts.chain - 1 - q) * waves + w) * kTok;
        const int n = static_cast<int>(p.T - t0 >= kTok ? kTok : p.T > t0 ? p.T - t0 : 0);
        const int64_t row = (at.seq * p.T + t0) * p.D;
        uint32_t xr[kTok], gr[kTok], br[kTok], dr[kTok];
        load_tokens<NT>(p.g, row, at, p.D, n, gr);
        load_tokens<NT>(p.dO, row, at, p.D, n, dr);
        load_tokens<NT>(p.x, row, at, p.D, n, xr);
        if constexpr (BETA) load_tokens<NT>(p.beta, row, at, p.D, n, br);
        float h[VEC];
        const bool here = at.nch > 0 && n > 0;
        {
            const float* s = p.states + (at.seq * blocks + t0 / kTok) * p.D + at.c;
#pragma unroll
            for (int v = 0; v < VEC; ++v) h[v] = here && v < at.nch ? s[v] : 0.f;
        }
        auto decay = [&](int i, float* a) {
            W::unpack(gr[i], a);
#pragma unroll
            for (int v = 0; v < VEC; ++v) a[v] = __expf(a[v]);
        };
        float A[VEC], r[VEC];
        auto reduce = [&](auto forgets) {
            float a[VEC], d[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) { A[v] = 1.f; r[v] = 0.f; }
#pragma unroll
            for (int i = kTok - 1; i >= 0; --i) {
                decay(i, a);
                W::unpack(dr[i], d);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float e = r[v] + d[v];
                    r[v] = forgets ? apply(a[v], e, 0.f) : a[v] * e;
                    A[v] = forgets ? join(A[v], a[v]) : A[v] * a[v];
                }
            }
        };
        reduce(std::false_type());
        bool forgets = any_forgets<VEC>(A);
        if (__builtin_expect(forgets, 0)) {
            forget_derived(gr);
            forget_derived(dr);
            reduce(std::true_type());
            forgets = any_forgets<VEC>(A);
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) J.wave[pos][lane * VEC + v] = make_float2(A[v], r[v]);
        forget_derived(gr);
        forget_derived(dr);
        wave_start<VEC>(J, ts, w, pos, waves, q, p.dhT, at.ch, channels, at.nch, r);
        if (here) {                            // all lanes go on to the next tile's barrier
            // The states before each token, from the one that the forward pass kept: those of
            // every fourth token first, then, from the last four tokens to the first, the
            // ones between (all sixteen at once do not fit beside the inputs in 128 registers).
            typedef typename W::T T;
            auto advance = [&](int i) {
                float a[VEC], u[VEC], b[VEC];
                decay(i, a);
                W::unpack(xr[i], u);
                if constexpr (BETA) W::unpack(br[i], b);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    if constexpr (BETA) u[v] *= b[v];
                    h[v] = fmaf(a[v], h[v], u[v]);
                }
            };
            if (forgets) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) J.start[w][lane * VEC + v] = r[v];
            }
            constexpr int kPart = 4;
            float start[kTok / kPart][VEC];
            bool finite = true;
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                if (i % kPart == 0) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) start[i / kPart][v] = h[v];
                }
                if (i < kTok - kPart) advance(i);
            }
#pragma unroll
            for (int part = kTok / kPart - 1; part >= 0; --part) {
                float before[kPart][VEC];
                forget_derived(gr);
                forget_derived(xr);
                if constexpr (BETA) forget_derived(br);
#pragma unroll
                for (int v = 0; v < VEC; ++v) h[v] = start[part][v];
#pragma unroll
                for (int i = 0; i < kPart; ++i) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) before[i][v] = h[v];
                    if (i + 1 < kPart) advance(part * kPart + i);
                }
                if (part == kTok / kPart - 1) finite = all_finite<VEC>(before[kPart - 1]);
#pragma unroll
                for (int j = kPart - 1; j >= 0; --j) {
                    const int i = part * kPart + j;
                    float a[VEC], e[VEC], x[VEC], b[VEC], dg[VEC];
                    decay(i, a);
                    W::unpack(dr[i], e);
                    W::unpack(xr[i], x);
                    if constexpr (BETA) W::unpack(br[i], b);
#pragma unroll
                    for (int v = 0; v < VEC; ++v) {
                        e[v] += r[v];
                        r[v] = a[v] * e[v];
                        dg[v] = r[v] * before[j][v];
                        if constexpr (BETA) {
                            x[v] *= e[v];
                            e[v] *= b[v];
                        }
                    }
                    if (i < n) {
                        const int64_t el = row + static_cast<int64_t>(i) * p.D;
                        W::template store<NT>(static_cast<T*>(p.dx) + el + at.c, e, at.lone);
                        W::template store<NT>(static_cast<T*>(p.dg) + el + at.c, dg, at.lone);
                        if constexpr (BETA) W::template store<NT>(static_cast<T*>(p.dbeta) + el + at.c, x, at.lone);
                    }
                }
            }
            if (__builtin_expect(forgets && !(finite && all_finite<VEC>(r)), 0)) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) r[v] = J.start[w][lane * VEC + v];
#pragma unroll 1
                for (int i = n - 1; i >= 0; --i) {
                    float a[VEC], e[VEC], x[VEC], b[VEC], dg[VEC];
                    const float* s = p.states + (at.seq * blocks + t0 / kTok) * p.D + at.c;
#pragma unroll
                    for (int v = 0; v < VEC; ++v) h[v] = v < at.nch ? s[v] : 0.f;
#pragma unroll 1
                    for (int k = 0;; ++k) {
                        const int64_t el = row + static_cast<int64_t>(k) * p.D;
                        W::unpack(load_token<W>(p.x, el, at), x);
                        W::unpack(load_token<W>(p.g, el, at), a);
                        if constexpr (BETA) W::unpack(load_token<W>(p.beta, el, at), b);
#pragma unroll
                        for (int v = 0; v < VEC; ++v) a[v] = __expf(a[v]);
                        if (k == i) break;
#pragma unroll
                        for (int v = 0; v < VEC; ++v) {
                            if constexpr (BETA) x[v] *= b[v];
                            h[v] = apply(a[v], h[v], x[v]);
                        }
                    }
                    const int64_t el = row + static_cast<int64_t>(i) * p.D;
                    W::unpack(load_token<W>(p.dO, el, at), e);
#pragma unroll
                    for (int v = 0; v < VEC; ++v) {
                        e[v] += r[v];
                        r[v] = apply(a[v], e[v], 0.f);
                        dg[v] = a[v] == 0.f ? 0.f : r[v] * h[v];
                        if constexpr (BETA) {
                            x[v] *= e[v];
                            e[v] *= b[v];
                        }
                    }
                    W::template store<NT>(static_cast<T*>(p.dx) + el + at.c, e, at.lone);
                    W::template store<NT>(static_cast<T*>(p.dg) + el + at.c, dg, at.lone);
                    if constexpr (BETA) W::template store<NT>(static_cast<T*>(p.dbeta) + el + at.c, x, at.lone);
                }
            }
            if (p.dh0 != nullptr && t0 == 0) {
#pragma unroll
                for (int v = 0; v < VEC; ++v)
                    if (v < at.nch) p.dh0[at.ch + v] = r[v];
            }
        }
    }
}

// All-ones over the workspace: nothing published, no tile handed out.
__global__ __launch_bounds__(256) void linrec_clear_kernel(uint4* ws, int64_t n) {
    const uint4 ones = make_uint4(~0u, ~0u, ~0u, ~0u);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256)
        ws[i] = ones;
}

// V consecutive channels from element i on: one access of 8 or 16 bytes for V = 4.
template <typename E, int V>
__device__ __forceinline__ void load_channels(const void* base, int64_t i, float* f) {
    if constexpr (V == 4) {
        const float4 v = load4<E>(base, i);
        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    } else {
        f[0] = load_elem<E>(base, i);
    }
}
template <typename E, int V>
__device__ __forceinline__ void store_channels(void* base, int64_t i, const float* f) {
    if constexpr (V == 1) {
        store_elem<E>(base, i, f[0]);
    } else if constexpr (E::bytes == 4) {
        *reinterpret_cast<float4*>(static_cast<float*>(base) + i) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + i) = make_uint2(Bf16Even::pack(f), Bf16Even::pack(f + 2));
    }
}

// One token per sequence: 8 bytes of state and 3 or 4 values per channel, HBM-bound for
// large batches, launch-bound for small ones (256 rows of 2048 channels bf16: 3.6 us).
// A workgroup takes 256 * V channels of one row; rows that share a page are all taken by
// the first of them, in order.
template <typename E, bool BETA, int V>
__global__ __launch_bounds__(kStepThreads) void linrec_step_kernel(LinrecStepArgs p, int per_row) {
    int b = blockIdx.x / per_row;
    const int c = ((blockIdx.x % per_row) * kStepThreads + threadIdx.x) * V;
    const bool on = c < p.D;      // lanes behind the row only help to scan the list
    int page = b;
    bool later = false;
    if (p.slots != nullptr) {
        bool earlier;
        page = slot_of_row(p.slots, p.B, b, &earlier, &later);
        if (page < 0 || page >= p.n_pages || earlier) return;
    }
    const int64_t state = static_cast<int64_t>(page) * p.D + c;
    float h[V];
    if (on) load_channels<F32, V>(p.h, state, h);
    do {
        if (on) {
            const int64_t at = static_cast<int64_t>(b) * p.D + c;
            float u[V], a[V], w[V];
            load_channels<E, V>(p.x, at, u);
            load_channels<E, V>(p.g, at, a);
            if constexpr (BETA) load_channels<E, V>(p.beta, at, w);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if constexpr (BETA) u[v] *= w[v];
                h[v] = apply(__expf(a[v]), h[v], u[v]);
            }
            store_channels<E, V>(p.o, at, h);
        }
        if (later) b = next_sharer(p.slots, p.B, b, page);
    } while (later && b < p.B);
    if (on) store_channels<F32, V>(p.h, state, h);
}

// ---- plans ----

// Tiles of a sequence.  One tile needs no counter, no maps and no clearing of them
// (B=32 T=200 D=2048 bf16: forward 26 us as two tiles, 23 us as one; backward 40 and 37).
int64_t chain_of(int T) {
    if (T <= kSingleWaves * kTok) return 1;
    return (static_cast<int64_t>(T) + kMaxWaves * kTok - 1) / (kMaxWaves * kTok);
}

// Workspace: the counters, the maps, the states; none if a tile covers T.
size_t counter_bytes(size_t channels) { return round_up_256((channels + 63) / 64 * kCounter * 4); }

size_t workspace_bytes(int B, int T, int D) {
    const size_t chain = static_cast<size_t>(chain_of(T)), channels = static_cast<size_t>(B) * D;
    if (chain == 1) return 0;
    return counter_bytes(channels) + round_up_256(chain * channels * 8) +
           round_up_256((chain + kGroup - 1) / kGroup * channels * 4);
}

Tiles plan(int B, int T, int D, int vec, void* ws) {
    Tiles t;
    t.row_lanes = static_cast<uint32_t>((D + vec - 1) / vec);
    t.lanes = static_cast<uint32_t>(B) * t.row_lanes;
    t.columns = (t.lanes + 63) / 64;
    t.chain = static_cast<int>(chain_of(T));
    t.n = t.columns * static_cast<uint32_t>(t.chain);
    char* at = static_cast<char*>(ws);
    t.ticket = reinterpret_cast<uint32_t*>(at);
    const size_t channels = static_cast<size_t>(B) * D;
    at += counter_bytes(channels);
    t.maps = reinterpret_cast<uint64_t*>(at);
    t.after = reinterpret_cast<uint32_t*>(at + round_up_256(t.chain * channels * 8));
    return t;
}

// Waves of a workgroup: what T needs if one tile covers it.
int waves_of(int T) { return chain_of(T) > 1 ? kMaxWaves : (T + kTok - 1) / kTok; }

struct FwdLaunch {
    template <typename W, bool BETA, bool UNI, bool NT>
    static void go(const LinrecArgs& a, const Tiles& t, dim3 grid, dim3 block, hipStream_t s) {
        hipLaunchKernelGGL((linrec_fwd_kernel<W, BETA, UNI, NT>), grid, block, 0, s, a, t);
    }
};
struct BwdLaunch {
    template <typename W, bool BETA, bool UNI, bool NT>
    static void go(const LinrecBwdArgs& a, const Tiles& t, dim3 grid, dim3 block, hipStream_t s) {
        hipLaunchKernelGGL((linrec_bwd_kernel<W, BETA, UNI, NT>), grid, block, 0, s, a, t);
    }
};

template <typename L, typename W, bool BETA, typename Args>
hipError_t launch_tiles(const Args& a, hipStream_t s) {
    const Tiles t = plan(a.B, a.T, a.D, W::VEC, a.ws);
    if (t.chain > 1) {
        const int64_t n = static_cast<int64_t>(workspace_bytes(a.B, a.T, a.D) / 16);
        const int64_t blocks = (n + 255) / 256;
        hipLaunchKernelGGL(linrec_clear_kernel, dim3(static_cast<unsigned>(blocks < 2048 ? blocks : 2048)), dim3(256), 0, s,
                           static_cast<uint4*>(a.ws), n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const dim3 grid(t.n < kMaxGrid ? t.n : kMaxGrid), block(static_cast<unsigned>(waves_of(a.T)) * 64);
    // Rows of whole words: whole waves of them have scalar row addresses (see Place), whole
    // cache lines (128 bytes, 32 words) are streamed.
    if constexpr (!W::kOdd) {
        if (t.row_lanes % 64 == 0) {
            L::template go<W, BETA, true, true>(a, t, grid, block, s);
            return hipGetLastError();
        }
        if (t.row_lanes % 32 == 0) {
            L::template go<W, BETA, false, true>(a, t, grid, block, s);
            return hipGetLastError();
        }
    }
    L::template go<W, BETA, false, false>(a, t, grid, block, s);
    return hipGetLastError();
}

template <typename L, typename W, typename Args>
hipError_t launch_beta(const Args& a, hipStream_t s) {
    return a.beta != nullptr ? launch_tiles<L, W, true>(a, s) : launch_tiles<L, W, false>(a, s);
}

template <typename L, typename Args>
hipError_t launch(int dtype, const Args& a, hipStream_t s) {
    if (dtype == 0) return launch_beta<L, Fp32>(a, s);
    return a.D % 2 == 0 ? launch_beta<L, Bf16Even>(a, s) : launch_beta<L, Bf16Odd>(a, s);
}

template <typename E, bool BETA>
hipError_t launch_step_beta(const LinrecStepArgs& a, hipStream_t s) {
    // four channels a lane where rows start on whole vectors, one otherwise
    const int V = a.D % 4 == 0 ? 4 : 1;
    const int per_row = (a.D + kStepThreads * V - 1) / (kStepThreads * V);
    const dim3 grid(static_cast<unsigned>(a.B) * static_cast<unsigned>(per_row)), block(kStepThreads);
    if (V == 4) hipLaunchKernelGGL((linrec_step_kernel<E, BETA, 4>), grid, block, 0, s, a, per_row);
    else hipLaunchKernelGGL((linrec_step_kernel<E, BETA, 1>), grid, block, 0, s, a, per_row);
    return hipGetLastError();
}

template <typename E>
hipError_t launch_step_dtype(const LinrecStepArgs& a, hipStream_t s) {
    return a.beta != nullptr ? launch_step_beta<E, true>(a, s) : launch_step_beta<E, false>(a, s);
}

}  // namespace

size_t linrec_fwd_workspace_bytes(int, int B, int T, int D) { return workspace_bytes(B, T, D); }
size_t linrec_bwd_workspace_bytes(int, int B, int T, int D) { return workspace_bytes(B, T, D); }

hipError_t launch_linrec_fwd(int dtype, const LinrecArgs& a, hipStream_t s) {
    return launch<FwdLaunch>(dtype, a, s);
}

hipError_t launch_linrec_bwd(int dtype, const LinrecBwdArgs& a, hipStream_t s) {
    return launch<BwdLaunch>(dtype, a, s);
}

hipError_t launch_linrec_step(int dtype, const LinrecStepArgs& a, hipStream_t s) {
    return dtype == 0 ? launch_step_dtype<F32>(a, s) : launch_step_dtype<BF16>(a, s);
}

}  // namespace dr
