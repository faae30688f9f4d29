// The gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t over packed
// sequences: forward, backward and the slot-pool step, with their C entry
// points (contract in include/gdr.h).
//
// The scan.  A token is the affine map h -> a h + b (a = exp(g), b = x), and
// maps compose: (A, B) then (a, b) is (a A, a B + b).  The packed token axis is
// cut into tiles of TT tokens by CC channels without regard to the sequences;
// a token that starts a sequence takes its state from h0 instead of from its
// left and cuts the composition there (a selection, not a product by 0, so that
// nothing of one sequence, NaN included, reaches the next).  One pass over the
// data: a tile is read once into registers, composed by runs of R tokens per
// thread and across the threads, waits for the state that reaches its first
// token, and is then evaluated from registers and written.
//   Between tiles: a tile publishes its composition (A, B), and its outgoing
// state once it knows its incoming one.  A tile looks back from its left
// neighbour to the nearest published state and folds the compositions between
// into it, always in token order and with the same fused multiply-adds, so that
// the bits do not depend on which of the two it found.  A published word says by
// itself that it is there (the workspace is cleared to a NaN pattern that no
// published value has), so that neither side needs a fence or a flag, and a tile
// whose neighbour is done learns its state in one trip to L2.  (With a flag per
// tile behind release and acquire, half of all cycles were waits at the barrier
// behind the look-back.)  Tiles are handed out by a counter in token order, so
// that a tile only ever waits for tiles that are already running; every wait has
// a limit.
//   The backward is the same scan from the end: with mu_t = a_t (dy_t + mu_{t+1})
// a token is the map mu -> a (mu + dy); dx = dy + mu_{t+1}, dg = mu_t h_{t-1}.
//
// Accuracy: a near 1 is applied thousands of times, so its error must have no
// mean.  The hardware's exponential is about 0.3 * 2^-24 low on average just
// below 0, which a memory of 4000 tokens turns into 6e-5 of the state; the
// Taylor polynomial, ending in a fused multiply-add with 1, has a mean error
// below 0.001 * 2^-24 there.  A run's decay is the exponential of its gates' sum:
// the product of its tokens' rounded decays left 1.0e-6 at that memory, the sum
// 3.5e-7 (fp32 states against 64 bits, channels of up to that memory; where all have
// it, 5e-7, and 8e-7 for the gradient of fp32 initial states, whose runs are shorter:
// the random walk of one rounding per run).
//
// What bounds it.  Less than two flops per byte: memory.  The floor of a call is
// its rows' bytes at the copy rate (6.69 TB/s measured); one GB300, device times:
//   forward  32768 x 4096  bf16, fp32 gates   167 us   96 %    (bf16 gates 148 us, 81 %;
//                          fp32, 16384 rows   123 us   98 %)
//   backward 32768 x 4096  bf16, bf16 gates   214 us   94 %    (fp32 gates 275 us, 102 %;
//                          fp32, 16384 rows   200 us  100 %)
//   backward 7001 x 1001   fp32, odd rows      42 us   50 %    (50000 rows 193 us, 78 %)
//   forward  6113 x 2048   bf16, 4 sequences   30 us   50 %
// Long calls of narrow types are held by the chain of one tile's steps (composition,
// fold, look-back, evaluation: about 10,500 cycles at two CTAs per SM, of which the
// look-back is a seventh), which longer tiles spread over more tokens: R is the most
// that registers hold, and tiles are narrow, which also leaves fewer tiles of one
// channel group in flight to look back over (64 channels by half the tokens: 172 and
// 226 us forward and backward; 16 channels by twice: 238 and 277).  Three and four
// smaller CTAs per SM (233 and 287 us forward), a larger window of the look-back (4
// instead of 2 rows: 195 -> 203 us; 16 rows a trip farther back instead of 8: 167 ->
// 172 us) and the look-back as a function of its own (173 -> 213 us) cost more in
// registers than they hid.  Short calls are bound by their first tile's latency and,
// like narrow ones, by the look-back over the tiles in flight; odd rows by
// element-wise copies and stores.
#include <cuda.h>
#include <math.h>

#include <atomic>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "gdr.h"
#include "launch.h"
#include "tc.cuh"

namespace gdr {
namespace {

struct LinrecParams {
    const void* x;   // forward: x; backward: dy
    const void* g;
    const void* h;   // backward: y, the forward's output
    void* out;       // forward: y; backward: dx
    void* dg;
    const float* h0;
    const float* start;  // state before the scan's first token: h0, or the final state's gradient
    float* last;         // state after its last: the final state, or the initial state's gradient
    const int32_t* cu;
    int64_t ldx, ldg, ldh, ldo, lddg;
    int64_t T;
    int N, D;
    int groups;          // channel groups of a tile row
    int rows;            // tile rows of T tokens
    int clustered;       // one cluster of `rows` CTAs per channel group; else more than one row looks back
    int lost;            // LOSE only: the tile row whose copies are not to complete
    unsigned int* head;  // workspace: [0] the tile counter, [1] set when a wait gave up
    unsigned int* words;  // [groups][rows][3][CC]: a tile's outgoing state, A, B; kNothing until published
    unsigned int* err;
};

constexpr int kMaxTileTokens = 512;         // a tile's at most: token numbers are 32-bit, a tile's last one included
constexpr unsigned kNothing = 0xffffffffu;  // a NaN that arithmetic does not give
constexpr int kHeadWords = 64;
constexpr unsigned kScanError = 0x200;  // device error word: a tile's wait gave up

// ---- exp(g) -------------------------------------------------------------------

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

constexpr float kTaylor = 0.25f;  // |g| up to here: the polynomial of degree 6 (next term 1.2e-8)

__device__ __forceinline__ float2 taylor_exp(float2 g) {
    float2 p = __ffma2_rn(g, both(1.f / 720), both(1.f / 120));
    p = __ffma2_rn(g, p, both(1.f / 24));
    p = __ffma2_rn(g, p, both(1.f / 6));
    p = __ffma2_rn(g, p, both(0.5f));
    p = __ffma2_rn(g, p, both(1.f));
    return __ffma2_rn(g, p, both(1.f));
}

__device__ __forceinline__ float taylor_exp(float g) {
    float p = fmaf(g, 1.f / 720, 1.f / 120);
    p = fmaf(g, p, 1.f / 24);
    p = fmaf(g, p, 1.f / 6);
    p = fmaf(g, p, 0.5f);
    p = fmaf(g, p, 1.f);
    return fmaf(g, p, 1.f);
}

// Any g: Cody and Waite's reduction ("Software Manual for the Elementary
// Functions", 1980), g = n ln 2 + r with |r| <= ln 2 / 2 and ln 2 in two parts, the
// polynomial of degree 7 in r (next term 5e-9), and 2^n put into the exponent.
// Below -87.3 the result is not a normal number: 0.
__device__ __forceinline__ float2 reduced_exp(float2 g) {
    constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it leaves the nearest integer in the low bits
    const float2 t = __ffma2_rn(g, both(1.44269504f), both(kRound));
    const float2 n = __fadd2_rn(t, both(-kRound));
    const float2 r = __ffma2_rn(n, both(1.90465e-9f), __ffma2_rn(n, both(-0.693147182f), g));
    float2 p = __ffma2_rn(r, both(1.f / 5040), both(1.f / 720));
    p = __ffma2_rn(r, p, both(1.f / 120));
    p = __ffma2_rn(r, p, both(1.f / 24));
    p = __ffma2_rn(r, p, both(1.f / 6));
    p = __ffma2_rn(r, p, both(0.5f));
    p = __ffma2_rn(r, p, both(1.f));
    p = __ffma2_rn(r, p, both(1.f));
    const float2 power = make_float2(__uint_as_float((__float_as_uint(t.x) << 23) + 0x3f800000u),
                                     __uint_as_float((__float_as_uint(t.y) << 23) + 0x3f800000u));
    const float2 e = __fmul2_rn(p, power);  // NaN stays NaN
    return make_float2(g.x < -87.3f ? 0.f : e.x, g.y < -87.3f ? 0.f : e.y);
}

template <int N>
__device__ __forceinline__ void exp_of(float (&g)[N], float2 (*f)(float2)) {
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        const int k = j + 1 < N ? j + 1 : j;
        const float2 e = f(make_float2(g[j], g[k]));
        g[j] = e.x;
        g[k] = e.y;
    }
}

// Of all N gates of a thread, in place.  Whether any is beyond the short
// polynomial is asked once, by the warp as a whole.
template <int N>
__device__ __forceinline__ void decays(float (&g)[N]) {
    float most[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < N; ++j) most[j % 4] = fmaxf(most[j % 4], fabsf(g[j]));
    if (__any_sync(0xffffffffu, fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])) > kTaylor)) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float far = expf(g[j]), near = taylor_exp(g[j]);
            g[j] = fabsf(g[j]) > kTaylor ? far : near;
        }
    } else {
        exp_of(g, taylor_exp);
    }
}

// ---- a thread's elements of a row, kept as they are stored -------------------------
//
// kNext: 8 neighbours, one 16-byte access of bf16.  kHalves: two runs of four, `d`
// elements from one another: a warp's 16-byte accesses to fp32 rows in shared memory
// then touch all banks in turn, and its stores whole sectors.  kApart: two elements 32
// apart, for rows of any alignment: a warp's accesses are 32 neighbours.  `n` says
// which lie inside the tensor: all or none (kNext), bit 0 and bit 1 for the runs
// (kHalves), how many (kApart).

enum Layout { kNext, kHalves, kApart };

template <typename T, Layout L> struct Row;

template <Layout L> struct Row<__nv_bfloat16, L> {
    uint4 v;
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p, int d) {
        if (L == kNext) {
            v = *reinterpret_cast<const uint4*>(p);
        } else {
            const uint2 a = *reinterpret_cast<const uint2*>(p), b = *reinterpret_cast<const uint2*>(p + d);
            v = make_uint4(a.x, a.y, b.x, b.y);
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[8], int n, int d) {
        const uint2 a = make_uint2(tc::pack_bf16(f[0], f[1]), tc::pack_bf16(f[2], f[3]));
        const uint2 b = make_uint2(tc::pack_bf16(f[4], f[5]), tc::pack_bf16(f[6], f[7]));
        if (L == kNext) {
            *reinterpret_cast<uint4*>(p) = make_uint4(a.x, a.y, b.x, b.y);
        } else {
            if (n & 1) *reinterpret_cast<uint2*>(p) = a;
            if (n & 2) *reinterpret_cast<uint2*>(p + d) = b;
        }
    }
};
template <> struct Row<__nv_bfloat16, kApart> {
    uint32_t v;
    __device__ __forceinline__ void zero() { v = 0; }
    __device__ __forceinline__ void load(const __nv_bfloat16* p, int) {
        const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
        v = u[0] | u[32] << 16;
    }
    __device__ __forceinline__ void get(float (&f)[2]) const {
        f[0] = __uint_as_float(v << 16);
        f[1] = __uint_as_float(v & 0xffff0000u);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[2], int n, int) {
        if (n > 0) p[0] = __float2bfloat16_rn(f[0]);
        if (n > 1) p[32] = __float2bfloat16_rn(f[1]);
    }
};
template <Layout L> struct Row<float, L> {
    float v[8];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
    }
    __device__ __forceinline__ void load(const float* p, int d, int n = 3) {
        if (n & 1) {
            const float4 a = *reinterpret_cast<const float4*>(p);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        }
        if (n & 2) {
            const float4 b = *reinterpret_cast<const float4*>(p + (L == kHalves ? d : 4));
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = v[j];
    }
    static __device__ __forceinline__ void store(float* p, const float (&f)[8], int n, int d) {
        if (n & 1) *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
        if (n & 2) *reinterpret_cast<float4*>(p + (L == kHalves ? d : 4)) = make_float4(f[4], f[5], f[6], f[7]);
    }
};
template <> struct Row<float, kApart> {
    float v[2];
    __device__ __forceinline__ void zero() { v[0] = v[1] = 0.f; }
    __device__ __forceinline__ void load(const float* p, int, int n = 2) {
        if (n > 0) v[0] = p[0];
        if (n > 1) v[1] = p[32];
    }
    __device__ __forceinline__ void get(float (&f)[2]) const {
        f[0] = v[0];
        f[1] = v[1];
    }
    static __device__ __forceinline__ void store(float* p, const float (&f)[2], int n, int) {
        if (n > 0) p[0] = f[0];
        if (n > 1) p[32] = f[1];
    }
};

template <int N> __device__ __forceinline__ float2 pair(const float (&f)[N], int i) {
    return make_float2(f[2 * i], f[2 * i + 1]);
}
template <int N> __device__ __forceinline__ void put(float (&f)[N], int i, float2 v) {
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
}

// One token of the scan: h <- a h + b, or h <- a (h + b) from the end.
template <bool BWD, int N>
__device__ __forceinline__ void advance(float (&h)[N], const float (&a)[N], const float (&b)[N]) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
        put(h, i, BWD ? __fmul2_rn(pair(a, i), __fadd2_rn(pair(h, i), pair(b, i)))
                      : __ffma2_rn(pair(a, i), pair(h, i), pair(b, i)));
}
template <int N> __device__ __forceinline__ void add(float (&f)[N], const float (&s)[N]) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) put(f, i, __fadd2_rn(pair(f, i), pair(s, i)));
}
template <int N> __device__ __forceinline__ void product(float (&o)[N], const float (&a)[N], const float (&b)[N]) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) put(o, i, __fmul2_rn(pair(a, i), pair(b, i)));
}

// ---- the tile kernel --------------------------------------------------------------

// WIDE: 32 channels per tile, 8 per thread, aligned rows, staged by TMA.  Otherwise 64
// channels, 2 per thread and a run of tokens per warp, so that the element-wise accesses
// of a warp are neighbours (with 8 per thread: backward 7001 x 1001 fp32 47 -> 43 us,
// 50000 x 1001 bf16 forward 125 -> 104, backward 215 -> 157).  Each row's segment is
// staged by a bulk copy of the 16-byte blocks around it, and read from where it lies in
// them: about 110 cycles of a warp each to issue, so six warps issue them while two look
// back (one warp for all took 17,600 cycles of a tile; 4-byte asynchronous copies by all
// warps before the fold took 3,200 to 10,700).
template <typename TX, typename TG, bool BWD, bool WIDE> struct Tile {
    static constexpr int THREADS = 256, CTAS = 2, WARPS = THREADS / 32;
    static constexpr int COPIERS = WARPS - 2;  // warps that issue bulk copies, while the others look back
    static constexpr int E = WIDE ? 8 : 2, LANES = WIDE ? 4 : 32, CC = E * LANES, RUNS = THREADS / LANES;  // runs of R tokens
    // Of 8 channels a token takes 8 registers for its decays and 4 or 8 for each of b
    // and h as stored; R is the most that fits beside the rest in 128 registers (one
    // more spilled: forward 151 -> 157 us with bf16 gates, backward 226 -> 235 us) and
    // in shared memory at two CTAs per SM.  Four times as many at 2 channels, where two
    // more fit but gain nothing.
    static constexpr int R = sizeof(TX) == 2 ? (BWD ? (WIDE ? 5 : 16) : WIDE ? 7 : 24) : (BWD ? (WIDE ? 3 : 12) : WIDE ? 5 : 20);
    static constexpr int TT = RUNS * R;
    // The fold over runs, in parts.  The 8 runs of the tiles that are not WIDE are one part,
    // folded by the two warps that look back while the others already copy (all warps in
    // four parts, then the copies: 7001 x 1001 backward 43.1 us, so 42.5).
    static constexpr int PARTS = WIDE ? THREADS / CC : 1, RUNS_PART = RUNS / PARTS;
    static constexpr Layout LAYOUT = !WIDE ? kApart : sizeof(TX) == 4 || sizeof(TG) == 4 ? kHalves : kNext;
    // bytes of a token in the stage, a row of x / h and one of g
    static constexpr int PITCH_X = CC * (int)sizeof(TX) + (WIDE ? 0 : 16), PITCH_G = CC * (int)sizeof(TG) + (WIDE ? 0 : 16);
    // shared memory (bytes)
    static constexpr int XS = 0, GS = XS + TT * PITCH_X, HS = GS + TT * PITCH_G, STAGE = HS + (BWD ? TT * PITCH_X : 0);
    static constexpr int CA = STAGE, CB = CA + RUNS * CC * 4, PA = CB + RUNS * CC * 4, PB = PA + PARTS * CC * 4;
    static constexpr int TA = PB + PARTS * CC * 4, TB = TA + CC * 4, CARRY = TB + CC * 4;
    static constexpr int FIRST = CARRY + CC * 4, LAST = FIRST + 2 * TT * 4, CUT = LAST + 2 * TT * 4;
    static constexpr int MISC = CUT + RUNS * 4, BYTES_SMEM = MISC + 64;
    static constexpr int BOX = TT > 256 ? TT / 2 : TT;  // tokens of a TMA copy
    static_assert(TT <= kMaxTileTokens, "T_total's limit");
    static_assert(RUNS % PARTS == 0 && STAGE % 128 == 0 && TT % BOX == 0 && BOX <= 256 && BOX * CC * 2 % 128 == 0, "tile shape");
    static_assert(CTAS * (BYTES_SMEM + 1024) <= 228 * 1024, "shared memory of the CTAs of an SM");
    // A lane's first channel, and how far its second run of four is (kHalves: runs of
    // odd number begin with the second half, so that the two runs that share a
    // quarter of a warp's access take different banks).
    static __device__ __forceinline__ int channel(int lane, int run) {
        return LAYOUT == kNext ? lane * 8 : LAYOUT == kHalves ? lane * 4 + (run & 1) * (CC / 2) : lane;
    }
    static __device__ __forceinline__ int apart(int run) { return LAYOUT == kHalves && (run & 1) ? -CC / 2 : CC / 2; }
    // Which of its channels lie below D, from its first one.
    static __device__ __forceinline__ int inside(int c, int d, int D) {
        return LAYOUT == kNext ? (c < D ? 3 : 0) : LAYOUT == kHalves ? (c < D ? 1 : 0) + (c + d < D ? 2 : 0)
                                                                     : (c < D ? 1 : 0) + (c + 32 < D ? 1 : 0);
    }
    // A run's values of a lane's channels in the arrays of compositions.
    static __device__ __forceinline__ float* place(float* c, int lane, int run, int k) {
        return c + run * CC + (WIDE ? lane * 4 + (LAYOUT == kHalves ? k ^ (run & 1) : k) * (CC / 2) : lane + k * 32);
    }
    static __device__ __forceinline__ void put_run(float* c, int lane, int run, const float (&f)[E]) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float* q = place(c, lane, run, k);
            if constexpr (WIDE)
                *reinterpret_cast<float4*>(q) = make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
            else
                *q = f[k];
        }
    }
    static __device__ __forceinline__ void get_run(float* c, int lane, int run, float (&f)[E]) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float* q = place(c, lane, run, k);
            if constexpr (WIDE) {
                const float4 u = *reinterpret_cast<const float4*>(q);
                f[4 * k] = u.x; f[4 * k + 1] = u.y; f[4 * k + 2] = u.z; f[4 * k + 3] = u.w;
            } else {
                f[k] = *q;
            }
        }
    }
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int c, int t, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        :: "r"(dst), "l"(map), "r"(c), "r"(t), "r"(mbar) : "memory");
}

__device__ __forceinline__ void expect_bytes(uint32_t mbar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(mbar), "r"(bytes) : "memory");
}

// The segment [c, c + 64) of one row of a tensor into its stage row: the 16-byte
// blocks around it by one bulk copy, and what of them lies outside the tensor (in
// rows near its ends) left out, the elements there copied one by one.
template <typename T>
__device__ __forceinline__ void copy_segment(unsigned char* dst, const void* tensor, int64_t ld, int64_t T_all, int D,
                                             int64_t row, int c, uint32_t mbar) {
    constexpr int ES = (int)sizeof(T);
    const uintptr_t base = reinterpret_cast<uintptr_t>(tensor), end = base + ((T_all - 1) * ld + D) * ES;
    const uintptr_t at = base + (row * ld + c) * ES, stop = at + min(64, D - c) * ES;
    const uintptr_t first = at & ~uintptr_t(15);  // where dst begins
    uintptr_t lo = first, hi = (stop + 15) & ~uintptr_t(15);
    if (lo < base) lo = (base + 15) & ~uintptr_t(15);
    if (hi > end) hi = end & ~uintptr_t(15);
    if (hi > lo) {
        const uint32_t bytes = (uint32_t)(hi - lo);
        expect_bytes(mbar, bytes);
        tc::bulk_g2s(tc::smem_u32(dst) + (uint32_t)(lo - first), reinterpret_cast<const void*>(lo), bytes, mbar);
    } else {
        lo = hi = stop;
    }
    for (uintptr_t e = at; e < stop; e += ES)
        if (e < lo || e >= hi) {
            *reinterpret_cast<T*>(dst + (e - first)) = *reinterpret_cast<const T*>(e);
        } else {
            e = hi - ES;
        }
}

__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float cluster_read(const void* own, unsigned rank) {
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(own)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ unsigned peek(const unsigned int* p) {
    unsigned v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void publish(unsigned int* p, float f) {
    unsigned v = __float_as_uint(f);
    if (v == kNothing) v = 0x7fffffffu;  // some other NaN
    asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" :: "l"(p), "r"(v) : "memory");
}

// The words of the rows left of `row` in one channel, nearest first.  `w`: that
// channel's words of row 0, rows `pitch` apart, fields `field` apart (state, A, B).
struct Neighbours {
    static constexpr int W = 2;
    unsigned s[W], a[W], b[W];

    __device__ __forceinline__ void peek_at(const unsigned int* w, int row, int64_t pitch, int field) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const unsigned int* q = w + max(row - 1 - i, 0) * pitch;
            s[i] = peek(q);
            a[i] = peek(q + field);
            b[i] = peek(q + 2 * field);
        }
    }
    // Whether a state is among them with every map behind it; `whole`: every row is
    // at least composed.
    __device__ __forceinline__ bool reach(float& state, bool& whole) const {
        bool known = false;
        float h = 0.f;
        whole = true;
#pragma unroll
        for (int i = W - 1; i >= 0; --i) {  // from the farthest: a state there starts anew, a map is applied
            if (s[i] != kNothing) {
                h = __uint_as_float(s[i]);
                known = true;
            } else if (a[i] != kNothing && b[i] != kNothing) {
                h = fmaf(__uint_as_float(a[i]), h, __uint_as_float(b[i]));
            } else {
                known = whole = false;
            }
        }
        state = h;
        return known;
    }
};

// The state that reaches a tile of row `row` in one channel, waited for.  False if
// a wait gave up.
__device__ __forceinline__ bool look_back(const unsigned int* w, int row, int64_t pitch, int field, float& state,
                                          const unsigned int* gave_up) {
    const uint64_t began = tc::globaltimer_ns();
    unsigned spin = 0;
    auto patience = [&]() {
        return (++spin & 63) != 0 || (!peek(gave_up) && tc::globaltimer_ns() - began < tc::kWaitLimitNs);
    };
    while (true) {
        Neighbours near;
        bool whole;
        near.peek_at(w, row, pitch, field);
        if (near.reach(state, whole)) return true;
        if (whole && row > Neighbours::W) break;
        if (!patience()) return false;
    }
    // further: the nearest state, then forward over the maps
    int k = row - 1 - Neighbours::W;
    constexpr int V = 8;
    while (true) {
        unsigned s[V];
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = peek(w + max(k - i, 0) * pitch);
        int at = -1;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
            if (s[i] != kNothing) at = i;
        if (at >= 0) {
            k = max(k - at, 0);
            state = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i == at) state = __uint_as_float(s[i]);
            break;
        }
        if (k >= V)
            k -= V;
        else if (!patience())
            return false;
    }
    for (++k; k < row;) {
        unsigned s[V], a[V], b[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const unsigned int* q = w + min(k + i, row - 1) * pitch;
            s[i] = peek(q);  // a tile that is cut publishes nothing else
            a[i] = peek(q + field);
            b[i] = peek(q + 2 * field);
        }
        bool ready = true;
        int n = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool map = a[i] != kNothing && b[i] != kNothing;
            ready = ready && k + i < row && (s[i] != kNothing || map);
            if (ready) {
                state = s[i] != kNothing ? __uint_as_float(s[i])
                                         : fmaf(__uint_as_float(a[i]), state, __uint_as_float(b[i]));
                ++n;
            }
        }
        k += n;
        if (!n && !patience()) return false;
    }
    return true;
}

// The sequences that begin and end in the tile of tokens [t0, t0 + TT): by the
// order of the scan, first[i] / last[i] is the sequence whose scan starts before
// token i / ends after it, or -1.  One warp; returns whether there is any.
template <int TT, bool BWD>
__device__ bool find_boundaries(const int32_t* cu, int N, int t0, int* first, int* last, int lane) {
    // smallest m in [0, N] with cu[m] >= t0 (N + 1 if none), 32 probes at a time
    int lo = 0, n = N + 1;
    while (n > 0) {
        const int step = (n + 31) / 32;
        const int m = lo + lane * step;  // the first element of this lane's piece
        const unsigned less = __ballot_sync(0xffffffffu, m < lo + n && cu[min(m, N)] < t0);
        if (!less) break;
        const int k = 31 - __clz(less);  // the boundary lies in piece k, behind its first element
        const int end = min(lo + (k + 1) * step, lo + n);
        lo += k * step + 1;
        n = end - lo;
    }
    int m = lo + lane, at = m <= N ? cu[m] : 0x7fffffff;
    bool in = at >= t0 && at - t0 <= TT;
    if (!__any_sync(0xffffffffu, in)) return false;
    for (int i = lane; i < TT; i += 32) first[i] = last[i] = -1;
    __syncwarp();
    while (true) {
        if (in) {
            const int k = at - t0;  // between tokens k - 1 and k of the tile
            if (k < TT && m < N && cu[m + 1] > at) (BWD ? last : first)[BWD ? TT - 1 - k : k] = m;
            if (k > 0 && m > 0 && cu[m - 1] < at) (BWD ? first : last)[BWD ? TT - k : k - 1] = m - 1;
        }
        // sorted: once a lane is beyond the tile, so is everything after it
        if (__any_sync(0xffffffffu, m >= N || (int64_t)at - t0 > TT)) break;
        m += 32;
        at = m <= N ? cu[m] : 0x7fffffff;
        in = at >= t0 && at - t0 <= TT;
    }
    return true;
}

// LOSE: tiles of row p.lost wait for 16 bytes that nobody copies, for the test of the
// way out.
template <typename TX, typename TG, bool BWD, bool WIDE, bool LOSE>
__global__ void __launch_bounds__(Tile<TX, TG, BWD, WIDE>::THREADS, Tile<TX, TG, BWD, WIDE>::CTAS)
linrec_tile_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_g,
                   const __grid_constant__ CUtensorMap map_h, const __grid_constant__ LinrecParams p) {
    using C = Tile<TX, TG, BWD, WIDE>;
    constexpr int CC = C::CC, E = C::E, R = C::R, TT = C::TT;
    constexpr Layout L = C::LAYOUT;
    extern __shared__ __align__(1024) unsigned char smem[];
    float* ca = reinterpret_cast<float*>(smem + C::CA);
    float* cb = reinterpret_cast<float*>(smem + C::CB);
    float* pa = reinterpret_cast<float*>(smem + C::PA);
    float* pb = reinterpret_cast<float*>(smem + C::PB);
    float* carry_s = reinterpret_cast<float*>(smem + C::CARRY);
    int* cut_s = reinterpret_cast<int*>(smem + C::CUT);
    uint64_t* mbar_s = reinterpret_cast<uint64_t*>(smem + C::MISC);
    // next tile, copies lost, boundaries of either buffer, cut, state lost
    int* misc = reinterpret_cast<int*>(smem + C::MISC + 16);
    // Either is set in front of one barrier and looked at behind it, and not set in
    // between, so that all threads of the CTA leave at the same place.
    volatile int* abort_s = misc + 1;  // the tile's copies did not land
    volatile int* stop_s = misc + 5;   // the state that reaches the tile did not arrive
    const uint32_t mbar = tc::smem_u32(mbar_s);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int lc = lane % C::LANES, run = warp * (32 / C::LANES) + lane / C::LANES;
    const int lane_c = C::channel(lc, run), apart = C::apart(run);
    const int part = tid / CC, pos = tid % CC;
    const bool many = p.rows > 1 && !p.clustered;

    if (tid == 0) {
        tc::mbar_init(mbar, WIDE ? 1 : 32 * C::COPIERS);
        tc::mbar_fence_init();
        *abort_s = *stop_s = 0;
    }
    const int valid = min((int64_t)max(p.cu[p.N], 0), p.T);
    const int rows = (valid + TT - 1) / TT;  // tile rows that hold a sequence's token
    const int64_t tiles = (int64_t)rows * p.groups;

    // tiles are taken in the order of the scan, all channel groups of a row first
    auto token0 = [&](int tile) -> int {
        const int row = tile / p.groups;
        return (BWD ? rows - 1 - row : row) * TT;
    };
    auto request = [&](int tile) {  // the tile's rows into the stage; one thread, or if not WIDE the copiers
        const int c = tile % p.groups * CC, t0 = token0(tile);
        if constexpr (WIDE) {
            tc::mbar_arrive_tx(mbar, C::STAGE + (LOSE && tile / p.groups == p.lost ? 16 : 0));
            for (int l = 0; l < TT; l += C::BOX) {
                tma_load_2d(tc::smem_u32(smem + C::XS + l * C::PITCH_X), &map_x, c, t0 + l, mbar);
                tma_load_2d(tc::smem_u32(smem + C::GS + l * C::PITCH_G), &map_g, c, t0 + l, mbar);
                if (BWD)  // row t - 1 beside token t
                    tma_load_2d(tc::smem_u32(smem + C::HS + l * C::PITCH_X), &map_h, c, t0 + l - 1, mbar);
            }
        } else {
            // What earlier tiles had copied into the stage element by element, and all have
            // read behind a barrier, before the bulk copies that may write the same bytes.
            tc::fence_proxy_async();
            for (int l = warp - 2 + C::COPIERS * lane; l < min(TT, valid - t0); l += 32 * C::COPIERS) {
                const int64_t t = t0 + l;
                copy_segment<TX>(smem + C::XS + l * C::PITCH_X, p.x, p.ldx, p.T, p.D, t, c, mbar);
                copy_segment<TG>(smem + C::GS + l * C::PITCH_G, p.g, p.ldg, p.T, p.D, t, c, mbar);
                if (BWD && t > 0) copy_segment<TX>(smem + C::HS + l * C::PITCH_X, p.h, p.ldh, p.T, p.D, t - 1, c, mbar);
            }
            if (LOSE && warp == 2 && lane == 0 && tile / p.groups == p.lost) expect_bytes(mbar, 16);
            tc::mbar_arrive(mbar);
        }
    };
    // where row t's segment from channel c on begins in its blocks
    auto shift = [&](const void* tensor, int64_t ld, int c, int t, int size) {
        return WIDE ? 0 : (int)(reinterpret_cast<uintptr_t>(tensor) + c * size + (t & 15) * ((int)ld & 15) * size) & 15;
    };

    if (many) tc::grid_dep_wait();  // the workspace has been cleared

    bool met = false;  // this CTA has been at its cluster's first meeting
    if (tid == 0) {
        int64_t t = blockIdx.x;  // one tile of each CTA: a row of the cluster, or a group of the only row
        if (many) t = atomicAdd(p.head, 1u);
        if (p.clustered) t = (int)(blockIdx.x % p.rows) < rows ? (int64_t)(blockIdx.x % p.rows) * p.groups + blockIdx.x / p.rows : tiles;
        misc[0] = t < tiles ? (int)t : -1;
    }
    __syncthreads();
    int tile = misc[0];
    __syncthreads();
    if (tile >= 0 && (WIDE ? tid == 0 : warp >= 2)) request(tile);
    if (tile >= 0 && warp == C::WARPS - 1) {
        const bool any = find_boundaries<TT, BWD>(p.cu, p.N, token0(tile), reinterpret_cast<int*>(smem + C::FIRST),
                                                  reinterpret_cast<int*>(smem + C::LAST), lane);
        if (lane == 0) misc[2] = any;
    }

    for (int it = 0; tile >= 0; ++it) {
        const int buf = it & 1;
        const int row = tile / p.groups, group = tile - row * p.groups, t0 = (BWD ? rows - 1 - row : row) * TT;
        const int c0 = group * CC + lane_c, inside = C::inside(c0, apart, p.D);
        const int* first = reinterpret_cast<int*>(smem + C::FIRST) + buf * TT;
        const int* last = reinterpret_cast<int*>(smem + C::LAST) + buf * TT;
        unsigned next = 0xffffffffu;  // looked at after the composition: the counter's answer takes its time
        if (many && tid == 0)
            asm volatile("atom.relaxed.gpu.global.add.u32 %0, [%1], 1;" : "=r"(next) : "l"(p.head) : "memory");
        if (!tc::mbar_wait(mbar, buf, abort_s)) {
            *abort_s = 1;
            atomicOr(p.err, kScanError);
        }
        __syncthreads();
        const bool bounded = misc[2 + buf] != 0;  // sequences begin or end in the tile

        // ---- into registers, and the composition of the thread's run.  The gates
        // first and their exponentials, then the rest: the most registers at a time are
        // those held to the tile's end anyway.  TMA has filled with zeros what lies
        // outside the tensors; what was not staged (channels that are none, the row
        // before the first) and rows behind the last sequence become the identity here.
        const bool full = t0 + TT <= valid;
        auto local = [&](int r) { return BWD ? TT - 1 - (run * R + r) : run * R + r; };  // the run's token r in the tile
        float a[R][E], A[E];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int l = local(r);
            Row<TG, L> gr;
            gr.load(reinterpret_cast<const TG*>(smem + C::GS + l * C::PITCH_G +
                                                shift(p.g, p.ldg, group * CC, t0 + l, sizeof(TG))) + lane_c, apart);
            gr.get(a[r]);
        }
        if (!full || (!WIDE && inside < E)) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int j = 0; j < E; ++j)
                    if (t0 + local(r) >= valid || (!WIDE && j >= inside)) a[r][j] = 0.f;  // exp(0) = 1
        }
        // The run's decay is the exponential of its gates' sum: the product of its
        // tokens' decays would carry the rounding of each, as the runs' do after it.
#pragma unroll
        for (int j = 0; j < E; ++j) A[j] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) add(A, a[r]);
        decays(A);
        C::put_run(ca, lc, run, A);
        decays(reinterpret_cast<float (&)[R * E]>(a));
        Row<TX, L> b[R], h[BWD ? R : 1];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int l = local(r);
            b[r].load(reinterpret_cast<const TX*>(smem + C::XS + l * C::PITCH_X +
                                                  shift(p.x, p.ldx, group * CC, t0 + l, sizeof(TX))) + lane_c, apart);
            if (BWD)
                h[r].load(reinterpret_cast<const TX*>(smem + C::HS + l * C::PITCH_X +
                                                      shift(p.h, p.ldh, group * CC, t0 + l - 1, sizeof(TX))) + lane_c, apart);
        }
        if (!full) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (t0 + local(r) >= valid) b[r].zero();
        }
        if (BWD && !WIDE && t0 == 0) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (local(r) == 0) h[r].zero();
        }
        float B[E];
#pragma unroll
        for (int j = 0; j < E; ++j) B[j] = 0.f;
        auto start_state = [&](int n, float (&f)[E]) {
            Row<float, L> s;
            s.zero();
            if (p.start && inside) s.load(p.start + (int64_t)n * p.D + c0, apart, inside);
            s.get(f);
        };
        int cut = 0;
        // twice in the code: tiles in which a sequence begins or ends, and the others
        auto compose = [&](auto cutting) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float f[E];
                b[r].get(f);
                if (decltype(cutting)::value) {
                    const int n = first[run * R + r];
                    if (n >= 0) {
                        start_state(n, B);
                        cut = 1;
                    }
                }
                advance<BWD, E>(B, a[r], f);
            }
        };
        bounded ? compose(std::true_type()) : compose(std::false_type());
        C::put_run(cb, lc, run, B);
        if (lc == 0) cut_s[run] = cut;
        if (tid == 0) misc[0] = (int64_t)next < tiles ? (int)next : -1;
        __syncthreads();
        if (*abort_s) {
            if (tid == 0) tc::mbar_wait_copies(mbar, buf);  // none may land after the CTA
            break;
        }
        const int ntile = misc[0];
        if (WIDE && tid == 0 && ntile >= 0) request(ntile);  // the stage has been read

        // The left neighbours' words are asked for before the fold, and looked at behind it.
        constexpr int64_t pitch = 3 * CC;
        unsigned int* words = p.words + (int64_t)group * p.rows * pitch + pos;
        Neighbours near;
        const bool looks = many && tid < CC && row > 0;
        if (looks) near.peek_at(words, row, pitch, CC);

        // ---- the runs of each part, then the parts: the tile's composition
        auto fold = [&](auto cutting) {
            float fa = 1.f, fb = 0.f;
#pragma unroll
            for (int i = 0; i < C::RUNS_PART; ++i) {
                const int at = part * C::RUNS_PART + i;
                const float ra = ca[at * CC + pos], rb = cb[at * CC + pos];
                if (decltype(cutting)::value && cut_s[at]) {
                    fb = rb;
                } else {
                    fb = fmaf(ra, fb, rb);
                    fa *= ra;
                }
            }
            pa[part * CC + pos] = fa;
            pb[part * CC + pos] = fb;
        };
        if (part < C::PARTS) bounded ? fold(std::true_type()) : fold(std::false_type());
        // whether a part is cut: read from cut_s by everyone alike
        auto part_cut = [&](int q) {
            int c = 0;
            if (bounded)
                for (int i = q * C::RUNS_PART; i < (q + 1) * C::RUNS_PART; ++i) c |= cut_s[i];
            return c != 0;
        };
        if (C::PARTS > 1) __syncthreads();
        if (warp == C::WARPS - 1 && ntile >= 0) {  // while others look back: the next tile's sequences
            const int nb = buf ^ 1;
            const bool any = find_boundaries<TT, BWD>(p.cu, p.N, token0(ntile),
                                                      reinterpret_cast<int*>(smem + C::FIRST) + nb * TT,
                                                      reinterpret_cast<int*>(smem + C::LAST) + nb * TT, lane);
            if (lane == 0) misc[2 + nb] = any;
        }
        if (!WIDE && warp >= 2 && ntile >= 0) request(ntile);  // and its rows, in many small copies
        float fa = 1.f, fb = 0.f;  // of the tile, in the threads of the first part
        bool cut_any = false;
        if (p.rows > 1 && tid < CC) {
#pragma unroll
            for (int q = 0; q < C::PARTS; ++q) {
                const float ra = pa[q * CC + pos], rb = pb[q * CC + pos];
                if (part_cut(q)) {
                    fb = rb;
                    cut_any = true;
                } else {
                    fb = fmaf(ra, fb, rb);
                    fa *= ra;
                }
            }
        }
        if (p.clustered) {  // the compositions of the cluster's tiles are read from their CTAs
            float* ta = reinterpret_cast<float*>(smem + C::TA);
            float* tb = reinterpret_cast<float*>(smem + C::TB);
            if (tid < CC) {
                ta[pos] = fa;
                tb[pos] = fb;
            }
            if (tid == 0) misc[4] = cut_any;
            cluster_meet();
            met = true;
            if (tid < CC) {
                float carry = 0.f;
                for (int k = 0; k < row; ++k) {
                    if (__float_as_int(cluster_read(misc + 1, k))) *stop_s = 1;  // that tile was not composed
                    const float ra = cluster_read(ta + pos, k), rb = cluster_read(tb + pos, k);
                    carry = __float_as_int(cluster_read(misc + 4, k)) || k == 0 ? rb : fmaf(ra, carry, rb);
                }
                carry_s[pos] = carry;
            }
        } else if (many && tid < CC) {
            unsigned int* own = words + row * pitch;
            const bool settled = cut_any || row == 0;  // the outgoing state does not depend on the incoming one
            float carry = 0.f;
            bool whole, known = looks && near.reach(carry, whole);
            if (settled) {
                publish(own, fb);
            } else if (!known) {
                publish(own + CC, fa);
                publish(own + 2 * CC, fb);
            }
            if (looks) {
                if (!known && !look_back(words, row, pitch, CC, carry, p.head + 1)) {
                    *stop_s = 1;
                    p.head[1] = 1;
                    atomicOr(p.err, kScanError);
                }
                if (!settled) publish(own, fmaf(fa, carry, fb));
            }
            carry_s[pos] = carry;
        }
        __syncthreads();
        if (*stop_s) {
            if (tid == 0 && ntile >= 0) tc::mbar_wait_copies(mbar, buf ^ 1);
            break;
        }
        // ---- the state that reaches each run
        auto walk = [&](auto cutting) {
            float f = p.rows > 1 ? carry_s[pos] : 0.f;
            for (int q = 0; q < part; ++q)
                f = decltype(cutting)::value && part_cut(q) ? pb[q * CC + pos] : fmaf(pa[q * CC + pos], f, pb[q * CC + pos]);
#pragma unroll
            for (int i = 0; i < C::RUNS_PART; ++i) {
                const int at = part * C::RUNS_PART + i;
                const float ra = ca[at * CC + pos], rb = cb[at * CC + pos];
                ca[at * CC + pos] = f;
                f = decltype(cutting)::value && cut_s[at] ? rb : fmaf(ra, f, rb);
            }
        };
        if (part < C::PARTS) bounded ? walk(std::true_type()) : walk(std::false_type());
        __syncthreads();
        if (inside) {
            float s[E];
            C::get_run(ca, lc, run, s);
            // ---- every token from its state
            const int64_t t_first = t0 + (BWD ? TT - 1 - run * R : run * R), dir = BWD ? -1 : 1;
            TX* out = static_cast<TX*>(p.out) + t_first * p.ldo + c0;
            TG* dg = BWD ? static_cast<TG*>(p.dg) + t_first * p.lddg + c0 : nullptr;
            auto evaluate = [&](auto cutting) {  // cutting: or rows behind the last sequence
#pragma unroll
                for (int r = 0; r < R; ++r, out += dir * p.ldo, dg += BWD ? -p.lddg : 0) {
                    int n_last = -1;
                    if (decltype(cutting)::value) {
                        if (t_first + dir * r >= valid) continue;
                        if (bounded) {
                            const int n = first[run * R + r];
                            n_last = last[run * R + r];
                            if (n >= 0) start_state(n, s);
                        }
                    }
                    float f[E];
                    b[r].get(f);
                    if (BWD) {
                        float before[E];
                        add(f, s);  // lam
                        Row<TX, L>::store(out, f, inside, apart);
                        product(s, a[r], f);  // mu
                        h[r].get(before);
                        if (decltype(cutting)::value && n_last >= 0) {  // before the first token: h0
                            Row<float, L> z;
                            z.zero();
                            if (p.h0) z.load(p.h0 + (int64_t)n_last * p.D + c0, apart, inside);
                            z.get(before);
                        }
                        product(before, before, s);
                        Row<TG, L>::store(dg, before, inside, apart);
                    } else {
                        advance<BWD, E>(s, a[r], f);
                        Row<TX, L>::store(out, s, inside, apart);
                    }
                    if (decltype(cutting)::value && n_last >= 0 && p.last)
                        Row<float, L>::store(p.last + (int64_t)n_last * p.D + c0, s, inside, apart);
                }
            };
            bounded || !full ? evaluate(std::true_type()) : evaluate(std::false_type());
        }
        tile = ntile;
    }

    if (p.clustered) {
        if (!met) cluster_meet();
        cluster_meet();  // nobody's shared memory goes before all have read
    }

    // sequences without a token pass their state on
    if (p.last) {
        for (int64_t n0 = (int64_t)blockIdx.x * C::THREADS + warp * 32; n0 < p.N; n0 += (int64_t)gridDim.x * C::THREADS) {
            const int64_t n = n0 + lane;
            unsigned empty = __ballot_sync(0xffffffffu, n < p.N && p.cu[min(n + 1, (int64_t)p.N)] <= p.cu[min(n, (int64_t)p.N)]);
            while (empty) {
                const int64_t m = n0 + __ffs(empty) - 1;
                empty &= empty - 1;
                for (int c = lane; c < p.D; c += 32) p.last[m * p.D + c] = p.start ? p.start[m * p.D + c] : 0.f;
            }
        }
    }
}

// Clears the workspace; the tile kernel behind it may start meanwhile.
__global__ void linrec_clear_kernel(uint4* w, int64_t n) {
    tc::grid_dep_launch();
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const unsigned v = i < kHeadWords / 4 ? 0u : kNothing;
        w[i] = make_uint4(v, v, v, v);
    }
}

// ---- workspace and launch ------------------------------------------------------------

// Up to 8 tile rows whose tiles all fit on the GPU at once are a cluster per channel
// group: one launch, no workspace.  On the device a little faster (1200 tokens by 1024
// channels 8.0 us, with the look-back 8.7 us); for the host one launch and one
// allocation less (16 instead of 22 us a call).
constexpr int kMaxCluster = 8, kMaxClusterTiles = 304;

struct ScanLayout {
    int groups, rows;
    bool clustered;
    size_t words, total;  // published words, bytes in all; 0 for a single row of tiles
};

ScanLayout scan_layout(int64_t T, int D, int TT, int CC) {
    ScanLayout l{};
    l.groups = (D + CC - 1) / CC;
    l.rows = (int)((T + TT - 1) / TT);
    l.clustered = l.rows > 1 && l.rows <= kMaxCluster && (int64_t)l.groups * l.rows <= kMaxClusterTiles;
    if (l.rows <= 1 || l.clustered) return l;
    l.words = (size_t)l.groups * l.rows * 3 * CC;
    l.total = (kHeadWords + l.words) * sizeof(unsigned);
    return l;
}

template <typename TX, typename TG, bool WIDE>
size_t scan_bytes(int64_t T, int D) {
    using F = Tile<TX, TG, false, WIDE>;
    using B = Tile<TX, TG, true, WIDE>;
    const size_t f = scan_layout(T, D, F::TT, F::CC).total, b = scan_layout(T, D, B::TT, B::CC).total;
    return f > b ? f : b;
}

template <typename TX, typename TG>
size_t scan_bytes(int64_t T, int D) {
    // whether rows are aligned is known only at the call
    const size_t n = scan_bytes<TX, TG, false>(T, D), w = D % 8 ? 0 : scan_bytes<TX, TG, true>(T, D);
    return n > w ? n : w;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static std::atomic<EncodeTiled> known{nullptr};
    EncodeTiled f = known.load(std::memory_order_acquire);
    if (f) return f;
    void* entry = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &entry, 12000, cudaEnableDefault, &found) !=
            cudaSuccess || found != cudaDriverEntryPointSuccess)
        return nullptr;
    f = reinterpret_cast<EncodeTiled>(entry);
    known.store(f, std::memory_order_release);
    return f;
}

// The [T, D] rows at `p`, in boxes of `tokens` by `channels`.
template <typename T>
bool encode_rows(CUtensorMap* map, const void* p, int64_t ld, int64_t tokens_all, int D, int tokens, int channels) {
    const EncodeTiled f = encode_tiled();
    if (!f) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)tokens_all}, strides[1] = {(cuuint64_t)ld * sizeof(T)};
    const cuuint32_t box[2] = {(cuuint32_t)channels, (cuuint32_t)tokens}, steps[2] = {1, 1};
    return f(map, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
             const_cast<void*>(p), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows that the wide tiles can read (TMA: 16-byte aligned rows, a stride that
// is one) and write (16-byte vectors).
template <typename T>
bool wide_rows(const void* p, int64_t ld, int D) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0 && ld >= D &&
           (uint64_t)ld * sizeof(T) < (1ull << 40);
}

template <typename TX, typename TG, bool BWD, bool WIDE, bool LOSE = false>
cudaError_t launch_tiles(LinrecParams p, void* ws, cudaStream_t s) {
    using C = Tile<TX, TG, BWD, WIDE>;
    auto kernel = linrec_tile_kernel<TX, TG, BWD, WIDE, LOSE>;
    // at every call: the attribute belongs to the context
    cudaError_t set = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES_SMEM);
    static std::atomic<int> resident{0};  // CTAs per SM
    int per_sm = resident.load(std::memory_order_relaxed);
    if (set == cudaSuccess && !per_sm) {
        set = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, C::THREADS, C::BYTES_SMEM);
        if (set == cudaSuccess && per_sm < 1) set = cudaErrorInvalidConfiguration;
        if (set == cudaSuccess) resident.store(per_sm, std::memory_order_relaxed);
    }
    if (set != cudaSuccess) return set;
    const ScanLayout l = scan_layout(p.T, p.D, C::TT, C::CC);
    p.groups = l.groups;
    p.rows = l.rows;
    p.clustered = l.clustered;
    CUtensorMap mx{}, mg{}, mh{};
    if (WIDE && !(encode_rows<TX>(&mx, p.x, p.ldx, p.T, p.D, C::BOX, C::CC) &&
                  encode_rows<TG>(&mg, p.g, p.ldg, p.T, p.D, C::BOX, C::CC) &&
                  (!BWD || encode_rows<TX>(&mh, p.h, p.ldh, p.T, p.D, C::BOX, C::CC))))
        return cudaErrorInvalidValue;
    p.err = device_error_word();
    if (!p.err) return cudaErrorInitializationError;
    const int64_t tiles = (int64_t)l.groups * l.rows, slots = (int64_t)per_sm * sm_count();
    if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
    if (l.rows <= 1) {
        KernelTimer kt(BWD ? "linrec_bwd" : "linrec_fwd", s);
        kernel<<<(unsigned)tiles, C::THREADS, C::BYTES_SMEM, s>>>(mx, mg, mh, p);
        return cudaGetLastError();
    }
    if (l.clustered) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)tiles);
        cfg.blockDim = dim3(C::THREADS);
        cfg.dynamicSmemBytes = C::BYTES_SMEM;
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)l.rows;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        KernelTimer kt(BWD ? "linrec_bwd" : "linrec_fwd", s);
        return cudaLaunchKernelEx(&cfg, kernel, mx, mg, mh, p);
    }
    char* w = static_cast<char*>(ws);
    p.head = reinterpret_cast<unsigned int*>(w);
    p.words = p.head + kHeadWords;
    {
        KernelTimer kt("linrec_clear", s);
        const int64_t quads = (int64_t)(l.total / 16), blocks = (quads + 511) / 512;
        linrec_clear_kernel<<<(unsigned)(blocks < 608 ? blocks : 608), 256, 0, s>>>(
            reinterpret_cast<uint4*>(p.head), quads);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    KernelTimer kt(BWD ? "linrec_bwd" : "linrec_fwd", s);
    return launch_dependent(kernel, dim3((unsigned)(tiles < slots ? tiles : slots)), dim3(C::THREADS), C::BYTES_SMEM, s,
                            mx, mg, mh, p);
}

template <typename TX, typename TG>
cudaError_t launch_scan_t(const LinrecParams& p, bool bwd, void* ws, cudaStream_t s) {
    const bool wide = p.D % 8 == 0 && wide_rows<TX>(p.x, p.ldx, p.D) && wide_rows<TG>(p.g, p.ldg, p.D) &&
                      wide_rows<TX>(p.out, p.ldo, p.D) &&
                      (!bwd || (wide_rows<TX>(p.h, p.ldh, p.D) && wide_rows<TG>(p.dg, p.lddg, p.D)));
    if (bwd)
        return wide ? launch_tiles<TX, TG, true, true>(p, ws, s) : launch_tiles<TX, TG, true, false>(p, ws, s);
    return wide ? launch_tiles<TX, TG, false, true>(p, ws, s) : launch_tiles<TX, TG, false, false>(p, ws, s);
}

// The forward on fp32 with the copies of tile row p.lost made to run out.
cudaError_t launch_scan_losing(const LinrecParams& p, void* ws, cudaStream_t s) {
    const bool wide = p.D % 8 == 0 && wide_rows<float>(p.x, p.ldx, p.D) && wide_rows<float>(p.g, p.ldg, p.D) &&
                      wide_rows<float>(p.out, p.ldo, p.D);
    return wide ? launch_tiles<float, float, false, true, true>(p, ws, s)
                : launch_tiles<float, float, false, false, true>(p, ws, s);
}

cudaError_t launch_scan(const LinrecParams& p, int dtype, int gate_dtype, bool bwd, void* ws, cudaStream_t s) {
    if (dtype == GDR_BF16)
        return gate_dtype == GDR_BF16 ? launch_scan_t<__nv_bfloat16, __nv_bfloat16>(p, bwd, ws, s)
                                      : launch_scan_t<__nv_bfloat16, float>(p, bwd, ws, s);
    return gate_dtype == GDR_BF16 ? launch_scan_t<float, __nv_bfloat16>(p, bwd, ws, s)
                                  : launch_scan_t<float, float>(p, bwd, ws, s);
}

// ---- the slot-pool step ------------------------------------------------------

struct StepParams {
    const void* x;
    const void* g;
    void* pool;
    const int32_t* idx;
    const int32_t* cu;
    void* y;
    void* states;
    int64_t ldx, ldg, ldy, T;
    int N, D, num_slots, steps, commit;
};

// VEC elements in one access (two for 8 fp32).
template <typename T, int VEC> struct alignas(sizeof(T) * VEC < 16 ? sizeof(T) * VEC : 16) Pack {
    T v[VEC];
};

// A thread owns VEC channels of a sequence and walks its tokens, those of the
// next TOKENS steps loaded at once.  Bound by latency at decode sizes (the slot
// and the sequence's place, then the rows), by memory at large ones: 4 x 2048
// channels 1.7 us, 256 x 4096 3.6 us (62 % of the copy rate, all of it in L2),
// 64 x 1..12 tokens x 4096 with every state kept 6.4 us (37 %).  All 12 tokens
// loaded at once instead of 4 was slower (9.7 us: a larger program than its run).
template <typename TX, typename TG, typename TP, int VEC>
__global__ void __launch_bounds__(128) linrec_step_kernel(StepParams p) {
    constexpr int TOKENS = VEC >= 8 ? 2 : 4;
    const int c = (blockIdx.x * blockDim.x + threadIdx.x) * VEC;
    if (c >= p.D) return;
    for (int64_t n = blockIdx.y; n < p.N; n += gridDim.y) {
        const int slot = p.idx[n];
        const int64_t lo = max((int64_t)p.cu[n], (int64_t)0), hi = min((int64_t)p.cu[n + 1], p.T);
        if (slot < 0 || slot >= p.num_slots || hi <= lo) continue;
        Pack<TP, VEC>* cell = reinterpret_cast<Pack<TP, VEC>*>(static_cast<TP*>(p.pool) + (int64_t)slot * p.D + c);
        const Pack<TP, VEC> before = *cell;
        const TX* x = static_cast<const TX*>(p.x) + lo * p.ldx + c;
        const TG* g = static_cast<const TG*>(p.g) + lo * p.ldg + c;
        TX* y = static_cast<TX*>(p.y) + lo * p.ldy + c;
        const int len = (int)(hi - lo), kept = p.states ? min(len, p.steps) : 0;
        TP* keep = kept ? static_cast<TP*>(p.states) + n * p.steps * p.D + c : nullptr;
        float h[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) h[j] = to_f(before.v[j]);
        for (int t0 = 0; t0 < len; t0 += TOKENS) {
            Pack<TX, VEC> xs[TOKENS];
            Pack<TG, VEC> gs[TOKENS];
#pragma unroll
            for (int i = 0; i < TOKENS; ++i)
                if (t0 + i < len) {
                    xs[i] = *reinterpret_cast<const Pack<TX, VEC>*>(x + (t0 + i) * p.ldx);
                    gs[i] = *reinterpret_cast<const Pack<TG, VEC>*>(g + (t0 + i) * p.ldg);
                }
#pragma unroll
            for (int i = 0; i < TOKENS; ++i)
                if (t0 + i < len) {
                    Pack<TX, VEC> out;
                    float a[VEC];
#pragma unroll
                    for (int j = 0; j < VEC; ++j) a[j] = to_f(gs[i].v[j]);
                    exp_of(a, reduced_exp);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        h[j] = fmaf(a[j], h[j], to_f(xs[i].v[j]));
                        out.v[j] = from_f<TX>(h[j]);
                    }
                    *reinterpret_cast<Pack<TX, VEC>*>(y + (t0 + i) * p.ldy) = out;
                    if (t0 + i < kept) {
                        Pack<TP, VEC> state;
#pragma unroll
                        for (int j = 0; j < VEC; ++j) state.v[j] = from_f<TP>(h[j]);
                        *reinterpret_cast<Pack<TP, VEC>*>(keep + (int64_t)(t0 + i) * p.D) = state;
                    }
                }
        }
        if (p.commit) {
            Pack<TP, VEC> state;
#pragma unroll
            for (int j = 0; j < VEC; ++j) state.v[j] = from_f<TP>(h[j]);
            *cell = state;
        }
    }
}

template <typename TX, typename TG, typename TP, int VEC>
cudaError_t launch_step_v(const StepParams& p, cudaStream_t s) {
    const dim3 grid((p.D + 128 * VEC - 1) / (128 * VEC), p.N < 65535 ? p.N : 65535);
    KernelTimer kt("linrec_step", s);
    linrec_step_kernel<TX, TG, TP, VEC><<<grid, 128, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename TX, typename TG, typename TP>
cudaError_t launch_step_t(const StepParams& p, cudaStream_t s) {
    if (p.D % 8 || !wide_rows<TX>(p.x, p.ldx, p.D) || !wide_rows<TG>(p.g, p.ldg, p.D) ||
        !wide_rows<TX>(p.y, p.ldy, p.D))
        return launch_step_v<TX, TG, TP, 1>(p, s);
    // 8 channels per thread where that still gives every SM's schedulers work (decode of
    // 256 x 4096: 3.6 us, with 4 channels 4.8, with 2 5.7), fewer otherwise (verify of 64
    // x 1..12 x 4096 with states kept: with 2 channels 6.4 us, with 4 7.4, with 8 9.0).
    // The number of tokens need not enter: verify of 128, 256 and 512 sequences takes
    // 9.5, 13.4 and 24.3 us by this rule (4, 8, 8 channels), the best of the others 9.0,
    // 13.8 and 24.6.
    const int64_t channels = (int64_t)p.N * p.D, full = (int64_t)sm_count() * 768;
    return channels >= full * 8 ? launch_step_v<TX, TG, TP, 8>(p, s)
         : channels >= full * 4 ? launch_step_v<TX, TG, TP, 4>(p, s) : launch_step_v<TX, TG, TP, 2>(p, s);
}

template <typename TX, typename TG>
cudaError_t launch_step_p(const StepParams& p, int pool_dtype, cudaStream_t s) {
    return pool_dtype == GDR_BF16 ? launch_step_t<TX, TG, __nv_bfloat16>(p, s) : launch_step_t<TX, TG, float>(p, s);
}

cudaError_t launch_step(const StepParams& p, int dtype, int gate_dtype, int pool_dtype, cudaStream_t s) {
    if (dtype == GDR_BF16)
        return gate_dtype == GDR_BF16 ? launch_step_p<__nv_bfloat16, __nv_bfloat16>(p, pool_dtype, s)
                                      : launch_step_p<__nv_bfloat16, float>(p, pool_dtype, s);
    return gate_dtype == GDR_BF16 ? launch_step_p<float, __nv_bfloat16>(p, pool_dtype, s)
                                  : launch_step_p<float, float>(p, pool_dtype, s);
}

// ---- GDR_VALIDATE --------------------------------------------------------------

enum : unsigned { L_CU = 1u, L_GATE = 2u, L_SLOT = 4u, L_DUP = 8u, L_STEPS = 16u };

static __device__ unsigned int g_linrec_findings;

template <typename TG>
__global__ void linrec_validate_kernel(const int32_t* cu, int N, int64_t T, const TG* g, int64_t ldg, int D,
                                       const int32_t* idx, int num_slots, int commit, int steps) {
    const int64_t tid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t nth = (int64_t)gridDim.x * blockDim.x;
    unsigned bad = 0;
    for (int64_t b = tid; b < N; b += nth) {
        const int lo = cu[b], hi = cu[b + 1];
        if (hi < lo) bad |= L_CU;
        if (idx) {
            const int slot = idx[b];
            if (slot >= num_slots) bad |= L_SLOT;
            if (slot >= 0 && steps > 0 && hi - lo > steps) bad |= L_STEPS;
            if (slot >= 0 && commit)
                for (int64_t j = 0; j < b; ++j)
                    if (idx[j] == slot) bad |= L_DUP;
        }
    }
    if (tid == 0 && (cu[0] != 0 || cu[N] < 0 || cu[N] > T)) bad |= L_CU;
    auto gates = [&](int64_t row, int64_t rows, int64_t i, int64_t step) {
        const TG* from = g + row * ldg;
        for (; i < rows * D; i += step)
            if (!(to_f(from[i / D * ldg + i % D]) <= 0.f)) bad |= L_GATE;
    };
    if (!idx) {
        gates(0, min(max((int64_t)cu[N], (int64_t)0), T), tid, nth);
    } else {  // a sequence per CTA: the rows of padding are not read
        for (int64_t b = blockIdx.x; b < N; b += gridDim.x) {
            const int64_t lo = max((int64_t)cu[b], (int64_t)0), hi = min((int64_t)cu[b + 1], T);
            if (idx[b] >= 0 && idx[b] < num_slots) gates(lo, hi - lo, threadIdx.x, blockDim.x);
        }
    }
    if (bad) atomicOr(&g_linrec_findings, bad);
}

int validate(const int32_t* cu, int N, int64_t T, const void* g, int64_t ldg, int D, int gate_dtype,
             const int32_t* idx, int num_slots, int commit, int steps, cudaStream_t s) {
    // one word for all: from its clearing to its reading it belongs to one call
    static std::mutex turn;
    const std::lock_guard<std::mutex> own(turn);
    void* word = nullptr;
    if (cudaGetSymbolAddress(&word, g_linrec_findings) != cudaSuccess)
        return set_last_error(GDR_ERR_LAUNCH, "validation word unavailable");
    cudaError_t e = cudaMemsetAsync(word, 0, sizeof(unsigned), s);
    if (e != cudaSuccess) return set_last_error(GDR_ERR_LAUNCH, "validation: %s", cudaGetErrorString(e));
    if (gate_dtype == GDR_BF16)
        linrec_validate_kernel<<<304, 256, 0, s>>>(cu, N, T, static_cast<const __nv_bfloat16*>(g), ldg, D, idx,
                                                   num_slots, commit, steps);
    else
        linrec_validate_kernel<<<304, 256, 0, s>>>(cu, N, T, static_cast<const float*>(g), ldg, D, idx, num_slots,
                                                   commit, steps);
    e = cudaGetLastError();
    unsigned found = 0;
    if (e == cudaSuccess) e = cudaMemcpyAsync(&found, word, sizeof(unsigned), cudaMemcpyDeviceToHost, s);
    const cudaError_t ended = cudaStreamSynchronize(s);  // also behind a copy that was refused: `found` is on this stack
    if (e == cudaSuccess) e = ended;
    if (e != cudaSuccess) return set_last_error(GDR_ERR_LAUNCH, "validation: %s", cudaGetErrorString(e));
    if (found)
        return set_last_error(GDR_ERR_VALIDATION, "input validation failed (0x%x):%s%s%s%s%s", found,
                              (found & L_CU) ? " cu_seqlens malformed;" : "",
                              (found & L_GATE) ? " gate NaN or > 0;" : "",
                              (found & L_SLOT) ? " state index >= num_slots;" : "",
                              (found & L_DUP) ? " duplicate state index;" : "",
                              (found & L_STEPS) ? " sequence longer than steps;" : "");
    return GDR_OK;
}

// ---- argument checks -----------------------------------------------------------

int check_sizes(int N, int64_t T, int D, int dtype, int gate_dtype) {
    if (N < 0 || T < 0) return set_last_error(GDR_ERR_INVALID_ARG, "negative N (%d) or T_total (%lld)", N, (long long)T);
    if (D <= 0) return set_last_error(GDR_ERR_INVALID_ARG, "D (%d) must be positive", D);
    if (dtype != GDR_BF16 && dtype != GDR_F32) return set_last_error(GDR_ERR_UNSUPPORTED, "dtype %d", dtype);
    if (gate_dtype != GDR_BF16 && gate_dtype != GDR_F32)
        return set_last_error(GDR_ERR_UNSUPPORTED, "gate_dtype %d", gate_dtype);
    if (T > 0x7fffffffLL - kMaxTileTokens + 1)
        return set_last_error(GDR_ERR_UNSUPPORTED, "T_total (%lld) above 2^31 - 512", (long long)T);
    if (N > 0x7fffffff / 2) return set_last_error(GDR_ERR_UNSUPPORTED, "N too large");
    if (D > 1 << 24) return set_last_error(GDR_ERR_UNSUPPORTED, "D (%d) above 2^24", D);
    return GDR_OK;
}

// The scans, as gdr_chunk_fwd: rows without a sequence.
int check_sequences(int N, int64_t T) {
    if (T > 0 && N == 0) return set_last_error(GDR_ERR_INVALID_ARG, "T_total > 0 with N == 0");
    return GDR_OK;
}

unsigned element(int dtype) { return dtype == GDR_BF16 ? 2 : 4; }

// cu_seqlens and state_indices.
int check_ints(const char* name, const void* p) {
    if (!p) return set_last_error(GDR_ERR_INVALID_ARG, "null pointer argument (%s)", name);
    if (reinterpret_cast<uintptr_t>(p) & 3u)
        return set_last_error(GDR_ERR_INVALID_ARG, "%s not 4-byte aligned", name);
    return GDR_OK;
}

// A sequence's last state may be written while another tile has yet to read its first.
// Both are [N, D], dense.
int check_apart(const char* name, const float* written, const float* read, int N, int D) {
    const uintptr_t w = reinterpret_cast<uintptr_t>(written), r = reinterpret_cast<uintptr_t>(read);
    const uintptr_t bytes = (uintptr_t)N * D * sizeof(float);
    if (written && read && (w < r ? r - w : w - r) < bytes)
        return set_last_error(GDR_ERR_INVALID_ARG, "%s must not overlap a state that the call reads", name);
    return GDR_OK;
}

int check_workspace(int N, int64_t T, int D, int dtype, int gate_dtype, const void* ws, size_t ws_bytes) {
    size_t need = 0;
    if (int rc = gdr_linrec_workspace_size(N, T, D, dtype, gate_dtype, &need)) return rc;
    if (need == 0) return GDR_OK;
    if (!ws || ws_bytes < need)
        return set_last_error(GDR_ERR_WORKSPACE, "workspace %zu bytes < required %zu", ws ? ws_bytes : (size_t)0, need);
    if (reinterpret_cast<uintptr_t>(ws) & 255u)
        return set_last_error(GDR_ERR_INVALID_ARG, "workspace not 256-byte aligned");
    return GDR_OK;
}

// No tokens at all: every sequence's last state is its first.
int pass_states(const float* start, float* last, int N, int D, cudaStream_t s) {
    if (N == 0 || !last) return set_ok();
    if (int rc = check_device()) return rc;
    const size_t bytes = sizeof(float) * (size_t)N * D;
    return launch_result(start ? cudaMemcpyAsync(last, start, bytes, cudaMemcpyDeviceToDevice, s)
                          : cudaMemsetAsync(last, 0, bytes, s), "empty recurrence");
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

int gdr_linrec_workspace_size(int N, int64_t T_total, int D, int dtype, int gate_dtype, size_t* bytes) {
    if (!bytes) return set_last_error(GDR_ERR_INVALID_ARG, "bytes is NULL");
    if (int rc = check_sizes(N, T_total, D, dtype, gate_dtype)) return rc;
    if (int rc = check_sequences(N, T_total)) return rc;
    if (dtype == GDR_BF16)
        *bytes = gate_dtype == GDR_BF16 ? scan_bytes<__nv_bfloat16, __nv_bfloat16>(T_total, D)
                                        : scan_bytes<__nv_bfloat16, float>(T_total, D);
    else
        *bytes = gate_dtype == GDR_BF16 ? scan_bytes<float, __nv_bfloat16>(T_total, D)
                                        : scan_bytes<float, float>(T_total, D);
    return set_ok();
}

int gdr_linrec_fwd(const void* x, int64_t x_stride, const void* g, int64_t g_stride, const float* initial_state,
                   const int32_t* cu_seqlens, int N, int64_t T_total, int D, int dtype, int gate_dtype, int flags,
                   void* y, int64_t y_stride, float* final_state, void* workspace, size_t ws_bytes,
                   gdr_stream_t stream) {
    if (int rc = check_sizes(N, T_total, D, dtype, gate_dtype)) return rc;
    if (int rc = check_sequences(N, T_total)) return rc;
    if (flags & ~GDR_VALIDATE)
        return set_last_error(GDR_ERR_INVALID_ARG, "unsupported flags 0x%x for gdr_linrec_fwd", flags);
    if (int rc = check_aligned16("initial_state", initial_state)) return rc;
    if (int rc = check_aligned16("final_state", final_state)) return rc;
    if (int rc = check_apart("final_state", final_state, initial_state, N, D)) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    if (T_total == 0) return pass_states(initial_state, final_state, N, D, s);
    if (int rc = check_rows("x", x, x_stride, 0, element(dtype))) return rc;
    if (int rc = check_rows("g", g, g_stride, 0, element(gate_dtype))) return rc;
    if (int rc = check_rows("y", y, y_stride, D, element(dtype))) return rc;
    if (int rc = check_ints("cu_seqlens", cu_seqlens)) return rc;
    if (int rc = check_workspace(N, T_total, D, dtype, gate_dtype, workspace, ws_bytes)) return rc;
    if (int rc = check_device()) return rc;
    if (flags & GDR_VALIDATE)
        if (int rc = validate(cu_seqlens, N, T_total, g, g_stride, D, gate_dtype, nullptr, 0, 0, 0, s)) return rc;
    LinrecParams p{};
    p.x = x; p.g = g; p.out = y; p.start = initial_state; p.last = final_state; p.cu = cu_seqlens;
    p.ldx = x_stride; p.ldg = g_stride; p.ldo = y_stride; p.T = T_total; p.N = N; p.D = D;
    return launch_result(launch_scan(p, dtype, gate_dtype, false, workspace, s), "gdr_linrec_fwd launch");
}

int gdr_selftest_linrec_lost_copy(const float* x, const float* g, const int32_t* cu_seqlens, int N, int64_t T_total,
                                  int D, int lost_row, float* y, float* final_state, void* workspace, size_t ws_bytes,
                                  gdr_stream_t stream) {
    if (int rc = check_sizes(N, T_total, D, GDR_F32, GDR_F32)) return rc;
    if (int rc = check_sequences(N, T_total)) return rc;
    if (T_total == 0) return set_ok();
    if (int rc = check_rows("x", x, D, 0, 4)) return rc;
    if (int rc = check_rows("g", g, D, 0, 4)) return rc;
    if (int rc = check_rows("y", y, D, D, 4)) return rc;
    if (int rc = check_aligned16("final_state", final_state)) return rc;
    if (int rc = check_ints("cu_seqlens", cu_seqlens)) return rc;
    if (int rc = check_workspace(N, T_total, D, GDR_F32, GDR_F32, workspace, ws_bytes)) return rc;
    if (int rc = check_device()) return rc;
    LinrecParams p{};
    p.x = x; p.g = g; p.out = y; p.last = final_state; p.cu = cu_seqlens;
    p.ldx = p.ldg = p.ldo = D; p.T = T_total; p.N = N; p.D = D; p.lost = lost_row;
    return launch_result(launch_scan_losing(p, workspace, (cudaStream_t)stream), "gdr_selftest_linrec_lost_copy launch");
}

int gdr_linrec_bwd(const void* dy, int64_t dy_stride, const void* g, int64_t g_stride, const void* y,
                   int64_t y_stride, const float* initial_state, const float* d_final_state,
                   const int32_t* cu_seqlens, int N, int64_t T_total, int D, int dtype, int gate_dtype, int flags,
                   void* dx, int64_t dx_stride, void* dg, int64_t dg_stride, float* d_initial_state,
                   void* workspace, size_t ws_bytes, gdr_stream_t stream) {
    if (int rc = check_sizes(N, T_total, D, dtype, gate_dtype)) return rc;
    if (int rc = check_sequences(N, T_total)) return rc;
    if (flags & ~GDR_VALIDATE)
        return set_last_error(GDR_ERR_INVALID_ARG, "unsupported flags 0x%x for gdr_linrec_bwd", flags);
    if (int rc = check_aligned16("initial_state", initial_state)) return rc;
    if (int rc = check_aligned16("d_final_state", d_final_state)) return rc;
    if (int rc = check_aligned16("d_initial_state", d_initial_state)) return rc;
    if (int rc = check_apart("d_initial_state", d_initial_state, initial_state, N, D)) return rc;
    if (int rc = check_apart("d_initial_state", d_initial_state, d_final_state, N, D)) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    if (T_total == 0) return pass_states(d_final_state, d_initial_state, N, D, s);
    if (int rc = check_rows("dy", dy, dy_stride, 0, element(dtype))) return rc;
    if (int rc = check_rows("g", g, g_stride, 0, element(gate_dtype))) return rc;
    if (int rc = check_rows("y", y, y_stride, 0, element(dtype))) return rc;
    if (int rc = check_rows("dx", dx, dx_stride, D, element(dtype))) return rc;
    if (int rc = check_rows("dg", dg, dg_stride, D, element(gate_dtype))) return rc;
    if (int rc = check_ints("cu_seqlens", cu_seqlens)) return rc;
    if (int rc = check_workspace(N, T_total, D, dtype, gate_dtype, workspace, ws_bytes)) return rc;
    if (int rc = check_device()) return rc;
    if (flags & GDR_VALIDATE)
        if (int rc = validate(cu_seqlens, N, T_total, g, g_stride, D, gate_dtype, nullptr, 0, 0, 0, s)) return rc;
    LinrecParams p{};
    p.x = dy; p.g = g; p.h = y; p.out = dx; p.dg = dg; p.h0 = initial_state; p.start = d_final_state;
    p.last = d_initial_state; p.cu = cu_seqlens; p.ldx = dy_stride; p.ldg = g_stride; p.ldh = y_stride;
    p.ldo = dx_stride; p.lddg = dg_stride; p.T = T_total; p.N = N; p.D = D;
    return launch_result(launch_scan(p, dtype, gate_dtype, true, workspace, s), "gdr_linrec_bwd launch");
}

int gdr_linrec_step(const void* x, int64_t x_stride, const void* g, int64_t g_stride, void* state_pool,
                    int pool_dtype, int num_slots, const int32_t* state_indices, const int32_t* cu_seqlens, int N,
                    int64_t T_total, int D, int dtype, int gate_dtype, int flags, void* y, int64_t y_stride,
                    void* intermediate_states, int steps, gdr_stream_t stream) {
    if (int rc = check_sizes(N, T_total, D, dtype, gate_dtype)) return rc;
    if (pool_dtype != GDR_BF16 && pool_dtype != GDR_F32)
        return set_last_error(GDR_ERR_UNSUPPORTED, "pool_dtype %d", pool_dtype);
    if (flags & ~(GDR_COMMIT | GDR_VALIDATE))
        return set_last_error(GDR_ERR_INVALID_ARG, "unsupported flags 0x%x for gdr_linrec_step", flags);
    if (N == 0 || T_total == 0) return set_ok();
    if (num_slots <= 0) return set_last_error(GDR_ERR_INVALID_ARG, "num_slots must be positive");
    if (intermediate_states && steps <= 0)
        return set_last_error(GDR_ERR_INVALID_ARG, "steps must be positive with intermediate_states");
    if (!state_pool) return set_last_error(GDR_ERR_INVALID_ARG, "null pointer argument (state_pool)");
    if (int rc = check_ints("state_indices", state_indices)) return rc;
    if (int rc = check_ints("cu_seqlens", cu_seqlens)) return rc;
    if (int rc = check_aligned16("state_pool", state_pool)) return rc;
    if (int rc = check_aligned16("intermediate_states", intermediate_states)) return rc;
    if (int rc = check_rows("x", x, x_stride, 0, element(dtype))) return rc;
    if (int rc = check_rows("g", g, g_stride, 0, element(gate_dtype))) return rc;
    if (int rc = check_rows("y", y, y_stride, D, element(dtype))) return rc;
    if (int rc = check_device()) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    if (flags & GDR_VALIDATE)
        if (int rc = validate(cu_seqlens, N, T_total, g, g_stride, D, gate_dtype, state_indices, num_slots,
                              (flags & GDR_COMMIT) ? 1 : 0, intermediate_states ? steps : 0, s))
            return rc;
    StepParams p{};
    p.x = x; p.g = g; p.pool = state_pool; p.idx = state_indices; p.cu = cu_seqlens; p.y = y;
    p.states = intermediate_states; p.ldx = x_stride; p.ldg = g_stride; p.ldy = y_stride; p.T = T_total; p.N = N;
    p.D = D; p.num_slots = num_slots; p.steps = intermediate_states ? steps : 0; p.commit = (flags & GDR_COMMIT) ? 1 : 0;
    return launch_result(launch_step(p, dtype, gate_dtype, pool_dtype, s), "gdr_linrec_step launch");
}

}  // extern "C"
