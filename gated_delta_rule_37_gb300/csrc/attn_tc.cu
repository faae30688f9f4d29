// Causal attention on the tensor cores (bf16): packed prompts, and the prefix that a
// batch shares in the paged cache.
//
// A CTA has one key head and two tiles of 128 query rows, a row being a (token, query
// head of the group) pair: the heads that read one key head share every key tile, and a
// causal tile has rows of 128 / group tokens only.  It walks over the keys by tiles of
// 128.  Per row tile and key tile, with S and O in tensor memory:
//   S = Q K^T     one thread issues it: Q and K from shared memory, 128 x 128 x D
//   P = 2^(S c - m)   a warpgroup, a row per thread, c = scale log2(e): P goes back into
//                 S's columns as bf16 (a product's operands have one type, V's), its sum stays fp32
//   O += P V      P from tensor memory, V from shared memory as it was loaded (rows of
//                 keys: the contraction runs down the tile)
// The two row tiles alternate: while one's P is formed the tensor cores work on the
// other's O += P V and next S.  S of one tile is free again when its O += P V has read P,
// and MMAs run in the order of their issue, so that needs no wait.
//   The maximum m that P refers to follows the row's maximum lazily: O and the sum are
// rescaled only when the maximum has risen by more than 2^8, so O's rescaling, a trip through
// registers, is rare.  P is taken 2^8 smaller for it and never above 1: values whose weighted
// sum fits in fp32 do not overflow on the way.  m cancels in O / sum.
//   A CTA of a prompt takes row tiles of any sequence one after the other; its copies run
// ahead into the next one's keys while the last rows of this one are rescaled and written.
// The grid has a place for every pair of row tiles: a CTA that is done asks the hardware for
// a CTA that has not started yet and takes its place, so whoever is free goes on, without a
// counter in memory.  Places are in the order of their keys, most first, for up to 64
// sequences; with more there are enough of them for any order.
//   Keys behind a sequence's last one are not another's to see: their V rows are cleared
// in shared memory (0 * NaN is a NaN), in the last tile alone.  Within a sequence a later
// token's infinity or NaN could still reach an earlier row as 0 * inf.  A row whose result is not
// finite is right if only keys that it sees have such values, which the values between its
// own token and the end of its last key tile tell; else those before tell whether it is a NaN or
// an infinity by its own keys too, and only if not it is computed once more, on the CUDA cores, from the
// keys that it sees: the rows within a key tile before a bad token.  (8192 tokens of 8 heads of 128, 0.103 ms:
// one early NaN in a key / a value 0.103 / 0.133, one in the middle 0.118, a channel of NaN / of infinities
// 0.147 / 0.276.)
//   Measured, heads of 128: 2900 cycles for a key tile of both row tiles, of which the four
// products are 2048 and most of the rest is the issuing warp's between them; 32768 tokens, 32 heads
// on 8, 5.55 ms, 1585 TFLOP/s.  Heads of 64 take 2700 for half of the products: there the softmax
// warps' chain of 1250 and the trips between them and the issuing warp bound it.
#include <math.h>

#include <atomic>

#include "attn.h"
#include "attn_copies.cuh"
#include "attn_step.cuh"
#include "common.cuh"
#include "gdr.h"
#include "launch.h"
#include "tc.cuh"

namespace gdr {
namespace {

using namespace tc;

static_assert(kFarTile == 128, "the prefix's key tile");
constexpr int kTile = 128;                // rows of a query tile, keys of a key tile
constexpr int kWarps = 12;                // 2 x 4 of softmax; copies, MMAs, values behind the end, places
// Registers: a softmax thread keeps a row of S.  The block is launched with 168 a thread,
// 3 x 168 for a thread of each warpgroup; the third one's go to the others.
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * kLaunchRegs, "more registers than the block has");
constexpr int kNoRow = 0x7fffffff;        // the limit of a lane without a row: it masks nothing
// How far P's reference may lag behind the maximum, log2 units (8 / 0: 32768 tokens 5.5 / 5.8 ms).
constexpr float kLag = 8.f;

template <int D> struct Shape {
    static constexpr int BLOCKS = D / 64;                  // 128-byte column blocks of a row
    static constexpr int BLOCK_BYTES = kTile * 128;
    static constexpr int TILE_BYTES = BLOCKS * BLOCK_BYTES;
    static constexpr int STAGES = D == 128 ? 4 : 8;
    static constexpr int OUT_BYTES = 32 * 128;             // 128 bytes of a warp's rows on their way out
    static constexpr int SMEM = 1024 + (2 + STAGES) * TILE_BYTES + 8 * OUT_BYTES;
    static constexpr uint32_t S = 0, O = 256;              // tensor memory columns: S of both row tiles, O of both
};

// Of each row tile: q, queries there; q_free, read for the last time; s, S there; p, P there;
// o, O there; o_free, O read.  Of the ring: full, empty, and fixed: values behind the end are
// cleared (of a stage: the copies may be jobs ahead of the MMAs, but a stage waits to be
// read).  Of the jobs: job, job_free; asked, its last copies are on their way (before, a wait
// for a stage could take the phase before for that one); ahead, the copies are at its last
// tiles; limits_free, the prefix's limits are read; place, the answer where to go on is there.
struct Barriers {
    uint64_t q[2], q_free[2], full[8], empty[8], s[2], p[2], o[2], o_free[2], job[2], job_free[2], fixed[8], asked[2], ahead,
        limits_free, place, drain;
};

struct TcParams {
    AttnArgs a;
    StepWork w;
    int tokens;  // of a row tile: 128 / group
    int box;     // rows of one copy of keys: 128, or a page's
    unsigned* err;
};

// One lane of a warp that is together, always the same.
__device__ __forceinline__ bool elect_one() {
    uint32_t x;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}\n" : "=r"(x));
    return x != 0;
}

// D += A B with A in tensor memory.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
                 :: "r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc));
}

#define GDR_R32(x, b)                                                                                                \
    x(b, 0), x(b, 1), x(b, 2), x(b, 3), x(b, 4), x(b, 5), x(b, 6), x(b, 7), x(b, 8), x(b, 9), x(b, 10), x(b, 11),    \
        x(b, 12), x(b, 13), x(b, 14), x(b, 15), x(b, 16), x(b, 17), x(b, 18), x(b, 19), x(b, 20), x(b, 21),          \
        x(b, 22), x(b, 23), x(b, 24), x(b, 25), x(b, 26), x(b, 27), x(b, 28), x(b, 29), x(b, 30), x(b, 31)
#define GDR_OUT(b, i) "=f"((b)[i])
#define GDR_INOUT(b, i) "+f"((b)[i])
#define GDR_IN(b, i) "r"((b)[i])
#define GDR_LIST32                                                                                                   \
    "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"    \
    "%29,%30,%31}"

// 32 columns of this thread's lane; the registers are there after arrived32.
__device__ __forceinline__ void tmem_fetch32(uint32_t addr, float* v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 " GDR_LIST32 ", [%32];" : GDR_R32(GDR_OUT, v) : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// ties the registers to what was waited for
__device__ __forceinline__ void arrived32(float* v) { asm volatile("" : GDR_R32(GDR_INOUT, v)); }
__device__ __forceinline__ void tmem_put32(uint32_t addr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], " GDR_LIST32 ";" :: GDR_R32(GDR_IN, v), "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two row tiles' work; n < 0: there is no more.
struct Job {
    int64_t t0;       // first token of their sequence (prompt), or 0
    int64_t i0;       // their first token, counted from t0
    int64_t end;      // tokens of the sequence, or of the batch
    int from, to[2];  // key tiles of the two row tiles: from .. to - 1
    int keys;         // end of the keys, counted from the sequence's first
    int n, h;
    int part;         // of the prefix's partial results
    bool clear;       // values behind the end are in the last tile
};

// Pairs of row tiles of sequence n.
__device__ __forceinline__ int pairs_of(const AttnArgs& a, int pair_tokens, int n) {
    if (n >= a.N) return 0;
    const int64_t L = min((int64_t)a.cu[n + 1], a.T) - max(a.cu[n], 0);
    return L > 0 ? (int)((L + pair_tokens - 1) / pair_tokens) : 0;
}

// Of the tokens first .. first + tokens - 1 of a batch the end of the prefix's keys that each
// sees, 0 for padding; by a warp.
__device__ __forceinline__ void mark_limits(const AttnArgs& a, int64_t first, int tokens, int* limits) {
    const int lane = threadIdx.x & 31;
    for (int i = lane; i < tokens; i += 32) limits[i] = 0;
    __syncwarp();
    // the last sequence that begins at or before the first token
    int lo = 0, hi = a.N - 1;
    while (hi > lo) {
        const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
        lo += __popc(__ballot_sync(0xffffffffu, at <= hi && a.cu[at] <= first)) * step;
        hi = min(lo + step - 1, hi);
    }
    for (int base = lo; base < a.N; base += 32) {
        const int n = base + lane;
        bool behind = true;
        if (n < a.N) {
            const int len = a.cache.lens[n];
            const int64_t begin = a.cu[n], end = min((int64_t)a.cu[n + 1], a.T);
            behind = begin >= first + tokens;
            if (len >= 0)
                for (int64_t t = max(begin, first); t < min(end, first + tokens); ++t)
                    limits[t - first] = (int)min((int64_t)a.cache.prefix_len, len + (t - begin) + 1);
        }
        if (__any_sync(0xffffffffu, behind)) break;
    }
    __syncwarp();
}

// Sequences, two of a lane.  (Sorted / in their own order: 4 prompts of 65 to 3000 tokens 60 / 63 us, 64
// of 16001 in all 50 / 53.)
constexpr int kSorted = 64;

// The pair of row tiles at a place of a prompt's call, by a warp; false where the place is
// empty.  Up to kSorted sequences (pairs: those of sequences lane and lane + 32): first all
// pairs number p, of sequences that have so many, then all number p - 1.  More sequences: the
// last one first; sequence n's places begin at cu[n] / (tokens of a pair) + n, which leaves
// room for its last, partly filled one and is found by search.
__device__ __forceinline__ bool find_job(const AttnArgs& a, int pair_tokens, const int (&pairs)[2], int64_t place,
                                         int64_t places, int h, Job& job) {
    const int lane = threadIdx.x & 31;
    int n, pair;
    if (a.N <= kSorted) {
        // pairs numbered p and above
        auto above = [&](int p) {
            return __reduce_add_sync(0xffffffffu, (unsigned)(max(0, pairs[0] - p) + max(0, pairs[1] - p)));
        };
        if (place >= above(0)) return false;
        int lo = 0, hi = (int)__reduce_max_sync(0xffffffffu, (unsigned)max(pairs[0], pairs[1]));
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (above(mid) > place) lo = mid; else hi = mid;
        }
        pair = lo;
        const int rank = (int)(place - above(lo + 1));
        const uint32_t has[2] = {__ballot_sync(0xffffffffu, pairs[0] > lo), __ballot_sync(0xffffffffu, pairs[1] > lo)};
        const int in_first = __popc(has[0]);
        n = rank < in_first ? (int)__fns(has[0], 0, rank + 1) : 32 + (int)__fns(has[1], 0, rank - in_first + 1);
    } else {
        place = places - 1 - place;
        int lo = 0, hi = a.N - 1;
        while (hi > lo) {
            const int step = (hi - lo + 31) / 32;
            const int at = lo + (lane + 1) * step;
            const bool below = at <= hi && max(a.cu[at], 0) / pair_tokens + (int64_t)at <= place;
            lo += __popc(__ballot_sync(0xffffffffu, below)) * step;
            hi = min(lo + step - 1, hi);
        }
        n = lo;
        const int64_t at = place - n - max(a.cu[n], 0) / pair_tokens;
        if (at < 0 || at >= pairs_of(a, pair_tokens, n)) return false;
        pair = (int)at;
    }
    job.t0 = max(a.cu[n], 0);
    const int64_t L = min((int64_t)a.cu[n + 1], a.T) - job.t0;
    job.i0 = (int64_t)pair * pair_tokens;
    const int64_t i1 = job.i0 + pair_tokens / 2;
    job.end = L;
    job.from = 0;
    job.to[0] = (int)((min(i1, L) + kTile - 1) / kTile);
    job.to[1] = i1 < L ? (int)((min(job.i0 + pair_tokens, L) + kTile - 1) / kTile) : 0;
    job.keys = (int)min(job.i0 + pair_tokens, L);
    job.n = n;
    job.h = h;
    // The sequence ends inside the last key tile: what follows there is another's.  (With several heads
    // to a key head a pair has fewer tokens than a key tile has keys: not the last pair alone.)  What lies
    // behind within the sequence is left to the rows that it spoils.
    job.clear = (int64_t)max(job.to[0], job.to[1]) * kTile > L;
    return true;
}

// Asks for a CTA of this grid that has not started, to take its place; the answer, 16 bytes,
// arrives on the barrier.
__device__ __forceinline__ void ask_place(uint32_t answer, uint32_t mbar) {
    mbar_arrive_tx(mbar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                 :: "r"(answer), "r"(mbar) : "memory");
}
// Its number, -1 where there was none.
__device__ __forceinline__ int read_place(uint32_t answer) {
    int x;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\tld.shared.b128 r, [%1];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tmov.b32 %0, -1;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}\n"
        : "=r"(x) : "r"(answer) : "memory");
    return x;
}

template <int D, bool PREFIX>
__global__ void __launch_bounds__(kWarps * 32, 1)
    attn_tc_kernel(const TcParams p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv) {
    using C = Shape<D>;
    extern __shared__ unsigned char raw[];
    __shared__ Barriers bars;
    __shared__ Job jobs[2];
    __shared__ __align__(16) unsigned char answer[16];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_busy[2];
    __shared__ int limits[PREFIX ? 2 * kTile : 1];            // per token of the job: end of the keys that it sees
    __shared__ uint32_t missing[PREFIX ? 16 : 1];             // per key tile: a bit per 16 keys without a page
    const AttnArgs& a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, group = a.group;
    if (PREFIX) grid_dep_launch();  // the own keys' CTAs start where this grid's have left
    volatile int* abort = abort_busy;  // a wait gave up; warps with rows to compute once more

    const uint32_t q_smem = (smem_u32(raw) + 1023) & ~1023u, ring = q_smem + 2 * C::TILE_BYTES;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars.q[i]), 1);
            mbar_init(smem_u32(&bars.q_free[i]), 1);
            mbar_init(smem_u32(&bars.s[i]), 1);
            mbar_init(smem_u32(&bars.p[i]), 4);
            mbar_init(smem_u32(&bars.o[i]), 1);
            mbar_init(smem_u32(&bars.o_free[i]), 4);
            mbar_init(smem_u32(&bars.job[i]), 1);
            mbar_init(smem_u32(&bars.asked[i]), 1);
            mbar_init(smem_u32(&bars.job_free[i]), 11);  // the MMAs' thread and ten warps
        }
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(smem_u32(&bars.full[i]), 1);
            mbar_init(smem_u32(&bars.empty[i]), 1);
            mbar_init(smem_u32(&bars.fixed[i]), 1);
        }
        mbar_init(smem_u32(&bars.ahead), 1);
        mbar_init(smem_u32(&bars.limits_free), 8);
        mbar_init(smem_u32(&bars.place), 1);
        mbar_init(smem_u32(&bars.drain), 1);
        mbar_fence_init();
        abort_busy[0] = abort_busy[1] = 0;
    }
    if (warp == 9) tmem_alloc(smem_u32(&tmem_slot), 512);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kOtherRegs));
        if (warp == 8) {
            // ---- copies ----
            int it = 0, count = 0, q_uses[2] = {0, 0};  // tiles of the ring (keys and values in turn) and jobs so far
            bool ok = true;
            const int pieces = kTile / p.box;
            auto page_of = [&](int piece) {
                const int64_t key = (int64_t)piece * p.box;
                return key < a.cache.prefix_len ? a.cache.prefix[key >> a.cache.page_bits] : -1;
            };
            for (;; ++count) {
                ok = mbar_wait_busy(smem_u32(&bars.job[count & 1]), (count / 2) & 1, abort);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                const Job job = jobs[count & 1];
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars.job_free[count & 1]));
                if (job.n < 0) break;
                const int from = job.from, to = max(job.to[0], job.to[1]), tiles = to - from, begin = it;
                for (int t = 0; t < 2 && ok; ++t) {
                    if (job.to[t] <= from) continue;
                    if (q_uses[t]) ok = mbar_wait_busy(smem_u32(&bars.q_free[t]), (q_uses[t] - 1) & 1, abort);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    ++q_uses[t];
                    if (lane == 0) {
                        const uint32_t mbar = smem_u32(&bars.q[t]);
                        mbar_arrive_tx(mbar, C::BLOCKS * p.tokens * group * 128);
                        for (int c = 0; c < C::BLOCKS; ++c)
                            tma_3d(q_smem + t * C::TILE_BYTES + c * C::BLOCK_BYTES, &mq, c * 64, job.h * group,
                                   (int)(job.t0 + job.i0 + t * p.tokens), mbar);
                    }
                }
                int held = 0, asked = PREFIX ? page_of(from * pieces + lane) : 0, at = -64;
                for (; it < begin + 2 * tiles && ok; ++it) {
                    // with a ring of tiles left to load the next place is looked for
                    if (lane == 0 && it == max(begin, begin + 2 * tiles - C::STAGES)) mbar_arrive(smem_u32(&bars.ahead));
                    const int stage = it % C::STAGES, j = from + ((it - begin) >> 1);
                    const bool value = (it - begin) & 1;
                    if (it >= C::STAGES) ok = mbar_wait_busy(smem_u32(&bars.empty[stage]), (it / C::STAGES - 1) & 1, abort);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    const uint32_t mbar = smem_u32(&bars.full[stage]), dst = ring + stage * C::TILE_BYTES;
                    const CUtensorMap* map = value ? &mv : &mk;
                    if (PREFIX) {
                        // piece `lane` of the tile; one without a page lies before the cache's first row, where a
                        // copy reads zeros (a weight of 0 would not keep another page's NaN out), and is
                        // masked.  The pages are those of 32 pieces, asked for 32 pieces ahead
                        const int first = j * pieces;
                        if (first + pieces > at + 32) {
                            at = first;
                            held = asked;
                            asked = page_of(at + 32 + lane);
                        }
                        const int page = __shfl_sync(0xffffffffu, held, (first - at + lane) & 31);
                        const int64_t key = (int64_t)j * kTile + lane * p.box;
                        bool gone = page < 0 || page >= a.cache.num_pages;
                        const int row = gone ? -p.box : (int)((((int64_t)page * a.Hkv + job.h) << a.cache.page_bits) +
                                                              (key & (a.cache.page_size - 1)));
                        gone = gone && key < a.cache.prefix_len;
                        const bool part = __shfl_sync(0xffffffffu, gone, lane * 16 / p.box & 31);
                        const uint32_t out = __ballot_sync(0xffffffffu, part && lane < kTile / 16);
                        if (lane == 0) {
                            // the ring holds 4 key tiles at most, and the MMAs are one ahead of the softmax
                            if (!value) missing[(it >> 1) & 15] = out;
                            mbar_arrive_tx(mbar, C::TILE_BYTES);
                        }
                        __syncwarp();
                        if (lane < pieces)
                            for (int c = 0; c < C::BLOCKS; ++c)
                                tma_2d(dst + c * C::BLOCK_BYTES + lane * p.box * 128, map, c * 64, row, mbar);
                    } else if (lane == 0) {
                        mbar_arrive_tx(mbar, C::TILE_BYTES);
                        for (int c = 0; c < C::BLOCKS; ++c)
                            tma_3d(dst + c * C::BLOCK_BYTES, map, c * 64, job.h, (int)(job.t0 + (int64_t)j * kTile), mbar);
                    }
                }
                if (!ok) break;
                if (lane == 0) mbar_arrive(smem_u32(&bars.asked[count & 1]));
            }
            if (!ok) *abort = 1;
            // nothing may still be arriving when the CTA leaves
            for (int i = max(0, it - C::STAGES); i < it; ++i)
                if (!mbar_wait_copies(smem_u32(&bars.full[i % C::STAGES]), (i / C::STAGES) & 1)) *abort = 1;
            for (int t = 0; t < 2; ++t)
                if (q_uses[t] && !mbar_wait_copies(smem_u32(&bars.q[t]), (q_uses[t] - 1) & 1)) *abort = 1;
        } else if (warp == 9) {
            // ---- MMAs ----
            // An MMA takes its operands from uniform registers, and one that a single lane has computed
            // costs a trip there each time, more than the MMA itself: so the whole warp walks
            // through the jobs, with values that are the same in all lanes, and one issues.
            constexpr uint32_t idesc_s = idesc_bf16(kTile, kTile, false, false);
            constexpr uint32_t idesc_o = idesc_bf16(kTile, D, false, true);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint64_t q0 = smem_desc(q_smem, 16, 1024, kSwizzle128);
            const uint64_t k0 = smem_desc(ring, 16, 1024, kSwizzle128);
            const uint64_t v0 = smem_desc(ring, C::BLOCK_BYTES, 1024, kSwizzle128);
            bool ok = true;
            auto wait = [&](uint64_t* bar, int phase) {
                ok = __all_sync(0xffffffffu, mbar_wait_busy(smem_u32(bar), phase & 1, abort));
                if (!ok) *abort = 1;
                return ok;
            };
            auto there = [&](int it) { return wait(&bars.full[it % C::STAGES], it / C::STAGES); };
            auto same = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
            auto commit = [&](uint64_t* bar) {
                if (elect_one()) mma_commit(smem_u32(bar));
            };
            // of the ring's tiles so far; of each row tile: the jobs that had it, its key tiles
            int begin = 0, uses[2] = {0, 0}, p_uses[2] = {0, 0};
            uint32_t fixes = 0;  // a bit per stage: the phase of its `fixed`
            for (int count = 0; ok; ++count) {
                if (!wait(&bars.job[count & 1], count / 2)) break;
                const Job& job = jobs[count & 1];
                const int n = same(job.n), from = same(job.from), clear = same(job.clear);
                const int mine[2] = {same(job.to[0]) - from, same(job.to[1]) - from};
                if (lane == 0) mbar_arrive(smem_u32(&bars.job_free[count & 1]));
                if (n < 0) break;
                const int tiles = max(mine[0], mine[1]);
                // S of key tile i follows the O += P V of the tile before
                for (int i = 0; i <= tiles && ok; ++i) {
                    const int ik = begin + 2 * i, iv = ik - 1;
                    if (i > 0 && !there(iv)) break;
                    if (i == tiles && clear) {
                        const int stage = iv % C::STAGES;
                        if (!wait(&bars.fixed[stage], fixes >> stage)) break;
                        fixes ^= 1u << stage;
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (!ok) break;
                        if (i > 0 && i <= mine[t]) {
                            // O of the job before is read before it is written again
                            if (i == 1 && uses[t] > 0 && !wait(&bars.o_free[t], uses[t] - 1)) break;
                            if (!wait(&bars.p[t], p_uses[t] + i - 1)) break;
                            fence_after();
                            const uint64_t v = v0 + iv % C::STAGES * (C::TILE_BYTES / 16);
                            if (elect_one()) {
#pragma unroll
                                for (int ks = 0; ks < kTile / 16; ++ks)
                                    mma_bf16_ta(tm + C::O + t * D, tm + C::S + t * kTile + ks * 8, v + ks * 128, idesc_o,
                                                i > 1 || ks > 0);
                            }
                            if (i == mine[t]) commit(&bars.o[t]);
                        }
                        if (i < mine[t]) {
                            if (!there(ik)) break;
                            if (i == 0 && !wait(&bars.q[t], uses[t])) break;
                            fence_after();
                            const uint64_t q = q0 + t * (C::TILE_BYTES / 16), k = k0 + ik % C::STAGES * (C::TILE_BYTES / 16);
                            if (elect_one()) {
#pragma unroll
                                for (int ks = 0; ks < D / 16; ++ks) {
                                    const uint32_t off = (ks >> 2) * (C::BLOCK_BYTES / 16) + (ks & 3) * 2;
                                    mma_bf16(tm + C::S + t * kTile, q + off, k + off, idesc_s, ks > 0);
                                }
                                mma_commit(smem_u32(&bars.s[t]));
                            }
                            if (i + 1 == mine[t]) commit(&bars.q_free[t]);
                        }
                    }
                    if (!ok) break;
                    if (i > 0) commit(&bars.empty[iv % C::STAGES]);
                    if (i < tiles) commit(&bars.empty[ik % C::STAGES]);
                }
                begin += 2 * tiles;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    uses[t] += mine[t] > 0;
                    p_uses[t] += max(mine[t], 0);
                }
            }
            // no MMA may still be running when tensor memory is given back
            commit(&bars.drain);
            if (!mbar_wait_copies(smem_u32(&bars.drain), 0)) *abort = 1;
            __syncwarp();
        } else if (warp == 10) {
            // ---- values behind the end ----
            int begin = 0;
            for (int count = 0;; ++count) {
                const int b = count & 1;
                auto wait = [&](uint64_t* bar, int phase) {
                    return __all_sync(0xffffffffu, mbar_wait_busy(smem_u32(bar), phase & 1, abort));
                };
                bool ok = wait(&bars.job[b], count / 2);
                if (ok) {
                    const Job& job = jobs[b];
                    if (job.n < 0) break;
                    const int to = max(job.to[0], job.to[1]);
                    begin += 2 * (to - job.from);
                    ok = wait(&bars.asked[b], count / 2);
                    if (ok && job.clear) {
                        const int last = begin - 1, stage = last % C::STAGES;
                        ok = wait(&bars.full[stage], last / C::STAGES);
                        if (ok) {
                            unsigned char* v = raw + (ring + stage * C::TILE_BYTES - smem_u32(raw));
                            for (int i = (job.keys - (to - 1) * kTile) * 8 + lane; i < kTile * 8; i += 32)
                                for (int c = 0; c < C::BLOCKS; ++c)
                                    *reinterpret_cast<uint4*>(v + c * C::BLOCK_BYTES + i * 16) = make_uint4(0, 0, 0, 0);
                            fence_proxy_async();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(smem_u32(&bars.fixed[stage]));
                        }
                    }
                    __syncwarp();
                    if (ok && lane == 0) mbar_arrive(smem_u32(&bars.job_free[b]));
                }
                if (!ok) {
                    *abort = 1;
                    break;
                }
            }
        } else {
            // ---- places ----
            const uint32_t at_answer = smem_u32(answer);
            const int pair_tokens = 2 * p.tokens;
            const int64_t places = PREFIX ? 1 : gridDim.x / a.Hkv;
            int pairs[2] = {0, 0};
            if (!PREFIX && a.N <= kSorted) {
                pairs[0] = pairs_of(a, pair_tokens, lane);
                pairs[1] = pairs_of(a, pair_tokens, lane + 32);
            }
            const int far_tiles = PREFIX ? (a.cache.prefix_len + kTile - 1) / kTile : 1;
            const int64_t units = PREFIX ? (a.T + pair_tokens - 1) / pair_tokens * a.Hkv * far_tiles : 1;
            int64_t unit = units * blockIdx.x / gridDim.x;
            const int64_t unit_end = units * (blockIdx.x + 1) / gridDim.x;
            bool ok = true;
            int count = 0;
            for (int place = blockIdx.x, asked = 0; place >= 0; ++asked) {
                Job job;
                bool found;
                if (PREFIX) {
                    // the next tiles of this CTA's share, up to the end of a block of rows
                    const int64_t block = unit / far_tiles;
                    const int from = (int)(unit - block * far_tiles);
                    const int to = (int)min((int64_t)far_tiles, from + unit_end - unit);
                    const int64_t first = block / a.Hkv * pair_tokens;
                    job.t0 = 0;
                    job.i0 = first;
                    job.end = a.T;
                    job.from = from;
                    job.to[0] = to;
                    job.to[1] = first + p.tokens < a.T ? to : from;
                    job.keys = a.cache.prefix_len;
                    job.n = 0;
                    job.h = (int)(block % a.Hkv);
                    job.part = (int)(blockIdx.x - cta_of(block * far_tiles, units, gridDim.x));
                    job.clear = job.keys < to * kTile;
                    unit += to - from;
                    found = true;
                } else {
                    found = find_job(a, pair_tokens, pairs, place / a.Hkv, places, place % a.Hkv, job);
                }
                if (found) {
                    if (count >= 2) ok = mbar_wait_busy(smem_u32(&bars.job_free[count & 1]), (count / 2 - 1) & 1, abort);
                    // the limits have one place, which those of the job before have to leave
                    if (PREFIX && ok && count >= 1) ok = mbar_wait_busy(smem_u32(&bars.limits_free), (count - 1) & 1, abort);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    if (PREFIX) mark_limits(a, job.i0, pair_tokens, limits);
                    if (lane == 0) {
                        jobs[count & 1] = job;
                        mbar_arrive(smem_u32(&bars.job[count & 1]));
                    }
                    ok = __all_sync(0xffffffffu, mbar_wait_busy(smem_u32(&bars.ahead), count & 1, abort));
                    ++count;
                    if (!ok) break;
                }
                if (PREFIX && unit == unit_end) break;
                if (PREFIX) continue;
                if (lane == 0) ask_place(at_answer, smem_u32(&bars.place));
                // it arrives whatever happens to the others, and none may be on its way when the CTA leaves
                ok = __all_sync(0xffffffffu, mbar_wait_copies(smem_u32(&bars.place), asked & 1));
                if (!ok) break;
                place = read_place(at_answer);
                fence_proxy_async();  // read before the next answer is written
                __syncwarp();
            }
            // no more jobs
            if (ok && count >= 2) ok = mbar_wait_busy(smem_u32(&bars.job_free[count & 1]), (count / 2 - 1) & 1, abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) *abort = 1;
            if (ok && lane == 0) {
                jobs[count & 1].n = -1;
                mbar_arrive(smem_u32(&bars.job[count & 1]));
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kSoftmaxRegs));
        // ---- softmax: a row per thread ----
        const int t = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // lane 32 (warp % 4) in the upper half
        const uint32_t ts = tmem + C::S + t * kTile + lanes, to_ = tmem + C::O + t * D + lanes;
        const float c = a.scale_log2;
        unsigned char* const out = raw + (ring + C::STAGES * C::TILE_BYTES - smem_u32(raw)) + warp * C::OUT_BYTES;
        int s_uses = 0, o_uses = 0;
        int tiles_before = 0;  // key tiles of the jobs so far
        for (int count = 0;; ++count) {
            bool ok = mbar_wait_busy(smem_u32(&bars.job[count & 1]), (count / 2) & 1, abort);
            if (!(ok = __all_sync(0xffffffffu, ok))) {
                *abort = 1;
                break;
            }
            const Job& job = jobs[count & 1];
            if (job.n < 0) break;
            const int from = job.from, end = job.to[t], first_tile = tiles_before;
            tiles_before += max(job.to[0], job.to[1]) - from;
            // what the loop does not need is read once more behind it: S takes the registers
            int limit = kNoRow;
            if (end > from) {
                const int local = row / group + t * p.tokens;  // token within the job
                if (row < p.tokens * group && job.i0 + local < job.end) {
                    limit = PREFIX ? limits[local] : (int)job.i0 + local + 1;
                    if (PREFIX && limit == 0) limit = kNoRow;  // padding has no row to leave
                }
            }
            __syncwarp();
            if (PREFIX && lane == 0) mbar_arrive(smem_u32(&bars.limits_free));
            if (end <= from) {
                if (lane == 0) mbar_arrive(smem_u32(&bars.job_free[count & 1]));
                continue;
            }
            float m = -INFINITY;
            float2 sum = make_float2(0.f, 0.f);
            for (int j = from, i = 0; j < end; ++j, ++i) {
                ok = mbar_wait_busy(smem_u32(&bars.s[t]), s_uses++ & 1, abort);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                fence_after();
                float s[kTile];
#pragma unroll
                for (int b = 0; b < 4; ++b) tmem_fetch32(ts + b * 32, s + b * 32);
                const uint32_t gone = PREFIX ? missing[(first_tile + i) & 15] : 0;
                tmem_wait_ld();
#pragma unroll
                for (int b = 0; b < 4; ++b) arrived32(s + b * 32);
                const int seen = limit - j * kTile;
                if (__any_sync(0xffffffffu, seen < kTile || (PREFIX && gone))) {
#pragma unroll
                    for (int k = 0; k < kTile; ++k)
                        if (k >= seen || (PREFIX && (gone >> (k / 16) & 1))) s[k] = -INFINITY;
                }
                float top = s[0];
#pragma unroll
                for (int k = 1; k < kTile; ++k) top = fmaxf(top, s[k]);
                top *= c;
                // (a lane without a row has what was left in shared memory: it does not decide)
                if (__any_sync(0xffffffffu, limit != kNoRow && top > m + kLag)) {
                    // to the new maximum where it has risen, by 1 where it has not
                    const float now = fmaxf(top, m), back = now == -INFINITY ? 1.f : ex2(m - now);
                    m = now;
                    sum.x *= back;
                    sum.y *= back;
                    if (i > 0) {
#pragma unroll
                        for (int b = 0; b < D; b += 32) {
                            float o[32];
                            tmem_fetch32(to_ + b, o);
                            tmem_wait_ld();
                            arrived32(o);
                            uint32_t u[32];
#pragma unroll
                            for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(o[k] * back);
                            tmem_put32(to_ + b, u);
                        }
                    }
                }
                const float base = m == -INFINITY ? 0.f : -kLag - m;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t pk[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const float2 x = __ffma2_rn(make_float2(s[b * 64 + 2 * k], s[b * 64 + 2 * k + 1]),
                                                    make_float2(c, c), make_float2(base, base));
                        const float2 e = make_float2(ex2(x.x), ex2(x.y));
                        sum = __fadd2_rn(sum, e);
                        pk[k] = pack_bf16(e.x, e.y);
                    }
                    tmem_put32(ts + b * 32, pk);
                }
                tmem_wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars.p[t]));
            }
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait_busy(smem_u32(&bars.o[t]), o_uses++ & 1, abort));
            if (!ok) {
                *abort = 1;
                break;
            }
            fence_after();
            const float l = sum.x + sum.y, inv = 1.f / l;
            const bool there = limit != kNoRow;
            const int h = job.h, part = PREFIX ? job.part : 0, local = row / group;
            const int64_t head = (int64_t)h * group + row - local * group;
            const int64_t token = job.i0 + local + t * p.tokens, t0 = job.t0;  // within the sequence
            const int64_t place = ((int64_t)part * a.T + t0 + token) * a.Hq + head;  // PREFIX
            char* to_row = PREFIX ? reinterpret_cast<char*>(p.w.far_sum + place * D)
                                  : reinterpret_cast<char*>(static_cast<__nv_bfloat16*>(a.o) + (t0 + token) * a.ldo + head * D);
            float any = 0.f;  // stays 0 but for an infinity or a NaN
            // a warp's rows through shared memory, 128 bytes of each at a time: what leaves are whole lines
            constexpr int COLS = PREFIX ? 32 : 64;
#pragma unroll
            for (int b = 0; b < D; b += COLS) {
                uint32_t w[32];
#pragma unroll
                for (int e = 0; e < COLS; e += 32) {
                    float o[32];
                    tmem_fetch32(to_ + b + e, o);
                    tmem_wait_ld();
                    arrived32(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k) any = fmaf(o[k], 0.f, any);
                    if (PREFIX) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(o[k]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; ++k) w[(e / 2 + k) & 31] = pack_bf16(o[2 * k] * inv, o[2 * k + 1] * inv);
                    }
                }
                if (b + COLS == D) {
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars.o_free[t]));
                }
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<uint4*>(out + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                        make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int r = k * 4 + (lane >> 3), ch = lane & 7;
                    char* to_it = reinterpret_cast<char*>(
                        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(there ? to_row : nullptr), r));
                    if (to_it)
                        *reinterpret_cast<uint4*>(to_it + b * (PREFIX ? 4 : 2) + ch * 16) =
                            *reinterpret_cast<const uint4*>(out + r * 128 + ((ch ^ (r & 7)) << 4));
                }
                __syncwarp();
            }
            if (PREFIX && there) p.w.far_stat[place] = make_float2(m + kLag, l);
            // A sum of weights that is a NaN comes from a score that the row sees, and the row is right as
            // it is; one of 0 from scores of -inf alone (the prefix's merge leaves such a part out).
            const uint32_t zero = PREFIX ? 0 : __ballot_sync(0xffffffffu, there && l == 0.f);
            const uint32_t bad = __ballot_sync(0xffffffffu, there && any != 0.f && l > 0.f);
            if (zero | bad) {
                if (lane == 0) atomicAdd(&abort_busy[1], 1);
                if (zero >> lane & 1)
                    for (int d = 0; d < D; d += 8) *reinterpret_cast<uint4*>(to_row + d * 2) = make_uint4(0, 0, 0, 0);
                if (bad) {
                    // by value: what the call takes by reference would live in local memory
                    const Paged cache = a.cache;
                    const int Hkv = a.Hkv;
                    const int64_t ldk = a.ldk, ldv = a.ldv;
                    const __nv_bfloat16* keys = static_cast<const __nv_bfloat16*>(a.k) + t0 * ldk + (int64_t)h * D;
                    const __nv_bfloat16* vals = static_cast<const __nv_bfloat16*>(a.v) + t0 * ldv + (int64_t)h * D;
                    const int loaded = job.clear ? min(job.keys, end * kTile) : end * kTile;
                    rows_again<D>(bad, PREFIX, static_cast<const __nv_bfloat16*>(a.q) + (t0 + token) * a.ldq + head * D,
                                  to_row, PREFIX ? p.w.far_stat + place : nullptr, limit, from * kTile, loaded, c,
                                  [=](int64_t key, const __nv_bfloat16*& kp, const __nv_bfloat16*& vp) {
                                      if (PREFIX) return cached_row<D>(cache, cache.prefix, Hkv, h, key, kp, vp);
                                      kp = keys + key * ldk;
                                      vp = vals + key * ldv;
                                      return true;
                                  });
                }
                __syncwarp();
                if (lane == 0) atomicSub(&abort_busy[1], 1);
            }
            if (lane == 0) mbar_arrive(smem_u32(&bars.job_free[count & 1]));
        }
    }
    fence_before();
    __syncwarp();
    __syncthreads();
    if (tid == 0 && abort_busy[0]) atomicOr(p.err, kAttnError);
    if (warp == 9) {
        fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---- launches -----------------------------------------------------------------------

template <int D, bool PREFIX>
cudaError_t launch_tc(TcParams p, dim3 grid, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                      cudaStream_t s) {
    static std::atomic<uint64_t> known{0};
    const cudaError_t set = allow_smem(attn_tc_kernel<D, PREFIX>, Shape<D>::SMEM, known);
    if (set != cudaSuccess) return set;
    // a warpgroup that asks for more registers than the block was launched with waits forever
    static std::atomic<bool> enough{false};
    if (!enough.load(std::memory_order_relaxed)) {
        cudaFuncAttributes f;
        const cudaError_t got = cudaFuncGetAttributes(&f, attn_tc_kernel<D, PREFIX>);
        if (got != cudaSuccess) return got;
        if (f.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
        enough.store(true, std::memory_order_relaxed);
    }
    p.err = device_error_word();
    KernelTimer kt(PREFIX ? "attn_prefix_tc" : "attn_prompt_tc", s);
    attn_tc_kernel<D, PREFIX><<<grid, kWarps * 32, Shape<D>::SMEM, s>>>(p, mq, mk, mv);
    return cudaGetLastError();
}

}  // namespace

uint64_t context_number() {
    using GetId = CUresult (*)(CUcontext, unsigned long long*);
    static std::atomic<GetId> known{nullptr};
    GetId get = known.load(std::memory_order_acquire);
    if (!get) {
        void* entry = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &entry, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return 0;
        get = reinterpret_cast<GetId>(entry);
        known.store(get, std::memory_order_release);
    }
    unsigned long long id = 0;
    return get(nullptr, &id) == CUDA_SUCCESS ? id + 1 : 0;
}

int prefix_block_tokens(int group) { return 2 * (kTile / group); }

cudaError_t launch_prompt_tc(const AttnArgs& a, cudaStream_t s) {
    TcParams p{};
    p.a = a;
    p.tokens = kTile / a.group;
    p.box = kTile;
    CUtensorMap mq, mk, mv;
    if (!encode_tokens(&mq, a.q, a.ldq, a.T, a.Hq, a.D, a.group, p.tokens) ||
        !encode_tokens(&mk, a.k, a.ldk, a.T, a.Hkv, a.D, 1, kTile) ||
        !encode_tokens(&mv, a.v, a.ldv, a.T, a.Hkv, a.D, 1, kTile))
        return cudaErrorInvalidValue;
    const dim3 grid((unsigned)((a.T / (2 * p.tokens) + a.N) * a.Hkv));
    return a.D == 128 ? launch_tc<128, false>(p, grid, mq, mk, mv, s) : launch_tc<64, false>(p, grid, mq, mk, mv, s);
}

cudaError_t launch_prefix_tc(const AttnArgs& a, const StepWork& w, cudaStream_t s) {
    TcParams p{};
    p.a = a;
    p.w = w;
    p.tokens = kTile / a.group;
    p.box = a.cache.page_size < kTile ? a.cache.page_size : kTile;
    CUtensorMap mq, mk, mv;
    const int64_t rows = (int64_t)a.cache.num_pages * a.Hkv << a.cache.page_bits;
    if (!encode_tokens(&mq, a.q, a.ldq, a.T, a.Hq, a.D, a.group, p.tokens) ||
        !encode_cache(&mk, a.cache.k, rows, a.D, p.box) || !encode_cache(&mv, a.cache.v, rows, a.D, p.box))
        return cudaErrorInvalidValue;
    const dim3 grid((unsigned)w.far_ctas);
    return a.D == 128 ? launch_tc<128, true>(p, grid, mq, mk, mv, s) : launch_tc<64, true>(p, grid, mq, mk, mv, s);
}

}  // namespace gdr
