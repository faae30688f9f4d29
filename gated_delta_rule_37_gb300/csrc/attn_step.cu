// The step over the paged cache in bf16: the sequences' own keys (contract in
// include/gdr.h, the cut of the work in attn_step.cuh).
//
// A step reads every key and value once for few rows (tokens times the heads that read
// one key head): memory bounds it, at 64 rows still.  What it takes is enough bytes in
// flight per SM and arithmetic that keeps out of the way: one warp copies tiles of 64
// keys and their values into a ring by TMA, pages in any order, across the borders of
// rows and sequences; eight warps work on them with the warp-wide matrix instructions
// (m16n8k16, bf16 in, fp32 out), whose 16 rows fit the few there are.  (tcgen05's tiles
// have 128 rows at least: with 4 to 64 of them filled it would read shared memory for
// empty ones.)
//   A warp has 16 rows and 16 or 32 of a tile's 64 keys, and a running maximum and sum of its
// own, so that no tile needs a barrier; the warps' results are joined at the end of a run.
// With up to 16 rows two sets of four warps take the tiles in turn; with more, rows are what
// the warps share out first: fewer results to join.
//   A row whose sums are not finite is written as it is.  Where the run has a key that the row does not
// see, whose value may have reached it as 0 * inf, the warps look at the values again: never in decode.
//   Measured: 256 sequences of up to 4096 keys, 32 heads of 128 on 8, 300 us, 6.5 TB/s; one of 65536
// 50 us, of which 5 pass before the first tile is there, the last ones in the merge; 230 of up to 1024 behind
// a prefix 80 us, 6.1 TB/s, where a run's beginning and end (1.9 us) count.
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

constexpr int kReaders = 8;  // warps that compute
constexpr int kStepBlock = (kReaders + 1) * 32;

// ROWS rows a run: GROUPS of 16, each with the warps that have its keys.
template <int D, int ROWS> struct StepShape {
    static constexpr int GROUPS = ROWS / 16, SHARE = kReaders / GROUPS;  // SHARE warps have the same rows
    static constexpr int KEYS = ROWS == 64 ? 32 : 16;                    // of a tile, per warp
    static constexpr bool TURNS = SHARE * KEYS > kKeyTile;               // two sets of warps take the tiles in turn
    static constexpr int BLOCKS = D / 64, BLOCK_BYTES = kKeyTile * 128, TILE_BYTES = BLOCKS * BLOCK_BYTES;
    static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
    // Where two sets take the tiles in turn a stage belongs to one of them, for good: a wait
    // by parity knows only its barrier's last phase, and a set that skips a stage's tile
    // could take the phase before the skipped one for its own.
    static constexpr int STAGES = D == 64 ? 10 : ROWS == 16 ? 6 : 5;
    static_assert(!TURNS || STAGES % 2 == 0, "a stage per set");
    static constexpr int Q_STRIDE = D * 2 + 16;   // a row of queries: 8 rows of a matrix on different banks
    // joined at a time: 8 rows of each group, half of the columns
    static constexpr int PART = D / 2, PART_LD = PART + 4;
    static constexpr int JOIN_BYTES = kReaders * 8 * PART_LD * 4;
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + 2 * ROWS * Q_STRIDE + JOIN_BYTES;
};

struct StepJob {
    int t0, len, least, most;  // first token; keys before the call's; the keys that some row sees: least .. most - 1
    int n, h, r0, rows, from, to, slot;
};

// A run with rows whose sums hold an infinity or a NaN, a bit each.
struct BadRun {
    StepJob job;
    uint32_t rows[2];
};

struct StepBarriers {
    uint64_t full[10], empty[10], q_full[2], q_empty[2];
};

struct StepParams {
    AttnArgs a;
    StepWork w;
    int box;  // rows of one copy: 64, or a page's
    unsigned* err;
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Barrier of the eight warps; whether any of their threads says so.  The threads of a warp
// come from a wait one by one and have to arrive together: a warp counts as a whole.
__device__ __forceinline__ bool any_reader(bool x) {
    uint32_t r;
    __syncwarp();
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred.aligned q, 1, %2, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}\n" : "=r"(r) : "r"((uint32_t)x), "n"(kReaders * 32) : "memory");
    return r != 0;
}

// These rows, by the eight warps: lane i of a warp has row 8 i + warp.  Of a row whose weights' sum is a
// NaN, from a score that it sees, all is one already.
template <int D, int ROWS>
__device__ __noinline__ void run_again(const StepParams& p, const BadRun& run, const float2 (*stats)[16]) {
    const AttnArgs& a = p.a;
    const StepJob& j = run.job;
    const int lane = threadIdx.x & 31, r = min(lane * kReaders + (int)(threadIdx.x >> 5), ROWS - 1);
    const bool mine = lane < ROWS / kReaders && (run.rows[r >> 5] >> (r & 31) & 1);
    using C = StepShape<D, ROWS>;
    float weights = 0.f;
    for (int w = 0; w < C::SHARE; ++w) weights += stats[w * C::GROUPS + r / 16][r % 16].y;
    const int64_t token = j.t0 + (j.r0 + r) / a.group;
    const int head = j.h * a.group + (j.r0 + r) % a.group;
    const bool whole = j.slot < 0 && p.w.splits == 0;
    const int64_t at = j.slot < 0 ? token * a.Hq + head : ((int64_t)blockIdx.x * 2 + j.slot) * ROWS + r;
    auto* const o = static_cast<__nv_bfloat16*>(a.o) + token * a.ldo + (int64_t)head * D;
    // scores of -inf alone weigh nothing, whatever the values (the merge leaves such a part out)
    if (whole && mine && weights == 0.f)
        for (int d = 0; d < D; d += 8) *reinterpret_cast<uint4*>(o + d) = make_uint4(0, 0, 0, 0);
    const uint32_t rows = __ballot_sync(0xffffffffu, mine && weights > 0.f);
    if (!rows) return;
    // the end of the run's keys, and of those that the row sees: a row that sees all has met its own alone
    const int last = min(j.to * kKeyTile, j.most);
    const int end = (int)min((int64_t)j.len + (j.r0 + r) / a.group + 1, (int64_t)last);
    void* const to = whole ? static_cast<void*>(o) : (j.slot < 0 ? p.w.row_sum : p.w.slot_sum) + at * D;
    const Paged cache = a.cache;
    const int32_t* pages = a.cache.table + j.n * a.cache.table_ld;
    const int h = j.h, Hkv = a.Hkv;
    rows_again<D>(rows, !whole, static_cast<const __nv_bfloat16*>(a.q) + token * a.ldq + (int64_t)head * D, to,
                  (j.slot < 0 ? p.w.row_stat : p.w.slot_stat) + at, end, max(j.from * kKeyTile, j.least), last,
                  a.scale_log2, [=](int64_t key, const __nv_bfloat16*& kp, const __nv_bfloat16*& vp) {
                      return cached_row<D>(cache, pages, Hkv, h, key, kp, vp);
                  });
}

template <int D, int ROWS>
__global__ void __launch_bounds__(kStepBlock, 1)
    step_kernel(const __grid_constant__ StepParams p, const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap mv) {
    using C = StepShape<D, ROWS>;
    extern __shared__ unsigned char raw[];
    __shared__ StepBarriers bars;
    __shared__ StepJob jobs[2];
    __shared__ uint32_t missing[C::STAGES];     // a bit per 16 keys without a page
    __shared__ float2 stats[kReaders][16];
    __shared__ uint32_t bad_rows[2];
    __shared__ BadRun bad_run;
    __shared__ int abort_busy[2];
    const AttnArgs& a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort = abort_busy;  // a wait gave up; warps with rows to compute once more
    const uint32_t ring = (smem_u32(raw) + 1023) & ~1023u;
    const uint32_t queries = ring + C::STAGES * C::STAGE_BYTES;
    unsigned char* const base = raw + (ring - smem_u32(raw));
    float* const join = reinterpret_cast<float*>(base + C::STAGES * C::STAGE_BYTES + 2 * ROWS * C::Q_STRIDE);

    if (tid == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(smem_u32(&bars.full[i]), 1);
            mbar_init(smem_u32(&bars.empty[i]), C::TURNS ? kReaders / 2 : kReaders);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars.q_full[i]), 1);
            mbar_init(smem_u32(&bars.q_empty[i]), kReaders);
        }
        mbar_fence_init();
        abort_busy[0] = abort_busy[1] = 0;
        bad_rows[0] = bad_rows[1] = 0;
    }
    grid_dep_launch();
    const Plan plan = make_plan(a, p.w, blockIdx.x);  // ends with a barrier of the block

    if (warp == kReaders) {
        // ---- copies ----
        int it = 0, count = 0;  // tiles and runs so far
        bool ok = true;
        const int pieces = kKeyTile / p.box;  // copies of a tile
        // lane l: the page of piece `at` + l of a sequence
        auto pages_from = [&](int n, int at) {
            const int slot = (int)((int64_t)(at + lane) * p.box >> a.cache.page_bits);
            return slot < a.cache.max_pages ? a.cache.table[n * a.cache.table_ld + slot] : -1;
        };
        Runs runs(a, p.w, plan);
        Run run;
        bool more = runs.next(run);
        int held = more ? pages_from(run.n, run.from * pieces) : 0;
        while (more && ok) {
            const Run r = run;
            int pages = held, at = r.from * pieces;
            // the next run is looked up, and its first pages, before this one's copies are waited for
            more = runs.next(run);
            if (more) held = pages_from(run.n, run.from * pieces);
            const int q = count & 1;
            if (count >= 2) ok = mbar_wait_busy(smem_u32(&bars.q_empty[q]), (count / 2 - 1) & 1, abort);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            const int r0 = r.row_tile * ROWS, rows = min(ROWS, r.s.rows - r0);
            if (lane == 0) {
                StepJob& j = jobs[q];
                j.t0 = r.s.t0; j.len = r.s.len; j.n = r.n; j.h = r.h; j.r0 = r0; j.rows = rows;
                j.from = r.from; j.to = r.to; j.slot = r.slot;
                j.least = a.cache.prefix_len;
                j.most = (int)min((int64_t)r.s.len + (r0 + rows - 1) / a.group + 1, (int64_t)r.s.end);
                mbar_arrive_tx(smem_u32(&bars.q_full[q]), rows * D * 2);
            }
            __syncwarp();
            for (int i = lane; i < rows; i += 32) {
                const int token = (r0 + i) / a.group, head = r.h * a.group + (r0 + i) - token * a.group;
                bulk_g2s(queries + (q * ROWS + i) * C::Q_STRIDE,
                         static_cast<const __nv_bfloat16*>(a.q) + (int64_t)(r.s.t0 + token) * a.ldq + (int64_t)head * D,
                         D * 2, smem_u32(&bars.q_full[q]));
            }
            if (lane == 0) leave_cut(p.w, plan, blockIdx.x, r);
            ++count;
            for (int k = r.from; k < r.to; ++k, ++it) {
                const int stage = it % C::STAGES, first = k * pieces;  // the tile's first piece
                if (first + pieces > at + 32) {
                    at = first;
                    pages = pages_from(r.n, at);
                }
                const int page = __shfl_sync(0xffffffffu, pages, first - at + (lane & (pieces - 1)));
                const int key = k * kKeyTile + (lane & (pieces - 1)) * p.box;
                const bool gone = page < 0 || page >= a.cache.num_pages;
                // a piece without a page is read from the cache's first rows and left out
                const int row = gone ? 0 : (int)((((int64_t)page * a.Hkv + r.h) << a.cache.page_bits) +
                                                 (key & (a.cache.page_size - 1)));
                const bool part = __shfl_sync(0xffffffffu, gone, (lane & 3) * 16 / p.box);
                const uint32_t out = __ballot_sync(0xffffffffu, part && lane < 4);
                if (it >= C::STAGES) ok = mbar_wait_busy(smem_u32(&bars.empty[stage]), (it / C::STAGES - 1) & 1, abort);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                const uint32_t mbar = smem_u32(&bars.full[stage]), dst = ring + stage * C::STAGE_BYTES;
                if (lane == 0) {
                    missing[stage] = out;
                    mbar_arrive_tx(mbar, C::STAGE_BYTES);
                }
                __syncwarp();
                // lanes 0 .. pieces - 1 copy the keys, the next ones the values
                if (lane < 2 * pieces) {
                    const bool value = lane >= pieces;
                    for (int b = 0; b < C::BLOCKS; ++b)
                        tma_2d(dst + (value ? C::TILE_BYTES : 0) + b * C::BLOCK_BYTES + (lane & (pieces - 1)) * p.box * 128,
                               value ? &mv : &mk, b * 64, row, mbar);
                }
            }
        }
        // nothing may still be arriving when the CTA leaves; the queries' barriers are waited for
        // before the end is announced through them
        bool landed = true;
        for (int i = max(0, it - C::STAGES); i < it; ++i)
            landed &= mbar_wait_copies(smem_u32(&bars.full[i % C::STAGES]), (i / C::STAGES) & 1);
        for (int i = max(0, count - 2); i < count; ++i)
            landed &= mbar_wait_copies(smem_u32(&bars.q_full[i & 1]), (i / 2) & 1);
        if (ok && count >= 2) ok = mbar_wait_busy(smem_u32(&bars.q_empty[count & 1]), (count / 2 - 1) & 1, abort);
        ok = __all_sync(0xffffffffu, ok && landed);
        if (ok && lane == 0) {
            jobs[count & 1].n = -1;
            mbar_arrive(smem_u32(&bars.q_full[count & 1]));
        }
        if (!ok) *abort = 1;
        // the merge waits for this grid alone, so this one ends behind the prefix's
        grid_dep_wait();
    } else {
        // ---- arithmetic ----
        const int group = warp % C::GROUPS, share = warp / C::GROUPS;
        const int set = C::TURNS ? share >> 2 : 0, part = C::TURNS ? share & 3 : share;  // the warp's keys of a tile
        const int quad = lane >> 2, pair = lane & 3;  // rows quad and quad + 8, keys or columns 2 pair, 2 pair + 1
        const float c = a.scale_log2;
        constexpr int NT = C::KEYS / 8;               // 8 keys each
        int it = 0;
        for (int count = 0;; ++count) {
            const int q = count & 1;
            bool ok = mbar_wait_busy(smem_u32(&bars.q_full[q]), (count / 2) & 1, abort);
            if (any_reader(!ok)) {
                *abort = 1;
                break;
            }
            const StepJob j = jobs[q];
            if (j.n < 0) break;
            uint32_t aq[D / 16][4];
            {
                const uint32_t at = queries + (q * ROWS + group * 16 + (lane & 15)) * C::Q_STRIDE + (lane >> 4) * 16;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) ldmatrix4(aq[ks], at + ks * 32);
            }
            float m[2], l[2], acc[D / 8][4];
            int limit[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[i] = -INFINITY;
                l[i] = 0.f;
                limit[i] = (int)min((int64_t)j.len + (j.r0 + group * 16 + i * 8 + quad) / a.group + 1, (int64_t)j.most);
            }
            const int all_see = (int)min((int64_t)j.len + j.r0 / a.group + 1, (int64_t)j.most);  // end of the keys that every row sees
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;

            for (int k = j.from; k < j.to; ++k, ++it) {
                if (C::TURNS && (it & 1) != set) continue;
                const int stage = it % C::STAGES;
                if (ok) ok = __all_sync(0xffffffffu, mbar_wait_busy(smem_u32(&bars.full[stage]), (it / C::STAGES) & 1, abort));
                if (!ok) continue;
                const uint32_t ks_ = ring + stage * C::STAGE_BYTES, vs = ks_ + C::TILE_BYTES;
                const int key0 = k * kKeyTile + part * C::KEYS;
                float s[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
                {
                    // matrices of a load: keys 0-7 and 8-15 (lane / 16), channels 0-7 and 8-15 (lane / 8 % 2)
                    const int r = part * C::KEYS + (lane >> 4) * 8 + (lane & 7), ch = (lane >> 3) & 1;
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                        for (int n = 0; n < NT; n += 2) {
                            uint32_t b[4];
                            ldmatrix4(b, ks_ + chunk_k128(r + n * 8, ks * 2 + ch, kKeyTile));
                            mma16816(s[n], aq[ks], b[0], b[1]);
                            mma16816(s[n + 1], aq[ks], b[2], b[3]);
                        }
                }
                const uint32_t gone = missing[stage] >> (part * C::KEYS / 16) & ((1u << C::KEYS / 16) - 1);
                const bool edge = gone || key0 < j.least || key0 + C::KEYS > all_see;
                float now[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (edge) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int key = key0 + n * 8 + pair * 2 + e;
                                if ((gone >> (n / 2) & 1) || key < j.least || key >= limit[i]) s[n][i * 2 + e] = -INFINITY;
                            }
                    }
                    float top = fmaxf(s[0][i * 2], s[0][i * 2 + 1]);
#pragma unroll
                    for (int n = 1; n < NT; ++n) top = fmaxf(top, fmaxf(s[n][i * 2], s[n][i * 2 + 1]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    now[i] = fmaxf(m[i], top * c);
                }
                if (__any_sync(0xffffffffu, now[0] > m[0] || now[1] > m[1])) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float back = now[i] == -INFINITY ? 1.f : ex2(m[i] - now[i]);
                        m[i] = now[i];
                        l[i] *= back;
#pragma unroll
                        for (int n = 0; n < D / 8; ++n) {
                            acc[n][i * 2] *= back;
                            acc[n][i * 2 + 1] *= back;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float off = m[i] == -INFINITY ? 0.f : -m[i];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float x = ex2(fmaf(s[n][i * 2 + e], c, off));
                            s[n][i * 2 + e] = x;
                            l[i] += x;
                        }
                }
#pragma unroll
                for (int half = 0; half < NT / 2; ++half) {
                    // the weights as they lie are the next product's left operand
                    const uint32_t pk[4] = {pack_bf16(s[2 * half][0], s[2 * half][1]), pack_bf16(s[2 * half][2], s[2 * half][3]),
                                            pack_bf16(s[2 * half + 1][0], s[2 * half + 1][1]),
                                            pack_bf16(s[2 * half + 1][2], s[2 * half + 1][3])};
                    // what no row sees may hold anything: a weight of 0 does not keep a NaN out
                    uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
                    if (edge) {
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const int key = key0 + half * 16 + n * 8 + pair * 2;
                            const bool there = !(gone >> half & 1);
                            keep[n] = (there && key >= j.least && key < j.most ? 0xffffu : 0u) |
                                      (there && key + 1 >= j.least && key + 1 < j.most ? 0xffff0000u : 0u);
                        }
                    }
                    // matrices of a load: keys 0-7 and 8-15 (lane / 8 % 2), channels 0-7 and 8-15 (lane / 16)
                    const int r = part * C::KEYS + half * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), ch = lane >> 4;
#pragma unroll
                    for (int n = 0; n < D / 16; ++n) {
                        uint32_t b[4];
                        ldmatrix4_t(b, vs + chunk_k128(r, n * 2 + ch, kKeyTile));
                        if (edge) {
                            b[0] &= keep[0];
                            b[1] &= keep[1];
                            b[2] &= keep[0];
                            b[3] &= keep[1];
                        }
                        mma16816(acc[2 * n], pk, b[0], b[1]);
                        mma16816(acc[2 * n + 1], pk, b[2], b[3]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars.empty[stage]));
            }

            // ---- the warps' results joined ----
            if (lane == 0) mbar_arrive(smem_u32(&bars.q_empty[q]));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x = l[i];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                if (pair == 0) stats[warp][i * 8 + quad] = make_float2(m[i], x);
            }
            constexpr int C4 = C::PART / 4;                    // threads of a row
            constexpr int ITEMS = C::GROUPS * 8 * C4;          // of a part
            bool stop = false;
#pragma unroll
            for (int half = 0; half < 2; ++half) {             // rows 0-7 and 8-15 of each group
                if (stop || (half && j.rows <= 8)) break;
#pragma unroll
                for (int b = 0; b < 2; ++b) {                  // halves of the columns
                    constexpr int N8 = C::PART / 8;
#pragma unroll
                    for (int n = 0; n < N8; ++n)
                        *reinterpret_cast<float2*>(join + (warp * 8 + quad) * C::PART_LD + n * 8 + pair * 2) =
                            make_float2(acc[b * N8 + n][half * 2], acc[b * N8 + n][half * 2 + 1]);
                    stop = any_reader(!ok);
                    if (stop) break;
#pragma unroll
                    for (int i = tid; i < ITEMS; i += kReaders * 32) {
                        const int g = i / C4 / 8, r8 = i / C4 % 8, col = i % C4 * 4, r = g * 16 + half * 8 + r8;
                        if (r >= j.rows) continue;
                        float2 st[C::SHARE];
                        float top = -INFINITY;
#pragma unroll
                        for (int w = 0; w < C::SHARE; ++w) {
                            st[w] = stats[w * C::GROUPS + g][half * 8 + r8];
                            top = fmaxf(top, st[w].x);
                        }
                        const float off = top == -INFINITY ? 0.f : top;
                        float sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int w = 0; w < C::SHARE; ++w) {
                            const float f = ex2(st[w].x - off);
                            const float4 y = *reinterpret_cast<const float4*>(
                                join + ((w * C::GROUPS + g) * 8 + r8) * C::PART_LD + col);
                            sum = fmaf(st[w].y, f, sum);
                            x[0] = fmaf(y.x, f, x[0]);
                            x[1] = fmaf(y.y, f, x[1]);
                            x[2] = fmaf(y.z, f, x[2]);
                            x[3] = fmaf(y.w, f, x[3]);
                        }
                        if (!(fabsf(x[0]) + fabsf(x[1]) + fabsf(x[2]) + fabsf(x[3]) + sum < INFINITY))
                            atomicOr(&bad_rows[r >> 5], 1u << (r & 31));  // the same word whatever the order
                        const int local = (j.r0 + r) / a.group, head = j.h * a.group + j.r0 + r - local * a.group;
                        const int64_t token = j.t0 + local;
                        if (j.slot < 0 && p.w.splits == 0) {
                            const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
                            for (int e = 0; e < 4; ++e) x[e] *= inv;
                            Vec<__nv_bfloat16, 4>::store(static_cast<__nv_bfloat16*>(a.o) + token * a.ldo +
                                                             (int64_t)head * D + b * C::PART + col, x);
                        } else {
                            const int64_t at = j.slot < 0 ? token * a.Hq + head
                                                          : ((int64_t)blockIdx.x * 2 + j.slot) * ROWS + r;
                            Vec<float, 4>::store((j.slot < 0 ? p.w.row_sum : p.w.slot_sum) + at * D + b * C::PART + col, x);
                            if (b == 0 && col == 0) (j.slot < 0 ? p.w.row_stat : p.w.slot_stat)[at] = make_float2(top, sum);
                        }
                    }
                    any_reader(false);  // before the next part, or the next run's stats
                }
            }
            if (stop) {
                *abort = 1;
                break;
            }
            // rows that an infinity or a NaN has reached
            if (bad_rows[0] | bad_rows[1]) {
                any_reader(false);  // all have read the words
                if (tid == 0) {
                    bad_run = BadRun{j, {bad_rows[0], bad_rows[1]}};
                    bad_rows[0] = bad_rows[1] = 0;
                }
                if (lane == 0) atomicAdd(&abort_busy[1], 1);
                any_reader(false);
                run_again<D, ROWS>(p, bad_run, stats);
                __syncwarp();
                if (lane == 0) atomicSub(&abort_busy[1], 1);
                any_reader(false);  // the words are clear before the next run's join
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (tid == 0 && abort_busy[0]) atomicOr(p.err, kAttnError);
}

template <int D, int ROWS>
cudaError_t launch_rows(StepParams p, cudaStream_t s) {
    using C = StepShape<D, ROWS>;
    CUtensorMap mk, mv;
    const int64_t rows = (int64_t)p.a.cache.num_pages * p.a.Hkv << p.a.cache.page_bits;
    if (!encode_cache(&mk, p.a.cache.k, rows, D, p.box) || !encode_cache(&mv, p.a.cache.v, rows, D, p.box))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> known{0};
    const cudaError_t set = allow_smem(step_kernel<D, ROWS>, C::SMEM, known);
    if (set != cudaSuccess) return set;
    KernelTimer kt("attn_step", s);
    // behind the prefix's kernel, which reads the same inputs and writes nothing that this one reads
    if (p.w.splits > 0)
        return launch_dependent(step_kernel<D, ROWS>, dim3(p.w.ctas), dim3(kStepBlock), C::SMEM, s, p, mk, mv);
    step_kernel<D, ROWS><<<p.w.ctas, kStepBlock, C::SMEM, s>>>(p, mk, mv);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_head(const StepParams& p, cudaStream_t s) {
    return p.w.rows == 16   ? launch_rows<D, 16>(p, s)
           : p.w.rows == 32 ? launch_rows<D, 32>(p, s)
                            : launch_rows<D, 64>(p, s);
}

}  // namespace

cudaError_t launch_step_own(const AttnArgs& a, const StepWork& w, cudaStream_t s) {
    StepParams p{};
    p.a = a;
    p.w = w;
    p.box = a.cache.page_size < kKeyTile ? a.cache.page_size : kKeyTile;
    p.err = device_error_word();
    return a.D == 128 ? launch_head<128>(p, s) : launch_head<64>(p, s);
}

}  // namespace gdr
