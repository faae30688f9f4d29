// How gdr_attn_step cuts its work, shared by its kernels.
//
// The keys of a step are the prefix's, which every row of the batch sees, and each
// sequence's own.  The prefix is one tall problem (all tokens' rows of a key head
// against the same keys), cut along the keys into `splits` so that it fills the GPU.
// The own parts are as many problems as there are sequences and key heads, of lengths
// that only the device knows: their key tiles are numbered (sequence, key head, row
// tile, key tile) and every CTA takes an equal run of the numbers, so that ragged
// batches are as balanced as even ones and one long sequence fills the GPU as well as
// many short ones.  A row tile that lies within one CTA's run is finished there; one
// that is cut leaves a partial result (unnormalised sums, running maximum and sum) in
// each CTA's slots, of which a CTA needs two, for its first and its last row tile.  The
// merge joins the partial results of a row in the order of its keys: no atomics, and
// the bits do not depend on which CTA ran first.
#pragma once

#include "attn.h"
#include "common.cuh"

namespace gdr {

constexpr int kKeyTile = 64;       // keys per tile of the own parts
constexpr int kStepThreads = 256;  // threads that form the plan (a block may have a warp or two more)
constexpr int kSms = 152;
constexpr int kMaxSplits = 64;

struct StepWork {
    int64_t* offsets;   // [N + 1]: number of the first tile of each sequence, and of all
    float2* slot_stat;  // [ctas][2][rows]: running maximum (log2 units) and sum
    float* slot_sum;    // [ctas][2][rows][D]
    float2* row_stat;   // [T][Hq]: rows that are whole but for the prefix
    float* row_sum;     // [T][Hq][D]
    float2* far_stat;   // [splits][T][Hq]: the prefix
    float* far_sum;     // [splits][T][Hq][D]
    int ctas, rows, splits;
};

struct Span {
    int rows;       // rows of one key head: tokens * group
    int row_tiles;
    int key_tiles;  // tiles of own keys
    int first;      // first of them, counted from position 0
    int64_t units;
};

__device__ __forceinline__ Span span_of(const AttnArgs& a, int rows_per_tile, int n) {
    const int64_t fresh = min((int64_t)a.cu[n + 1], a.T) - max(a.cu[n], 0);
    const int len = a.cache.lens[n];
    Span s{0, 0, 0, 0, 0};
    if (fresh <= 0 || len < 0) return s;
    // what lies behind the table's last page has no row
    const int64_t end = min(len + fresh, (int64_t)a.cache.max_pages << a.cache.page_bits);
    s.rows = (int)min(fresh * a.group, (int64_t)0x7fffffff);
    s.row_tiles = (s.rows + rows_per_tile - 1) / rows_per_tile;
    s.first = a.cache.prefix_len / kKeyTile;
    if (end > a.cache.prefix_len) s.key_tiles = (int)((end + kKeyTile - 1) / kKeyTile) - s.first;
    s.units = (int64_t)s.row_tiles * s.key_tiles * a.Hkv;
    return s;
}

// The CTAs that take part: each at least `kLeast` tiles, as long as there are fewer than
// would give all of them that.
constexpr int kLeast = 1;
__device__ __forceinline__ int64_t taking_part(int64_t units, int ctas) {
    return max((int64_t)1, min((int64_t)ctas, (units + kLeast - 1) / kLeast));
}

struct Plan {
    int64_t from, to;  // this CTA's tiles
    int64_t offset;    // number of the first tile of sequence n
    int n;             // the sequence of its first tile
};

// Formed by kStepThreads threads: thread i sums the tiles of a run of sequences.
// CTA 0 leaves the sequences' numbers for the merge.  Every thread of the block calls it.
__device__ __forceinline__ Plan make_plan(const AttnArgs& a, const StepWork& w, int cta) {
    __shared__ int64_t warp_units[kStepThreads / 32 + 2];
    __shared__ Plan plan;
    const int tid = threadIdx.x, per = (a.N + kStepThreads - 1) / kStepThreads;
    const int lo = min(tid * per, a.N), hi = min(lo + per, a.N);
    int64_t mine = 0;
    for (int n = lo; n < hi; ++n) mine += span_of(a, w.rows, n).units;
    int64_t upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
        const int64_t left = __shfl_up_sync(0xffffffffu, upto, off);
        if ((tid & 31) >= off) upto += left;
    }
    if ((tid & 31) == 31) warp_units[tid >> 5] = upto;
    __syncthreads();
    int64_t all = 0, before = upto - mine;
#pragma unroll
    for (int i = 0; i < kStepThreads / 32; ++i) {
        if (i < (tid >> 5)) before += warp_units[i];
        all += warp_units[i];
    }
    const int64_t ctas = taking_part(all, w.ctas);
    const int64_t from = cta < ctas ? all * cta / ctas : all, to = cta < ctas ? all * (cta + 1) / ctas : all;
    if (tid == 0) plan = Plan{from, to, 0, 0};
    __syncthreads();
    int64_t at = before;
    if (cta == 0 || (from >= before && from < before + mine))
        for (int n = lo; n < hi; ++n) {
            const int64_t units = span_of(a, w.rows, n).units;
            if (from >= at && from < at + units) {
                plan.offset = at;
                plan.n = n;
            }
            if (cta == 0) w.offsets[n] = at;
            at += units;
        }
    if (cta == 0 && tid == 0) w.offsets[a.N] = all;
    __syncthreads();
    return plan;
}

// cta_of: the CTA whose run holds tile u.
__device__ __forceinline__ int64_t cta_of(int64_t u, int64_t all, int64_t ctas) { return ((u + 1) * ctas - 1) / all; }

// Calls job(n, span, key head, row tile, first key tile, last key tile + 1, slot) for every
// run of key tiles of one row tile in the plan, until it says false: slot -1 where it is whole.
template <typename F>
__device__ __forceinline__ void walk(const AttnArgs& a, const StepWork& w, const Plan& plan, F job) {
    int64_t u = plan.from, offset = plan.offset;
    int n = plan.n;
    while (u < plan.to && n < a.N) {
        const Span s = span_of(a, w.rows, n);
        while (u < plan.to && u < offset + s.units) {
            const int64_t local = u - offset, tile = local / s.key_tiles;
            const int begin = (int)(local - tile * s.key_tiles);
            const int end = (int)min((int64_t)s.key_tiles, begin + (plan.to - u));
            const int slot = begin == 0 && end == s.key_tiles ? -1 : begin > 0 ? 0 : 1;
            if (!job(n, s, (int)(tile / s.row_tiles), (int)(tile % s.row_tiles), s.first + begin, s.first + end, slot))
                return;
            u += end - begin;
        }
        offset += s.units;
        ++n;
    }
}

}  // namespace gdr
