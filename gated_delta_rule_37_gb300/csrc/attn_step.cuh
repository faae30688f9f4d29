// How gdr_attn_step cuts its work, shared by its kernels.
//
// The keys of a step are the prefix's, which every row of the batch sees, and each
// sequence's own.  The prefix is one tall problem (all tokens' rows of a key head
// against the same keys), cut along the keys so that it fills the GPU: on the tensor
// cores its (block of rows, key head, key tile) are numbered and shared out like the own
// parts' tiles below, elsewhere every block is cut into `splits`.
// The own parts are as many problems as there are sequences and key heads, of lengths
// that only the device knows: their key tiles are numbered (sequence, key head, row
// tile, key tile) and every CTA takes an equal run of the numbers, so that ragged
// batches are as balanced as even ones and one long sequence fills the GPU as well as
// many short ones.  A row tile's first tile follows kStart numbers without one: what its
// beginning and end cost, in tiles.  A row tile that lies within one CTA's run is finished
// there; one that is cut leaves a partial result (unnormalised sums, running maximum and
// sum) in each CTA's slots, of which a CTA needs two, for its first and its last row tile.
// The merge joins the partial results of a row in the order of its keys: no atomics, and
// the bits do not depend on which CTA ran first.
#pragma once

#include "attn.h"
#include "common.cuh"

namespace gdr {

constexpr int kKeyTile = 64;       // keys per tile of the own parts
constexpr int kFarTile = 128;      // keys per tile of the prefix, on the tensor cores
constexpr int kStepThreads = 256;  // threads that form the plan (a block may have a warp or two more)
constexpr int kSms = 152;          // GB300's: the workspace's size, which the host alone tells, follows it
constexpr int kMaxSplits = 64;

// A row tile that begins in a CTA's run and ends in another's: rows rows from r0 on of the
// sequence that begins at token t0, in the last slot of this CTA and the first of the
// parts - 1 next ones.  rows 0: there is none.
struct Cut {
    int t0, h, r0, rows, parts;
};

struct StepWork {
    int64_t* offsets;   // [N + 1]: first number of each sequence, and of all (with a prefix)
    Cut* cuts;          // [ctas] (without)
    float2* slot_stat;  // [ctas][2][rows]: running maximum (log2 units) and sum
    float* slot_sum;    // [ctas][2][rows][D]
    float2* row_stat;   // [T][Hq]: rows that are whole but for the prefix
    float* row_sum;     // [T][Hq][D]
    float2* far_stat;   // [splits][T][Hq]: the prefix
    float* far_sum;     // [splits][T][Hq][D]
    int ctas, rows;
    int splits;               // partial results of a row of the prefix, at most
    int far_ctas, far_tokens; // of the tensor cores' kernel, and tokens of a block (far_ctas 0: another kernel)
};

// (Measured, decode of 230 ragged sequences of up to 1024 own keys behind a prefix of 16000,
// all three kernels: 0: 175 us, 1: 166, 2: 158, 4: 152, 6: 154; longer or fewer sequences and
// 64 rows do not tell them apart.)
constexpr int kStart = 4;

struct Span {
    int rows;       // rows of one key head: tokens * group
    int row_tiles;
    int key_tiles;  // tiles of own keys
    int first;      // first of them, counted from position 0
    int t0;         // first token
    int len;        // tokens in the cache before the call's
    int end;        // end of the positions that have a place in the table
    int64_t units;
};

// Of cu[n], cu[n + 1] and lens[n].
__device__ __forceinline__ Span span_of(const AttnArgs& a, int rows_per_tile, int begin, int stop, int len) {
    Span s{0, 0, 0, 0, 0, 0, 0, 0};
    s.t0 = max(begin, 0);
    const int fresh = (int)min((int64_t)stop, a.T) - s.t0;
    if (fresh <= 0 || len < 0) return s;
    s.len = len;
    // what lies behind the table's last page has no row
    s.end = (int)min((int64_t)len + fresh, (int64_t)a.cache.max_pages << a.cache.page_bits);
    s.rows = fresh * a.group;
    s.row_tiles = (s.rows + rows_per_tile - 1) / rows_per_tile;
    s.first = a.cache.prefix_len / kKeyTile;
    if (s.end > a.cache.prefix_len) s.key_tiles = (s.end + kKeyTile - 1) / kKeyTile - s.first;
    if (s.key_tiles > 0) s.units = (int64_t)s.row_tiles * (s.key_tiles + kStart) * a.Hkv;
    return s;
}
__device__ __forceinline__ Span span_of(const AttnArgs& a, int rows_per_tile, int n) {
    return span_of(a, rows_per_tile, a.cu[n], a.cu[n + 1], a.cache.lens[n]);
}

// The CTAs that take part, if there is less work than CTAs.
__device__ __forceinline__ int64_t taking_part(int64_t units, int ctas) {
    return max((int64_t)1, min((int64_t)ctas, units));
}

struct Plan {
    int64_t from, to;  // this CTA's numbers
    int64_t offset;    // first number of sequence n
    int64_t all, ctas; // numbers, and CTAs that share them
    int n;             // the sequence of its first number
};

// Formed by kStepThreads threads: thread i sums the numbers of a run of sequences.
// CTA 0 leaves the sequences' first ones for a merge with a prefix, which goes over all
// rows; without, the CTAs leave the row tiles that are cut.  Every thread of the block calls it.
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
    if (tid == 0) {
        plan = Plan{from, to, 0, all, ctas, 0};
        w.cuts[cta].rows = 0;
    }
    __syncthreads();
    int64_t at = before;
    const bool leave = cta == 0 && w.splits > 0;
    if (leave || (from >= before && from < before + mine))
        for (int n = lo; n < hi; ++n) {
            const int64_t units = span_of(a, w.rows, n).units;
            if (from >= at && from < at + units) {
                plan.offset = at;
                plan.n = n;
            }
            if (leave) w.offsets[n] = at;
            at += units;
        }
    if (leave && tid == 0) w.offsets[a.N] = all;
    __syncthreads();
    return plan;
}

// The CTA whose run holds number u.
__device__ __forceinline__ int64_t cta_of(int64_t u, int64_t all, int64_t ctas) { return ((u + 1) * ctas - 1) / all; }

// One run of key tiles of one row tile.
struct Run {
    Span s;
    int n, h, row_tile;
    int from, to;  // key tiles, counted from position 0
    int slot;      // -1: the row tile is whole; else where its partial result goes
    int64_t last;  // number of the row tile's last key tile
};

// The partial results that a row of `token` has of the prefix.
__device__ __forceinline__ int far_parts(const AttnArgs& a, const StepWork& w, int64_t token, int h) {
    if (w.far_ctas == 0) return w.splits;
    const int64_t tiles = (a.cache.prefix_len + kFarTile - 1) / kFarTile, blocks = (a.T + w.far_tokens - 1) / w.far_tokens;
    const int64_t all = blocks * a.Hkv * tiles, u = (token / w.far_tokens * a.Hkv + h) * tiles;
    return (int)(cta_of(u + tiles - 1, all, w.far_ctas) - cta_of(u, all, w.far_ctas)) + 1;
}

// A run that goes on in other CTAs, for the merge; by one thread.
__device__ __forceinline__ void leave_cut(const StepWork& w, const Plan& plan, int cta, const Run& r) {
    if (r.slot != 1) return;
    const int r0 = r.row_tile * w.rows;
    w.cuts[cta] = Cut{r.s.t0, r.h, r0, min(w.rows, r.s.rows - r0), (int)(cta_of(r.last, plan.all, plan.ctas) - cta) + 1};
}

// The runs of a plan one after the other.  The next sequence's numbers are asked for before
// they are needed.
class Runs {
  public:
    __device__ __forceinline__ Runs(const AttnArgs& args, const StepWork& w, const Plan& plan)
        : a(args), rows(w.rows), u(plan.from), stop(plan.to), n(plan.n), h(0), row_tile(0), begin(0) {
        if (u >= stop) return;
        s = span_of(a, rows, n);
        ask();
        const int64_t local = u - plan.offset, tile = local / (s.key_tiles + kStart);
        begin = (int)(local - tile * (s.key_tiles + kStart));
        h = (int)(tile / s.row_tiles);
        row_tile = (int)(tile - (int64_t)h * s.row_tiles);
    }
    __device__ __forceinline__ bool next(Run& r) {
        while (u < stop) {
            while (h == a.Hkv || s.units == 0) {
                if (++n >= a.N) return false;
                s = span_of(a, rows, c0, c1, len);
                ask();
                h = 0;
            }
            const int end = (int)min((int64_t)s.key_tiles + kStart, begin + (stop - u));
            const int from = max(begin - kStart, 0), to = max(end - kStart, 0);
            r.s = s;
            r.n = n;
            r.h = h;
            r.row_tile = row_tile;
            r.from = s.first + from;
            r.to = s.first + to;
            r.slot = from == 0 && to == s.key_tiles ? -1 : from > 0 ? 0 : 1;
            r.last = u - begin + s.key_tiles + kStart - 1;
            u += end - begin;
            begin = 0;
            if (++row_tile == s.row_tiles) {
                row_tile = 0;
                ++h;
            }
            if (to > from) return true;
        }
        return false;
    }

  private:
    __device__ __forceinline__ void ask() {
        if (n + 1 >= a.N) return;
        c0 = a.cu[n + 1];
        c1 = a.cu[n + 2];
        len = a.cache.lens[n + 1];
    }
    const AttnArgs& a;
    int rows;
    int64_t u, stop;
    Span s;
    int n, h, row_tile, begin;
    int c0, c1, len;  // of sequence n + 1
};

}  // namespace gdr
