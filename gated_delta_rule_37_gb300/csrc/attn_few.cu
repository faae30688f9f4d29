// The step over the paged cache in fp32 for few rows (up to 8 on a key head: decode): the
// sequences' own keys (contract in include/gdr.h, the cut of the work in attn_step.cuh).
//
// Every key and value is read once and multiplied with 4 or 8 rows: a few operations a
// byte, which the CUDA cores do at the memory's pace as long as nothing goes through
// shared memory, where each row would read the keys again.  So 16 lanes take a key, D / 16
// of its channels each, straight from memory; the rows' queries and sums stay in
// registers, and a score is the lanes' sum by four shuffles.  A warp has 8 consecutive keys
// of a tile, which lie in one page, and a running maximum and sum of its own; the eight
// warps' results are joined at the end of a run.
//   Measured (against the tiles of 16 rows through shared memory): 64 sequences of up to 4096
// keys, 8 heads of 128 with 4 rows each, 174 us (409; 0.92 GB: 5.3 TB/s), 16 heads of 64 with
// one row 176 us (487); 256 of up to 300, 2 heads with 7 rows, 46 us (61).  What bounds it is the
// rows under way: a warp waits for its 4 or 8 keys before it asks for the next.
#include <math.h>

#include "attn.h"
#include "attn_step.cuh"
#include "common.cuh"
#include "gdr.h"
#include "launch.h"
#include "tc.cuh"

namespace gdr {
namespace {

constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32;
constexpr int kWarpKeys = kKeyTile / kFewWarps;  // of a tile

__device__ __forceinline__ void prefetch_line(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" :: "l"(p));
}

template <int D, int ROWS>
__global__ void __launch_bounds__(kFewThreads, ROWS == 4 ? 2 : 1) step_few_kernel(const AttnArgs a, const StepWork w) {
    constexpr int CH = D / 16, NV = CH / 4;            // channels of a lane, in pieces of 4
    constexpr int PAIRS = ROWS == 4 ? 2 : 4;           // pairs of keys whose rows are under way
    __shared__ __align__(16) float join[kFewWarps][ROWS][D];
    __shared__ float2 stats[kFewWarps][ROWS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = lane & 15, second = lane >> 4;
    tc::grid_dep_launch();
    const Plan plan = make_plan(a, w, blockIdx.x);
    Runs runs(a, w, plan);
    for (Run run; runs.next(run);) {
        if (tid == 0) leave_cut(w, plan, blockIdx.x, run);
        const int r0 = run.row_tile * ROWS, rows = min(ROWS, run.s.rows - r0), h = run.h;
        const int32_t* pages = a.cache.table + run.n * a.cache.table_ld;
        const int least = a.cache.prefix_len;
        auto sees = [&](int r) {
            return (int)min((int64_t)run.s.len + (r0 + min(r, rows - 1)) / a.group + 1, (int64_t)run.s.end);
        };
        const int most = sees(ROWS - 1), all_see = sees(0);
        float q[ROWS][CH], acc[ROWS][CH], m[ROWS], l[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int row = r0 + min(r, rows - 1), token = row / a.group, head = h * a.group + row - token * a.group;
            const float* from = static_cast<const float*>(a.q) + (int64_t)(run.s.t0 + token) * a.ldq + (int64_t)head * D;
#pragma unroll
            for (int v = 0; v < NV; ++v) Vec<float, 4>::load(from + v * 64 + sub * 4, q[r] + v * 4);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                q[r][c] *= a.scale_log2;
                acc[r][c] = 0.f;
            }
            m[r] = -INFINITY;
            l[r] = 0.f;
        }
        auto page_of = [&](int k) {
            const int64_t j = (int64_t)k * kKeyTile + warp * kWarpKeys;
            return k < run.to && j < most ? pages[j >> a.cache.page_bits] : -1;
        };
        auto row_of = [&](int page, int j) {
            return (((int64_t)page * a.Hkv + h) << a.cache.page_bits) + (j & (a.cache.page_size - 1));
        };
        // With 4 rows the next tile's rows go to L2 while this one's are worked on (64 sequences of up
        // to 4096 keys, 8 heads of 128: 174 / 212 us); with 8 registers are short (256 of up to 300: 62 / 46).
        constexpr bool FETCH = ROWS == 4;
        int ahead = page_of(run.from), next = FETCH ? page_of(run.from + 1) : 0;
        for (int k = run.from; k < run.to; ++k) {
            const int page = ahead, j0 = k * kKeyTile + warp * kWarpKeys;
            if (FETCH) {
                ahead = next;
                next = page_of(k + 2);
                if (ahead >= 0 && ahead < a.cache.num_pages) {
                    constexpr int LINES = kWarpKeys * D / 32;  // of 128 bytes: a warp's keys are dense
                    const int64_t at = row_of(ahead, j0 + kKeyTile) * D;
#pragma unroll
                    for (int i = lane; i < 2 * LINES; i += 32)
                        prefetch_line(static_cast<const float*>(i < LINES ? a.cache.k : a.cache.v) + at + i % LINES * 32);
                }
            } else {
                ahead = page_of(k + 1);
            }
            if (page < 0 || page >= a.cache.num_pages || j0 >= most || j0 + kWarpKeys <= least) continue;
            const int64_t row = row_of(page, j0);
            const float* kp = static_cast<const float*>(a.cache.k) + (row + second) * D + sub * 4;
            const float* vp = static_cast<const float*>(a.cache.v) + (row + second) * D + sub * 4;
            const bool edge = j0 < least || j0 + kWarpKeys > all_see;
#pragma unroll
            for (int g = 0; g < kWarpKeys / 2; g += PAIRS) {
                float x[PAIRS][CH], y[PAIRS][CH], s[ROWS][PAIRS];
#pragma unroll
                for (int i = 0; i < PAIRS; ++i)
#pragma unroll
                    for (int v = 0; v < NV; ++v) Vec<float, 4>::load(kp + (int64_t)(g + i) * 2 * D + v * 64, x[i] + v * 4);
#pragma unroll
                for (int i = 0; i < PAIRS; ++i)
#pragma unroll
                    for (int v = 0; v < NV; ++v) Vec<float, 4>::load(vp + (int64_t)(g + i) * 2 * D + v * 64, y[i] + v * 4);
#pragma unroll
                for (int r = 0; r < ROWS; ++r)
#pragma unroll
                    for (int i = 0; i < PAIRS; ++i) {
                        float2 d = make_float2(0.f, 0.f);
#pragma unroll
                        for (int c = 0; c < CH; c += 2)
                            d = __ffma2_rn(make_float2(q[r][c], q[r][c + 1]), make_float2(x[i][c], x[i][c + 1]), d);
                        s[r][i] = d.x + d.y;
                    }
#pragma unroll
                for (int off = 8; off; off /= 2)
#pragma unroll
                    for (int r = 0; r < ROWS; ++r)
#pragma unroll
                        for (int i = 0; i < PAIRS; ++i) s[r][i] += __shfl_xor_sync(0xffffffffu, s[r][i], off);
                if (edge) {
                    // what a row does not see; what none does may hold anything
#pragma unroll
                    for (int i = 0; i < PAIRS; ++i) {
                        const int j = j0 + (g + i) * 2 + second;
#pragma unroll
                        for (int r = 0; r < ROWS; ++r)
                            if (j < least || j >= sees(r)) s[r][i] = -INFINITY;
                    }
                }
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    float top = s[r][0];
#pragma unroll
                    for (int i = 1; i < PAIRS; ++i) top = fmaxf(top, s[r][i]);
                    top = fmaxf(m[r], fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16)));
                    const float base = top == -INFINITY ? 0.f : top, back = exp2f(m[r] - base);
                    m[r] = top;
                    l[r] *= back;
#pragma unroll
                    for (int c = 0; c < CH; ++c) acc[r][c] *= back;
#pragma unroll
                    for (int i = 0; i < PAIRS; ++i) {
                        const float p = exp2f(s[r][i] - base);
                        l[r] += p;
                        // a weight of 0 at the edge is of a key that the row does not see
                        if (edge && p == 0.f) continue;
#pragma unroll
                        for (int c = 0; c < CH; c += 2) {
                            const float2 z = __ffma2_rn(make_float2(p, p), make_float2(y[i][c], y[i][c + 1]),
                                                        make_float2(acc[r][c], acc[r][c + 1]));
                            acc[r][c] = z.x;
                            acc[r][c + 1] = z.y;
                        }
                    }
                }
            }
        }

        // ---- the warps' results joined ----
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 16);
#pragma unroll
            for (int c = 0; c < CH; ++c) acc[r][c] += __shfl_xor_sync(0xffffffffu, acc[r][c], 16);
            if (second == 0)
#pragma unroll
                for (int v = 0; v < NV; ++v) Vec<float, 4>::store(&join[warp][r][v * 64 + sub * 4], acc[r] + v * 4);
            if (lane == 0) stats[warp][r] = make_float2(m[r], l[r]);
        }
        __syncthreads();
        for (int i = tid; i < rows * (D / 4); i += kFewThreads) {
            const int r = i / (D / 4), col = i % (D / 4) * 4;
            float top = -INFINITY;
#pragma unroll
            for (int x = 0; x < kFewWarps; ++x) top = fmaxf(top, stats[x][r].x);
            const float base = top == -INFINITY ? 0.f : top;
            float sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int n = 0; n < kFewWarps; ++n) {
                const float2 st = stats[n][r];
                if (st.x == -INFINITY && st.y == 0.f) continue;  // no key, or scores of -inf alone: no weight
                const float f = exp2f(st.x - base);
                const float4 y = *reinterpret_cast<const float4*>(&join[n][r][col]);
                sum = fmaf(st.y, f, sum);
                x[0] = fmaf(y.x, f, x[0]);
                x[1] = fmaf(y.y, f, x[1]);
                x[2] = fmaf(y.z, f, x[2]);
                x[3] = fmaf(y.w, f, x[3]);
            }
            const int local = (r0 + r) / a.group, head = h * a.group + r0 + r - local * a.group;
            const int64_t token = run.s.t0 + local;
            if (run.slot < 0 && w.splits == 0) {
                const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] *= inv;
                Vec<float, 4>::store(static_cast<float*>(a.o) + token * a.ldo + (int64_t)head * D + col, x);
            } else {
                const int64_t at = run.slot < 0 ? token * a.Hq + head : ((int64_t)blockIdx.x * 2 + run.slot) * ROWS + r;
                Vec<float, 4>::store((run.slot < 0 ? w.row_sum : w.slot_sum) + at * D + col, x);
                if (col == 0) (run.slot < 0 ? w.row_stat : w.slot_stat)[at] = make_float2(top, sum);
            }
        }
        __syncthreads();
    }
}

template <int D, int ROWS>
cudaError_t launch_rows(const AttnArgs& a, const StepWork& w, cudaStream_t s) {
    KernelTimer kt("attn_step_few", s);
    step_few_kernel<D, ROWS><<<w.ctas, kFewThreads, 0, s>>>(a, w);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_step_few(const AttnArgs& a, const StepWork& w, cudaStream_t s) {
    if (a.D == 128) return w.rows == 4 ? launch_rows<128, 4>(a, w, s) : launch_rows<128, 8>(a, w, s);
    return w.rows == 4 ? launch_rows<64, 4>(a, w, s) : launch_rows<64, 8>(a, w, s);
}

}  // namespace gdr
