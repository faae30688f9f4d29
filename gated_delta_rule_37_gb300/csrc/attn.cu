// Attention in fp32 on the CUDA cores (packed prompts, the step over the paged
// cache), the merge of the step's partial results, and the layer's entry points
// (contract in include/gdr.h).
//
// One pass over the keys with the running maximum m and sum l of a row's softmax, in
// log2 units: with s_j = scale log2(e) q . k_j and m' = max(m, max_j s_j),
//   l <- l 2^(m - m') + sum_j 2^(s_j - m'),   acc <- acc 2^(m - m') + sum_j 2^(s_j - m') v_j,
// o = acc / l.  Two partial results join by the same rule.
//   On the CUDA cores the products bound it: a tile of 128 rows by 64 keys reads 12 pieces of
// 16 bytes from shared memory for 128 multiply-adds of a thread, copies run beside them.  Measured:
// 4000 tokens of 32 heads of 128 on 8 3.2 ms, 41 of 74 TFLOP/s.
#include <math.h>

#include "attn.h"
#include "attn_step.cuh"
#include "common.cuh"
#include "gdr.h"
#include "launch.h"
#include "tc.cuh"

namespace gdr {
namespace {

using tc::grid_dep_wait;

constexpr float kNone = -INFINITY;

// ---- rows by keys on the CUDA cores ------------------------------------------------

// RT rows by 64 keys, 256 threads as TR x TK: thread (tr, tk) has the rows tr + TR i, the
// keys tk + TK j of the scores and D / TK channels of the sums.  TK threads of one warp
// share a row, so that its maximum and sum are shuffles.
template <typename T, int D, int RT> struct Simt {
    static constexpr int TK = RT >= 64 ? 16 : 32, TR = 256 / TK, RR = RT / TR, KK = kKeyTile / TK;
    static constexpr int CV = D / TK < 4 ? D / TK : 4, CG = D / TK / CV;
    static constexpr int LDQ = D + 4, LDP = kKeyTile + 4;  // rows of the products on different banks
    struct Smem {
        float q[RT][LDQ], k[kKeyTile][LDQ], v[kKeyTile][D], p[RT][LDP];
        int64_t limit[RT];
        int there[2][kKeyTile];  // of this tile and the next
    };

    float m[RR], l[RR], acc[RR][CG * CV];

    // rows(r): the address of row r's query, nullptr where there is none; limit(r): the
    // end of the keys that it sees
    template <typename R, typename L>
    __device__ void start(Smem& s, R rows, L limit, float scale) {
        __syncthreads();
        constexpr int C = D / 4;
        for (int i = threadIdx.x; i < RT * C; i += 256) {
            const T* from = rows(i / C);
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            if (from) Vec<T, 4>::load(from + i % C * 4, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) s.q[i / C][i % C * 4 + e] = x[e] * scale;
        }
        for (int r = threadIdx.x; r < RT; r += 256) s.limit[r] = limit(r);
#pragma unroll
        for (int i = 0; i < RR; ++i) {
            m[i] = kNone;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < CG * CV; ++c) acc[i][c] = 0.f;
        }
    }

    // Rows of keys or values from position j0 on to shared memory, zeros where there are none;
    // fp32 by asynchronous copies.  keys(j, kp, vp) gives a key's rows, false where it has none.
    template <bool VALUES, int LD, typename K>
    __device__ void load(float (&to)[kKeyTile][LD], int* there, int64_t j0, int64_t least, int64_t most, K keys) {
        constexpr int C = D / 4;
#pragma unroll 4
        for (int i = threadIdx.x; i < kKeyTile * C; i += 256) {
            const int64_t j = j0 + i / C;
            const T *kp = nullptr, *vp = nullptr;
            const bool has = j >= least && j < most && keys(j, kp, vp);
            if (!VALUES && i % C == 0) there[i / C] = has;
            float* row = &to[i / C][i % C * 4];
            const T* from = (VALUES ? vp : kp) + i % C * 4;
            if (sizeof(T) == 4) {
                const uint32_t dst = (uint32_t)__cvta_generic_to_shared(row), bytes = has ? 16 : 0;
                const void* src = has ? static_cast<const void*>(from) : a_row;  // read only if there are bytes
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
            } else {
                float x[4] = {0.f, 0.f, 0.f, 0.f};
                if (has) Vec<T, 4>::load(from, x);
                Vec<float, 4>::store(row, x);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // All of this thread's copies but the last set.
    __device__ static void landed() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

    const void* a_row;  // an address that may be given where nothing is read

    // The tiles of keys from position j0 to j1, those below `least` and from `most` on left out.
    // A tile's values arrive while its scores are formed, the next one's keys during the
    // product with the values.
    template <typename K>
    __device__ void tiles(Smem& s, int64_t j0, int64_t j1, int64_t least, int64_t most, K keys) {
        if (j0 >= j1) return;
        __syncthreads();
        load<false>(s.k, s.there[0], j0, least, most, keys);
        for (int b = 0; j0 < j1; j0 += kKeyTile, b ^= 1) {
            load<true>(s.v, nullptr, j0, least, most, keys);
            landed();
            __syncthreads();
            const int tk = threadIdx.x % TK, tr = threadIdx.x / TK;
            // a key that a row does not see may be an infinity, which a weight of 0 does not
            // keep out: where the tile has such pairs each is asked for
            const bool masked = __syncthreads_or(scores(s, s.there[b], j0, tr, tk));
            if (j0 + kKeyTile < j1) load<false>(s.k, s.there[b ^ 1], j0 + kKeyTile, least, most, keys);
            else asm volatile("cp.async.commit_group;" ::: "memory");
            landed();
            __syncthreads();
            if (!masked) product<false>(s, j0, tr, tk);
            else product<true>(s, j0, tr, tk);
            __syncthreads();
        }
    }

    // One tile's scores and weights; whether a row does not see one of its keys.
    __device__ bool scores(Smem& s, const int* there, int64_t j0, int tr, int tk) {
        // even and odd channels apart: two fused multiply-adds an instruction
        float2 part[RR][KK];
#pragma unroll
        for (int i = 0; i < RR; ++i)
#pragma unroll
            for (int j = 0; j < KK; ++j) part[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            float4 qf[RR], kf[KK];
#pragma unroll
            for (int i = 0; i < RR; ++i) qf[i] = *reinterpret_cast<const float4*>(&s.q[tr + TR * i][d]);
#pragma unroll
            for (int j = 0; j < KK; ++j) kf[j] = *reinterpret_cast<const float4*>(&s.k[tk + TK * j][d]);
#pragma unroll
            for (int i = 0; i < RR; ++i)
#pragma unroll
                for (int j = 0; j < KK; ++j)
                    part[i][j] = __ffma2_rn(make_float2(qf[i].x, qf[i].y), make_float2(kf[j].x, kf[j].y),
                                            __ffma2_rn(make_float2(qf[i].z, qf[i].w), make_float2(kf[j].z, kf[j].w),
                                                       part[i][j]));
        }
        float sc[RR][KK];
#pragma unroll
        for (int i = 0; i < RR; ++i)
#pragma unroll
            for (int j = 0; j < KK; ++j) sc[i][j] = part[i][j].x + part[i][j].y;
        bool masked = false;
#pragma unroll
        for (int i = 0; i < RR; ++i) {
            const int64_t end = s.limit[tr + TR * i];
            float top = m[i];
#pragma unroll
            for (int j = 0; j < KK; ++j) {
                const int k = tk + TK * j;
                if (!there[k] || j0 + k >= end) {
                    sc[i][j] = kNone;
                    masked = true;
                }
                top = fmaxf(top, sc[i][j]);
            }
#pragma unroll
            for (int off = TK / 2; off; off /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float base = top == kNone ? 0.f : top, back = exp2f(m[i] - base);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < KK; ++j) {
                const float e = exp2f(sc[i][j] - base);
                s.p[tr + TR * i][tk + TK * j] = e;
                sum += e;
            }
#pragma unroll
            for (int off = TK / 2; off; off /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            m[i] = top;
            l[i] = l[i] * back + sum;
#pragma unroll
            for (int c = 0; c < CG * CV; ++c) acc[i][c] *= back;
        }
        return masked;
    }

    template <bool MASKED>
    __device__ void product(Smem& s, int64_t j0, int tr, int tk) {
        int64_t end[RR];
#pragma unroll
        for (int i = 0; i < RR; ++i) end[i] = MASKED ? s.limit[tr + TR * i] - j0 : 0;
#pragma unroll 2
        for (int k = 0; k < kKeyTile; k += 4) {
            float4 pf[RR];
#pragma unroll
            for (int i = 0; i < RR; ++i) pf[i] = *reinterpret_cast<const float4*>(&s.p[tr + TR * i][k]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v[CG * CV];
#pragma unroll
                for (int g = 0; g < CG; ++g) Vec<float, CV>::load(&s.v[k + e][(tk + TK * g) * CV], v + g * CV);
#pragma unroll
                for (int i = 0; i < RR; ++i) {
                    const float p = e == 0 ? pf[i].x : e == 1 ? pf[i].y : e == 2 ? pf[i].z : pf[i].w;
                    if (MASKED && k + e >= end[i]) continue;
#pragma unroll
                    for (int c = 0; c < CG * CV; c += 2) {
                        const float2 a = __ffma2_rn(make_float2(p, p), make_float2(v[c], v[c + 1]),
                                                    make_float2(acc[i][c], acc[i][c + 1]));
                        acc[i][c] = a.x;
                        acc[i][c + 1] = a.y;
                    }
                }
            }
        }
    }

    // out(r): where row r's result goes, nullptr where it is not wanted; o = acc / l
    template <typename O>
    __device__ void finish(O out) {
        const int tk = threadIdx.x % TK, tr = threadIdx.x / TK;
#pragma unroll
        for (int i = 0; i < RR; ++i) {
            T* to = out(tr + TR * i);
            if (!to) continue;
            const float inv = l[i] > 0.f ? 1.f / l[i] : l[i];  // a NaN stays one
            // (scores of -inf alone weigh nothing, whatever the values)
#pragma unroll
            for (int c = 0; c < CG * CV; ++c) acc[i][c] = l[i] == 0.f ? 0.f : acc[i][c] * inv;
#pragma unroll
            for (int g = 0; g < CG; ++g) Vec<T, CV>::store(to + (tk + TK * g) * CV, acc[i] + g * CV);
        }
    }

    // sum(r) and stat(r): where row r's partial result goes
    template <typename S, typename P>
    __device__ void leave(S sum, P stat) {
        const int tk = threadIdx.x % TK, tr = threadIdx.x / TK;
#pragma unroll
        for (int i = 0; i < RR; ++i) {
            float* to = sum(tr + TR * i);
            if (!to) continue;
#pragma unroll
            for (int g = 0; g < CG; ++g) Vec<float, CV>::store(to + (tk + TK * g) * CV, acc[i] + g * CV);
            if (tk == 0) *stat(tr + TR * i) = make_float2(m[i], l[i]);
        }
    }
};

// Key j's rows in the caches, of key head h.
template <typename T, int D>
__device__ __forceinline__ bool cached(const Paged& c, const int32_t* pages, int Hkv, int h, int64_t j, const T*& kp,
                                       const T*& vp) {
    const int page = pages[j >> c.page_bits];
    if (page < 0 || page >= c.num_pages) return false;
    const int64_t row = (((int64_t)page * Hkv + h) << c.page_bits) + (j & (c.page_size - 1));
    kp = static_cast<const T*>(c.k) + row * D;
    vp = static_cast<const T*>(c.v) + row * D;
    return true;
}

template <typename T, int D, int RT>
__global__ void __launch_bounds__(256) prompt_simt_kernel(const AttnArgs a) {
    extern __shared__ float4 raw[];
    using E = Simt<T, D, RT>;
    typename E::Smem& s = *reinterpret_cast<typename E::Smem*>(raw);
    // blockIdx.x numbers the row tiles of all sequences, the last first: their rows see most keys
    __shared__ int at_n, at_tile;
    if (threadIdx.x == 0) at_n = -1;
    __syncthreads();
    if (threadIdx.x < 32) {
        int64_t left = gridDim.x - 1 - blockIdx.x;
        for (int base = 0; base < a.N && left >= 0; base += 32) {
            const int n = base + threadIdx.x;
            int64_t tiles = 0;
            if (n < a.N) {
                const int64_t rows = (min((int64_t)a.cu[n + 1], a.T) - max(a.cu[n], 0)) * a.group;
                tiles = rows > 0 ? (rows + RT - 1) / RT : 0;
            }
            int64_t upto = tiles;
#pragma unroll
            for (int off = 1; off < 32; off *= 2) {
                const int64_t l = __shfl_up_sync(0xffffffffu, upto, off);
                if ((int)threadIdx.x >= off) upto += l;
            }
            if (left < upto && left >= upto - tiles) {
                at_n = n;
                at_tile = (int)(left - (upto - tiles));
            }
            const int64_t all = __shfl_sync(0xffffffffu, upto, 31);
            left = left < all ? -1 : left - all;
        }
    }
    __syncthreads();
    if (at_n < 0) return;
    const int n = at_n, h = blockIdx.y;
    const int64_t t0 = max(a.cu[n], 0), L = min((int64_t)a.cu[n + 1], a.T) - t0;
    const int64_t r0 = (int64_t)at_tile * RT, rows = min((int64_t)RT, L * a.group - r0);
    auto element = [&](int64_t r, int64_t ld) { return (t0 + r / a.group) * ld + ((int64_t)h * a.group + r % a.group) * D; };
    E e;
    e.start(s, [&](int r) { return r < rows ? static_cast<const T*>(a.q) + element(r0 + r, a.ldq) : nullptr; },
            [&](int r) { return r < rows ? (r0 + r) / a.group + 1 : 0; }, a.scale_log2);
    const int64_t most = (r0 + rows - 1) / a.group + 1;
    e.a_row = a.q;
    e.tiles(s, 0, most, 0, most, [&](int64_t i, const T*& kp, const T*& vp) {
        kp = static_cast<const T*>(a.k) + (t0 + i) * a.ldk + (int64_t)h * D;
        vp = static_cast<const T*>(a.v) + (t0 + i) * a.ldv + (int64_t)h * D;
        return true;
    });
    e.finish([&](int r) { return r < rows ? static_cast<T*>(a.o) + element(r0 + r, a.ldo) : nullptr; });
}

// The sequences' own keys.
template <typename T, int D, int RT>
__global__ void __launch_bounds__(256) step_simt_kernel(const AttnArgs a, const StepWork w) {
    extern __shared__ float4 raw[];
    using E = Simt<T, D, RT>;
    typename E::Smem& s = *reinterpret_cast<typename E::Smem*>(raw);
    const Plan plan = make_plan(a, w, blockIdx.x);
    Runs runs(a, w, plan);
    for (Run run; runs.next(run);) {
        if (threadIdx.x == 0) leave_cut(w, plan, blockIdx.x, run);
        const int64_t t0 = run.s.t0, len = run.s.len;
        const int r0 = run.row_tile * RT, rows = min(RT, run.s.rows - r0), h = run.h;
        const int64_t most = min(len + (r0 + rows - 1) / a.group + 1, (int64_t)run.s.end);
        const int32_t* pages = a.cache.table + run.n * a.cache.table_ld;
        auto row = [&](int r) { return (t0 + (r0 + r) / a.group) * a.Hq + h * a.group + (r0 + r) % a.group; };
        auto element = [&](int r, int64_t ld) {
            return (t0 + (r0 + r) / a.group) * ld + (int64_t)(h * a.group + (r0 + r) % a.group) * D;
        };
        E e;
        e.start(s, [&](int r) { return r < rows ? static_cast<const T*>(a.q) + element(r, a.ldq) : nullptr; },
                [&](int r) { return r < rows ? len + (r0 + r) / a.group + 1 : 0; }, a.scale_log2);
        e.a_row = a.q;
        e.tiles(s, (int64_t)run.from * kKeyTile, (int64_t)run.to * kKeyTile, a.cache.prefix_len, most,
                [&](int64_t j, const T*& kp, const T*& vp) { return cached<T, D>(a.cache, pages, a.Hkv, h, j, kp, vp); });
        if (run.slot >= 0) {
            const int64_t base = ((int64_t)blockIdx.x * 2 + run.slot) * w.rows;
            e.leave([&](int r) { return r < rows ? w.slot_sum + (base + r) * D : nullptr; },
                    [&](int r) { return w.slot_stat + base + r; });
        } else if (a.cache.prefix_len > 0) {
            e.leave([&](int r) { return r < rows ? w.row_sum + row(r) * D : nullptr; },
                    [&](int r) { return w.row_stat + row(r); });
        } else {
            e.finish([&](int r) { return r < rows ? static_cast<T*>(a.o) + element(r, a.ldo) : nullptr; });
        }
    }
}

// The prefix: blockIdx = (row tile of all tokens' rows, key head, split).
template <typename T, int D, int RT>
__global__ void __launch_bounds__(256) prefix_simt_kernel(const AttnArgs a, const StepWork w) {
    extern __shared__ float4 raw[];
    using E = Simt<T, D, RT>;
    typename E::Smem& s = *reinterpret_cast<typename E::Smem*>(raw);
    const int h = blockIdx.y, tiles = (a.cache.prefix_len + kKeyTile - 1) / kKeyTile;
    const int64_t r0 = (int64_t)blockIdx.x * RT, rows = min((int64_t)RT, a.T * a.group - r0);
    const int from = (int)((int64_t)tiles * blockIdx.z / w.splits), to = (int)((int64_t)tiles * (blockIdx.z + 1) / w.splits);
    auto row = [&](int r) {
        return ((int64_t)blockIdx.z * a.T + (r0 + r) / a.group) * a.Hq + h * a.group + (int)((r0 + r) % a.group);
    };
    E e;
    e.start(s, [&](int r) {
                return r < rows ? static_cast<const T*>(a.q) + (r0 + r) / a.group * a.ldq +
                                      (h * a.group + (r0 + r) % a.group) * D : nullptr;
            },
            [&](int r) -> int64_t {
                if (r >= rows) return 0;
                // the last sequence that starts at or before the token
                const int64_t t = (r0 + r) / a.group;
                int lo = 0, hi = a.N;
                while (hi > lo) {
                    const int mid = (lo + hi + 1) / 2;
                    if (a.cu[mid] <= t) lo = mid; else hi = mid - 1;
                }
                if (lo >= a.N || a.cu[lo] > t || t >= a.cu[lo + 1] || a.cache.lens[lo] < 0) return 0;
                return min((int64_t)a.cache.prefix_len, a.cache.lens[lo] + (t - a.cu[lo]) + 1);
            }, a.scale_log2);
    e.a_row = a.q;
    e.tiles(s, (int64_t)from * kKeyTile, (int64_t)to * kKeyTile, 0, a.cache.prefix_len,
            [&](int64_t j, const T*& kp, const T*& vp) {
                return cached<T, D>(a.cache, a.cache.prefix, a.Hkv, h, j, kp, vp);
            });
    e.leave([&](int r) { return r < rows ? w.far_sum + row(r) * D : nullptr; },
            [&](int r) { return w.far_stat + row(r); });
}

// ---- the merge ----------------------------------------------------------------------

constexpr int kMergeThreads = 128, kMergeWarps = kMergeThreads / 32;
constexpr int kBatch = 8;  // partial results that a warp has under way

// The partial results first, first + step, ... below count of one row, by a warp: adds them up
// relative to the maximum of all `count`.  stat_at(i), sum_at(i): where they are.
template <int C, typename S, typename P>
__device__ __forceinline__ void join_parts(int count, int first, int step, S stat_at, P sum_at, float (&acc)[C], float& l) {
    const int lane = threadIdx.x & 31;
    float top = kNone;
    for (int i = lane; i < count; i += 32) top = fmaxf(top, stat_at(i)->x);
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
    l = 0.f;
    float base = 0.f;
    for (int i0 = first; i0 < count; i0 += step * kBatch) {
        float2 st[kBatch];
        float x[kBatch][C];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int i = i0 + k * step;
            st[k] = make_float2(kNone, 0.f);
            if (i >= count) continue;
            st[k] = *stat_at(i);
            Vec<float, C>::load(sum_at(i) + lane * C, x[k]);
        }
        if (i0 == first) {  // with the first loads under way
#pragma unroll
            for (int off = 16; off; off /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            base = top == kNone ? 0.f : top;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (st[k].x == kNone && st[k].y == 0.f) continue;  // no key, or scores of -inf alone: no weight
            const float f = exp2f(st[k].x - base);
            l = fmaf(st[k].y, f, l);
#pragma unroll
            for (int c = 0; c < C; ++c) acc[c] = fmaf(x[k][c], f, acc[c]);
        }
    }
}

// Without a prefix: the row tiles that are cut, blockIdx = (CTA that has the first part, share
// of its rows); the block's warps share the parts of a row, of which one long sequence has many.
template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) step_merge_kernel(const AttnArgs a, const StepWork w) {
    constexpr int C = D / 32;
    __shared__ __align__(16) float sums[kMergeWarps][D];
    __shared__ float ls[kMergeWarps];
    grid_dep_wait();
    const Cut cut = w.cuts[blockIdx.x];
    const int cta = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = threadIdx.x * 2;
    for (int r = blockIdx.y; r < cut.rows; r += gridDim.y) {
        auto place = [&](int i) { return ((int64_t)(cta + i) * 2 + (i == 0)) * w.rows + r; };
        float acc[C], l;
        join_parts(cut.parts, warp, kMergeWarps, [&](int i) { return w.slot_stat + place(i); },
                   [&](int i) { return w.slot_sum + place(i) * D; }, acc, l);
        Vec<float, C>::store(&sums[warp][lane * C], acc);
        if (lane == 0) ls[warp] = l;
        __syncthreads();
        if (d < D) {
            float x[2] = {0.f, 0.f}, y = 0.f;
#pragma unroll
            for (int i = 0; i < kMergeWarps; ++i) {
                x[0] += sums[i][d];
                x[1] += sums[i][d + 1];
                y += ls[i];
            }
            const float inv = y > 0.f ? 1.f / y : y == 0.f ? 0.f : y;
            x[0] *= inv;
            x[1] *= inv;
            const int row = cut.r0 + r, local = row / a.group, head = cut.h * a.group + row - local * a.group;
            Vec<T, 2>::store(static_cast<T*>(a.o) + (int64_t)(cut.t0 + local) * a.ldo + (int64_t)head * D + d, x);
        }
        __syncthreads();
    }
}

// With a prefix, which every row has partial results of: blockIdx = (sequence, key head, share
// of its rows); a warp per row.
template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) step_merge_prefix_kernel(const AttnArgs a, const StepWork w) {
    constexpr int C = D / 32;
    const int n = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31;
    const Span s = span_of(a, w.rows, n);
    grid_dep_wait();
    const int64_t all = w.offsets[a.N], ctas = taking_part(all, w.ctas);
    const int64_t t0 = s.t0;
    for (int r = blockIdx.z * kMergeWarps + (threadIdx.x >> 5); r < s.rows; r += gridDim.z * kMergeWarps) {
        const int64_t row = (t0 + r / a.group) * a.Hq + h * a.group + r % a.group;
        int64_t first = 0;
        int near = 0;  // partial results of the own keys
        if (s.key_tiles > 0) {
            const int64_t u = w.offsets[n] + ((int64_t)h * s.row_tiles + r / w.rows) * (s.key_tiles + kStart) + kStart;
            first = cta_of(u, all, ctas);
            near = (int)(cta_of(u + s.key_tiles - 1, all, ctas) - first) + 1;
        }
        auto slot = [&](int c) { return ((first + c) * 2 + (c == 0)) * w.rows + r % w.rows; };
        float acc[C], l;
        const int far = far_parts(a, w, t0 + r / a.group, h);
        join_parts(far + near, 0, 1,
                   [&](int i) -> const float2* {
                       return i < far ? w.far_stat + i * a.T * a.Hq + row
                              : near == 1  ? w.row_stat + row
                                           : w.slot_stat + slot(i - far);
                   },
                   [&](int i) -> const float* {
                       return i < far ? w.far_sum + (i * a.T * a.Hq + row) * D
                              : near == 1  ? w.row_sum + row * D
                                           : w.slot_sum + slot(i - far) * D;
                   }, acc, l);
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] *= inv;
        Vec<T, C>::store(static_cast<T*>(a.o) + (t0 + r / a.group) * a.ldo +
                             (int64_t)(h * a.group + r % a.group) * D + lane * C, acc);
    }
}

// ---- launches -----------------------------------------------------------------------

// Tokens that a tensor map takes: none overlaps its neighbour.
bool tiled(int64_t ld, int heads, int D) { return ld >= (int64_t)heads * D; }

template <typename T, int D, int RT>
cudaError_t launch_prompt_rows(const AttnArgs& a, cudaStream_t s) {
    const size_t bytes = sizeof(typename Simt<T, D, RT>::Smem);
    static std::atomic<uint64_t> known{0};
    const cudaError_t e = allow_smem(prompt_simt_kernel<T, D, RT>, (int)bytes, known);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (a.T * a.group + RT - 1) / RT + a.N;
    KernelTimer kt("attn_prompt_simt", s);
    prompt_simt_kernel<T, D, RT><<<dim3((unsigned)tiles, a.Hkv), 256, bytes, s>>>(a);
    return cudaGetLastError();
}

// The largest tiles that leave no SM without one: 128 rows by heads of 128, 64, else 16.
// (Measured with fp32.  128 rows against 64: 32 heads of 128 on 8, 4000 tokens 3.5 / 4.5 ms, 16 on
// 2, 2000 tokens 461 / 519 us; heads of 64, of which 64 rows leave room for two CTAs, 2.0 / 1.9 ms.
// 16 rows against 64: 2 heads of 64, 128 tokens 9.9 / 16.2 us, 512 tokens 28 / 49; 8 heads of 128 on
// one key head, 1000 tokens 114 / 158; 16 of 128, 512 tokens, nearly a tile for each SM, 93 / 83;
// 32 of 128 on 8, 4000 tokens 6.8 / 4.8 ms.)
template <typename T, int D>
cudaError_t launch_prompt_simt(const AttnArgs& a, cudaStream_t s) {
    const auto tiles = [&](int rows) { return (a.T * a.group + rows - 1) / rows * a.Hkv; };
    if (D == 128 && tiles(128) >= kSms) return launch_prompt_rows<T, D, D == 128 ? 128 : 64>(a, s);
    return tiles(64) >= kSms ? launch_prompt_rows<T, D, 64>(a, s) : launch_prompt_rows<T, D, 16>(a, s);
}

template <typename T, int D, int RT>
cudaError_t launch_prefix_simt(const AttnArgs& a, const StepWork& w, cudaStream_t s) {
    const size_t bytes = sizeof(typename Simt<T, D, RT>::Smem);
    static std::atomic<uint64_t> known{0};
    const cudaError_t e = allow_smem(prefix_simt_kernel<T, D, RT>, (int)bytes, known);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (a.T * a.group + RT - 1) / RT;
    KernelTimer kt("attn_prefix_simt", s);
    prefix_simt_kernel<T, D, RT><<<dim3((unsigned)tiles, a.Hkv, w.splits), 256, bytes, s>>>(a, w);
    return cudaGetLastError();
}

template <int D, int RT>
cudaError_t launch_step_simt(const AttnArgs& a, const StepWork& w, cudaStream_t s) {
    const size_t bytes = sizeof(typename Simt<float, D, RT>::Smem);
    static std::atomic<uint64_t> known{0};
    const cudaError_t e = allow_smem(step_simt_kernel<float, D, RT>, (int)bytes, known);
    if (e != cudaSuccess) return e;
    KernelTimer kt("attn_step_simt", s);
    step_simt_kernel<float, D, RT><<<w.ctas, 256, bytes, s>>>(a, w);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_merge(const AttnArgs& a, const StepWork& w, cudaStream_t s) {
    KernelTimer kt("attn_step_merge", s);
    if (w.splits == 0)
        return launch_dependent(step_merge_kernel<T, D>, dim3(w.ctas, w.rows < 16 ? w.rows : 16), dim3(kMergeThreads), 0,
                                s, a, w);
    const int64_t rows = (a.T + a.N - 1) / a.N * a.group;  // of a sequence and key head, on average
    const int64_t shares = (rows + kMergeWarps - 1) / kMergeWarps;
    return launch_dependent(step_merge_prefix_kernel<T, D>, dim3(a.N, a.Hkv, (unsigned)(shares < 64 ? shares : 64)),
                            dim3(kMergeThreads), 0, s, a, w);
}

// Rows per tile of the own keys' part, by the rows that a sequence has on average: a
// tile's cost grows with it, and rows beyond the first tile read the keys again.  (bf16, own
// keys of up to 2000: 16 rows against 32, 64 sequences with 18 rows 26 / 27 us, with 26, 32 heads of 64
// on 8, 71 / 65; 32 against 64, 64 with 51 rows 44 / 47, the same behind a prefix 70 / 68, 4 with 1037
// rows 217 / 176.  fp32, 32 rows against 64, which leave room for one CTA on an SM: 20 sequences
// of up to 12 tokens and 4000 keys, 16 heads of 128 on 2, 117 / 156 us; 28 of few keys 20 / 23; 100 of
// up to 1000, 32 heads of 64 on 8, 242 / 248.)
int rows_per_tile(int N, int64_t T, int group, int dtype) {
    const int64_t rows = (T + N - 1) / (N > 0 ? N : 1) * group;
    if (dtype == GDR_F32 && rows <= 8) return rows <= 4 ? 4 : 8;
    return rows <= 16 ? 16 : rows <= 32 || dtype == GDR_F32 ? 32 : 64;
}

// Rows per tile of the prefix in fp32, by the rows that the batch has on a key head.  (All
// kernels, 128 against 64: 32 sequences of up to 12 tokens behind 4000, 16 heads of 128 on 2, 270 / 304 us;
// 64 against 16: 200 of one token behind 3000, 8 heads of 64 on one, 68 / 100 us.)
int far_rows(int64_t T, int group, int D) {
    const int64_t rows = T * group;
    return rows >= 128 && D == 128 ? 128 : rows > 16 ? 64 : 16;
}

// Cuts of the prefix along its keys: about as many CTAs as the GPU holds at once.
void prefix_cuts(StepWork* w, int64_t T, int Hkv, int group, int D, int prefix_len, int dtype) {
    w->splits = w->far_ctas = w->far_tokens = 0;
    if (prefix_len == 0) return;
    const int64_t tiles = (prefix_len + kFarTile - 1) / kFarTile;
    if (dtype == GDR_BF16) {
        w->far_tokens = prefix_block_tokens(group);
        const int64_t blocks = (T + w->far_tokens - 1) / w->far_tokens * Hkv, all = blocks * tiles;
        int64_t ctas = all < kSms ? all : kSms;
        if (ctas > blocks * kMaxSplits) ctas = blocks * kMaxSplits;
        const int64_t least = all / ctas;  // tiles of a CTA
        const int64_t parts = (tiles + least - 1) / least + 1;
        w->far_ctas = (int)ctas;
        w->splits = (int)(parts < tiles ? parts : tiles);
        return;
    }
    const int rows = far_rows(T, group, D);
    const int64_t blocks = (T * group + rows - 1) / rows * Hkv;
    int64_t splits = (rows >= 64 && D == 128 ? 1 : 2) * kSms / blocks;  // CTAs that the GPU holds at once
    if (splits > tiles) splits = tiles;
    if (splits < 1) splits = 1;
    w->splits = (int)(splits < kMaxSplits ? splits : kMaxSplits);
}

// The workspace's parts (from `base`; a null one for the size alone).
size_t step_layout(StepWork* w, char* base, int N, int64_t T, int Hq, int Hkv, int D, int prefix_len,
                   int dtype) {
    size_t at = 0;
    auto part = [&](size_t bytes) {
        char* p = base + at;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    w->rows = rows_per_tile(N, T, Hq / Hkv, dtype);
    w->ctas = dtype == GDR_BF16 || w->rows == 8 ? kSms : 2 * kSms;  // what the GPU holds at once
    prefix_cuts(w, T, Hkv, Hq / Hkv, D, prefix_len, dtype);
    const size_t slots = (size_t)w->ctas * 2 * w->rows, rows = w->splits ? (size_t)T * Hq : 0;
    w->offsets = reinterpret_cast<int64_t*>(part(sizeof(int64_t) * ((size_t)N + 1)));
    w->cuts = reinterpret_cast<Cut*>(part(sizeof(Cut) * w->ctas));
    w->slot_stat = reinterpret_cast<float2*>(part(sizeof(float2) * slots));
    w->slot_sum = reinterpret_cast<float*>(part(sizeof(float) * slots * D));
    w->row_stat = reinterpret_cast<float2*>(part(sizeof(float2) * rows));
    w->row_sum = reinterpret_cast<float*>(part(sizeof(float) * rows * D));
    w->far_stat = reinterpret_cast<float2*>(part(sizeof(float2) * rows * w->splits));
    w->far_sum = reinterpret_cast<float*>(part(sizeof(float) * rows * w->splits * D));
    return at;
}

template <int D>
cudaError_t launch_step(const AttnArgs& a, StepWork w, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    if (a.dtype == GDR_BF16) {
        if (!tiled(a.ldq, a.Hq, D)) w.far_ctas = 0;
        if (w.splits > 0) e = w.far_ctas ? launch_prefix_tc(a, w, s) : launch_prefix_simt<__nv_bfloat16, D, 64>(a, w, s);
        if (e == cudaSuccess) e = launch_step_own(a, w, s);
        return e == cudaSuccess ? launch_merge<__nv_bfloat16, D>(a, w, s) : e;
    }
    if (w.splits > 0) {
        const int rows = far_rows(a.T, a.group, D);
        e = rows == 16   ? launch_prefix_simt<float, D, 16>(a, w, s)
            : rows == 64 ? launch_prefix_simt<float, D, 64>(a, w, s)
                         : launch_prefix_simt<float, D, D == 128 ? 128 : 64>(a, w, s);
    }
    if (e == cudaSuccess)
        e = w.rows <= 8    ? launch_step_few(a, w, s)
            : w.rows == 16 ? launch_step_simt<D, 16>(a, w, s)
                           : launch_step_simt<D, 32>(a, w, s);
    return e == cudaSuccess ? launch_merge<float, D>(a, w, s) : e;
}

// scale: the maximum of the scores is that of the products only for one above 0
int check_scale(float scale) {
    if (!(scale > 0.f) || scale > 1e30f)
        return set_last_error(GDR_ERR_INVALID_ARG, "scale must be positive and finite");
    return GDR_OK;
}

int check_attention(int N, int64_t T, int Hq, int Hkv, int D, int dtype) {
    if (int rc = check_heads(N, T, Hq, Hkv, D, dtype)) return rc;
    if (Hq == 0) return set_last_error(GDR_ERR_INVALID_ARG, "Hq must be positive");
    // (the bf16 prompt looks at N * Hkv places at least)
    if ((int64_t)N * Hkv > 1 << 24)
        return set_last_error(GDR_ERR_UNSUPPORTED, "N (%d) * Hkv (%d) above 2^24", N, Hkv);
    if (T * Hq > 0x7fffffffLL - 512)
        return set_last_error(GDR_ERR_UNSUPPORTED, "T_total (%lld) * Hq too large", (long long)T);
    return GDR_OK;
}

// The prefix's positions, as the table's: its tiles' ends are counted in 32 bits.
int check_prefix(int prefix_len) {
    if (prefix_len < 0) return set_last_error(GDR_ERR_INVALID_ARG, "prefix_len (%d) negative", prefix_len);
    if (prefix_len > 0x7fffffff - 256)
        return set_last_error(GDR_ERR_UNSUPPORTED, "prefix_len (%d) above 2^31 - 257", prefix_len);
    return GDR_OK;
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

int gdr_attn_fwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                 const int32_t* cu_seqlens, int N, int64_t T_total, int Hq, int Hkv, int D, float scale, int dtype,
                 int flags, void* o, int64_t o_stride, gdr_stream_t stream) {
    if (int rc = check_attention(N, T_total, Hq, Hkv, D, dtype)) return rc;
    if (flags & ~GDR_VALIDATE) return set_last_error(GDR_ERR_INVALID_ARG, "unsupported flags 0x%x for gdr_attn_fwd", flags);
    if (int rc = check_scale(scale)) return rc;
    if (N == 0 || T_total == 0) return set_ok();
    if (int rc = check_token_rows("q", q, q_stride, 0, dtype)) return rc;
    if (int rc = check_token_rows("k", k, k_stride, 0, dtype)) return rc;
    if (int rc = check_token_rows("v", v, v_stride, 0, dtype)) return rc;
    if (int rc = check_token_rows("o", o, o_stride, (int64_t)Hq * D, dtype)) return rc;
    if (int rc = check_int32s("cu_seqlens", cu_seqlens)) return rc;
    const int64_t e = dtype == GDR_BF16 ? 2 : 4;
    const MemRows out{"o", o, (int64_t)Hq * D * e, o_stride * e, T_total};
    if (int rc = check_apart(out, {"q", q, (int64_t)Hq * D * e, q_stride * e, T_total})) return rc;
    if (int rc = check_apart(out, {"k", k, (int64_t)Hkv * D * e, k_stride * e, T_total})) return rc;
    if (int rc = check_apart(out, {"v", v, (int64_t)Hkv * D * e, v_stride * e, T_total})) return rc;
    if (int rc = check_device()) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    if (flags & GDR_VALIDATE)
        if (int rc = validate_attention(cu_seqlens, N, T_total, nullptr, s)) return rc;
    AttnArgs a{};
    a.q = q; a.k = k; a.v = v; a.o = o;
    a.ldq = q_stride; a.ldk = k_stride; a.ldv = v_stride; a.ldo = o_stride;
    a.cu = cu_seqlens; a.N = N; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.group = Hq / Hkv; a.T = T_total;
    a.scale_log2 = scale * 1.44269504088896341f;
    a.dtype = dtype;
    const cudaError_t launched = dtype == GDR_BF16 && tiled(q_stride, Hq, D) && tiled(k_stride, Hkv, D) && tiled(v_stride, Hkv, D)
                              ? launch_prompt_tc(a, s)
                          : dtype == GDR_BF16 ? (D == 128 ? launch_prompt_simt<__nv_bfloat16, 128>(a, s)
                                                          : launch_prompt_simt<__nv_bfloat16, 64>(a, s))
                                            : (D == 128 ? launch_prompt_simt<float, 128>(a, s)
                                                        : launch_prompt_simt<float, 64>(a, s));
    return launch_result(launched, "gdr_attn_fwd launch");
}

int gdr_attn_step_workspace_size(int N, int64_t T_total, int Hq, int Hkv, int D, int prefix_len, int dtype,
                                 size_t* bytes) {
    if (!bytes) return set_last_error(GDR_ERR_INVALID_ARG, "bytes is NULL");
    if (int rc = check_attention(N, T_total, Hq, Hkv, D, dtype)) return rc;
    if (int rc = check_prefix(prefix_len)) return rc;
    StepWork w{};
    *bytes = N == 0 || T_total == 0 ? 0 : step_layout(&w, nullptr, N, T_total, Hq, Hkv, D, prefix_len, dtype);
    return set_ok();
}

int gdr_attn_step(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache, int num_pages,
                  int page_size, const int32_t* block_table, int64_t table_stride, int max_pages,
                  const int32_t* cache_lens, const int32_t* prefix_pages, int prefix_len, const int32_t* cu_seqlens,
                  int N, int64_t T_total, int Hq, int Hkv, int D, float scale, int dtype, int flags, void* o,
                  int64_t o_stride, void* workspace, size_t ws_bytes, gdr_stream_t stream) {
    if (int rc = check_attention(N, T_total, Hq, Hkv, D, dtype)) return rc;
    if (flags & ~GDR_VALIDATE) return set_last_error(GDR_ERR_INVALID_ARG, "unsupported flags 0x%x for gdr_attn_step", flags);
    if (int rc = check_prefix(prefix_len)) return rc;
    if ((prefix_len > 0) != (prefix_pages != nullptr))
        return set_last_error(GDR_ERR_INVALID_ARG, "prefix_pages goes with prefix_len (%d) > 0", prefix_len);
    if (int rc = check_scale(scale)) return rc;
    if (N == 0 || T_total == 0) return set_ok();
    AttnArgs a{};
    a.cache = Paged{const_cast<void*>(k_cache), const_cast<void*>(v_cache), block_table, table_stride, cache_lens,
                    prefix_pages, prefix_len, max_pages, num_pages, page_size, 0};
    if (int rc = check_paged(a.cache, N, Hkv, D, dtype)) return rc;
    while ((1 << a.cache.page_bits) < page_size) ++a.cache.page_bits;
    if (prefix_pages)
        if (int rc = check_int32s("prefix_pages", prefix_pages)) return rc;
    if (int rc = check_token_rows("q", q, q_stride, 0, dtype)) return rc;
    if (int rc = check_token_rows("o", o, o_stride, (int64_t)Hq * D, dtype)) return rc;
    if (int rc = check_int32s("cu_seqlens", cu_seqlens)) return rc;
    StepWork w{};
    const size_t need = step_layout(&w, static_cast<char*>(workspace), N, T_total, Hq, Hkv, D, prefix_len,
                                    dtype);
    if (!workspace || ws_bytes < need)
        return set_last_error(GDR_ERR_WORKSPACE, "workspace %zu bytes < required %zu", workspace ? ws_bytes : (size_t)0, need);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return set_last_error(GDR_ERR_INVALID_ARG, "workspace not 256-byte aligned");
    const int64_t e = dtype == GDR_BF16 ? 2 : 4, cache = (int64_t)num_pages * Hkv * page_size * D * e;
    const MemRows out{"o", o, (int64_t)Hq * D * e, o_stride * e, T_total};
    const MemRows in[3] = {{"q", q, (int64_t)Hq * D * e, q_stride * e, T_total}, {"k_cache", k_cache, cache, cache, 1},
                           {"v_cache", v_cache, cache, cache, 1}};
    for (const MemRows& x : in)
        if (int rc = check_apart(out, x)) return rc;
    const MemRows scratch{"workspace", workspace, (int64_t)need, (int64_t)need, 1};
    if (int rc = check_apart(scratch, out)) return rc;
    for (const MemRows& x : in)
        if (int rc = check_apart(scratch, x)) return rc;
    if (int rc = check_device()) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    if (flags & GDR_VALIDATE)
        if (int rc = validate_attention(cu_seqlens, N, T_total, &a.cache, s)) return rc;
    a.q = q; a.o = o; a.ldq = q_stride; a.ldo = o_stride;
    a.cu = cu_seqlens; a.N = N; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.group = Hq / Hkv; a.T = T_total;
    a.scale_log2 = scale * 1.44269504088896341f;
    a.dtype = dtype;
    const cudaError_t launched = D == 128 ? launch_step<128>(a, w, s) : launch_step<64>(a, w, s);
    return launch_result(launched, "gdr_attn_step launch");
}

}  // extern "C"
