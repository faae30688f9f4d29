// Tensor maps and copies of the attention kernels (bf16), and the slow way for single rows.
#pragma once

#include <cuda.h>
#include <math.h>

#include <atomic>

#include "attn.h"
#include "common.cuh"
#include "tc.cuh"

namespace gdr {
namespace {

using namespace tc;

constexpr unsigned kAttnError = 0x800;  // device error word: a wait gave up

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        :: "r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(mbar) : "memory");
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        :: "r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(mbar) : "memory");
}

// mbar_wait for those that may wait for a warp with rows to compute once more, which can take
// longer than the limit: it counts itself in abort[1].
__device__ __forceinline__ bool mbar_wait_busy(uint32_t mbar, uint32_t parity, volatile int* abort) {
    if (mbar_test(mbar, parity)) return true;
    uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try(mbar, parity)) return true;
        if ((i & 255) == 0) {
            if (abort[0]) return false;
            if (abort[1]) t0 = globaltimer_ns();
            if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
        }
    }
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Key j's rows of head h in the caches, false where it has no page.
template <int D>
__device__ __forceinline__ bool cached_row(const Paged& c, const int32_t* pages, int Hkv, int h, int64_t j,
                                           const __nv_bfloat16*& kp, const __nv_bfloat16*& vp) {
    const int page = pages[j >> c.page_bits];
    if (page < 0 || page >= c.num_pages) return false;
    const int64_t row = (((int64_t)page * Hkv + h) << c.page_bits) + (j & (c.page_size - 1));
    kp = static_cast<const __nv_bfloat16*>(c.k) + row * D;
    vp = static_cast<const __nv_bfloat16*>(c.v) + row * D;
    return true;
}

// ---- rows once more ----------------------------------------------------------------------

// One row, a warp together: the keys [from, end) that it sees, read by rows(j, k, v).  A lane has
// a key's score, then channels (D / 32) lane .. of the sums, which are left undivided.
template <int D, typename R>
__device__ __noinline__ void row_again(const __nv_bfloat16* q, int64_t from, int64_t end, float scale, R rows,
                                       float (&acc)[D / 32], float& m, float& l) {
    constexpr int C = D / 32;
    const int lane = threadIdx.x & 31;
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
    for (int64_t j0 = from; j0 < end; j0 += 32) {
        const __nv_bfloat16 *kp = nullptr, *vp = nullptr;
        float s = -INFINITY;
        if (j0 + lane < end && rows(j0 + lane, kp, vp)) {
            float dot[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
            for (int d = 0; d < D; d += 8) {
                float x[8], k[8];
                Vec<__nv_bfloat16, 8>::load(q + d, x);
                Vec<__nv_bfloat16, 8>::load(kp + d, k);
#pragma unroll
                for (int e = 0; e < 8; ++e) dot[e & 3] = fmaf(x[e], k[e], dot[e & 3]);
            }
            s = (dot[0] + dot[1] + (dot[2] + dot[3])) * scale;
        } else {
            vp = nullptr;
        }
        float top = s;
#pragma unroll
        for (int off = 16; off; off /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        top = fmaxf(m, top);
        const float base = top == -INFINITY ? 0.f : top, back = exp2f(m - base), p = exp2f(s - base);
        m = top;
        l = fmaf(l, back, p);
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] *= back;
#pragma unroll 8
        for (int k = 0; k < 32; ++k) {
            const float w = __shfl_sync(0xffffffffu, p, k);
            const auto* value = reinterpret_cast<const __nv_bfloat16*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(vp), k));
            if (!value) continue;
            float v[C];
            Vec<__nv_bfloat16, C>::load(value + lane * C, v);
#pragma unroll
            for (int c = 0; c < C; ++c) acc[c] = fmaf(w, v[c], acc[c]);
        }
    }
    l = warp_sum(l);
}

// The largest of a lane's values (as packed bf16 bits) at keys [from, end), by their bits as signed
// and as unsigned numbers: what is above +inf in the one and above -inf in the other is a NaN.  Up to where
// every lane's are NaN in the channels of `want` (ones in their halves of the words).
template <int W, typename R>
__device__ __forceinline__ void largest_bits(int64_t from, int64_t end, R rows, const uint32_t (&want)[W],
                                             uint32_t (&as_signed)[W], uint32_t (&as_unsigned)[W]) {
    constexpr int KEYS = 96 / W;  // under way
    const int lane = threadIdx.x & 31;
    const bool mine = (want[0] | want[W - 1]) != 0;  // the other lanes' are left in memory
#pragma unroll
    for (int w = 0; w < W; ++w) {
        as_signed[w] = 0x80008000u;
        as_unsigned[w] = 0;
    }
    auto look = [&](auto key_of) {
        uint32_t v[KEYS][W];
#pragma unroll
        for (int i = 0; i < KEYS; ++i) {
            const __nv_bfloat16 *kp, *vp;
#pragma unroll
            for (int w = 0; w < W; ++w) v[i][w] = 0;
            if (rows(key_of(i), kp, vp) && mine) {
                const uint32_t* at = reinterpret_cast<const uint32_t*>(vp) + lane * W;
                if constexpr (W == 2) {
                    const uint2 x = *reinterpret_cast<const uint2*>(at);
                    v[i][0] = x.x;
                    v[i][1] = x.y;
                } else {
                    v[i][0] = *at;
                }
            }
        }
        bool more = false;
#pragma unroll
        for (int w = 0; w < W; ++w) {
#pragma unroll
            for (int i = 0; i < KEYS; ++i) {
                as_signed[w] = __vmaxs2(as_signed[w], v[i][w]);
                as_unsigned[w] = __vmaxu2(as_unsigned[w], v[i][w]);
            }
            const uint32_t nan = __vcmpgts2(as_signed[w], 0x7f807f80u) | __vcmpgtu2(as_unsigned[w], 0xff80ff80u);
            more |= (want[w] & ~nan) != 0;
        }
        return __any_sync(0xffffffffu, more) != 0;
    };
    int64_t j0 = from;
    for (; j0 + KEYS <= end; j0 += KEYS)
        if (!look([&](int i) { return j0 + i; })) return;
    // (the last key several times, not one behind it)
    if (j0 < end) look([&](int i) { return min(j0 + i, end - 1); });
}

// A warp's rows (bad: a bit for each lane that has one; its query, result, statistics and the end
// of the keys that it sees) whose sums hold an infinity or a NaN, although those of the weights do
// not: it comes from the values of keys from .. end - 1, which is what the products took.  They are
// right where only keys that the row sees have such values.  A channel in which one does that the row
// does not see (a weight of 0 makes it a NaN) is a NaN or an infinity by the row's own keys, which their
// values tell, or the row is computed once more.  partial: the result is sums, fp32.
template <int D, typename R>
__device__ __noinline__ void rows_again(uint32_t bad, bool partial, const __nv_bfloat16* q, void* to, float2* stat,
                                        int limit, int from, int end, float scale, R rows) {
    constexpr int C = D / 32, NEVER = 0x7fffffff;
    const int lane = threadIdx.x & 31;
    const bool mine = bad >> lane & 1;
    const int least = __reduce_min_sync(0xffffffffu, mine ? limit : NEVER);
    // of each channel the last such key, and the first of each kind (-1: one that all rows see)
    int last[C], nan[C], inf[2][C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        last[c] = -1;
        nan[c] = inf[0][c] = inf[1][c] = NEVER;
    }
    // the keys that not all rows see
    constexpr int KEYS = 64 / C;
    for (int64_t j0 = max(least, from); j0 < end; j0 += KEYS) {
        float v[KEYS][C];
#pragma unroll
        for (int i = 0; i < KEYS; ++i) {
            const __nv_bfloat16 *kp, *vp;
#pragma unroll
            for (int c = 0; c < C; ++c) v[i][c] = 0.f;
            if (rows(min(j0 + i, (int64_t)end - 1), kp, vp)) Vec<__nv_bfloat16, C>::load(vp + lane * C, v[i]);
        }
#pragma unroll
        for (int i = 0; i < KEYS; ++i)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int j = min((int)j0 + i, end - 1);  // the last key several times, not one behind it
                if (fabsf(v[i][c]) < INFINITY) continue;
                last[c] = j;
                if (v[i][c] != v[i][c]) nan[c] = min(nan[c], j);
                else if (v[i][c] > 0.f) inf[0][c] = min(inf[0][c], j);
                else inf[1][c] = min(inf[1][c], j);
            }
    }
    bool any = false;
    uint32_t want[C / 2], as_signed[C / 2], as_unsigned[C / 2];
#pragma unroll
    for (int w = 0; w < C / 2; ++w) {
        want[w] = (last[2 * w] < 0 ? 0 : 0xffffu) | (last[2 * w + 1] < 0 ? 0 : 0xffff0000u);
        any |= want[w] != 0;
    }
    if (!__any_sync(0xffffffffu, any)) return;
    // those that all see
    largest_bits<C / 2>(from, min(least, end), rows, want, as_signed, as_unsigned);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const uint32_t s = as_signed[c / 2] >> c % 2 * 16 & 0xffff, u = as_unsigned[c / 2] >> c % 2 * 16 & 0xffff;
        if ((s > 0x7f80u && s < 0x8000u) || u > 0xff80u) nan[c] = -1;
        if (s == 0x7f80u) inf[0][c] = -1;
        if (u == 0xff80u) inf[1][c] = -1;
    }
    auto of = [](const void* x, int who) {
        return __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(x), who);
    };
    for (; bad; bad &= bad - 1) {
        const int who = __ffs(bad) - 1, sees = __shfl_sync(0xffffffffu, limit, who);
        auto* const result = reinterpret_cast<char*>(of(to, who));
        auto* const its = reinterpret_cast<float2*>(of(stat, who));
        const auto* query = reinterpret_cast<const __nv_bfloat16*>(of(q, who));
        bool open = false;
#pragma unroll
        for (int c = 0; c < C; ++c) open |= last[c] >= sees && min(nan[c], min(inf[0][c], inf[1][c])) >= sees;
        if (__any_sync(0xffffffffu, open)) {
            float acc[C], m, l;
            row_again<D>(query, from, min(sees, end), scale, rows, acc, m, l);
            if (partial) {
                Vec<float, C>::store(reinterpret_cast<float*>(result) + lane * C, acc);
                if (lane == 0) *its = make_float2(m, l);
            } else {
#pragma unroll
                for (int c = 0; c < C; ++c) acc[c] /= l;
                Vec<__nv_bfloat16, C>::store(reinterpret_cast<__nv_bfloat16*>(result) + lane * C, acc);
            }
            continue;
        }
        // (a NaN is there already)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (last[c] < sees || nan[c] < sees || (inf[0][c] < sees && inf[1][c] < sees)) continue;
            const float x = inf[0][c] < sees ? INFINITY : -INFINITY;
            if (partial) reinterpret_cast<float*>(result)[lane * C + c] = x;
            else reinterpret_cast<__nv_bfloat16*>(result)[lane * C + c] = __float2bfloat16(x);
        }
    }
}

// ---- tensor maps (host) ----------------------------------------------------------------

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

bool encode(CUtensorMap* map, const void* p, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
    const EncodeTiled f = encode_tiled();
    const cuuint32_t steps[3] = {1, 1, 1};
    return f && f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(p), dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [T, heads, D] rows in boxes of 64 channels, `hb` heads and `tb` tokens.
bool encode_tokens(CUtensorMap* map, const void* p, int64_t ld, int64_t T, int heads, int D, int hb, int tb) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)hb, (cuuint32_t)tb};
    return encode(map, p, 3, dims, strides, box);
}

// The cache's rows in boxes of 64 channels and `rows` rows.
bool encode_cache(CUtensorMap* map, const void* p, int64_t all, int D, int rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)all};
    const cuuint64_t strides[1] = {(cuuint64_t)D * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)rows};
    return encode(map, p, 2, dims, strides, box);
}

}  // namespace
}  // namespace gdr
