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

// One row once more, a warp together: the keys [from, end) that it sees, read by
// rows(j, k, v).  Lane l has channels (D / 32) l ..  Leaves the sums, not divided.
template <int D, typename R>
__device__ __noinline__ void row_again(const __nv_bfloat16* q, int64_t from, int64_t end, float scale, R rows,
                                       float (&acc)[D / 32], float& m, float& l) {
    constexpr int C = D / 32;
    const int lane = threadIdx.x & 31;
    float x[C];
    Vec<__nv_bfloat16, C>::load(q + lane * C, x);
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
    for (int64_t j = from; j < end; ++j) {
        const __nv_bfloat16 *kp, *vp;
        if (!rows(j, kp, vp)) continue;
        float k[C], v[C], dot = 0.f;
        Vec<__nv_bfloat16, C>::load(kp + lane * C, k);
        Vec<__nv_bfloat16, C>::load(vp + lane * C, v);
#pragma unroll
        for (int c = 0; c < C; ++c) dot = fmaf(x[c], k[c], dot);
        const float s = warp_sum(dot) * scale, top = fmaxf(m, s);
        const float base = top == -INFINITY ? 0.f : top, back = exp2f(m - base), p = exp2f(s - base);
        m = top;
        l = fmaf(l, back, p);
        // a weight of 0 (a score of -inf) takes nothing from the value
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] = p == 0.f ? acc[c] * back : fmaf(acc[c], back, p * v[c]);
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
