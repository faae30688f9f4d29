// Root-mean-square norm with the residual's addition (output in the input's
// type or e4m3 with scales) and its backward, with their C entry points
// (contract in include/gdr.h).
//
// Every tensor is read and written once; bound by memory as long as a row's
// arithmetic is kept short (packed fp32 pairs, the scale group a compile-time
// length, no division per element: e4m3 at 32768 x 4096 went 212 -> 149 us on
// that alone).  One GB300, device times, of the copy rate (6.69 TB/s measured):
//   forward  32768 x 4096  bf16 + residual, e4m3 by 128   153 us   92 %
//            16384 x 4096  bf16 + residual, bf16           84 us   95 %
//            16384 x 4096  fp32 + residual                172 us   93 %
//             8192 x 8192  bf16 + residual, e4m3 by row    88 us   80 %
//            98000 x 128   bf16                            18 us   42 %
//             3001 x 1001  fp32, e4m3 by row, odd rows     11 us   20 % (in L2)
//                8 x 4096  bf16 + residual                2.5 us   (latency)
//   backward 16384 x 4096  bf16 + residual gradient        90 us   89 %
//            16384 x 4096  fp32 + residual gradient       167 us   96 %
//             8192 x 7168  bf16 + residual gradient        82 us   86 %
//             4096 x 16384 bf16 + residual gradient       160 us   50 %
//             4096 x 16384 fp32 + residual gradient       583 us   28 %
//            65536 x 256   bf16 + residual gradient        36 us   55 %
//             9000 x 1001  fp32, odd rows                  41 us   52 %
// A row of 128 is one load of each of its sixteen threads, which meet before the next
// row's is asked for.  Registers do not hold the widest rows: the compiler spills 24
// bytes of the forward at 8 bf16 pieces per thread and a scale per row, 80 to 128 at 8
// fp32 pieces, 220 to 240 and 1260 to 1860 at 32 and 64 single elements; backward 310 in
// the ring of 4 bf16 pieces (8200 to 16384 columns), 120 and 260 at 2 pieces from memory
// (136 to 504 columns, bf16 and fp32), 1410 and 2650 at 8 (wider than the ring), 50 and
// 1400 to 1700 at 16 and 64 single elements.
#include <cuda_fp8.h>
#include <math.h>

#include "common.cuh"
#include "gdr.h"
#include "launch.h"
#include "tc.cuh"

namespace gdr {
namespace {

constexpr float kE4m3Max = 448.f;     // largest finite e4m3 value
constexpr float kAmaxFloor = 1e-12f;  // a group of zeros gets a scale too

struct NormParams {
    const void* x;
    const void* residual;
    const float* w;
    void* sum;
    void* y;
    float* scales;
    int64_t ldx, ldr, lds, ldy, M;
    int D, group, groups;
    int tpr;  // threads of a row, a power of two
    float eps;
};

// ---- 8 consecutive elements, kept as they are stored, worked on in pairs ----------

template <typename T> struct Cells;

template <> struct Cells<__nv_bfloat16> {
    uint32_t w[4];
    __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const {
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ float2 get(int i) const {
        return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    __device__ __forceinline__ void set(int i, float2 f) { w[i] = tc::pack_bf16(f.x, f.y); }
    // the rounded sum: a bf16 sum is the same rounded once or through fp32 (where fp32 has to
    // round, the smaller term is below 2^-16 of the larger, and no midpoint is that near a bf16 value)
    __device__ __forceinline__ void add(const Cells& o) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 r = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]),
                                             *reinterpret_cast<const __nv_bfloat162*>(&o.w[i]));
            w[i] = *reinterpret_cast<const uint32_t*>(&r);
        }
    }
};
template <> struct Cells<float> {
    float2 w[4];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = make_float2(0.f, 0.f);
    }
    __device__ __forceinline__ void load(const float* p) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        w[0] = make_float2(a.x, a.y); w[1] = make_float2(a.z, a.w);
        w[2] = make_float2(b.x, b.y); w[3] = make_float2(b.z, b.w);
    }
    __device__ __forceinline__ void store(float* p) const {
        reinterpret_cast<float4*>(p)[0] = make_float4(w[0].x, w[0].y, w[1].x, w[1].y);
        reinterpret_cast<float4*>(p)[1] = make_float4(w[2].x, w[2].y, w[3].x, w[3].y);
    }
    __device__ __forceinline__ float2 get(int i) const { return w[i]; }
    __device__ __forceinline__ void set(int i, float2 f) { w[i] = f; }
    __device__ __forceinline__ void add(const Cells& o) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __fadd2_rn(w[i], o.w[i]);
    }
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ void store_codes(__nv_fp8_storage_t* p, const float2 (&f)[4]) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(f[2 * i], __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(f[2 * i + 1], __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | hi << 16;
    }
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// A group's scale, amax / 448, and its values' quotients by it: products with the
// reciprocal, each corrected by its exact remainder (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990), which finds a
// quotient that fp32 holds to the last bit whatever the reciprocal's own rounding.  So a
// value half-way between two codes is seen to be half-way; by the product alone about
// half of those went to the wrong code.  (At 32768 x 4096 by the product alone 149 us,
// by division 163, so 153.)  Where the scale is infinite there is no remainder: finite
// values give 0.  Where it is NaN, so is every code.
struct Scale {
    float scale, inverse, minus;
    __device__ __forceinline__ explicit Scale(float amax) {
        const float a = amax < kAmaxFloor ? kAmaxFloor : amax, q = __fmul_rn(a, 1.f / kE4m3Max);
        const bool finite = a < INFINITY;
        scale = finite ? fmaf(fmaf(q, -kE4m3Max, a), 1.f / kE4m3Max, q) : a;
        inverse = __fdividef(1.f, scale);
        minus = finite ? -scale : 0.f;
    }
    __device__ __forceinline__ float2 operator()(float2 f) const {
        const float2 q = __fmul2_rn(f, both(inverse));
        return __ffma2_rn(__ffma2_rn(q, both(minus), f), both(inverse), q);
    }
    __device__ __forceinline__ float operator()(float f) const {
        const float q = __fmul_rn(f, inverse);
        return fmaf(fmaf(q, minus, f), inverse, q);
    }
};

// The larger of two, NaN if either is: a NaN reaches its group's scale.
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// Reductions over the tpr threads of a row: shuffles, and above a warp one
// exchange of the warps' results behind a barrier of the row's threads.  `turn`
// alternates from call to call (two buffers: one barrier each suffices).
constexpr int kMaxThreads = 512;

struct RowReduce {
    float2 (*buf)[kMaxThreads / 32];
    int tpr, slot, turn;

    template <typename F>
    __device__ __forceinline__ float2 all(float2 v, F op) {
        for (int off = min(tpr, 32) >> 1; off >= 1; off >>= 1) {
            const float2 o = make_float2(__shfl_xor_sync(0xffffffffu, v.x, off), __shfl_xor_sync(0xffffffffu, v.y, off));
            v = op(v, o);
        }
        if (tpr > 32) {
            const int warps = tpr >> 5, at = slot * warps;
            if ((threadIdx.x & 31) == 0) buf[turn][threadIdx.x >> 5] = v;
            tc::bar_sync(1 + slot, tpr);
            v = buf[turn][at];
            for (int i = 1; i < warps; ++i) v = op(v, buf[turn][at + i]);
            turn ^= 1;
        }
        return v;
    }
    __device__ __forceinline__ float2 sum(float2 v) {
        return all(v, [](float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); });
    }
    __device__ __forceinline__ float max(float v) {
        return all(make_float2(v, 0.f), [](float2 a, float2 b) { return make_float2(max_nan(a.x, b.x), 0.f); }).x;
    }
};

// Forward on aligned rows.  A row belongs to tpr threads, CH pieces of 8 elements
// each, and is held as stored from its one read to its output.  CH = 8 where there
// are rows enough (bf16 at 16384 x 4096: 4: 84 -> 89 us, 2: 93 us).  MODE: kSame for
// the input's type, kRow for codes with one scale per row, else the group's
// length: its 8-element pieces lie in neighbouring threads.
constexpr int kSame = -1, kRow = 0;

template <typename T, int CH, int MODE>
__global__ void __launch_bounds__(kMaxThreads, 1) rmsnorm_fwd_kernel(NormParams p) {
    __shared__ float2 exchange[2][kMaxThreads / 32];
    const int tpr = p.tpr, slots = blockDim.x / tpr, slot = threadIdx.x / tpr, l = threadIdx.x % tpr;
    RowReduce reduce{exchange, tpr, slot, 0};
    const float mean = 1.f / p.D;
    for (int64_t m0 = (int64_t)blockIdx.x * slots; m0 < p.M; m0 += (int64_t)gridDim.x * slots) {
        const int64_t m = m0 + slot;
        const int width = m < p.M ? p.D : 0;  // a missing row has no elements
        const T* x = static_cast<const T*>(p.x) + m * p.ldx;
        Cells<T> s[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * tpr + l) * 8;
            s[c].zero();
            if (e < width) s[c].load(x + e);
        }
        if (p.residual) {
            const T* res = static_cast<const T*>(p.residual) + m * p.ldr;
            T* sum = static_cast<T*>(p.sum) + m * p.lds;
            Cells<T> r[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int e = (c * tpr + l) * 8;
                r[c].zero();
                if (e < width) r[c].load(res + e);
            }
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int e = (c * tpr + l) * 8;
                s[c].add(r[c]);  // the stored sum is what the norm is taken of
                if (e < width) s[c].store(sum + e);
            }
        }
        float2 ss = both(0.f);
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = s[c].get(i);
                ss = __ffma2_rn(f, f, ss);
            }
        const float rstd = 1.f / sqrtf(fmaf(reduce.sum(make_float2(ss.x + ss.y, 0.f)).x, mean, p.eps));

        auto norm = [&](int c, float2 (&f)[4]) {
            const int e = (c * tpr + l) * 8;
            Cells<float> w;
            w.zero();
            if (e < p.D) w.load(p.w + e);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = __fmul2_rn(__fmul2_rn(s[c].get(i), both(rstd)), w.get(i));
        };
        auto largest = [](const float2 (&f)[4]) {
            float a = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) a = max_nan(a, max_nan(fabsf(f[i].x), fabsf(f[i].y)));
            return a;
        };
        if (MODE == kSame) {
            T* y = static_cast<T*>(p.y) + m * p.ldy;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int e = (c * tpr + l) * 8;
                float2 f[4];
                norm(c, f);
                Cells<T> out;
#pragma unroll
                for (int i = 0; i < 4; ++i) out.set(i, f[i]);
                if (e < width) out.store(y + e);
            }
            continue;
        }
        __nv_fp8_storage_t* y = static_cast<__nv_fp8_storage_t*>(p.y) + m * p.ldy;
        float* scales = p.scales + m * p.groups;
        if (MODE == kRow) {
            float most = 0.f;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                float2 f[4];
                norm(c, f);
                most = max_nan(most, largest(f));
            }
            const Scale by(reduce.max(most));
            if (l == 0 && width) *scales = by.scale;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int e = (c * tpr + l) * 8;
                float2 f[4];
                norm(c, f);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = by(f[i]);
                if (e < width) store_codes(y + e, f);
            }
        } else {
            constexpr int SPAN = MODE > 0 ? MODE / 8 : 1;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int e = (c * tpr + l) * 8;
                float2 f[4];
                norm(c, f);
                float most = largest(f);
#pragma unroll
                for (int off = SPAN / 2; off >= 1; off >>= 1)
                    most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, off));
                const Scale by(most);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = by(f[i]);
                if (e < width) {
                    store_codes(y + e, f);
                    if (l % SPAN == 0) scales[e / (SPAN * 8)] = by.scale;
                }
            }
        }
    }
}

// Forward on any rows: one element at a time, CH per thread, neighbours in
// neighbouring threads.  Held to 64 registers up to CH = 8, for the loads of 1024
// threads per SM (9000 x 1001 fp32: 47 -> 34 us).
template <typename T, int CH, bool FP8>
__global__ void __launch_bounds__(kMaxThreads, CH <= 8 ? 2 : 1) rmsnorm_fwd_any_kernel(NormParams p) {
    __shared__ float2 exchange[2][kMaxThreads / 32];
    __shared__ int amax_s[FP8 ? 1024 : 1];
    const int tpr = p.tpr, slots = blockDim.x / tpr, slot = threadIdx.x / tpr, l = threadIdx.x % tpr;
    RowReduce reduce{exchange, tpr, slot, 0};
    const float mean = 1.f / p.D;
    for (int64_t m0 = (int64_t)blockIdx.x * slots; m0 < p.M; m0 += (int64_t)gridDim.x * slots) {
        const int64_t m = m0 + slot;
        const int width = m < p.M ? p.D : 0;
        const T* x = static_cast<const T*>(p.x) + m * p.ldx;
        float s[CH], ss = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) s[c] = c * tpr + l < width ? to_f(x[c * tpr + l]) : 0.f;
        if (p.residual) {
            const T* res = static_cast<const T*>(p.residual) + m * p.ldr;
            T* sum = static_cast<T*>(p.sum) + m * p.lds;
            float r[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) r[c] = c * tpr + l < width ? to_f(res[c * tpr + l]) : 0.f;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const T q = from_f<T>(s[c] + r[c]);
                s[c] = to_f(q);
                if (c * tpr + l < width) sum[c * tpr + l] = q;
            }
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) ss = fmaf(s[c], s[c], ss);
        const float rstd = 1.f / sqrtf(fmaf(reduce.sum(make_float2(ss, 0.f)).x, mean, p.eps));
#pragma unroll
        for (int c = 0; c < CH; ++c)
            s[c] = c * tpr + l < p.D ? __fmul_rn(__fmul_rn(s[c], rstd), p.w[c * tpr + l]) : 0.f;
        if (!FP8) {
            T* y = static_cast<T*>(p.y) + m * p.ldy;
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (c * tpr + l < width) y[c * tpr + l] = from_f<T>(s[c]);
            continue;
        }
        __nv_fp8_storage_t* y = static_cast<__nv_fp8_storage_t*>(p.y) + m * p.ldy;
        float* scales = p.scales + m * p.groups;
        if (p.groups == 1) {
            float most = 0.f;
#pragma unroll
            for (int c = 0; c < CH; ++c) most = max_nan(most, fabsf(s[c]));
            const Scale by(reduce.max(most));
            if (l == 0 && width) *scales = by.scale;
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (c * tpr + l < width) y[c * tpr + l] = __nv_cvt_float_to_fp8(by(s[c]), __NV_SATFINITE, __NV_E4M3);
            continue;
        }
        // a group crosses warps: its largest magnitude in shared memory (the order of a maximum does not
        // matter), a warp's 32 neighbours, which lie in one group, reduced before; the bits of magnitudes
        // are ordered as they are, NaN above all numbers
        int* amax = amax_s + slot * p.groups;
        const int shift = p.group == 32 ? 5 : p.group == 64 ? 6 : 7;
        auto meet = [&]() {
            if (tpr <= 32)
                __syncwarp();
            else
                tc::bar_sync(1 + slot, tpr);
        };
        for (int i = l; i < p.groups; i += tpr) amax[i] = 0;
        meet();
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const unsigned most = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(s[c])));
            if ((l & 31) == 0 && c * tpr + l < p.D) atomicMax(amax + ((c * tpr + l) >> shift), (int)most);
        }
        meet();
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = c * tpr + l;
            if (e < width) {
                const Scale by(__int_as_float(amax[e >> shift]));
                y[e] = __nv_cvt_float_to_fp8(by(s[c]), __NV_SATFINITE, __NV_E4M3);
                if ((e & (p.group - 1)) == 0) scales[e >> shift] = by.scale;
            }
        }
        meet();
    }
}

// Threads of a row that holds `pieces` pieces, ch of them per thread.
int row_threads(int pieces, int ch, int least) {
    int t = least;
    while (t * ch < pieces && t < kMaxThreads) t *= 2;
    return t;
}

struct Shape {
    unsigned grid, block;
};

// CTAs of at least 256 threads, at most 32 per SM, which then walk the rows.
Shape shape_of(const NormParams& p) {
    const int block = p.tpr > 256 ? p.tpr : 256, slots = block / p.tpr;
    const int64_t want = (p.M + slots - 1) / slots, most = (int64_t)sm_count() * 32;
    return {(unsigned)(want < most ? want : most), (unsigned)block};
}

template <typename T, int CH>
cudaError_t launch_fwd_ch(const NormParams& p, bool fp8, cudaStream_t s) {
    const Shape h = shape_of(p);
    KernelTimer kt("rmsnorm_fwd", s);
    switch (!fp8 ? kSame : p.groups == 1 ? kRow : p.group) {
        case kSame: rmsnorm_fwd_kernel<T, CH, kSame><<<h.grid, h.block, 0, s>>>(p); break;
        case kRow: rmsnorm_fwd_kernel<T, CH, kRow><<<h.grid, h.block, 0, s>>>(p); break;
        case 32: rmsnorm_fwd_kernel<T, CH, 32><<<h.grid, h.block, 0, s>>>(p); break;
        case 64: rmsnorm_fwd_kernel<T, CH, 64><<<h.grid, h.block, 0, s>>>(p); break;
        default: rmsnorm_fwd_kernel<T, CH, 128><<<h.grid, h.block, 0, s>>>(p); break;
    }
    return cudaGetLastError();
}

template <typename T, int CH>
cudaError_t launch_fwd_any(const NormParams& p, bool fp8, cudaStream_t s) {
    const Shape h = shape_of(p);
    KernelTimer kt("rmsnorm_fwd", s);
    if (fp8)
        rmsnorm_fwd_any_kernel<T, CH, true><<<h.grid, h.block, 0, s>>>(p);
    else
        rmsnorm_fwd_any_kernel<T, CH, false><<<h.grid, h.block, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_fwd(NormParams p, bool fp8, bool wide, cudaStream_t s) {
    // About as many pieces per thread as registers hold, and fewer where there are too
    // few rows to fill the GPU.
    const int64_t full = (int64_t)sm_count() * 1024;
    if (!wide) {
        int ch = p.D > 32 * kMaxThreads ? 64 : p.D > 8 * kMaxThreads ? 32 : 8;
        if (p.D <= 2 * kMaxThreads && (p.D <= 64 || p.M * row_threads(p.D, 8, 32) < full)) ch = 2;
        p.tpr = row_threads(p.D, ch, 32);
        switch (ch) {
            case 2: return launch_fwd_any<T, 2>(p, fp8, s);
            case 8: return launch_fwd_any<T, 8>(p, fp8, s);
            case 32: return launch_fwd_any<T, 32>(p, fp8, s);
            default: return launch_fwd_any<T, 64>(p, fp8, s);
        }
    }
    const int pieces = p.D / 8;
    int ch = 8;
    while (ch > 1 && row_threads(pieces, ch / 2, 16) * (ch / 2) >= pieces &&
           (row_threads(pieces, ch, 16) == row_threads(pieces, ch / 2, 16) ||
            p.M * row_threads(pieces, ch, 16) < full))
        ch /= 2;
    p.tpr = row_threads(pieces, ch, 16);
    switch (ch) {
        case 1: return launch_fwd_ch<T, 1>(p, fp8, s);
        case 2: return launch_fwd_ch<T, 2>(p, fp8, s);
        case 4: return launch_fwd_ch<T, 4>(p, fp8, s);
        default: return launch_fwd_ch<T, 8>(p, fp8, s);
    }
}

// ---- backward ----------------------------------------------------------------

struct NormBwdParams {
    const void* dy;
    const void* s;
    const float* w;
    const void* ds;
    void* dx;
    float* dw;
    float* partial;  // [parts, D]: dw summed over each CTA's rows
    int64_t lddy, lds, ldds, lddx, M;
    int D, parts, tpr, stages;
    float eps;
    unsigned int* err;
    int64_t lost;  // LOSE only: the row whose copies are not to complete
};

constexpr unsigned kNormError = 0x400;  // device error word: a row's copies did not land
constexpr int kMaxStages = 8;
constexpr int kMaxParts = 608;  // CTAs of the backward: four per SM

int norm_parts(int64_t M) { return (int)(M < kMaxParts ? M : kMaxParts); }

// Rows are walked by the CTAs of one grid, so that a thread meets the same
// columns in every row and sums dw in registers; one [D] part per CTA goes to
// memory.
template <typename T, int CH>
__global__ void __launch_bounds__(kMaxThreads, CH <= 2 ? 2 : 1) rmsnorm_bwd_kernel(NormBwdParams p) {
    __shared__ float2 exchange[2][kMaxThreads / 32];
    extern __shared__ float dw_s[];
    const int tpr = p.tpr, slots = blockDim.x / tpr, slot = threadIdx.x / tpr, l = threadIdx.x % tpr;
    RowReduce reduce{exchange, tpr, slot, 0};
    const float mean = 1.f / p.D;
    float2 dw[CH][4];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[c][i] = both(0.f);
    for (int64_t m0 = (int64_t)blockIdx.x * slots; m0 < p.M; m0 += (int64_t)gridDim.x * slots) {
        const int64_t m = m0 + slot;
        const int width = m < p.M ? p.D : 0;  // a missing row has no elements
        const T* dy_row = static_cast<const T*>(p.dy) + m * p.lddy;
        const T* s_row = static_cast<const T*>(p.s) + m * p.lds;
        const T* ds_row = p.ds ? static_cast<const T*>(p.ds) + m * p.ldds : nullptr;
        T* dx_row = static_cast<T*>(p.dx) + m * p.lddx;
        Cells<T> dy[CH], s[CH], ds[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * tpr + l) * 8;
            dy[c].zero();
            s[c].zero();
            ds[c].zero();
            if (e < width) {
                dy[c].load(dy_row + e);
                s[c].load(s_row + e);
                if (ds_row) ds[c].load(ds_row + e);
            }
        }
        float2 square = both(0.f), dot = both(0.f);  // sums of s^2 and of s z
        auto weight = [&](int c) {
            const int e = (c * tpr + l) * 8;
            Cells<float> w;
            w.zero();
            if (e < p.D) w.load(p.w + e);
            return w;
        };
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const Cells<float> w = weight(c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = s[c].get(i);
                square = __ffma2_rn(v, v, square);
                dot = __ffma2_rn(v, __fmul2_rn(dy[c].get(i), w.get(i)), dot);
            }
        }
        const float2 sums = reduce.sum(make_float2(square.x + square.y, dot.x + dot.y));
        float rstd = 1.f / sqrtf(fmaf(sums.x, mean, p.eps));
        if (!width) rstd = 0.f;  // with eps = 0 a missing row's would be infinite, and reach dw as NaN
        const float proj = sums.y * mean * rstd * rstd;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * tpr + l) * 8;
            const Cells<float> w = weight(c);
            Cells<T> out;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 d = dy[c].get(i), v = s[c].get(i);
                const float2 t = __ffma2_rn(d, w.get(i), __fmul2_rn(v, both(-proj)));
                out.set(i, __ffma2_rn(both(rstd), t, ds[c].get(i)));
                dw[c][i] = __ffma2_rn(d, __fmul2_rn(v, both(rstd)), dw[c][i]);
            }
            if (e < width) out.store(dx_row + e);
        }
    }
    if (!p.dw) return;
    // the CTA's rows at once: slot after slot
    float2* dw2 = reinterpret_cast<float2*>(dw_s);
    for (int k = 0; k < slots; ++k) {
        if (slot == k)
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int e = (c * tpr + l) * 8;
                if (k > 0)
#pragma unroll
                    for (int i = 0; i < 4; ++i) dw[c][i] = __fadd2_rn(dw2[e / 2 + i], dw[c][i]);
                if (k + 1 < slots) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) dw2[e / 2 + i] = dw[c][i];
                } else if (e < p.D) {
                    Cells<float> out;
#pragma unroll
                    for (int i = 0; i < 4; ++i) out.set(i, dw[c][i]);
                    out.store(p.partial + (int64_t)blockIdx.x * p.D + e);
                }
            }
        __syncthreads();
    }
}

// The same for rows of 512 elements and more, whose rows (dy, s, d_residual) come
// through a ring of `stages` rows in shared memory per row's threads (32 or more),
// filled by bulk copies: the next rows are on their way while one is reduced
// (16384 x 4096 bf16: 110 us from registers, 90 us through the ring).  A row whose
// copies do not land ends its threads' rows: that row and the later ones stay
// unwritten, and the CTA's part of dw is NaN.  LOSE: row p.lost waits for 16 bytes that
// nobody copies, for the test of that.
template <typename T, int CH, int MAX_THREADS, int MIN_CTAS, bool LOSE>
__global__ void __launch_bounds__(MAX_THREADS, MIN_CTAS) rmsnorm_bwd_ring_kernel(NormBwdParams p) {
    __shared__ float2 exchange[2][kMaxThreads / 32];
    __shared__ uint64_t full_s[kMaxThreads / 32][kMaxStages];
    __shared__ int never, lost_s[kMaxThreads / 32];  // per row's threads: the step that lost its copies
    extern __shared__ __align__(128) unsigned char ring[];
    const int tpr = p.tpr, slots = blockDim.x / tpr, slot = threadIdx.x / tpr, l = threadIdx.x % tpr;
    RowReduce reduce{exchange, tpr, slot, 0};
    const float mean = 1.f / p.D;
    const uint32_t row_bytes = p.D * (uint32_t)sizeof(T), rows = p.ds ? 3 : 2;
    const uint32_t own = tc::smem_u32(ring) + slot * p.stages * rows * row_bytes;
    const uint32_t full = tc::smem_u32(full_s[slot]);
    const int64_t stride = (int64_t)gridDim.x * slots;
    auto request = [&](int stage, int64_t m) {  // one thread of the row's
        const uint32_t at = own + stage * rows * row_bytes, bar = full + stage * 8;
        tc::mbar_arrive_tx(bar, rows * row_bytes + (LOSE && m == p.lost ? 16 : 0));
        tc::bulk_g2s(at, static_cast<const T*>(p.dy) + m * p.lddy, row_bytes, bar);
        tc::bulk_g2s(at + row_bytes, static_cast<const T*>(p.s) + m * p.lds, row_bytes, bar);
        if (p.ds) tc::bulk_g2s(at + 2 * row_bytes, static_cast<const T*>(p.ds) + m * p.ldds, row_bytes, bar);
    };
    const int64_t first = (int64_t)blockIdx.x * slots + slot;
    if (l == 0) {
        never = 0;
        lost_s[slot] = 0x7fffffff;
        for (int k = 0; k < p.stages; ++k) tc::mbar_init(full + k * 8, 1);
        tc::mbar_fence_init();
        for (int k = 0; k < p.stages; ++k)
            if (first + k * stride < p.M) request(k, first + k * stride);
    }
    float2 dw[CH][4];
    Cells<float> w[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int e = (c * tpr + l) * 8;
        w[c].zero();
        if (e < p.D) w[c].load(p.w + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[c][i] = both(0.f);
    }
    __syncthreads();
    volatile int* lost_at = lost_s + slot;
    int stage = 0, parity = 0, step = 0;
    bool lost = false;
    for (int64_t m = first; m < p.M; m += stride, ++step) {
        if (!tc::mbar_wait(full + stage * 8, parity, &never)) {
            *lost_at = step;
            atomicOr(p.err, kNormError);
        }
        const unsigned char* at = ring + (own - tc::smem_u32(ring)) + stage * rows * row_bytes;
        Cells<T> dy[CH], s[CH], ds[CH];
        float2 square = both(0.f), dot = both(0.f);  // sums of s^2 and of s z
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * tpr + l) * 8;
            dy[c].zero();
            s[c].zero();
            ds[c].zero();
            if (e < p.D) {
                dy[c].load(reinterpret_cast<const T*>(at) + e);
                s[c].load(reinterpret_cast<const T*>(at + row_bytes) + e);
                if (p.ds) ds[c].load(reinterpret_cast<const T*>(at + 2 * row_bytes) + e);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = s[c].get(i);
                square = __ffma2_rn(v, v, square);
                dot = __ffma2_rn(v, __fmul2_rn(dy[c].get(i), w[c].get(i)), dot);
            }
        }
        const float2 sums = reduce.sum(make_float2(square.x + square.y, dot.x + dot.y));
        if (tpr == 32) __syncwarp();
        // one thread's wait may run out where another's did not: all have met since
        if (*lost_at <= step) {
            lost = true;
            if (l == 0)  // none of the copies on their way may land behind this
                for (int k = 0; k < p.stages && m + k * stride < p.M; ++k) {
                    tc::mbar_wait_copies(full + stage * 8, parity);
                    if (++stage == p.stages) {
                        stage = 0;
                        parity ^= 1;
                    }
                }
            break;
        }
        if (l == 0 && m + p.stages * stride < p.M) request(stage, m + p.stages * stride);  // read by all
        if (++stage == p.stages) {
            stage = 0;
            parity ^= 1;
        }
        const float rstd = 1.f / sqrtf(fmaf(sums.x, mean, p.eps)), proj = sums.y * mean * rstd * rstd;
        T* dx_row = static_cast<T*>(p.dx) + m * p.lddx;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = (c * tpr + l) * 8;
            Cells<T> out;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 d = dy[c].get(i), v = s[c].get(i);
                const float2 t = __ffma2_rn(d, w[c].get(i), __fmul2_rn(v, both(-proj)));
                out.set(i, __ffma2_rn(both(rstd), t, ds[c].get(i)));
                dw[c][i] = __ffma2_rn(d, __fmul2_rn(v, both(rstd)), dw[c][i]);
            }
            if (e < p.D) out.store(dx_row + e);
        }
    }
    if (!p.dw) return;
    if (lost)
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) dw[c][i] = both(NAN);
    __syncthreads();  // the ring becomes the place of the sums
    float2* dw2 = reinterpret_cast<float2*>(ring);
    for (int k = 0; k < slots; ++k) {
        if (slot == k)
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int e = (c * tpr + l) * 8;
                if (k > 0)
#pragma unroll
                    for (int i = 0; i < 4; ++i) dw[c][i] = __fadd2_rn(dw2[e / 2 + i], dw[c][i]);
                if (k + 1 < slots) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) dw2[e / 2 + i] = dw[c][i];
                } else if (e < p.D) {
                    Cells<float> out;
#pragma unroll
                    for (int i = 0; i < 4; ++i) out.set(i, dw[c][i]);
                    out.store(p.partial + (int64_t)blockIdx.x * p.D + e);
                }
            }
        __syncthreads();
    }
}

// The same on any rows: one element at a time.
template <typename T, int CH>
__global__ void __launch_bounds__(kMaxThreads, CH <= 8 ? 2 : 1) rmsnorm_bwd_any_kernel(NormBwdParams p) {
    __shared__ float2 exchange[2][kMaxThreads / 32];
    extern __shared__ float dw_s[];
    const int tpr = p.tpr, slots = blockDim.x / tpr, slot = threadIdx.x / tpr, l = threadIdx.x % tpr;
    RowReduce reduce{exchange, tpr, slot, 0};
    const float mean = 1.f / p.D;
    float dw[CH], w[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        dw[c] = 0.f;
        w[c] = c * tpr + l < p.D ? p.w[c * tpr + l] : 0.f;
    }
    for (int64_t m0 = (int64_t)blockIdx.x * slots; m0 < p.M; m0 += (int64_t)gridDim.x * slots) {
        const int64_t m = m0 + slot;
        const int width = m < p.M ? p.D : 0;
        const T* dy_row = static_cast<const T*>(p.dy) + m * p.lddy;
        const T* s_row = static_cast<const T*>(p.s) + m * p.lds;
        const T* ds_row = p.ds ? static_cast<const T*>(p.ds) + m * p.ldds : nullptr;
        T* dx_row = static_cast<T*>(p.dx) + m * p.lddx;
        T dy[CH], s[CH], ds[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = c * tpr + l;
            dy[c] = e < width ? dy_row[e] : from_f<T>(0.f);
            s[c] = e < width ? s_row[e] : from_f<T>(0.f);
            ds[c] = e < width && ds_row ? ds_row[e] : from_f<T>(0.f);
        }
        float2 sums = both(0.f);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const float v = to_f(s[c]);
            sums.x = fmaf(v, v, sums.x);
            sums.y = fmaf(v, __fmul_rn(to_f(dy[c]), w[c]), sums.y);
        }
        sums = reduce.sum(sums);
        float rstd = 1.f / sqrtf(fmaf(sums.x, mean, p.eps));
        if (!width) rstd = 0.f;
        const float proj = sums.y * mean * rstd * rstd;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = c * tpr + l;
            const float d = to_f(dy[c]), v = to_f(s[c]);
            const float o = fmaf(rstd, fmaf(d, w[c], __fmul_rn(v, -proj)), to_f(ds[c]));
            dw[c] = fmaf(d, __fmul_rn(v, rstd), dw[c]);
            if (e < width) dx_row[e] = from_f<T>(o);
        }
    }
    if (!p.dw) return;
    for (int k = 0; k < slots; ++k) {
        if (slot == k)
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int e = c * tpr + l;
                if (k > 0) dw[c] = dw_s[e] + dw[c];
                if (k + 1 < slots)
                    dw_s[e] = dw[c];
                else if (e < p.D)
                    p.partial[(int64_t)blockIdx.x * p.D + e] = dw[c];
            }
        __syncthreads();
    }
}

// The sum of the parts: 32 columns per CTA, 16 slices of the parts, in a fixed order.
__global__ void rmsnorm_dw_kernel(const float* __restrict__ partial, int parts, int D, float* dw) {
    __shared__ float slice[16][33];
    tc::grid_dep_wait();
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), q = threadIdx.x >> 5;
    float v = 0.f;
    if (c < D) {
#pragma unroll 8
        for (int i = q; i < parts; i += 16) v += partial[(int64_t)i * D + c];
    }
    slice[q][threadIdx.x & 31] = v;
    __syncthreads();
    if (q == 0 && c < D) {
        for (int i = 1; i < 16; ++i) v += slice[i][threadIdx.x];
        dw[c] = v;
    }
}

// A single part is written as dw itself.
void place_parts(NormBwdParams& p) {
    if (p.parts == 1) p.partial = p.dw;
}

cudaError_t launch_dw(const NormBwdParams& p, cudaStream_t s) {
    if (p.parts == 1) return cudaSuccess;
    KernelTimer kt("rmsnorm_dw", s);
    return launch_dependent(rmsnorm_dw_kernel, dim3((p.D + 31) / 32), dim3(512), 0, s, p.partial, p.parts, p.D, p.dw);
}

template <typename T, int CH, bool WIDE>
cudaError_t launch_bwd_ch(NormBwdParams p, cudaStream_t s) {
    const int block = p.tpr > 256 ? p.tpr : 256, slots = block / p.tpr;
    const int64_t want = (p.M + slots - 1) / slots;
    p.parts = norm_parts(want);
    place_parts(p);
    const size_t smem = slots > 1 ? (size_t)p.tpr * CH * (WIDE ? 8 : 1) * sizeof(float) : 0;
    {
        KernelTimer kt("rmsnorm_bwd", s);
        if constexpr (WIDE)
            rmsnorm_bwd_kernel<T, CH><<<p.parts, block, smem, s>>>(p);
        else
            rmsnorm_bwd_any_kernel<T, CH><<<p.parts, block, smem, s>>>(p);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess && p.dw ? launch_dw(p, s) : e;
}

// CTAS CTAs per SM; the ring takes their share of its 227 KB.
template <typename T, int CH, int THREADS, int CTAS, bool LOSE = false>
cudaError_t launch_bwd_ring(NormBwdParams p, cudaStream_t s) {
    auto kernel = rmsnorm_bwd_ring_kernel<T, CH, THREADS, CTAS, LOSE>;
    constexpr int kShare = 227 * 1024 / CTAS - 2048;
    const int slots = THREADS / p.tpr, stage = slots * 3 * p.D * (int)sizeof(T);
    p.stages = kShare / stage < kMaxStages ? kShare / stage : kMaxStages;
    // at every call: the attribute belongs to the context
    const cudaError_t set = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kShare);
    if (set != cudaSuccess) return set;
    p.err = device_error_word();
    if (!p.err) return cudaErrorInitializationError;
    const int64_t want = (p.M + slots - 1) / slots, most = (int64_t)CTAS * sm_count();
    p.parts = norm_parts(want < most ? want : most);
    place_parts(p);
    {
        KernelTimer kt("rmsnorm_bwd", s);
        kernel<<<p.parts, THREADS, p.stages * stage, s>>>(p);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess && p.dw ? launch_dw(p, s) : e;
}

template <typename T>
cudaError_t launch_bwd(NormBwdParams p, bool wide, cudaStream_t s) {
    if (wide && p.D >= 512 && p.D * sizeof(T) <= 32768) {
        const int pieces = p.D / 8;
        if (pieces <= 512) {
            p.tpr = row_threads(pieces, 2, 32);
            return launch_bwd_ring<T, 2, 256, 2>(p, s);
        }
        if (pieces <= 1024) {
            p.tpr = 512;
            return launch_bwd_ring<T, 2, 512, 1>(p, s);
        }
        if constexpr (sizeof(T) == 2) {  // 32768 bytes of fp32 are 1024 pieces already
            p.tpr = 512;
            return launch_bwd_ring<T, 4, 512, 1>(p, s);
        }
    }
    if (!wide) {
        const int ch = p.D <= 4 * kMaxThreads ? 4 : p.D <= 16 * kMaxThreads ? 16 : 64;
        p.tpr = row_threads(p.D, ch, 32);
        return ch == 4 ? launch_bwd_ch<T, 4, false>(p, s) : ch == 16 ? launch_bwd_ch<T, 16, false>(p, s)
                                                                     : launch_bwd_ch<T, 64, false>(p, s);
    }
    // narrow rows, and those of which the ring does not hold two
    const int pieces = p.D / 8, ch = pieces <= 16 ? 1 : pieces <= 64 ? 2 : 8;
    p.tpr = row_threads(pieces, ch, 16);
    return ch == 1 ? launch_bwd_ch<T, 1, true>(p, s) : ch == 2 ? launch_bwd_ch<T, 2, true>(p, s)
                                                               : launch_bwd_ch<T, 8, true>(p, s);
}

// Rows of 8 aligned elements of `esize` bytes (16-byte vectors; codes: 8).
bool wide_rows(const void* p, int64_t ld, int esize) {
    return (reinterpret_cast<uintptr_t>(p) & (esize == 1 ? 7u : 15u)) == 0 && ld % 8 == 0;
}

// ---- argument checks -----------------------------------------------------------

int check_sizes(int64_t M, int D, float eps, int dtype) {
    if (M < 0 || D <= 0) return set_last_error(GDR_ERR_INVALID_ARG, "bad M (%lld) or D (%d)", (long long)M, D);
    if (D > GDR_RMSNORM_MAX_D) return set_last_error(GDR_ERR_UNSUPPORTED, "D (%d) above %d", D, GDR_RMSNORM_MAX_D);
    if (dtype != GDR_BF16 && dtype != GDR_F32) return set_last_error(GDR_ERR_UNSUPPORTED, "dtype %d", dtype);
    if (!(eps >= 0.f)) return set_last_error(GDR_ERR_INVALID_ARG, "eps must be >= 0");
    return GDR_OK;
}

int check_floats(const char* name, const void* p) {
    if (!p) return set_last_error(GDR_ERR_INVALID_ARG, "null pointer argument (%s)", name);
    return check_aligned16(name, p);
}

// One tensor on another: the same pointer and stride, or neither.
int check_in_place(const char* name, const void* p, int64_t ld, const char* other, const void* q, int64_t ldq, int64_t M) {
    if (p == q && ld != ldq && M > 1)
        return set_last_error(GDR_ERR_INVALID_ARG, "%s is %s with another row stride", name, other);
    return GDR_OK;
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

int gdr_rmsnorm_fwd(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                    const float* weight, int64_t M, int D, float eps, int dtype, void* residual_out,
                    int64_t residual_out_stride, void* y, int64_t y_stride, int y_dtype, float* scales,
                    int scale_group, gdr_stream_t stream) {
    if (int rc = check_sizes(M, D, eps, dtype)) return rc;
    if (y_dtype != dtype && y_dtype != GDR_E4M3)
        return set_last_error(GDR_ERR_UNSUPPORTED, "y_dtype %d with dtype %d", y_dtype, dtype);
    if ((residual == nullptr) != (residual_out == nullptr))
        return set_last_error(GDR_ERR_INVALID_ARG, "residual and residual_out go together");
    const bool fp8 = y_dtype == GDR_E4M3;
    if (fp8 ? (scale_group != 0 && scale_group != 32 && scale_group != 64 && scale_group != 128) : scale_group != 0)
        return set_last_error(GDR_ERR_INVALID_ARG, "scale_group %d", scale_group);
    if (!fp8 && scales) return set_last_error(GDR_ERR_INVALID_ARG, "scales are GDR_E4M3's only");
    if (M == 0) return set_ok();
    const unsigned esize = dtype == GDR_BF16 ? 2 : 4;
    if (int rc = check_rows("x", x, x_stride, 0, esize)) return rc;
    if (residual) {
        if (int rc = check_rows("residual", residual, residual_stride, 0, esize)) return rc;
        if (int rc = check_rows("residual_out", residual_out, residual_out_stride, D, esize)) return rc;
        if (int rc = check_in_place("residual_out", residual_out, residual_out_stride, "residual", residual, residual_stride, M))
            return rc;
        if (int rc = check_in_place("residual_out", residual_out, residual_out_stride, "x", x, x_stride, M)) return rc;
    }
    if (int rc = check_rows("y", y, y_stride, D, fp8 ? 1 : esize)) return rc;
    if (int rc = check_floats("weight", weight)) return rc;
    if (fp8)
        if (int rc = check_floats("scales", scales)) return rc;
    if (int rc = check_device()) return rc;
    NormParams p{};
    p.x = x; p.residual = residual; p.w = weight; p.sum = residual_out; p.y = y; p.scales = scales;
    p.ldx = x_stride; p.ldr = residual_stride; p.lds = residual_out_stride; p.ldy = y_stride; p.M = M; p.D = D;
    p.group = fp8 ? (scale_group ? scale_group : D) : 1;
    p.groups = fp8 ? (D + p.group - 1) / p.group : 0;
    p.eps = eps;
    cudaStream_t s = (cudaStream_t)stream;
    const bool wide = D % 8 == 0 && wide_rows(x, x_stride, esize) && wide_rows(y, y_stride, fp8 ? 1 : esize) &&
                      (!residual || (wide_rows(residual, residual_stride, esize) &&
                                     wide_rows(residual_out, residual_out_stride, esize)));
    return launch_result(dtype == GDR_BF16 ? launch_fwd<__nv_bfloat16>(p, fp8, wide, s) : launch_fwd<float>(p, fp8, wide, s),
                    "gdr_rmsnorm_fwd launch");
}

int gdr_rmsnorm_bwd_workspace_size(int64_t M, int D, size_t* bytes) {
    if (!bytes) return set_last_error(GDR_ERR_INVALID_ARG, "bytes is NULL");
    if (int rc = check_sizes(M, D, 0.f, GDR_F32)) return rc;
    *bytes = ((size_t)norm_parts(M) * D * sizeof(float) + 255) / 256 * 256;
    return set_ok();
}

int gdr_rmsnorm_bwd(const void* dy, int64_t dy_stride, const void* s, int64_t s_stride, const float* weight,
                    const void* d_residual_out, int64_t d_residual_out_stride, int64_t M, int D, float eps, int dtype,
                    void* dx, int64_t dx_stride, float* dweight, void* workspace, size_t ws_bytes,
                    gdr_stream_t stream) {
    if (int rc = check_sizes(M, D, eps, dtype)) return rc;
    cudaStream_t st = (cudaStream_t)stream;
    if (dweight)
        if (int rc = check_floats("dweight", dweight)) return rc;
    if (M == 0) {
        if (!dweight) return set_ok();
        if (int rc = check_device()) return rc;
        return launch_result(cudaMemsetAsync(dweight, 0, sizeof(float) * (size_t)D, st), "gdr_rmsnorm_bwd launch");
    }
    const unsigned esize = dtype == GDR_BF16 ? 2 : 4;
    if (int rc = check_rows("dy", dy, dy_stride, 0, esize)) return rc;
    if (int rc = check_rows("s", s, s_stride, 0, esize)) return rc;
    if (d_residual_out)
        if (int rc = check_rows("d_residual_out", d_residual_out, d_residual_out_stride, 0, esize)) return rc;
    if (int rc = check_rows("dx", dx, dx_stride, D, esize)) return rc;
    if (int rc = check_in_place("dx", dx, dx_stride, "dy", dy, dy_stride, M)) return rc;
    if (int rc = check_in_place("dx", dx, dx_stride, "d_residual_out", d_residual_out, d_residual_out_stride, M)) return rc;
    if (int rc = check_floats("weight", weight)) return rc;
    if (dweight) {
        size_t need = 0;
        if (int rc = gdr_rmsnorm_bwd_workspace_size(M, D, &need)) return rc;
        if (!workspace || ws_bytes < need)
            return set_last_error(GDR_ERR_WORKSPACE, "workspace %zu bytes < required %zu",
                                  workspace ? ws_bytes : (size_t)0, need);
        if (reinterpret_cast<uintptr_t>(workspace) & 255u)
            return set_last_error(GDR_ERR_INVALID_ARG, "workspace not 256-byte aligned");
    }
    if (int rc = check_device()) return rc;
    NormBwdParams p{};
    p.dy = dy; p.s = s; p.w = weight; p.ds = d_residual_out; p.dx = dx; p.dw = dweight;
    p.partial = static_cast<float*>(workspace);
    p.lddy = dy_stride; p.lds = s_stride; p.ldds = d_residual_out_stride; p.lddx = dx_stride;
    p.M = M; p.D = D; p.eps = eps;
    const bool wide = D % 8 == 0 && wide_rows(dy, dy_stride, esize) && wide_rows(s, s_stride, esize) &&
                      wide_rows(dx, dx_stride, esize) &&
                      (!d_residual_out || wide_rows(d_residual_out, d_residual_out_stride, esize));
    return launch_result(dtype == GDR_BF16 ? launch_bwd<__nv_bfloat16>(p, wide, st) : launch_bwd<float>(p, wide, st),
                    "gdr_rmsnorm_bwd launch");
}

int gdr_selftest_rmsnorm_lost_copy(const void* dy, const void* s, const float* weight, int64_t M, int D,
                                   int64_t lost_row, void* dx, float* dweight, void* workspace, size_t ws_bytes,
                                   gdr_stream_t stream) {
    if (int rc = check_sizes(M, D, 1e-6f, GDR_BF16)) return rc;
    if (D % 8 || D < 512 || D > 4096) return set_last_error(GDR_ERR_UNSUPPORTED, "D %d", D);
    if (M == 0) return set_ok();
    const void* all[] = {dy, s, weight, dx, dweight};
    for (const void* p : all)
        if (int rc = check_floats("tensor", p)) return rc;
    size_t need = 0;
    if (int rc = gdr_rmsnorm_bwd_workspace_size(M, D, &need)) return rc;
    if (!workspace || ws_bytes < need) return set_last_error(GDR_ERR_WORKSPACE, "workspace too small");
    if (int rc = check_device()) return rc;
    NormBwdParams p{};
    p.dy = dy; p.s = s; p.w = weight; p.dx = dx; p.dw = dweight;
    p.partial = static_cast<float*>(workspace);
    p.lddy = p.lds = p.lddx = D;
    p.M = M; p.D = D; p.eps = 1e-6f; p.lost = lost_row;
    p.tpr = row_threads(D / 8, 2, 32);
    return launch_result(launch_bwd_ring<__nv_bfloat16, 2, 256, 2, true>(p, (cudaStream_t)stream),
                         "gdr_selftest_rmsnorm_lost_copy launch");
}

}  // extern "C"
