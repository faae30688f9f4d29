// Root-mean-square norm with the residual's addition (output in the input's
// type or e4m3 with scales) and its backward, with their C entry points
// (contract in include/gdr.h).
#include <cuda_fp8.h>
#include <math.h>

#include "common.cuh"
#include "gdr.h"
#include "launch.h"

namespace gdr {
namespace {

constexpr float kE4m3Max = 448.f;    // largest finite e4m3 value
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
    float eps;
};

__device__ __forceinline__ float block_sum(float v, float* shared) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    v = threadIdx.x < (blockDim.x >> 5) ? shared[threadIdx.x] : 0.f;
    if (threadIdx.x < 32) {
        v = warp_sum(v);
        if (threadIdx.x == 0) shared[32] = v;
    }
    __syncthreads();
    return shared[32];
}

template <typename T, bool FP8>
__global__ void rmsnorm_row_kernel(NormParams p) {
    __shared__ float shared[33];
    __shared__ int amax[GDR_RMSNORM_MAX_D / 32];
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        const T* x = static_cast<const T*>(p.x) + m * p.ldx;
        const T* r = p.residual ? static_cast<const T*>(p.residual) + m * p.ldr : nullptr;
        T* sum = p.residual ? static_cast<T*>(p.sum) + m * p.lds : nullptr;
        const T* s = sum ? sum : x;
        float ss = 0.f;
        for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
            float v = to_f(x[c]);
            if (r) {
                const T q = from_f<T>(v + to_f(r[c]));
                sum[c] = q;
                v = to_f(q);
            }
            ss += v * v;
        }
        if (FP8)
            for (int i = threadIdx.x; i < p.groups; i += blockDim.x) amax[i] = 0;
        const float rstd = 1.f / sqrtf(block_sum(ss, shared) / p.D + p.eps);
        if (!FP8) {
            T* y = static_cast<T*>(p.y) + m * p.ldy;
            for (int c = threadIdx.x; c < p.D; c += blockDim.x) y[c] = from_f<T>(to_f(s[c]) * rstd * p.w[c]);
        } else {
            for (int c = threadIdx.x; c < p.D; c += blockDim.x)
                atomicMax(&amax[c / p.group], __float_as_int(fmaxf(fabsf(to_f(s[c]) * rstd * p.w[c]), kAmaxFloor)));
            __syncthreads();
            __nv_fp8_storage_t* y = static_cast<__nv_fp8_storage_t*>(p.y) + m * p.ldy;
            for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
                const float scale = __int_as_float(amax[c / p.group]) / kE4m3Max;
                y[c] = __nv_cvt_float_to_fp8(to_f(s[c]) * rstd * p.w[c] / scale, __NV_SATFINITE, __NV_E4M3);
            }
            for (int i = threadIdx.x; i < p.groups; i += blockDim.x)
                p.scales[m * p.groups + i] = __int_as_float(amax[i]) / kE4m3Max;
            __syncthreads();
        }
    }
}

template <typename T>
cudaError_t launch_fwd(const NormParams& p, bool fp8, cudaStream_t s) {
    const unsigned grid = (unsigned)(p.M < 65535 ? p.M : 65535);
    KernelTimer kt("rmsnorm_fwd", s);
    if (fp8)
        rmsnorm_row_kernel<T, true><<<grid, 256, 0, s>>>(p);
    else
        rmsnorm_row_kernel<T, false><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
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
    int D, parts;
    float eps;
};

constexpr int kMaxParts = 304;

int norm_parts(int64_t M) { return (int)(M < kMaxParts ? M : kMaxParts); }

template <typename T>
__global__ void rmsnorm_bwd_kernel(NormBwdParams p) {
    __shared__ float shared[33];
    if (p.dw)
        for (int c = threadIdx.x; c < p.D; c += blockDim.x) p.partial[(int64_t)blockIdx.x * p.D + c] = 0.f;
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        const T* dy = static_cast<const T*>(p.dy) + m * p.lddy;
        const T* s = static_cast<const T*>(p.s) + m * p.lds;
        const T* ds = p.ds ? static_cast<const T*>(p.ds) + m * p.ldds : nullptr;
        T* dx = static_cast<T*>(p.dx) + m * p.lddx;
        float ss = 0.f, sz = 0.f;
        for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
            const float v = to_f(s[c]);
            ss += v * v;
            sz += v * to_f(dy[c]) * p.w[c];
        }
        const float rstd = 1.f / sqrtf(block_sum(ss, shared) / p.D + p.eps);
        const float proj = block_sum(sz, shared) * rstd * rstd / p.D;
        for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
            const float v = to_f(s[c]), d = to_f(dy[c]);
            // one rounding each, written out: the same bits with and without dw
            const float out = fmaf(rstd, fmaf(d, p.w[c], -__fmul_rn(v, proj)), ds ? to_f(ds[c]) : 0.f);
            if (p.dw) p.partial[(int64_t)blockIdx.x * p.D + c] += rstd * d * v;
            dx[c] = from_f<T>(out);
        }
    }
}

__global__ void rmsnorm_dw_kernel(const float* partial, int parts, int D, float* dw) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= D) return;
    float v = 0.f;
    for (int i = 0; i < parts; ++i) v += partial[(int64_t)i * D + c];
    dw[c] = v;
}

template <typename T>
cudaError_t launch_bwd(const NormBwdParams& p, cudaStream_t s) {
    {
        KernelTimer kt("rmsnorm_bwd", s);
        rmsnorm_bwd_kernel<T><<<p.parts, 256, 0, s>>>(p);
    }
    if (p.dw) {
        KernelTimer kt("rmsnorm_dw", s);
        rmsnorm_dw_kernel<<<(p.D + 127) / 128, 128, 0, s>>>(p.partial, p.parts, p.D, p.dw);
    }
    return cudaGetLastError();
}

// ---- argument checks -----------------------------------------------------------

int check_sizes(int64_t M, int D, float eps, int dtype) {
    if (M < 0 || D <= 0) return set_last_error(GDR_ERR_INVALID_ARG, "bad M (%lld) or D (%d)", (long long)M, D);
    if (D > GDR_RMSNORM_MAX_D) return set_last_error(GDR_ERR_UNSUPPORTED, "D (%d) above %d", D, GDR_RMSNORM_MAX_D);
    if (dtype != GDR_BF16 && dtype != GDR_F32) return set_last_error(GDR_ERR_UNSUPPORTED, "dtype %d", dtype);
    if (!(eps >= 0.f)) return set_last_error(GDR_ERR_INVALID_ARG, "eps must be >= 0");
    return GDR_OK;
}

int check_rows(const char* name, const void* p, int64_t stride, int64_t least, unsigned esize) {
    if (!p) return set_last_error(GDR_ERR_INVALID_ARG, "null pointer argument (%s)", name);
    if (reinterpret_cast<uintptr_t>(p) & (esize - 1))
        return set_last_error(GDR_ERR_INVALID_ARG, "%s not aligned to its element", name);
    if (stride < least)
        return set_last_error(GDR_ERR_INVALID_ARG, "%s: row stride %lld too small", name, (long long)stride);
    return GDR_OK;
}

int check_floats(const char* name, const void* p) {
    if (!p) return set_last_error(GDR_ERR_INVALID_ARG, "null pointer argument (%s)", name);
    if (reinterpret_cast<uintptr_t>(p) & 15u)
        return set_last_error(GDR_ERR_INVALID_ARG, "%s not 16-byte aligned", name);
    return GDR_OK;
}

int launched(cudaError_t e, const char* what) {
    if (e != cudaSuccess) return set_last_error(GDR_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
    return set_ok();
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
    return launched(dtype == GDR_BF16 ? launch_fwd<__nv_bfloat16>(p, fp8, s) : launch_fwd<float>(p, fp8, s),
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
        return launched(cudaMemsetAsync(dweight, 0, sizeof(float) * (size_t)D, st), "gdr_rmsnorm_bwd launch");
    }
    const unsigned esize = dtype == GDR_BF16 ? 2 : 4;
    if (int rc = check_rows("dy", dy, dy_stride, 0, esize)) return rc;
    if (int rc = check_rows("s", s, s_stride, 0, esize)) return rc;
    if (d_residual_out)
        if (int rc = check_rows("d_residual_out", d_residual_out, d_residual_out_stride, 0, esize)) return rc;
    if (int rc = check_rows("dx", dx, dx_stride, D, esize)) return rc;
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
    p.M = M; p.D = D; p.parts = norm_parts(M); p.eps = eps;
    return launched(dtype == GDR_BF16 ? launch_bwd<__nv_bfloat16>(p, st) : launch_bwd<float>(p, st),
                    "gdr_rmsnorm_bwd launch");
}

}  // extern "C"
