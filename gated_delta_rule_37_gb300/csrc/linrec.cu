// The gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t over packed
// sequences: forward, backward and the slot-pool step, with their C entry
// points (contract in include/gdr.h).
#include <math.h>

#include "common.cuh"
#include "gdr.h"
#include "launch.h"

namespace gdr {
namespace {

struct LinrecParams {
    const void* x;   // forward: x; backward: dy
    const void* g;
    const void* h;   // backward: y, the forward's output
    void* out;       // forward: y; backward: dx
    void* dg;
    const float* h0;
    const float* start;  // state before the scan's first token: h0, or the final state's gradient
    float* last;         // state after its last: the final state, or the initial state's gradient
    const int32_t* cu;
    int64_t ldx, ldg, ldh, ldo, lddg;
    int64_t T;
    int N, D;
};

// One thread per (sequence, channel), token after token.
template <typename TX, typename TG, bool BWD>
__global__ void linrec_serial_kernel(LinrecParams p) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= p.D) return;
    const TX* x = static_cast<const TX*>(p.x);
    const TG* g = static_cast<const TG*>(p.g);
    const TX* hs = static_cast<const TX*>(p.h);
    TX* out = static_cast<TX*>(p.out);
    TG* dg = static_cast<TG*>(p.dg);
    for (int64_t n = blockIdx.y; n < p.N; n += gridDim.y) {
        const int64_t lo = max((int64_t)p.cu[n], (int64_t)0), hi = min((int64_t)p.cu[n + 1], p.T);
        float h = p.start ? p.start[n * p.D + c] : 0.f;
        for (int64_t i = 0; i < hi - lo; ++i) {
            const int64_t t = BWD ? hi - 1 - i : lo + i;
            const float a = expf(to_f(g[t * p.ldg + c])), b = to_f(x[t * p.ldx + c]);
            if (BWD) {
                const float lam = b + h;
                out[t * p.ldo + c] = from_f<TX>(lam);
                h = a * lam;
                const float before = t > lo ? to_f(hs[(t - 1) * p.ldh + c]) : p.h0 ? p.h0[n * p.D + c] : 0.f;
                dg[t * p.lddg + c] = from_f<TG>(h * before);
            } else {
                h = fmaf(a, h, b);
                out[t * p.ldo + c] = from_f<TX>(h);
            }
        }
        if (p.last) p.last[n * p.D + c] = h;
    }
}

template <typename TX, typename TG>
cudaError_t launch_serial(const LinrecParams& p, bool bwd, cudaStream_t s) {
    const dim3 grid((p.D + 127) / 128, p.N < 65535 ? p.N : 65535);
    KernelTimer kt(bwd ? "linrec_bwd" : "linrec_fwd", s);
    if (bwd)
        linrec_serial_kernel<TX, TG, true><<<grid, 128, 0, s>>>(p);
    else
        linrec_serial_kernel<TX, TG, false><<<grid, 128, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_scan(const LinrecParams& p, int dtype, int gate_dtype, bool bwd, cudaStream_t s) {
    if (dtype == GDR_BF16)
        return gate_dtype == GDR_BF16 ? launch_serial<__nv_bfloat16, __nv_bfloat16>(p, bwd, s)
                                      : launch_serial<__nv_bfloat16, float>(p, bwd, s);
    return gate_dtype == GDR_BF16 ? launch_serial<float, __nv_bfloat16>(p, bwd, s)
                                  : launch_serial<float, float>(p, bwd, s);
}

// ---- the slot-pool step ------------------------------------------------------

struct StepParams {
    const void* x;
    const void* g;
    void* pool;
    const int32_t* idx;
    const int32_t* cu;
    void* y;
    void* states;
    int64_t ldx, ldg, ldy, T;
    int N, D, num_slots, steps, commit;
};

template <typename TX, typename TG, typename TP>
__global__ void linrec_step_kernel(StepParams p) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= p.D) return;
    const TX* x = static_cast<const TX*>(p.x);
    const TG* g = static_cast<const TG*>(p.g);
    TX* y = static_cast<TX*>(p.y);
    for (int64_t n = blockIdx.y; n < p.N; n += gridDim.y) {
        const int slot = p.idx[n];
        if (slot < 0 || slot >= p.num_slots) continue;
        const int64_t lo = max((int64_t)p.cu[n], (int64_t)0), hi = min((int64_t)p.cu[n + 1], p.T);
        if (hi <= lo) continue;
        TP* cell = static_cast<TP*>(p.pool) + (int64_t)slot * p.D + c;
        TP* keep = p.states ? static_cast<TP*>(p.states) + n * p.steps * p.D + c : nullptr;
        float h = to_f(*cell);
        for (int64_t t = lo; t < hi; ++t) {
            h = fmaf(expf(to_f(g[t * p.ldg + c])), h, to_f(x[t * p.ldx + c]));
            y[t * p.ldy + c] = from_f<TX>(h);
            if (keep && t - lo < p.steps) keep[(t - lo) * p.D] = from_f<TP>(h);
        }
        if (p.commit) *cell = from_f<TP>(h);
    }
}

template <typename TX, typename TG, typename TP>
cudaError_t launch_step_t(const StepParams& p, cudaStream_t s) {
    const dim3 grid((p.D + 127) / 128, p.N < 65535 ? p.N : 65535);
    KernelTimer kt("linrec_step", s);
    linrec_step_kernel<TX, TG, TP><<<grid, 128, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename TX, typename TG>
cudaError_t launch_step_p(const StepParams& p, int pool_dtype, cudaStream_t s) {
    return pool_dtype == GDR_BF16 ? launch_step_t<TX, TG, __nv_bfloat16>(p, s) : launch_step_t<TX, TG, float>(p, s);
}

cudaError_t launch_step(const StepParams& p, int dtype, int gate_dtype, int pool_dtype, cudaStream_t s) {
    if (dtype == GDR_BF16)
        return gate_dtype == GDR_BF16 ? launch_step_p<__nv_bfloat16, __nv_bfloat16>(p, pool_dtype, s)
                                      : launch_step_p<__nv_bfloat16, float>(p, pool_dtype, s);
    return gate_dtype == GDR_BF16 ? launch_step_p<float, __nv_bfloat16>(p, pool_dtype, s)
                                  : launch_step_p<float, float>(p, pool_dtype, s);
}

// ---- GDR_VALIDATE --------------------------------------------------------------

enum : unsigned { L_CU = 1u, L_GATE = 2u, L_SLOT = 4u, L_DUP = 8u, L_STEPS = 16u };

static __device__ unsigned int g_linrec_findings;

template <typename TG>
__global__ void linrec_validate_kernel(const int32_t* cu, int N, int64_t T, const TG* g, int64_t ldg, int D,
                                       const int32_t* idx, int num_slots, int commit, int steps) {
    const int64_t tid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t nth = (int64_t)gridDim.x * blockDim.x;
    unsigned bad = 0;
    for (int64_t b = tid; b < N; b += nth) {
        const int lo = cu[b], hi = cu[b + 1];
        if (hi < lo) bad |= L_CU;
        if (idx) {
            const int slot = idx[b];
            if (slot >= num_slots) bad |= L_SLOT;
            if (slot >= 0 && steps > 0 && hi - lo > steps) bad |= L_STEPS;
            if (slot >= 0 && commit)
                for (int64_t j = 0; j < b; ++j)
                    if (idx[j] == slot) bad |= L_DUP;
        }
    }
    if (tid == 0 && (cu[0] != 0 || cu[N] < 0 || cu[N] > T)) bad |= L_CU;
    const int64_t rows = min(max((int64_t)cu[N], (int64_t)0), T);
    for (int64_t i = tid; i < rows * D; i += nth)
        if (!(to_f(g[i / D * ldg + i % D]) <= 0.f)) bad |= L_GATE;
    if (bad) atomicOr(&g_linrec_findings, bad);
}

int validate(const int32_t* cu, int N, int64_t T, const void* g, int64_t ldg, int D, int gate_dtype,
             const int32_t* idx, int num_slots, int commit, int steps, cudaStream_t s) {
    void* word = nullptr;
    if (cudaGetSymbolAddress(&word, g_linrec_findings) != cudaSuccess)
        return set_last_error(GDR_ERR_LAUNCH, "validation word unavailable");
    cudaMemsetAsync(word, 0, sizeof(unsigned), s);
    if (gate_dtype == GDR_BF16)
        linrec_validate_kernel<<<304, 256, 0, s>>>(cu, N, T, static_cast<const __nv_bfloat16*>(g), ldg, D, idx,
                                                   num_slots, commit, steps);
    else
        linrec_validate_kernel<<<304, 256, 0, s>>>(cu, N, T, static_cast<const float*>(g), ldg, D, idx, num_slots,
                                                   commit, steps);
    unsigned found = 0;
    cudaMemcpyAsync(&found, word, sizeof(unsigned), cudaMemcpyDeviceToHost, s);
    const cudaError_t e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return set_last_error(GDR_ERR_LAUNCH, "validation: %s", cudaGetErrorString(e));
    if (found)
        return set_last_error(GDR_ERR_VALIDATION, "input validation failed (0x%x):%s%s%s%s%s", found,
                              (found & L_CU) ? " cu_seqlens malformed;" : "",
                              (found & L_GATE) ? " gate NaN or > 0;" : "",
                              (found & L_SLOT) ? " state index >= num_slots;" : "",
                              (found & L_DUP) ? " duplicate state index;" : "",
                              (found & L_STEPS) ? " sequence longer than steps;" : "");
    return GDR_OK;
}

// ---- argument checks -----------------------------------------------------------

int check_sizes(int N, int64_t T, int D, int dtype, int gate_dtype) {
    if (N < 0 || T < 0) return set_last_error(GDR_ERR_INVALID_ARG, "negative N (%d) or T_total (%lld)", N, (long long)T);
    if (D <= 0) return set_last_error(GDR_ERR_INVALID_ARG, "D (%d) must be positive", D);
    if (dtype != GDR_BF16 && dtype != GDR_F32) return set_last_error(GDR_ERR_UNSUPPORTED, "dtype %d", dtype);
    if (gate_dtype != GDR_BF16 && gate_dtype != GDR_F32)
        return set_last_error(GDR_ERR_UNSUPPORTED, "gate_dtype %d", gate_dtype);
    if (T > 0x7fffffffLL) return set_last_error(GDR_ERR_UNSUPPORTED, "T_total (%lld) above 2^31 - 1", (long long)T);
    if (N > 0x7fffffff / 2) return set_last_error(GDR_ERR_UNSUPPORTED, "N too large");
    if (T > 0 && N == 0) return set_last_error(GDR_ERR_INVALID_ARG, "T_total > 0 with N == 0");
    return GDR_OK;
}

// A token tensor: present, aligned to its element, its stride in range.
int check_rows(const char* name, const void* p, int64_t stride, int D, int dtype, bool written) {
    if (!p) return set_last_error(GDR_ERR_INVALID_ARG, "null pointer argument (%s)", name);
    if (reinterpret_cast<uintptr_t>(p) & (dtype == GDR_BF16 ? 1u : 3u))
        return set_last_error(GDR_ERR_INVALID_ARG, "%s not aligned to its element", name);
    if (stride < (written ? D : 0))
        return set_last_error(GDR_ERR_INVALID_ARG, "%s: row stride %lld too small", name, (long long)stride);
    return GDR_OK;
}

int check_state(const char* name, const void* p) {
    if (reinterpret_cast<uintptr_t>(p) & 15u)
        return set_last_error(GDR_ERR_INVALID_ARG, "%s not 16-byte aligned", name);
    return GDR_OK;
}

int check_workspace(int N, int64_t T, int D, int dtype, int gate_dtype, const void* ws, size_t ws_bytes) {
    size_t need = 0;
    if (int rc = gdr_linrec_workspace_size(N, T, D, dtype, gate_dtype, &need)) return rc;
    if (need == 0) return GDR_OK;
    if (!ws || ws_bytes < need)
        return set_last_error(GDR_ERR_WORKSPACE, "workspace %zu bytes < required %zu", ws ? ws_bytes : (size_t)0, need);
    if (reinterpret_cast<uintptr_t>(ws) & 255u)
        return set_last_error(GDR_ERR_INVALID_ARG, "workspace not 256-byte aligned");
    return GDR_OK;
}

int launched(cudaError_t e, const char* what) {
    if (e != cudaSuccess) return set_last_error(GDR_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
    return set_ok();
}

// No tokens at all: every sequence's last state is its first.
int pass_states(const float* start, float* last, int N, int D, cudaStream_t s) {
    if (N == 0 || !last) return set_ok();
    if (int rc = check_device()) return rc;
    const size_t bytes = sizeof(float) * (size_t)N * D;
    return launched(start ? cudaMemcpyAsync(last, start, bytes, cudaMemcpyDeviceToDevice, s)
                          : cudaMemsetAsync(last, 0, bytes, s), "empty recurrence");
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

int gdr_linrec_workspace_size(int N, int64_t T_total, int D, int dtype, int gate_dtype, size_t* bytes) {
    if (!bytes) return set_last_error(GDR_ERR_INVALID_ARG, "bytes is NULL");
    if (int rc = check_sizes(N, T_total, D, dtype, gate_dtype)) return rc;
    *bytes = 0;
    return set_ok();
}

int gdr_linrec_fwd(const void* x, int64_t x_stride, const void* g, int64_t g_stride, const float* initial_state,
                   const int32_t* cu_seqlens, int N, int64_t T_total, int D, int dtype, int gate_dtype, int flags,
                   void* y, int64_t y_stride, float* final_state, void* workspace, size_t ws_bytes,
                   gdr_stream_t stream) {
    if (int rc = check_sizes(N, T_total, D, dtype, gate_dtype)) return rc;
    if (flags & ~GDR_VALIDATE)
        return set_last_error(GDR_ERR_INVALID_ARG, "unsupported flags 0x%x for gdr_linrec_fwd", flags);
    if (int rc = check_state("initial_state", initial_state)) return rc;
    if (int rc = check_state("final_state", final_state)) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    if (T_total == 0) return pass_states(initial_state, final_state, N, D, s);
    if (int rc = check_rows("x", x, x_stride, D, dtype, false)) return rc;
    if (int rc = check_rows("g", g, g_stride, D, gate_dtype, false)) return rc;
    if (int rc = check_rows("y", y, y_stride, D, dtype, true)) return rc;
    if (!cu_seqlens) return set_last_error(GDR_ERR_INVALID_ARG, "null pointer argument (cu_seqlens)");
    if (int rc = check_workspace(N, T_total, D, dtype, gate_dtype, workspace, ws_bytes)) return rc;
    if (int rc = check_device()) return rc;
    if (flags & GDR_VALIDATE)
        if (int rc = validate(cu_seqlens, N, T_total, g, g_stride, D, gate_dtype, nullptr, 0, 0, 0, s)) return rc;
    LinrecParams p{};
    p.x = x; p.g = g; p.out = y; p.start = initial_state; p.last = final_state; p.cu = cu_seqlens;
    p.ldx = x_stride; p.ldg = g_stride; p.ldo = y_stride; p.T = T_total; p.N = N; p.D = D;
    return launched(launch_scan(p, dtype, gate_dtype, false, s), "gdr_linrec_fwd launch");
}

int gdr_linrec_bwd(const void* dy, int64_t dy_stride, const void* g, int64_t g_stride, const void* y,
                   int64_t y_stride, const float* initial_state, const float* d_final_state,
                   const int32_t* cu_seqlens, int N, int64_t T_total, int D, int dtype, int gate_dtype, int flags,
                   void* dx, int64_t dx_stride, void* dg, int64_t dg_stride, float* d_initial_state,
                   void* workspace, size_t ws_bytes, gdr_stream_t stream) {
    if (int rc = check_sizes(N, T_total, D, dtype, gate_dtype)) return rc;
    if (flags & ~GDR_VALIDATE)
        return set_last_error(GDR_ERR_INVALID_ARG, "unsupported flags 0x%x for gdr_linrec_bwd", flags);
    if (int rc = check_state("initial_state", initial_state)) return rc;
    if (int rc = check_state("d_final_state", d_final_state)) return rc;
    if (int rc = check_state("d_initial_state", d_initial_state)) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    if (T_total == 0) return pass_states(d_final_state, d_initial_state, N, D, s);
    if (int rc = check_rows("dy", dy, dy_stride, D, dtype, false)) return rc;
    if (int rc = check_rows("g", g, g_stride, D, gate_dtype, false)) return rc;
    if (int rc = check_rows("y", y, y_stride, D, dtype, false)) return rc;
    if (int rc = check_rows("dx", dx, dx_stride, D, dtype, true)) return rc;
    if (int rc = check_rows("dg", dg, dg_stride, D, gate_dtype, true)) return rc;
    if (!cu_seqlens) return set_last_error(GDR_ERR_INVALID_ARG, "null pointer argument (cu_seqlens)");
    if (int rc = check_workspace(N, T_total, D, dtype, gate_dtype, workspace, ws_bytes)) return rc;
    if (int rc = check_device()) return rc;
    if (flags & GDR_VALIDATE)
        if (int rc = validate(cu_seqlens, N, T_total, g, g_stride, D, gate_dtype, nullptr, 0, 0, 0, s)) return rc;
    LinrecParams p{};
    p.x = dy; p.g = g; p.h = y; p.out = dx; p.dg = dg; p.h0 = initial_state; p.start = d_final_state;
    p.last = d_initial_state; p.cu = cu_seqlens; p.ldx = dy_stride; p.ldg = g_stride; p.ldh = y_stride;
    p.ldo = dx_stride; p.lddg = dg_stride; p.T = T_total; p.N = N; p.D = D;
    return launched(launch_scan(p, dtype, gate_dtype, true, s), "gdr_linrec_bwd launch");
}

int gdr_linrec_step(const void* x, int64_t x_stride, const void* g, int64_t g_stride, void* state_pool,
                    int pool_dtype, int num_slots, const int32_t* state_indices, const int32_t* cu_seqlens, int N,
                    int64_t T_total, int D, int dtype, int gate_dtype, int flags, void* y, int64_t y_stride,
                    void* intermediate_states, int steps, gdr_stream_t stream) {
    if (int rc = check_sizes(N, T_total, D, dtype, gate_dtype)) return rc;
    if (pool_dtype != GDR_BF16 && pool_dtype != GDR_F32)
        return set_last_error(GDR_ERR_UNSUPPORTED, "pool_dtype %d", pool_dtype);
    if (flags & ~(GDR_COMMIT | GDR_VALIDATE))
        return set_last_error(GDR_ERR_INVALID_ARG, "unsupported flags 0x%x for gdr_linrec_step", flags);
    if (N == 0 || T_total == 0) return set_ok();
    if (num_slots <= 0) return set_last_error(GDR_ERR_INVALID_ARG, "num_slots must be positive");
    if (intermediate_states && steps <= 0)
        return set_last_error(GDR_ERR_INVALID_ARG, "steps must be positive with intermediate_states");
    if (!state_pool || !state_indices || !cu_seqlens)
        return set_last_error(GDR_ERR_INVALID_ARG, "null pointer argument");
    if (int rc = check_state("state_pool", state_pool)) return rc;
    if (int rc = check_state("intermediate_states", intermediate_states)) return rc;
    if (int rc = check_rows("x", x, x_stride, D, dtype, false)) return rc;
    if (int rc = check_rows("g", g, g_stride, D, gate_dtype, false)) return rc;
    if (int rc = check_rows("y", y, y_stride, D, dtype, true)) return rc;
    if (int rc = check_device()) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    if (flags & GDR_VALIDATE)
        if (int rc = validate(cu_seqlens, N, T_total, g, g_stride, D, gate_dtype, state_indices, num_slots,
                              (flags & GDR_COMMIT) ? 1 : 0, intermediate_states ? steps : 0, s))
            return rc;
    StepParams p{};
    p.x = x; p.g = g; p.pool = state_pool; p.idx = state_indices; p.cu = cu_seqlens; p.y = y;
    p.states = intermediate_states; p.ldx = x_stride; p.ldg = g_stride; p.ldy = y_stride; p.T = T_total; p.N = N;
    p.D = D; p.num_slots = num_slots; p.steps = intermediate_states ? steps : 0; p.commit = (flags & GDR_COMMIT) ? 1 : 0;
    return launched(launch_step(p, dtype, gate_dtype, pool_dtype, s), "gdr_linrec_step launch");
}

}  // extern "C"
