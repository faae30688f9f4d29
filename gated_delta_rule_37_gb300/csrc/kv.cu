// The paged key / value cache: new tokens appended, rotary positions applied on
// the way (contract in include/gdr.h).
//
// Token i of sequence n has position p = cache_lens[n] + i.  The pair of channels
// (a, b) with frequency f turns by the angle p f:
//   a' = a cos(p f) - b sin(p f),  b' = b cos(p f) + a sin(p f).
// The angle counts only up to whole turns, and in 32 bits a far position has no
// fraction of a turn left.  So f / 2 pi is kept as a fixed-point fraction of a turn
// in 64 bits, off by less than 2^-63 turns for f <= 1, and p times it wraps modulo one
// turn by itself: the upper 32 bits are the angle, off by at most p 2^-63 + 2^-32
// turns, and a sine of half a turn or less remains.  (All in integers: fp64 is two
// operations a clock on an SM, which bound prompts of few heads.)
//   Every byte is read and written once; memory bounds it: 32768 tokens of 32 + 8 heads of 128, keys
// returned, 142 us, 6.1 TB/s.
#include <math.h>

#include <mutex>

#include "attn.h"
#include "common.cuh"
#include "gdr.h"
#include "launch.h"

namespace gdr {
namespace {

struct AppendParams {
    const void* q;
    const void* k;
    const void* v;
    void* q_out;
    void* k_out;
    int64_t ldq, ldk, ldv, ldqo, ldko;
    const float* freqs;
    const int32_t* cu;
    int64_t T;
    int N, Hq, Hkv, R, pairs;
    int tokens;  // of a block
    Paged c;
};

constexpr int kAppendThreads = 128;

// The last n with cu[n] <= t (t >= cu[0]); the block looks at blockDim.x entries a
// time, so that a search costs one trip to memory for a batch of that size, two for
// its square.  Never reads outside cu[0 .. N].
__device__ __forceinline__ int find_sequence(const int32_t* cu, int N, int64_t t) {
    int lo = 0, hi = N;
    while (hi > lo) {
        const int step = (hi - lo + (int)blockDim.x - 1) / (int)blockDim.x;
        const int64_t at = lo + (int64_t)(threadIdx.x + 1) * step;
        const int below = __syncthreads_count(at <= hi && cu[at] <= t);
        lo += below * step;
        hi = min(lo + step - 1, hi);
    }
    return lo;
}

// VEC consecutive channels, 16 bytes of them.
template <typename T> struct Pack16;
template <> struct Pack16<float> {
    static constexpr int VEC = 4;
};
template <> struct Pack16<__nv_bfloat16> {
    static constexpr int VEC = 8;
};

__device__ __forceinline__ void spread(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void spread(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store16(float* p, const float (&f)[4]) { Vec<float, 4>::store(p, f); }
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&f)[8]) {
    uint4 u;
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    u.x = *reinterpret_cast<uint32_t*>(&h[0]);
    u.y = *reinterpret_cast<uint32_t*>(&h[1]);
    u.z = *reinterpret_cast<uint32_t*>(&h[2]);
    u.w = *reinterpret_cast<uint32_t*>(&h[3]);
    *reinterpret_cast<uint4*>(p) = u;
}

// f / 2 pi modulo 1 in 64 bits.  With f = m 2^e, m of 24 bits, and K = 2^64 / 2 pi rounded, it is
// m K 2^e: a product of 86 bits, shifted.
__device__ __forceinline__ uint64_t turn_of(float f) {
    constexpr uint64_t K = 0x28be60db9391054aull;
    const uint32_t bits = __float_as_uint(f), field = bits >> 23 & 255;
    const uint64_t m = (bits & 0x7fffffu) | (field ? 0x800000u : 0u);
    const int right = 150 - (int)max(field, 1u);  // -e
    const uint64_t lo = m * K, hi = __umul64hi(m, K);
    uint64_t unit = 0;
    if (right > 0 && right < 64) unit = lo >> right | hi << (64 - right);
    else if (right >= 64 && right < 128) unit = hi >> (right - 64);
    else if (right <= 0 && right > -64) unit = lo << -right;
    return bits >> 31 ? 0 - unit : unit;
}

// The row of position pos of sequence n in the caches, of head 0; -1 where it has none.
__device__ __forceinline__ int64_t cache_row(const AppendParams& p, int n, int64_t pos) {
    const int64_t slot = pos >> p.c.page_bits;
    if (slot >= p.c.max_pages) return -1;
    const int page = p.c.table[n * p.c.table_ld + slot];
    if (page < 0 || page >= p.c.num_pages) return -1;
    return ((int64_t)page * p.Hkv << p.c.page_bits) + (pos & (p.c.page_size - 1));
}

constexpr int kMostTokens = 8;  // of a block

// One block per (token, share of the heads), or with MANY per p.tokens tokens.  A thread owns
// two 16-byte pieces of a head's row, the pieces x and x + R / 2 where those turn with one
// another, and walks over the heads.  What it reads of its first head does not depend on
// the token's place, which takes four trips to memory in turn: it is asked for before them,
// and each next head's before this one is turned and written.
template <typename T, int D, bool MANY>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendParams p) {
    constexpr int VEC = Pack16<T>::VEC, PIECES = D / (2 * VEC), LANES = kAppendThreads / PIECES;
    constexpr int TOKENS = MANY ? kMostTokens : 1;
    __shared__ float2 turn[TOKENS][D / 2];
    __shared__ int64_t places[TOKENS], rows[TOKENS];  // MANY: position, -1 for none, and row in the caches
    const int64_t t0 = MANY ? (int64_t)blockIdx.x * p.tokens : blockIdx.x;
    const int count = MANY ? (int)min((int64_t)p.tokens, p.T - t0) : 1;
    const int half = p.R / 2;
    const int piece = threadIdx.x % PIECES, lane = threadIdx.x / PIECES + LANES * blockIdx.y;
    const int heads = p.Hq + 2 * p.Hkv, items = heads * count;  // of one token after the other
    // the pieces' channels, and whether they turn with one another element by element
    const bool across = !p.pairs && piece * VEC < half;
    const int c0 = across ? piece * VEC : p.pairs ? piece * 2 * VEC : 2 * half + (piece - half / VEC) * 2 * VEC;
    const int c1 = across ? c0 + half : c0 + VEC;
    uint4 next[2];
    auto ask = [&](int item) {
        const int tok = MANY ? item / heads : 0, h = item - tok * heads;
        const int64_t t = t0 + tok;
        const T* from = h < p.Hq           ? static_cast<const T*>(p.q) + t * p.ldq + (int64_t)h * D
                        : h < p.Hq + p.Hkv ? static_cast<const T*>(p.k) + t * p.ldk + (int64_t)(h - p.Hq) * D
                                           : static_cast<const T*>(p.v) + t * p.ldv + (int64_t)(h - p.Hq - p.Hkv) * D;
        next[0] = *reinterpret_cast<const uint4*>(from + c0);
        next[1] = *reinterpret_cast<const uint4*>(from + c1);
    };
    if (lane < items) ask(lane);
    int n = 0;
    int64_t pos = 0, row = -1;
    if (MANY) {
        if (threadIdx.x < count) {
            // the last sequence that begins at or before the token
            const int64_t t = t0 + threadIdx.x;
            int hi = p.N;
            while (hi > n) {
                const int mid = (n + hi + 1) / 2;
                if (p.cu[mid] <= t) n = mid; else hi = mid - 1;
            }
            pos = -1;
            if (n < p.N && p.cu[n] <= t && t < p.cu[n + 1]) {
                const int len = p.c.lens[n];
                if (len >= 0) {
                    pos = (int64_t)len + (t - p.cu[n]);
                    row = cache_row(p, n, pos);
                }
            }
            places[threadIdx.x] = pos;
            rows[threadIdx.x] = row;
        }
        __syncthreads();
    } else {
        if (p.cu[0] > t0) return;
        n = find_sequence(p.cu, p.N, t0);
        if (n >= p.N || t0 >= p.cu[n + 1]) return;  // behind the last sequence
        const int len = p.c.lens[n];
        if (len < 0) return;
        pos = (int64_t)len + (t0 - p.cu[n]);
    }
    for (int i = threadIdx.x; i < half * count; i += kAppendThreads) {
        const int tok = MANY ? i / half : 0, j = i - tok * half;
        const uint64_t angle = turn_of(p.freqs[j]) * (uint64_t)(MANY ? places[tok] : pos);
        float s, c;
        sincospif((float)(int)(angle >> 32) * 0x1p-31f, &s, &c);
        turn[tok][j] = make_float2(c, s);
    }
    __syncthreads();

    if (!MANY) row = cache_row(p, n, pos);
    const int step = LANES * gridDim.y;
    for (int item = lane; item < items; item += step) {
        const int tok = MANY ? item / heads : 0, h = item - tok * heads;
        const int64_t t = t0 + tok;
        if (MANY) row = rows[tok];
        float x[VEC], y[VEC];
        spread(next[0], x);
        spread(next[1], y);
        if (item + step < items) ask(item + step);
        if (MANY && places[tok] < 0) continue;
        T* dense = nullptr;
        T* cached = nullptr;
        if (h < p.Hq) {
            dense = static_cast<T*>(p.q_out) + t * p.ldqo + (int64_t)h * D;
        } else {
            const int kv = h < p.Hq + p.Hkv ? h - p.Hq : h - p.Hq - p.Hkv;
            const bool key = h < p.Hq + p.Hkv;
            if (key && p.k_out) dense = static_cast<T*>(p.k_out) + t * p.ldko + (int64_t)kv * D;
            if (row >= 0)
                cached = static_cast<T*>(key ? p.c.k : p.c.v) + (row + ((int64_t)kv << p.c.page_bits)) * D;
        }
        if (h < p.Hq + p.Hkv && half > 0) {
            const float2* const w_of = turn[tok];
            if (across) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float2 w = w_of[c0 + i];
                    const float a = x[i], b = y[i];
                    x[i] = a * w.x - b * w.y;
                    y[i] = b * w.x + a * w.y;
                }
            } else if (p.pairs) {
#pragma unroll
                for (int i = 0; i < VEC; i += 2) {
                    if (c0 + i < p.R) {
                        const float2 w = w_of[(c0 + i) / 2];
                        const float a = x[i], b = x[i + 1];
                        x[i] = a * w.x - b * w.y;
                        x[i + 1] = b * w.x + a * w.y;
                    }
                    if (c1 + i < p.R) {
                        const float2 w = w_of[(c1 + i) / 2];
                        const float a = y[i], b = y[i + 1];
                        y[i] = a * w.x - b * w.y;
                        y[i + 1] = b * w.x + a * w.y;
                    }
                }
            }
        }
        if (dense) {
            store16(dense + c0, x);
            store16(dense + c1, y);
        }
        if (cached) {
            store16(cached + c0, x);
            store16(cached + c1, y);
        }
    }
}

template <typename T, int D>
cudaError_t launch_append(AppendParams p, cudaStream_t s) {
    constexpr int LANES = kAppendThreads / (D / (2 * Pack16<T>::VEC));
    // few tokens: their heads over several blocks; many of few heads: several to a block, as long
    // as that leaves eight blocks to an SM and gives a thread no more than four pairs of pieces
    // (measured, several / one, when the angles still took fp64: 14998 tokens of 2 + 2 heads of 128
    // 22 / 35 us, 16000 of 8 + 1 of 64 18 / 33, 7001 of 12 + 4 of 64 in fp32 19.5 / 20.8; with integers
    // 17, 15 and 19.  A prompt of 32768 tokens of 32 + 8 heads has one to a block: 143 us, 6.1 TB/s.)
    const int heads = p.Hq + 2 * p.Hkv, most = (heads + LANES - 1) / LANES;
    const int64_t full = (int64_t)sm_count() * 8;
    const int64_t share = p.T < full ? full / (p.T > 0 ? p.T : 1) : 1;
    p.tokens = 1;
    while (p.tokens < kMostTokens && p.T / (2 * p.tokens) >= full && 2 * p.tokens * heads <= 4 * LANES) p.tokens *= 2;
    KernelTimer kt("kv_append", s);
    if (p.tokens > 1)
        kv_append_kernel<T, D, true><<<(unsigned)((p.T + p.tokens - 1) / p.tokens), kAppendThreads, 0, s>>>(p);
    else
        kv_append_kernel<T, D, false><<<dim3((unsigned)p.T, (unsigned)(share < most ? share : most)), kAppendThreads, 0, s>>>(p);
    return cudaGetLastError();
}

// ---- GDR_VALIDATE ----------------------------------------------------------------

enum : unsigned { A_CU = 1u, A_PAGE = 2u, A_LONG = 4u, A_PREFIX = 8u };

static __device__ unsigned int g_attention_findings;

__global__ void attention_validate_kernel(const int32_t* cu, int N, int64_t T, int paged, Paged c) {
    const int64_t tid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t nth = (int64_t)gridDim.x * blockDim.x;
    unsigned bad = 0;
    if (tid == 0 && (cu[0] != 0 || cu[N] < 0 || cu[N] > T)) bad |= A_CU;
    for (int64_t b = tid; b < N; b += nth)
        if (cu[b + 1] < cu[b]) bad |= A_CU;
    if (paged) {
        for (int64_t b = blockIdx.x; b < N; b += gridDim.x) {
            const int64_t fresh = (int64_t)cu[b + 1] - cu[b];
            if (c.lens[b] < 0 || fresh <= 0) continue;
            const int64_t end = c.lens[b] + fresh;  // positions 0 .. end - 1, the prefix's in its own pages
            if (end <= c.prefix_len) continue;          // no page of its own
            const int64_t pages = (end + c.page_size - 1) >> c.page_bits;
            if (pages > c.max_pages) bad |= A_LONG;
            // a call without a prefix that only writes reaches the new tokens' pages alone
            const int64_t from = c.prefix_len < 0 ? c.lens[b] : c.prefix_len;
            for (int64_t j = (from >> c.page_bits) + threadIdx.x; j < min(pages, (int64_t)c.max_pages); j += blockDim.x) {
                const int page = c.table[b * c.table_ld + j];
                if (page < 0 || page >= c.num_pages) bad |= A_PAGE;
            }
        }
        for (int64_t j = tid; j < (c.prefix_len + c.page_size - 1) >> c.page_bits; j += nth)
            if (c.prefix[j] < 0 || c.prefix[j] >= c.num_pages) bad |= A_PREFIX;
    }
    if (bad) atomicOr(&g_attention_findings, bad);
}

}  // namespace

int validate_attention(const int32_t* cu, int N, int64_t T, const Paged* c, cudaStream_t s) {
    // one word for all: from its clearing to its reading it belongs to one call
    static std::mutex turn;
    const std::lock_guard<std::mutex> own(turn);
    void* word = nullptr;
    if (cudaGetSymbolAddress(&word, g_attention_findings) != cudaSuccess)
        return set_last_error(GDR_ERR_LAUNCH, "validation word unavailable");
    cudaError_t e = cudaMemsetAsync(word, 0, sizeof(unsigned), s);
    if (e != cudaSuccess) return set_last_error(GDR_ERR_LAUNCH, "validation: %s", cudaGetErrorString(e));
    attention_validate_kernel<<<304, 256, 0, s>>>(cu, N, T, c != nullptr, c ? *c : Paged{});
    e = cudaGetLastError();
    unsigned found = 0;
    if (e == cudaSuccess) e = cudaMemcpyAsync(&found, word, sizeof(unsigned), cudaMemcpyDeviceToHost, s);
    const cudaError_t ended = cudaStreamSynchronize(s);  // also behind a copy that was refused: `found` is on this stack
    if (e == cudaSuccess) e = ended;
    if (e != cudaSuccess) return set_last_error(GDR_ERR_LAUNCH, "validation: %s", cudaGetErrorString(e));
    if (found)
        return set_last_error(GDR_ERR_VALIDATION, "input validation failed (0x%x):%s%s%s%s", found,
                              (found & A_CU) ? " cu_seqlens malformed;" : "",
                              (found & A_PAGE) ? " page number outside the cache;" : "",
                              (found & A_LONG) ? " sequence longer than its pages;" : "",
                              (found & A_PREFIX) ? " prefix page outside the cache;" : "");
    return GDR_OK;
}

// ---- argument checks ---------------------------------------------------------------

int check_heads(int N, int64_t T, int Hq, int Hkv, int D, int dtype) {
    if (N < 0 || T < 0) return set_last_error(GDR_ERR_INVALID_ARG, "negative N (%d) or T_total (%lld)", N, (long long)T);
    if (Hkv <= 0 || Hq < 0 || Hq % Hkv != 0)
        return set_last_error(GDR_ERR_INVALID_ARG, "Hq (%d) must be a multiple of Hkv (%d > 0)", Hq, Hkv);
    if (Hq > 4096 || Hkv > 4096) return set_last_error(GDR_ERR_UNSUPPORTED, "more than 4096 heads");
    if (Hq / Hkv > GDR_ATTN_MAX_GROUP)
        return set_last_error(GDR_ERR_UNSUPPORTED, "Hq / Hkv (%d) above %d", Hq / Hkv, GDR_ATTN_MAX_GROUP);
    if (dtype != GDR_BF16 && dtype != GDR_F32) return set_last_error(GDR_ERR_UNSUPPORTED, "dtype %d", dtype);
    if (D != 64 && D != 128) return set_last_error(GDR_ERR_UNSUPPORTED, "D (%d) must be 64 or 128", D);
    if (T > 0x7fffffffLL - 512) return set_last_error(GDR_ERR_UNSUPPORTED, "T_total (%lld) too large", (long long)T);
    if (N > 65535) return set_last_error(GDR_ERR_UNSUPPORTED, "N (%d) above 65535 sequences per call", N);
    if (T > 0 && N == 0) return set_last_error(GDR_ERR_INVALID_ARG, "T_total > 0 with N == 0");
    return GDR_OK;
}

int check_token_rows(const char* name, const void* p, int64_t stride, int64_t least, int dtype) {
    const int64_t vec = dtype == GDR_BF16 ? 8 : 4;
    if (!p) return set_last_error(GDR_ERR_INVALID_ARG, "null pointer argument (%s)", name);
    if (int rc = check_aligned16(name, p)) return rc;
    if (stride < least || stride % vec != 0 || stride >= (1LL << 32))
        return set_last_error(GDR_ERR_INVALID_ARG, "%s: token stride %lld must be a multiple of 16 bytes, at least %lld",
                              name, (long long)stride, (long long)least);
    return GDR_OK;
}

int check_apart(const MemRows& a, const MemRows& b) {
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0) return GDR_OK;
    const int64_t pa = (int64_t)reinterpret_cast<uintptr_t>(a.p), pb = (int64_t)reinterpret_cast<uintptr_t>(b.p);
    if (pa + (a.rows - 1) * a.ld + a.row <= pb || pb + (b.rows - 1) * b.ld + b.row <= pa) return GDR_OK;
    if (a.ld == b.ld && a.ld > 0) {
        const int64_t d = ((pb - pa) % a.ld + a.ld) % a.ld;  // where b's rows begin within a's
        if (d >= a.row && d + b.row <= a.ld) return GDR_OK;
    }
    return set_last_error(GDR_ERR_INVALID_ARG, "%s is written and overlaps %s", a.name, b.name);
}

int check_int32s(const char* name, const void* p) {
    if (!p) return set_last_error(GDR_ERR_INVALID_ARG, "null pointer argument (%s)", name);
    if (reinterpret_cast<uintptr_t>(p) & 3u)
        return set_last_error(GDR_ERR_INVALID_ARG, "%s not 4-byte aligned", name);
    return GDR_OK;
}

int check_paged(const Paged& c, int N, int Hkv, int D, int dtype) {
    if (c.page_size < 16 || c.page_size > 256 || (c.page_size & (c.page_size - 1)))
        return set_last_error(GDR_ERR_UNSUPPORTED, "page_size (%d) must be 16, 32, 64, 128 or 256", c.page_size);
    if (c.num_pages <= 0 || c.max_pages <= 0)
        return set_last_error(GDR_ERR_INVALID_ARG, "num_pages (%d) and max_pages (%d) must be positive", c.num_pages,
                              c.max_pages);
    if ((int64_t)c.num_pages * Hkv * c.page_size > 0x7fffffffLL)
        return set_last_error(GDR_ERR_UNSUPPORTED, "caches of more than 2^31 - 1 rows");
    if ((int64_t)c.max_pages * c.page_size > 0x7fffffffLL - 256)
        return set_last_error(GDR_ERR_UNSUPPORTED, "block_table of more than 2^31 - 257 positions");
    if (!c.k || !c.v) return set_last_error(GDR_ERR_INVALID_ARG, "null pointer argument (cache)");
    if (int rc = check_aligned16("k_cache", c.k)) return rc;
    if (int rc = check_aligned16("v_cache", c.v)) return rc;
    if (int rc = check_int32s("block_table", c.table)) return rc;
    if (int rc = check_int32s("cache_lens", c.lens)) return rc;
    if (c.table_ld < c.max_pages && N > 1)
        return set_last_error(GDR_ERR_INVALID_ARG, "block_table: row stride %lld below max_pages", (long long)c.table_ld);
    return GDR_OK;
}

}  // namespace gdr

using namespace gdr;

extern "C" {

int gdr_kv_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                  const float* freqs, int rotary_dim, const int32_t* cache_lens, const int32_t* block_table,
                  int64_t table_stride, int max_pages, const int32_t* cu_seqlens, int N, int64_t T_total, int Hq,
                  int Hkv, int D, int dtype, int flags, void* q_out, int64_t q_out_stride, void* k_out,
                  int64_t k_out_stride, void* k_cache, void* v_cache, int num_pages, int page_size,
                  gdr_stream_t stream) {
    if (int rc = check_heads(N, T_total, Hq, Hkv, D, dtype)) return rc;
    if (flags & ~(GDR_ROPE_PAIRS | GDR_VALIDATE))
        return set_last_error(GDR_ERR_INVALID_ARG, "unsupported flags 0x%x for gdr_kv_append", flags);
    const int unit = flags & GDR_ROPE_PAIRS ? 2 : 16;
    if (rotary_dim < 0 || rotary_dim > D || rotary_dim % unit)
        return set_last_error(GDR_ERR_INVALID_ARG, "rotary_dim (%d) must be a multiple of %d, up to D", rotary_dim, unit);
    if (N == 0 || T_total == 0) return set_ok();
    AppendParams p{};
    p.c = Paged{k_cache, v_cache, block_table, table_stride, cache_lens, nullptr, 0, max_pages, num_pages, page_size, 0};
    if (int rc = check_paged(p.c, N, Hkv, D, dtype)) return rc;
    while ((1 << p.c.page_bits) < page_size) ++p.c.page_bits;
    const int64_t wide = (int64_t)Hq * D, narrow = (int64_t)Hkv * D;
    if ((q != nullptr) != (Hq > 0) || (q_out != nullptr) != (Hq > 0))
        return set_last_error(GDR_ERR_INVALID_ARG, "q and q_out go together with Hq > 0");
    if (q)
        if (int rc = check_token_rows("q", q, q_stride, 0, dtype)) return rc;
    if (int rc = check_token_rows("k", k, k_stride, 0, dtype)) return rc;
    if (int rc = check_token_rows("v", v, v_stride, 0, dtype)) return rc;
    if (q)
        if (int rc = check_token_rows("q_out", q_out, q_out_stride, wide, dtype)) return rc;
    if (k_out)
        if (int rc = check_token_rows("k_out", k_out, k_out_stride, narrow, dtype)) return rc;
    if ((q && q == q_out && q_stride != q_out_stride) || (k == k_out && k_stride != k_out_stride))
        return set_last_error(GDR_ERR_INVALID_ARG, "rows turned in place keep their stride");
    if (rotary_dim > 0 && (!freqs || (reinterpret_cast<uintptr_t>(freqs) & 3u)))
        return set_last_error(GDR_ERR_INVALID_ARG, "freqs missing or not 4-byte aligned");
    if (int rc = check_int32s("cu_seqlens", cu_seqlens)) return rc;
    {
        const int64_t e = dtype == GDR_BF16 ? 2 : 4, cache = (int64_t)num_pages * Hkv * page_size * D * e;
        const MemRows in[3] = {{"q", q, wide * e, q_stride * e, T_total}, {"k", k, narrow * e, k_stride * e, T_total},
                               {"v", v, narrow * e, v_stride * e, T_total}};
        const MemRows out[4] = {{"q_out", q_out, wide * e, q_out_stride * e, T_total},
                                {"k_out", k_out, narrow * e, k_out_stride * e, T_total},
                                {"k_cache", k_cache, cache, cache, 1}, {"v_cache", v_cache, cache, cache, 1}};
        for (int i = 0; i < 4; ++i) {
            for (int j = 0; j < 3; ++j)
                if (!(i < 2 && i == j && out[i].p == in[j].p))  // in place
                    if (int rc = check_apart(out[i], in[j])) return rc;
            for (int j = i + 1; j < 4; ++j)
                if (int rc = check_apart(out[i], out[j])) return rc;
        }
    }
    if (int rc = check_device()) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    if (flags & GDR_VALIDATE) {
        Paged c = p.c;
        c.prefix_len = -1;
        if (int rc = validate_attention(cu_seqlens, N, T_total, &c, s)) return rc;
    }
    p.q = q; p.k = k; p.v = v; p.q_out = q_out; p.k_out = k_out;
    p.ldq = q_stride; p.ldk = k_stride; p.ldv = v_stride; p.ldqo = q_out_stride; p.ldko = k_out_stride;
    p.freqs = freqs; p.cu = cu_seqlens; p.T = T_total; p.N = N; p.Hq = Hq; p.Hkv = Hkv; p.R = rotary_dim;
    p.pairs = flags & GDR_ROPE_PAIRS ? 1 : 0;
    const cudaError_t e = dtype == GDR_BF16 ? (D == 128 ? launch_append<__nv_bfloat16, 128>(p, s)
                                                        : launch_append<__nv_bfloat16, 64>(p, s))
                                            : (D == 128 ? launch_append<float, 128>(p, s) : launch_append<float, 64>(p, s));
    return launch_result(e, "gdr_kv_append launch");
}

}  // extern "C"
