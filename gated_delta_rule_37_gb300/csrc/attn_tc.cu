// Causal attention on the tensor cores (bf16): packed prompts, and the prefix that a
// batch shares in the paged cache.
//
// A CTA has one key head and two tiles of 128 query rows, a row being a (token, query
// head of the group) pair: the heads that read one key head share every key tile, and a
// causal tile has rows of 128 / group tokens only.  It walks over the keys by tiles of
// 128.  Per row tile and key tile, with S and O in tensor memory:
//   S = Q K^T     one thread issues it: Q and K from shared memory, 128 x 128 x D
//   P = 2^(S c - m)   a warpgroup, a row per thread, c = scale log2(e): P goes back into
//                 S's columns as bf16, its sum stays in fp32
//   O += P V      P from tensor memory, V from shared memory as it was loaded (rows of
//                 keys: the contraction runs down the tile)
// The two row tiles alternate: while one's P is formed the tensor cores work on the
// other's O += P V and next S.  S of one tile is free again when its O += P V has read P,
// and MMAs run in the order of their issue, so that needs no wait.
//   The maximum m that P refers to follows the row's maximum lazily: O and the sum are
// rescaled only when the maximum has risen by more than 2^8, so P stays within 2^8 and
// O's rescaling, a trip through registers, is rare.  m cancels in O / sum.
//   Keys behind a sequence's last one are not another's to see: their V rows are cleared
// in shared memory (0 * NaN is a NaN), in the last tile alone.  Within a sequence a later
// token's infinity or NaN could still reach an earlier row as 0 * inf; a row whose result
// is not finite is computed once more, on the CUDA cores, from the keys that it sees.
#include <math.h>

#include <atomic>

#include "attn.h"
#include "attn_copies.cuh"
#include "attn_step.cuh"
#include "common.cuh"
#include "gdr.h"
#include "launch.h"
#include "tc.cuh"

namespace gdr {
namespace {

using namespace tc;

constexpr int kTile = 128;                // rows of a query tile, keys of a key tile
constexpr int kWarps = 12;                // 2 x 4 of softmax; the copies', the MMAs' and two that only leave
// Registers: a softmax thread keeps a row of S.  The block is launched with 168 a thread,
// 3 x 168 for a thread of each warpgroup; the third one's go to the others.
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * kLaunchRegs, "more registers than the block has");
constexpr float kLag = 8.f;               // how far P's reference may lag behind the maximum, log2 units

template <int D> struct Shape {
    static constexpr int BLOCKS = D / 64;                  // 128-byte column blocks of a row
    static constexpr int BLOCK_BYTES = kTile * 128;
    static constexpr int TILE_BYTES = BLOCKS * BLOCK_BYTES;
    static constexpr int STAGES = D == 128 ? 5 : 8;
    static constexpr int SMEM = 1024 + (2 + STAGES) * TILE_BYTES;
    static constexpr uint32_t S = 0, O = 256;              // tensor memory columns: S of both row tiles, O of both
};

struct Barriers {
    uint64_t q[2], full[8], empty[8], s[2], p[2], o[2], fixed, drain;
};

struct TcParams {
    AttnArgs a;
    StepWork w;
    int tokens;  // of a row tile: 128 / group
    int box;     // rows of one copy of keys: 128, or a page's
    unsigned* err;
};

// D += A B with A in tensor memory.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
                 :: "r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc));
}

#define GDR_R32(x, b)                                                                                                \
    x(b, 0), x(b, 1), x(b, 2), x(b, 3), x(b, 4), x(b, 5), x(b, 6), x(b, 7), x(b, 8), x(b, 9), x(b, 10), x(b, 11),    \
        x(b, 12), x(b, 13), x(b, 14), x(b, 15), x(b, 16), x(b, 17), x(b, 18), x(b, 19), x(b, 20), x(b, 21),          \
        x(b, 22), x(b, 23), x(b, 24), x(b, 25), x(b, 26), x(b, 27), x(b, 28), x(b, 29), x(b, 30), x(b, 31)
#define GDR_OUT(b, i) "=f"((b)[i])
#define GDR_INOUT(b, i) "+f"((b)[i])
#define GDR_IN(b, i) "r"((b)[i])
#define GDR_LIST32                                                                                                   \
    "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"    \
    "%29,%30,%31}"

// 32 columns of this thread's lane; the registers are there after arrived32.
__device__ __forceinline__ void tmem_fetch32(uint32_t addr, float* v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 " GDR_LIST32 ", [%32];" : GDR_R32(GDR_OUT, v) : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// ties the registers to what was waited for
__device__ __forceinline__ void arrived32(float* v) { asm volatile("" : GDR_R32(GDR_INOUT, v)); }
__device__ __forceinline__ void tmem_put32(uint32_t addr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], " GDR_LIST32 ";" :: GDR_R32(GDR_IN, v), "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// What a CTA works on.
struct Job {
    int64_t t0;       // first token of its rows' sequence (prompt), or 0
    int64_t i0;       // its first token, counted from t0
    int64_t end;      // tokens of the sequence, or of the batch
    int from, to[2];  // key tiles of the two row tiles: from .. to - 1
    int keys;         // end of the keys, counted from the sequence's first
    int n;
};

template <int D, bool PREFIX>
__global__ void __launch_bounds__(kWarps * 32, 1)
    attn_tc_kernel(const TcParams p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv) {
    using C = Shape<D>;
    extern __shared__ unsigned char raw[];
    __shared__ Barriers bars;
    __shared__ Job job;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ int limits[PREFIX ? 2 * kTile : 1];            // per token of the CTA: end of the keys that it sees
    __shared__ uint32_t missing[PREFIX ? 16 : 1];             // per key tile: a bit per 16 keys without a page
    const AttnArgs& a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, group = a.group;
    const int h = PREFIX ? blockIdx.y : blockIdx.x % a.Hkv;
    volatile int* abort = &abort_flag;

    // ---- what to do ----
    if (PREFIX) {
        const int64_t first = (int64_t)blockIdx.x * 2 * p.tokens;
        const int tiles = (a.cache.prefix_len + kTile - 1) / kTile;
        if (tid == 0) {
            job.t0 = 0;
            job.i0 = first;
            job.end = a.T;
            job.from = (int)((int64_t)tiles * blockIdx.z / p.w.splits);
            job.to[0] = (int)((int64_t)tiles * (blockIdx.z + 1) / p.w.splits);
            job.to[1] = first + p.tokens < a.T ? job.to[0] : job.from;
            job.keys = a.cache.prefix_len;
        }
        for (int i = tid; i < 2 * kTile; i += kWarps * 32) limits[i] = 0;
        __syncthreads();
        // every sequence marks its tokens that the CTA has
        for (int n = tid; n < a.N; n += kWarps * 32) {
            const int len = a.cache.lens[n];
            const int64_t lo = a.cu[n], hi = min((int64_t)a.cu[n + 1], a.T);
            if (len < 0) continue;
            for (int64_t t = max(lo, first); t < min(hi, first + 2 * p.tokens); ++t)
                limits[t - first] = (int)min((int64_t)a.cache.prefix_len, len + (t - lo) + 1);
        }
    } else {
        if (tid == 0) job.n = -1;
        __syncthreads();
        if (warp == 0) {
            // the CTAs of all sequences in a row, the last first: their rows see most keys
            int64_t left = gridDim.x / a.Hkv - 1 - blockIdx.x / a.Hkv;
            for (int base = 0; base < a.N && left >= 0; base += 32) {
                const int n = base + lane;
                int64_t t0 = 0, L = 0, count = 0;
                if (n < a.N) {
                    t0 = max(a.cu[n], 0);
                    L = min((int64_t)a.cu[n + 1], a.T) - t0;
                    count = L > 0 ? (L + 2 * p.tokens - 1) / (2 * p.tokens) : 0;
                }
                int64_t upto = count;
#pragma unroll
                for (int off = 1; off < 32; off *= 2) {
                    const int64_t u = __shfl_up_sync(0xffffffffu, upto, off);
                    if (lane >= off) upto += u;
                }
                if (left < upto && left >= upto - count) {
                    job.t0 = t0;
                    job.i0 = (left - (upto - count)) * 2 * p.tokens;
                    job.end = L;
                    job.from = 0;
                    const int64_t i1 = job.i0 + p.tokens;
                    job.to[0] = (int)((min(i1, L) + kTile - 1) / kTile);
                    job.to[1] = i1 < L ? (int)((min(i1 + p.tokens, L) + kTile - 1) / kTile) : 0;
                    job.keys = (int)min(job.i0 + 2 * p.tokens, L);
                    job.n = n;
                }
                const int64_t all = __shfl_sync(0xffffffffu, upto, 31);
                left = left < all ? -1 : left - all;
            }
        }
        __syncthreads();
        if (job.n < 0) return;
    }

    // ---- barriers, tensor memory ----
    const uint32_t q_smem = (smem_u32(raw) + 1023) & ~1023u, ring = q_smem + 2 * C::TILE_BYTES;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars.q[i]), 1);
            mbar_init(smem_u32(&bars.s[i]), 1);
            mbar_init(smem_u32(&bars.p[i]), 4);
            mbar_init(smem_u32(&bars.o[i]), 1);
        }
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(smem_u32(&bars.full[i]), 1);
            mbar_init(smem_u32(&bars.empty[i]), 1);
        }
        mbar_init(smem_u32(&bars.fixed), 1);
        mbar_init(smem_u32(&bars.drain), 1);
        mbar_fence_init();
        abort_flag = 0;
    }
    if (warp == 9) tmem_alloc(smem_u32(&tmem_slot), 512);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;
    const int from = job.from, to0 = job.to[0], to1 = job.to[1], to = max(to0, to1), count = to - from;
    const bool tail = job.keys < to * kTile;  // the last tile has rows that are not the sequence's

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kOtherRegs));
        if (warp == 8) {
            // ---- copies ----
            int issued = 0;
            bool ok = true;
            if (lane == 0) {
                for (int t = 0; t < 2; ++t) {
                    if ((t ? to1 : to0) <= from) continue;
                    const uint32_t mbar = smem_u32(&bars.q[t]);
                    mbar_arrive_tx(mbar, C::BLOCKS * p.tokens * group * 128);
                    for (int b = 0; b < C::BLOCKS; ++b)
                        tma_3d(q_smem + t * C::TILE_BYTES + b * C::BLOCK_BYTES, &mq, b * 64, h * group,
                               (int)(job.t0 + job.i0 + t * p.tokens), mbar);
                }
            }
            const int pieces = kTile / p.box;
            auto page_of = [&](int piece) {
                const int64_t key = (int64_t)piece * p.box;
                return key < a.cache.prefix_len ? a.cache.prefix[key >> a.cache.page_bits] : -1;
            };
            int held = 0, asked = PREFIX ? page_of(from * pieces + lane) : 0, at = -64;
            for (int it = 0; it < 2 * count && ok; ++it) {
                const int stage = it % C::STAGES, j = from + (it >> 1);
                if (it >= C::STAGES) ok = mbar_wait(smem_u32(&bars.empty[stage]), (it / C::STAGES - 1) & 1, abort);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                const uint32_t mbar = smem_u32(&bars.full[stage]), dst = ring + stage * C::TILE_BYTES;
                const CUtensorMap* map = it & 1 ? &mv : &mk;
                if (PREFIX) {
                    // piece `lane` of the tile; one without a page is read from the cache's first rows and
                    // masked.  The pages are those of 32 pieces, asked for 32 pieces ahead
                    const int first = j * pieces;
                    if (first + pieces > at + 32) {
                        at = first;
                        held = asked;
                        asked = page_of(at + 32 + lane);
                    }
                    const int page = __shfl_sync(0xffffffffu, held, (first - at + lane) & 31);
                    const int64_t key = (int64_t)j * kTile + lane * p.box;
                    bool gone = page < 0 || page >= a.cache.num_pages;
                    const int row = gone ? 0 : (int)((((int64_t)page * a.Hkv + h) << a.cache.page_bits) +
                                                     (key & (a.cache.page_size - 1)));
                    gone = gone && key < a.cache.prefix_len;
                    const bool part = __shfl_sync(0xffffffffu, gone, lane * 16 / p.box & 31);
                    const uint32_t out = __ballot_sync(0xffffffffu, part && lane < kTile / 16);
                    if (lane == 0) {
                        // the ring holds 4 key tiles at most, and the MMAs are one ahead of the softmax
                        if (!(it & 1)) missing[(it >> 1) & 15] = out;
                        mbar_arrive_tx(mbar, C::TILE_BYTES);
                    }
                    __syncwarp();
                    if (lane < pieces)
                        for (int b = 0; b < C::BLOCKS; ++b)
                            tma_2d(dst + b * C::BLOCK_BYTES + lane * p.box * 128, map, b * 64, row, mbar);
                } else if (lane == 0) {
                    mbar_arrive_tx(mbar, C::TILE_BYTES);
                    for (int b = 0; b < C::BLOCKS; ++b)
                        tma_3d(dst + b * C::BLOCK_BYTES, map, b * 64, h, (int)(job.t0 + (int64_t)j * kTile), mbar);
                }
                issued = it + 1;
            }
            if (ok && tail) {
                // the last tile's values behind the end
                const int it = 2 * count - 1, stage = it % C::STAGES, first = job.keys - (to - 1) * kTile;
                ok = mbar_wait_copies(smem_u32(&bars.full[stage]), (it / C::STAGES) & 1);
                if (ok) {
                    unsigned char* v = raw + (ring + stage * C::TILE_BYTES - smem_u32(raw));
                    for (int i = first * 8 + lane; i < kTile * 8; i += 32)
                        for (int b = 0; b < C::BLOCKS; ++b)
                            *reinterpret_cast<uint4*>(v + b * C::BLOCK_BYTES + i * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars.fixed));
                }
            }
            if (!ok) *abort = 1;
            // nothing may still be arriving when the CTA leaves
            for (int it = max(0, issued - C::STAGES); it < issued; ++it)
                if (!mbar_wait_copies(smem_u32(&bars.full[it % C::STAGES]), (it / C::STAGES) & 1)) *abort = 1;
            for (int t = 0; t < 2; ++t)
                if ((t ? to1 : to0) > from && !mbar_wait_copies(smem_u32(&bars.q[t]), 0)) *abort = 1;
        } else if (warp == 9) {
            // ---- MMAs ----
            if (lane == 0) {
                constexpr uint32_t idesc_s = idesc_bf16(kTile, kTile, false, false);
                constexpr uint32_t idesc_o = idesc_bf16(kTile, D, false, true);
                auto wait = [&](uint64_t* bar, int parity) {
                    const bool ok = mbar_spin(smem_u32(bar), parity & 1, abort);
                    if (!ok) *abort = 1;
                    return ok;
                };
                auto scores = [&](int t, int stage) {
                    const uint64_t q = smem_desc(q_smem + t * C::TILE_BYTES, 16, 1024, kSwizzle128);
                    const uint64_t k = smem_desc(ring + stage * C::TILE_BYTES, 16, 1024, kSwizzle128);
    #pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t off = (ks >> 2) * (C::BLOCK_BYTES / 16) + (ks & 3) * 2;
                        mma_bf16(tmem + C::S + t * kTile, q + off, k + off, idesc_s, ks > 0);
                    }
                    mma_commit(smem_u32(&bars.s[t]));
                };
                auto values = [&](int t, int stage, bool first) {
                    const uint64_t v = smem_desc(ring + stage * C::TILE_BYTES, C::BLOCK_BYTES, 1024, kSwizzle128);
    #pragma unroll
                    for (int ks = 0; ks < kTile / 16; ++ks)
                        mma_bf16_ta(tmem + C::O + t * D, tmem + C::S + t * kTile + ks * 8, v + ks * 128, idesc_o,
                                    !(first && ks == 0));
                };
                bool ok = count == 0 || wait(&bars.full[0], 0);
                for (int t = 0; t < 2 && ok; ++t)
                    if ((t ? to1 : to0) > from) {
                        ok = wait(&bars.q[t], 0);
                        if (ok) {
                            fence_after();
                            scores(t, 0);
                        }
                    }
                if (ok && count) mma_commit(smem_u32(&bars.empty[0]));
                for (int i = 0; i < count && ok; ++i) {
                    const int iv = 2 * i + 1, ik = 2 * i + 2, j = from + i;
                    ok = wait(&bars.full[iv % C::STAGES], iv / C::STAGES);
                    if (ok && i == count - 1 && tail) ok = wait(&bars.fixed, 0);
                    bool have_k = false;
                    for (int t = 0; t < 2 && ok; ++t) {
                        const int end = t ? to1 : to0;
                        if (j >= end) continue;
                        ok = wait(&bars.p[t], i);
                        if (!ok) break;
                        fence_after();
                        values(t, iv % C::STAGES, i == 0);
                        if (j + 1 < end) {
                            if (!have_k) ok = wait(&bars.full[ik % C::STAGES], ik / C::STAGES);
                            if (!ok) break;
                            have_k = true;
                            fence_after();
                            scores(t, ik % C::STAGES);
                        } else {
                            mma_commit(smem_u32(&bars.o[t]));
                        }
                    }
                    if (ok) {
                        mma_commit(smem_u32(&bars.empty[iv % C::STAGES]));
                        if (have_k) mma_commit(smem_u32(&bars.empty[ik % C::STAGES]));
                    }
                }
                // no MMA may still be running when tensor memory is given back
                mma_commit(smem_u32(&bars.drain));
                if (!mbar_wait_copies(smem_u32(&bars.drain), 0)) *abort = 1;
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kSoftmaxRegs));
        // ---- softmax: a row per thread ----
        const int t = warp >> 2, row = tid & 127, end = t ? to1 : to0;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // lane 32 (warp % 4) in the upper half
        const uint32_t ts = tmem + C::S + t * kTile + lanes, to_ = tmem + C::O + t * D + lanes;
        const int local = row / group + t * p.tokens;                // token within the CTA
        const int64_t token = job.i0 + local;                        // within the sequence
        const bool there = row < p.tokens * group && token < job.end;
        const int limit = !there ? 0x7fffffff : PREFIX ? limits[local] : (int)token + 1;
        const float c = a.scale_log2;
        float m = -INFINITY;
        float2 sum = make_float2(0.f, 0.f);
        bool ok = true;
        for (int j = from, i = 0; j < end; ++j, ++i) {
            ok = mbar_wait(smem_u32(&bars.s[t]), i & 1, abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                *abort = 1;
                break;
            }
            fence_after();
            float s[kTile];
#pragma unroll
            for (int b = 0; b < 4; ++b) tmem_fetch32(ts + b * 32, s + b * 32);
            tmem_wait_ld();
#pragma unroll
            for (int b = 0; b < 4; ++b) arrived32(s + b * 32);
            const int seen = limit - j * kTile;
            if (__any_sync(0xffffffffu, seen < kTile)) {
#pragma unroll
                for (int k = 0; k < kTile; ++k)
                    if (k >= seen) s[k] = -INFINITY;
            }
            if (PREFIX) {
                const uint32_t gone = missing[i & 15];
                if (gone) {
#pragma unroll
                    for (int k = 0; k < kTile; ++k)
                        if (gone >> (k / 16) & 1) s[k] = -INFINITY;
                }
            }
            float top = s[0];
#pragma unroll
            for (int k = 1; k < kTile; ++k) top = fmaxf(top, s[k]);
            top *= c;
            if (__any_sync(0xffffffffu, top > m + kLag)) {
                // to the new maximum where it has risen, by 1 where it has not
                const float now = fmaxf(top, m), back = now == -INFINITY ? 1.f : ex2(m - now);
                m = now;
                sum.x *= back;
                sum.y *= back;
                if (i > 0) {
#pragma unroll
                    for (int b = 0; b < D; b += 32) {
                        float o[32];
                        tmem_fetch32(to_ + b, o);
                        tmem_wait_ld();
                        arrived32(o);
                        uint32_t u[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(o[k] * back);
                        tmem_put32(to_ + b, u);
                    }
                }
            }
            const float base = m == -INFINITY ? 0.f : -m;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t pk[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const float2 x = __ffma2_rn(make_float2(s[b * 64 + 2 * k], s[b * 64 + 2 * k + 1]),
                                                make_float2(c, c), make_float2(base, base));
                    const float2 e = make_float2(ex2(x.x), ex2(x.y));
                    sum = __fadd2_rn(sum, e);
                    pk[k] = pack_bf16(e.x, e.y);
                }
                tmem_put32(ts + b * 32, pk);
            }
            tmem_wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars.p[t]));
        }
        if (end > from && ok) {
            ok = mbar_wait(smem_u32(&bars.o[t]), 0, abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) *abort = 1;
        }
        if (end > from && ok) {
            fence_after();
            float l = sum.x + sum.y;
            float o[D];
#pragma unroll
            for (int b = 0; b < D; b += 32) tmem_fetch32(to_ + b, o + b);
            tmem_wait_ld();
#pragma unroll
            for (int b = 0; b < D; b += 32) arrived32(o + b);
            const int64_t at = job.t0 + token;
            const int64_t head = (int64_t)h * group + row % group;
            float any = 0.f;
#pragma unroll
            for (int k = 0; k < D; ++k) any = fmaf(o[k], 0.f, any);  // 0 but for an infinity or a NaN
            const bool finite = any == 0.f && l < INFINITY && (PREFIX || l > 0.f);
            const int64_t place = ((int64_t)blockIdx.z * a.T + at) * a.Hq + head;  // PREFIX
            if (there && finite) {
                if (PREFIX) {
                    float* to_sum = p.w.far_sum + place * D;
#pragma unroll
                    for (int k = 0; k < D; k += 4) Vec<float, 4>::store(to_sum + k, o + k);
                    p.w.far_stat[place] = make_float2(m, l);
                } else {
                    const float inv = 1.f / l;
                    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o) + at * a.ldo + head * D;
#pragma unroll
                    for (int k = 0; k < D; k += 8) {
                        uint4 u;
                        u.x = pack_bf16(o[k] * inv, o[k + 1] * inv);
                        u.y = pack_bf16(o[k + 2] * inv, o[k + 3] * inv);
                        u.z = pack_bf16(o[k + 4] * inv, o[k + 5] * inv);
                        u.w = pack_bf16(o[k + 6] * inv, o[k + 7] * inv);
                        *reinterpret_cast<uint4*>(out + k) = u;
                    }
                }
            }
            // rows that an infinity or a NaN has reached, one after the other
            for (uint32_t bad = __ballot_sync(0xffffffffu, there && !finite); bad; bad &= bad - 1) {
                const int who = __ffs(bad) - 1;
                const int64_t at_w = __shfl_sync(0xffffffffu, at, who), head_w = __shfl_sync(0xffffffffu, head, who);
                const int64_t place_w = __shfl_sync(0xffffffffu, place, who);
                const int limit_w = __shfl_sync(0xffffffffu, limit, who);
                float acc[D / 32], mw, lw;
                // by value: what the call takes by reference would live in local memory
                const Paged cache = a.cache;
                const int Hkv = a.Hkv;
                const int64_t ldk = a.ldk, ldv = a.ldv;
                const __nv_bfloat16* keys = static_cast<const __nv_bfloat16*>(a.k) + job.t0 * ldk + (int64_t)h * D;
                const __nv_bfloat16* vals = static_cast<const __nv_bfloat16*>(a.v) + job.t0 * ldv + (int64_t)h * D;
                row_again<D>(static_cast<const __nv_bfloat16*>(a.q) + at_w * a.ldq + head_w * D, (int64_t)from * kTile,
                             min(limit_w, end * kTile), c,
                             [=](int64_t key, const __nv_bfloat16*& kp, const __nv_bfloat16*& vp) {
                                 if (PREFIX) return cached_row<D>(cache, cache.prefix, Hkv, h, key, kp, vp);
                                 kp = keys + key * ldk;
                                 vp = vals + key * ldv;
                                 return true;
                             }, acc, mw, lw);
                if (PREFIX) {
                    Vec<float, D / 32>::store(p.w.far_sum + place_w * D + lane * (D / 32), acc);
                    if (lane == 0) p.w.far_stat[place_w] = make_float2(mw, lw);
                } else {
                    const float inv = lw > 0.f ? 1.f / lw : lw == 0.f ? 0.f : lw;
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) acc[k] *= inv;
                    Vec<__nv_bfloat16, D / 32>::store(static_cast<__nv_bfloat16*>(a.o) + at_w * a.ldo + head_w * D +
                                                          lane * (D / 32), acc);
                }
            }
        }
    }
    fence_before();
    __syncwarp();
    __syncthreads();
    if (tid == 0 && abort_flag) atomicOr(p.err, kAttnError);
    if (warp == 9) {
        fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---- launches -----------------------------------------------------------------------

template <int D, bool PREFIX>
cudaError_t launch_tc(TcParams p, dim3 grid, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                      cudaStream_t s) {
    // at every call: the attribute belongs to the context
    const cudaError_t set = cudaFuncSetAttribute(attn_tc_kernel<D, PREFIX>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 Shape<D>::SMEM);
    if (set != cudaSuccess) return set;
    // a warpgroup that asks for more registers than the block was launched with waits forever
    static std::atomic<bool> enough{false};
    if (!enough.load(std::memory_order_relaxed)) {
        cudaFuncAttributes f;
        const cudaError_t got = cudaFuncGetAttributes(&f, attn_tc_kernel<D, PREFIX>);
        if (got != cudaSuccess) return got;
        if (f.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
        enough.store(true, std::memory_order_relaxed);
    }
    p.err = device_error_word();
    KernelTimer kt(PREFIX ? "attn_prefix_tc" : "attn_prompt_tc", s);
    attn_tc_kernel<D, PREFIX><<<grid, kWarps * 32, Shape<D>::SMEM, s>>>(p, mq, mk, mv);
    return cudaGetLastError();
}

}  // namespace

int prefix_tile_tokens(int group) { return kTile / group; }

cudaError_t launch_prompt_tc(const AttnArgs& a, cudaStream_t s) {
    TcParams p{};
    p.a = a;
    p.tokens = kTile / a.group;
    p.box = kTile;
    CUtensorMap mq, mk, mv;
    if (!encode_tokens(&mq, a.q, a.ldq, a.T, a.Hq, a.D, a.group, p.tokens) ||
        !encode_tokens(&mk, a.k, a.ldk, a.T, a.Hkv, a.D, 1, kTile) ||
        !encode_tokens(&mv, a.v, a.ldv, a.T, a.Hkv, a.D, 1, kTile))
        return cudaErrorInvalidValue;
    // a sequence's last CTA may be in part empty: one more for each
    const int64_t tiles = a.T / (2 * p.tokens) + (a.N < a.T ? a.N : a.T);
    const dim3 grid((unsigned)(tiles * a.Hkv));
    return a.D == 128 ? launch_tc<128, false>(p, grid, mq, mk, mv, s) : launch_tc<64, false>(p, grid, mq, mk, mv, s);
}

cudaError_t launch_prefix_tc(const AttnArgs& a, const StepWork& w, cudaStream_t s) {
    TcParams p{};
    p.a = a;
    p.w = w;
    p.tokens = kTile / a.group;
    p.box = a.cache.page_size < kTile ? a.cache.page_size : kTile;
    CUtensorMap mq, mk, mv;
    const int64_t rows = (int64_t)a.cache.num_pages * a.Hkv << a.cache.page_bits;
    if (!encode_tokens(&mq, a.q, a.ldq, a.T, a.Hq, a.D, a.group, p.tokens) ||
        !encode_cache(&mk, a.cache.k, rows, a.D, p.box) || !encode_cache(&mv, a.cache.v, rows, a.D, p.box))
        return cudaErrorInvalidValue;
    const int64_t tiles = (a.T + 2 * p.tokens - 1) / (2 * p.tokens);
    const dim3 grid((unsigned)tiles, a.Hkv, w.splits);
    return a.D == 128 ? launch_tc<128, true>(p, grid, mq, mk, mv, s) : launch_tc<64, true>(p, grid, mq, mk, mv, s);
}

}  // namespace gdr
