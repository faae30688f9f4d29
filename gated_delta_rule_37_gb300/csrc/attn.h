// Internal interface of the attention layer's translation units: the paged
// cache (kv.cu), the argument checks and entry points (attn.cu), the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace gdr {

// A pair of paged caches and the sequences' pages.
struct Paged {
    void* k;  // [num_pages, Hkv, page_size, D]
    void* v;
    const int32_t* table;  // [N, max_pages], row stride table_ld
    int64_t table_ld;
    const int32_t* lens;    // [N] tokens in the cache before the call's; < 0: padding
    const int32_t* prefix;  // pages of the first prefix_len keys (nullptr: none)
    int prefix_len;
    int max_pages, num_pages, page_size, page_bits;  // page_size = 1 << page_bits
};

struct AttnArgs {
    const void* q;
    const void* k;  // packed keys and values (gdr_attn_fwd)
    const void* v;
    void* o;
    int64_t ldq, ldk, ldv, ldo;  // elements from one token to the next
    const int32_t* cu;
    int N, Hq, Hkv, D, group;  // group = Hq / Hkv
    int64_t T;
    float scale_log2;  // scale * log2(e): scores are kept in log2 units
    int dtype;
    Paged cache;  // gdr_attn_step
};

// The checks that every call of the layer makes; GDR_OK or a status with its message set.
int check_heads(int N, int64_t T, int Hq, int Hkv, int D, int dtype);
int check_token_rows(const char* name, const void* p, int64_t stride, int64_t least, int dtype);
int check_int32s(const char* name, const void* p);
int check_paged(const Paged& c, int N, int Hkv, int D, int dtype);

// Rows in memory: `rows` of them, `row` bytes each, `ld` bytes from one to the next.
struct MemRows {
    const char* name;
    const void* p;
    int64_t row, ld, rows;
};
// GDR_OK if what is written shares no byte with the other (column blocks of the same rows do
// not), else a status with its message set.  A null pointer shares nothing.
int check_apart(const MemRows& written, const MemRows& other);

// GDR_VALIDATE of the layer: cu_seqlens, and where `c` is given that every page
// that the call reaches is there.  Synchronises the stream.
int validate_attention(const int32_t* cu, int N, int64_t T, const Paged* c, cudaStream_t s);

struct StepWork;

// A number of the current context that no other one of this process has; 0 if there is none.
uint64_t context_number();

// Allows `kernel` its dynamic shared memory.  The attribute belongs to the context, and setting
// it costs a fifth of a launch: `known` (one per kernel) keeps the context that has it.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t>& known) {
    const uint64_t now = context_number();
    if (now != 0 && known.load(std::memory_order_relaxed) == now) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) known.store(now, std::memory_order_relaxed);
    return e;
}

// Tensor-core paths (bf16).
cudaError_t launch_prompt_tc(const AttnArgs& a, cudaStream_t s);
int prefix_block_tokens(int group);  // tokens of a block of rows of the prefix's kernel
cudaError_t launch_prefix_tc(const AttnArgs& a, const StepWork& w, cudaStream_t s);
cudaError_t launch_step_own(const AttnArgs& a, const StepWork& w, cudaStream_t s);

// The own keys' part in fp32 for w.rows 4 or 8.
cudaError_t launch_step_few(const AttnArgs& a, const StepWork& w, cudaStream_t s);

}  // namespace gdr
