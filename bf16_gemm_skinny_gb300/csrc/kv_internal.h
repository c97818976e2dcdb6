// kv_internal.h -- the paged key/value cache as the cache and attention kernels
// see it: where a token's row lies, what an E4M3 row's scale byte stands for,
// and the launchers of kv_cache.cu and kv_attention.cu (not part of the C ABI).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace bsk {

// Codes a kernel writes into the device status word (beside those of
// bsk_internal.h): a sequence brings more new tokens than the caller's bound.
constexpr int kDevErrChunkTooLong = 0x201;

enum CacheType : int { kCacheBF16 = 0, kCacheE4M3 = 1 };

// A paged cache and a batch over it.
//   k, v            [num_blocks, block_size, num_kv_heads, head_dim] BF16 or E4M3
//   k_scales, ...   [num_blocks, block_size, num_kv_heads] E8M0 (E4M3 caches only)
//   block_tables    [num_seqs, max_blocks];  seq_lens [num_seqs], new tokens included
//   cu_tokens       [num_seqs + 1]: the new tokens of sequence s are cu_tokens[s] ..
//                   cu_tokens[s+1]-1 and its last ones; nullptr: one token per sequence
struct KvBatch {
    void* k = nullptr;
    void* v = nullptr;
    uint8_t* k_scales = nullptr;
    uint8_t* v_scales = nullptr;
    const int32_t* cu_tokens = nullptr;
    const int32_t* block_tables = nullptr;
    const int32_t* seq_lens = nullptr;
    int type = kCacheBF16;
    int num_seqs = 0, num_tokens = 0;
    int num_kv_heads = 0, head_dim = 0, block_size = 0, max_blocks = 0, num_blocks = 0;
    // > 0: k and v are not the pages but copies of their positions, position t of
    // sequence s in row s * flat_len + t (the block table still says which exist)
    int flat_len = 0;
    int* status = nullptr;
};

struct KvCopyLaunch {
    KvBatch b;
    // append: sources; gather: destinations (BF16, elements between tokens in *_stride)
    const uint16_t* k_in = nullptr;
    const uint16_t* v_in = nullptr;
    uint16_t* k_out = nullptr;
    uint16_t* v_out = nullptr;
    long long k_stride = 0, v_stride = 0;
    int num_sms = 1;
    bool pdl = true;
};
int launch_kv_append(const KvCopyLaunch& a, cudaStream_t stream, char* msg, size_t msg_len);
int launch_kv_gather(const KvCopyLaunch& a, cudaStream_t stream, char* msg, size_t msg_len);
// The positions of an E4M3 cache that the new tokens see, as BF16 in the layout of
// KvBatch::flat_len.
int launch_kv_flatten(const KvBatch& b, uint16_t* k_out, uint16_t* v_out, int flat_len, int max_seq_len, int window,
                      int sinks, bool pdl, cudaStream_t stream, char* msg, size_t msg_len);

struct KvAttnLaunch {
    KvBatch b;
    const uint16_t* q = nullptr;   // [num_tokens, num_q_heads, head_dim], q_stride elements between tokens
    uint16_t* out = nullptr;       // the same shape, out_stride elements between tokens
    long long q_stride = 0, out_stride = 0;
    int num_q_heads = 0;
    int max_chunk = 1;             // most new tokens of a sequence
    int max_seq_len = 0;
    float scale = 1.f;
    int window = 0, sinks = 0;     // window 0: every earlier position is visible
    int kernel = 0;                // 0 automatic, 1 many rows (tcgen05), 2 few rows
    int segments = 1;              // kv_attention_segments()
    bool flat_copy = true;         // false: no flat copy of an E4M3 cache (no memory for it)
    float* workspace = nullptr;    // kv_attention_workspace() bytes, or nullptr when that is 0
    int num_sms = 1;
    unsigned long long wait_limit_ns = 2000000000ull;
    bool pdl = true;
};
// The caller's bounds as far as the batch can reach: a sequence brings no more new
// tokens than there are (without cu_tokens: one).  max_chunk decides the kernel, the
// grid and the flat copy, and row numbers up to max_chunk * (query heads per KV head)
// are 32-bit in the kernels; num_tokens * num_q_heads is known to fit.
void kv_attention_limit(KvAttnLaunch& a);
// What the call launches (for the planner hook).
struct KvAttnPlan {
    int cta_rows = 0;    // query rows per CTA
    int tiles = 0;       // CTAs' row tiles per sequence and KV head
    int segments = 1;
    int flat_rows = 0;   // rows per sequence of the flat copy, or 0
};
KvAttnPlan kv_attention_plan(const KvAttnLaunch& a);
// Segments that a call without a choice of its own splits the keys into (>= 1).
int kv_attention_segments(const KvAttnLaunch& a);
size_t kv_attention_workspace(const KvAttnLaunch& a);
int launch_kv_attention(const KvAttnLaunch& a, cudaStream_t stream, char* msg, size_t msg_len);

// What the entry points of kv_api.cu share with api.cu: the device check (sets
// the SM count and the device status word), the status of a finished stream.
int api_prepare(int* sms, int** status);
int api_sync_and_check(cudaStream_t s);
// The library's own memory pool of the current device, which keeps its memory
// mapped when a stream is synchronised (up to 2 GiB).
int api_pool(cudaMemPool_t* pool);

#ifdef __CUDACC__

// 2^(b - 127), the value of the E8M0 byte b; NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t b)
{
    return __uint_as_float(b == 255u ? 0x7FC00000u : (b == 0u ? 0x00400000u : b << 23));
}

// Row of the cache that holds position `pos` of the sequence whose block table
// is `table`: block * block_size + slot (or its row in a flat copy), or -1 (and a status code) when the
// table does not reach that far or its entry is no block.
__device__ __forceinline__ long long kv_row(const KvBatch& b, const int32_t* table, int pos)
{
    const int i = pos / b.block_size;
    if (i < b.max_blocks) {
        const int blk = table[i];
        if (blk >= 0 && blk < b.num_blocks && b.flat_len > 0)
            return (table - b.block_tables) / b.max_blocks * b.flat_len + pos;
        if (blk >= 0 && blk < b.num_blocks)
            return static_cast<long long>(blk) * b.block_size + (pos - i * b.block_size);
    }
    *reinterpret_cast<volatile int*>(b.status) = 0x200;   // kDevErrBadIndex
    return -1;
}

// Whole warp: the sequence that new token `t` belongs to (num_seqs if none):
// the number of ends cu_tokens[1..] at or before t, found 32 at a time.
__device__ __forceinline__ int kv_sequence_of(const KvBatch& b, int t)
{
    if (b.cu_tokens == nullptr) return t;
    const int lane = threadIdx.x & 31;
    int lo = 0, n = b.num_seqs;
    while (n > 0) {
        const int step = (n + 31) / 32;
        const int i = (lane + 1) * step - 1;
        const bool before = i < n && b.cu_tokens[lo + i + 1] <= t;
        const int c = __popc(__ballot_sync(0xffffffffu, before));
        lo += c * step;
        const int left = n - c * step;
        n = step - 1 < left ? step - 1 : left;
    }
    return lo;
}

#endif

}  // namespace bsk
