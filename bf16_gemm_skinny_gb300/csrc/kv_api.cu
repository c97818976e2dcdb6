// kv_api.cu -- the C entry points of the paged KV cache and of the attention
// over it: argument checks, workspace, launch, completion.  No compute here.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "bsk.h"
#include "bsk_internal.h"
#include "bsk_tuning.h"
#include "kv_internal.h"

namespace {

int fail(int status, const char* fmt, ...)
{
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    bsk::record_error(msg);
    return status;
}

// Stream-ordered workspace, freed in stream order after use.  From the library's
// pool: the default one gives its memory back at every synchronisation, and a
// blocking call would map it anew each time (some 200 us).  A capturing stream
// takes the default pool, whose allocations become nodes of the graph.
struct Workspace {
    void* ptr = nullptr;
    cudaStream_t s;
    explicit Workspace(cudaStream_t stream) : s(stream) {}
    Workspace(const Workspace&) = delete;
    Workspace& operator=(const Workspace&) = delete;
    ~Workspace()
    {
        if (ptr != nullptr) cudaFreeAsync(ptr, s);
    }
    cudaError_t take(size_t bytes)
    {
        const long long limit_kb = bsk_get_option(BSK_OPT_KV_WORKSPACE_KB);
        if (limit_kb > 0 && bytes > static_cast<unsigned long long>(limit_kb) * 1024ull) return cudaErrorMemoryAllocation;
        cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
        cudaError_t e = cudaStreamIsCapturing(s, &capture);
        cudaMemPool_t pool = nullptr;
        if (e == cudaSuccess) {
            if (capture != cudaStreamCaptureStatusNone || bsk::api_pool(&pool) != BSK_OK)
                e = cudaMallocAsync(&ptr, bytes, s);
            else
                e = cudaMallocFromPoolAsync(&ptr, bytes, pool, s);
        }
        if (e != cudaSuccess) {
            cudaGetLastError();
            ptr = nullptr;
        }
        return e;
    }
};

struct Span {
    const void* p;
    long long bytes;
};

bool overlap(const Span& a, const Span& b)
{
    if (a.p == nullptr || b.p == nullptr || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + static_cast<uintptr_t>(b.bytes) && b0 < a0 + static_cast<uintptr_t>(a.bytes);
}

bool unaligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// Bytes that `rows` rows of `width` 16-bit elements, `stride` elements apart, span.
long long row_bytes(long long rows, long long stride, long long width)
{
    return rows > 0 ? ((rows - 1) * stride + width) * 2 : 0;
}

long long cache_elems(const bsk::KvBatch& b)
{
    return static_cast<long long>(b.num_blocks) * b.block_size * b.num_kv_heads * b.head_dim;
}
Span cache_span(const bsk::KvBatch& b, const void* p)
{
    return {p, cache_elems(b) * (b.type == bsk::kCacheBF16 ? 2 : 1)};
}
Span scale_span(const bsk::KvBatch& b, const void* p) { return {p, cache_elems(b) / b.head_dim}; }

// The checks that all four calls share.  BSK_OK with *empty set: nothing to do.
int check_batch(const bsk::KvBatch& b, bool* empty)
{
    *empty = false;
    if (b.type != BSK_CACHE_BF16 && b.type != BSK_CACHE_E4M3)
        return fail(BSK_ERR_INVALID_ARG, "unknown cache_type %d", b.type);
    if (b.num_seqs < 0 || b.num_tokens < 0 || b.num_kv_heads <= 0 || b.block_size <= 0 || b.max_blocks <= 0 ||
        b.num_blocks <= 0)
        return fail(BSK_ERR_INVALID_ARG, "bad cache sizes (seqs=%d tokens=%d kv_heads=%d block_size=%d max_blocks=%d "
                    "num_blocks=%d)", b.num_seqs, b.num_tokens, b.num_kv_heads, b.block_size, b.max_blocks,
                    b.num_blocks);
    if (b.head_dim != 64 && b.head_dim != 128 && b.head_dim != 256)
        return fail(BSK_ERR_INVALID_ARG, "head_dim must be 64, 128 or 256 (got %d)", b.head_dim);
    if (b.num_seqs > 65535 || b.num_kv_heads > 65535)
        return fail(BSK_ERR_INVALID_ARG, "num_seqs and num_kv_heads must be at most 65535");
    if (static_cast<long long>(b.num_blocks) * b.block_size > INT_MAX)
        return fail(BSK_ERR_INVALID_ARG, "num_blocks * block_size exceeds 2^31 - 1 tokens");
    if (b.cu_tokens == nullptr && b.num_tokens != b.num_seqs)
        return fail(BSK_ERR_INVALID_ARG, "without cu_tokens there is one new token per sequence (%d tokens, %d "
                    "sequences)", b.num_tokens, b.num_seqs);
    if (b.num_seqs == 0 || b.num_tokens == 0) {
        *empty = true;
        return BSK_OK;
    }
    if (!b.k || !b.v || !b.block_tables || !b.seq_lens)
        return fail(BSK_ERR_INVALID_ARG, "a pointer argument is NULL");
    if (unaligned16(b.k) || unaligned16(b.v))
        return fail(BSK_ERR_INVALID_ARG, "k_cache and v_cache must be 16-byte aligned");
    if (b.type == BSK_CACHE_E4M3 && (!b.k_scales || !b.v_scales))
        return fail(BSK_ERR_INVALID_ARG, "an E4M3 cache needs k_scales and v_scales");
    if (b.type == BSK_CACHE_BF16 && (b.k_scales || b.v_scales))
        return fail(BSK_ERR_INVALID_ARG, "a BF16 cache has no scales: pass NULL");
    return BSK_OK;
}

int check_rows(const char* name, const void* p, long long stride, long long width)
{
    if (p == nullptr) return fail(BSK_ERR_INVALID_ARG, "%s is NULL", name);
    if (unaligned16(p)) return fail(BSK_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
    if (stride < width || stride % 8 != 0)
        return fail(BSK_ERR_INVALID_ARG, "the stride of %s (%lld) must be a multiple of 8 and at least %lld", name,
                    stride, width);
    return BSK_OK;
}

bsk::KvBatch make_batch(int cache_type, const void* k_cache, const void* v_cache, const uint8_t* k_scales,
                        const uint8_t* v_scales, const int32_t* cu_tokens, const int32_t* block_tables,
                        const int32_t* seq_lens, int num_seqs, int num_tokens, int num_kv_heads, int head_dim,
                        int block_size, int max_blocks, int num_blocks)
{
    bsk::KvBatch b;
    b.type = cache_type;
    b.k = const_cast<void*>(k_cache);
    b.v = const_cast<void*>(v_cache);
    b.k_scales = const_cast<uint8_t*>(k_scales);
    b.v_scales = const_cast<uint8_t*>(v_scales);
    b.cu_tokens = cu_tokens;
    b.block_tables = block_tables;
    b.seq_lens = seq_lens;
    b.num_seqs = num_seqs;
    b.num_tokens = num_tokens;
    b.num_kv_heads = num_kv_heads;
    b.head_dim = head_dim;
    b.block_size = block_size;
    b.max_blocks = max_blocks;
    b.num_blocks = num_blocks;
    return b;
}

int enqueue_append(bsk::KvCopyLaunch& a, cudaStream_t s)
{
    bool empty = false;
    int st = check_batch(a.b, &empty);
    if (st != BSK_OK || empty) return st;
    const bsk::KvBatch& b = a.b;
    const long long width = static_cast<long long>(b.num_kv_heads) * b.head_dim;
    if ((st = check_rows("k", a.k_in, a.k_stride, width)) != BSK_OK) return st;
    if ((st = check_rows("v", a.v_in, a.v_stride, width)) != BSK_OK) return st;
    const Span in[2] = {{a.k_in, row_bytes(b.num_tokens, a.k_stride, width)},
                        {a.v_in, row_bytes(b.num_tokens, a.v_stride, width)}};
    const Span out[4] = {cache_span(b, b.k), cache_span(b, b.v), scale_span(b, b.k_scales),
                         scale_span(b, b.v_scales)};
    for (int i = 0; i < 4; ++i) {
        for (const Span& x : in)
            if (overlap(out[i], x)) return fail(BSK_ERR_INVALID_ARG, "the cache overlaps k or v");
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return fail(BSK_ERR_INVALID_ARG, "the parts of the cache overlap");
    }
    if ((st = bsk::api_prepare(&a.num_sms, &a.b.status)) != BSK_OK) return st;
    a.pdl = bsk_get_option(BSK_OPT_PDL) != 1;
    char msg[256] = "";
    if (bsk::launch_kv_append(a, s, msg, sizeof(msg))) return fail(BSK_ERR_CUDA, "%s", msg);
    return BSK_OK;
}

int enqueue_gather(bsk::KvCopyLaunch& a, cudaStream_t s)
{
    bool empty = false;
    int st = check_batch(a.b, &empty);
    if (st != BSK_OK || empty) return st;
    const bsk::KvBatch& b = a.b;
    const long long width = static_cast<long long>(b.num_kv_heads) * b.head_dim;
    a.k_stride = a.v_stride = width;
    if ((st = check_rows("k_out", a.k_out, width, width)) != BSK_OK) return st;
    if ((st = check_rows("v_out", a.v_out, width, width)) != BSK_OK) return st;
    const Span out[2] = {{a.k_out, row_bytes(b.num_tokens, width, width)},
                         {a.v_out, row_bytes(b.num_tokens, width, width)}};
    const Span in[4] = {cache_span(b, b.k), cache_span(b, b.v), scale_span(b, b.k_scales), scale_span(b, b.v_scales)};
    if (overlap(out[0], out[1])) return fail(BSK_ERR_INVALID_ARG, "k_out overlaps v_out");
    for (const Span& x : in)
        if (overlap(out[0], x) || overlap(out[1], x)) return fail(BSK_ERR_INVALID_ARG, "an output overlaps the cache");
    if ((st = bsk::api_prepare(&a.num_sms, &a.b.status)) != BSK_OK) return st;
    a.pdl = bsk_get_option(BSK_OPT_PDL) != 1;
    char msg[256] = "";
    if (bsk::launch_kv_gather(a, s, msg, sizeof(msg))) return fail(BSK_ERR_CUDA, "%s", msg);
    return BSK_OK;
}

void plan_attention(bsk::KvAttnLaunch& a, int num_segments)
{
    bsk::kv_attention_limit(a);
    a.kernel = static_cast<int>(bsk_get_option(BSK_OPT_KV_KERNEL));
    a.segments = num_segments > 0 ? num_segments : bsk::kv_attention_segments(a);
}

int enqueue_attention(bsk::KvAttnLaunch& a, int num_segments, cudaStream_t s)
{
    bool empty = false;
    int st = check_batch(a.b, &empty);
    if (st != BSK_OK) return st;
    const bsk::KvBatch& b = a.b;
    if (a.num_q_heads <= 0 || a.num_q_heads % b.num_kv_heads != 0)
        return fail(BSK_ERR_INVALID_ARG, "num_q_heads (%d) is not a positive multiple of num_kv_heads (%d)",
                    a.num_q_heads, b.num_kv_heads);
    if (a.max_chunk <= 0 && !empty) return fail(BSK_ERR_INVALID_ARG, "max_chunk must be positive (got %d)", a.max_chunk);
    if (a.max_seq_len < 0 || static_cast<long long>(a.max_seq_len) > static_cast<long long>(b.max_blocks) * b.block_size)
        return fail(BSK_ERR_INVALID_ARG, "max_seq_len %d is negative or exceeds max_blocks * block_size", a.max_seq_len);
    if (a.max_seq_len > INT_MAX - 255)   // whole tiles of positions are counted in 32 bits
        return fail(BSK_ERR_INVALID_ARG, "max_seq_len %d exceeds 2^31 - 256", a.max_seq_len);
    if (!std::isfinite(a.scale * 1.4426950408889634f))   // the kernels' factor, for powers of two
        return fail(BSK_ERR_INVALID_ARG, "softmax_scale must be finite, and so must softmax_scale * log2(e)");
    if (a.window < 0 || a.sinks < 0)
        return fail(BSK_ERR_INVALID_ARG, "window (%d) and sinks (%d) must not be negative", a.window, a.sinks);
    if (num_segments < 0 || num_segments > 256)
        return fail(BSK_ERR_INVALID_ARG, "num_segments %d out of range (0 = automatic, else 1..256)", num_segments);
    if (empty) return BSK_OK;
    const long long width = static_cast<long long>(a.num_q_heads) * b.head_dim;
    if ((st = check_rows("q", a.q, a.q_stride, width)) != BSK_OK) return st;
    if ((st = check_rows("out", a.out, a.out_stride, width)) != BSK_OK) return st;
    if (static_cast<long long>(b.num_tokens) * a.num_q_heads > INT_MAX)
        return fail(BSK_ERR_INVALID_ARG, "num_tokens * num_q_heads exceeds 2^31 - 1");
    const Span out = {a.out, row_bytes(b.num_tokens, a.out_stride, width)};
    const Span in[5] = {{a.q, row_bytes(b.num_tokens, a.q_stride, width)}, cache_span(b, b.k), cache_span(b, b.v),
                        scale_span(b, b.k_scales), scale_span(b, b.v_scales)};
    for (const Span& x : in)
        if (overlap(out, x)) return fail(BSK_ERR_INVALID_ARG, "out overlaps an input");
    if ((st = bsk::api_prepare(&a.num_sms, &a.b.status)) != BSK_OK) return st;
    const long long limit_us = bsk_get_option(BSK_OPT_WAIT_LIMIT_US);
    if (limit_us > 0) a.wait_limit_ns = static_cast<unsigned long long>(limit_us) * 1000ull;
    a.pdl = bsk_get_option(BSK_OPT_PDL) != 1;
    plan_attention(a, num_segments);
    Workspace ws(s);
    size_t bytes = bsk::kv_attention_workspace(a);
    cudaError_t e = bytes > 0 ? ws.take(bytes) : cudaSuccess;
    // The flat copy and segments of the library's own choice are for speed: without room
    // for them the cache is converted tile by tile, and read in one segment.
    if (e == cudaErrorMemoryAllocation && bsk::kv_attention_plan(a).flat_rows > 0) {
        a.flat_copy = false;
        plan_attention(a, num_segments);
        bytes = bsk::kv_attention_workspace(a);
        e = bytes > 0 ? ws.take(bytes) : cudaSuccess;
    }
    if (e == cudaErrorMemoryAllocation && num_segments == 0) {
        a.segments = 1;
        bytes = 0;
        e = cudaSuccess;
    }
    if (e != cudaSuccess)
        return fail(BSK_ERR_NO_MEMORY, "cudaMallocAsync(%zu bytes) for a workspace failed: %s", bytes,
                    cudaGetErrorString(e));
    a.workspace = static_cast<float*>(ws.ptr);
    char msg[512] = "";
    if (bsk::launch_kv_attention(a, s, msg, sizeof(msg))) return fail(BSK_ERR_CUDA, "%s", msg);
    return BSK_OK;
}

}  // namespace

extern "C" {

int bsk_kv_cache_append_enqueue(int cache_type, void* k_cache, void* v_cache, uint8_t* k_scales, uint8_t* v_scales,
                                const uint16_t* k, int k_stride, const uint16_t* v, int v_stride,
                                const int32_t* cu_tokens, const int32_t* block_tables, const int32_t* seq_lens,
                                int num_seqs, int num_tokens, int num_kv_heads, int head_dim, int block_size,
                                int max_blocks, int num_blocks, void* stream)
{
    bsk::KvCopyLaunch a;
    a.b = make_batch(cache_type, k_cache, v_cache, k_scales, v_scales, cu_tokens, block_tables, seq_lens, num_seqs,
                     num_tokens, num_kv_heads, head_dim, block_size, max_blocks, num_blocks);
    a.k_in = k;
    a.v_in = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    return enqueue_append(a, static_cast<cudaStream_t>(stream));
}

int kv_cache_append(int cache_type, void* k_cache, void* v_cache, uint8_t* k_scales, uint8_t* v_scales,
                    const uint16_t* k, int k_stride, const uint16_t* v, int v_stride, const int32_t* cu_tokens,
                    const int32_t* block_tables, const int32_t* seq_lens, int num_seqs, int num_tokens,
                    int num_kv_heads, int head_dim, int block_size, int max_blocks, int num_blocks, void* stream)
{
    const int st = bsk_kv_cache_append_enqueue(cache_type, k_cache, v_cache, k_scales, v_scales, k, k_stride, v,
                                               v_stride, cu_tokens, block_tables, seq_lens, num_seqs, num_tokens,
                                               num_kv_heads, head_dim, block_size, max_blocks, num_blocks, stream);
    if (st != BSK_OK || num_seqs == 0 || num_tokens == 0) return st;
    return bsk::api_sync_and_check(static_cast<cudaStream_t>(stream));
}

int bsk_kv_cache_gather_enqueue(int cache_type, const void* k_cache, const void* v_cache, const uint8_t* k_scales,
                                const uint8_t* v_scales, uint16_t* k_out, uint16_t* v_out, const int32_t* cu_tokens,
                                const int32_t* block_tables, const int32_t* seq_lens, int num_seqs, int num_tokens,
                                int num_kv_heads, int head_dim, int block_size, int max_blocks, int num_blocks,
                                void* stream)
{
    bsk::KvCopyLaunch a;
    a.b = make_batch(cache_type, k_cache, v_cache, k_scales, v_scales, cu_tokens, block_tables, seq_lens, num_seqs,
                     num_tokens, num_kv_heads, head_dim, block_size, max_blocks, num_blocks);
    a.k_out = k_out;
    a.v_out = v_out;
    return enqueue_gather(a, static_cast<cudaStream_t>(stream));
}

int kv_cache_gather(int cache_type, const void* k_cache, const void* v_cache, const uint8_t* k_scales,
                    const uint8_t* v_scales, uint16_t* k_out, uint16_t* v_out, const int32_t* cu_tokens,
                    const int32_t* block_tables, const int32_t* seq_lens, int num_seqs, int num_tokens,
                    int num_kv_heads, int head_dim, int block_size, int max_blocks, int num_blocks, void* stream)
{
    const int st = bsk_kv_cache_gather_enqueue(cache_type, k_cache, v_cache, k_scales, v_scales, k_out, v_out,
                                               cu_tokens, block_tables, seq_lens, num_seqs, num_tokens, num_kv_heads,
                                               head_dim, block_size, max_blocks, num_blocks, stream);
    if (st != BSK_OK || num_seqs == 0 || num_tokens == 0) return st;
    return bsk::api_sync_and_check(static_cast<cudaStream_t>(stream));
}

int bsk_chunk_attention_enqueue(int cache_type, const void* k_cache, const void* v_cache, const uint8_t* k_scales,
                                const uint8_t* v_scales, const uint16_t* q, int q_stride, uint16_t* out,
                                int out_stride, const int32_t* cu_tokens, const int32_t* block_tables,
                                const int32_t* seq_lens, int num_seqs, int num_tokens, int max_chunk,
                                int num_q_heads, int num_kv_heads, int head_dim, int block_size, int max_blocks,
                                int num_blocks, int max_seq_len, float softmax_scale, int window, int sinks,
                                int num_segments, void* stream)
{
    bsk::KvAttnLaunch a;
    a.b = make_batch(cache_type, k_cache, v_cache, k_scales, v_scales, cu_tokens, block_tables, seq_lens, num_seqs,
                     num_tokens, num_kv_heads, head_dim, block_size, max_blocks, num_blocks);
    a.q = q;
    a.q_stride = q_stride;
    a.out = out;
    a.out_stride = out_stride;
    a.max_chunk = max_chunk;
    a.num_q_heads = num_q_heads;
    a.max_seq_len = max_seq_len;
    a.scale = softmax_scale;
    a.window = window;
    a.sinks = sinks;
    return enqueue_attention(a, num_segments, static_cast<cudaStream_t>(stream));
}

int chunk_attention(int cache_type, const void* k_cache, const void* v_cache, const uint8_t* k_scales,
                    const uint8_t* v_scales, const uint16_t* q, int q_stride, uint16_t* out, int out_stride,
                    const int32_t* cu_tokens, const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                    int num_tokens, int max_chunk, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                    int max_blocks, int num_blocks, int max_seq_len, float softmax_scale, int window, int sinks,
                    int num_segments, void* stream)
{
    const int st = bsk_chunk_attention_enqueue(cache_type, k_cache, v_cache, k_scales, v_scales, q, q_stride, out,
                                               out_stride, cu_tokens, block_tables, seq_lens, num_seqs, num_tokens,
                                               max_chunk, num_q_heads, num_kv_heads, head_dim, block_size,
                                               max_blocks, num_blocks, max_seq_len, softmax_scale, window, sinks,
                                               num_segments, stream);
    if (st != BSK_OK || num_seqs == 0 || num_tokens == 0) return st;
    return bsk::api_sync_and_check(static_cast<cudaStream_t>(stream));
}

int bsk_decode_attention_enqueue(int cache_type, const void* k_cache, const void* v_cache, const uint8_t* k_scales,
                                 const uint8_t* v_scales, const uint16_t* q, int q_stride, uint16_t* out,
                                 int out_stride, const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                                 int num_q_heads, int num_kv_heads, int head_dim, int block_size, int max_blocks,
                                 int num_blocks, int max_seq_len, float softmax_scale, int window, int sinks,
                                 int num_segments, void* stream)
{
    return bsk_chunk_attention_enqueue(cache_type, k_cache, v_cache, k_scales, v_scales, q, q_stride, out, out_stride,
                                       nullptr, block_tables, seq_lens, num_seqs, num_seqs, 1, num_q_heads,
                                       num_kv_heads, head_dim, block_size, max_blocks, num_blocks, max_seq_len,
                                       softmax_scale, window, sinks, num_segments, stream);
}

int decode_attention(int cache_type, const void* k_cache, const void* v_cache, const uint8_t* k_scales,
                     const uint8_t* v_scales, const uint16_t* q, int q_stride, uint16_t* out, int out_stride,
                     const int32_t* block_tables, const int32_t* seq_lens, int num_seqs, int num_q_heads,
                     int num_kv_heads, int head_dim, int block_size, int max_blocks, int num_blocks,
                     int max_seq_len, float softmax_scale, int window, int sinks, int num_segments, void* stream)
{
    return chunk_attention(cache_type, k_cache, v_cache, k_scales, v_scales, q, q_stride, out, out_stride, nullptr,
                           block_tables, seq_lens, num_seqs, num_seqs, 1, num_q_heads, num_kv_heads, head_dim,
                           block_size, max_blocks, num_blocks, max_seq_len, softmax_scale, window, sinks,
                           num_segments, stream);
}

int bsk_plan_kv_attention(int cache_type, int one_token_each, int num_seqs, int num_tokens, int max_chunk,
                          int num_q_heads, int num_kv_heads, int head_dim, int max_seq_len, int window, int sinks,
                          int num_segments, int sms, int* plan)
{
    if (plan == nullptr || num_seqs < 1 || num_tokens < 1 || max_chunk < 1 || num_kv_heads < 1 ||
        num_q_heads < num_kv_heads || head_dim < 1 || max_seq_len < 0 || window < 0 || sinks < 0 || num_segments < 0 ||
        sms < 1)
        return fail(BSK_ERR_INVALID_ARG, "plan query: sizes and SM count must be positive, plan non-NULL");
    static const int32_t some = 0;   // stands for a prefix sum; not read
    bsk::KvAttnLaunch a;
    a.b = make_batch(cache_type, nullptr, nullptr, nullptr, nullptr, one_token_each ? nullptr : &some, nullptr, nullptr,
                     num_seqs, num_tokens, num_kv_heads, head_dim, 1, 1, 1);
    a.max_chunk = max_chunk;
    a.num_q_heads = num_q_heads;
    a.max_seq_len = max_seq_len;
    a.window = window;
    a.sinks = sinks;
    a.num_sms = sms;
    plan_attention(a, num_segments);
    const bsk::KvAttnPlan p = bsk::kv_attention_plan(a);
    plan[0] = p.cta_rows;
    plan[1] = p.tiles;
    plan[2] = p.segments;
    plan[3] = p.flat_rows;
    return BSK_OK;
}

}  // extern "C"
