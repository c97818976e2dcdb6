// kv_attention.cu -- attention of new tokens over the paged cache.
#include <cmath>
#include <cstdio>

#include "bsk_internal.h"
#include "kv_internal.h"

namespace bsk {
namespace {

struct RowParams {
    KvBatch b;
    const uint16_t* q;
    uint16_t* out;
    long long q_stride, out_stride;
    int num_q_heads, group, max_chunk, max_seq_len;
    float scale_log2;   // softmax scale * log2(e)
    int window, sinks;
};

// EPL values of one lane's slice of a cache row.
template <bool E4M3, int EPL>
__device__ __forceinline__ void load_slice(const void* cache, long long elem, float (&f)[EPL])
{
    if constexpr (E4M3) {
        const uint8_t* c = static_cast<const uint8_t*>(cache) + elem;
#pragma unroll
        for (int i = 0; i < EPL; i += 2) {
            const uint16_t two = *reinterpret_cast<const uint16_t*>(c + i);
            uint32_t h;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
            asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
                : "=f"(f[i]), "=f"(f[i + 1])
                : "r"(h));
        }
    } else {
        const uint16_t* c = static_cast<const uint16_t*>(cache) + elem;
#pragma unroll
        for (int i = 0; i < EPL; i += 2) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(c + i);
            f[i] = __uint_as_float(w << 16);
            f[i + 1] = __uint_as_float(w & 0xffff0000u);
        }
    }
}

// One warp, one query row: adds the positions [t0, t1) to the running maximum
// m (of scale * log2 e * q.k), sum l and unnormalised output o, in FP32.
template <bool E4M3, int HD>
__device__ __forceinline__ void row_add(const KvBatch& b, const int32_t* table, int kvh, const float (&q)[HD / 32],
                                        float scale_log2, int t0, int t1, float& m, float& l, float (&o)[HD / 32])
{
    constexpr int EPL = HD / 32;
    const int lane = threadIdx.x & 31;
    for (int t = t0; t < t1; ++t) {
        const long long row = kv_row(b, table, t);
        if (row < 0) continue;
        const long long hr = row * b.num_kv_heads + kvh;
        float k[EPL], v[EPL];
        load_slice<E4M3, EPL>(b.k, hr * HD + lane * EPL, k);
        load_slice<E4M3, EPL>(b.v, hr * HD + lane * EPL, v);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
        if constexpr (E4M3) s *= e8m0_value(b.k_scales[hr]);
        s *= scale_log2;
        const float vs = E4M3 ? e8m0_value(b.v_scales[hr]) : 1.f;
        const float mn = fmaxf(m, s);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float corr = exp2f(m - base);   // m = -inf: 0
        const float w = exp2f(s - base);      // s = NaN or +inf: NaN
        l = l * corr + w;
        m = mn;
#pragma unroll
        for (int i = 0; i < EPL; ++i) o[i] = o[i] * corr + w * (v[i] * vs);
    }
}

template <bool E4M3, int HD>
__global__ void __launch_bounds__(256) kv_attention_row_kernel(const RowParams p)
{
    constexpr int EPL = HD / 32;
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int t = static_cast<int>(w / p.num_q_heads);
    const int h = static_cast<int>(w - static_cast<long long>(t) * p.num_q_heads);
    griddep_wait();
    griddep_launch_dependents();
    if (t >= p.b.num_tokens) return;
    const int s = kv_sequence_of(p.b, t);
    if (s >= p.b.num_seqs) return;
    const int first = p.b.cu_tokens != nullptr ? p.b.cu_tokens[s] : t;
    const int end = p.b.cu_tokens != nullptr ? p.b.cu_tokens[s + 1] : t + 1;
    if (end - first > p.max_chunk && lane == 0)
        *reinterpret_cast<volatile int*>(p.b.status) = kDevErrChunkTooLong;
    int len = p.b.seq_lens[s];
    len = len < 0 ? 0 : (len > p.max_seq_len ? p.max_seq_len : len);
    const int pos = len - (end - t);
    const int32_t* table = p.b.block_tables + static_cast<long long>(s) * p.b.max_blocks;
    float q[EPL], o[EPL];
    load_slice<false, EPL>(p.q, t * p.q_stride + static_cast<long long>(h) * HD + lane * EPL, q);
#pragma unroll
    for (int i = 0; i < EPL; ++i) o[i] = 0.f;
    float m = -INFINITY, l = 0.f;
    const int kvh = h / p.group;
    int lo = 0;
    if (p.window > 0 && pos - p.window + 1 > 0) lo = pos - p.window + 1;
    row_add<E4M3, HD>(p.b, table, kvh, q, p.scale_log2, 0, min(p.sinks, lo), m, l, o);
    row_add<E4M3, HD>(p.b, table, kvh, q, p.scale_log2, lo, pos + 1, m, l, o);
    uint16_t* out = p.out + t * p.out_stride + static_cast<long long>(h) * HD + lane * EPL;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < EPL; i += 2) {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(o[i + 1] * inv), "f"(o[i] * inv));
        *reinterpret_cast<uint32_t*>(out + i) = r;
    }
}

template <bool E4M3, int HD>
cudaError_t launch_rows(const KvAttnLaunch& a, cudaStream_t stream)
{
    RowParams p;
    p.b = a.b;
    p.q = a.q;
    p.out = a.out;
    p.q_stride = a.q_stride;
    p.out_stride = a.out_stride;
    p.num_q_heads = a.num_q_heads;
    p.group = a.num_q_heads / a.b.num_kv_heads;
    p.max_chunk = a.max_chunk;
    p.max_seq_len = a.max_seq_len;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.window = a.window;
    p.sinks = a.sinks;
    const long long blocks = (static_cast<long long>(a.b.num_tokens) * a.num_q_heads + 7) / 8;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_kernel(kv_attention_row_kernel<E4M3, HD>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream,
                         a.pdl, p);
}

}  // namespace

int launch_kv_attention(const KvAttnLaunch& a, cudaStream_t stream, char* msg, size_t msg_len)
{
    const bool q = a.b.type == kCacheE4M3;
    cudaError_t e = cudaErrorInvalidValue;
    switch (a.b.head_dim) {
    case 64: e = q ? launch_rows<true, 64>(a, stream) : launch_rows<false, 64>(a, stream); break;
    case 128: e = q ? launch_rows<true, 128>(a, stream) : launch_rows<false, 128>(a, stream); break;
    case 256: e = q ? launch_rows<true, 256>(a, stream) : launch_rows<false, 256>(a, stream); break;
    default: break;
    }
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "cache attention launch failed: %s", cudaGetErrorString(e));
        return 1;
    }
    return 0;
}

}  // namespace bsk
