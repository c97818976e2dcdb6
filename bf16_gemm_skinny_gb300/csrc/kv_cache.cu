// kv_cache.cu -- a paged key/value cache, written and read back.
//
// Append: the new tokens' K and V rows go to the pages, copied in BF16 or
// quantised to E4M3.  Each row x (one token, one KV head, head_dim values) has
// one scale 2^e, held as an E8M0 byte: with a = max|x|, e is the least integer
// with a <= 448 * 2^e (448 is E4M3's largest value), kept within [-117, 120];
// the codes are x * 2^-e rounded to nearest even.  A power of two makes both
// directions exact but for that one rounding: x * 2^-e is a scaled BF16 value,
// and code * 2^e has at most 4 significant bits and lies at or above 2^-126, so
// BF16 holds it exactly (at e = 120 the codes stop at 240, whose next one would
// stand for 2^128).  Against a scale of a / 448 it costs less than one binade of
// the 15 that E4M3's normal values span.  A row with an Inf or a NaN gets the
// scale byte 255 (NaN) and reads back as NaN.
//
// Gather: the last tokens of each sequence, BF16 again, side by side.
//
// Bound: HBM (K and V in once, out once).  A warp moves U x 512 bytes of one
// token's K and as much of its V, all loads issued before the first use; one
// lane holds 8 values, so head_dim / 8 lanes share a row and its maximum.
// Measured, 4 KV heads of 256: 20.6 k tokens quantised in 27 us (4.7 TB/s), 30 k read
// back in 30.5 us (6.0 TB/s); 20 k tokens of 8 heads of 128 stored in BF16 26.8 us (6.1 TB/s,
// 0.90 of the measured copy rate).  One token each of 16 sequences: 2 us on the GPU.
#include <cstdio>

#include "bsk_internal.h"
#include "kv_internal.h"

namespace bsk {
namespace {

constexpr int kWarps = 8;

struct CopyParams {
    KvBatch b;
    const uint16_t* k_in;
    const uint16_t* v_in;
    uint16_t* k_out;
    uint16_t* v_out;
    long long k_stride, v_stride;
    int groups;   // warps per token
};

// Where new token t lies in the cache (its row index); -1: its position does not
// exist; -2: it belongs to no sequence.
__device__ __forceinline__ long long token_row(const KvBatch& b, int t)
{
    const int s = kv_sequence_of(b, t);
    if (s >= b.num_seqs) return -2;
    if (b.cu_tokens != nullptr && t < b.cu_tokens[s]) return -2;   // before the first sequence's rows
    const int end = b.cu_tokens != nullptr ? b.cu_tokens[s + 1] : t + 1;
    const long long pos = static_cast<long long>(b.seq_lens[s]) - (static_cast<long long>(end) - t);
    if (pos < 0 || pos > 0x7fffffffLL) return -1;   // more new tokens than the sequence is long
    return kv_row(b, b.block_tables + static_cast<long long>(s) * b.max_blocks, static_cast<int>(pos));
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two E4M3 codes (x in the low byte), rounded to nearest even.
__device__ __forceinline__ uint32_t e4m3x2(float x, float y)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
    return r;
}

// Eight BF16 values of a row shared by LPR lanes -> eight codes and, in `byte`, the row's scale.
template <int LPR>
__device__ __forceinline__ uint2 quantise(const uint4& x, uint32_t& byte)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);   // magnitudes compare as integers
    m = max(m & 0xffffu, m >> 16);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m >= 0x7f80u) {
        byte = 255u;
        return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
    }
    // m = 1.f * 2^(E - 127) with f in the low 7 bits; 448 = 1.75 * 2^8
    const int e = static_cast<int>(m >> 7) - 8 + ((m & 0x7fu) > 0x60u ? 1 : 0);
    byte = static_cast<uint32_t>(min(max(e, 10), 247));
    const float inv = __uint_as_float((254u - byte) << 23);   // 2^-(byte - 127)
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo = bf16_lo(w[i]) * inv, hi = bf16_hi(w[i]) * inv;
        if (byte == 247u) {   // 256 * 2^120 would be 2^128: the codes stop at 240
            lo = fminf(fmaxf(lo, -240.f), 240.f);
            hi = fminf(fmaxf(hi, -240.f), 240.f);
        }
        c[i] = e4m3x2(lo, hi);
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Eight codes times their scale, as BF16 (exact).
__device__ __forceinline__ uint4 dequantise(const uint2& codes, float scale)
{
    const uint32_t w[2] = {codes.x, codes.y};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h, o;
        const uint16_t two = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
        float lo, hi;
        asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(lo), "=f"(hi)
            : "r"(h));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o) : "f"(hi * scale), "f"(lo * scale));
        r[i] = o;
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

template <bool E4M3, int HD, int U>
__global__ void __launch_bounds__(kWarps * 32) kv_append_kernel(const CopyParams p)
{
    constexpr int LPR = HD / 8;   // lanes per row
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long t = w / p.groups;
    const int chunks = p.b.num_kv_heads * LPR;   // 16-byte chunks of a token's K (or V)
    const int c0 = static_cast<int>(w - t * p.groups) * (U * 32) + lane;
    griddep_wait();
    griddep_launch_dependents();
    if (t >= p.b.num_tokens) return;
    const uint4* k = reinterpret_cast<const uint4*>(p.k_in + t * p.k_stride);
    const uint4* v = reinterpret_cast<const uint4*>(p.v_in + t * p.v_stride);
    uint4 x[2][U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = c0 + u * 32;
        x[0][u] = c < chunks ? k[c] : make_uint4(0, 0, 0, 0);
        x[1][u] = c < chunks ? v[c] : make_uint4(0, 0, 0, 0);
    }
    const long long row = token_row(p.b, static_cast<int>(t));
    if (row < 0) return;   // the whole warp
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = c0 + u * 32;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            void* cache = i == 0 ? p.b.k : p.b.v;
            if constexpr (E4M3) {
                uint32_t byte;
                const uint2 codes = quantise<LPR>(x[i][u], byte);
                if (c < chunks) {
                    static_cast<uint2*>(cache)[row * chunks + c] = codes;
                    if (c % LPR == 0)
                        (i == 0 ? p.b.k_scales : p.b.v_scales)[row * p.b.num_kv_heads + c / LPR] =
                            static_cast<uint8_t>(byte);
                }
            } else {
                if (c < chunks) static_cast<uint4*>(cache)[row * chunks + c] = x[i][u];
            }
        }
    }
}

template <bool E4M3, int HD, int U>
__global__ void __launch_bounds__(kWarps * 32) kv_gather_kernel(const CopyParams p)
{
    constexpr int LPR = HD / 8;
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long t = w / p.groups;
    const int chunks = p.b.num_kv_heads * LPR;
    const int c0 = static_cast<int>(w - t * p.groups) * (U * 32) + lane;
    griddep_wait();
    griddep_launch_dependents();
    if (t >= p.b.num_tokens) return;
    const long long row = token_row(p.b, static_cast<int>(t));
    if (row == -2) return;   // the whole warp
    uint4* k = reinterpret_cast<uint4*>(p.k_out + t * p.k_stride);
    uint4* v = reinterpret_cast<uint4*>(p.v_out + t * p.v_stride);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 x[2][U];
    if constexpr (E4M3) {
        uint2 codes[2][U];
        uint32_t byte[2][U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * 32;
            const bool in = row >= 0 && c < chunks;
            codes[0][u] = in ? static_cast<const uint2*>(p.b.k)[row * chunks + c] : make_uint2(0, 0);
            codes[1][u] = in ? static_cast<const uint2*>(p.b.v)[row * chunks + c] : make_uint2(0, 0);
            byte[0][u] = in ? p.b.k_scales[row * p.b.num_kv_heads + c / LPR] : 127u;
            byte[1][u] = in ? p.b.v_scales[row * p.b.num_kv_heads + c / LPR] : 127u;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) x[i][u] = dequantise(codes[i][u], e8m0_value(byte[i][u]));
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * 32;
            const bool in = row >= 0 && c < chunks;
            x[0][u] = in ? static_cast<const uint4*>(p.b.k)[row * chunks + c] : zero;
            x[1][u] = in ? static_cast<const uint4*>(p.b.v)[row * chunks + c] : zero;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = c0 + u * 32;
        if (c < chunks) {
            k[c] = x[0][u];
            v[c] = x[1][u];
        }
    }
}

// An E4M3 cache as BF16, sequence by sequence: position t of sequence s at row
// s * flat_len + t of k_out and v_out.  Only positions that some new token sees
// (at or after `lo` = the first one's window, or before `sinks`); one whose page is
// none gives zeros.  A warp moves 4 x 512 bytes of one position's K and V.
template <int HD>
__global__ void __launch_bounds__(kWarps * 32) kv_flatten_kernel(const CopyParams p, int flat_len, int max_seq_len,
                                                                 int window, int sinks)
{
    constexpr int LPR = HD / 8, U = 4;
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int t = static_cast<int>(w / p.groups);
    const int chunks = p.b.num_kv_heads * LPR;
    const int c0 = static_cast<int>(w - static_cast<long long>(t) * p.groups) * (U * 32) + lane;
    const int s = blockIdx.y;
    griddep_wait();
    griddep_launch_dependents();
    const int len = min(p.b.seq_lens[s], max_seq_len);
    if (t >= len) return;
    const int n = p.b.cu_tokens != nullptr ? p.b.cu_tokens[s + 1] - p.b.cu_tokens[s] : 1;
    if (n <= 0 || (window > 0 && t >= sinks && t < static_cast<long long>(len) - n - window + 1)) return;
    const long long row = kv_row(p.b, p.b.block_tables + static_cast<long long>(s) * p.b.max_blocks, t);
    const long long to = (static_cast<long long>(s) * flat_len + t) * chunks;
    uint2 codes[2][U];
    uint32_t byte[2][U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = c0 + u * 32;
        const bool in = row >= 0 && c < chunks;
        codes[0][u] = in ? static_cast<const uint2*>(p.b.k)[row * chunks + c] : make_uint2(0, 0);
        codes[1][u] = in ? static_cast<const uint2*>(p.b.v)[row * chunks + c] : make_uint2(0, 0);
        byte[0][u] = in ? p.b.k_scales[row * p.b.num_kv_heads + c / LPR] : 127u;
        byte[1][u] = in ? p.b.v_scales[row * p.b.num_kv_heads + c / LPR] : 127u;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = c0 + u * 32;
        if (c < chunks) {
            reinterpret_cast<uint4*>(p.k_out)[to + c] = dequantise(codes[0][u], e8m0_value(byte[0][u]));
            reinterpret_cast<uint4*>(p.v_out)[to + c] = dequantise(codes[1][u], e8m0_value(byte[1][u]));
        }
    }
}

template <bool APPEND, bool E4M3, int HD, int U>
cudaError_t launch_copy(const KvCopyLaunch& a, cudaStream_t stream)
{
    CopyParams p;
    p.b = a.b;
    p.k_in = a.k_in;
    p.v_in = a.v_in;
    p.k_out = a.k_out;
    p.v_out = a.v_out;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    const int chunks = a.b.num_kv_heads * (HD / 8);
    p.groups = (chunks + U * 32 - 1) / (U * 32);
    const long long warps = static_cast<long long>(a.b.num_tokens) * p.groups;
    const long long blocks = (warps + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto kern = APPEND ? kv_append_kernel<E4M3, HD, U> : kv_gather_kernel<E4M3, HD, U>;
    return launch_kernel(kern, dim3(static_cast<unsigned>(blocks)), dim3(kWarps * 32), 0, stream, a.pdl, p);
}

template <bool APPEND, bool E4M3, int HD>
cudaError_t launch_copy_u(const KvCopyLaunch& a, cudaStream_t stream)
{
    // With work for every warp slot a warp takes four times as much, for more loads in
    // flight per look-up.  20k tokens quantised, 4 heads of 256: 33.0 us with 1, 27.8 with
    // 2, 26.5 with 4; 28k tokens read back 37.0, 30.6, 30.7.
    const long long warps = static_cast<long long>(a.b.num_tokens) * ((a.b.num_kv_heads * (HD / 8) + 31) / 32);
    if (warps >= 8LL * a.num_sms) return launch_copy<APPEND, E4M3, HD, 4>(a, stream);
    return launch_copy<APPEND, E4M3, HD, 1>(a, stream);
}

template <bool APPEND>
int launch_copy_any(const KvCopyLaunch& a, cudaStream_t stream, char* msg, size_t msg_len)
{
    const bool q = a.b.type == kCacheE4M3;
    cudaError_t e = cudaErrorInvalidValue;
    switch (a.b.head_dim) {
    case 64: e = q ? launch_copy_u<APPEND, true, 64>(a, stream) : launch_copy_u<APPEND, false, 64>(a, stream); break;
    case 128: e = q ? launch_copy_u<APPEND, true, 128>(a, stream) : launch_copy_u<APPEND, false, 128>(a, stream); break;
    case 256: e = q ? launch_copy_u<APPEND, true, 256>(a, stream) : launch_copy_u<APPEND, false, 256>(a, stream); break;
    default: break;
    }
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "kv cache %s launch failed: %s", APPEND ? "append" : "gather", cudaGetErrorString(e));
        return 1;
    }
    return 0;
}

}  // namespace

int launch_kv_append(const KvCopyLaunch& a, cudaStream_t stream, char* msg, size_t msg_len)
{
    return launch_copy_any<true>(a, stream, msg, msg_len);
}

int launch_kv_flatten(const KvBatch& b, uint16_t* k_out, uint16_t* v_out, int flat_len, int max_seq_len, int window,
                      int sinks, bool pdl, cudaStream_t stream, char* msg, size_t msg_len)
{
    CopyParams p = {};
    p.b = b;
    p.k_out = k_out;
    p.v_out = v_out;
    const int chunks = b.num_kv_heads * (b.head_dim / 8);
    p.groups = (chunks + 127) / 128;
    const long long blocks = (static_cast<long long>(max_seq_len) * p.groups + kWarps - 1) / kWarps;
    cudaError_t e = cudaErrorInvalidConfiguration;
    if (blocks <= 0x7fffffffLL) {
        auto kern = b.head_dim == 64 ? kv_flatten_kernel<64> : (b.head_dim == 128 ? kv_flatten_kernel<128> : kv_flatten_kernel<256>);
        e = launch_kernel(kern, dim3(static_cast<unsigned>(blocks), b.num_seqs), dim3(kWarps * 32), 0, stream, pdl, p,
                          flat_len, max_seq_len, window, sinks);
    }
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "kv cache dequantisation launch failed: %s", cudaGetErrorString(e));
        return 1;
    }
    return 0;
}

int launch_kv_gather(const KvCopyLaunch& a, cudaStream_t stream, char* msg, size_t msg_len)
{
    return launch_copy_any<false>(a, stream, msg, msg_len);
}

}  // namespace bsk
