// kv_attention.cuh -- what the two attention kernels over the paged cache share:
// parameters, the keys that a CTA's rows see, small arithmetic, and one row's
// result by one warp.  (kv_attention.cu: many query rows, on tcgen05;
// kv_few_rows.cu: few, from registers.)
#pragma once

#include <cmath>

#include "kv_internal.h"

namespace bsk {
namespace kv {

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
          "l"(*reinterpret_cast<unsigned long long*>(&c)));
    return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
    return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
    return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// 2^x, the hardware approximation (2^-22 relative): 2^-inf = 0.
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two E4M3 codes -> two FP16 values (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
    return h;
}
// Two E4M3 codes -> their values.
__device__ __forceinline__ float2 e4m3x2_values(uint32_t two)
{
    uint32_t h;
    float2 f;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}
// The score factor of a query row that was multiplied by 2^-e: never 0, since it also
// multiplies the -inf of a position out of sight, and never infinite, since it also
// multiplies scores of 0.  FP32's least number stands for what is smaller (scores up to
// FP32's largest times it are within 2^-21 of 0), its largest for what is larger.
__device__ __forceinline__ float row_factor(float scale_log2, int e)
{
    return fminf(fmaxf(scale_log2 * exp2f(static_cast<float>(e)), __uint_as_float(1u)), __uint_as_float(0x7f7fffffu));
}
// Scales of E4M3 values.  A row's scale 2^s goes into its FP16 values, not into the
// weights: a value is code * 2^(s - E + 5), which FP16 holds exactly for s - E from -20
// (E4M3's least step 2^-9 becomes 2^-24) to 2 (448 becomes 57344), and O is multiplied
// by 2^(E' - E'') when E moves.  E follows the largest scale in sight, from -40 up, in
// steps of more than 2.  Weights are stored times 2^7: at most 2^15 (the running maximum
// may lag by 2^8), off by 2^-11 of themselves at most down to 2^-21 of the row's largest
// and by 2^-32 of it below that.  (The scale in the weights instead, w * 2^(s - E) in
// FP16, lost the weights of ordinary rows beside one large value that no row attends to.)
// A row further below E, or one whose O would shrink past FP32, makes the CTA's rows
// be computed one by one (repair_row).  Rows at the least scale, 2^-117, may be zeros,
// which mind no factor: they stay out of the range, their factor is 0 (E is -40 at
// least), and the first code among them that is not 0 does the same.
struct ScaleRange {
    int E = -40, low = 1000;
    // New rows' largest and least exponent (-1000, 1000: none); true: out of range
    __device__ __forceinline__ bool take(int top, int least)
    {
        if (top > E + 2) E = top;
        low = min(low, least);
        return least < E - 20 || low < E - 90;
    }
    // 2^(s - E + 5) in FP16 for the scale byte b of a row in sight; 0 when that is too small
    __device__ __forceinline__ uint32_t factor(uint32_t b) const
    {
        const int g = static_cast<int>(b) - 127 - E + 5;
        if (b == 255u) return 0x7e00u;
        return g >= -14 ? static_cast<uint32_t>(g + 15) << 10 : (g == -15 ? 0x0200u : 0u);
    }
};
constexpr float kWeightLog2 = 7.f;   // weights are stored times 2^this
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
struct AttnParams {
    KvBatch b;
    const uint16_t* q;
    uint16_t* out;
    long long q_stride, out_stride;
    int num_q_heads, group, max_chunk, max_seq_len;
    int tiles, segments;          // row tiles (128 rows, or 8) per sequence and KV head, key segments per tile
    int segment_keys;             // positions of a segment, a multiple of 128 (the last one takes the rest)
    int box;                      // rows per TMA box, or 4: pages of an odd size, gathers only
    int tile_rows;                // cache rows that boxes of a tile's rows may cover
    float scale_log2;             // |softmax scale| * log2(e), > 0 (a scale of 0: FP32's least number)
    uint32_t q_sign;              // 0x80008000 for a negative scale
    int window, sinks;
    float* part_o;                // [rows][segments][HD] unnormalised O
    float2* part_ml;              // [rows][segments] (m, l)
    unsigned long long wait_limit_ns;
};

// The first position in the window of a query at `pos` (which may be negative, and the
// window up to 2^31 - 1); no window: 0.
__device__ __forceinline__ int window_start(int pos, int window)
{
    return window > 0 && pos >= window ? pos - window + 1 : 0;
}

// The key tiles that some row of a CTA sees: those of the sinks, then those from
// the window's first on.  A position holds a key when it is below kv_end and not
// between sink_end and lo.
template <int kTile>
struct Keys {
    int sink_tiles, lo_tile;      // tile i lies at i, or at i - sink_tiles + lo_tile
    int begin, end;               // this segment's tiles
    int lo, sink_end, kv_end;
    __device__ __forceinline__ int base(int i) const { return (i < sink_tiles ? i : i - sink_tiles + lo_tile) * kTile; }
    __device__ __forceinline__ bool holds(int t) const { return t < kv_end && (t >= lo || t < sink_end); }
    // all of t .. t + n - 1 hold a key / none does
    __device__ __forceinline__ bool all(int t, int n) const { return t + n <= kv_end && (t >= lo || t + n <= sink_end); }
    __device__ __forceinline__ bool none(int t, int n) const { return t >= kv_end || (t >= sink_end && t + n <= lo); }
};

// The k lowest of 64 bits.
__device__ __forceinline__ unsigned long long low_bits(int k)
{
    return k <= 0 ? 0ull : (k >= 64 ? ~0ull : (1ull << k) - 1);
}

// One row by one warp, in FP32: for rows whose O is not finite although their
// weights are, which happens when a value that the row does not see holds an
// Inf or a NaN (its weight 0 times that is NaN on the tensor cores).
template <bool E4M3, int EPL>
__device__ __forceinline__ void load_slice(const void* cache, long long elem, float (&f)[EPL])
{
#pragma unroll
    for (int i = 0; i < EPL; i += 2) {
        if constexpr (E4M3) {
            const float2 v =
                e4m3x2_values(*reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(cache) + elem + i));
            f[i] = v.x;
            f[i + 1] = v.y;
        } else {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(cache) + elem + i);
            f[i] = __uint_as_float(w << 16);
            f[i + 1] = __uint_as_float(w & 0xffff0000u);
        }
    }
}

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
        const float ks = E4M3 ? e8m0_value(b.k_scales[hr]) : 1.f;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) s = fmaf(q[i], k[i] * ks, s);
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
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

// The row's positions are those it sees among the keys' tiles begin .. end - 1.
template <bool E4M3, int HD, int kTile>
__device__ __noinline__ void repair_row(const AttnParams& p, const int32_t* table, const Keys<kTile>& keys, int kvh,
                                        int token, int head, int pos, int seg)
{
    constexpr int EPL = HD / 32;
    const int lane = threadIdx.x & 31;
    float q[EPL], o[EPL];
    load_slice<false, EPL>(p.q, token * p.q_stride + static_cast<long long>(head) * HD + lane * EPL, q);
    const float sign = p.q_sign ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        q[i] *= sign;
        o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const int lo = window_start(pos, p.window);
    const int sinks = min(p.sinks, lo);
    for (int part = 0; part < 2; ++part) {   // the segment's sink tiles, then its window tiles
        const int i0 = part == 0 ? keys.begin : max(keys.begin, keys.sink_tiles);
        const int i1 = part == 0 ? min(keys.end, keys.sink_tiles) : keys.end;
        if (i0 >= i1) continue;
        const int a = keys.base(i0), e = keys.base(i1 - 1) + kTile;
        row_add<E4M3, HD>(p.b, table, kvh, q, p.scale_log2, a, min(min(e, sinks), pos + 1), m, l, o);
        row_add<E4M3, HD>(p.b, table, kvh, q, p.scale_log2, max(a, lo), min(e, pos + 1), m, l, o);
    }
    if (p.segments == 1) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t* out = p.out + token * p.out_stride + static_cast<long long>(head) * HD + lane * EPL;
#pragma unroll
        for (int i = 0; i < EPL; i += 2) *reinterpret_cast<uint32_t*>(out + i) = bf16x2(o[i] * inv, o[i + 1] * inv);
    } else {
        const long long at = (static_cast<long long>(token) * p.num_q_heads + head) * p.segments + seg;
#pragma unroll
        for (int i = 0; i < EPL; ++i) p.part_o[at * HD + lane * EPL + i] = o[i];
        if (lane == 0) p.part_ml[at] = make_float2(m, l);
    }
}

// A score is (sum of 2^-e q * code) * K scale * row_factor, and the sum up to 2^32 (q up to
// 2^15, codes to 448, 256 of them), so that beside a K scale above 2^95 it may pass FP32
// although q.k does not: such a key in sight makes the CTA's rows be computed one by one.
__device__ __forceinline__ bool k_scale_too_large(uint32_t b) { return b - 223u < 32u; }

// Launches the kernel for few query rows over an E4M3 cache: `rows` (8, or 16 with
// HD < 256) per CTA, p.tiles of them per sequence and KV head.
template <int HD>
cudaError_t launch_few_rows(const AttnParams& p, int rows, bool pdl, cudaStream_t stream);

}  // namespace kv
}  // namespace bsk
