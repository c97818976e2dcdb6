// kv_few_rows.cu -- attention over the paged cache for few query rows per KV
// head: single tokens, and a few drafted ones.
//
// The same one-pass sums as kv_attention.cu, but the cache is read once for at
// most 8 rows, so what counts is the stream from HBM; the tcgen05 path would send
// every key through shared memory twice for an MMA of 128 rows.  Here keys and
// values go from global memory to registers and from there into mma.sync, with
// the positions as the M of the products:
//   S^T (16 positions x 8 rows) = K Q^T,   O^T (16 dimensions x 8 rows) += V^T P^T
// The order of the dimensions within a product is free, so each lane loads 16
// contiguous bytes of a key's row and uses them as its fragments of several MMAs
// (Q is read in the same order); a value's row likewise, two positions' values
// put side by side with byte permutations.  P goes from the layout of S^T to that
// of P^T by movmatrix.  E4M3 codes become FP16 pairs by one instruction each
// (exact), and Q, scaled by a power of two per row, FP16 too.
//
// A warp takes every fourth group of 16 positions of its CTA's segment; the next
// group's keys load while this one's values are used and the other way round.
// The CTA's four warps are joined in shared memory, the segments by kv_join_kernel.
#include <cstdio>

#include "bsk_internal.h"
#include "kv_attention.cuh"

namespace bsk {
namespace kv {
namespace {

constexpr int kWarps = 4;
constexpr int kGroup = 16;   // positions per step of a warp
constexpr int kRows8 = 8;    // query rows per CTA (the N of the MMAs)

template <bool E4M3>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    if constexpr (E4M3)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// A 16-byte load that leaves no line in L1 (the cache is read once).
__device__ __forceinline__ uint4 load_once(const void* p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

template <bool E4M3, int HD>
__global__ void __launch_bounds__(kWarps * 32, 2) kv_few_rows_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int kElem = E4M3 ? 1 : 2;
    constexpr int kVec = 16 / kElem;             // values in 16 bytes
    constexpr int kKeyVecs = HD / (4 * kVec);    // 16-byte loads of a key's row per lane (4 lanes a row)
    // values: 8 lanes a row.  With HD = 64 in E4M3 a lane's share is 8 bytes; it
    // loads the 16 around them and uses its half.
    constexpr bool kHalf = E4M3 && HD == 64;
    constexpr int kValVecs = kHalf ? 1 : HD / (8 * kVec);
    constexpr int kDim = HD / 16;                // O^T tiles
    constexpr int kPitch = HD + 8;               // Q rows in shared memory, padded against bank conflicts
    __shared__ __align__(16) uint16_t s_q[kRows8 * kPitch];
    __shared__ float s_o[kWarps][kRows8][HD];
    __shared__ float s_m[kWarps][kRows8], s_l[kWarps][kRows8], s_scale[kRows8];
    __shared__ int s_flag;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;

    griddep_wait();
    griddep_launch_dependents();

    int idx = blockIdx.x;
    const int tile = p.tiles - 1 - idx % p.tiles;
    idx /= p.tiles;
    const int kvh = idx % p.b.num_kv_heads;
    idx /= p.b.num_kv_heads;
    const int seq = idx % p.b.num_seqs;
    const int seg = idx / p.b.num_seqs;
    int first = seq, n = 1;
    if (p.b.cu_tokens != nullptr) {
        first = p.b.cu_tokens[seq];
        n = p.b.cu_tokens[seq + 1] - first;
        if (first < 0 || n < 0 || first > p.b.num_tokens - n) n = 0;   // not a prefix sum: nothing is read
    }
    if (n > p.max_chunk) {
        if (threadIdx.x == 0) *reinterpret_cast<volatile int*>(p.b.status) = kDevErrChunkTooLong;
        n = p.max_chunk;
    }
    int len = p.b.seq_lens[seq];
    len = len < 0 ? 0 : (len > p.max_seq_len ? p.max_seq_len : len);
    const int row0 = tile * kRows8;
    const int rows = min(kRows8, n * p.group - row0);
    if (rows <= 0) return;
    const int pos0 = len - n;
    const int pmin = pos0 + row0 / p.group, pmax = pos0 + (row0 + rows - 1) / p.group;
    Keys<kGroup> keys;
    keys.kv_end = max(pmax + 1, 0);
    keys.lo = p.window > 0 && pmin - p.window + 1 > 0 ? pmin - p.window + 1 : 0;
    keys.sink_end = min(p.sinks, keys.lo);
    keys.lo_tile = keys.lo / kGroup;
    keys.sink_tiles = min((keys.sink_end + kGroup - 1) / kGroup, keys.lo_tile);
    {
        const int total = keys.kv_end > 0 ? keys.sink_tiles + (keys.kv_end + kGroup - 1) / kGroup - keys.lo_tile : 0;
        keys.begin = static_cast<int>(static_cast<long long>(total) * seg / p.segments);
        keys.end = static_cast<int>(static_cast<long long>(total) * (seg + 1) / p.segments);
    }
    const int32_t* table = p.b.block_tables + static_cast<long long>(seq) * p.b.max_blocks;

    // ---- Q: 16-bit rows in shared memory; rows that do not exist are zero ----
    if (threadIdx.x == 0) s_flag = 0;
    for (int r = warp; r < kRows8; r += kWarps) {
        constexpr int kPairs = HD / 64;   // 32-bit pairs per lane
        uint32_t w[kPairs];
        const int my = row0 + min(r, rows - 1);
        const uint32_t* src = reinterpret_cast<const uint32_t*>(
            p.q + (first + my / p.group) * p.q_stride + (static_cast<long long>(kvh) * p.group + my % p.group) * HD);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            w[i] = r < rows ? src[i * 32 + lane] ^ p.q_sign : 0u;
            m = __vmaxu2(m, w[i] & 0x7fff7fffu);
        }
        float scale = p.scale_log2;
        if constexpr (E4M3) {
            // times a power of two that brings the row's largest value to [2^14, 2^15)
            m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
            const int e = max(-126, min(static_cast<int>(m >> 7) - 127 - 14, 113));
            const float f = exp2f(static_cast<float>(-e));
            scale *= exp2f(static_cast<float>(e));
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                w[i] = f16x2(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
        }
        if (lane == 0) s_scale[r] = scale;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) *reinterpret_cast<uint32_t*>(s_q + r * kPitch + (i * 32 + lane) * 2) = w[i];
    }
    __syncthreads();

    // this lane's two rows (columns 2c, 2c+1 of S^T)
    float row_scale[2], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int row_pos[2], row_lo[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        row_scale[i] = s_scale[2 * c + i];
        row_pos[i] = 2 * c + i < rows ? pos0 + (row0 + 2 * c + i) / p.group : -1;
        row_lo[i] = p.window > 0 && row_pos[i] - p.window + 1 > 0 ? row_pos[i] - p.window + 1 : 0;
    }
    const int lo_max = p.window > 0 ? pmax - p.window + 1 : 0;
    float o[kDim][4];
#pragma unroll
    for (int d = 0; d < kDim; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][i] = 0.f;
    // E4M3 (as in kv_attention.cu): o and l hold 2^(3 - E) of their values
    int E = 0, low_e = 1000;
    bool wide = false;

    const uint8_t* kc = static_cast<const uint8_t*>(p.b.k) + static_cast<long long>(kvh) * HD * kElem;
    const uint8_t* vc = static_cast<const uint8_t*>(p.b.v) + static_cast<long long>(kvh) * HD * kElem;
    const long long pitch = static_cast<long long>(p.b.num_kv_heads) * HD * kElem;
    const int mine = lane & 15;   // the position of a group whose page this lane looks up
    int entry = -1, row = -1;     // block-table entry of the group after next, cache row in the next
    uint32_t kb = 127u, vb = 127u;
    auto look_up = [&](int i) {
        entry = -1;
        if (i < keys.end) {
            const int at = (keys.base(i) + mine) / p.b.block_size;
            if (at < p.b.max_blocks) entry = table[at];
        }
    };
    auto find = [&](int i) {   // the group looked up last
        row = -1;
        kb = vb = 127u;
        if (i < keys.end) {
            const int t = keys.base(i) + mine;
            if (keys.holds(t)) {
                if (static_cast<unsigned>(entry) < static_cast<unsigned>(p.b.num_blocks)) {
                    row = entry * p.b.block_size + t % p.b.block_size;
                    if constexpr (E4M3) {
                        kb = p.b.k_scales[static_cast<long long>(row) * p.b.num_kv_heads + kvh];
                        vb = p.b.v_scales[static_cast<long long>(row) * p.b.num_kv_heads + kvh];
                    }
                } else {
                    *reinterpret_cast<volatile int*>(p.b.status) = 0x200;   // kDevErrBadIndex
                }
            }
        }
    };
    uint4 kreg[2][kKeyVecs], vreg[4][kValVecs];
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    auto load_keys = [&]() {   // of the group whose rows `row` holds
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = __shfl_sync(0xffffffffu, row, g + 8 * i);
            const uint8_t* src = kc + r * pitch + c * 16;
#pragma unroll
            for (int v = 0; v < kKeyVecs; ++v) kreg[i][v] = r >= 0 ? load_once(src + v * 64) : zero;
        }
    };
    auto load_values = [&]() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = __shfl_sync(0xffffffffu, row, 2 * c + (i & 1) + 8 * (i >> 1));
            const uint8_t* src = vc + r * pitch + (kHalf ? (g >> 1) : g) * 16;
#pragma unroll
            for (int v = 0; v < kValVecs; ++v) vreg[i][v] = r >= 0 ? load_once(src + v * 128) : zero;
        }
    };

    int i0 = keys.begin + warp;
    look_up(i0);
    find(i0);
    look_up(i0 + kWarps);
    load_keys();
    load_values();
    for (int i = i0; i < keys.end; i += kWarps) {
        const int base = keys.base(i);
        const uint32_t have = __ballot_sync(0xffffffffu, row >= 0) & 0xffffu;   // positions that hold a key
        const uint32_t kb_now = kb, vb_now = vb;
        // S^T
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int v = 0; v < kKeyVecs; ++v) {
            const uint32_t x[2][4] = {{kreg[0][v].x, kreg[0][v].y, kreg[0][v].z, kreg[0][v].w},
                                      {kreg[1][v].x, kreg[1][v].y, kreg[1][v].z, kreg[1][v].w}};
            const uint4* qs = reinterpret_cast<const uint4*>(s_q + g * kPitch + v * 4 * kVec + c * kVec);
            if constexpr (E4M3) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 q = qs[h];   // 8 values: two MMAs
                    mma16816<true>(s[0], e4m3x2_f16x2(x[0][2 * h]), e4m3x2_f16x2(x[1][2 * h]),
                                   e4m3x2_f16x2(x[0][2 * h] >> 16), e4m3x2_f16x2(x[1][2 * h] >> 16), q.x, q.y);
                    mma16816<true>(s[1], e4m3x2_f16x2(x[0][2 * h + 1]), e4m3x2_f16x2(x[1][2 * h + 1]),
                                   e4m3x2_f16x2(x[0][2 * h + 1] >> 16), e4m3x2_f16x2(x[1][2 * h + 1] >> 16), q.z, q.w);
                }
            } else {
                const uint4 q = qs[0];
                mma16816<false>(s[0], x[0][0], x[1][0], x[0][1], x[1][1], q.x, q.y);
                mma16816<false>(s[1], x[0][2], x[1][2], x[0][3], x[1][3], q.z, q.w);
            }
        }
        // the next group's rows, and its keys on their way
        find(i + kWarps);
        look_up(i + 2 * kWarps);
        load_keys();
        // weights: lane (g, c) has positions g, g + 8 and rows 2c, 2c + 1
        float x[4] = {s[0][0] + s[1][0], s[0][1] + s[1][1], s[0][2] + s[1][2], s[0][3] + s[1][3]};
        float grow_e = 1.f, vf[2] = {1.f, 1.f};
        if constexpr (E4M3) {
            const uint32_t k0 = __shfl_sync(0xffffffffu, kb_now, g), k1 = __shfl_sync(0xffffffffu, kb_now, g + 8);
            const float f0 = e8m0_value(k0), f1 = e8m0_value(k1);
            x[0] *= f0;
            x[1] *= f0;
            x[2] *= f1;
            x[3] *= f1;
            vf[0] = e8m0_value(__shfl_sync(0xffffffffu, vb_now, g));
            vf[1] = e8m0_value(__shfl_sync(0xffffffffu, vb_now, g + 8));
            // the range of V's exponents, all-zero rows (the least scale) left out
            const bool h = ((have >> mine) & 1u) != 0 && vb_now > 10u && vb_now != 255u;
            const int top = __reduce_max_sync(0xffffffffu, h ? static_cast<int>(vb_now) - 127 : -1000);
            const int low = __reduce_min_sync(0xffffffffu, h ? static_cast<int>(vb_now) - 127 : 1000);
            if (top > -1000) {
                if (low_e == 1000 || top > E + 4) {
                    grow_e = exp2_fast(static_cast<float>(E - top));
                    E = top;
                }
                low_e = min(low_e, low);
                wide = wide || E - low_e > 20 || top > 60 || low_e < -60;
            }
        }
        if (have != 0xffffu || base + kGroup - 1 > pmin || (base < lo_max && base + kGroup > p.sinks) || rows < kRows8) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int at = g + 8 * (k >> 1), t = base + at;
                const bool seen = ((have >> at) & 1u) != 0 && t <= row_pos[k & 1] && (t >= row_lo[k & 1] || t < p.sinks);
                if (!seen) x[k] = -INFINITY;
            }
        }
        float mn[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float t = fmaxf(x[k], x[k + 2]);
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
            mn[k] = fmaxf(m[k], t * row_scale[k]);
        }
        // O and l move to a new maximum only once it is 2^8 larger (or E changes)
        if (__any_sync(0xffffffffu, mn[0] > m[0] + 8.f || mn[1] > m[1] + 8.f) || grow_e != 1.f) {
            float f[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                f[k] = grow_e;
                if (mn[k] > m[k] + 8.f) {
                    f[k] *= exp2_fast(m[k] - mn[k]);
                    m[k] = mn[k];
                }
                l[k] *= f[k];
            }
#pragma unroll
            for (int d = 0; d < kDim; ++d) {
                o[d][0] *= f[0];
                o[d][1] *= f[1];
                o[d][2] *= f[0];
                o[d][3] *= f[1];
            }
        }
        uint32_t pt[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {   // positions g + 8 k
            float w[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float b = m[q] == -INFINITY ? 0.f : m[q];
                if constexpr (E4M3) b -= static_cast<float>(3 - E);
                w[q] = exp2_fast(fmaf(x[2 * k + q], row_scale[q], -b));
                l[q] += w[q];
            }
            pt[k] = transpose8x8(E4M3 ? f16x2(w[0] * vf[k], w[1] * vf[k]) : bf16x2(w[0], w[1]));
        }
        // O^T
#pragma unroll
        for (int v = 0; v < kValVecs; ++v) {
            uint32_t y[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                y[k][0] = vreg[k][v].x;
                y[k][1] = vreg[k][v].y;
                y[k][2] = vreg[k][v].z;
                y[k][3] = vreg[k][v].w;
                if constexpr (kHalf) {
                    if (g & 1) {
                        y[k][0] = y[k][2];
                        y[k][1] = y[k][3];
                    }
                }
            }
            constexpr int kPairs = kHalf ? 4 : kVec / 2;   // pairs of dimensions a lane has per position
#pragma unroll
            for (int d = 0; d < kPairs; ++d) {
                uint32_t u[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    u[k] = E4M3 ? e4m3x2_f16x2(y[k][(d >> 1) & 3] >> (16 * (d & 1))) : y[k][d & 3];
                mma16816<E4M3>(o[v * kPairs + d], __byte_perm(u[0], u[1], 0x5410), __byte_perm(u[0], u[1], 0x7632),
                               __byte_perm(u[2], u[3], 0x5410), __byte_perm(u[2], u[3], 0x7632), pt[0], pt[1]);
            }
        }
        load_values();
    }

    // ---- the warps' results ---------------------------------------------------
    const float plain = E4M3 ? exp2f(static_cast<float>(E - 3)) : 1.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], 4);
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], 8);
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], 16);
        if (g == 0) {
            s_m[warp][2 * c + k] = m[k];
            s_l[warp][2 * c + k] = l[k] * plain;
        }
    }
    constexpr int kPairs = kHalf ? 4 : kVec / 2;
#pragma unroll
    for (int d = 0; d < kDim; ++d) {
        const int dim = kHalf ? g * 8 + d * 2 : (d / kPairs) * (8 * kVec) + g * kVec + (d % kPairs) * 2;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            *reinterpret_cast<float2*>(&s_o[warp][2 * c + k][dim]) = make_float2(o[d][k] * plain, o[d][2 + k] * plain);
    }
    if (wide && lane == 0) atomicOr(&s_flag, 0xff);
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (HD / 4); i += kWarps * 32) {
        const int r = i / (HD / 4), d = (i % (HD / 4)) * 4;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][r]);
        const float b = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2f(s_m[w][r] - b);
            const float4 v = *reinterpret_cast<const float4*>(&s_o[w][r][d]);
            L = fmaf(f, s_l[w][r], L);
            O.x = fmaf(f, v.x, O.x);
            O.y = fmaf(f, v.y, O.y);
            O.z = fmaf(f, v.z, O.z);
            O.w = fmaf(f, v.w, O.w);
        }
        const int my = row0 + r, token = first + my / p.group, head = kvh * p.group + my % p.group;
        if (p.segments == 1) {
            const float inv = L == 0.f ? 0.f : 1.f / L;
            *reinterpret_cast<uint2*>(p.out + token * p.out_stride + static_cast<long long>(head) * HD + d) =
                make_uint2(bf16x2(O.x * inv, O.y * inv), bf16x2(O.z * inv, O.w * inv));
        } else {
            const long long at = (static_cast<long long>(token) * p.num_q_heads + head) * p.segments + seg;
            *reinterpret_cast<float4*>(p.part_o + at * HD + d) = O;
            if (d == 0) p.part_ml[at] = make_float2(M, L);
        }
        // an Inf or NaN among values that the row may not see: repair_row below
        const float odd = fmaf(O.x, 0.f, fmaf(O.y, 0.f, fmaf(O.z, 0.f, O.w * 0.f)));
        if (odd != 0.f && L - L == 0.f) atomicOr(&s_flag, 1 << r);
    }
    __syncthreads();
    if (s_flag != 0) {
        for (int r = warp; r < rows; r += kWarps) {
            if (!((s_flag >> r) & 1)) continue;
            const int my = row0 + r;
            repair_row<E4M3, HD, kGroup>(p, table, keys, kvh, first + my / p.group, kvh * p.group + my % p.group,
                                         pos0 + my / p.group, seg);
        }
    }
}

}  // namespace

template <bool E4M3, int HD>
cudaError_t launch_few_rows(const AttnParams& p, bool pdl, cudaStream_t stream)
{
    const long long ctas = static_cast<long long>(p.tiles) * p.b.num_kv_heads * p.b.num_seqs * p.segments;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_kernel(kv_few_rows_kernel<E4M3, HD>, dim3(static_cast<unsigned>(ctas)), dim3(kWarps * 32), 0, stream,
                         pdl, p);
}

template cudaError_t launch_few_rows<false, 64>(const AttnParams&, bool, cudaStream_t);
template cudaError_t launch_few_rows<false, 128>(const AttnParams&, bool, cudaStream_t);
template cudaError_t launch_few_rows<false, 256>(const AttnParams&, bool, cudaStream_t);
template cudaError_t launch_few_rows<true, 64>(const AttnParams&, bool, cudaStream_t);
template cudaError_t launch_few_rows<true, 128>(const AttnParams&, bool, cudaStream_t);
template cudaError_t launch_few_rows<true, 256>(const AttnParams&, bool, cudaStream_t);

}  // namespace kv
}  // namespace bsk
