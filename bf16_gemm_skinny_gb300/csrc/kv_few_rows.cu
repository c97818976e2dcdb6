// kv_few_rows.cu -- attention over a paged E4M3 cache for few query rows per KV
// head: single tokens, and a few drafted ones.
//
// The same one-pass sums as kv_attention.cu, but the cache is read once for at
// most 8 rows, so what counts is the stream from HBM; the tcgen05 path would send
// every key through shared memory twice for an MMA of 128 rows.  Here each lane
// copies (cp.async) what it will itself need, a few groups ahead, and feeds it
// from registers into mma.sync, with the positions as the M of the products:
//   S^T (16 positions x 8 rows) = K Q^T,   O^T (16 dimensions x 8 rows) += V^T P^T
// The order of the dimensions within a product is free, so each lane loads 16
// contiguous bytes of a key's row and uses them as its fragments of several MMAs
// (Q is read in the same order); a value's row likewise, two positions' values
// put side by side with byte permutations.  P goes from the layout of S^T to that
// of P^T by movmatrix.  E4M3 codes become FP16 pairs by one instruction each
// (exact), the values by a second one times their row's scale (ScaleRange, exact), and
// Q, scaled by a power of two per row, FP16 too.
//
// The warps of a CTA take the 32-position steps of its segment in turn.  They are
// joined in shared memory, the segments by kv_join_kernel.
//
// Bound: the latency of a warp's step (some 750 instructions, 6 to 16 warps per SM);
// without its MMAs, or on a few pages read over and over, it was under 4% faster.
// Measured: 64 sequences of up to 8000 tokens, 64 heads over 8 KV heads of 128: 148 to
// 150 us, 3.7 TB/s (0.55 of the measured copy rate; 231 us with loads into registers, 181
// with 16 positions a step); one of 32768, 16 heads over 4 of 256: 28 us, 2.4 TB/s, of
// which some 19 us do not depend on the length.
#include <cstdio>

#include "bsk_internal.h"
#include "kv_attention.cuh"

namespace bsk {
namespace kv {
namespace {

// D (16 x 8, FP32) += A (16 x 16, FP16, row-major) * B (16 x 8, FP16, column-major).
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// 16 bytes global -> shared, asynchronous; `in` false: zeros.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
// The aligned 4 bytes that hold the byte at `src`, to shared memory.
__device__ __forceinline__ void cp_async_word_of(uint32_t dst, const uint8_t* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst),
                 "l"(reinterpret_cast<uintptr_t>(src) & ~static_cast<uintptr_t>(3))
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Sizes.  `kAhead` steps per warp are on their way: the CTAs of an SM have 64 to
// 200 KB in flight; the latency times HBM's rate needs about 45 KB.  More warps count
// for more than more steps ahead.  Microseconds with 4 CTAs of one step ahead / 3 of
// two (head_dim 64: three): 64 sequences of up to 8000 tokens, head_dim 128, 149 / 156;
// 32 of up to 4000, head_dim 64, 27 / 37; 5 or 6 CTAs spill (167; 33).  With head_dim 256
// twice the warps at one step ahead are the same (27.1 / 27.4, one sequence of 32768).
template <int HD, int R>
struct Few {
    static constexpr int kRows = 8 * R;                 // query rows per CTA (R MMAs of N = 8)
    static constexpr int kVec = 16;                     // codes in 16 bytes
    static constexpr int kKeyVecs = HD / 64;            // 16-byte pieces of a key's row per lane (4 lanes a row)
    // values: 8 lanes a row.  With HD = 64 a lane's share is 8 bytes; it takes the 16
    // around them and uses its half.
    static constexpr bool kHalf = HD == 64;
    static constexpr int kValVecs = kHalf ? 1 : HD / 128;
    // A warp's step is 32 positions: the work that does not depend on their number is
    // over half of that of 16.
    static constexpr int kSub = 2;
    static constexpr int kGroup = 16 * kSub;
    static constexpr int kWarps = HD == 256 ? 3 : 4;
    static constexpr int kAhead = HD == 256 ? 2 : 1;
    static constexpr int kCtas = R > 1 || HD == 256 ? 2 : 4;   // of an SM
    static constexpr int kKeyBytes = kSub * 2 * kKeyVecs * 512, kValBytes = kSub * 4 * kValVecs * 512;   // of a step
    static constexpr int kWarpRing = kAhead * (kKeyBytes + kValBytes);
    static constexpr int kRing = kWarps * kWarpRing;
    static constexpr int kOut = kWarps * kRows * HD * 4;   // the warps' O, over the ring
    // Q rows, padded so that the 8 lanes of a 16-byte read's quarter meet distinct banks
    static constexpr int kPitch = HD + 8;
    static constexpr int kBytes = (kRing > kOut ? kRing : kOut) + kRows * kPitch * 2;
};

template <int HD, int R>
__global__ void __launch_bounds__(Few<HD, R>::kWarps * 32, Few<HD, R>::kCtas) kv_few_rows_kernel(const __grid_constant__ AttnParams p)
{
    using F = Few<HD, R>;
    constexpr int kWarps = F::kWarps, kVec = F::kVec, kKeyVecs = F::kKeyVecs, kValVecs = F::kValVecs;
    constexpr bool kHalf = F::kHalf;
    constexpr int A = F::kAhead, SUB = F::kSub;
    constexpr int kDim = HD / 16;                // O^T tiles
    constexpr int kPitch = F::kPitch;
    extern __shared__ __align__(16) uint8_t smem[];
    uint16_t* s_q = reinterpret_cast<uint16_t*>(smem + F::kBytes - F::kRows * kPitch * 2);
    float* s_o = reinterpret_cast<float*>(smem);          // [kWarps][F::kRows][HD], once the ring is done with
    // per position of the steps on their way: which byte of s_sk / s_sv holds its scale
    // (bits 0-1, 2-3), and bit 4: it holds a key
    __shared__ uint32_t s_meta[kWarps][A + 1][32];
    __shared__ uint32_t s_sk[kWarps][A + 1][32], s_sv[kWarps][A + 1][32];
    __shared__ float s_m[kWarps][F::kRows], s_l[kWarps][F::kRows], s_scale[F::kRows];
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
    const int seg = p.segments - 1 - idx / p.b.num_seqs;   // what only long sequences have, first
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
    const int row0 = tile * F::kRows;
    const int rows = min(F::kRows, n * p.group - row0);
    if (rows <= 0) return;
    const int pos0 = len - n;
    const int pmin = pos0 + row0 / p.group, pmax = pos0 + (row0 + rows - 1) / p.group;
    Keys<F::kGroup> keys;
    keys.kv_end = max(pmax + 1, 0);
    keys.lo = window_start(pmin, p.window);
    keys.sink_end = min(p.sinks, keys.lo);
    keys.lo_tile = keys.lo / F::kGroup;
    keys.sink_tiles = min((keys.sink_end + F::kGroup - 1) / F::kGroup, keys.lo_tile);
    {
        const int total = keys.kv_end > 0 ? keys.sink_tiles + (keys.kv_end + F::kGroup - 1) / F::kGroup - keys.lo_tile : 0;
        const int each = p.segment_keys / F::kGroup;
        keys.begin = static_cast<int>(min(static_cast<long long>(total), static_cast<long long>(each) * seg));
        keys.end = seg + 1 == p.segments ? total : min(total, keys.begin + each);
    }
    const int32_t* table = p.b.block_tables + static_cast<long long>(seq) * p.b.max_blocks;

    const uint8_t* kc = static_cast<const uint8_t*>(p.b.k) + static_cast<long long>(kvh) * HD;
    const uint8_t* vc = static_cast<const uint8_t*>(p.b.v) + static_cast<long long>(kvh) * HD;
    const long long pitch = static_cast<long long>(p.b.num_kv_heads) * HD;
    const int mine = lane & (F::kGroup - 1);   // the position of a step whose page this lane looks up
    int entry = -1, row = -1;     // block-table entry of the group looked up last, cache row of the one found last
    // page and place in it of the group to look up next, stepped from group to group
    const int bs = p.b.block_size;
    const int step_pages = kWarps * F::kGroup / bs, step_slots = kWarps * F::kGroup - step_pages * bs;
    int page = 0, off = 0, entry_off = 0;
    bool fresh = true, in_sinks = false;
    auto look_up = [&](int i) {
        entry = -1;
        if (i < keys.end) {
            if (fresh || (in_sinks && i >= keys.sink_tiles)) {
                const int t = keys.base(i) + mine;
                page = t / bs;
                off = t - page * bs;
                fresh = false;
                in_sinks = i < keys.sink_tiles;
            }
            if (page < p.b.max_blocks) entry = table[page];
            entry_off = off;
            page += step_pages;
            off += step_slots;
            if (off >= bs) {
                off -= bs;
                ++page;
            }
        }
    };
    auto find = [&](int i) {   // the step looked up last
        row = -1;
        if (i < keys.end && keys.holds(keys.base(i) + mine)) {
            if (static_cast<unsigned>(entry) < static_cast<unsigned>(p.b.num_blocks))
                row = entry * bs + entry_off;
            else
                *reinterpret_cast<volatile int*>(p.b.status) = kDevErrBadIndex;
        }
    };
    const uint8_t* scales_end[2] = {nullptr, nullptr};
    const long long n_scales = static_cast<long long>(p.b.num_blocks) * bs * p.b.num_kv_heads;
    scales_end[0] = p.b.k_scales + n_scales;
    scales_end[1] = p.b.v_scales + n_scales;
    // A scale byte on its way to word `w`; returns its place there.  The word around it
    // is copied where it lies within the scales, else the byte is loaded.
    auto load_scale = [&](uint32_t* w, const uint8_t* scales, const uint8_t* end, long long i) -> uint32_t {
        const uint8_t* src = scales + i;
        const uint32_t b = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src) & 3u);
        if (src - b >= scales && src - b + 4 <= end) {
            cp_async_word_of(static_cast<uint32_t>(__cvta_generic_to_shared(w)), src);
            return b;
        }
        *w = *src;
        return 0u;
    };
    // the step whose rows `row` holds: its note, and its scales in the next group of copies
    auto note = [&](int slot) {
        uint32_t meta = 0u;
        if (row >= 0) {
            meta = 16u;
            const long long at = static_cast<long long>(row) * p.b.num_kv_heads + kvh;
            meta |= load_scale(&s_sk[warp][slot][lane], p.b.k_scales, scales_end[0], at);
            meta |= load_scale(&s_sv[warp][slot][lane], p.b.v_scales, scales_end[1], at) << 2;
        }
        s_meta[warp][slot][lane] = meta;
    };
    uint8_t* ring = smem + warp * F::kWarpRing + lane * 16;   // this lane's 16 bytes of each 512
    const uint32_t ring32 = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    auto load_keys = [&](int at) {     // of the step whose rows `row` holds
#pragma unroll
        for (int i = 0; i < 2 * SUB; ++i) {
            const int r = __shfl_sync(0xffffffffu, row, g + 8 * i);
            const uint8_t* src = kc + (r < 0 ? 0 : r) * pitch + c * 16;
#pragma unroll
            for (int v = 0; v < kKeyVecs; ++v)
                cp_async_16(ring32 + at * F::kKeyBytes + (i * kKeyVecs + v) * 512, src + v * 64, r >= 0);
        }
        cp_async_commit();
    };
    auto load_values = [&](int at) {
#pragma unroll
        for (int i = 0; i < 4 * SUB; ++i) {
            const int r = __shfl_sync(0xffffffffu, row, 2 * c + (i & 1) + 8 * (i >> 1));
            const uint8_t* src = vc + (r < 0 ? 0 : r) * pitch + (kHalf ? (g >> 1) : g) * 16;
#pragma unroll
            for (int v = 0; v < kValVecs; ++v)
                cp_async_16(ring32 + A * F::kKeyBytes + at * F::kValBytes + (i * kValVecs + v) * 512, src + v * 128, r >= 0);
        }
        cp_async_commit();
    };
    // Steps in turn: copies are issued A steps ahead of their use, rows found one step
    // before that, block-table entries loaded one before that.
    const int i0 = keys.begin + warp;
    look_up(i0);
    find(i0);
    look_up(i0 + kWarps);
#pragma unroll
    for (int a = 0; a < A; ++a) {
        note(a);
        load_keys(a);
        load_values(a);
        find(i0 + (a + 1) * kWarps);
        look_up(i0 + (a + 2) * kWarps);
    }
    // ---- Q: 16-bit rows in shared memory; rows that do not exist are zero ----
    if (threadIdx.x == 0) s_flag = 0;
    for (int r = warp; r < F::kRows; r += kWarps) {
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
        // times a power of two that brings the row's largest value to [2^14, 2^15)
        m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
        const int e = max(-126, min(static_cast<int>(m >> 7) - 127 - 14, 113));
        const float f = exp2f(static_cast<float>(-e));
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
            w[i] = f16x2(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
        if (lane == 0) s_scale[r] = row_factor(p.scale_log2, e);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) *reinterpret_cast<uint32_t*>(s_q + r * kPitch + (i * 32 + lane) * 2) = w[i];
    }
    __syncthreads();

    // this lane's rows: 8 n + 2c and 8 n + 2c + 1 (columns 2c, 2c + 1 of S^T n)
    float row_scale[R][2], m[R][2], l[R][2];
    int row_pos[R][2], row_lo[R][2];
    float o[R][kDim][4];
#pragma unroll
    for (int n8 = 0; n8 < R; ++n8) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 8 * n8 + 2 * c + i;
            row_scale[n8][i] = s_scale[r];
            row_pos[n8][i] = r < rows ? pos0 + (row0 + r) / p.group : -1;
            row_lo[n8][i] = window_start(row_pos[n8][i], p.window);
            m[n8][i] = -INFINITY;
            l[n8][i] = 0.f;
        }
#pragma unroll
        for (int d = 0; d < kDim; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n8][d][i] = 0.f;
    }
    const int lo_max = window_start(pmax, p.window);
    // o holds 2^(5 - E) of its values (ScaleRange), and weights, o and l 2^7 more
    ScaleRange scales;
    bool wide = false;

    int at = 0, slot = 0, slot_in = A;   // ring place; places of this step's note and of the next one written
    for (int i = i0; i < keys.end; i += kWarps) {
        const int base = keys.base(i);
        cp_async_wait<2 * A - 1>();      // this step's keys and scales
        __syncwarp();
        const uint32_t meta = s_meta[warp][slot][mine];
        const bool holds = (meta & 16u) != 0;
        uint32_t kb_now = 127u, vb_now = 127u;
        if (holds) {
            kb_now = (s_sk[warp][slot][mine] >> (8 * (meta & 3u))) & 255u;
            vb_now = (s_sv[warp][slot][mine] >> (8 * ((meta >> 2) & 3u))) & 255u;
        }
        if (++slot > A) slot = 0;
        const uint32_t have = __ballot_sync(0xffffffffu, holds);   // positions that hold a key
        const uint8_t* ks = ring + at * F::kKeyBytes;
        // S^T, 16 positions at a time
        float s[R][SUB][4];
#pragma unroll
        for (int b = 0; b < SUB; ++b) {
            float t[R][2][4];   // two chains of MMAs
#pragma unroll
            for (int n8 = 0; n8 < R; ++n8)
#pragma unroll
                for (int k = 0; k < 4; ++k) t[n8][0][k] = t[n8][1][k] = 0.f;
#pragma unroll
            for (int v = 0; v < kKeyVecs; ++v) {
                const uint4 k0 = *reinterpret_cast<const uint4*>(ks + (2 * b * kKeyVecs + v) * 512);
                const uint4 k1 = *reinterpret_cast<const uint4*>(ks + ((2 * b + 1) * kKeyVecs + v) * 512);
                const uint32_t x[2][4] = {{k0.x, k0.y, k0.z, k0.w}, {k1.x, k1.y, k1.z, k1.w}};
                const uint16_t* qs = s_q + g * kPitch + v * 4 * kVec + c * kVec;
#pragma unroll
                for (int h = 0; h < 2; ++h) {   // 8 values of each row: two MMAs
                    uint32_t a[2][4];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        a[u][0] = e4m3x2_f16x2(x[0][2 * h + u]);
                        a[u][1] = e4m3x2_f16x2(x[1][2 * h + u]);
                        a[u][2] = e4m3x2_f16x2(x[0][2 * h + u] >> 16);
                        a[u][3] = e4m3x2_f16x2(x[1][2 * h + u] >> 16);
                    }
#pragma unroll
                    for (int n8 = 0; n8 < R; ++n8) {
                        const uint4 q = *reinterpret_cast<const uint4*>(qs + n8 * 8 * kPitch + h * 8);
                        mma16816(t[n8][0], a[0][0], a[0][1], a[0][2], a[0][3], q.x, q.y);
                        mma16816(t[n8][1], a[1][0], a[1][1], a[1][2], a[1][3], q.z, q.w);
                    }
                }
            }
#pragma unroll
            for (int n8 = 0; n8 < R; ++n8)
#pragma unroll
                for (int k = 0; k < 4; ++k) s[n8][b][k] = t[n8][0][k] + t[n8][1][k];
        }
        // a later step's keys on their way to this one's place
        note(slot_in);
        if (++slot_in > A) slot_in = 0;
        load_keys(at);
        // weights: lane (g, c) has positions g + 8 k and rows 8 n + 2c, 8 n + 2c + 1
        float kf[2 * SUB];
        const float own_k = e8m0_value(kb_now);
#pragma unroll
        for (int k = 0; k < 2 * SUB; ++k) kf[k] = __shfl_sync(0xffffffffu, own_k, g + 8 * k);
        // the range of V's exponents, the least scale (that of all-zero rows) left out
        const bool h = holds && vb_now > 10u && vb_now != 255u;
        const int top = __reduce_max_sync(0xffffffffu, h ? static_cast<int>(vb_now) - 127 : -1000);
        const bool far = holds && k_scale_too_large(kb_now);   // out of any range
        const int low = __reduce_min_sync(0xffffffffu, far ? -1000 : (h ? static_cast<int>(vb_now) - 127 : 1000));
        const int before = scales.E;
        wide = scales.take(top, low) || wide;
        const float grow_e = exp2_fast(static_cast<float>(before - scales.E));
        // this lane's values: positions 2c + 8k and 2c + 8k + 1
        uint32_t vf[2 * SUB];
        {
            uint32_t pair = holds ? scales.factor(vb_now) : 0x3c00u;
            pair |= __shfl_down_sync(0xffffffffu, pair, 1) << 16;
#pragma unroll
            for (int k = 0; k < 2 * SUB; ++k) vf[k] = __shfl_sync(0xffffffffu, pair, 2 * c + 8 * k);
        }
        const bool masked = have != 0xffffffffu || base + F::kGroup - 1 > pmin ||
                            (base < lo_max && base + F::kGroup > p.sinks);
        uint32_t pt[R][2 * SUB];
#pragma unroll
        for (int n8 = 0; n8 < R; ++n8) {
            float x[2 * SUB][2];
#pragma unroll
            for (int k = 0; k < 2 * SUB; ++k)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    x[k][q] = s[n8][k >> 1][2 * (k & 1) + q];
                    x[k][q] *= kf[k];
                }
            if (masked) {
#pragma unroll
                for (int k = 0; k < 2 * SUB; ++k)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int pl = g + 8 * k, t = base + pl;
                        const bool seen = ((have >> pl) & 1u) != 0 && t <= row_pos[n8][q] &&
                                          (t >= row_lo[n8][q] || t < p.sinks);
                        if (!seen) x[k][q] = -INFINITY;
                    }
            }
            float mn[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float t = fmaxf(x[0][q], x[1][q]);
                if constexpr (SUB == 2) t = max3(t, x[2][q], x[3][q]);
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                mn[q] = fmaxf(m[n8][q], t * row_scale[n8][q]);
            }
            // O and l move to a new maximum only once it is 2^8 larger (O also with E)
            if (__any_sync(0xffffffffu, mn[0] > m[n8][0] + 8.f || mn[1] > m[n8][1] + 8.f) || grow_e != 1.f) {
                float f[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    f[k] = 1.f;
                    if (mn[k] > m[n8][k] + 8.f) {
                        f[k] = exp2_fast(m[n8][k] - mn[k]);
                        m[n8][k] = mn[k];
                    }
                    l[n8][k] *= f[k];
                    f[k] *= grow_e;
                }
#pragma unroll
                for (int d = 0; d < kDim; ++d) {
                    o[n8][d][0] *= f[0];
                    o[n8][d][1] *= f[1];
                    o[n8][d][2] *= f[0];
                    o[n8][d][3] *= f[1];
                }
            }
            float b[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                b[q] = m[n8][q] == -INFINITY ? 0.f : m[n8][q];
                b[q] -= kWeightLog2;
            }
#pragma unroll
            for (int k = 0; k < 2 * SUB; ++k) {   // positions g + 8 k
                float w[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    w[q] = exp2_fast(fmaf(x[k][q], row_scale[n8][q], -b[q]));
                    l[n8][q] += w[q];
                }
                pt[n8][k] = transpose8x8(f16x2(w[0], w[1]));
            }
        }
        // O^T
        cp_async_wait<2 * A - 1>();      // this group's values
        const uint8_t* vs = ring + A * F::kKeyBytes + at * F::kValBytes;
        if (__any_sync(0xffffffffu, holds && vb_now <= 10u)) {
            // rows at the least scale: all zeros, or a code whose value this sum leaves out?
#pragma unroll
            for (int k = 0; k < 4 * SUB; ++k) {
                const bool none = ((k & 1) != 0 ? vf[k >> 1] >> 16 : vf[k >> 1] & 0xffffu) == 0u;
#pragma unroll
                for (int v = 0; v < kValVecs; ++v) {
                    const uint4 x = *reinterpret_cast<const uint4*>(vs + (k * kValVecs + v) * 512);
                    wide = wide || (none && ((x.x | x.y | x.z | x.w) & 0x7f7f7f7fu) != 0u);
                }
            }
        }
#pragma unroll
        for (int b = 0; b < SUB; ++b) {
#pragma unroll
            for (int v = 0; v < kValVecs; ++v) {
                uint32_t y[4][4];   // positions 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 x = *reinterpret_cast<const uint4*>(vs + ((4 * b + k) * kValVecs + v) * 512);
                    y[k][0] = x.x;
                    y[k][1] = x.y;
                    y[k][2] = x.z;
                    y[k][3] = x.w;
                    if constexpr (kHalf) {
                        if (g & 1) {
                            y[k][0] = y[k][2];
                            y[k][1] = y[k][3];
                        }
                    }
                }
                constexpr int kPairs = kHalf ? 4 : kVec / 2;   // pairs of dimensions a lane has per position
                // two positions' codes byte by byte beside each other, four dimensions at a time
#pragma unroll
                for (int d = 0; d < kPairs; d += 2) {
                    const uint32_t u0 = __byte_perm(y[0][d >> 1], y[1][d >> 1], 0x5140);
                    const uint32_t u1 = __byte_perm(y[0][d >> 1], y[1][d >> 1], 0x7362);
                    const uint32_t u2 = __byte_perm(y[2][d >> 1], y[3][d >> 1], 0x5140);
                    const uint32_t u3 = __byte_perm(y[2][d >> 1], y[3][d >> 1], 0x7362);
                    const uint32_t f0 = vf[2 * b], f1 = vf[2 * b + 1];
                    const uint32_t a[2][4] = {
                        {mul_f16x2(e4m3x2_f16x2(u0), f0), mul_f16x2(e4m3x2_f16x2(u0 >> 16), f0),
                         mul_f16x2(e4m3x2_f16x2(u2), f1), mul_f16x2(e4m3x2_f16x2(u2 >> 16), f1)},
                        {mul_f16x2(e4m3x2_f16x2(u1), f0), mul_f16x2(e4m3x2_f16x2(u1 >> 16), f0),
                         mul_f16x2(e4m3x2_f16x2(u3), f1), mul_f16x2(e4m3x2_f16x2(u3 >> 16), f1)}};
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int n8 = 0; n8 < R; ++n8)
                            mma16816(o[n8][v * kPairs + d + u], a[u][0], a[u][1], a[u][2], a[u][3],
                                           pt[n8][2 * b], pt[n8][2 * b + 1]);
                }
            }
        }
        load_values(at);
        if (++at == A) at = 0;
        find(i + (A + 1) * kWarps);
        look_up(i + (A + 2) * kWarps);
    }
    cp_async_wait<0>();
    __syncthreads();   // the ring becomes s_o

    // ---- the warps' results ---------------------------------------------------
    const float plain = exp2f(static_cast<float>(scales.E - 5) - kWeightLog2);
    constexpr int kPairs = kHalf ? 4 : kVec / 2;
#pragma unroll
    for (int n8 = 0; n8 < R; ++n8) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float t = l[n8][k];
            t += __shfl_xor_sync(0xffffffffu, t, 4);
            t += __shfl_xor_sync(0xffffffffu, t, 8);
            t += __shfl_xor_sync(0xffffffffu, t, 16);
            if (g == 0) {
                s_m[warp][8 * n8 + 2 * c + k] = m[n8][k];
                s_l[warp][8 * n8 + 2 * c + k] = t * exp2f(-kWeightLog2);
            }
        }
#pragma unroll
        for (int d = 0; d < kDim; ++d) {
            const int dim = kHalf ? g * 8 + d * 2 : (d / kPairs) * (8 * kVec) + g * kVec + (d % kPairs) * 2;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                *reinterpret_cast<float2*>(s_o + (warp * F::kRows + 8 * n8 + 2 * c + k) * HD + dim) =
                    make_float2(o[n8][d][k] * plain, o[n8][d][2 + k] * plain);
        }
    }
    if (__any_sync(0xffffffffu, wide) && lane == 0) atomicOr(&s_flag, 0xffff);
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
            const float4 v = *reinterpret_cast<const float4*>(s_o + (w * F::kRows + r) * HD + d);
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
            repair_row<true, HD, F::kGroup>(p, table, keys, kvh, first + my / p.group, kvh * p.group + my % p.group,
                                         pos0 + my / p.group, seg);
        }
    }
}

}  // namespace

template <int HD>
cudaError_t launch_few_rows(const AttnParams& p, int rows, bool pdl, cudaStream_t stream)
{
    const long long ctas = static_cast<long long>(p.tiles) * p.b.num_kv_heads * p.b.num_seqs * p.segments;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto launch = [&](auto kern, int threads, int bytes, SmemOptIn& smem_opt) {
        const cudaError_t e = smem_opt.ensure(reinterpret_cast<const void*>(kern), bytes);
        if (e != cudaSuccess) return e;
        return launch_kernel(kern, dim3(static_cast<unsigned>(ctas)), dim3(threads), bytes, stream, pdl, p);
    };
    static SmemOptIn one, two;
    if constexpr (HD < 256) {
        if (rows > 8) return launch(kv_few_rows_kernel<HD, 2>, Few<HD, 2>::kWarps * 32, Few<HD, 2>::kBytes, two);
    }
    return launch(kv_few_rows_kernel<HD, 1>, Few<HD, 1>::kWarps * 32, Few<HD, 1>::kBytes, one);
}

template cudaError_t launch_few_rows<64>(const AttnParams&, int, bool, cudaStream_t);
template cudaError_t launch_few_rows<128>(const AttnParams&, int, bool, cudaStream_t);
template cudaError_t launch_few_rows<256>(const AttnParams&, int, bool, cudaStream_t);

}  // namespace kv
}  // namespace bsk
