// kv_attention.cu -- attention of new tokens over the paged cache, on the
// tensor cores (kv_attention_kernel), and the join of split rows (kv_join_kernel).
//
//   out = sum_t w_t v_t / sum_t w_t,  w_t = 2^(x_t - m),  x_t = scale * log2(e) * q.k_t
//
// over the positions t that a query sees, in one pass over the keys: the running
// maximum m, the sum l of the weights and the weighted sum O of the values are
// kept per query row in FP32, and O and l are multiplied by 2^(m - m') when the
// maximum moves to m'.  It is moved only once it is 2^8 too small (the weights
// then stay below 2^8, which costs no precision), so O is seldom touched.
//
// A CTA has 128 query rows (token x query head, the heads of one KV head side by
// side, so they share the keys) and walks 128-position tiles of the keys:
//   S = Q K^T   tcgen05.mma, Q and K from shared memory, S in TMEM, two buffers
//   P = 2^(..)  eight warps, S from TMEM to registers and P back, as BF16, over S
//   O += P V    tcgen05.mma, P from TMEM, V from shared memory, O in TMEM
// The MMAs of S for tile j+1 and of PV for tile j-1 run while the warps work on
// tile j.  TMEM: 2 x 128 columns of S, head_dim columns of O.
#include <cmath>
#include <cstdio>

#include "bsk_internal.h"
#include "kv_internal.h"
#include "ptx.cuh"

namespace bsk {
namespace {

// ---------------------------------------------------------------------------
// PTX that only this kernel needs
// ---------------------------------------------------------------------------

// Four rows of a 2-D tensor (box: one row of 64 elements), 128 bytes each.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int4 rows)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(rows.x), "r"(rows.y), "r"(rows.z), "r"(rows.w)
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem desc], A 128 x 16 BF16, two values per column.
__device__ __forceinline__ void mma_f16_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void named_barrier(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

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
// 16 bytes global -> shared, asynchronous; `in` false: zeros.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// ---------------------------------------------------------------------------
// Geometry
// ---------------------------------------------------------------------------
constexpr int kRows = 128;        // query rows per CTA (the M of the MMAs)
constexpr int kTile = 128;        // key positions per tile
constexpr int kProducers = 128;   // threads of warps 0..3
constexpr int kSoftmax = 256;     // threads of warps 4..11
constexpr int kThreads = kProducers + kSoftmax + 32;   // warp 12 issues the MMAs
constexpr int kStageBytes = 16384;
constexpr int kSlots = 8;         // tiles whose masks and scales are kept
constexpr int kStaging = 4;       // E4M3: stages of raw codes on their way

enum AttnSite : int { kSiteKvEmpty = 0x30, kSiteKvFull, kSiteKvQ, kSiteKvScores, kSiteKvWeights, kSiteKvOutput, kSiteKvDrain };

template <bool E4M3, int HD>
struct Geo {
    static constexpr int kBlocks = HD / 64;                    // 64-element (128-byte) blocks of a row
    static constexpr int kQBytes = kRows * HD * 2;
    // K stage: 128 positions x 64 dimensions; V stage: kVTok positions x HD
    static constexpr int kVTok = kStageBytes / (HD * 2);
    static constexpr int kStages = HD == 256 ? (E4M3 ? 7 : 9) : (E4M3 ? 8 : 10);
    static constexpr int kStagingBytes = E4M3 ? kStaging * 8192 : 0;
    static constexpr int kScaleBytes = E4M3 ? kSlots * kTile * 12 : 0;   // K and V factors, row indexes
    static constexpr int kMisc = kSlots * 16 + 2 * 2 * kRows * 4 + kRows * 4 + (2 * kStages + 8) * 8 + 16;
    static constexpr int kBytes = 1024 + kQBytes + kStages * kStageBytes + kStagingBytes + kScaleBytes + kMisc;
    static_assert(kBytes <= 232448, "shared memory of one CTA");
};

struct AttnParams {
    KvBatch b;
    const uint16_t* q;
    uint16_t* out;
    long long q_stride, out_stride;
    int num_q_heads, group, max_chunk, max_seq_len;
    int tiles, segments;          // row tiles per sequence and KV head, key segments per tile
    float scale_log2;             // |softmax scale| * log2(e), > 0
    uint32_t q_sign;              // 0x80008000 for a negative scale
    int window, sinks;
    float* part_o;                // [rows][segments][HD] unnormalised O
    float2* part_ml;              // [rows][segments] (m, l)
    unsigned long long wait_limit_ns;
};

// The key tiles that some row of a CTA sees: those of the sinks, then those from
// the window's first on.  A position holds a key when it is below kv_end and not
// between sink_end and lo.
struct Keys {
    int sink_tiles, lo_tile;      // tile i lies at i, or at i - sink_tiles + lo_tile
    int begin, end;               // this segment's tiles
    int lo, sink_end, kv_end;
    __device__ __forceinline__ int base(int i) const { return (i < sink_tiles ? i : i - sink_tiles + lo_tile) * kTile; }
    __device__ __forceinline__ bool holds(int t) const { return t < kv_end && (t >= lo || t < sink_end); }
};

// ---------------------------------------------------------------------------
// One row by one warp, in FP32: for rows whose O is not finite although their
// weights are, which happens when a value that the row does not see holds an
// Inf or a NaN (its weight 0 times that is NaN on the tensor cores).
// ---------------------------------------------------------------------------
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
__device__ __noinline__ void repair_row(const AttnParams& p, const int32_t* table, const Keys& keys, int kvh, int token,
                                        int head, int pos, int seg)
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
    const int lo = p.window > 0 && pos - p.window + 1 > 0 ? pos - p.window + 1 : 0;
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

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
template <bool E4M3, int HD>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attention_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ AttnParams p)
{
    using G = Geo<E4M3, HD>;
    constexpr int S = G::kStages;
    constexpr int NB = G::kBlocks;      // K stages of a tile
    constexpr int VT = G::kVTok;
    constexpr uint32_t kIdescS = idesc_f16(true, false, false, kRows, kTile);
    constexpr uint32_t kIdescO = idesc_f16(true, false, true, kRows, HD);

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* sQ = smem;
    uint8_t* ring = sQ + G::kQBytes;
    uint8_t* staging = ring + S * kStageBytes;
    float* s_kf = reinterpret_cast<float*>(staging + G::kStagingBytes);   // E4M3: [kSlots][kTile] K scales
    float* s_vf = s_kf + (E4M3 ? kSlots * kTile : 0);                     //       V scales
    int* s_row = reinterpret_cast<int*>(s_vf + (E4M3 ? kSlots * kTile : 0));   //  cache rows (-1: none)
    uint32_t* s_mask = reinterpret_cast<uint32_t*>(s_row + (E4M3 ? kSlots * kTile : 0));   // [kSlots][4] positions that hold a key
    float* s_max = reinterpret_cast<float*>(s_mask + kSlots * 4);         // [2][2][kRows]
    int* s_flag = reinterpret_cast<int*>(s_max + 4 * kRows);              // [kRows] rows to repair
    uint64_t* bars = reinterpret_cast<uint64_t*>(s_flag + kRows);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 8);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    const uint32_t full0 = smem_u32(bars);          // S: stage filled
    const uint32_t empty0 = full0 + 8 * S;          // S: stage read
    const uint32_t q_full = empty0 + 8 * S;         // Q in shared memory
    const uint32_t s_full0 = q_full + 8;            // 2: scores ready
    const uint32_t p_full0 = s_full0 + 16;          // 2: weights ready
    // 2 (tiles in turn): a tile's PV done.  One barrier would not do: with tile j's
    // scores at hand, PV of j - 2 is done, but those of j - 1 and j may or may not
    // be, and a wait tells two neighbouring phases apart, not three.
    const uint32_t o_done0 = p_full0 + 16;
    const uint32_t drain = o_done0 + 16;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    griddep_wait();
    griddep_launch_dependents();

    // ---- which rows, which keys -------------------------------------------
    int idx = blockIdx.x;
    const int tile = p.tiles - 1 - idx % p.tiles;   // the tiles with the most keys first
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
    const int row0 = tile * kRows;
    const int rows = min(kRows, n * p.group - row0);
    if (rows <= 0) return;
    const int pos0 = len - n;                              // position of the sequence's first new token
    const int pmin = pos0 + row0 / p.group, pmax = pos0 + (row0 + rows - 1) / p.group;
    Keys keys;
    keys.kv_end = max(pmax + 1, 0);
    keys.lo = p.window > 0 && pmin - p.window + 1 > 0 ? pmin - p.window + 1 : 0;
    keys.sink_end = min(p.sinks, keys.lo);
    keys.lo_tile = keys.lo / kTile;
    keys.sink_tiles = min((keys.sink_end + kTile - 1) / kTile, keys.lo_tile);
    {
        const int total = keys.kv_end > 0 ? keys.sink_tiles + (keys.kv_end + kTile - 1) / kTile - keys.lo_tile : 0;
        keys.begin = static_cast<int>(static_cast<long long>(total) * seg / p.segments);
        keys.end = static_cast<int>(static_cast<long long>(total) * (seg + 1) / p.segments);
    }
    const int32_t* table = p.b.block_tables + static_cast<long long>(seq) * p.b.max_blocks;
    const int nt = keys.end - keys.begin;
    if (nt <= 0) {
        // nothing to see in this segment
        if (p.segments == 1) {
            for (int i = threadIdx.x; i < rows * (HD / 8); i += kThreads) {
                const int r = row0 + i / (HD / 8);
                uint16_t* o = p.out + (first + r / p.group) * p.out_stride +
                              (static_cast<long long>(kvh) * p.group + r % p.group) * HD + (i % (HD / 8)) * 8;
                *reinterpret_cast<uint4*>(o) = make_uint4(0, 0, 0, 0);
            }
        } else {
            for (int i = threadIdx.x; i < rows; i += kThreads) {
                const int r = row0 + i;
                const long long at = (static_cast<long long>(first + r / p.group) * p.num_q_heads +
                                      kvh * p.group + r % p.group) * p.segments + seg;
                p.part_ml[at] = make_float2(-INFINITY, 0.f);
            }
        }
        return;
    }

    // ---- barriers, TMEM ----------------------------------------------------
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, E4M3 ? kProducers / 32 : 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(q_full, kSoftmax / 32);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full0 + 8 * i, 1);
            mbar_init(p_full0 + 8 * i, kSoftmax / 32);
            mbar_init(o_done0 + 8 * i, 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == 12) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish_alloc_permit();
    }
    if (warp >= 4 && warp < 12) {
        for (int i = threadIdx.x - kProducers; i < kRows; i += kSoftmax) s_flag[i] = 0;
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const WaitCtl wc{abort_flag, p.b.status, p.wait_limit_ns};
    uint32_t never = 0u;
    const WaitCtl wc_drain{&never, p.b.status, p.wait_limit_ns};
    // V stages of tile i: positions past kv_end are not multiplied
    auto v_stages = [&](int i) { return (min(kTile, keys.kv_end - keys.base(i)) + VT - 1) / VT; };

    if (warp < 4) {
        // ------------------------------------------------------------------
        // Producers: K of tile 0, K 1, V 0, K 2, V 1, ... (the MMAs' order)
        // ------------------------------------------------------------------
        int stage = 0;
        uint32_t phase = 0;
        if constexpr (!E4M3) {
            // warp 0: lane i holds the cache rows of positions 4i .. 4i+3 of a tile and
            // gathers them; a position without a key reads past the last row: zeros
            if (warp == 0) {
                const int none = p.b.num_blocks * p.b.block_size;
                long long issued = 0;
                bool ok = true;
                auto rows_of = [&](int i) {
                    int r[4];
                    uint32_t have = 0;
                    const int t = keys.base(i) + 4 * lane;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const long long row = keys.holds(t + u) ? kv_row(p.b, table, t + u) : -1;
                        r[u] = row < 0 ? none : static_cast<int>(row);
                        have |= (row < 0 ? 0u : 1u) << u;
                    }
                    // 8 lanes' bits make one word of the tile's mask
                    have <<= 4 * (lane & 7);
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) have |= __shfl_xor_sync(0xffffffffu, have, o);
                    if ((lane & 7) == 0) s_mask[((i - keys.begin) % kSlots) * 4 + (lane >> 3)] = have;
                    __syncwarp();
                    return make_int4(r[0], r[1], r[2], r[3]);
                };
                auto next = [&](uint32_t& dst, uint32_t& bar) {
                    ok = __all_sync(0xffffffffu, mbar_wait(empty0 + 8 * stage, phase ^ 1u, wc, kSiteKvEmpty));
                    if (!ok) return;
                    dst = smem_u32(ring + stage * kStageBytes);
                    bar = full0 + 8 * stage;
                    if (lane == 0) mbar_arrive_expect_tx(bar, kStageBytes);
                    __syncwarp();
                    ++issued;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                };
                auto load_k = [&](const int4& r) {
                    for (int kb = 0; kb < NB && ok; ++kb) {
                        uint32_t dst, bar;
                        next(dst, bar);
                        if (ok) tma_gather4(dst + lane * 512, &tmK, bar, kvh * HD + kb * 64, r);
                    }
                };
                auto load_v = [&](const int4& r, int count) {
                    constexpr int GR = VT / 4;   // gathers per 64-element block of a stage
                    const int g = lane % GR, blk = lane / GR;
                    for (int v = 0; v < count && ok; ++v) {
                        uint32_t dst, bar;
                        next(dst, bar);
                        int4 x;
                        x.x = __shfl_sync(0xffffffffu, r.x, v * GR + g);
                        x.y = __shfl_sync(0xffffffffu, r.y, v * GR + g);
                        x.z = __shfl_sync(0xffffffffu, r.z, v * GR + g);
                        x.w = __shfl_sync(0xffffffffu, r.w, v * GR + g);
                        if (ok) tma_gather4(dst + blk * (VT * 128) + g * 512, &tmV, bar, kvh * HD + blk * 64, x);
                    }
                };
                int4 cur = rows_of(keys.begin);
                load_k(cur);
                for (int i = keys.begin; i < keys.end && ok; ++i) {
                    int4 nxt = cur;
                    if (i + 1 < keys.end) {
                        nxt = rows_of(i + 1);
                        load_k(nxt);
                    }
                    if (ok) load_v(cur, v_stages(i));
                    cur = nxt;
                }
                if (!ok) {
                    // abort: the loads already issued land before the CTA exits
                    const long long pending = issued < S ? issued : S;
                    for (long long j = 1; j <= pending; ++j) {
                        const int s = (stage - static_cast<int>(j) + S) % S;
                        const uint32_t ph = (stage - static_cast<int>(j) < 0) ? (phase ^ 1u) : phase;
                        mbar_wait(full0 + 8 * s, ph, wc_drain, kSiteKvDrain);
                    }
                }
            }
        } else {
            // All four warps: each thread copies 16-code chunks of the rows into its own
            // places of a staging ring (cp.async, kStaging - 1 stages ahead) and later
            // writes them, as BF16, where the MMAs read them.
            const int tid = threadIdx.x;
            const uint8_t* kc = static_cast<const uint8_t*>(p.b.k);
            const uint8_t* vc = static_cast<const uint8_t*>(p.b.v);
            // Rows, scales and mask of a tile, one position per thread, in two steps
            // a tile apart, so that the loads of each are in flight meanwhile.
            int pend_row = -1;
            uint32_t pend_k = 127u, pend_v = 127u;
            auto look_up = [&](int i) {
                pend_row = -1;
                pend_k = pend_v = 127u;
                if (i >= keys.end) return;
                const int t = keys.base(i) + tid;
                if (!keys.holds(t)) return;
                const long long row = kv_row(p.b, table, t);
                if (row < 0) return;
                pend_row = static_cast<int>(row);
                pend_k = p.b.k_scales[row * p.b.num_kv_heads + kvh];
                pend_v = p.b.v_scales[row * p.b.num_kv_heads + kvh];
            };
            auto publish = [&](int i) {   // what look_up(i) found
                const int slot = (i - keys.begin) % kSlots;
                const uint32_t have = __ballot_sync(0xffffffffu, pend_row >= 0);
                if (lane == 0) s_mask[slot * 4 + warp] = have;
                s_row[slot * kTile + tid] = pend_row;
                s_kf[slot * kTile + tid] = e8m0_value(pend_k);
                s_vf[slot * kTile + tid] = e8m0_value(pend_v);
                named_barrier(5, kProducers);
            };
            // The stages in order, as (tile, K or V, index); kept twice: for the copies
            // and, kStaging - 1 stages behind, for the conversion.
            struct Cursor {
                int i, j;      // tile; stage of it: 0 .. NB-1 K, then V of the tile before
                bool v;
            };
            auto advance = [&](Cursor& c) -> bool {   // to the next stage; false at the end
                // K of tile i, then V of tile i - 1
                while (true) {
                    ++c.j;
                    if (!c.v) {
                        if (c.i < keys.end && c.j < NB) return true;
                        c.v = true;
                        c.j = -1;
                    } else {
                        const int vi = c.i - 1;
                        if (vi >= keys.begin && c.j < v_stages(vi)) return true;
                        c.v = false;
                        c.j = -1;
                        if (++c.i > keys.end) return false;
                    }
                }
            };
            auto copy = [&](const Cursor& c, int buf) {
                const int i = c.v ? c.i - 1 : c.i;
                const int slot = (i - keys.begin) % kSlots;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int ch = u * kProducers + tid;
                    int t, off;
                    if (!c.v) {
                        t = ch >> 2;
                        off = c.j * 64 + (ch & 3) * 16;
                    } else {
                        t = c.j * VT + ch / (HD / 16);
                        off = (ch % (HD / 16)) * 16;
                    }
                    const int row = s_row[slot * kTile + t];
                    const uint8_t* src = (c.v ? vc : kc) +
                                         (static_cast<long long>(row < 0 ? 0 : row) * p.b.num_kv_heads + kvh) * HD + off;
                    cp_async_16(smem_u32(staging + buf * 8192 + ch * 16), src, row >= 0);
                }
            };
            auto convert = [&](const Cursor& c, int buf) {
                mbar_wait(empty0 + 8 * stage, phase ^ 1u, wc, kSiteKvEmpty);
                uint8_t* dst = ring + stage * kStageBytes;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int ch = u * kProducers + tid;
                    const uint4 x = *reinterpret_cast<const uint4*>(staging + buf * 8192 + ch * 16);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    uint32_t o[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float2 f = e4m3x2_values(w[k >> 1] >> (16 * (k & 1)));
                        o[k] = bf16x2(f.x, f.y);
                    }
                    // 128-byte rows of 64 values, their 16-byte chunks permuted by the row
                    int r, blk, c16;
                    if (!c.v) {
                        r = ch >> 2;
                        blk = 0;
                        c16 = (ch & 3) * 2;
                    } else {
                        r = ch / (HD / 16);
                        const int e = ch % (HD / 16);
                        blk = e >> 2;
                        c16 = (e & 3) * 2;
                    }
                    uint8_t* d = dst + blk * (VT * 128) + r * 128;
                    *reinterpret_cast<uint4*>(d + ((c16 ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4*>(d + (((c16 + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full0 + 8 * stage);
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            };
            Cursor ahead{keys.begin, -1, false}, behind{keys.begin, -1, false};
            look_up(keys.begin);
            publish(keys.begin);
            look_up(keys.begin + 1);
            bool more = true;
            int in = 0;
            auto step_ahead = [&]() {
                if (more) {
                    more = advance(ahead);
                    if (more) {
                        if (!ahead.v && ahead.j == 0 && ahead.i > keys.begin) {
                            publish(ahead.i);
                            look_up(ahead.i + 1);
                        }
                        copy(ahead, in % kStaging);
                    }
                }
                ++in;
                cp_async_commit();
            };
            for (int k = 0; k < kStaging - 1; ++k) step_ahead();
            for (int k = 0; advance(behind); ++k) {
                cp_async_wait<kStaging - 2>();
                convert(behind, k % kStaging);
                step_ahead();
            }
            cp_async_wait<0>();
        }
    } else if (warp == 12) {
        // ------------------------------------------------------------------
        // MMA issuer
        // ------------------------------------------------------------------
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = mbar_wait(q_full, 0, wc, kSiteKvQ);
            tc_fence_after_sync();
            const uint32_t q_base = smem_u32(sQ);
            const uint32_t o_tmem = tmem + 256;
            auto next = [&]() {
                ok = ok && mbar_wait(full0 + 8 * stage, phase, wc, kSiteKvFull);
                tc_fence_after_sync();
                return smem_u32(ring + stage * kStageBytes);
            };
            auto done = [&]() {
                mma_commit(empty0 + 8 * stage);
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            };
            auto scores = [&](int j) {
                for (int kb = 0; kb < NB && ok; ++kb) {
                    const uint32_t b = next();
                    if (!ok) break;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f16(tmem + (j & 1) * 128, smem_desc_sw128(q_base + kb * (kRows * 128) + kk * 32, 16, 1024),
                                smem_desc_sw128(b + kk * 32, 16, 1024), kIdescS, (kb | kk) != 0 ? 1u : 0u);
                    done();
                }
                if (ok) mma_commit(s_full0 + 8 * (j & 1));
            };
            auto weighted = [&](int j) {
                ok = ok && mbar_wait(p_full0 + 8 * (j & 1), (j >> 1) & 1, wc, kSiteKvWeights);
                tc_fence_after_sync();
                const int count = v_stages(keys.begin + j);
                for (int v = 0; v < count && ok; ++v) {
                    const uint32_t b = next();
                    if (!ok) break;
#pragma unroll
                    for (int kk = 0; kk < VT / 16; ++kk)
                        mma_f16_tmem_a(o_tmem, tmem + (j & 1) * 128 + (v * VT / 16 + kk) * 8,
                                       smem_desc_sw128(b + kk * 2048, VT * 128, 1024), kIdescO,
                                       (j | v | kk) != 0 ? 1u : 0u);
                    done();
                }
                if (ok) mma_commit(o_done0 + 8 * (j & 1));
            };
            if (ok) scores(0);
            for (int j = 0; j < nt && ok; ++j) {
                if (j + 1 < nt) scores(j + 1);
                if (ok) weighted(j);
            }
            if (!ok) {
                // abort: every MMA issued so far finishes before TMEM is freed
                mma_commit(drain);
                mbar_wait(drain, 0u, wc_drain, kSiteKvDrain);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------------
        // Softmax: warp (quarter, half) has TMEM lanes 32 * quarter .. and half of
        // the columns: of S positions 64 * half .., of O dimensions HD/2 * half ..
        // A failed wait (abort flag up) does not leave the loop: the barriers below
        // stay matched, the waits return at once and the output is undefined.
        // ------------------------------------------------------------------
        const int quarter = warp & 3;
        const int half = (warp - 4) >> 2;
        const int r = quarter * 32 + lane;
        const bool idle = quarter * 32 >= rows;   // the whole warp
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const int my = row0 + min(r, rows - 1);
        const int token = first + my / p.group;
        const int head = kvh * p.group + my % p.group;
        const int pos = pos0 + my / p.group;
        {
            // Q: row r's chunks, the two halves of the warps taking turns; 128-byte rows of
            // 64 values, their 16-byte chunks permuted by the row
            const uint4* src = reinterpret_cast<const uint4*>(p.q + token * p.q_stride + static_cast<long long>(head) * HD);
#pragma unroll
            for (int c = 0; c < HD / 16; ++c) {
                const int ch = half * (HD / 16) + c;
                uint4 x = make_uint4(0, 0, 0, 0);
                if (r < rows) {
                    x = src[ch];
                    x.x ^= p.q_sign;
                    x.y ^= p.q_sign;
                    x.z ^= p.q_sign;
                    x.w ^= p.q_sign;
                }
                *reinterpret_cast<uint4*>(sQ + (ch >> 3) * (kRows * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = x;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        const int lo = p.window > 0 && pos - p.window + 1 > 0 ? pos - p.window + 1 : 0;   // this row's window
        const int lo_max = p.window > 0 ? pmax - p.window + 1 : 0;                        // the last row's
        float m = -INFINITY;
        float2 l2 = make_float2(0.f, 0.f);
        for (int j = 0; j < nt; ++j) {
            const int buf = j & 1;
            const int slot = j % kSlots;
            mbar_wait(s_full0 + 8 * buf, (j >> 1) & 1, wc, kSiteKvScores);
            tc_fence_after_sync();
            if (!idle) {
                const uint32_t s_addr = lane_addr + buf * 128 + half * 64;
                uint32_t raw[2][32];
                tmem_ld_32x32b_x32(s_addr, raw[0]);
                tmem_ld_32x32b_x32(s_addr + 32, raw[1]);
                tmem_ld_wait();
                float2 x[32];
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    x[c] = make_float2(__uint_as_float(raw[c >> 4][(2 * c) & 31]), __uint_as_float(raw[c >> 4][(2 * c + 1) & 31]));
                if constexpr (E4M3) {
                    const float4* kf = reinterpret_cast<const float4*>(s_kf + slot * kTile + half * 64);
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float4 f = kf[c];
                        x[2 * c] = mul2(x[2 * c], make_float2(f.x, f.y));
                        x[2 * c + 1] = mul2(x[2 * c + 1], make_float2(f.z, f.w));
                    }
                }
                // positions that hold no key, or that this row does not see
                const int t0 = keys.base(keys.begin + j) + half * 64;
                const uint2 have = *reinterpret_cast<const uint2*>(s_mask + slot * 4 + half * 2);
                if ((have.x & have.y) != 0xffffffffu || t0 + 63 > pmin || (t0 < lo_max && t0 + 64 > p.sinks)) {
                    auto below = [](int k) {   // the k lowest of 64 bits
                        return k <= 0 ? 0ull : (k >= 64 ? ~0ull : (1ull << k) - 1);
                    };
                    const unsigned long long seen = (static_cast<unsigned long long>(have.y) << 32 | have.x) &
                                                    below(pos + 1 - t0) & (~below(lo - t0) | below(p.sinks - t0));
                    const uint32_t lo32 = static_cast<uint32_t>(seen), hi32 = static_cast<uint32_t>(seen >> 32);
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const uint32_t w = c < 16 ? lo32 : hi32;
                        if (!((w >> ((2 * c) & 31)) & 1u)) x[c].x = -INFINITY;
                        if (!((w >> ((2 * c + 1) & 31)) & 1u)) x[c].y = -INFINITY;
                    }
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 32; ++c) mx[c & 3] = max3(mx[c & 3], x[c].x, x[c].y);
                float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
                // the row's other half; also: both warps have read S, P may go over it
                float* sm = s_max + buf * 2 * kRows;
                sm[half * kRows + r] = top;
                named_barrier(1 + quarter, 64);
                top = fmaxf(top, sm[(half ^ 1) * kRows + r]) * p.scale_log2;
                const float mn = fmaxf(m, top);
                if (j == 0) {
                    m = mn;
                } else if (__any_sync(0xffffffffu, mn > m + 8.f)) {
                    float f = 1.f;
                    if (mn > m + 8.f) {
                        f = exp2_fast(m - mn);
                        m = mn;
                    }
                    const float2 f2 = make_float2(f, f);
                    l2 = mul2(l2, f2);
                    mbar_wait(o_done0 + 8 * ((j - 1) & 1), ((j - 1) >> 1) & 1, wc, kSiteKvOutput);   // PV of j - 1
                    tc_fence_after_sync();
                    // this half of the row's O
                    for (int c = 0; c < HD / 64; ++c) {
                        const uint32_t o_addr = lane_addr + 256 + half * (HD / 2) + c * 32;
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(o_addr, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st_32x32b_x32(o_addr, o);
                    }
                }
                const float base = m == -INFINITY ? 0.f : m;
                const float2 sc = make_float2(p.scale_log2, p.scale_log2), nb = make_float2(-base, -base);
                uint32_t w[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    float2 e = fma2(x[c], sc, nb);
                    e.x = exp2_fast(e.x);
                    e.y = exp2_fast(e.y);
                    l2 = add2(l2, e);
                    if constexpr (E4M3) {
                        const float2 f = *reinterpret_cast<const float2*>(s_vf + slot * kTile + half * 64 + 2 * c);
                        e = mul2(e, f);
                    }
                    w[c] = bf16x2(e.x, e.y);
                }
                tmem_st_32x32b_x32(lane_addr + buf * 128 + half * 32, w);
                tmem_st_wait();
                tc_fence_before_sync();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full0 + 8 * buf);
        }
        // ---- the rows' results ---------------------------------------------
        mbar_wait(o_done0 + 8 * ((nt - 1) & 1), ((nt - 1) >> 1) & 1, wc, kSiteKvOutput);
        tc_fence_after_sync();
        if (!idle) {
            float l = l2.x + l2.y;
            float* sm = s_max + (nt & 1) * 2 * kRows;
            sm[half * kRows + r] = l;
            named_barrier(1 + quarter, 64);
            l = sm[r] + sm[kRows + r];   // the same order for both halves
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const long long at = (static_cast<long long>(token) * p.num_q_heads + head) * p.segments + seg;
            float odd = 0.f;   // NaN once a value is not finite
            for (int c = 0; c < HD / 64; ++c) {
                const int d0 = half * (HD / 2) + c * 32;
                uint32_t o[32];
                tmem_ld_32x32b_x32(lane_addr + 256 + d0, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) odd = fmaf(__uint_as_float(o[i]), 0.f, odd);
                if (r < rows) {
                    if (p.segments == 1) {
                        uint4* dst = reinterpret_cast<uint4*>(p.out + token * p.out_stride +
                                                              static_cast<long long>(head) * HD + d0);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t h[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                h[k] = bf16x2(__uint_as_float(o[8 * i + 2 * k]) * inv, __uint_as_float(o[8 * i + 2 * k + 1]) * inv);
                            dst[i] = make_uint4(h[0], h[1], h[2], h[3]);
                        }
                    } else {
                        uint4* dst = reinterpret_cast<uint4*>(p.part_o + at * HD + d0);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
            }
            if (p.segments > 1 && half == 0 && r < rows) p.part_ml[at] = make_float2(m, l);
            if (odd != 0.f && l - l == 0.f && r < rows) s_flag[r] = 1;   // odd is NaN, l is finite
            named_barrier(1 + quarter, 64);
            for (int i = half; i < 32; i += 2) {
                const int rr = quarter * 32 + i;
                if (rr < rows && s_flag[rr]) {
                    const int row = row0 + rr;
                    repair_row<E4M3, HD>(p, table, keys, kvh, first + row / p.group, kvh * p.group + row % p.group,
                                         pos0 + row / p.group, seg);
                }
            }
        }
        tc_fence_before_sync();
    }
    __syncthreads();
    if (warp == 12) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// Joins the segments of split rows: M = max m_s, out = sum_s O_s 2^(m_s - M) /
// sum_s l_s 2^(m_s - M), in segment order.  LANES = HD / 4 threads have a row's
// four values each; with WIDE the 256 threads share one row's segments, else
// they take 256 / LANES rows.
// ---------------------------------------------------------------------------
template <int HD, bool WIDE>
__global__ void __launch_bounds__(256) kv_join_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int LANES = HD / 4;
    constexpr int GROUPS = 256 / LANES;
    __shared__ float4 s_o[GROUPS][LANES];
    __shared__ float s_l[GROUPS];
    const int g = threadIdx.x / LANES, e = threadIdx.x % LANES;
    griddep_wait();
    griddep_launch_dependents();
    const long long row = WIDE ? blockIdx.x : static_cast<long long>(blockIdx.x) * GROUPS + g;
    const int token = static_cast<int>(row / p.num_q_heads);
    // a row of some sequence
    const bool in = token < p.b.num_tokens &&
                    (p.b.cu_tokens == nullptr || (token >= p.b.cu_tokens[0] && token < p.b.cu_tokens[p.b.num_seqs]));
    const float2* ml = p.part_ml + row * p.segments;
    const float4* po = reinterpret_cast<const float4*>(p.part_o + row * p.segments * HD) + e;
    float M = -INFINITY, L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
        for (int s = 0; s < p.segments; ++s) M = fmaxf(M, ml[s].x);
        const float base = M == -INFINITY ? 0.f : M;
        const int step = WIDE ? GROUPS : 1;
#pragma unroll 4
        for (int s = WIDE ? g : 0; s < p.segments; s += step) {
            const float2 x = ml[s];
            if (x.y == 0.f) continue;   // saw nothing: its O was not written
            const float w = exp2f(x.x - base);
            const float4 v = po[static_cast<long long>(s) * LANES];
            L = fmaf(w, x.y, L);
            o.x = fmaf(w, v.x, o.x);
            o.y = fmaf(w, v.y, o.y);
            o.z = fmaf(w, v.z, o.z);
            o.w = fmaf(w, v.w, o.w);
        }
    }
    if constexpr (WIDE) {
        s_o[g][e] = o;
        if (e == 0) s_l[g] = L;
        __syncthreads();
        if (g != 0) return;
#pragma unroll
        for (int i = 1; i < GROUPS; ++i) {
            const float4 v = s_o[i][e];
            o.x += v.x;
            o.y += v.y;
            o.z += v.z;
            o.w += v.w;
            L += s_l[i];
        }
    }
    if (in) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        uint16_t* out = p.out + token * p.out_stride + (row - static_cast<long long>(token) * p.num_q_heads) * HD + 4 * e;
        *reinterpret_cast<uint2*>(out) = make_uint2(bf16x2(o.x * inv, o.y * inv), bf16x2(o.z * inv, o.w * inv));
    }
}

template <bool E4M3, int HD>
cudaError_t launch_hd(const KvAttnLaunch& a, cudaStream_t stream, char* msg, size_t msg_len)
{
    AttnParams p;
    p.b = a.b;
    p.q = a.q;
    p.out = a.out;
    p.q_stride = a.q_stride;
    p.out_stride = a.out_stride;
    p.num_q_heads = a.num_q_heads;
    p.group = a.num_q_heads / a.b.num_kv_heads;
    p.max_chunk = a.max_chunk;
    p.max_seq_len = a.max_seq_len;
    const long long max_rows = static_cast<long long>(a.max_chunk) * p.group;
    p.tiles = static_cast<int>((max_rows + kRows - 1) / kRows);
    p.segments = a.segments;
    // a zero scale still has to keep -inf (a position not seen) at -inf
    p.scale_log2 = a.scale == 0.f ? 1e-37f : std::fabs(a.scale) * 1.4426950408889634f;
    p.q_sign = a.scale < 0.f ? 0x80008000u : 0u;
    p.window = a.window;
    p.sinks = a.sinks;
    p.part_o = a.workspace;
    const long long rows = static_cast<long long>(a.b.num_tokens) * a.num_q_heads;
    p.part_ml = reinterpret_cast<float2*>(a.workspace + rows * a.segments * HD);
    p.wait_limit_ns = a.wait_limit_ns;
    CUtensorMap maps[2] = {};
    if constexpr (!E4M3) {
        TmapEncodeFn enc = tmap_encoder();
        if (enc == nullptr) {
            snprintf(msg, msg_len, "cuTensorMapEncodeTiled is not available from the driver");
            return cudaErrorNotSupported;
        }
        const cuuint64_t width = static_cast<cuuint64_t>(a.b.num_kv_heads) * HD;
        const cuuint64_t dims[2] = {width, static_cast<cuuint64_t>(a.b.num_blocks) * a.b.block_size};
        const cuuint64_t strides[1] = {width * 2};
        const cuuint32_t box[2] = {64, 1}, ones[2] = {1, 1};
        for (int i = 0; i < 2; ++i) {
            const CUresult r = enc(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, i == 0 ? a.b.k : a.b.v, dims, strides,
                                   box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
            if (r != CUDA_SUCCESS) {
                snprintf(msg, msg_len, "cuTensorMapEncodeTiled failed (%d) for the cache", static_cast<int>(r));
                return cudaErrorInvalidValue;
            }
        }
    }
    auto kern = kv_attention_kernel<E4M3, HD>;
    static SmemOptIn smem_opt;
    cudaError_t e = smem_opt.ensure(reinterpret_cast<const void*>(kern), Geo<E4M3, HD>::kBytes);
    if (e != cudaSuccess) return e;
    const long long ctas = static_cast<long long>(p.tiles) * a.b.num_kv_heads * a.b.num_seqs * a.segments;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    e = launch_kernel(kern, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), Geo<E4M3, HD>::kBytes, stream, a.pdl,
                      maps[0], maps[1], p);
    if (e != cudaSuccess || a.segments == 1) return e;
    constexpr int kPerCta = 256 / (HD / 4);
    if (rows < 4 * a.num_sms)
        return launch_kernel(kv_join_kernel<HD, true>, dim3(static_cast<unsigned>(rows)), dim3(256), 0, stream, a.pdl, p);
    return launch_kernel(kv_join_kernel<HD, false>, dim3(static_cast<unsigned>((rows + kPerCta - 1) / kPerCta)), dim3(256),
                         0, stream, a.pdl, p);
}

}  // namespace

int kv_attention_segments(const KvAttnLaunch& a)
{
    const long long group = a.num_q_heads / a.b.num_kv_heads;
    const long long per_seq = (static_cast<long long>(a.max_chunk) * group + kRows - 1) / kRows;
    long long row_tiles = (static_cast<long long>(a.b.num_tokens) * group + kRows - 1) / kRows + a.b.num_seqs - 1;
    if (row_tiles > per_seq * a.b.num_seqs) row_tiles = per_seq * a.b.num_seqs;
    const long long ctas = row_tiles * a.b.num_kv_heads;
    long long keys = a.max_seq_len;
    if (a.window > 0 && static_cast<long long>(a.window) + a.max_chunk + a.sinks < keys)
        keys = static_cast<long long>(a.window) + a.max_chunk + a.sinks;
    const long long tiles = (keys + kTile - 1) / kTile;
    const double rows = static_cast<double>(a.b.num_tokens) * a.num_q_heads;
    // Time in units of one tile's work on one CTA: a CTA starts and ends in about
    // 6, a join costs about 6 more and the traffic of the partial rows.
    double best = 0;
    int segments = 1;
    for (int s = 1; s <= 64 && (s == 1 || s <= tiles); ++s) {
        const long long waves = (ctas * s + a.num_sms - 1) / a.num_sms;
        double t = static_cast<double>(waves) * (6 + static_cast<double>((tiles + s - 1) / s));
        if (s > 1) t += 6 + rows * s * a.b.head_dim * 8 / 3.5e6;
        if (s == 1 || t < best) {
            best = t;
            segments = s;
        }
    }
    return segments;
}

size_t kv_attention_workspace(const KvAttnLaunch& a)
{
    if (a.segments <= 1) return 0;
    return static_cast<size_t>(a.b.num_tokens) * a.num_q_heads * a.segments * (a.b.head_dim + 2) * sizeof(float);
}

int launch_kv_attention(const KvAttnLaunch& a, cudaStream_t stream, char* msg, size_t msg_len)
{
    msg[0] = '\0';
    const bool q = a.b.type == kCacheE4M3;
    cudaError_t e = cudaErrorInvalidValue;
    switch (a.b.head_dim) {
    case 64: e = q ? launch_hd<true, 64>(a, stream, msg, msg_len) : launch_hd<false, 64>(a, stream, msg, msg_len); break;
    case 128: e = q ? launch_hd<true, 128>(a, stream, msg, msg_len) : launch_hd<false, 128>(a, stream, msg, msg_len); break;
    case 256: e = q ? launch_hd<true, 256>(a, stream, msg, msg_len) : launch_hd<false, 256>(a, stream, msg, msg_len); break;
    default: break;
    }
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        if (msg[0] == '\0') snprintf(msg, msg_len, "cache attention launch failed: %s", cudaGetErrorString(e));
        return 1;
    }
    return 0;
}

}  // namespace bsk
