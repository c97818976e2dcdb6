// linear_tcgen05.cuh -- the products of the feed-forward layer calls on the
// tcgen05 tensor cores: linear layer with bias, activation and residual, gated
// pair of linear layers, and the gradients' products (linear_internal.h has the
// formulas).  Instantiated per 16-bit type in linear_bf16.cu and linear_f16.cu.
//
// A tile is 128 rows by bn accumulator columns on one CTA, or 256 rows by bn on
// a CTA pair (two SMs, each staging half of A's rows and half of B's columns).
// The result's rows are the MMA's rows (TMEM lanes), its columns, contiguous in
// memory, the registers of a lane: a lane writes whole 32-byte sectors, reads its
// part of a residual likewise, and two neighbouring outputs are rounded by one
// packed conversion.
//
// Gated: the tile's B is bn/2 rows of Wg above bn/2 rows of Wu, so one MMA gives
// g in the accumulator's first half and u in its second, at the cost of a plain
// product of the same width; the epilogue reads both and stores act(g) * u.
// Neither g nor u goes through memory unless they are kept for a backward pass.
//
// Gradients: dx (rows are tokens, k are features) and dW (rows are features, k are
// tokens) are tiles of one launch, the longer k loops first, so that neither waits
// for the other's last wave.  Both read dz where it is, along k or along rows.  dx
// of a gated layer (dg Wg + du Wu) is one k loop over both sources and rounded once.
// The epilogue warps, idle until the first accumulator, add up the bias gradients'
// partial sums.
//
// Roles (320 threads): warp 0 loads by TMA into a ring of k slices, warp 1 issues
// the MMAs, warps 2..9 are the epilogue, overlapped with the next tile's loop by a
// second accumulator.  Tile sizes are run-time values (TMA boxes, instruction
// descriptor, ring depth): with few rows only those are staged -- the MMA reads
// on into whatever follows in shared memory, and those rows are not stored.
//
// Split k (one-CTA tiles, few tiles): the CTAs of a cluster share a tile's k
// loop; each stores its FP32 sums into the shared memory of the CTAs that finish the
// columns, which add them up in rank order (the result does not depend on timing).
//
// Bound and figures (GB300, back to back): few rows, the weights from HBM (gated
// 17408 x 5120, 1 token: 55.4 us, 6.4 TB/s); many, the power limit (gated 4096 x 17408 x 5120:
// 838 us, 1740 TFLOP/s) and in short bursts the MMAs (709 us, 2060 TFLOP/s); between, the latency
// of a k loop's operands from L2 (95 GB/s an SM) and of the launch (4 us).
#pragma once

#include <cstdio>
#include <type_traits>

#include "bsk_internal.h"
#include "linear_math.cuh"
#include "ptx.cuh"

namespace bsk {
namespace {

constexpr int kLinEpiWarps = 8;                  // two per quarter of the TMEM lanes: every other kCh columns
constexpr int kLinThreads = 64 + 32 * kLinEpiWarps;
constexpr int kLinBK = 64;                       // k values per stage: one 128-byte swizzle row
constexpr int kLinMaxStages = 24;
constexpr int kCh = 16;                          // columns per epilogue step: 32 bytes of 16-bit values
constexpr int kBlockBytes = 128;                 // a row of a warp's staging buffer: one line of memory
static_assert(kLinStageBytes == kLinEpiWarps * 32 * kBlockBytes, "staging buffers");
// Gradients: k-blocks summed in an accumulator before they are added to FP32 registers.  A
// tensor-core accumulation cuts each of its sums (toward zero), so an error grows with their number: FP32 dW
// over 8192 tokens came out 2e-5 off, in segments of 768 tokens 7e-7, as much as FP32 arithmetic gives.  Results
// of 16 bits take longer segments: with operands of one sign the error is 2.5e-5 of the sum for 4096 terms, a
// twentieth of FP16's half step, and in one accumulation passed it (400,003 tokens: 2.5e-3).  That costs
// nothing: segments of 64, 128, 256 k-blocks and none took 290 us each for the gradients of 32768 x 2048 x 2048,
// 432, 434, 440 and 436 for the gated ones of 16384 x 4096 x 1024.
constexpr int kSegmentKb32 = 12;
constexpr int kSegmentKb16 = 64;

enum LinearWaitSite {
    kSiteLinEmpty = 0x30,
    kSiteLinFull = 0x31,
    kSiteLinTmemEmpty = 0x32,
    kSiteLinTmemFull = 0x33,
    kSiteLinDrain = 0x34,
};

// A product of a launch: `tiles` tiles of one result.
struct LinearJob {
    int rows, cols;           // of the result (weight gradient: of each source's)
    int kbs, k_sources;       // k-blocks per source, sources one after the other along k
    int num_m, num_m1;        // tile rows in all, of the first source (weight gradient)
    int num_n, num_tiles;
    int a_mn;                 // A read along its rows (weight gradient)
    int seg_kb;               // k-blocks per segment (a multiple of a turn's, or all)
    uint32_t idesc;
    void* out[2];
    long long ldo;
    int out_f32, accumulate, vec_out;
};

struct LinearParams {
    LinearJob job[2];         // [1]: gradients only, may have no tiles
    int extra;                // gradients: see tile_of()
    int wide_z, wide_w, wide_x;   // operands read along rows or columns: all 64-element blocks by one load
    int group_m;
    int a_rows;               // rows of A staged per CTA (128, or the few there are)
    int bn;                   // accumulator columns per tile
    int wcols;                // result columns per tile: bn, gated bn / 2
    int stages;               // ring depth, in groups of `group` k-blocks
    int group;                // k-blocks per wait of the MMA warp
    int a_bytes, b_bytes;     // of a k-block
    int ring_bytes;           // the stages (and staging buffers), before the barriers
    int stage_at;             // results go through staging buffers here; -1: row by row
    int acc_cols, tmem_cols;  // TMEM columns of an accumulator, in all
    int split;                // CTAs that share a tile's k loop (a cluster); 1: none
    int prefetch_kb;          // k-blocks of the first tile's weights brought into L2 ahead
    const uint8_t* w_rows[2];
    long long w_ld_bytes;
    const uint16_t* bias[2];
    const uint16_t* residual;
    long long ldr;
    uint16_t* keep[2];
    long long ldk;
    int act;
    int vec_res, vec_keep, vec_bias;   // 16-byte accesses allowed
    const float* db_partial;
    int db_chunks, db_parts, db_M, db_f32, db_accumulate;
    void* db[2];
    int* status;
    unsigned long long wait_limit_ns;
};

// Tensor maps.  Forward: x, W (Wg), Wu.  Gradients: dz_0, dz_1, W_0, W_1, x, read along rows or
// columns, then dz_0, dz_1 read along k.
struct LinearMaps {
    CUtensorMap m[7];
};

// The i-th tile of this CTA (or pair) in `pass`; false when there is none.
// Without split k there is one pass: tiles go to the `units` CTAs (pairs) in turn, job
// 0 first.  With it, pass 0 is job 0, a tile per cluster (unit / split), and pass 1 job 1, a tile per
// CTA.  Units that got one tile of job 0 fewer than the others take p.extra tiles of job 1
// before all units go on with the rest.
template <bool SPLIT>
__device__ __forceinline__ bool tile_of(const LinearParams& p, int pass, int unit, int units, int i, int* job, int* tile)
{
    const int t0 = p.job[0].num_tiles;
    int h;   // units up to here have one tile of job 0 more than the others (0: all the same)
    if constexpr (SPLIT) {
        if (pass == 0) {
            *job = 0;
            *tile = unit / p.split;
            return i == 0 && *tile < t0;
        }
        h = t0 * p.split;
    } else {
        const int rounds = t0 / units;
        h = t0 - rounds * units;
        const int mine = rounds + (unit < h ? 1 : 0);
        if (i < mine) {
            *job = 0;
            *tile = unit + i * units;
            return true;
        }
        i -= mine;
    }
    const int late = units - h;
    const int extra = h != 0 ? p.extra : 0;
    *job = 1;
    if (unit >= h && i < extra) {
        *tile = i * late + (unit - h);
    } else {
        if (unit >= h) i -= extra;
        *tile = extra * late + i * units + unit;
    }
    return *tile < p.job[1].num_tiles;
}

__device__ __forceinline__ bool lin_elect()
{
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

__device__ __forceinline__ void lin_tmem_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// A hint, as prefetch_l2().
__device__ __forceinline__ void prefetch_l1(const void* addr)
{
    asm volatile("prefetch.global.L1 [%0];" ::"l"(addr) : "memory");
}

template <int CH>
__device__ __forceinline__ void lin_tmem_ld(uint32_t taddr, uint32_t (&r)[CH])
{
    static_assert(CH == 16 || CH == 32, "16 or 32 columns");
    if constexpr (CH == 16) lin_tmem_ld16(taddr, r);
    else tmem_ld_32x32b_x32(taddr, r);
}

// Whole warp: the wait's answer, the same for all lanes.  Looks at the clock and the
// abort flag only after many tries (each suspends the warp for a while by itself).
__device__ __forceinline__ bool lin_wait(uint32_t bar, uint32_t parity, const WaitCtl& w, int site)
{
    for (int i = 0; i < 256; ++i)
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, w, site));
}
__device__ __forceinline__ bool lin_wait_cluster(uint32_t bar, uint32_t parity, const WaitCtl& w, int site)
{
    for (int i = 0; i < 256; ++i)
        if (__all_sync(0xffffffffu, mbar_try_wait_cluster(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, w, site));
}

// Arrive on an mbarrier of the cluster without ordering this thread's earlier writes: the
// accumulator that it hands back has been read (tcgen05.wait::ld).  A release at cluster scope would
// wait for the results' stores to memory, every tile (6992 x 8512 x 320 on pairs: 57 us).
__device__ __forceinline__ void mbar_arrive_remote_relaxed(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// A 3-D box, {64 elements, 64 rows, blocks}, from row y of block z on.
template <bool PAIR>
__device__ __forceinline__ void tma_load_blocks(uint32_t dst, const CUtensorMap* map, uint32_t bar, int y, int z)
{
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(y), "r"(z)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(y), "r"(z)
            : "memory");
}

// 16-byte store to the shared memory of a CTA of the cluster (address from mapa_shared).
__device__ __forceinline__ void st_shared_cluster_v4(uint32_t cluster_addr, float a, float b, float c, float d)
{
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "f"(a), "f"(b), "f"(c), "f"(d)
                 : "memory");
}

// ---------------------------------------------------------------------------
// Epilogue, row by row: each lane reads and writes its own row's CH columns, n of them there.
// For few rows, and for the parts of split k.
// ---------------------------------------------------------------------------
template <int TYPE, int CH>
__device__ __forceinline__ void load_row(float (&v)[CH], const uint16_t* p, int n, bool vec)
{
    if (vec && n == CH) {
#pragma unroll
        for (int i = 0; i < CH; i += 8) {
            const uint4 w = *reinterpret_cast<const uint4*>(p + i);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 f = unpack2<TYPE>(u[k]);
                v[i + 2 * k] = f.x;
                v[i + 2 * k + 1] = f.y;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < CH; ++i) v[i] = i < n ? to_f32<TYPE>(p[i]) : 0.f;
    }
}

template <int TYPE, int CH>
__device__ __forceinline__ void store_row16(uint16_t* p, const float (&v)[CH], int n, bool vec)
{
    uint32_t w[CH / 2];
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) w[i] = pack2<TYPE>(v[2 * i], v[2 * i + 1]);
    if (vec && n == CH) {
#pragma unroll
        for (int i = 0; i < CH / 8; ++i)
            reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (i < n) p[i] = static_cast<uint16_t>(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
    }
}

template <int CH>
__device__ __forceinline__ void store_row32(float* p, const float (&v)[CH], int n, bool vec, bool accumulate)
{
    if (vec && n == CH) {
#pragma unroll
        for (int i = 0; i < CH; i += 4) {
            float4 t = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            if (accumulate) {
                const float4 w = *reinterpret_cast<const float4*>(p + i);
                t = make_float4(t.x + w.x, t.y + w.y, t.z + w.z, t.w + w.w);
            }
            *reinterpret_cast<float4*>(p + i) = t;
        }
    } else {
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (i < n) p[i] = accumulate ? p[i] + v[i] : v[i];
    }
}

template <int CH>
__device__ __forceinline__ void act_switch(float (&v)[CH], int act)
{
    if (act == kActSilu) act_values<kActSilu, false, CH>(v, v);
    else if (act == kActGeluTanh) act_values<kActGeluTanh, false, CH>(v, v);
    else if (act == kActGelu) act_values<kActGelu, false, CH>(v, v);
    else if (act == kActRelu) act_values<kActRelu, false, CH>(v, v);
}

// v += bias[c0 ..], if there is one.
template <int TYPE, int CH>
__device__ __forceinline__ void add_bias_row(float (&v)[CH], const uint16_t* bias, int c0, int n, bool vec)
{
    if (bias == nullptr) return;
    float t[CH];
    load_row<TYPE, CH>(t, bias + c0, n, vec);
#pragma unroll
    for (int i = 0; i < CH; ++i) v[i] += t[i];
}

// a (and b, gated: u) hold the sums of `row`, columns c0 .. c0 + n - 1 of source `src`.
template <int TYPE, int MODE, int CH>
__device__ __forceinline__ void finish_row(const LinearParams& p, const LinearJob& job, float (&a)[CH], float (&b)[CH],
                                           int src, long long row, int c0, int n)
{
    if constexpr (MODE == kModeLinear || MODE == kModeGated) {
        add_bias_row<TYPE, CH>(a, p.bias[0], c0, n, p.vec_bias);
        if (MODE == kModeGated) add_bias_row<TYPE, CH>(b, p.bias[1], c0, n, p.vec_bias);
        if (p.keep[0] != nullptr) {
            store_row16<TYPE, CH>(p.keep[0] + row * p.ldk + c0, a, n, p.vec_keep);
            if (MODE == kModeGated) store_row16<TYPE, CH>(p.keep[1] + row * p.ldk + c0, b, n, p.vec_keep);
        }
        act_switch<CH>(a, p.act);
        if constexpr (MODE == kModeGated) {
#pragma unroll
            for (int i = 0; i < CH; ++i) a[i] *= b[i];
        }
        if (MODE == kModeLinear && p.residual != nullptr) {
            float t[CH];
            load_row<TYPE, CH>(t, p.residual + row * p.ldr + c0, n, p.vec_res);
#pragma unroll
            for (int i = 0; i < CH; ++i) a[i] += t[i];
        }
        store_row16<TYPE, CH>(static_cast<uint16_t*>(job.out[0]) + row * job.ldo + c0, a, n, job.vec_out);
    } else if (job.out_f32) {
        store_row32<CH>(static_cast<float*>(job.out[src]) + row * job.ldo + c0, a, n, job.vec_out, job.accumulate != 0);
    } else {
        uint16_t* o = static_cast<uint16_t*>(job.out[src]) + row * job.ldo + c0;
        if (job.accumulate) {
            float t[CH];
            load_row<TYPE, CH>(t, o, n, job.vec_out);
#pragma unroll
            for (int i = 0; i < CH; ++i) a[i] += t[i];
        }
        store_row16<TYPE, CH>(o, a, n, job.vec_out);
    }
}

// ---------------------------------------------------------------------------
// Epilogue through shared memory: a warp gathers a block of 32 rows by up to 128 bytes
// (64 columns of 16 bits, 32 of FP32) in its staging buffer and moves it in whole lines, neighbouring
// lanes on neighbouring addresses whatever the rows' alignment.  With every lane storing its own
// row's 32 bytes, outputs went out at 11 GB/s an SM (6992 x 8512 x 320: 69 us).
// Piece q (16 bytes) of row r lies at r * 128 + (q ^ (r & 7)) * 16: no bank conflicts either way.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint4* block_piece(uint8_t* buf, int row, int piece)
{
    return reinterpret_cast<uint4*>(buf + row * kBlockBytes + ((piece ^ (row & 7)) << 4));
}
template <typename E>
__device__ __forceinline__ E* block_element(uint8_t* buf, int row, int col)
{
    const int byte = col * static_cast<int>(sizeof(E));
    return reinterpret_cast<E*>(buf + row * kBlockBytes + (((byte >> 4) ^ (row & 7)) << 4) + (byte & 15));
}

// Element by element, all of a turn's reads before its writes (the compiler cannot tell that
// they do not touch).
template <typename E, bool LOAD, int ROWS>
__device__ __forceinline__ void block_move_elements(uint8_t* buf, E* g, long long ld, int rows, int n)
{
    constexpr int kRows = ROWS;
    constexpr int kCols = kBlockBytes / static_cast<int>(sizeof(E)) / 32;   // of a lane: 2 of 16 bits, 1 of FP32
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += kRows) {
        E v[kRows][kCols];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
            for (int h = 0; h < kCols; ++h) {
                const int c = 32 * h + lane;
                if constexpr (LOAD) {
                    if (r0 + i < rows && c < n) v[i][h] = g[(r0 + i) * ld + c];
                } else {
                    v[i][h] = *block_element<E>(buf, r0 + i, c);
                }
            }
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
            for (int h = 0; h < kCols; ++h) {
                const int c = 32 * h + lane;
                if (r0 + i < rows && c < n) {
                    if constexpr (LOAD) *block_element<E>(buf, r0 + i, c) = v[i][h];
                    else g[(r0 + i) * ld + c] = v[i][h];
                }
            }
    }
}

// The same, not inlined: in the linear kernels its registers and code slow the common path down, by
// more than unaligned rows gain (inlined / called, us: 6992 x 8512 x 320 with SiLU 78 / 72, 777 x 1031 x 4099 with
// kept z 21.8 / 22.2, 333 x 2731 x 1024 13.1 / 13.6); in the gated ones they do not (6992 x 4256 x 320 63.5 / 64.3,
// 333 x 2731 x 1024 with kept g and u 12.5 / 14.6, 2000 x 2731 x 1024 23.0 / 25.0).
template <typename E, bool LOAD>
__device__ __noinline__ void block_move_elements_call(uint8_t* buf, E* g, long long ld, int rows, int n)
{
    block_move_elements<E, LOAD, 8>(buf, g, ld, rows, n);
}

// Whole warp: rows [0, rows) x n elements between the buffer and memory (first element at `g`, rows ld
// elements apart).
// (FLIGHT: 16-byte accesses of a lane in flight; 2: few, beside a tile in registers.  There unaligned
// rows are stored by eight all the same, and loaded, when all of the tile is still in registers, one by
// one.  ANY: not all is whole aligned 16-byte units.)
template <typename E, bool LOAD, int FLIGHT, bool INLINE, bool ANY = true>
__device__ __forceinline__ void block_move(uint8_t* buf, E* g, long long ld, int rows, int n, bool vec)
{
    constexpr int kPer = 16 / static_cast<int>(sizeof(E));
    const int lane = threadIdx.x & 31;
    if (vec && n == 8 * kPer) {
        const int piece = lane & 7;
#pragma unroll FLIGHT
        for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3);
            uint4* at = reinterpret_cast<uint4*>(g + r * ld + piece * kPer);
            if (r < rows) {
                if constexpr (LOAD) *block_piece(buf, r, piece) = *at;
                else *at = *block_piece(buf, r, piece);
            }
        }
    } else if (vec && n % kPer == 0) {
        const int pieces = n / kPer;
        for (int e = lane; e < rows * pieces; e += 32) {
            const int r = e / pieces, piece = e - r * pieces;
            uint4* at = reinterpret_cast<uint4*>(g + r * ld + piece * kPer);
            if constexpr (LOAD) *block_piece(buf, r, piece) = *at;
            else *at = *block_piece(buf, r, piece);
        }
    } else if constexpr (FLIGHT == 8) {
        if constexpr (INLINE) block_move_elements<E, LOAD, 8>(buf, g, ld, rows, n);
        else block_move_elements_call<E, LOAD>(buf, g, ld, rows, n);
    } else if constexpr (ANY) {
        block_move_elements<E, LOAD, LOAD ? 1 : 8>(buf, g, ld, rows, n);
    }
    __syncwarp();
}

// This lane's row, CH columns of 16 bits from piece `first`: read, or rounded and written.
template <int TYPE, int CH>
__device__ __forceinline__ void block_get16(float (&v)[CH], uint8_t* buf, int row, int first)
{
#pragma unroll
    for (int i = 0; i < CH / 8; ++i) {
        const uint4 w = *block_piece(buf, row, first + i);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = unpack2<TYPE>(u[k]);
            v[8 * i + 2 * k] = f.x;
            v[8 * i + 2 * k + 1] = f.y;
        }
    }
}
template <int TYPE, int CH>
__device__ __forceinline__ void block_put16(uint8_t* buf, int row, int first, const float (&v)[CH])
{
#pragma unroll
    for (int i = 0; i < CH / 8; ++i)
        *block_piece(buf, row, first + i) =
            make_uint4(pack2<TYPE>(v[8 * i], v[8 * i + 1]), pack2<TYPE>(v[8 * i + 2], v[8 * i + 3]),
                       pack2<TYPE>(v[8 * i + 4], v[8 * i + 5]), pack2<TYPE>(v[8 * i + 6], v[8 * i + 7]));
}

// Forward, one block: up to 64 columns c0 .. of 32 rows from `row0` (the first `rows` of them there); the
// accumulator's columns at `t_col` (gated: u's at t_col + u_cols).  32 columns at a time: what a
// step waits for (TMEM, the special functions, shared memory) is then shared by 32.
template <int TYPE, int MODE>
__device__ __forceinline__ void finish_block(const LinearParams& p, const LinearJob& job, uint8_t* buf, uint32_t t_col,
                                             uint32_t u_cols, long long row0, int rows, int c0, int n)
{
    constexpr bool kGated = MODE == kModeGated;
    constexpr int CH = 32;
    const int lane = threadIdx.x & 31;
    if (p.keep[0] != nullptr) {
        // the kept pre-activations first
#pragma unroll 1
        for (int o = 0; o < (kGated ? 2 : 1); ++o) {
#pragma unroll 1
            for (int c = 0; c < n; c += CH) {
                const int left = n - c < CH ? n - c : CH;
                uint32_t ra[CH];
                lin_tmem_ld<CH>(t_col + o * u_cols + c, ra);
                tmem_ld_wait();
                float a[CH];
#pragma unroll
                for (int i = 0; i < CH; ++i) a[i] = __uint_as_float(ra[i]);
                add_bias_row<TYPE, CH>(a, p.bias[o], c0 + c, left, p.vec_bias);
                block_put16<TYPE, CH>(buf, lane, c / 8, a);
            }
            __syncwarp();
            block_move<uint16_t, false, 8, kGated>(buf, p.keep[o] + row0 * p.ldk + c0, p.ldk, rows, n, p.vec_keep);
        }
    }
    if (MODE == kModeLinear && p.residual != nullptr)
        block_move<uint16_t, true, 8, kGated>(buf, const_cast<uint16_t*>(p.residual) + row0 * p.ldr + c0, p.ldr, rows, n, p.vec_res);
#pragma unroll 1
    for (int c = 0; c < n; c += CH) {
        const int left = n - c < CH ? n - c : CH;
        uint32_t ra[CH], rb[CH];
        lin_tmem_ld<CH>(t_col + c, ra);
        if constexpr (kGated) lin_tmem_ld<CH>(t_col + u_cols + c, rb);
        tmem_ld_wait();
        float a[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) a[i] = __uint_as_float(ra[i]);
        add_bias_row<TYPE, CH>(a, p.bias[0], c0 + c, left, p.vec_bias);
        act_switch<CH>(a, p.act);
        if constexpr (kGated) {
            float b[CH];
#pragma unroll
            for (int i = 0; i < CH; ++i) b[i] = __uint_as_float(rb[i]);
            add_bias_row<TYPE, CH>(b, p.bias[1], c0 + c, left, p.vec_bias);
#pragma unroll
            for (int i = 0; i < CH; ++i) a[i] *= b[i];
        } else if (p.residual != nullptr) {
            float t[CH];
            block_get16<TYPE, CH>(t, buf, lane, c / 8);
#pragma unroll
            for (int i = 0; i < CH; ++i) a[i] += t[i];
        }
        block_put16<TYPE, CH>(buf, lane, c / 8, a);
    }
    __syncwarp();
    block_move<uint16_t, false, 8, kGated>(buf, static_cast<uint16_t*>(job.out[0]) + row0 * job.ldo + c0, job.ldo, rows, n, job.vec_out);
}

// Gradients: a warp's columns of a tile, 16 * i from c0 in sum[i], n of them there.
template <int TYPE, bool ANY>
__device__ __forceinline__ void finish_sums(const LinearJob& job, uint8_t* buf, float (&sum)[8][kCh], int src, long long row0,
                                            int rows, int c0, int n)
{
    const int lane = threadIdx.x & 31;
    const bool acc = job.accumulate != 0;
    if (job.out_f32) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {   // blocks of 32 columns
            const int left = n - 32 * g < 32 ? n - 32 * g : 32;
            if (left > 0) {
                float* o = static_cast<float*>(job.out[src]) + row0 * job.ldo + c0 + 32 * g;
                if (acc) block_move<float, true, 2, true, ANY>(buf, o, job.ldo, rows, left, job.vec_out);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    float4 v = make_float4(sum[2 * g + q / 4][q % 4 * 4], sum[2 * g + q / 4][q % 4 * 4 + 1],
                                           sum[2 * g + q / 4][q % 4 * 4 + 2], sum[2 * g + q / 4][q % 4 * 4 + 3]);
                    float4* at = reinterpret_cast<float4*>(block_piece(buf, lane, q));
                    if (acc) {
                        const float4 w = *at;
                        v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
                    }
                    *at = v;
                }
                __syncwarp();
                block_move<float, false, 2, true, ANY>(buf, o, job.ldo, rows, left, job.vec_out);
            }
        }
    } else {
#pragma unroll
        for (int g = 0; g < 2; ++g) {   // blocks of 64 columns
            const int left = n - 64 * g < 64 ? n - 64 * g : 64;
            if (left > 0) {
                uint16_t* o = static_cast<uint16_t*>(job.out[src]) + row0 * job.ldo + c0 + 64 * g;
                if (acc) block_move<uint16_t, true, 2, true, ANY>(buf, o, job.ldo, rows, left, job.vec_out);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (acc) {
                        float t[kCh];
                        block_get16<TYPE, kCh>(t, buf, lane, 2 * q);
#pragma unroll
                        for (int i = 0; i < kCh; ++i) sum[4 * g + q][i] += t[i];
                    }
                    block_put16<TYPE, kCh>(buf, lane, 2 * q, sum[4 * g + q]);
                }
                __syncwarp();
                block_move<uint16_t, false, 2, true, ANY>(buf, o, job.ldo, rows, left, job.vec_out);
            }
        }
    }
}

// The bias gradients: their partial sums added up, by the epilogue warps of all CTAs:
// 32 columns a CTA and turn, every eighth chunk a warp, the warps' sums in order.
template <int TYPE>
__device__ __forceinline__ void sum_bias_grads(const LinearParams& p, float* sums)
{
    const int w = static_cast<int>(threadIdx.x >> 5) - 2, lane = threadIdx.x & 31;
    const long long total = static_cast<long long>(p.db_parts) * p.db_M;
    for (long long e0 = static_cast<long long>(blockIdx.x) * 32; e0 < total; e0 += static_cast<long long>(gridDim.x) * 32) {
        const long long e = e0 + lane;
        float v = 0.f;
        if (e < total) {
#pragma unroll 8
            for (int i = w; i < p.db_chunks; i += kLinEpiWarps) v += p.db_partial[i * total + e];
        }
        sums[w * 32 + lane] = v;
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kLinEpiWarps) : "memory");
        if (w == 0 && e < total) {
            v = 0.f;
#pragma unroll
            for (int i = 0; i < kLinEpiWarps; ++i) v += sums[i * 32 + lane];
            const int q = e >= p.db_M ? 1 : 0;
            const long long c = e - static_cast<long long>(q) * p.db_M;
            if (p.db[q] != nullptr) {
                if (p.db_f32) {
                    float* o = static_cast<float*>(p.db[q]) + c;
                    *o = p.db_accumulate ? *o + v : v;
                } else {
                    uint16_t* o = static_cast<uint16_t*>(p.db[q]) + c;
                    *o = to_16<TYPE>(p.db_accumulate ? to_f32<TYPE>(*o) + v : v);
                }
            }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kLinEpiWarps) : "memory");
    }
}

// A tile of split k: its place, and the layout of its partial sums in the shared memory of
// the CTA that finishes `slice` of its columns: [CTA][part][slice / 4][row][4 columns], so that the
// 32 rows of a warp's 16-byte stores to another SM lie side by side.
struct SplitTile {
    int job, src, row0, col0;
    int rows, width, slice;
};
__host__ __device__ __forceinline__ int split_slice(int width, int split)
{
    return ((width + split - 1) / split + 7) / 8 * 8;   // 16-byte accesses of results stay aligned
}
template <bool GRAD>
__device__ __forceinline__ SplitTile split_tile(const LinearParams& p, int j, int tile)
{
    const LinearJob& job = p.job[GRAD ? j : 0];
    SplitTile t;
    int pm, pn;
    tile_coord(tile, job.num_m, job.num_n, p.group_m, &pm, &pn);
    t.job = j;
    t.src = GRAD && pm >= job.num_m1 ? 1 : 0;
    t.row0 = (pm - t.src * job.num_m1) * 128;
    t.col0 = pn * p.wcols;
    t.rows = job.rows - t.row0 < 128 ? job.rows - t.row0 : 128;
    t.width = job.cols - t.col0 < p.wcols ? job.cols - t.col0 : p.wcols;
    t.slice = split_slice(t.width, p.split);
    return t;
}

// Kinds of kernel: results row by row (forward, few rows or one narrow tile per CTA), through shared
// memory, split k, CTA pairs.  With few rows two CTAs fit on an SM by registers and shared memory, so
// that the next launch's CTAs set up while this one's finish; split k of a forward pass likewise.
// ANY, gradients: results of any alignment and width.  Without them the code for unaligned rows costs no
// registers (spill stores of 36 to 48 bytes on one CTA and pairs, with it 204 to 268; split k 220 and 356; gated
// backward 4096 x 17408 x 5120 1% faster), with it they are stored by eight rows (linear backward
// 187 x 7695 x 2339 64 us, row by row 86).  Forward kernels spill nothing.
enum LinearKind : int { kKindDirect = 0, kKindOne = 1, kKindSplit = 2, kKindPair = 3 };

template <int TYPE, int MODE, int KIND, bool ANY>
__global__ void __launch_bounds__(kLinThreads, KIND == kKindDirect || (KIND == kKindSplit && MODE != kModeGrad) ? 2 : 1)
    linear_kernel(const __grid_constant__ LinearMaps maps, const __grid_constant__ LinearParams p)
{
    constexpr bool kGated = MODE == kModeGated;
    constexpr bool kGrad = MODE == kModeGrad;
    constexpr bool PAIR = KIND == kKindPair;
    constexpr bool SPLIT = KIND == kKindSplit;
    constexpr int kTileRows = PAIR ? 256 : 128;
    const int S = p.stages;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t sA = smem_u32(smem);
    const uint32_t sB = sA + static_cast<uint32_t>(S * p.group * p.a_bytes);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.ring_bytes);
    const uint32_t full0 = smem_u32(bars);                 // kLinMaxStages each: stage loaded, consumed
    const uint32_t empty0 = full0 + 8 * kLinMaxStages;
    const uint32_t tfull0 = empty0 + 8 * kLinMaxStages;    // 2 each: accumulator ready, drained
    const uint32_t tempty0 = tfull0 + 16;
    const uint32_t drain_bar = tempty0 + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kLinMaxStages + 5);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    static_assert((2 * kLinMaxStages + 5) * 8 + 8 <= 512, "barrier area too small");

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = PAIR || SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
    const bool leader = !PAIR || rank == 0;   // issues the MMAs
    const int unit = static_cast<int>(blockIdx.x) / (PAIR ? 2 : 1);
    const int units = static_cast<int>(gridDim.x) / (PAIR ? 2 : 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull0 + 8 * a, 1);
            mbar_init(tempty0 + 8 * a, PAIR ? 2 * kLinEpiWarps : kLinEpiWarps);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0u;
        fence_mbar_init();
        prefetch_tmap(&maps.m[0]);
        prefetch_tmap(&maps.m[1]);
        if (kGated || kGrad) prefetch_tmap(&maps.m[2]);
    }
    __syncwarp();
    if (warp == 1) {
        if constexpr (PAIR) {
            tmem_alloc_pair(smem_u32(tmem_slot), static_cast<uint32_t>(p.tmem_cols));
            tmem_relinquish_alloc_permit_pair();
        } else {
            tmem_alloc(smem_u32(tmem_slot), static_cast<uint32_t>(p.tmem_cols));
            tmem_relinquish_alloc_permit();
        }
    }
    tc_fence_before_sync();
    if constexpr (PAIR) cluster_sync();
    else __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    if constexpr (!kGrad && (KIND == kKindDirect || SPLIT)) {
        // The epilogue warps bring the first weights into L2 while the kernel before
        // this one may still run (a prefetch is coherent and delivers nothing).
        if (warp >= 2 && p.prefetch_kb > 0) {
            int job, tile, pm, pn;
            if (tile_of<SPLIT>(p, 0, unit, units, 0, &job, &tile)) {
                tile_coord(tile, p.job[0].num_m, p.job[0].num_n, p.group_m, &pm, &pn);
                const int kb_all = p.job[0].kbs;
                const int kb0 = static_cast<int>(static_cast<long long>(rank) * kb_all / p.split);
                int lines = static_cast<int>(static_cast<long long>(rank + 1) * kb_all / p.split) - kb0;
                if (lines > p.prefetch_kb) lines = p.prefetch_kb;
                for (int r = static_cast<int>(threadIdx.x) - 64; r < p.bn; r += 32 * kLinEpiWarps) {
                    const int half = kGated && r >= p.wcols ? 1 : 0;
                    const int col = pn * p.wcols + r - half * p.wcols;
                    if (col >= p.job[0].cols) continue;
                    const uint8_t* w = p.w_rows[half] + col * p.w_ld_bytes + static_cast<long long>(kb0) * 128;
                    for (int i = 0; i < lines; ++i) prefetch_l2(w + i * 128);
                }
            }
        }
    }
    // global memory is read and written only once the kernel before this one in the stream has completed
    // (all CTAs of this launch have their TMEM by the time the next launch's may start)
    griddep_launch_dependents();
    griddep_wait();
    const WaitCtl wc{abort_flag, p.status, p.wait_limit_ns};
    uint32_t never = 0u;
    const WaitCtl wc_drain{&never, p.status, p.wait_limit_ns};
    // Each warp's place in the rings of stages and accumulators, over all tiles and passes.
    int stage = 0, it = 0;
    uint32_t phase = 0;
    long long issued = 0;
    bool ok = true;
    if constexpr (kGrad) {
        if (warp >= 2 && p.db_partial != nullptr) sum_bias_grads<TYPE>(p, reinterpret_cast<float*>(smem + p.ring_bytes + 512));
        __syncwarp();
    }
    // One pass over this CTA's tiles.  PARTIAL (pass 0 of split k): its share of a tile's k-blocks,
    // the sums left in shared memory.
    auto run = [&](auto partial_tag, const int pass) {
        constexpr bool PARTIAL = decltype(partial_tag)::value;
        // k-blocks [begin, end) of a tile of `job`
        auto k_range = [&](const LinearJob& job, int* begin, int* end) {
            const int all = job.kbs * job.k_sources;
            *begin = PARTIAL ? static_cast<int>(static_cast<long long>(rank) * all / p.split) : 0;
            *end = PARTIAL ? static_cast<int>(static_cast<long long>(rank + 1) * all / p.split) : all;
        };
        if (warp == 0) {
            // ------------------------------------------------------------------
            // loads: this CTA's rows of A and of B
            // ------------------------------------------------------------------
            const uint32_t lead_full0 = PAIR ? mapa_shared(full0, 0) : full0;
            auto load = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
                if constexpr (PAIR) tma_load_2d_pair(dst, map, bar, x, y);
                else tma_load_2d(dst, map, bar, x, y);
            };
            // 64 k rows of `blocks` 64-element blocks from element x on
            auto load_blocks = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int k0, int blocks, bool wide) {
                if (wide) {
                    tma_load_blocks<PAIR>(dst, map, bar, k0, x / 64);
                } else {
                    for (int b = 0; b < blocks; ++b) load(dst + static_cast<uint32_t>(b) * 8192u, map, bar, x + 64 * b, k0);
                }
            };
            const int b_rows = PAIR ? p.bn / 2 : p.bn;   // rows of B (columns of the tile) staged by this CTA
            const uint32_t tx = static_cast<uint32_t>(p.a_bytes + p.b_bytes) * (PAIR ? 2u : 1u);
            int j, tile;
            for (int i = 0; ok && tile_of<SPLIT>(p, pass, unit, units, i, &j, &tile); ++i) {
                const LinearJob& job = p.job[kGrad ? j : 0];
                int pm, pn, kb_begin, kb_end;
                tile_coord(tile, job.num_m, job.num_n, p.group_m, &pm, &pn);
                k_range(job, &kb_begin, &kb_end);
                const int row_src = kGrad && pm >= job.num_m1 ? 1 : 0;
                const int m0 = (pm - row_src * job.num_m1) * kTileRows + (PAIR ? rank * 128 : 0);
                const int n0 = pn * p.wcols;
                for (int kb0 = kb_begin; kb0 < kb_end; kb0 += p.group) {
                    const int count = kb_end - kb0 < p.group ? kb_end - kb0 : p.group;
                    ok = lin_wait(empty0 + 8 * stage, phase ^ 1u, wc, kSiteLinEmpty);
                    if (!ok) break;
                    if (lin_elect()) {
                        if (leader) mbar_arrive_expect_tx(full0 + 8 * stage, tx * static_cast<uint32_t>(count));
                        const uint32_t bar = lead_full0 + 8 * stage;
                        uint32_t a_dst = sA + static_cast<uint32_t>(stage * p.group * p.a_bytes);
                        uint32_t b_dst = sB + static_cast<uint32_t>(stage * p.group * p.b_bytes);
                        for (int kb = kb0; kb < kb0 + count; ++kb) {
                            if constexpr (kGrad) {
                                const int k_src = kb >= job.kbs ? 1 : 0;
                                const int k0 = (kb - k_src * job.kbs) * kLinBK;
                                const int nb = n0 + (PAIR ? rank * b_rows : 0);
                                if (job.a_mn) {
                                    load_blocks(a_dst, &maps.m[row_src], bar, m0, k0, 2, p.wide_z != 0);
                                    load_blocks(b_dst, &maps.m[4], bar, nb, k0, b_rows / 64, p.wide_x != 0);
                                } else {
                                    load(a_dst, &maps.m[5 + k_src], bar, k0, m0);
                                    load_blocks(b_dst, &maps.m[2 + k_src], bar, nb, k0, b_rows / 64, p.wide_w != 0);
                                }
                            } else {
                                const int k0 = kb * kLinBK;
                                load(a_dst, &maps.m[0], bar, k0, m0);
                                if constexpr (kGated) {
                                    if constexpr (PAIR) {
                                        load(b_dst, &maps.m[1 + rank], bar, k0, n0);
                                    } else {
                                        load(b_dst, &maps.m[1], bar, k0, n0);
                                        load(b_dst + static_cast<uint32_t>(p.b_bytes / 2), &maps.m[2], bar, k0, n0);
                                    }
                                } else {
                                    load(b_dst, &maps.m[1], bar, k0, n0 + (PAIR ? rank * b_rows : 0));
                                }
                            }
                            a_dst += static_cast<uint32_t>(p.a_bytes);
                            b_dst += static_cast<uint32_t>(p.b_bytes);
                        }
                    }
                    __syncwarp();
                    ++issued;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            __syncwarp();
            if constexpr (PARTIAL) cluster_sync();   // (the epilogue warps' one)
        } else if (warp == 1) {
            // ------------------------------------------------------------------
            // MMAs
            // ------------------------------------------------------------------
            if (leader) {
                int j, tile;
                for (int i = 0; ok && tile_of<SPLIT>(p, pass, unit, units, i, &j, &tile); ++i) {
                    const LinearJob& job = p.job[kGrad ? j : 0];
                    int kb_begin, kb_end;
                    k_range(job, &kb_begin, &kb_end);
                    const bool a_mn = kGrad && job.a_mn != 0;
                    const uint32_t idesc = job.idesc;
                    // Operand descriptors of the first stage; addresses count 16 bytes.  An MMA's 16 k
                    // values are 32 bytes of every 128-byte row of an operand read along k, and 16 rows of
                    // 128 bytes of one read along rows or columns (64-element blocks 8 KB apart).
                    const uint64_t desc_a = a_mn ? smem_desc_sw128(sA, 8192, 1024) : smem_desc_sw128(sA, 16, 1024);
                    const uint64_t desc_b = kGrad ? smem_desc_sw128(sB, 8192, 1024) : smem_desc_sw128(sB, 16, 1024);
                    const uint32_t step_a = a_mn ? 128u : 2u;
                    constexpr uint32_t kStepB = kGrad ? 128u : 2u;
                    const uint32_t step_ga = static_cast<uint32_t>(p.a_bytes) / 16u, step_gb = static_cast<uint32_t>(p.b_bytes) / 16u;
                    const uint32_t stage_a = step_ga * static_cast<uint32_t>(p.group), stage_b = step_gb * static_cast<uint32_t>(p.group);
                    for (int seg = kb_begin; ok && seg < kb_end; seg += job.seg_kb, ++it) {
                        const int acc = it & 1;
                        const uint32_t aph = static_cast<uint32_t>(it >> 1) & 1u;
                        ok = PAIR ? lin_wait_cluster(tempty0 + 8 * acc, aph ^ 1u, wc, kSiteLinTmemEmpty)
                                  : lin_wait(tempty0 + 8 * acc, aph ^ 1u, wc, kSiteLinTmemEmpty);
                        if (!ok) break;
                        tc_fence_after_sync();
                        const uint32_t d = tmem_base + static_cast<uint32_t>(acc * p.acc_cols);
                        const int seg_end = kb_end - seg < job.seg_kb ? kb_end : seg + job.seg_kb;
                        for (int kb0 = seg; kb0 < seg_end; kb0 += p.group) {
                            const int count = seg_end - kb0 < p.group ? seg_end - kb0 : p.group;
                            ok = lin_wait(full0 + 8 * stage, phase, wc, kSiteLinFull);
                            if (!ok) break;
                            tc_fence_after_sync();
                            const uint64_t a0 = desc_a + static_cast<uint32_t>(stage) * stage_a;
                            const uint64_t b0 = desc_b + static_cast<uint32_t>(stage) * stage_b;
                            if (lin_elect()) {
                                auto issue = [&](uint64_t a, uint64_t b, uint32_t more) {
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk) {
                                        const uint32_t add = kk != 0 ? 1u : more;
                                        if constexpr (PAIR) mma_f16_pair(d, a + kk * step_a, b + kk * kStepB, idesc, add);
                                        else mma_f16(d, a + kk * step_a, b + kk * kStepB, idesc, add);
                                    }
                                };
                                issue(a0, b0, kb0 != seg ? 1u : 0u);
                                for (int g = 1; g < count; ++g) issue(a0 + g * step_ga, b0 + g * step_gb, 1u);
                                if constexpr (PAIR) mma_commit_pair_multicast(empty0 + 8 * stage, 0x3);
                                else mma_commit(empty0 + 8 * stage);
                            }
                            __syncwarp();
                            ++issued;
                            if (++stage == S) {
                                stage = 0;
                                phase ^= 1u;
                            }
                        }
                        if (!ok) break;
                        if (lin_elect()) {
                            if constexpr (PAIR) mma_commit_pair_multicast(tfull0 + 8 * acc, 0x3);
                            else mma_commit(tfull0 + 8 * acc);
                        }
                        __syncwarp();
                    }
                }
            }
            __syncwarp();
            if constexpr (PARTIAL) cluster_sync();
        } else {
            // ------------------------------------------------------------------
            // epilogue: 32 rows a warp (the TMEM lanes it may read), every other kCh columns
            // ------------------------------------------------------------------
            const int quarter = warp & 3;
            const int half = (warp - 2) >> 2;
            const uint32_t lead_tempty0 = PAIR ? mapa_shared(tempty0, 0) : tempty0;
            uint8_t* staging = smem + p.stage_at + (warp - 2) * 32 * kBlockBytes;   // (one tile or split k: set)
            auto hand_back = [&](int acc) {   // this warp has read its part of the accumulator
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR) mbar_arrive_remote_relaxed(lead_tempty0 + 8 * acc);
                    else mbar_arrive(tempty0 + 8 * acc);
                }
            };
            // Gradients: this warp's half of the accumulator's columns, from `half * bn / 2`, summed
            // over a tile's segments
            const int c_half = half * (p.bn / 2);
            auto add_segments = [&](float (&sum)[8][kCh], const LinearJob& job, int kb_begin, int kb_end, bool any) {
                const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
                for (int c = 0; c < 8; ++c)
#pragma unroll
                    for (int e = 0; e < kCh; ++e) sum[c][e] = 0.f;
                for (int seg = kb_begin; seg < kb_end; seg += job.seg_kb, ++it) {
                    const int acc = it & 1;
                    ok = lin_wait(tfull0 + 8 * acc, static_cast<uint32_t>(it >> 1) & 1u, wc, kSiteLinTmemFull);
                    if (!ok) break;
                    tc_fence_after_sync();
                    if (any) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            if (q * kCh < p.bn / 2) {
                                uint32_t r[kCh];
                                lin_tmem_ld16(t_row + acc * p.acc_cols + c_half + q * kCh, r);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < kCh; ++e) sum[q][e] += __uint_as_float(r[e]);
                            }
                        }
                    }
                    hand_back(acc);
                }
            };
            int j = 0, tile = 0;
            if constexpr (PARTIAL) {
                // The CTA's only tile: its sums go to the CTAs of the cluster that finish their columns,
                // over those CTAs' rings, once all have read their stages.
                const bool have = tile_of<SPLIT>(p, 0, unit, units, 0, &j, &tile);
                const SplitTile t = split_tile<kGrad>(p, have ? j : 0, have ? tile : 0);
                const LinearJob& job = p.job[kGrad ? t.job : 0];
                const bool any = have && quarter * 32 < t.rows;
                const int lrow = quarter * 32 + lane;
                // 8 columns c .. of this lane's row, part 0 or (gated) 1
                auto push = [&](const float* v, int part, int c) {
                    const int owner = c / t.slice;
                    const int group = ((rank * (kGated ? 2 : 1) + part) * t.slice + c - owner * t.slice) / 4;
                    const uint32_t to = mapa_shared(sA, static_cast<uint32_t>(owner)) + static_cast<uint32_t>((group * t.rows + lrow) * 16);
                    st_shared_cluster_v4(to, v[0], v[1], v[2], v[3]);
                    st_shared_cluster_v4(to + static_cast<uint32_t>(t.rows * 16), v[4], v[5], v[6], v[7]);
                };
                if constexpr (kGrad) {
                    int kb_begin, kb_end;
                    k_range(job, &kb_begin, &kb_end);
                    float sum[8][kCh];
                    add_segments(sum, job, kb_begin, have ? kb_end : kb_begin, any);
                    fence_proxy_async_smem();
                    cluster_sync();
                    if (ok && any && lrow < t.rows) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const int c = c_half + q * kCh;
                            if (q * kCh < p.bn / 2 && c < t.width) push(sum[q], 0, c);
                            if (q * kCh < p.bn / 2 && c + 8 < t.width) push(sum[q] + 8, 0, c + 8);
                        }
                    }
                } else {
                    if (have) ok = lin_wait(tfull0, 0u, wc, kSiteLinTmemFull);
                    tc_fence_after_sync();
                    fence_proxy_async_smem();
                    cluster_sync();
                    if (ok && any) {
                        const uint32_t t_acc = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
                        for (int c = half * kCh; c < t.width; c += 2 * kCh) {
#pragma unroll
                            for (int part = 0; part < (kGated ? 2 : 1); ++part) {
                                uint32_t r[kCh];
                                lin_tmem_ld16(t_acc + part * p.wcols + c, r);
                                tmem_ld_wait();
                                float v[kCh];
#pragma unroll
                                for (int e = 0; e < kCh; ++e) v[e] = __uint_as_float(r[e]);
                                if (lrow < t.rows) {
                                    push(v, part, c);
                                    if (c + 8 < t.width) push(v + 8, part, c + 8);
                                }
                            }
                        }
                    }
                }
            } else {
                for (int i = 0; ok && tile_of<SPLIT>(p, pass, unit, units, i, &j, &tile); ++i) {
                    const LinearJob& job = p.job[kGrad ? j : 0];
                    int pm, pn;
                    tile_coord(tile, job.num_m, job.num_n, p.group_m, &pm, &pn);
                    const int src = kGrad && pm >= job.num_m1 ? 1 : 0;
                    const int m0 = (pm - src * job.num_m1) * kTileRows + (PAIR ? rank * 128 : 0) + quarter * 32;
                    const int n0 = pn * p.wcols;
                    const int row = m0 + lane;
                    const bool any = m0 < job.rows;   // rows of this warp's to store
                    const int left = job.cols - n0;
                    const int width = left < p.wcols ? left : p.wcols;
                    if constexpr (kGrad) {
                        int kb_begin, kb_end;
                        k_range(job, &kb_begin, &kb_end);
                        float sum[8][kCh];
                        add_segments(sum, job, kb_begin, kb_end, any);
                        if (!ok) break;
                        if (any)
                            finish_sums<TYPE, ANY>(job, staging, sum, src, m0, job.rows - m0 < 32 ? job.rows - m0 : 32, n0 + c_half,
                                              width - c_half < p.bn / 2 ? width - c_half : p.bn / 2);
                    } else {
                        // what the epilogue reads from memory, on its way while the k loop runs
                        if (p.bias[0] != nullptr && lane * 64 < width) {
                            prefetch_l1(p.bias[0] + n0 + lane * 64);
                            if (kGated && p.bias[1] != nullptr) prefetch_l1(p.bias[1] + n0 + lane * 64);
                        }
                        if (MODE == kModeLinear && p.residual != nullptr && row < job.rows)
                            for (int c = half * 64; c < width; c += 128) prefetch_l2(p.residual + row * p.ldr + n0 + c);
                        const int acc = it & 1;
                        ok = lin_wait(tfull0 + 8 * acc, static_cast<uint32_t>(it >> 1) & 1u, wc, kSiteLinTmemFull);
                        if (!ok) break;
                        ++it;
                        tc_fence_after_sync();
                        const uint32_t t_acc = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                               static_cast<uint32_t>(acc * p.acc_cols);
                        if constexpr (KIND == kKindDirect) {
                            if (any) {
#pragma unroll 1
                                for (int c = half * kCh; c < width; c += 2 * kCh) {
                                    uint32_t ra[kCh], rb[kCh];
                                    lin_tmem_ld16(t_acc + c, ra);
                                    if constexpr (kGated) lin_tmem_ld16(t_acc + p.wcols + c, rb);
                                    tmem_ld_wait();
                                    float a[kCh], b[kCh];
#pragma unroll
                                    for (int e = 0; e < kCh; ++e) {
                                        a[e] = __uint_as_float(ra[e]);
                                        b[e] = kGated ? __uint_as_float(rb[e]) : 0.f;
                                    }
                                    if (row < job.rows)
                                        finish_row<TYPE, MODE, kCh>(p, job, a, b, 0, row, n0 + c,
                                                                    width - c < kCh ? width - c : kCh);
                                }
                            }
                        } else if (any) {
                            // this warp's half of the columns, a multiple of 32, in blocks of up to 64
                            const int mid = ((width + 31) / 32 + 1) / 2 * 32;
                            const int end = half == 0 && mid < width ? mid : width;
#pragma unroll 1
                            for (int c = half * mid; c < end; c += 64)
                                finish_block<TYPE, MODE>(p, job, staging, t_acc + c, p.wcols, m0,
                                                         job.rows - m0 < 32 ? job.rows - m0 : 32, n0 + c,
                                                         end - c < 64 ? end - c : 64);
                        }
                        hand_back(acc);
                    }
                }
            }
            __syncwarp();
        }
    };
    if constexpr (!SPLIT) {
        run(std::false_type{}, 0);
    } else {
        run(std::true_type{}, 0);
        // all partial sums of this CTA's columns are in its shared memory
        cluster_sync();
        int j, tile;
        if (warp >= 2 && tile_of<SPLIT>(p, 0, unit, units, 0, &j, &tile)) {
            // 8 columns of a row per thread and turn, neighbouring threads on neighbouring
            // rows; summed in rank order
            constexpr int kW = 8;
            const SplitTile t = split_tile<kGrad>(p, j, tile);
            const int c_begin = rank * t.slice;
            const int c_end = c_begin + t.slice < t.width ? c_begin + t.slice : t.width;
            const int items = c_begin < c_end ? (c_end - c_begin + kW - 1) / kW * t.rows : 0;
            const LinearJob& job = p.job[kGrad ? t.job : 0];
            const bool whole = job.vec_out && (kGrad || ((p.vec_res || p.residual == nullptr) && (p.vec_keep || p.keep[0] == nullptr)));
            for (int e = static_cast<int>(threadIdx.x) - 64; e < items; e += 32 * kLinEpiWarps) {
                const int lrow = e % t.rows;
                const int cl = e / t.rows * kW;
                const float4* from = reinterpret_cast<const float4*>(smem) + cl / 4 * t.rows + lrow;
                const int part = t.slice / 4 * t.rows;   // of 16 bytes
                float a[kW] = {}, b[kW] = {};
                for (int q = 0; q < p.split; ++q, from += (kGated ? 2 : 1) * part) {
#pragma unroll
                    for (int h = 0; h < kW; h += 4) {
                        const float4 v = from[h / 4 * t.rows];
                        a[h] += v.x;
                        a[h + 1] += v.y;
                        a[h + 2] += v.z;
                        a[h + 3] += v.w;
                        if constexpr (kGated) {
                            const float4 w = from[part + h / 4 * t.rows];
                            b[h] += w.x;
                            b[h + 1] += w.y;
                            b[h + 2] += w.z;
                            b[h + 3] += w.w;
                        }
                    }
                }
                const int c = c_begin + cl;
                if (whole) {
                    finish_row<TYPE, MODE, kW>(p, job, a, b, t.src, t.row0 + lrow, t.col0 + c, c_end - c < kW ? c_end - c : kW);
                    continue;
                }
                // rows at any alignment: the results go back to where this thread's sums of CTA 0 (kept
                // values) and CTA 1 (outputs) were, for the warps to write row by row
                float4* kept = reinterpret_cast<float4*>(smem) + cl / 4 * t.rows + lrow;
                float4* done = kept + (kGated ? 2 : 1) * part;
                if constexpr (!kGrad) {
                    const int n = c_end - c < kW ? c_end - c : kW;
                    add_bias_row<TYPE, kW>(a, p.bias[0], t.col0 + c, n, p.vec_bias);
                    if constexpr (kGated) add_bias_row<TYPE, kW>(b, p.bias[1], t.col0 + c, n, p.vec_bias);
#pragma unroll
                    for (int h = 0; h < kW; h += 4) {
                        kept[h / 4 * t.rows] = make_float4(a[h], a[h + 1], a[h + 2], a[h + 3]);
                        if constexpr (kGated) kept[part + h / 4 * t.rows] = make_float4(b[h], b[h + 1], b[h + 2], b[h + 3]);
                    }
                    act_switch<kW>(a, p.act);
                    if constexpr (kGated) {
#pragma unroll
                        for (int h = 0; h < kW; ++h) a[h] *= b[h];
                    }
                }
#pragma unroll
                for (int h = 0; h < kW; h += 4) done[h / 4 * t.rows] = make_float4(a[h], a[h + 1], a[h + 2], a[h + 3]);
            }
            if (!whole) {
                asm volatile("bar.sync 1, %0;" ::"n"(32 * kLinEpiWarps) : "memory");
                const int part = t.slice * t.rows;   // of floats
                const float* vals = reinterpret_cast<const float*>(smem);
                for (int r = warp - 2; r < t.rows; r += kLinEpiWarps) {
                    const long long row = t.row0 + r;
                    for (int c = c_begin + lane; c < c_end; c += 32) {
                        const int at = ((c - c_begin) / 4 * t.rows + r) * 4 + (c - c_begin) % 4;
                        const int col = t.col0 + c;
                        float v = vals[(kGated ? 2 : 1) * part + at];
                        if constexpr (kGrad) {
                            if (job.out_f32) {
                                float* o = static_cast<float*>(job.out[t.src]) + row * job.ldo + col;
                                *o = job.accumulate ? *o + v : v;
                            } else {
                                uint16_t* o = static_cast<uint16_t*>(job.out[t.src]) + row * job.ldo + col;
                                *o = to_16<TYPE>(job.accumulate ? to_f32<TYPE>(*o) + v : v);
                            }
                        } else {
                            if (p.keep[0] != nullptr) p.keep[0][row * p.ldk + col] = to_16<TYPE>(vals[at]);
                            if (kGated && p.keep[1] != nullptr) p.keep[1][row * p.ldk + col] = to_16<TYPE>(vals[part + at]);
                            if (MODE == kModeLinear && p.residual != nullptr) v += to_f32<TYPE>(p.residual[row * p.ldr + col]);
                            static_cast<uint16_t*>(job.out[0])[row * job.ldo + col] = to_16<TYPE>(v);
                        }
                    }
                }
            }
        }
        if constexpr (kGrad) {
            // the ring's stages are loaded again over the partials once all have read them
            fence_proxy_async_smem();
            __syncthreads();
            run(std::false_type{}, 1);
        }
    }
    if (!ok && leader && warp == 0) {
        // abort: the loads already issued land (waits with a limit) before the CTA can exit
        const int pending = static_cast<int>(issued < S ? issued : S);
        for (int b = 1; b <= pending; ++b) {
            const int s = (stage - b + S) % S;
            mbar_wait(full0 + 8 * s, stage - b < 0 ? phase ^ 1u : phase, wc_drain, kSiteLinDrain);
        }
    }
    if (!ok && leader && warp == 1 && issued > 0) {
        // abort: every MMA issued so far finishes before TMEM is freed
        if (lin_elect()) {
            if constexpr (PAIR) mma_commit_pair_multicast(drain_bar, 0x1);
            else mma_commit(drain_bar);
        }
        __syncwarp();
        mbar_wait(drain_bar, 0u, wc_drain, kSiteLinDrain);
    }
    __syncwarp();
    tc_fence_before_sync();
    if constexpr (PAIR) cluster_sync();
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        if constexpr (PAIR) tmem_dealloc_pair(tmem_base, static_cast<uint32_t>(p.tmem_cols));
        else tmem_dealloc(tmem_base, static_cast<uint32_t>(p.tmem_cols));
    }
}

// Tensor map, 128-byte swizzle, of `inner` contiguous elements in `outer` lines.  blocks 0: boxes of
// 64 x box_outer.  blocks > 0: the line as 64-element blocks, boxes of {64, box_outer, blocks}.
inline bool lin_map(CUtensorMap* map, int type, const void* base, long long inner, long long outer, long long ld,
                    int box_outer, int blocks, char* msg, size_t msg_len)
{
    TmapEncodeFn enc = tmap_encoder();
    if (enc == nullptr) {
        snprintf(msg, msg_len, "cuTensorMapEncodeTiled is not available from the driver");
        return false;
    }
    const bool flat = blocks == 0;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(flat ? inner : 64), static_cast<cuuint64_t>(outer),
                                static_cast<cuuint64_t>((inner + 63) / 64)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2u, 128u};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(kLinBK), static_cast<cuuint32_t>(box_outer),
                               static_cast<cuuint32_t>(flat ? 1 : blocks)};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(map, type == kTypeBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                           flat ? 2 : 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        snprintf(msg, msg_len, "cuTensorMapEncodeTiled failed (%d) for %lld x %lld, stride %lld, box 64 x %d x %d",
                 static_cast<int>(r), inner, outer, ld, box_outer, blocks);
        return false;
    }
    return true;
}

inline bool lin_aligned16(const void* p, long long ld_bytes)
{
    return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld_bytes)) & 15u) == 0;
}

// A job's tiles, of tile_rows x wcols.
inline LinearJob lin_job(int rows, int cols, int k, int k_sources, int row_sources, int tile_rows, int wcols)
{
    LinearJob j = {};
    j.rows = rows;
    j.cols = cols;
    j.kbs = (k + kLinBK - 1) / kLinBK;
    j.k_sources = k_sources;
    j.num_m1 = (rows + tile_rows - 1) / tile_rows;
    j.num_m = j.num_m1 * row_sources;
    j.num_n = (cols + wcols - 1) / wcols;
    j.num_tiles = j.num_m * j.num_n;
    j.seg_kb = j.kbs * k_sources;
    return j;
}

// LinearParams::extra: the number of tiles of job 1 that the units with fewer tiles of job 0 take
// first, so that the last of all is done earliest.  Times in microseconds: a k-block's operands at 95
// GB/s an SM, or 0.3; with split k 2.5 for the sums; a tile's results 0.0165 a column of 16 bits.
inline int lin_extra(const LinearParams& p, int bn, long long units)
{
    const long long t0 = p.job[0].num_tiles * static_cast<long long>(p.split), t1 = p.job[1].num_tiles;
    const long long late = units - (p.split > 1 ? t0 : t0 % units);
    if (t1 == 0 || late <= 0 || late == units) return 0;
    const double block = (128 + bn) * 0.00135 > 0.3 ? (128 + bn) * 0.00135 : 0.3;
    const double store = (p.job[1].out_f32 ? 0.033 : 0.0165) * bn, loop = p.job[1].kbs * p.job[1].k_sources * block;
    const double c0 = p.job[0].kbs * p.job[0].k_sources / p.split * block + (p.split > 1 ? 2.5 : 0.0);
    const double c1 = loop > store ? loop : store;
    double best = -1.0;
    int extra = 0;
    for (int e = 0; e <= 4096; ++e) {
        const long long rest = t1 > e * late ? (t1 - e * late + units - 1) / units : 0;   // rounds of all units
        const long long most = (t1 + late - 1) / late;
        const double end0 = c0 + c1 * static_cast<double>(rest), end1 = c1 * static_cast<double>((e < most ? e : most) + rest);
        const double end = end0 > end1 ? end0 : end1;
        if (best < 0.0 || end < best) {
            best = end;
            extra = e;
        }
        if (e * late >= t1 || end1 > end0) break;
    }
    return extra;
}

template <int TYPE, int MODE, bool PAIR>
int launch_linear_instance(const LinearLaunch& g, cudaStream_t stream, char* msg, size_t msg_len)
{
    constexpr bool kGated = MODE == kModeGated;
    constexpr bool kGrad = MODE == kModeGrad;
    constexpr int kTileRows = PAIR ? 256 : 128;
    const int bn_unit = PAIR ? (kGrad ? 128 : 32) : (kGrad ? 64 : kGated ? 32 : 16);
    if (g.bn < bn_unit || g.bn > 256 || g.bn % bn_unit != 0) {
        snprintf(msg, msg_len, "linear product: bad tile width %d", g.bn);
        return 1;
    }
    LinearParams p = {};
    p.bn = g.bn;
    p.wcols = kGated ? g.bn / 2 : g.bn;
    p.group_m = g.group_m;
    if constexpr (kGrad) {
        int jobs = 0;
        if (g.dx != nullptr) {
            LinearJob& j = p.job[jobs++];
            j = lin_job(g.n, g.K, g.M, g.parts, 1, kTileRows, p.wcols);
            j.idesc = idesc_f16(TYPE == kTypeBF16, false, true, kTileRows, g.bn);
            j.out[0] = g.dx;
            j.ldo = g.ld_dx;
            if (j.seg_kb > kSegmentKb16) j.seg_kb = kSegmentKb16;
            j.vec_out = lin_aligned16(g.dx, g.ld_dx * 2);
        }
        if (g.dW[0] != nullptr) {
            LinearJob& j = p.job[jobs++];
            j = lin_job(g.M, g.K, g.n, 1, g.parts, kTileRows, p.wcols);
            j.a_mn = 1;
            j.idesc = idesc_f16(TYPE == kTypeBF16, true, true, kTileRows, g.bn);
            j.out[0] = g.dW[0];
            j.out[1] = g.dW[1];
            j.ldo = g.ld_dw;
            j.out_f32 = g.grad_f32;
            j.accumulate = g.accumulate;
            if (g.grad_f32 || j.seg_kb > kSegmentKb16) j.seg_kb = g.grad_f32 ? kSegmentKb32 : kSegmentKb16;
            j.vec_out = lin_aligned16(g.dW[0], g.ld_dw * (g.grad_f32 ? 4 : 2)) && lin_aligned16(g.dW[1], 0);
        }
        if (jobs == 2 && p.job[1].kbs * p.job[1].k_sources > p.job[0].kbs * p.job[0].k_sources) {
            const LinearJob t = p.job[0];   // longer k loops first
            p.job[0] = p.job[1];
            p.job[1] = t;
        }
        if (jobs == 1) {
            p.job[1] = p.job[0];
            p.job[1].num_tiles = 0;
        }
    } else {
        LinearJob& j = p.job[0];
        j = lin_job(g.n, g.M, g.K, 1, 1, kTileRows, p.wcols);
        j.idesc = idesc_f16(TYPE == kTypeBF16, false, false, kTileRows, g.bn);
        j.out[0] = g.out;
        j.ldo = g.ldo;
        j.vec_out = lin_aligned16(g.out, g.ldo * 2);
    }
    const long long tiles = static_cast<long long>(p.job[0].num_tiles) + p.job[1].num_tiles;
    p.split = PAIR || g.split < 2 ? 1 : g.split;
    const int kb0 = p.job[0].kbs * p.job[0].k_sources;
    while (p.split > kb0) p.split /= 2;   // every CTA of a cluster has a k-block
    p.bias[0] = static_cast<const uint16_t*>(g.bias[0]);
    p.bias[1] = static_cast<const uint16_t*>(g.bias[1]);
    p.keep[0] = static_cast<uint16_t*>(g.keep[0]);
    p.keep[1] = static_cast<uint16_t*>(g.keep[1]);
    p.ldk = g.ldk;
    p.residual = static_cast<const uint16_t*>(g.residual);
    p.ldr = g.ldr;
    p.act = g.act;
    p.vec_res = lin_aligned16(g.residual, g.ldr * 2);
    p.vec_keep = lin_aligned16(g.keep[0], g.ldk * 2) && lin_aligned16(g.keep[1], 0);
    p.vec_bias = lin_aligned16(g.bias[0], 0) && lin_aligned16(g.bias[1], 0);
    p.db_partial = g.db_partial;
    p.db_chunks = g.db_chunks;
    p.db_parts = g.parts;
    p.db_M = g.M;
    p.db_f32 = g.grad_f32;
    p.db_accumulate = g.accumulate;
    p.db[0] = g.db[0];
    p.db[1] = g.db[1];
    p.status = g.status;
    p.wait_limit_ns = g.wait_limit_ns;

    // Few rows: the weights' stream is the bound, and two CTAs fit on an SM, each with half of the
    // shared memory and of TMEM; the next launch's CTAs can be there when this one's finish.
    p.acc_cols = 32;   // (the epilogue reads 32 columns at a time)
    while (p.acc_cols < (kGated ? p.wcols + (p.wcols + 31) / 32 * 32 : g.bn)) p.acc_cols *= 2;
    const long long sms = g.num_sms > 0 ? g.num_sms : 1;
    const bool few = !PAIR && !kGrad && g.n <= kFewRows &&
                     (p.acc_cols <= 128 || tiles * p.split <= 2 * sms || p.split > 1);
    // Units: each gets the same number of tiles (the last wave is not left partial).
    const int share = PAIR ? 2 : p.split;
    long long units = static_cast<long long>(p.job[0].num_tiles) * p.split;
    long long per_unit = 1;
    if (p.split > 1) {
        if (p.job[1].num_tiles > 0) {
            // clusters that fit on the device at once; job 0 has no more tiles than that
            long long clusters = split_k_capacity(p.split);
            if (clusters > sms / p.split) clusters = sms / p.split;
            if (clusters < p.job[0].num_tiles) clusters = p.job[0].num_tiles;
            units = clusters * p.split;
            per_unit = 2;
        }
    } else {
        units = tiles;
        const long long most = PAIR ? sms / 2 : few ? 2 * sms : sms;
        const long long cap = most > 0 ? most : 1;
        per_unit = (units + cap - 1) / cap;
        units = kGrad && p.job[1].num_tiles > 0 ? (units < cap ? units : cap) : (units + per_unit - 1) / per_unit;
    }
    // TMEM: two accumulators unless every unit has one tile of one segment.
    const bool one = per_unit == 1 && (!kGrad || p.job[1].num_tiles == 0) && p.job[0].seg_kb >= kb0;
    if constexpr (kGrad) p.extra = lin_extra(p, g.bn, units);
    p.tmem_cols = one ? p.acc_cols : 2 * p.acc_cols;

    // Shared memory: the ring, the staging buffers behind it, the barriers.
    p.a_rows = PAIR || kGrad || g.n >= 128 ? 128 : (g.n + 7) / 8 * 8;
    p.a_bytes = p.a_rows * 128;
    const int b_rows = PAIR ? g.bn / 2 : g.bn;
    p.b_bytes = b_rows * 128;
    // One narrow tile per CTA: its rows are written as they are, which takes less time from the last
    // MMA to the end (261 x 128 x 64: 3.9 us, through shared memory 4.8).
    const bool direct = few || (!PAIR && !kGrad && per_unit == 1 && g.bn <= 64 && p.job[0].vec_out &&
                                (p.vec_res || g.residual == nullptr) && (p.vec_keep || g.keep[0] == nullptr));
    const bool staged = kGrad || (!direct && p.split == 1);
    const int stage_bytes = p.a_bytes + p.b_bytes;
    const int fit = linear_ring_room(few, staged) / stage_bytes;
    p.group = linear_group(g, PAIR, g.bn, few, staged);
    p.stages = fit / p.group;
    // one tile per CTA: no more than its k loop takes, so that the next launch's CTAs find room
    if (per_unit == 1 && !kGrad) {
        const int turns = ((kb0 + p.split - 1) / p.split + p.group - 1) / p.group;
        if (p.stages > turns) p.stages = turns;
    }
    if (p.stages > kLinMaxStages) p.stages = kLinMaxStages;
    // (with few rows the MMA reads up to 16 KB from the start of the last k-block's A: inside this)
    int ring = p.stages * p.group * stage_bytes;
    const int reach = (p.stages * p.group - 1) * p.a_bytes + 16384;
    if (ring < reach) ring = reach;
    const int rows = g.n < 128 && !kGrad ? g.n : 128;
    const int partial = p.split > 1 ? p.split * rows * (g.bn / p.wcols) * split_slice(p.wcols, p.split) * 4 : 0;
    if (ring < partial) ring = partial;
    ring = (ring + 1023) / 1024 * 1024;
    p.stage_at = staged ? ring : -1;
    p.ring_bytes = ring + (staged ? kLinStageBytes : 0);
    // Clusters: no CTA of one can wait for TMEM columns that a CTA of a cluster waiting for it holds.  Split k
    // of a forward pass: at most two CTAs per SM, of 256 columns at most; the others one, by their
    // registers; and none beside a cluster's CTA of the GEMMs (190 KB and more).
    int smem_bytes = 1024 + p.ring_bytes + kLinBarBytes;
    if (share > 1 && smem_bytes < 80 * 1024) smem_bytes = 80 * 1024;
    if (smem_bytes > kLinSmemBytes) {
        snprintf(msg, msg_len, "linear product: %d bytes of shared memory needed", smem_bytes);
        return 1;
    }

    if constexpr (!kGrad) {
        // as much as the launch before leaves HBM idle for; beyond the ring's own loads it is worth nothing
        p.prefetch_kb = few ? 8 : 0;
        p.w_rows[0] = static_cast<const uint8_t*>(g.W[0]);
        p.w_rows[1] = static_cast<const uint8_t*>(g.W[1]);
        p.w_ld_bytes = g.ldw * 2;
    }

    LinearMaps maps;
    bool ok = true;
    if constexpr (kGrad) {
        // one load for a tile's blocks where a line's last block may be read whole
        p.wide_z = g.z_padded || g.M % 64 == 0;
        p.wide_w = g.w_padded || g.K % 64 == 0;
        p.wide_x = g.x_padded || g.K % 64 == 0;
        const int blocks = b_rows / 64;
        for (int s = 0; s < 2 && ok; ++s) {
            const int q = s < g.parts ? s : 0;
            ok = lin_map(&maps.m[s], g.type, g.dz[q], g.M, g.n, g.ldz, kLinBK, p.wide_z ? 2 : 0, msg, msg_len) &&
                 lin_map(&maps.m[5 + s], g.type, g.dz[q], g.M, g.n, g.ldz, 128, 0, msg, msg_len);
            if (g.dx != nullptr)
                ok = ok && lin_map(&maps.m[2 + s], g.type, g.W[q], g.K, g.M, g.ldw, kLinBK, p.wide_w ? blocks : 0, msg, msg_len);
            else
                maps.m[2 + s] = maps.m[0];
        }
        if (g.dW[0] != nullptr)
            ok = ok && lin_map(&maps.m[4], g.type, g.x, g.K, g.n, g.ldx, kLinBK, p.wide_x ? blocks : 0, msg, msg_len);
        else
            maps.m[4] = maps.m[0];
    } else {
        const int box = kGated ? g.bn / 2 : b_rows;
        ok = lin_map(&maps.m[0], g.type, g.x, g.K, g.n, g.ldx, p.a_rows, 0, msg, msg_len) &&
             lin_map(&maps.m[1], g.type, g.W[0], g.K, g.M, g.ldw, box, 0, msg, msg_len);
        if (kGated && ok) ok = lin_map(&maps.m[2], g.type, g.W[1], g.K, g.M, g.ldw, box, 0, msg, msg_len);
        else maps.m[2] = maps.m[1];
        for (int i = 3; i < 7; ++i) maps.m[i] = maps.m[1];
    }
    if (!ok) return 1;

    constexpr int kWhole = PAIR ? kKindPair : kKindOne;
    bool any = true;
    if constexpr (kGrad) any = g.K % 8 != 0 || (p.job[0].num_tiles > 0 && !p.job[0].vec_out) || (p.job[1].num_tiles > 0 && !p.job[1].vec_out);
    auto kern = linear_kernel<TYPE, MODE, kWhole, true>;
    int kind = kWhole;
    if constexpr (kGrad) {
        if (!any) kern = linear_kernel<TYPE, MODE, kWhole, false>;
    }
    if constexpr (!PAIR) {
        if (p.split > 1) {
            kern = linear_kernel<TYPE, MODE, kKindSplit, true>;
            kind = kKindSplit;
            if constexpr (kGrad) {
                if (!any) kern = linear_kernel<TYPE, MODE, kKindSplit, false>;
            }
        }
        if constexpr (!kGrad) {
            if (p.split == 1 && direct) {
                kern = linear_kernel<TYPE, MODE, kKindDirect, true>;
                kind = kKindDirect;
            }
        }
    }
    static SmemOptIn smem_opt[8];
    cudaError_t e = smem_opt[kind + (any ? 4 : 0)].ensure(reinterpret_cast<const void*>(kern), kLinSmemBytes);
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        return 1;
    }
    cudaLaunchAttribute attr[2];
    int attrs = 0;
    if (share > 1) {
        attr[attrs].id = cudaLaunchAttributeClusterDimension;
        attr[attrs].val.clusterDim.x = static_cast<unsigned>(share);
        attr[attrs].val.clusterDim.y = 1;
        attr[attrs].val.clusterDim.z = 1;
        ++attrs;
    }
    if (g.pdl) {
        attr[attrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[attrs].val.programmaticStreamSerializationAllowed = 1;
        ++attrs;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(units * (PAIR ? 2 : 1)), 1, 1);
    cfg.blockDim = dim3(kLinThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem_bytes);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = static_cast<unsigned>(attrs);
    e = cudaLaunchKernelEx(&cfg, kern, maps, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "linear product launch failed: %s", cudaGetErrorString(e));
        return 1;
    }
    return 0;
}

template <int TYPE>
int launch_linear_type(const LinearLaunch& g, cudaStream_t stream, char* msg, size_t msg_len)
{
    switch (g.mode) {
    case kModeLinear:
        return g.pair ? launch_linear_instance<TYPE, kModeLinear, true>(g, stream, msg, msg_len)
                      : launch_linear_instance<TYPE, kModeLinear, false>(g, stream, msg, msg_len);
    case kModeGated:
        return g.pair ? launch_linear_instance<TYPE, kModeGated, true>(g, stream, msg, msg_len)
                      : launch_linear_instance<TYPE, kModeGated, false>(g, stream, msg, msg_len);
    case kModeGrad:
        return g.pair ? launch_linear_instance<TYPE, kModeGrad, true>(g, stream, msg, msg_len)
                      : launch_linear_instance<TYPE, kModeGrad, false>(g, stream, msg, msg_len);
    default:
        snprintf(msg, msg_len, "unknown linear mode %d", g.mode);
        return 1;
    }
}

}  // namespace
}  // namespace bsk
