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
// Two k sources (dx = dg Wg + du Wu): one k loop over both, one accumulator, so
// that dx is rounded once.
//
// Roles (320 threads): warp 0 loads by TMA into a ring of k slices, warp 1 issues
// the MMAs, warps 2..9 are the epilogue, overlapped with the next tile's loop by a
// second accumulator.  Tile sizes are run-time values (TMA boxes, instruction
// descriptor, ring depth): with few rows only those are staged -- the MMA reads
// on into whatever follows in shared memory, and those rows are not stored.
//
// Split k (one-CTA tiles, few tiles): the CTAs of a cluster share a tile's k
// loop, leave FP32 partials in their own shared memory and each finish a part of
// the columns from all of them, summed in rank order (the result does not depend
// on timing).
#pragma once

#include <cstdio>

#include "bsk_internal.h"
#include "linear_math.cuh"
#include "ptx.cuh"

namespace bsk {
namespace {

constexpr int kLinEpiWarps = 8;                  // two per quarter of the TMEM lanes: every other kCh columns
constexpr int kLinThreads = 64 + 32 * kLinEpiWarps;
constexpr int kLinBK = 64;                       // k values per stage: one 128-byte swizzle row
constexpr int kLinBarBytes = 512;
constexpr int kLinSmemBytes = 232448;            // all of it: one CTA per SM, so that 512 TMEM columns are free
constexpr int kLinRingBytes = kLinSmemBytes - 1024 - kLinBarBytes;
constexpr int kLinMaxStages = 24;
constexpr int kLinAccCols = 256;                 // TMEM columns of one accumulator (two of them)
constexpr int kCh = 16;                          // columns per epilogue step: 32 bytes of 16-bit values
constexpr int kStagePitch = 9;                   // words per row of a warp's staging buffer (odd: no bank conflicts)
constexpr int kStageBytes = kLinEpiWarps * 32 * kStagePitch * 4;
// FP32 weight gradients: k-blocks summed in an accumulator before they are added to
// FP32 registers.  A tensor-core accumulation cuts each of its sums (toward zero), so
// an error grows with their number: dW over 8192 tokens came out 2e-5 off, in segments of 256
// tokens 1e-6, as much as FP32 arithmetic gives.
constexpr int kSegmentKb = 16;

enum LinearWaitSite {
    kSiteLinEmpty = 0x30,
    kSiteLinFull = 0x31,
    kSiteLinTmemEmpty = 0x32,
    kSiteLinTmemFull = 0x33,
    kSiteLinDrain = 0x34,
};

struct LinearParams {
    int rows, cols;           // of the result (weight gradient: of each source's)
    int kbs, k_sources;       // k-blocks per source
    int num_m, num_m1;        // tile rows in all, of the first source (weight gradient)
    int num_n, num_tiles, group_m;
    int a_rows;               // rows of A staged per CTA (128, or the few there are)
    int bn;                   // accumulator columns per tile
    int wcols;                // result columns per tile: bn, gated bn / 2
    int stages, a_bytes, b_bytes;
    int seg_kb;               // weight gradient: k-blocks per segment
    int stage_out;            // rows that no 16-byte accesses reach go through the staging buffers
    int split;                // CTAs that share a tile's k loop (a cluster); 1: none
    uint32_t idesc;
    void* out[2];
    long long ldo;
    const uint16_t* bias[2];
    const uint16_t* residual;
    long long ldr;
    uint16_t* keep[2];
    long long ldk;
    int act;
    int out_f32, accumulate;
    int vec_out, vec_res, vec_keep, vec_bias;   // 16-byte accesses allowed
    int* status;
    unsigned long long wait_limit_ns;
};

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

// Whole warp: the wait's answer, the same for all lanes.
__device__ __forceinline__ bool lin_wait(uint32_t bar, uint32_t parity, const WaitCtl& w, int site)
{
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, w, site));
}

// ---------------------------------------------------------------------------
// Epilogue arithmetic on CH columns of one row per lane, c0 .. c0 + n - 1 of them there.
//
// Where rows cannot be read or written 16 bytes at a time (odd strides), a
// whole warp exchanges its 32 rows through its staging buffer, so that neighbouring lanes
// touch neighbouring elements; `stage` is that buffer, or NULL (each lane by itself).
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

// Rows row - lane .. of a matrix with stride ld (base at column c0), one per lane of a
// converged warp; lanes with `valid` have a row.
template <int TYPE, int CH>
__device__ __forceinline__ void load_rows(float (&v)[CH], const uint16_t* base, long long ld, long long row, int n,
                                          bool vec, bool valid, uint32_t* stage)
{
    if (stage == nullptr || vec) {
        if (valid) load_row<TYPE, CH>(v, base + row * ld, n, vec);
    } else if constexpr (CH == 16) {
        const int lane = threadIdx.x & 31;
        const int rows = __popc(__ballot_sync(0xffffffffu, valid));   // the first lanes'
        const int r0 = lane >> 4, c = lane & 15;
        const long long first = row - lane;
        uint16_t* st = reinterpret_cast<uint16_t*>(stage);
#pragma unroll 4
        for (int i = 0; i < 32; i += 2) {
            const int r = i + r0;
            if (r < rows && c < n) st[r * (2 * kStagePitch) + c] = base[(first + r) * ld + c];
        }
        __syncwarp();
        load_row<TYPE, CH>(v, st + lane * (2 * kStagePitch), valid ? n : 0, false);
        __syncwarp();
    }
}

template <int TYPE, int CH>
__device__ __forceinline__ void store_rows16(uint16_t* base, long long ld, long long row, const float (&v)[CH], int n,
                                             bool vec, bool valid, uint32_t* stage)
{
    uint32_t w[CH / 2];
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) w[i] = pack2<TYPE>(v[2 * i], v[2 * i + 1]);
    if (vec && n == CH) {
        if (valid) {
            uint4* p = reinterpret_cast<uint4*>(base + row * ld);
#pragma unroll
            for (int i = 0; i < CH / 8; ++i) p[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
    } else if (CH != 16 || stage == nullptr || vec) {
        if (valid) {
            uint16_t* p = base + row * ld;
#pragma unroll
            for (int i = 0; i < CH; ++i)
                if (i < n) p[i] = static_cast<uint16_t>(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
        }
    } else if constexpr (CH == 16) {
        const int lane = threadIdx.x & 31;
        const int rows = __popc(__ballot_sync(0xffffffffu, valid));
        const int r0 = lane >> 4, c = lane & 15;
        const long long first = row - lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) stage[lane * kStagePitch + i] = w[i];
        __syncwarp();
        const uint16_t* st = reinterpret_cast<const uint16_t*>(stage);
#pragma unroll 4
        for (int i = 0; i < 32; i += 2) {
            const int r = i + r0;
            if (r < rows && c < n) base[(first + r) * ld + c] = st[r * (2 * kStagePitch) + c];
        }
        __syncwarp();
    }
}

template <int CH>
__device__ __forceinline__ void store_rows32(float* base, long long ld, long long row, const float (&v)[CH], int n,
                                             bool vec, bool accumulate, bool valid, uint32_t* stage)
{
    if (vec && n == CH) {
        if (valid) {
            float* p = base + row * ld;
#pragma unroll
            for (int i = 0; i < CH; i += 4) {
                float4 t = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                if (accumulate) {
                    const float4 w = *reinterpret_cast<const float4*>(p + i);
                    t = make_float4(t.x + w.x, t.y + w.y, t.z + w.z, t.w + w.w);
                }
                *reinterpret_cast<float4*>(p + i) = t;
            }
        }
    } else if (stage == nullptr || vec) {
        if (valid) {
            float* p = base + row * ld;
#pragma unroll
            for (int i = 0; i < CH; ++i)
                if (i < n) p[i] = accumulate ? p[i] + v[i] : v[i];
        }
    } else {
        const int lane = threadIdx.x & 31;
        const int rows = __popc(__ballot_sync(0xffffffffu, valid));
        const int r0 = lane >> 3, c = lane & 7;
        const long long first = row - lane;
#pragma unroll
        for (int h = 0; h < CH; h += 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) stage[lane * kStagePitch + i] = __float_as_uint(v[h + i]);
            __syncwarp();
#pragma unroll 4
            for (int i = 0; i < 32; i += 4) {
                const int r = i + r0;
                if (r < rows && h + c < n) {
                    float* p = base + (first + r) * ld + h + c;
                    const float t = __uint_as_float(stage[r * kStagePitch + c]);
                    *p = accumulate ? *p + t : t;
                }
            }
            __syncwarp();
        }
    }
}

template <int ACT, int CH>
__device__ __forceinline__ void act_all(float (&v)[CH])
{
#pragma unroll
    for (int i = 0; i < CH; ++i) v[i] = act_value<ACT>(v[i]);
}
template <int CH>
__device__ __forceinline__ void act_switch(float (&v)[CH], int act)
{
    if (act == kActSilu) act_all<kActSilu>(v);
    else if (act == kActGeluTanh) act_all<kActGeluTanh>(v);
    else if (act == kActGelu) act_all<kActGelu>(v);
    else if (act == kActRelu) act_all<kActRelu>(v);
}

// a (and b, gated: u) hold the sums of `row`, columns c0 .. c0 + n - 1 of source `src`.
// With `stage`, all lanes of a converged warp hold consecutive rows.
template <int TYPE, int MODE, int CH>
__device__ __forceinline__ void finish_rows(const LinearParams& p, float (&a)[CH], float (&b)[CH], int src, long long row,
                                            int c0, int n, bool valid, uint32_t* stage)
{
    if constexpr (MODE == kModeLinear || MODE == kModeGated) {
        if (p.bias[0] != nullptr) {
            float t[CH];
            load_row<TYPE, CH>(t, p.bias[0] + c0, n, p.vec_bias);
#pragma unroll
            for (int i = 0; i < CH; ++i) a[i] += t[i];
        }
        if (MODE == kModeGated && p.bias[1] != nullptr) {
            float t[CH];
            load_row<TYPE, CH>(t, p.bias[1] + c0, n, p.vec_bias);
#pragma unroll
            for (int i = 0; i < CH; ++i) b[i] += t[i];
        }
        if (p.keep[0] != nullptr) {
            store_rows16<TYPE, CH>(p.keep[0] + c0, p.ldk, row, a, n, p.vec_keep, valid, stage);
            if (MODE == kModeGated) store_rows16<TYPE, CH>(p.keep[1] + c0, p.ldk, row, b, n, p.vec_keep, valid, stage);
        }
        act_switch<CH>(a, p.act);
        if constexpr (MODE == kModeGated) {
#pragma unroll
            for (int i = 0; i < CH; ++i) a[i] *= b[i];
        }
        if (MODE == kModeLinear && p.residual != nullptr) {
            float t[CH] = {};
            load_rows<TYPE, CH>(t, p.residual + c0, p.ldr, row, n, p.vec_res, valid, stage);
#pragma unroll
            for (int i = 0; i < CH; ++i) a[i] += t[i];
        }
        store_rows16<TYPE, CH>(static_cast<uint16_t*>(p.out[0]) + c0, p.ldo, row, a, n, p.vec_out, valid, stage);
    } else if constexpr (MODE == kModeGradInput) {
        store_rows16<TYPE, CH>(static_cast<uint16_t*>(p.out[0]) + c0, p.ldo, row, a, n, p.vec_out, valid, stage);
    } else if (p.out_f32) {
        store_rows32<CH>(static_cast<float*>(p.out[src]) + c0, p.ldo, row, a, n, p.vec_out, p.accumulate != 0, valid, stage);
    } else {
        uint16_t* o = static_cast<uint16_t*>(p.out[src]) + c0;
        if (p.accumulate) {
            float t[CH] = {};
            load_rows<TYPE, CH>(t, o, p.ldo, row, n, p.vec_out, valid, stage);
#pragma unroll
            for (int i = 0; i < CH; ++i) a[i] += t[i];
        }
        store_rows16<TYPE, CH>(o, p.ldo, row, a, n, p.vec_out, valid, stage);
    }
}

template <int TYPE, int MODE, bool PAIR>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
                  const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
                  const __grid_constant__ LinearParams p)
{
    constexpr bool kGated = MODE == kModeGated;
    constexpr bool kAMn = MODE == kModeGradWeight;                              // A read along its rows
    constexpr bool kBMn = MODE == kModeGradWeight || MODE == kModeGradInput;   // B read along its columns
    constexpr int kTileRows = PAIR ? 256 : 128;
    const int S = p.stages;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t sA = smem_u32(smem);
    const uint32_t sB = sA + static_cast<uint32_t>(S * p.a_bytes);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kLinRingBytes);
    const uint32_t full0 = smem_u32(bars);                 // kLinMaxStages each: stage loaded, consumed
    const uint32_t empty0 = full0 + 8 * kLinMaxStages;
    const uint32_t tfull0 = empty0 + 8 * kLinMaxStages;    // 2 each: accumulator ready, drained
    const uint32_t tempty0 = tfull0 + 16;
    const uint32_t drain_bar = tempty0 + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kLinMaxStages + 5);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    static_assert((2 * kLinMaxStages + 5) * 8 + 8 <= kLinBarBytes, "barrier area too small");

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = PAIR || p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const bool leader = !PAIR || rank == 0;   // issues the MMAs

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
        prefetch_tmap(&tmA0);
        prefetch_tmap(&tmB0);
    }
    __syncwarp();
    if (warp == 1) {
        if constexpr (PAIR) {
            tmem_alloc_pair(smem_u32(tmem_slot), 2 * kLinAccCols);
            tmem_relinquish_alloc_permit_pair();
        } else {
            tmem_alloc(smem_u32(tmem_slot), 2 * kLinAccCols);
            tmem_relinquish_alloc_permit();
        }
    }
    tc_fence_before_sync();
    if constexpr (PAIR) cluster_sync();
    else __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    // global memory is read and written only once the kernel before this one in the stream has completed
    griddep_wait();
    griddep_launch_dependents();
    const WaitCtl wc{abort_flag, p.status, p.wait_limit_ns};
    uint32_t never = 0u;
    const WaitCtl wc_drain{&never, p.status, p.wait_limit_ns};

    // This CTA's (or pair's) tiles: unit, unit + units, ...; k-blocks [kb_begin, kb_end) of each.
    const int share = PAIR ? 2 : p.split;
    const int unit = static_cast<int>(blockIdx.x) / share;
    const int units = static_cast<int>(gridDim.x) / share;
    const int kb_all = p.kbs * p.k_sources;
    const int kb_begin = PAIR ? 0 : static_cast<int>(static_cast<long long>(rank) * kb_all / p.split);
    const int kb_end = PAIR ? kb_all : static_cast<int>(static_cast<long long>(rank + 1) * kb_all / p.split);

    if (warp == 0) {
        // ------------------------------------------------------------------
        // loads: this CTA's rows of A and of B
        // ------------------------------------------------------------------
        const uint32_t lead_full0 = PAIR ? mapa_shared(full0, 0) : full0;
        auto load = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
            if constexpr (PAIR) tma_load_2d_pair(dst, map, bar, x, y);
            else tma_load_2d(dst, map, bar, x, y);
        };
        const int b_rows = PAIR ? p.bn / 2 : p.bn;   // rows of B (columns of the tile) staged by this CTA
        const uint32_t tx = static_cast<uint32_t>(p.a_bytes + p.b_bytes) * (PAIR ? 2u : 1u);
        int stage = 0;
        uint32_t phase = 0;
        long long issued = 0;
        bool ok = true;
        for (int tile = unit; ok && tile < p.num_tiles; tile += units) {
            int pm, pn;
            tile_coord(tile, p.num_m, p.num_n, p.group_m, &pm, &pn);
            const int row_src = MODE == kModeGradWeight && pm >= p.num_m1 ? 1 : 0;
            const int m0 = (pm - row_src * p.num_m1) * kTileRows + (PAIR ? rank * 128 : 0);
            const int n0 = pn * p.wcols;
            for (int kb = kb_begin; kb < kb_end; ++kb) {
                ok = lin_wait(empty0 + 8 * stage, phase ^ 1u, wc, kSiteLinEmpty);
                if (!ok) break;
                if (lin_elect()) {
                    if (leader) mbar_arrive_expect_tx(full0 + 8 * stage, tx);
                    const uint32_t bar = lead_full0 + 8 * stage;
                    const uint32_t a_dst = sA + static_cast<uint32_t>(stage * p.a_bytes);
                    const uint32_t b_dst = sB + static_cast<uint32_t>(stage * p.b_bytes);
                    const int k_src = MODE == kModeGradInput && kb >= p.kbs ? 1 : 0;
                    const int k0 = (kb - k_src * p.kbs) * kLinBK;
                    const CUtensorMap* ma = (MODE == kModeGradWeight ? row_src : k_src) != 0 ? &tmA1 : &tmA0;
                    if constexpr (kAMn) {
                        load(a_dst, ma, bar, m0, k0);
                        load(a_dst + 8192, ma, bar, m0 + 64, k0);
                    } else {
                        load(a_dst, ma, bar, k0, m0);
                    }
                    if constexpr (kGated) {
                        if constexpr (PAIR) {
                            load(b_dst, rank != 0 ? &tmB1 : &tmB0, bar, k0, n0);
                        } else {
                            load(b_dst, &tmB0, bar, k0, n0);
                            load(b_dst + static_cast<uint32_t>(p.b_bytes / 2), &tmB1, bar, k0, n0);
                        }
                    } else {
                        const int nb = n0 + (PAIR ? rank * b_rows : 0);
                        if constexpr (kBMn) {
                            const CUtensorMap* mb = k_src != 0 ? &tmB1 : &tmB0;
                            for (int i = 0; i < b_rows / 64; ++i)
                                load(b_dst + static_cast<uint32_t>(i) * 8192u, mb, bar, nb + 64 * i, k0);
                        } else {
                            load(b_dst, &tmB0, bar, k0, nb);
                        }
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
        if (!ok && leader) {
            // abort: the loads already issued land (waits with a limit) before the CTA can exit
            const int pending = static_cast<int>(issued < S ? issued : S);
            for (int j = 1; j <= pending; ++j) {
                const int s = (stage - j + S) % S;
                mbar_wait(full0 + 8 * s, stage - j < 0 ? phase ^ 1u : phase, wc_drain, kSiteLinDrain);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------------
        // MMAs
        // ------------------------------------------------------------------
        if (leader) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            bool issued_any = false;
            int it = 0;
            const int seg_kb = MODE == kModeGradWeight ? p.seg_kb : kb_end - kb_begin;
            for (int tile = unit; ok && tile < p.num_tiles; tile += units) {
                for (int seg = kb_begin; ok && seg < kb_end; seg += seg_kb, ++it) {
                    const int acc = it & 1;
                    const uint32_t aph = static_cast<uint32_t>(it >> 1) & 1u;
                    ok = PAIR ? mbar_wait_cluster(tempty0 + 8 * acc, aph ^ 1u, wc, kSiteLinTmemEmpty)
                              : mbar_wait(tempty0 + 8 * acc, aph ^ 1u, wc, kSiteLinTmemEmpty);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint32_t d = tmem_base + static_cast<uint32_t>(acc * kLinAccCols);
                    const int seg_end = kb_end - seg < seg_kb ? kb_end : seg + seg_kb;
                    for (int kb = seg; kb < seg_end; ++kb) {
                        ok = lin_wait(full0 + 8 * stage, phase, wc, kSiteLinFull);
                        if (!ok) break;
                        tc_fence_after_sync();
                        const uint32_t a = sA + static_cast<uint32_t>(stage * p.a_bytes);
                        const uint32_t b = sB + static_cast<uint32_t>(stage * p.b_bytes);
                        if (lin_elect()) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                // read along k: 32 bytes of every 128-byte row; read along rows
                                // (columns): 16 k rows of 128 bytes, 64-element blocks 8 KB apart
                                const uint64_t ad = kAMn ? smem_desc_sw128(a + kk * 2048, 8192, 1024)
                                                         : smem_desc_sw128(a + kk * 32, 16, 1024);
                                const uint64_t bd = kBMn ? smem_desc_sw128(b + kk * 2048, 8192, 1024)
                                                         : smem_desc_sw128(b + kk * 32, 16, 1024);
                                const uint32_t more = kb != seg || kk != 0 ? 1u : 0u;
                                if constexpr (PAIR) mma_f16_pair(d, ad, bd, p.idesc, more);
                                else mma_f16(d, ad, bd, p.idesc, more);
                            }
                            if constexpr (PAIR) mma_commit_pair_multicast(empty0 + 8 * stage, 0x3);
                            else mma_commit(empty0 + 8 * stage);
                        }
                        __syncwarp();
                        issued_any = true;
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
            if (!ok && issued_any) {
                // abort: every MMA issued so far finishes before TMEM is freed
                if (lin_elect()) {
                    if constexpr (PAIR) mma_commit_pair_multicast(drain_bar, 0x1);
                    else mma_commit(drain_bar);
                }
                __syncwarp();
                mbar_wait(drain_bar, 0u, wc_drain, kSiteLinDrain);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------------
        // epilogue: 32 rows a warp (the TMEM lanes it may read), every other kCh columns
        // ------------------------------------------------------------------
        const int quarter = warp & 3;
        const int half = (warp - 2) >> 2;
        const uint32_t lead_tempty0 = PAIR ? mapa_shared(tempty0, 0) : tempty0;
        uint32_t* stage = p.stage_out
                              ? reinterpret_cast<uint32_t*>(smem + kLinRingBytes - kStageBytes) + (warp - 2) * 32 * kStagePitch
                              : nullptr;
        auto hand_back = [&](int acc) {   // this warp has read its part of the accumulator
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) mbar_arrive_remote(lead_tempty0 + 8 * acc);
                else mbar_arrive(tempty0 + 8 * acc);
            }
        };
        bool ok = true;
        int it = 0;
        for (int tile = unit; ok && tile < p.num_tiles; tile += units) {
            int pm, pn;
            tile_coord(tile, p.num_m, p.num_n, p.group_m, &pm, &pn);
            const int src = MODE == kModeGradWeight && pm >= p.num_m1 ? 1 : 0;
            const int m0 = (pm - src * p.num_m1) * kTileRows + (PAIR ? rank * 128 : 0) + quarter * 32;
            const int n0 = pn * p.wcols;
            const int row = m0 + lane;
            const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
            const bool any = m0 < p.rows;   // rows of this warp's to store
            const bool valid = row < p.rows;
            const int left = p.cols - n0;
            const int width = left < p.wcols ? left : p.wcols;
            // split k: partials stay in this CTA's shared memory, over the ring (whose stages the
            // MMAs have finished reading), bn + 4 floats a row
            float* part = reinterpret_cast<float*>(smem) + (quarter * 32 + lane) * (p.bn + 4);
            if constexpr (MODE == kModeGradWeight) {
                float sum[8][kCh];
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int i = 0; i < kCh; ++i) sum[j][i] = 0.f;
                for (int seg = kb_begin; seg < kb_end; seg += p.seg_kb, ++it) {
                    const int acc = it & 1;
                    ok = lin_wait(tfull0 + 8 * acc, static_cast<uint32_t>(it >> 1) & 1u, wc, kSiteLinTmemFull);
                    if (!ok) break;
                    tc_fence_after_sync();
                    if (any) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int c = (2 * j + half) * kCh;
                            if (c < p.bn) {
                                uint32_t r[kCh];
                                lin_tmem_ld16(t_row + acc * kLinAccCols + c, r);
                                tmem_ld_wait();
#pragma unroll
                                for (int i = 0; i < kCh; ++i) sum[j][i] += __uint_as_float(r[i]);
                            }
                        }
                    }
                    hand_back(acc);
                }
                if (!ok) break;
                if (any) {
                    if (p.split > 1) fence_proxy_async_smem();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int c = (2 * j + half) * kCh;
                        if (p.split > 1) {
                            if (c < p.bn && valid) {
#pragma unroll
                                for (int i = 0; i < kCh; i += 4)
                                    *reinterpret_cast<float4*>(part + c + i) =
                                        make_float4(sum[j][i], sum[j][i + 1], sum[j][i + 2], sum[j][i + 3]);
                            }
                        } else if (c < width) {
                            finish_rows<TYPE, MODE, kCh>(p, sum[j], sum[j], src, row, n0 + c,
                                                         width - c < kCh ? width - c : kCh, valid, stage);
                        }
                    }
                }
            } else {
                const int acc = it & 1;
                ok = lin_wait(tfull0 + 8 * acc, static_cast<uint32_t>(it >> 1) & 1u, wc, kSiteLinTmemFull);
                if (!ok) break;
                ++it;
                tc_fence_after_sync();
                const uint32_t t_acc = t_row + static_cast<uint32_t>(acc * kLinAccCols);
                if (any && p.split == 1) {
#pragma unroll 1
                    for (int c = half * kCh; c < width; c += 2 * kCh) {
                        uint32_t ra[kCh], rb[kCh];
                        lin_tmem_ld16(t_acc + c, ra);
                        if constexpr (kGated) lin_tmem_ld16(t_acc + p.wcols + c, rb);
                        tmem_ld_wait();
                        float a[kCh], b[kCh];
#pragma unroll
                        for (int i = 0; i < kCh; ++i) {
                            a[i] = __uint_as_float(ra[i]);
                            b[i] = kGated ? __uint_as_float(rb[i]) : 0.f;
                        }
                        finish_rows<TYPE, MODE, kCh>(p, a, b, src, row, n0 + c, width - c < kCh ? width - c : kCh, valid,
                                                     stage);
                    }
                } else if (any) {
                    fence_proxy_async_smem();
#pragma unroll 1
                    for (int c = half * kCh; c < p.bn; c += 2 * kCh) {
                        uint32_t r[kCh];
                        lin_tmem_ld16(t_acc + c, r);
                        tmem_ld_wait();
                        if (valid) {
#pragma unroll
                            for (int i = 0; i < kCh; i += 4)
                                *reinterpret_cast<uint4*>(part + c + i) = make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
                        }
                    }
                }
                hand_back(acc);
            }
        }
        __syncwarp();
    }

    if constexpr (!PAIR) {
        if (p.split > 1) {
            // One tile per cluster.  Barrier 1: every CTA's partial is in its shared memory.
            cluster_sync();
            if (warp >= 2) {
                // This CTA's columns of the tile (a multiple of 8, so that 16-byte accesses stay
                // aligned), 8 columns of a row per thread and turn, neighbouring threads on
                // neighbouring rows.
                constexpr int kW = 8;
                int pm, pn;
                tile_coord(unit, p.num_m, p.num_n, p.group_m, &pm, &pn);
                const int src = MODE == kModeGradWeight && pm >= p.num_m1 ? 1 : 0;
                const int r0 = (pm - src * p.num_m1) * 128;
                const int n0 = pn * p.wcols;
                const int left = p.cols - n0;
                const int width = left < p.wcols ? left : p.wcols;
                const int rows = p.rows - r0 < 128 ? p.rows - r0 : 128;
                const int slice = ((width + p.split - 1) / p.split + kW - 1) / kW * kW;
                const int c_begin = rank * slice;
                const int c_end = c_begin + slice < width ? c_begin + slice : width;
                const int items = c_begin < c_end ? (c_end - c_begin + kW - 1) / kW * rows : 0;
                for (int e = static_cast<int>(threadIdx.x) - 64; e < items; e += 32 * kLinEpiWarps) {
                    const int lrow = e % rows;
                    const int c = c_begin + e / rows * kW;
                    const uint32_t base = sA + static_cast<uint32_t>((lrow * (p.bn + 4) + c) * 4);
                    float a[kW] = {}, b[kW] = {};
                    // four partials' loads in flight; summed in rank order
                    for (int q0 = 0; q0 < p.split; q0 += 4) {
                        float4 v[4][2], w[4][2];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if (q0 + q < p.split) {
                                const uint32_t peer = mapa_shared(base, static_cast<uint32_t>(q0 + q));
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    v[q][i] = ld_shared_cluster_v4(peer + 16u * i);
                                    if constexpr (kGated) w[q][i] = ld_shared_cluster_v4(peer + static_cast<uint32_t>(p.wcols) * 4u + 16u * i);
                                }
                            }
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if (q0 + q < p.split) {
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    a[4 * i] += v[q][i].x;
                                    a[4 * i + 1] += v[q][i].y;
                                    a[4 * i + 2] += v[q][i].z;
                                    a[4 * i + 3] += v[q][i].w;
                                    if constexpr (kGated) {
                                        b[4 * i] += w[q][i].x;
                                        b[4 * i + 1] += w[q][i].y;
                                        b[4 * i + 2] += w[q][i].z;
                                        b[4 * i + 3] += w[q][i].w;
                                    }
                                }
                            }
                        }
                    }
                    finish_rows<TYPE, MODE, kW>(p, a, b, src, r0 + lrow, n0 + c, c_end - c < kW ? c_end - c : kW, true,
                                                nullptr);
                }
            }
            // Barrier 2: no CTA leaves while a peer may still read its shared memory.
            cluster_sync();
        }
    }
    tc_fence_before_sync();
    if constexpr (PAIR) cluster_sync();
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        if constexpr (PAIR) tmem_dealloc_pair(tmem_base, 2 * kLinAccCols);
        else tmem_dealloc(tmem_base, 2 * kLinAccCols);
    }
}

// 2-D tensor map, 128-byte swizzle: `inner` contiguous elements in `outer` lines.
inline bool lin_map(CUtensorMap* map, int type, const void* base, long long inner, long long outer, long long ld,
                    int box_inner, int box_outer, char* msg, size_t msg_len)
{
    TmapEncodeFn enc = tmap_encoder();
    if (enc == nullptr) {
        snprintf(msg, msg_len, "cuTensorMapEncodeTiled is not available from the driver");
        return false;
    }
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2u};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_outer)};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, type == kTypeBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                           2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        snprintf(msg, msg_len, "cuTensorMapEncodeTiled failed (%d) for %lld x %lld, stride %lld, box %d x %d",
                 static_cast<int>(r), inner, outer, ld, box_inner, box_outer);
        return false;
    }
    return true;
}

inline bool lin_aligned16(const void* p, long long ld_bytes)
{
    return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld_bytes)) & 15u) == 0;
}

template <int TYPE, int MODE, bool PAIR>
int launch_linear_instance(const LinearLaunch& g, cudaStream_t stream, char* msg, size_t msg_len)
{
    constexpr bool kGated = MODE == kModeGated;
    constexpr bool kAMn = MODE == kModeGradWeight;
    constexpr bool kBMn = MODE == kModeGradWeight || MODE == kModeGradInput;
    constexpr int kTileRows = PAIR ? 256 : 128;
    const int unit_cols = kGated ? 32 : kBMn ? 64 : 16;
    const int bn_unit = PAIR && kBMn ? 128 : PAIR ? 32 : unit_cols;
    if (g.bn < bn_unit || g.bn > 256 || g.bn % bn_unit != 0) {
        snprintf(msg, msg_len, "linear product: bad tile width %d", g.bn);
        return 1;
    }
    LinearParams p = {};
    p.rows = g.rows;
    p.cols = g.cols;
    p.kbs = (g.k + kLinBK - 1) / kLinBK;
    p.k_sources = MODE == kModeGradInput ? g.sources : 1;
    p.num_m1 = (g.rows + kTileRows - 1) / kTileRows;
    p.num_m = p.num_m1 * (MODE == kModeGradWeight ? g.sources : 1);
    p.bn = g.bn;
    p.wcols = kGated ? g.bn / 2 : g.bn;
    p.num_n = (g.cols + p.wcols - 1) / p.wcols;
    p.num_tiles = p.num_m * p.num_n;
    p.group_m = g.group_m;
    p.a_rows = PAIR || kAMn || g.rows >= 128 ? 128 : (g.rows + 7) / 8 * 8;
    p.a_bytes = p.a_rows * 128;
    const int b_rows = PAIR ? g.bn / 2 : g.bn;
    p.b_bytes = b_rows * 128;
    const int ob = g.out_f32 ? 4 : 2;
    p.vec_out = lin_aligned16(g.out[0], g.ldo * ob) && lin_aligned16(g.out[1], 0);
    p.vec_res = lin_aligned16(g.residual, g.ldr * 2);
    p.vec_keep = lin_aligned16(g.keep[0], g.ldk * 2) && lin_aligned16(g.keep[1], 0);
    p.vec_bias = lin_aligned16(g.bias[0], 0) && lin_aligned16(g.bias[1], 0);
    p.stage_out = !(p.vec_out && (p.vec_res || g.residual == nullptr) && (p.vec_keep || g.keep[0] == nullptr));
    // (with few rows the MMA reads up to 16 KB from the start of the last stage's A, into B's stages)
    p.stages = (kLinRingBytes - (p.stage_out ? kStageBytes : 0)) / (p.a_bytes + p.b_bytes);
    if (p.stages > kLinMaxStages) p.stages = kLinMaxStages;
    p.split = PAIR || g.split < 2 ? 1 : g.split;
    while (p.split > p.kbs * p.k_sources) p.split /= 2;   // every CTA of a cluster has a k-block
    p.seg_kb = g.out_f32 ? kSegmentKb : p.kbs * p.k_sources;
    p.idesc = idesc_f16(TYPE == kTypeBF16, kAMn, kBMn, kTileRows, g.bn);
    for (int i = 0; i < 2; ++i) {
        p.out[i] = g.out[i];
        p.bias[i] = static_cast<const uint16_t*>(g.bias[i]);
        p.keep[i] = static_cast<uint16_t*>(g.keep[i]);
    }
    p.ldo = g.ldo;
    p.residual = static_cast<const uint16_t*>(g.residual);
    p.ldr = g.ldr;
    p.ldk = g.ldk;
    p.act = g.act;
    p.out_f32 = g.out_f32;
    p.accumulate = g.accumulate;
    p.status = g.status;
    p.wait_limit_ns = g.wait_limit_ns;

    CUtensorMap tmA[2], tmB[2];
    const int b_box = kBMn ? 64 : kGated ? g.bn / 2 : b_rows;
    const int srcs = MODE == kModeGradInput || MODE == kModeGradWeight ? g.sources : 1;
    for (int s = 0; s < 2; ++s) {
        const void* a = s < srcs ? g.A[s] : g.A[0];
        const bool ok_a = kAMn ? lin_map(&tmA[s], g.type, a, g.rows, g.k, g.lda, 64, kLinBK, msg, msg_len)
                               : lin_map(&tmA[s], g.type, a, g.k, g.rows, g.lda, kLinBK, p.a_rows, msg, msg_len);
        const void* b = s == 0 || g.B[1] == nullptr ? g.B[0] : g.B[1];
        const bool ok_b = ok_a && (kBMn ? lin_map(&tmB[s], g.type, b, g.cols, g.k, g.ldb, 64, kLinBK, msg, msg_len)
                                        : lin_map(&tmB[s], g.type, b, g.k, g.cols, g.ldb, kLinBK, b_box, msg, msg_len));
        if (!ok_b) return 1;
    }

    auto kern = linear_kernel<TYPE, MODE, PAIR>;
    static SmemOptIn smem_opt;
    cudaError_t e = smem_opt.ensure(reinterpret_cast<const void*>(kern), kLinSmemBytes);
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        return 1;
    }
    const int share = PAIR ? 2 : p.split;
    long long units = p.num_tiles;
    if (p.split == 1) {
        // every unit gets the same number of tiles (the last wave is not left partial)
        const long long most = PAIR ? g.num_sms / 2 : g.num_sms;
        const long long cap = most > 0 ? most : 1;
        const long long per = (units + cap - 1) / cap;
        units = (units + per - 1) / per;
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
    cfg.gridDim = dim3(static_cast<unsigned>(units * share), 1, 1);
    cfg.blockDim = dim3(kLinThreads, 1, 1);
    cfg.dynamicSmemBytes = kLinSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = static_cast<unsigned>(attrs);
    e = cudaLaunchKernelEx(&cfg, kern, tmA[0], tmA[1], tmB[0], tmB[1], p);
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
    case kModeGradInput:
        return g.pair ? launch_linear_instance<TYPE, kModeGradInput, true>(g, stream, msg, msg_len)
                      : launch_linear_instance<TYPE, kModeGradInput, false>(g, stream, msg, msg_len);
    case kModeGradWeight:
        return g.pair ? launch_linear_instance<TYPE, kModeGradWeight, true>(g, stream, msg, msg_len)
                      : launch_linear_instance<TYPE, kModeGradWeight, false>(g, stream, msg, msg_len);
    default:
        snprintf(msg, msg_len, "unknown linear mode %d", g.mode);
        return 1;
    }
}

}  // namespace
}  // namespace bsk
