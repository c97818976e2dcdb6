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
// side, so they share the keys) and walks the keys in tiles of kTile positions:
//   S = Q K^T   tcgen05.mma, Q from TMEM, K from shared memory, S in TMEM (two buffers)
//   P = 2^(..)  four or eight warps, S from TMEM to registers and P back, 16 bits, over S
//   O += P V    tcgen05.mma, P from TMEM, V from shared memory, O in TMEM
// The MMAs of S for tile j+1 and of PV for tile j-1 run while the warps work on
// tile j.  Q lies in TMEM, so that shared memory holds nothing but keys and values
// on their way and an MMA reads one operand from it (with Q there too, head_dim 256
// took 1040 us where this took 927).
//
// Bound, long chunks: a tile is 1024 clocks of MMAs (head_dim 128 and 256) and takes about
// 1850.  Its 64 KB of keys and values come from the TMA unit in 1150 (57 bytes a clock at
// best); the rest is one set of softmax warps that takes tile after tile (load S,
// exchange the maximum, exponentials, store P).  2048 tokens over 30720 (16 query heads,
// 4 KV heads of 256, BF16): 856 to 883 us by box, 1200 to 1240 TFLOP/s, 0.63 to 0.65 of
// the tensor cores' measured rate.  head_dim 64: the same per tile, and the start and end
// of a CTA, some 6 us each over 3.5 waves of CTAs (a windowed chunk of 4097 tokens, 32
// heads, 73 us, of which the exponentials alone would be 25).  Few rows: HBM and a CTA's
// start and end (8 sequences decoded through a window of 4096, BF16: 31 us, 4.3 TB/s).
#include <cmath>
#include <cstdio>
#include <limits>

#include "bsk_internal.h"
#include "kv_attention.cuh"
#include "kv_internal.h"
#include "ptx.cuh"

namespace bsk {
using namespace kv;
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

// Cache rows of one KV head, a multiple of 8 of them, from the 4-D view below.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int y, int z, int w)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem desc], A 128 x 16 16-bit values, two values per column.
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
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
// Each lane reads 16 consecutive columns of its TMEM lane.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One lane of a converged warp, always the same.  A branch on this (and not on
// lane == 0) tells the compiler that a single thread issues the TMA or MMA
// instruction in it; otherwise it takes the active lanes one after the other, at
// 80 to 100 clocks an instruction.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

__device__ __forceinline__ void named_barrier(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// mbar_wait for waits that come several times a microsecond: it looks at the
// clock and the abort flag only after many tries (each try suspends the warp for
// a while by itself).
__device__ __forceinline__ bool wait_long(uint32_t bar, uint32_t parity, const WaitCtl& w, int site)
{
    for (int i = 0; i < 256; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait(bar, parity, w, site);
}

// ---------------------------------------------------------------------------
// Geometry
// ---------------------------------------------------------------------------
constexpr int kRows = 128;        // query rows per CTA (the M of the MMAs)
// Warps 12 .. convert E4M3 codes, four of them keys and four values.  32 sequences of
// up to 4000 tokens, 16 rows of head_dim 256: 105 us with four warps for both in turn,
// 89 with eight, 77 with four for each (78 now).
constexpr int kConvertWarps = 4;
constexpr int kSlots = 8;         // tiles whose cache rows, masks and scales are kept

// Warps 0..3: keys' loads, MMAs, values' loads, look-ups in the block table.
enum AttnWarp : int { kWarpK = 0, kWarpMma = 1, kWarpV = 2, kWarpPages = 3 };
// How a tile is loaded: its rows lie side by side (one box), its boxes are each
// whole or without a key, or some box is neither.
enum LoadKind : int { kLoadTile = 0, kLoadBoxes = 1, kLoadRows = 2 };
enum AttnSite : int {
    kSiteKvEmpty = 0x30, kSiteKvFull, kSiteKvQ, kSiteKvScores, kSiteKvWeights, kSiteKvOutput, kSiteKvDrain,
    kSiteKvRaw, kSiteKvMeta
};

template <bool E4M3, int HD>
struct Geo {
    static constexpr int kBlocks = HD / 64;                    // 64-element (128-byte) blocks of a row
    // CTAs per SM.  A CTA alternates between waiting for its own scores and working on
    // them; a second one fills the gaps, and one's start and end.  With HD = 64 two fit
    // TMEM with 64-position tiles: a windowed chunk of 4097 tokens took 76 us with two
    // (72 now), 110 with one of 128-position tiles.  With HD = 128 a second one leaves room for one S
    // tile only and lost (325 against 276 us for four ragged chunks).
    static constexpr int kCtas = !E4M3 && HD == 64 ? 2 : 1;
    // Positions per tile, S tiles in TMEM.  TMEM's columns (512, or 256 for each of two
    // CTAs) hold the S tiles, Q (HD / 2 columns) and O (HD).
    static constexpr int kTile = HD == 256 || kCtas == 2 ? 64 : 128;
    static constexpr int kTmem = 512 / kCtas;
    // Softmax warps: four have a row per lane; eight, two lanes a row.
    static constexpr int kHalves = kCtas == 2 ? 1 : 2;
    static constexpr int kSoftmaxWarps = 4 * kHalves;          // warps 4 ..
    static constexpr int kCols = kTile / kHalves;              // S columns per softmax warp
    static constexpr int kColQ = 2 * kTile;               // TMEM columns of Q and O
    static constexpr int kColO = HD == 64 ? kColQ + 32 : kTmem - HD;
    static_assert(kColQ + HD / 2 <= kColO && kColO + HD <= kTmem, "TMEM columns of one CTA");
    // A stage: one tile's keys or values in 16 bits, [kTile / 8][kBlocks] swizzle atoms
    // of 8 rows x 128 bytes.  Keys are read as a K-major operand (8-row groups
    // kBlocks * 1024 bytes apart), values as an MN-major one (64-dimension blocks 1024
    // bytes apart, groups as before): one layout and one kind of load serves both.
    static constexpr int kStageBytes = kTile * HD * 2;
    static constexpr int kStages = E4M3 && HD != 64 ? 2 : 3;   // of keys, and of values
    static constexpr int kRawBytes = E4M3 ? kTile * HD : 0;    // a tile's codes, rows side by side
    static constexpr int kRawStages = E4M3 ? 2 : 0;
    static constexpr int kThreads = E4M3 ? 384 + 64 * kConvertWarps : 128 + 32 * kSoftmaxWarps;
    static constexpr int kBars = 4 * kStages + 4 * kRawStages + 2 * kSlots + 8;
    static constexpr int kScaleBytes = E4M3 ? kSlots * (kTile * 8 + 4) : 0;
    static constexpr int kMisc = kScaleBytes + kSlots * (kTile + 36) * 4 + kSlots * 16 + 2 * 2 * kRows * 4 + kRows * 4 + kBars * 8 + 16;
    static constexpr int kBytes = 1024 + 2 * kStages * kStageBytes + 2 * kRawStages * kRawBytes + kMisc;
    static_assert(kBytes <= 232448 / kCtas - (kCtas - 1) * 1024, "shared memory of one CTA");
};

// Tensor maps of the cache.  Gathers see it as [num_blocks * block_size] rows of
// heads * HD values.  Boxes are `box` rows of one head: of a BF16 cache as the stages
// want them ([rows / 8][heads * HD / 64][8][64]), of an E4M3 cache in lines of at
// most 128 codes, each swizzled: without
// swizzling the TMA unit writes 31 bytes a clock, with it 57.  Tile boxes are the
// same with a tile's rows.
struct KvMaps {
    CUtensorMap k_tile, v_tile, k_box, v_box, k_row, v_row;
};

// Of the positions k .. k + box - 1 (box a power of two), by a tile's mask: 0 none
// holds a key, 1 all do, 2 some.
__device__ __forceinline__ int box_state(const uint32_t* mask, int k, int box)
{
    const uint32_t bits = box >= 32 ? 0xffffffffu : (1u << box) - 1u;
    uint32_t all = bits, any = 0u;
    for (int w = k; w < k + box; w += 32) {
        const uint32_t m = (mask[w >> 5] >> (w & 31)) & bits;
        all &= m;
        any |= m;
    }
    return all == bits ? 1 : (any == 0u ? 0 : 2);
}

// Where 16-byte piece c of row r goes, of rows of N pieces one after the other: piece
// c ^ row_swizzle(r), so that 8 neighbouring rows' same pieces meet distinct banks.
template <int N>
__device__ __forceinline__ int row_swizzle(int r)
{
    return N >= 8 ? r & 7 : (r >> 1) & 3;
}

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
template <bool E4M3, int HD>
__global__ void __launch_bounds__(Geo<E4M3, HD>::kThreads, Geo<E4M3, HD>::kCtas)
    kv_attention_kernel(const __grid_constant__ KvMaps maps, const __grid_constant__ AttnParams p)
{
    using G = Geo<E4M3, HD>;
    constexpr int S = G::kStages;
    constexpr int RS = E4M3 ? G::kRawStages : 1;
    constexpr int NB = G::kBlocks;
    constexpr int kTile = G::kTile;
    constexpr int C = G::kCols;
    constexpr int H = G::kHalves;
    constexpr uint32_t kIdescS = idesc_f16(!E4M3, false, false, kRows, kTile);
    constexpr uint32_t kIdescO = idesc_f16(!E4M3, false, true, kRows, HD);

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* s_k = smem;                                            // [S] keys
    uint8_t* s_v = s_k + S * G::kStageBytes;                        // [S] values
    uint8_t* r_k = s_v + S * G::kStageBytes;                        // E4M3: [RS] keys' codes
    uint8_t* r_v = r_k + G::kRawStages * G::kRawBytes;              //       [RS] values' codes
    float* s_kf = reinterpret_cast<float*>(r_v + G::kRawStages * G::kRawBytes);   // E4M3: [kSlots][kTile] K scales
    uint32_t* s_vf = reinterpret_cast<uint32_t*>(s_kf + (E4M3 ? kSlots * kTile : 0));   //       V rows' FP16 factors, twice
    int* s_exp = reinterpret_cast<int*>(s_vf + (E4M3 ? kSlots * kTile : 0));    // [kSlots] V scales' E
    int* s_row = reinterpret_cast<int*>(s_exp + (E4M3 ? kSlots : 0));   // [kSlots][kTile] cache row of each position
    int* s_box = s_row + kSlots * kTile;                            // [kSlots][32] cache row of each box
    int* s_kind = s_box + kSlots * 32;                              // [kSlots][4] (first used) LoadKind of the tile
    uint32_t* s_mask = reinterpret_cast<uint32_t*>(s_kind + kSlots * 4);          // [kSlots][4] positions that hold a key
    float* s_max = reinterpret_cast<float*>(s_mask + kSlots * 4);   // [2][2][kRows]
    int* s_flag = reinterpret_cast<int*>(s_max + 4 * kRows);        // [kRows] rows to repair
    uint64_t* bars = reinterpret_cast<uint64_t*>(s_flag + kRows);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + G::kBars);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    volatile uint32_t* s_wide = tmem_slot + 2;              // E4M3: a V scale is out of range
    const uint32_t k_full0 = smem_u32(bars);                // S: a tile's keys are there
    const uint32_t k_empty0 = k_full0 + 8 * S;              // S: ... and read
    const uint32_t v_full0 = k_empty0 + 8 * S;
    const uint32_t v_empty0 = v_full0 + 8 * S;
    const uint32_t rk_full0 = v_empty0 + 8 * S;             // kRawStages: codes are there
    const uint32_t rk_empty0 = rk_full0 + 8 * G::kRawStages;
    const uint32_t rv_full0 = rk_empty0 + 8 * G::kRawStages;
    const uint32_t rv_empty0 = rv_full0 + 8 * G::kRawStages;
    const uint32_t m_full0 = rv_empty0 + 8 * G::kRawStages; // kSlots: a tile's rows, mask and scales
    const uint32_t m_empty0 = m_full0 + 8 * kSlots;
    const uint32_t q_full = m_empty0 + 8 * kSlots;          // Q in TMEM
    const uint32_t s_full0 = q_full + 8;                    // 2: scores ready
    const uint32_t p_full0 = s_full0 + 16;                  // 2: weights ready
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
    const int row0 = tile * kRows;
    const int rows = min(kRows, n * p.group - row0);
    if (rows <= 0) return;
    const int pos0 = len - n;                              // position of the sequence's first new token
    const int pmin = pos0 + row0 / p.group, pmax = pos0 + (row0 + rows - 1) / p.group;
    Keys<kTile> keys;
    keys.kv_end = max(pmax + 1, 0);
    keys.lo = window_start(pmin, p.window);
    keys.sink_end = min(p.sinks, keys.lo);
    keys.lo_tile = keys.lo / kTile;
    keys.sink_tiles = min((keys.sink_end + kTile - 1) / kTile, keys.lo_tile);
    {
        const int total = keys.kv_end > 0 ? keys.sink_tiles + (keys.kv_end + kTile - 1) / kTile - keys.lo_tile : 0;
        const int each = p.segment_keys / kTile;
        keys.begin = static_cast<int>(min(static_cast<long long>(total), static_cast<long long>(each) * seg));
        keys.end = seg + 1 == p.segments ? total : min(total, keys.begin + each);
    }
    const int32_t* table = p.b.block_tables + static_cast<long long>(seq) * p.b.max_blocks;
    const int nt = keys.end - keys.begin;
    if (nt <= 0) {
        // nothing to see in this segment
        if (p.segments == 1) {
            for (int i = threadIdx.x; i < rows * (HD / 8); i += G::kThreads) {
                const int r = row0 + i / (HD / 8);
                uint16_t* o = p.out + (first + r / p.group) * p.out_stride +
                              (static_cast<long long>(kvh) * p.group + r % p.group) * HD + (i % (HD / 8)) * 8;
                *reinterpret_cast<uint4*>(o) = make_uint4(0, 0, 0, 0);
            }
        } else {
            for (int i = threadIdx.x; i < rows; i += G::kThreads) {
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
            mbar_init(k_full0 + 8 * s, E4M3 ? kConvertWarps : 1);
            mbar_init(k_empty0 + 8 * s, 1);
            mbar_init(v_full0 + 8 * s, E4M3 ? kConvertWarps : 1);
            mbar_init(v_empty0 + 8 * s, 1);
        }
        for (int s = 0; s < G::kRawStages; ++s) {
            mbar_init(rk_full0 + 8 * s, 1);
            mbar_init(rk_empty0 + 8 * s, kConvertWarps);
            mbar_init(rv_full0 + 8 * s, 1);
            mbar_init(rv_empty0 + 8 * s, kConvertWarps);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(m_full0 + 8 * s, 1);
            mbar_init(m_empty0 + 8 * s, G::kSoftmaxWarps + 1 + (E4M3 ? kConvertWarps : 0));
        }
        mbar_init(q_full, G::kSoftmaxWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full0 + 8 * i, 1);
            mbar_init(p_full0 + 8 * i, G::kSoftmaxWarps);
            mbar_init(o_done0 + 8 * i, 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0u;
        *s_wide = 0u;
        fence_mbar_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32(tmem_slot), G::kTmem);
        tmem_relinquish_alloc_permit();
    }
    if (warp >= 4 && warp < 8) s_flag[threadIdx.x - 128] = 0;
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const WaitCtl wc{abort_flag, p.b.status, p.wait_limit_ns};
    uint32_t never = 0u;
    const WaitCtl wc_drain{&never, p.b.status, p.wait_limit_ns};

    if (warp == kWarpK || warp == kWarpV) {
        // ------------------------------------------------------------------
        // Loads: one warp for the keys, one for the values.  `box` positions lie in
        // one page, side by side (box divides the page size), and come as one TMA box
        // when all of them hold a key.  Others are gathered four by four, a position
        // without a key from past the last row: zeros.  A box costs its warp about 57
        // clocks and 2.2 for each 128 bytes that the TMA unit writes (so 57 bytes a
        // clock at best); with two warps one's overhead hides behind the other's.
        // ------------------------------------------------------------------
        const bool is_k = warp == kWarpK;
        const CUtensorMap* tile_map = is_k ? &maps.k_tile : &maps.v_tile;
        const CUtensorMap* box_map = is_k ? &maps.k_box : &maps.v_box;
        const CUtensorMap* row_map = is_k ? &maps.k_row : &maps.v_row;
        constexpr int RING = E4M3 ? RS : S;
        constexpr int kBytes = E4M3 ? G::kRawBytes : G::kStageBytes;
        const uint32_t full0 = E4M3 ? (is_k ? rk_full0 : rv_full0) : (is_k ? k_full0 : v_full0);
        const uint32_t empty0 = E4M3 ? (is_k ? rk_empty0 : rv_empty0) : (is_k ? k_empty0 : v_empty0);
        const uint32_t dst0 = smem_u32(E4M3 ? (is_k ? r_k : r_v) : (is_k ? s_k : s_v));
        const int box = p.box, pad = max(box, 16);
        // the rows from `row` on, as positions k .. of a tile
        auto load_box = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar, int k, int row) {
            if constexpr (!E4M3 && HD > 64) {
                tma_load_4d(dst + (k >> 3) * (NB * 1024), map, bar, 0, kvh * NB, row >> 3);
            } else if constexpr (!E4M3) {
                tma_load_2d(dst + k * 128, map, bar, kvh * HD, row);
            } else if constexpr (HD == 256) {
                // two lines of 128 codes a row, kTile lines apart
                tma_load_2d(dst + k * 128, map, bar, kvh * HD, row);
                tma_load_2d(dst + kTile * 128 + k * 128, map, bar, kvh * HD + 128, row);
            } else {
                tma_load_2d(dst + k * HD, map, bar, kvh * HD, row);
            }
        };
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        int issued = 0;
        for (int j = 0; j < nt; ++j) {
            const int slot = j % kSlots;
            ok = wait_long(m_full0 + 8 * slot, (j / kSlots) & 1, wc, kSiteKvMeta) &&
                 wait_long(empty0 + 8 * stage, phase ^ 1u, wc, kSiteKvEmpty);
            if (!E4M3 && j == S - 1) ok = ok && wait_long(q_full, 0, wc, kSiteKvQ);   // Q came through this stage
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ++issued;
            // Positions past the last key, to the next group of 16 (or box), are not loaded:
            // their scores are masked, and PV leaves their groups out.
            const int upto = min(kTile, (keys.kv_end - keys.base(keys.begin + j) + pad - 1) & -pad);
            if (elect_one()) {
                const uint32_t bar = full0 + 8 * stage;
                const uint32_t dst = dst0 + stage * kBytes;
                const int kind = s_kind[slot * 4];
                const int4* boxes = reinterpret_cast<const int4*>(s_box + slot * 32);
                mbar_arrive_expect_tx(bar, kBytes / kTile * upto);
                if (kind == kLoadTile) {
                    load_box(dst, tile_map, bar, 0, boxes[0].x);
                } else if (kind == kLoadBoxes) {
                    for (int k = 0; k < upto; k += 4 * box) {
                        const int4 r = boxes[k / box >> 2];
                        load_box(dst, box_map, bar, k, r.x);
                        if (k + box < upto) load_box(dst, box_map, bar, k + box, r.y);
                        if (k + 2 * box < upto) load_box(dst, box_map, bar, k + 2 * box, r.z);
                        if (k + 3 * box < upto) load_box(dst, box_map, bar, k + 3 * box, r.w);
                    }
                } else {
                    const int* rows_of = s_row + slot * kTile;
                    const uint32_t* mask = s_mask + slot * 4;
                    for (int k = 0; k < upto; k += box) {
                        if (box >= 8 && box_state(mask, k, box) != 2) {
                            load_box(dst, box_map, bar, k, rows_of[k]);
                            continue;
                        }
                        for (int u = k; u < k + box; u += 4) {
                            const int4 r = *reinterpret_cast<const int4*>(rows_of + u);
                            if constexpr (!E4M3) {
                                for (int blk = 0; blk < NB; ++blk)
                                    tma_gather4(dst + ((u >> 3) * NB + blk) * 1024 + (u & 7) * 128, row_map, bar,
                                                kvh * HD + blk * 64, r);
                            } else if constexpr (HD == 256) {
                                for (int h = 0; h < 2; ++h)
                                    tma_gather4(dst + h * (kTile * 128) + u * 128, row_map, bar, kvh * HD + h * 128, r);
                            } else {
                                tma_gather4(dst + u * HD, row_map, bar, kvh * HD, r);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (!is_k && lane == 0) mbar_arrive(m_empty0 + 8 * slot);
            if (++stage == RING) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (!ok) {
            // abort: the loads already issued land before the CTA exits
            const int pending = issued < RING ? issued : RING;
            for (int j = 1; j <= pending; ++j) {
                const int s = (stage - j + RING) % RING;
                mbar_wait(full0 + 8 * s, stage - j < 0 ? phase ^ 1u : phase, wc_drain, kSiteKvDrain);
            }
        }
    } else if (warp == kWarpMma) {
        // ------------------------------------------------------------------
        // MMA issuer
        // ------------------------------------------------------------------
        {
            bool ok = __all_sync(0xffffffffu, wait_long(q_full, 0, wc, kSiteKvQ));
            tc_fence_after_sync();
            const uint32_t q_tmem = tmem + G::kColQ, o_tmem = tmem + G::kColO;
            int ks = 0, vs = 0;
            uint32_t kph = 0, vph = 0;
            auto scores = [&](int j) {
                ok = __all_sync(0xffffffffu, ok && wait_long(k_full0 + 8 * ks, kph, wc, kSiteKvFull));
                if (!ok) return;
                tc_fence_after_sync();
                const uint32_t b = smem_u32(s_k + ks * G::kStageBytes);
                if (elect_one()) {
#pragma unroll
                    for (int kb = 0; kb < NB; ++kb)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_f16_tmem_a(tmem + (j & 1) * kTile, q_tmem + (kb * 4 + kk) * 8,
                                           smem_desc_sw128(b + kb * 1024 + kk * 32, 16, NB * 1024), kIdescS,
                                           (kb | kk) != 0 ? 1u : 0u);
                    mma_commit(s_full0 + 8 * (j & 1));
                    mma_commit(k_empty0 + 8 * ks);
                }
                __syncwarp();
                if (++ks == S) {
                    ks = 0;
                    kph ^= 1u;
                }
            };
            auto weighted = [&](int j) {
                ok = ok && wait_long(v_full0 + 8 * vs, vph, wc, kSiteKvFull);
                ok = ok && wait_long(p_full0 + 8 * (j & 1), (j >> 1) & 1, wc, kSiteKvWeights);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                tc_fence_after_sync();
                const uint32_t b = smem_u32(s_v + vs * G::kStageBytes);
                // 16 positions an MMA; those past kv_end are not multiplied
                const int steps = min(kTile / 16, (keys.kv_end - keys.base(keys.begin + j) + 15) / 16);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        if (kk < steps)
                            mma_f16_tmem_a(o_tmem, tmem + (j & 1) * kTile + kk * 8,
                                           smem_desc_sw128(b + kk * (NB * 2048), 1024, NB * 1024), kIdescO,
                                           (j | kk) != 0 ? 1u : 0u);
                    mma_commit(o_done0 + 8 * (j & 1));
                    mma_commit(v_empty0 + 8 * vs);
                }
                __syncwarp();
                if (++vs == S) {
                    vs = 0;
                    vph ^= 1u;
                }
            };
            if (ok) scores(0);
            for (int j = 0; j < nt && ok; ++j) {
                if (j + 1 < nt) scores(j + 1);
                if (ok) weighted(j);
            }
            if (!ok) {
                // abort: every MMA issued so far finishes before TMEM is freed
                if (elect_one()) mma_commit(drain);
                __syncwarp();
                mbar_wait(drain, 0u, wc_drain, kSiteKvDrain);
            }
        }
        __syncwarp();
    } else if (warp == kWarpPages) {
        // ------------------------------------------------------------------
        // Look-ups, some tiles ahead of the loads: each position's cache row (past the
        // last row where it holds no key), the mask and the scales; kTile / 32
        // positions per lane.  Block-table entries are loaded two tiles before they
        // are published, scales one.
        // ------------------------------------------------------------------
        constexpr int PL = kTile / 32;
        const int bs = p.b.block_size;
        const int flat = p.b.flat_len > 0 ? seq * p.b.flat_len : -1;   // rows of a flat copy
        const int none = p.b.flat_len > 0 ? p.b.num_seqs * p.b.flat_len : p.b.num_blocks * bs;
        const int tile_pages = kTile / bs, tile_slots = kTile - tile_pages * bs;
        int page[PL], off[PL];              // of the next tile to look up
        int entry[PL], entry_off[PL];       // looked up: block-table entry and place in the page
        int row[PL];                        // of the next tile to publish
        uint32_t kb[PL], vb[PL], have = 0;
        ScaleRange scales;
        auto look_up = [&](int i) {         // tiles in turn
            if (i >= keys.end) return;
            if (i == keys.begin || i == keys.sink_tiles) {
#pragma unroll
                for (int u = 0; u < PL; ++u) {
                    const int t = keys.base(i) + u * 32 + lane;
                    page[u] = t / bs;
                    off[u] = t - page[u] * bs;
                }
            }
#pragma unroll
            for (int u = 0; u < PL; ++u) {
                entry[u] = page[u] < p.b.max_blocks ? table[page[u]] : -1;
                entry_off[u] = off[u];
                page[u] += tile_pages;
                off[u] += tile_slots;
                if (off[u] >= bs) {
                    off[u] -= bs;
                    ++page[u];
                }
            }
        };
        auto fetch = [&](int i) {           // the tile looked up last
            if (i >= keys.end) return;
            const int base = keys.base(i);
            const bool inside = keys.all(base, kTile);   // the usual case: all positions in sight
            have = 0;
            bool bad = false;
#pragma unroll
            for (int u = 0; u < PL; ++u) {
                const int t = base + u * 32 + lane;
                const bool h = inside || keys.holds(t);
                const bool g = static_cast<unsigned>(entry[u]) < static_cast<unsigned>(p.b.num_blocks);
                bad = bad || (h && !g);
                row[u] = h && g ? (flat >= 0 ? flat + t : entry[u] * bs + entry_off[u]) : none;
                have |= (h && g ? 1u : 0u) << u;
                if constexpr (E4M3) {
                    kb[u] = vb[u] = 127u;
                    if (h && g) {
                        const long long at = static_cast<long long>(row[u]) * p.b.num_kv_heads + kvh;
                        kb[u] = p.b.k_scales[at];
                        vb[u] = p.b.v_scales[at];
                    }
                }
            }
            if (bad) *reinterpret_cast<volatile int*>(p.b.status) = kDevErrBadIndex;
        };
        const int box_shift = 31 - __clz(p.box);
        look_up(keys.begin);
        fetch(keys.begin);
        look_up(keys.begin + 1);
        bool ok = true;
        for (int j = 0; j < nt && ok; ++j) {
            const int slot = j % kSlots;
            ok = __all_sync(0xffffffffu, wait_long(m_empty0 + 8 * slot, ((j / kSlots) & 1) ^ 1, wc, kSiteKvMeta));
            if (!ok) break;
            const bool full = __all_sync(0xffffffffu, have == (1u << PL) - 1u);
            const int row0 = __shfl_sync(0xffffffffu, row[0], 0);
            bool run = full && p.tile_rows > 0 && row0 + kTile <= p.tile_rows && (E4M3 || HD == 64 || (row0 & 7) == 0);
#pragma unroll
            for (int u = 0; u < PL; ++u) run = run && row[u] == row0 + u * 32 + lane;
            run = __all_sync(0xffffffffu, run);
            int kind = kLoadTile;
            if (run) {
                if (lane < PL) s_mask[slot * 4 + lane] = 0xffffffffu;
                if (lane == 0) s_box[slot * 32] = row0;
            } else {
#pragma unroll
                for (int u = 0; u < PL; ++u) {
                    const uint32_t word = __ballot_sync(0xffffffffu, (have >> u) & 1u);
                    if (lane == 0) s_mask[slot * 4 + u] = word;
                    const int k = u * 32 + lane;
                    s_row[slot * kTile + k] = row[u];
                    if ((k & (p.box - 1)) == 0) s_box[slot * 32 + (k >> box_shift)] = row[u];
                }
                __syncwarp();
                const bool mixed = !full && lane * p.box < kTile && box_state(s_mask + slot * 4, lane * p.box, p.box) == 2;
                kind = p.box >= 8 && !__any_sync(0xffffffffu, mixed) ? kLoadBoxes : kLoadRows;
            }
            if (lane == 0) s_kind[slot * 4] = kind;
            if constexpr (E4M3) {
                // the range of V's exponents, the least scale (that of all-zero rows) left out
                int top = -1000, low = 1000;
#pragma unroll
                for (int u = 0; u < PL; ++u) {
                    s_kf[slot * kTile + u * 32 + lane] = e8m0_value(kb[u]);
                    if (((have >> u) & 1u) != 0 && vb[u] > 10u && vb[u] != 255u) {
                        top = max(top, static_cast<int>(vb[u]) - 127);
                        low = min(low, static_cast<int>(vb[u]) - 127);
                    }
                    if (k_scale_too_large(kb[u])) low = -1000;   // out of any range
                }
                top = __reduce_max_sync(0xffffffffu, top);
                low = __reduce_min_sync(0xffffffffu, low);
                const bool wide = scales.take(top, low);
#pragma unroll
                for (int u = 0; u < PL; ++u)
                    s_vf[slot * kTile + u * 32 + lane] =
                        0x10001u * (((have >> u) & 1u) != 0 ? scales.factor(vb[u]) : 0x3c00u);
                if (lane == 0) {
                    s_exp[slot] = scales.E;
                    if (wide) *s_wide = 1u;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(m_full0 + 8 * slot);
            fetch(keys.begin + j + 1);
            look_up(keys.begin + j + 2);
        }
    } else if (warp >= 12) {
        if constexpr (E4M3) {
            // ----------------------------------------------------------------
            // Codes -> FP16, where the MMAs read them; values times their row's factor.
            // A failed wait does not leave the loop (see the softmax warps).
            // ----------------------------------------------------------------
            const int tid = (threadIdx.x - 384) % (32 * kConvertWarps);
            constexpr int kChunks = G::kRawBytes / 16 / (32 * kConvertWarps);   // 16 codes each, per thread
            constexpr int CPR = HD / 16;                       // chunks per row
            auto convert = [&](int j, bool v) {
                const int rs = j % RS, ss = j % S;
                const uint8_t* raw = (v ? r_v : r_k) + rs * G::kRawBytes;
                uint8_t* dst = (v ? s_v : s_k) + ss * G::kStageBytes;
                wait_long((v ? rv_full0 : rk_full0) + 8 * rs, (j / RS) & 1, wc, kSiteKvRaw);
                auto codes = [&](int u) {
                    const int ch = u * (32 * kConvertWarps) + tid;
                    const int r = ch / CPR, e = ch % CPR;
                    // the line (128 bytes; 64 with HD = 64) of row r's codes, and the chunk in it,
                    // swizzled by the line's place
                    const int line = ((e >> 3) * kTile + r) * (HD == 64 ? 64 : 128);
                    const int c = (e & 7) ^ ((line >> 7) & (HD == 64 ? 3 : 7));
                    return *reinterpret_cast<const uint4*>(raw + line + c * 16);
                };
                wait_long((v ? v_empty0 : k_empty0) + 8 * ss, ((j / S) & 1) ^ 1, wc, kSiteKvEmpty);
                if (j == S - 1) wait_long(q_full, 0, wc, kSiteKvQ);   // Q came through this stage
                // One or two chunks at a time: the warps of a CTA run six different loops, and more
                // code here costs them all.  Chunks of a few tokens over 2000 to 9000, head_dim 256:
                // 56.5 us with one, 53.5 with two, 56.4 with four, 63.4 with all eight; 2048 rows over
                // 30000 positions without the flat copy, head_dim 64: 221 us with one, 244 with two.
                constexpr int kAtOnce = HD == 256 ? 2 : 1;
#pragma unroll 1
                for (int u0 = 0; u0 < kChunks; u0 += kAtOnce) {
                    uint4 x[kAtOnce];
                    uint32_t factor[kAtOnce];
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u) {
                        x[u] = codes(u0 + u);
                        factor[u] = v ? s_vf[(j % kSlots) * kTile + ((u0 + u) * (32 * kConvertWarps) + tid) / CPR] : 0x3c003c00u;
                    }
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u) {
                        const int ch = (u0 + u) * (32 * kConvertWarps) + tid;
                        const int r = ch / CPR, e = ch % CPR;
                        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                        // factor 0, the least scale: all zeros, or a code whose value this sum leaves out?
                        if (factor[u] == 0u && ((w[0] | w[1] | w[2] | w[3]) & 0x7f7f7f7fu) != 0u) *s_wide = 1u;
                        uint32_t o[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) o[k] = e4m3x2_f16x2(w[k >> 1] >> (16 * (k & 1)));
                        if (v) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) o[k] = mul_f16x2(o[k], factor[u]);
                        }
                        uint8_t* d = dst + ((r >> 3) * NB + (e >> 2)) * 1024 + (r & 7) * 128;
                        // 16-byte chunks permuted by the row; lanes of odd blocks write the later one
                        // first, so that a row's lanes meet distinct banks
                        const int c16 = (e & 3) * 2, flip = (e >> 2) & 1;
                        const uint4 a = make_uint4(o[0], o[1], o[2], o[3]), b = make_uint4(o[4], o[5], o[6], o[7]);
                        *reinterpret_cast<uint4*>(d + (((c16 + flip) ^ (r & 7)) << 4)) = flip ? b : a;
                        *reinterpret_cast<uint4*>(d + (((c16 + 1 - flip) ^ (r & 7)) << 4)) = flip ? a : b;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive((v ? rv_empty0 : rk_empty0) + 8 * rs);
                    mbar_arrive((v ? v_full0 : k_full0) + 8 * ss);
                    if (v) mbar_arrive(m_empty0 + 8 * (j % kSlots));
                }
            };
            for (int j = 0; j < nt; ++j) convert(j, warp >= 12 + kConvertWarps);
        }
    } else {
        // ------------------------------------------------------------------
        // Softmax: warp (quarter, half) has TMEM lanes 32 * quarter .. and half of
        // the columns: of S positions kTile/2 * half .., of O dimensions HD/2 * half ..
        // A failed wait (abort flag up) does not leave the loop: the barriers below
        // stay matched, the waits return at once and the output is undefined.
        // ------------------------------------------------------------------
        const int quarter = warp & 3;
        const int half = H == 2 ? (warp - 4) >> 2 : 0;
        const int r = quarter * 32 + lane;
        const bool idle = quarter * 32 >= rows;   // the whole warp
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const int my = row0 + min(r, rows - 1);
        const int token = first + my / p.group;
        const int head = kvh * p.group + my % p.group;
        const int pos = pos0 + my / p.group;
        float row_scale = p.scale_log2;
        if (!idle) {
            // This half of Q's row: 16-bit pairs, one per TMEM column.  Neighbouring lanes load
            // neighbouring 16 bytes, and the rows go to their lanes through the last stages
            // of keys and values (a lane loading its own row takes 32 cache lines an
            // instruction, and the look-ups queue behind them: 2000 to 5000 clocks).
            constexpr int QW = HD / 2 / H;   // pairs
            constexpr int LPR = QW / 4;      // lanes per row
            constexpr int kMine = 32 * QW * 4;
            static_assert(4 * H * kMine <= 2 * G::kStageBytes, "Q's rows in two stages");
            const int at = (quarter * H + half) * kMine;
            uint4* mine = reinterpret_cast<uint4*>((at < G::kStageBytes ? s_k : s_v - G::kStageBytes) +
                                                   (S - 1) * G::kStageBytes + at);
            const long long q_row = token * p.q_stride + static_cast<long long>(head) * HD + half * (HD / H);
            constexpr int kRound = E4M3 && LPR > 8 ? 8 : LPR;   // loads at a time (as registers allow)
#pragma unroll 1
            for (int c0 = 0; c0 < LPR; c0 += kRound) {
                uint4 x[kRound];
#pragma unroll
                for (int c = 0; c < kRound; ++c) {
                    const int i = (c0 + c) * 32 + lane;
                    x[c] = *reinterpret_cast<const uint4*>(p.q + __shfl_sync(0xffffffffu, q_row, i / LPR) + i % LPR * 8);
                }
#pragma unroll
                for (int c = 0; c < kRound; ++c) {
                    const int i = (c0 + c) * 32 + lane;
                    mine[i / LPR * LPR + (i % LPR ^ row_swizzle<LPR>(i / LPR))] = x[c];
                }
            }
            __syncwarp();
            float f = 1.f;
            if constexpr (E4M3) {
                // FP16 beside FP16 keys: the row times a power of two that brings its largest
                // value to [2^14, 2^15).  What FP16 then drops is under 2^-39 of the largest.
                uint32_t m = 0;
#pragma unroll
                for (int c = 0; c < LPR; ++c) {
                    const uint4 x = mine[lane * LPR + (c ^ row_swizzle<LPR>(lane))];
                    m = __vmaxu2(__vmaxu2(m, x.x & 0x7fff7fffu), x.y & 0x7fff7fffu);
                    m = __vmaxu2(__vmaxu2(m, x.z & 0x7fff7fffu), x.w & 0x7fff7fffu);
                }
                m = max(m & 0xffffu, m >> 16);
                uint32_t* sm = reinterpret_cast<uint32_t*>(s_max);
                sm[half * kRows + r] = m;
                named_barrier(1 + quarter, 64);
                m = max(m, sm[(half ^ 1) * kRows + r]);
                int e = static_cast<int>(m >> 7) - 127 - 14;               // q * 2^-e
                e = max(-126, min(e, 113));
                f = exp2f(static_cast<float>(-e));
                row_scale = row_factor(p.scale_log2, e);
                named_barrier(1 + quarter, 64);   // s_max is free again
            }
            constexpr int kPart = QW < 32 ? 16 : 32;   // columns at a time
#pragma unroll
            for (int c0 = 0; c0 < QW; c0 += kPart) {
                uint32_t t[kPart];
#pragma unroll
                for (int c = 0; c < kPart; c += 4) {
                    const uint4 x = mine[lane * LPR + ((c0 + c) / 4 ^ row_swizzle<LPR>(lane))];
                    t[c] = x.x ^ p.q_sign;
                    t[c + 1] = x.y ^ p.q_sign;
                    t[c + 2] = x.z ^ p.q_sign;
                    t[c + 3] = x.w ^ p.q_sign;
                }
                if constexpr (E4M3) {
#pragma unroll
                    for (int c = 0; c < kPart; ++c)
                        t[c] = f16x2(__uint_as_float(t[c] << 16) * f, __uint_as_float(t[c] & 0xffff0000u) * f);
                }
                const uint32_t q_addr = lane_addr + G::kColQ + half * QW + c0;
                if constexpr (kPart == 32)
                    tmem_st_32x32b_x32(q_addr, t);
                else
                    tmem_st_32x32b_x16(q_addr, t);
            }
            fence_proxy_async_smem();   // the stage is the TMA unit's from here on
            tmem_st_wait();
            tc_fence_before_sync();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        const int lo = window_start(pos, p.window);        // this row's
        const int lo_max = window_start(pmax, p.window);   // the last row's
        float m = -INFINITY;
        float2 l2 = make_float2(0.f, 0.f);
        // E4M3 (ScaleRange): O holds 2^(5 - E) of its values, and weights, O and l 2^7 more.
        int E = 0;
        for (int j = 0; j < nt; ++j) {
            const int buf = j & 1;
            const int slot = j % kSlots;
            if constexpr (E4M3) wait_long(m_full0 + 8 * slot, (j / kSlots) & 1, wc, kSiteKvMeta);
            wait_long(s_full0 + 8 * buf, (j >> 1) & 1, wc, kSiteKvScores);
            tc_fence_after_sync();
            if (!idle) {
                const uint32_t s_addr = lane_addr + (j & 1) * kTile + half * C;
                float2 x[C / 2];
                {
                    uint32_t raw[C / 32][32];
#pragma unroll
                    for (int c = 0; c < C / 32; ++c) tmem_ld_32x32b_x32(s_addr + 32 * c, raw[c]);
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < C / 2; ++c)
                        x[c] = make_float2(__uint_as_float(raw[c >> 4][(2 * c) & 31]),
                                           __uint_as_float(raw[c >> 4][(2 * c + 1) & 31]));
                }
                float grow_e = 1.f;   // E4M3: factor of O for a new E
                if constexpr (E4M3) {
                    const float4* kf = reinterpret_cast<const float4*>(s_kf + slot * kTile + half * C);
#pragma unroll
                    for (int c = 0; c < C / 4; ++c) {
                        const float4 f = kf[c];
                        x[2 * c] = mul2(x[2 * c], make_float2(f.x, f.y));
                        x[2 * c + 1] = mul2(x[2 * c + 1], make_float2(f.z, f.w));
                        if (c % 4 == 3) asm volatile("" ::: "memory");   // no more loads ahead: registers
                    }
                    const int now = s_exp[slot];
                    if (j > 0) grow_e = exp2_fast(static_cast<float>(E - now));
                    E = now;
                }
                // positions that hold no key, or that this row does not see
                const int t0 = keys.base(keys.begin + j) + half * C;
                uint2 have;
                if constexpr (C == 64)
                    have = *reinterpret_cast<const uint2*>(s_mask + slot * 4 + half * 2);
                else
                    have = make_uint2(s_mask[slot * 4 + half], 0xffffffffu);
                if ((have.x & have.y) != 0xffffffffu || t0 + C - 1 > pmin || (t0 < lo_max && t0 + C > p.sinks)) {
                    const unsigned long long seen = (static_cast<unsigned long long>(have.y) << 32 | have.x) &
                                                    low_bits(pos + 1 - t0) & (~low_bits(lo - t0) | low_bits(p.sinks - t0));
                    const uint32_t lo32 = static_cast<uint32_t>(seen), hi32 = static_cast<uint32_t>(seen >> 32);
#pragma unroll
                    for (int c = 0; c < C / 2; ++c) {
                        const uint32_t w = c < 16 ? lo32 : hi32;
                        if (!((w >> ((2 * c) & 31)) & 1u)) x[c].x = -INFINITY;
                        if (!((w >> ((2 * c + 1) & 31)) & 1u)) x[c].y = -INFINITY;
                    }
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < C / 2; ++c) mx[c & 3] = max3(mx[c & 3], x[c].x, x[c].y);
                float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
                if constexpr (H == 2) {
                    // the row's other half; also: both warps have read S, P may go over it
                    float* sm = s_max + buf * 2 * kRows;
                    sm[half * kRows + r] = top;
                    named_barrier(1 + quarter, 64);
                    top = fmaxf(top, sm[(half ^ 1) * kRows + r]);
                }
                top *= row_scale;
                const float mn = fmaxf(m, top);
                if (j == 0) {
                    m = mn;
                } else if (__any_sync(0xffffffffu, mn > m + 8.f) || (E4M3 && grow_e != 1.f)) {
                    float f = 1.f;
                    if (mn > m + 8.f) {
                        f = exp2_fast(m - mn);
                        m = mn;
                    }
                    l2 = mul2(l2, make_float2(f, f));
                    f *= grow_e;
                    wait_long(o_done0 + 8 * ((j - 1) & 1), ((j - 1) >> 1) & 1, wc, kSiteKvOutput);   // PV of j - 1
                    tc_fence_after_sync();
                    // this half of the row's O, 16 columns at a time (beside x in registers)
#pragma unroll 1
                    for (int c = 0; c < HD / H / 16; ++c) {
                        const uint32_t o_addr = lane_addr + G::kColO + half * (HD / H) + c * 16;
                        uint32_t o[16];
                        tmem_ld_32x32b_x16(o_addr, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st_32x32b_x16(o_addr, o);
                    }
                }
                float base = m == -INFINITY ? 0.f : m;
                if constexpr (E4M3) base -= kWeightLog2;
                const float2 sc = make_float2(row_scale, row_scale), nb = make_float2(-base, -base);
                const uint32_t p_addr = lane_addr + (j & 1) * kTile + half * (C / 2);
#pragma unroll
                for (int g = 0; g < C / 32; ++g) {   // 32 columns, 16 of P, at a time
                    uint32_t w[16];
#pragma unroll
                    for (int c = 0; c < 16; c += 2) {
                        float2 e0 = fma2(x[16 * g + c], sc, nb), e1 = fma2(x[16 * g + c + 1], sc, nb);
                        e0.x = exp2_fast(e0.x);
                        e0.y = exp2_fast(e0.y);
                        e1.x = exp2_fast(e1.x);
                        e1.y = exp2_fast(e1.y);
                        l2 = add2(l2, add2(e0, e1));
                        if constexpr (E4M3) {
                            w[c] = f16x2(e0.x, e0.y);
                            w[c + 1] = f16x2(e1.x, e1.y);
                        } else {
                            // BF16, since an MMA's operands have one type and FP16 does not hold BF16
                            // values: 2^-8 of a weight at most (outputs are 0.0023 off in the mean,
                            // where weights in FP32 give 0.0017, the output's own rounding)
                            w[c] = bf16x2(e0.x, e0.y);
                            w[c + 1] = bf16x2(e1.x, e1.y);
                        }
                    }
                    tmem_st_32x32b_x16(p_addr + 16 * g, w);
                }
                tmem_st_wait();
                tc_fence_before_sync();
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(p_full0 + 8 * buf);
                mbar_arrive(m_empty0 + 8 * slot);
            }
        }
        // ---- the rows' results ---------------------------------------------
        wait_long(o_done0 + 8 * ((nt - 1) & 1), ((nt - 1) >> 1) & 1, wc, kSiteKvOutput);
        tc_fence_after_sync();
        if (!idle) {
            float l = l2.x + l2.y;
            if constexpr (H == 2) {
                float* sm = s_max + (nt & 1) * 2 * kRows;
                sm[half * kRows + r] = l;
                named_barrier(1 + quarter, 64);
                l = sm[r] + sm[kRows + r];   // the same order for both halves
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const long long at = (static_cast<long long>(token) * p.num_q_heads + head) * p.segments + seg;
            // E4M3: out of the weighted mean, O / l; a split row's partial sums leave out 2^7 too
            const float mean = E4M3 ? exp2f(static_cast<float>(E - 5)) : 1.f;
            const float plain = E4M3 ? exp2f(static_cast<float>(E - 5) - kWeightLog2) : 1.f;
            const bool wide = E4M3 && *s_wide != 0u;
            const long long out_at = p.segments == 1 ? token * p.out_stride + static_cast<long long>(head) * HD : at * HD;
            uint4* stage = reinterpret_cast<uint4*>(s_k + (warp - 4) * 4096);
            static_assert(2 * S * G::kStageBytes >= 4 * H * 4096, "rows of 32 FP32 in the stages");
            float odd = 0.f;   // NaN once a value is not finite
            for (int c = 0; c < HD / H / 32; ++c) {
                const int d0 = half * (HD / H) + c * 32;
                uint32_t o[32];
                tmem_ld_32x32b_x32(lane_addr + G::kColO + d0, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) odd = fmaf(__uint_as_float(o[i]), 0.f, odd);
                // through shared memory (the stages are done with), so that neighbouring
                // lanes write neighbouring 16 bytes
                __syncwarp();
                if (p.segments == 1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t h[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            h[k] = bf16x2(__uint_as_float(o[8 * i + 2 * k]) * inv * mean,
                                          __uint_as_float(o[8 * i + 2 * k + 1]) * inv * mean);
                        stage[lane * 4 + (i ^ row_swizzle<4>(lane))] = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int rr = i * 8 + (lane >> 2);
                        const long long to = __shfl_sync(0xffffffffu, out_at, rr);
                        if (quarter * 32 + rr < rows)
                            *reinterpret_cast<uint4*>(p.out + to + d0 + (lane & 3) * 8) =
                                stage[rr * 4 + ((lane & 3) ^ row_swizzle<4>(rr))];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        stage[lane * 8 + (i ^ row_swizzle<8>(lane))] =
                            make_uint4(__float_as_uint(__uint_as_float(o[4 * i]) * plain),
                                       __float_as_uint(__uint_as_float(o[4 * i + 1]) * plain),
                                       __float_as_uint(__uint_as_float(o[4 * i + 2]) * plain),
                                       __float_as_uint(__uint_as_float(o[4 * i + 3]) * plain));
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int rr = i * 4 + (lane >> 3);
                        const long long to = __shfl_sync(0xffffffffu, out_at, rr);
                        if (quarter * 32 + rr < rows)
                            *reinterpret_cast<uint4*>(p.part_o + to + d0 + (lane & 7) * 4) =
                                stage[rr * 8 + ((lane & 7) ^ row_swizzle<8>(rr))];
                    }
                }
            }
            if (p.segments > 1 && half == 0 && r < rows) p.part_ml[at] = make_float2(m, E4M3 ? l * exp2f(-kWeightLog2) : l);
            if (((odd != 0.f && l - l == 0.f) || wide) && r < rows) s_flag[r] = 1;   // odd is NaN, l is finite
            if constexpr (H == 2)
                named_barrier(1 + quarter, 64);
            else
                __syncwarp();
            for (uint32_t left = __ballot_sync(0xffffffffu, s_flag[r] != 0); left != 0; left &= left - 1) {
                const int rr = quarter * 32 + __ffs(left) - 1, row = row0 + rr;
                if (H == 2 && (rr & 1) != half) continue;
                repair_row<E4M3, HD, kTile>(p, table, keys, kvh, first + row / p.group, kvh * p.group + row % p.group,
                                            pos0 + row / p.group, seg);
            }
        }
        tc_fence_before_sync();
    }
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, G::kTmem);
    }
}

// ---------------------------------------------------------------------------
// Joins the segments of split rows: M = max m_s, out = sum_s O_s 2^(m_s - M) /
// sum_s l_s 2^(m_s - M), in a fixed order.  256 threads have 64 dimensions of one
// row (WIDE: few rows, up to 256 segments; 16 groups of 16 threads share the
// segments) or of 16 rows (a group each).  Latency is what counts: the loads of
// (m, l) are one round, those of O as many as the registers allow.  One row of 256 by
// 74 segments: some 3 us between the attention's last store and the next call.
// ---------------------------------------------------------------------------
template <int HD, bool WIDE>
__global__ void __launch_bounds__(256) kv_join_kernel(const __grid_constant__ AttnParams p)
{
    __shared__ float4 s_o[16][16];
    __shared__ float s_w[256], s_red[8], s_l[8];
    const int g = threadIdx.x >> 4, e = threadIdx.x & 15;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_wait();
    griddep_launch_dependents();
    const long long row = WIDE ? blockIdx.x : static_cast<long long>(blockIdx.x) * 16 + g;
    const int token = static_cast<int>(row / p.num_q_heads);
    // a row of some sequence
    const bool in = token < p.b.num_tokens &&
                    (p.b.cu_tokens == nullptr || (token >= p.b.cu_tokens[0] && token < p.b.cu_tokens[p.b.num_seqs]));
    if (WIDE ? !in : false) return;
    const float2* ml = p.part_ml + row * p.segments;
    const float4* po = reinterpret_cast<const float4*>(p.part_o + row * p.segments * HD) + blockIdx.y * 16 + e;
    constexpr int kStride = HD / 4;
    float L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float w, const float4& v) {
        o.x = fmaf(w, v.x, o.x);
        o.y = fmaf(w, v.y, o.y);
        o.z = fmaf(w, v.z, o.z);
        o.w = fmaf(w, v.w, o.w);
    };
    if constexpr (WIDE) {
        const bool mine = threadIdx.x < p.segments;
        const float2 x = mine ? ml[threadIdx.x] : make_float2(-INFINITY, 0.f);
        float M = x.x;
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, i));
        if (lane == 0) s_red[warp] = M;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) M = fmaxf(M, s_red[i]);
        const float w = x.y == 0.f ? 0.f : exp2f(x.x - (M == -INFINITY ? 0.f : M));   // l = 0: saw nothing, O not written
        s_w[threadIdx.x] = w;
        float t = w * x.y;
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) t += __shfl_xor_sync(0xffffffffu, t, i);
        if (lane == 0) s_l[warp] = t;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) L += s_l[i];
        for (int s0 = g; s0 < p.segments; s0 += 16 * 8) {
            float4 v[8];
            float f[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int s = s0 + 16 * u;
                f[u] = s < p.segments ? s_w[s] : 0.f;
                // (a weight of NaN has its O)
                v[u] = s < p.segments && f[u] != 0.f ? po[static_cast<long long>(s) * kStride] : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) add(f[u], v[u]);
        }
        s_o[g][e] = o;
        __syncthreads();
        if (g != 0) return;
#pragma unroll
        for (int i = 1; i < 16; ++i) add(1.f, s_o[i][e]);
    } else if (in) {
        float M = -INFINITY;
#pragma unroll 4
        for (int s = 0; s < p.segments; ++s) M = fmaxf(M, ml[s].x);
        const float base = M == -INFINITY ? 0.f : M;
#pragma unroll 4
        for (int s = 0; s < p.segments; ++s) {
            const float2 x = ml[s];
            const bool some = x.y != 0.f;
            const float w = some ? exp2f(x.x - base) : 0.f;
            const float4 v = some ? po[static_cast<long long>(s) * kStride] : make_float4(0.f, 0.f, 0.f, 0.f);
            L = fmaf(w, x.y, L);
            add(w, v);
        }
    }
    if (in) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        uint16_t* out = p.out + token * p.out_stride + (row - static_cast<long long>(token) * p.num_q_heads) * HD +
                        blockIdx.y * 64 + 4 * e;
        *reinterpret_cast<uint2*>(out) = make_uint2(bf16x2(o.x * inv, o.y * inv), bf16x2(o.z * inv, o.w * inv));
    }
}

// The most positions that the rows of a CTA may see.
long long most_keys(const KvAttnLaunch& a)
{
    const long long seen = static_cast<long long>(a.window) + a.max_chunk + a.sinks;
    return a.window > 0 && seen < a.max_seq_len ? seen : a.max_seq_len;
}

// Rows per CTA of the kernel for few query rows per KV head, or 0: the call takes
// the other kernel.  An E4M3 cache read for few rows would spend its time in the
// other kernel's shared memory.  Measured in microseconds, many-row / few-row kernel
// (32 sequences of up to 4000 tokens; one of 30000): head_dim 256, 8 rows 79 / 79, 31 / 30,
// 16 rows 78 / 129, 31 / 43; 128, 8 rows 135 / 68, 42 / 25, 16 rows 123 / 80, 42 / 30, 24 rows
// 123 / 131, 43 / 43; 64, 16 rows 62 / 45, 22 / 18, 32 rows 63 / 68, 24 / 23.  On a BF16 cache
// it did not pay: 8 rows of 256 83 / 130, of 128 91 / 117, of 64 46 / 45.
int few_rows(const KvAttnLaunch& a)
{
    const long long rows = static_cast<long long>(a.max_chunk) * (a.num_q_heads / a.b.num_kv_heads);
    const int few = rows <= 8 || a.b.head_dim == 256 ? 8 : 16;
    if (a.b.type != kCacheE4M3 || a.kernel == 1) return 0;
    return a.kernel == 2 || rows <= (a.b.head_dim == 256 ? 8 : 16) ? few : 0;
}

int cta_rows_of(const KvAttnLaunch& a)
{
    const int few = few_rows(a);
    return few > 0 ? few : kRows;
}

// Row tiles per sequence and KV head: at most num_tokens * num_q_heads (kv_attention_limit).
int row_tiles_of(const KvAttnLaunch& a)
{
    const int cta_rows = cta_rows_of(a);
    const long long rows = static_cast<long long>(a.max_chunk) * (a.num_q_heads / a.b.num_kv_heads);
    return static_cast<int>((rows + cta_rows - 1) / cta_rows);
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
    const int few = few_rows(a);
    p.tiles = row_tiles_of(a);
    p.segments = a.segments;
    // Segments are as many positions for short sequences as for long ones, so that
    // CTAs have equal work in a batch of uneven lengths.
    p.segment_keys = static_cast<int>((most_keys(a) + a.segments * 128LL - 1) / (a.segments * 128LL) * 128);
    // a zero scale still has to keep -inf (a position not seen) at -inf
    p.scale_log2 = a.scale == 0.f ? std::numeric_limits<float>::denorm_min() : std::fabs(a.scale) * 1.4426950408889634f;
    p.q_sign = a.scale < 0.f ? 0x80008000u : 0u;
    p.window = a.window;
    p.sinks = a.sinks;
    p.part_o = a.workspace;
    const long long rows = static_cast<long long>(a.b.num_tokens) * a.num_q_heads;
    p.part_ml = reinterpret_cast<float2*>(a.workspace + rows * a.segments * HD);
    p.wait_limit_ns = a.wait_limit_ns;
    auto join = [&]() {
        if (a.segments == 1) return cudaSuccess;
        if (rows < 16 * a.num_sms)
            return launch_kernel(kv_join_kernel<HD, true>, dim3(static_cast<unsigned>(rows), HD / 64), dim3(256), 0, stream,
                                 a.pdl, p);
        return launch_kernel(kv_join_kernel<HD, false>, dim3(static_cast<unsigned>((rows + 15) / 16), HD / 64), dim3(256), 0,
                             stream, a.pdl, p);
    };
    if constexpr (E4M3) {
        if (few > 0) {
            const cudaError_t e = launch_few_rows<HD>(p, few, a.pdl, stream);
            return e != cudaSuccess ? e : join();
        }
    }
    KvMaps maps = {};
    TmapEncodeFn enc = tmap_encoder();
    if (enc == nullptr) {
        snprintf(msg, msg_len, "cuTensorMapEncodeTiled is not available from the driver");
        return cudaErrorNotSupported;
    }
    // a box is whole 8-row atoms of one page and fits a stage
    p.box = 4;
    for (int r = 8; r <= Geo<E4M3, HD>::kTile; r *= 2)
        if (a.b.block_size % r == 0) p.box = r;
    if (a.b.flat_len > 0) p.box = 16;   // (whole tiles are one box; of the last one, boxes)
    const cuuint64_t width = static_cast<cuuint64_t>(a.b.num_kv_heads) * HD;
    const cuuint64_t cache_rows = a.b.flat_len > 0 ? static_cast<cuuint64_t>(a.b.num_seqs) * a.b.flat_len
                                                   : static_cast<cuuint64_t>(a.b.num_blocks) * a.b.block_size;
    const cuuint64_t pitch = E4M3 ? width : width * 2;
    const cuuint32_t rows8 = static_cast<cuuint32_t>(p.box);
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    constexpr int kBoxDims = !E4M3 && HD > 64 ? 4 : 2;   // as in the kernel
    constexpr int kTile = Geo<E4M3, HD>::kTile;
    constexpr cuuint32_t kLine = E4M3 ? (HD < 128 ? HD : 128) : 64;   // elements of a swizzled line
    p.tile_rows = static_cast<int>(cache_rows / 8 * 8);
    const cuuint64_t dims2[2] = {width, cache_rows}, dims4[4] = {64, 8, width / 64, cache_rows / 8};
    const cuuint64_t strides2[1] = {pitch}, strides4[3] = {pitch, 128, pitch * 8};
    CUtensorMap* const map[6] = {&maps.k_row, &maps.v_row, &maps.k_tile, &maps.v_tile, &maps.k_box, &maps.v_box};
    for (int i = 0; i < (p.box >= 8 ? 6 : (p.tile_rows > 0 ? 4 : 2)); ++i) {
        const int d = i < 2 ? 2 : kBoxDims;
        const cuuint32_t r8 = i < 2 ? 1 : (i < 4 ? kTile : rows8);
        const cuuint32_t box2[2] = {kLine, r8}, box4[4] = {64, 8, HD / 64, r8 / 8};
        const CUresult r =
            enc(map[i], E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                static_cast<cuuint32_t>(d), i % 2 == 0 ? a.b.k : a.b.v, d == 2 ? dims2 : dims4,
                d == 2 ? strides2 : strides4, d == 2 ? box2 : box4, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                E4M3 && HD == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) {
            snprintf(msg, msg_len, "cuTensorMapEncodeTiled failed (%d) for the cache", static_cast<int>(r));
            return cudaErrorInvalidValue;
        }
    }
    auto kern = kv_attention_kernel<E4M3, HD>;
    static SmemOptIn smem_opt;
    cudaError_t e = smem_opt.ensure(reinterpret_cast<const void*>(kern), Geo<E4M3, HD>::kBytes);
    if (e != cudaSuccess) return e;
    const long long ctas = static_cast<long long>(p.tiles) * a.b.num_kv_heads * a.b.num_seqs * a.segments;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    e = launch_kernel(kern, dim3(static_cast<unsigned>(ctas)), dim3(Geo<E4M3, HD>::kThreads), Geo<E4M3, HD>::kBytes, stream, a.pdl,
                      maps, p);
    return e != cudaSuccess ? e : join();
}

}  // namespace

namespace {

size_t partial_bytes(const KvAttnLaunch& a)
{
    if (a.segments <= 1) return 0;
    const size_t bytes = static_cast<size_t>(a.b.num_tokens) * a.num_q_heads * a.segments * (a.b.head_dim + 2) * sizeof(float);
    return (bytes + 255) / 256 * 256;
}

// Rows of a sequence in the flat BF16 copy of an E4M3 cache, or 0: no copy is made.
// It costs one pass over the positions in sight; without it every 128 query rows
// convert them again.  Microseconds without / with it, 30000 positions: head_dim 256,
// 512 rows 94 / 105, 1024 rows 159 / 150, 2048 rows 304 / 257; 128, 256 rows 79 / 75,
// 512 rows 142 / 99, 2048 rows 521 / 261; 64, 256 rows 37 / 36, 2048 rows 217 / 114.
// In a batch of prompts and single tokens it also passes over the sequences that few
// rows read, so the rows per sequence count too, on average.  8000 positions, one
// prompt among single tokens (4 among 12 for the last of 256), 8 rows a token (256: 4):
// head_dim 256, 19 rows on average 353 / 829, 131 330 / 501, 515 735 / 791, 1026 607 / 573;
// 128, 39 rows 774 / 884, 135 572 / 526, 519 1332 / 934; 64, 39 rows 686 / 589.
int flat_rows(const KvAttnLaunch& a)
{
    const long long all_rows = static_cast<long long>(a.b.num_tokens) * (a.num_q_heads / a.b.num_kv_heads);
    const int average = a.b.head_dim == 256 ? 1024 : (a.b.head_dim == 128 ? 96 : 32);
    if (all_rows < static_cast<long long>(average) * a.b.num_seqs) return 0;
    const long long rows = static_cast<long long>(a.max_chunk) * (a.num_q_heads / a.b.num_kv_heads);
    if (!a.flat_copy || a.b.type != kCacheE4M3 || few_rows(a) > 0 || a.kernel == 1 || rows < (a.b.head_dim == 256 ? 1024 : 256)) return 0;
    const long long len = (a.max_seq_len + 127LL) / 128 * 128;
    const long long bytes = len * a.b.num_seqs * a.b.num_kv_heads * a.b.head_dim * 4;
    return len * a.b.num_seqs <= 0x7fffffffLL && bytes <= (2LL << 30) ? static_cast<int>(len) : 0;
}

}  // namespace

// An estimate: it counts tiles of 64 or 128 positions, while a segment's positions are
// rounded to 128 (so that the last of many segments may be empty: 10 of 74 for one
// sequence of 32768), and two CTAs of the few-row kernel per SM, which has four below
// head_dim 256.  One sequence of 32768, E4M3, head_dim 256: 607 us in one segment, 116 in
// 6, 34 in 32, 28 in the 74 it takes; 8 chunks of 1-6 tokens over 2000-9000: 160, 46,
// 74, and 53 in its 7; three chunks of 300 tokens over 9000, BF16: 136 (its choice), 167, 353.
int kv_attention_segments(const KvAttnLaunch& a)
{
    const int few = few_rows(a);
    const int cta_rows = cta_rows_of(a);
    const bool two = a.b.head_dim == 64 && (a.b.type == kCacheBF16 || flat_rows(a) > 0);   // CTAs per SM
    const int tile = few || two || a.b.head_dim == 256 ? 64 : 128;
    const long long group = a.num_q_heads / a.b.num_kv_heads;
    const long long per_seq = (static_cast<long long>(a.max_chunk) * group + cta_rows - 1) / cta_rows;
    long long row_tiles = (static_cast<long long>(a.b.num_tokens) * group + cta_rows - 1) / cta_rows + a.b.num_seqs - 1;
    if (row_tiles > per_seq * a.b.num_seqs) row_tiles = per_seq * a.b.num_seqs;
    const long long ctas = row_tiles * a.b.num_kv_heads;
    const long long tiles = (most_keys(a) + tile - 1) / tile;
    const double rows = static_cast<double>(a.b.num_tokens) * a.num_q_heads;
    // Time in units of one tile's work on one CTA: a CTA starts and ends in about
    // `fixed`, a join costs about as much and the traffic of the partial rows.
    const double fixed = few ? 4 : (tile == 64 ? 8 : 3);
    const long long slots = few || two ? 2LL * a.num_sms : a.num_sms;
    double best = 0;
    int segments = 1;
    for (int s = 1; s <= 256 && (s == 1 || s <= tiles); ++s) {
        const double each = static_cast<double>((tiles + s - 1) / s);
        double t;
        const double full = static_cast<double>((ctas * s + slots - 1) / slots) * (fixed + each);   // whole waves
        if (a.b.num_seqs == 1 || a.window > 0) {
            t = full;   // equal CTAs
        } else {
            // Lengths anywhere up to the longest: 0.6 of it on average.  Fewer CTAs than
            // slots end together; else it is the average work, and the last CTA's.  The
            // kernel for many rows has few CTAs, so that one wave more or less counts:
            // there, against the chance that all are as long as the longest.
            const double n = s > 1 ? static_cast<double>(ctas) * (0.6 * s + 0.5) : static_cast<double>(ctas);
            const double spread = (static_cast<double>(ctas) * 0.6 * static_cast<double>(tiles) + n * fixed) / static_cast<double>(slots) + each;
            t = few ? spread : 0.6 * (n <= static_cast<double>(slots) ? fixed + each : spread) + 0.4 * full;
        }
        if (s > 1) t += fixed + rows * s * a.b.head_dim * 8 / 3.5e6;
        if (s == 1 || t < best) {
            best = t;
            segments = s;
        }
    }
    return segments;
}

void kv_attention_limit(KvAttnLaunch& a)
{
    const int most = a.b.cu_tokens != nullptr ? a.b.num_tokens : 1;
    if (a.max_chunk > most) a.max_chunk = most;
}

KvAttnPlan kv_attention_plan(const KvAttnLaunch& a)
{
    KvAttnPlan plan;
    plan.cta_rows = cta_rows_of(a);
    plan.tiles = row_tiles_of(a);
    plan.segments = a.segments;
    plan.flat_rows = flat_rows(a);
    return plan;
}

size_t kv_attention_workspace(const KvAttnLaunch& a)
{
    return partial_bytes(a) +
           static_cast<size_t>(flat_rows(a)) * a.b.num_seqs * a.b.num_kv_heads * a.b.head_dim * 2 * sizeof(uint16_t);
}

int launch_kv_attention(const KvAttnLaunch& launch, cudaStream_t stream, char* msg, size_t msg_len)
{
    KvAttnLaunch a = launch;
    if (const int flat = flat_rows(a); flat > 0) {
        uint16_t* k = reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(a.workspace) + partial_bytes(a));
        uint16_t* v = k + static_cast<size_t>(flat) * a.b.num_seqs * a.b.num_kv_heads * a.b.head_dim;
        if (launch_kv_flatten(a.b, k, v, flat, a.max_seq_len, a.window, a.sinks, a.pdl, stream, msg, msg_len)) return 1;
        a.b.k = k;
        a.b.v = v;
        a.b.k_scales = a.b.v_scales = nullptr;
        a.b.type = kCacheBF16;
        a.b.flat_len = flat;
    }
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
