// linear_grad.cu -- the element-wise part of the feed-forward layers' backward
// passes, and the bias gradients.
//
//   dz = dy act'(z);   gated: dg = dh u act'(g),  du = dh act(g)
//
// One pass over the tokens: every value is read once, FP32 inside, dz rounded
// once to the type, because it is an operand of the tensor cores' products next
// (2^-8 of each term at most in BF16, 2^-11 in FP16, either way: the gradients' sums
// see about as much as from their own rounding).  A bias gradient is the column sum
// of the unrounded dz: each thread keeps its columns' sums over its tokens, a
// block adds its threads' in a fixed order and leaves one FP32 row; the products'
// kernel, or one of its own without products, adds those rows in order.  No
// atomics: the same call gives the same bits.
// Bound: HBM (6 bytes read and 4 written per value of a gated layer), of which it gets 0.8
// (4096 x 17408: 129 us, 5.5 TB/s).  An asynchronous copy ring per warp and blocks of 2048 columns
// were tried: the ring gained 2% there and lost 12% on 200 x 1000 x 1024, wide blocks lost everywhere.
#include <cstdio>

#include "bsk_internal.h"
#include "linear_math.cuh"

namespace bsk {
namespace {

constexpr int kGradThreads = 256;
constexpr int kGradCols = 8;                        // columns per thread: 16 bytes
constexpr int kGradTileCols = 32 * kGradCols;       // columns per block
constexpr int kGradRowThreads = kGradThreads / 32;  // rows a block works on at once

struct ActBackwardParams {
    int n, M, rows_per_chunk;
    const uint16_t* z[2];
    long long ldz;
    const uint16_t* dy;
    long long ld_dy;
    uint16_t* dz[2];
    long long ld_dz;
    float* partial;
};

// 8 values of 16 bits from p on, n of them there.  Without ALIGNED a row may start at any
// element: the values lie in two 16-byte units, and only units that hold one of them are read.  Either
// way what else such a unit holds (the next columns of wider rows, say) is read and not used.
template <bool ALIGNED>
struct GradValues {
    uint4 lo, hi;
};
template <bool ALIGNED>
__device__ __forceinline__ GradValues<ALIGNED> grad_load(const uint16_t* p, int n)
{
    GradValues<ALIGNED> v;
    if constexpr (ALIGNED) {
        v.lo = *reinterpret_cast<const uint4*>(p);
    } else {
        const uint4* u = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) & ~static_cast<uintptr_t>(15));
        v.lo = *u;
        if ((reinterpret_cast<uintptr_t>(p) & 15u) + 2u * static_cast<uint32_t>(n) > 16u) v.hi = u[1];
    }
    return v;
}
// The values as words, two each (shift: bytes from the first unit's start to the first value).
template <bool ALIGNED>
__device__ __forceinline__ void grad_words(uint32_t (&o)[4], const GradValues<ALIGNED>& v, uint32_t shift)
{
    if constexpr (ALIGNED) {
        o[0] = v.lo.x;
        o[1] = v.lo.y;
        o[2] = v.lo.z;
        o[3] = v.lo.w;
    } else {
        uint32_t w[8] = {v.lo.x, v.lo.y, v.lo.z, v.lo.w, v.hi.x, v.hi.y, v.hi.z, v.hi.w};
        if (shift & 8u) {
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        }
        if (shift & 4u) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
        }
        if (shift & 2u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = w[i];
    }
}
template <int TYPE>
__device__ __forceinline__ void grad_floats(float (&f)[4], uint32_t a, uint32_t b)
{
    const float2 s = unpack2<TYPE>(a), t = unpack2<TYPE>(b);
    f[0] = s.x;
    f[1] = s.y;
    f[2] = t.x;
    f[3] = t.y;
}

// (dz is a workspace: 16-byte aligned rows)
__device__ __forceinline__ void grad_store(uint16_t* p, const uint32_t (&w)[4], int n)
{
    if (n == kGradCols) {
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kGradCols; ++i)
            if (i < n) p[i] = static_cast<uint16_t>(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
    }
}

template <int TYPE, bool GATED, int ACT, bool ALIGNED>
__global__ void __launch_bounds__(kGradThreads, 3) act_backward_kernel(const ActBackwardParams p)
{
    constexpr int kParts = GATED ? 2 : 1;
    constexpr bool kNeedZ = ACT != kActNone || GATED;
    __shared__ float sums[kParts][kGradRowThreads][kGradTileCols];
    griddep_wait();
    griddep_launch_dependents();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int first = blockIdx.x * kGradTileCols;
    const int c0 = first + tx * kGradCols;
    const int n = p.M - c0 < kGradCols ? p.M - c0 : kGradCols;
    const long long r0 = static_cast<long long>(blockIdx.y) * p.rows_per_chunk;
    const long long r1 = r0 + p.rows_per_chunk < p.n ? r0 + p.rows_per_chunk : p.n;
    float sum[kParts][kGradCols] = {};
    if (n > 0) {
        // kAhead rows' values are loaded before the first of them is worked on: with one row's
        // loads of a thread in flight HBM gave half its rate.
        constexpr int kAhead = (GATED ? 2 : 3) - (ALIGNED ? 0 : 1);
        auto shift_of = [](const uint16_t* q) { return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(q)) & 15u; };
        for (long long r = r0 + ty; r < r1; r += kAhead * kGradRowThreads) {
            GradValues<ALIGNED> vy[kAhead], vz[kAhead], vu[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const long long q = r + a * kGradRowThreads;
                if (q < r1) {
                    vy[a] = grad_load<ALIGNED>(p.dy + q * p.ld_dy + c0, n);
                    if (kNeedZ) vz[a] = grad_load<ALIGNED>(p.z[0] + q * p.ldz + c0, n);
                    if (GATED) vu[a] = grad_load<ALIGNED>(p.z[1] + q * p.ldz + c0, n);
                }
            }
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const long long q = r + a * kGradRowThreads;
                if (q >= r1) break;
                uint32_t wy[4], wz[4] = {}, wu[4] = {}, w0[4], w1[4];
                grad_words<ALIGNED>(wy, vy[a], shift_of(p.dy + q * p.ld_dy));
                if (kNeedZ) grad_words<ALIGNED>(wz, vz[a], shift_of(p.z[0] + q * p.ldz));
                if (GATED) grad_words<ALIGNED>(wu, vu[a], shift_of(p.z[1] + q * p.ldz));
                // Four values at a time.  Past a row's end: zeros, because the reciprocals of a group of
                // values go by their product and a value's last bits are not to depend on what lies there.
                if (kNeedZ && n < kGradCols) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) wz[i] = 2 * i + 1 < n ? wz[i] : 2 * i < n ? wz[i] & 0xFFFFu : 0u;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float dy[4], z[4], u[4], slope[4], d0[4], d1[4];
                    grad_floats<TYPE>(dy, wy[2 * h], wy[2 * h + 1]);
                    grad_floats<TYPE>(z, wz[2 * h], wz[2 * h + 1]);
                    grad_floats<TYPE>(u, wu[2 * h], wu[2 * h + 1]);
                    if (kNeedZ) act_values<ACT, true, 4>(z, slope);   // z becomes act(z)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        d0[i] = !kNeedZ ? dy[i] : GATED ? dy[i] * u[i] * slope[i] : dy[i] * slope[i];
                        d1[i] = GATED ? dy[i] * z[i] : 0.f;
                        sum[0][4 * h + i] += d0[i];
                        if (GATED) sum[kParts - 1][4 * h + i] += d1[i];
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        w0[2 * h + i] = pack2<TYPE>(d0[2 * i], d0[2 * i + 1]);
                        w1[2 * h + i] = pack2<TYPE>(d1[2 * i], d1[2 * i + 1]);
                    }
                }
                if (p.dz[0] != nullptr) {
                    grad_store(p.dz[0] + q * p.ld_dz + c0, w0, n);
                    if (GATED) grad_store(p.dz[1] + q * p.ld_dz + c0, w1, n);
                }
            }
        }
    }
    if (p.partial != nullptr) {
        // a thread's i-th column lies at i * 32 + tx
#pragma unroll
        for (int q = 0; q < kParts; ++q)
#pragma unroll
            for (int i = 0; i < kGradCols; ++i) sums[q][ty][i * 32 + tx] = sum[q][i];
        __syncthreads();
        for (int e = threadIdx.x; e < kParts * kGradTileCols; e += kGradThreads) {
            const int q = e / kGradTileCols, c = e % kGradTileCols;
            if (first + c >= p.M) continue;
            const int at = (c % kGradCols) * 32 + c / kGradCols;
            float v = 0.f;
#pragma unroll
            for (int y = 0; y < kGradRowThreads; ++y) v += sums[q][y][at];
            p.partial[(static_cast<long long>(blockIdx.y) * kParts + q) * p.M + first + c] = v;
        }
    }
}

// 32 columns a block, every eighth chunk a warp, the warps' sums in order.
template <int TYPE>
__global__ void __launch_bounds__(256)
    bias_grad_kernel(const float* __restrict__ partial, int chunks, int parts, int M, void* db0, void* db1, int f32,
                     int accumulate)
{
    __shared__ float sums[8][32];
    griddep_wait();
    griddep_launch_dependents();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long total = static_cast<long long>(parts) * M;
    const long long e = static_cast<long long>(blockIdx.x) * 32 + lane;
    float v = 0.f;
    if (e < total) {
#pragma unroll 8
        for (int i = w; i < chunks; i += 8) v += partial[i * total + e];
    }
    sums[w][lane] = v;
    __syncthreads();
    if (w != 0 || e >= total) return;
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += sums[i][lane];
    const int q = e >= M ? 1 : 0;
    const long long c = e - static_cast<long long>(q) * M;
    void* db = q == 0 ? db0 : db1;
    if (db == nullptr) return;
    if (f32) {
        float* o = static_cast<float*>(db) + c;
        *o = accumulate ? *o + v : v;
    } else {
        uint16_t* o = static_cast<uint16_t*>(db) + c;
        *o = to_16<TYPE>(accumulate ? to_f32<TYPE>(*o) + v : v);
    }
}

template <int TYPE, bool GATED, int ACT>
cudaError_t launch_act(const ActBackwardLaunch& a, const ActBackwardParams& p, bool aligned, cudaStream_t stream)
{
    const dim3 grid((a.M + kGradTileCols - 1) / kGradTileCols, a.chunks);
    auto kern = aligned ? act_backward_kernel<TYPE, GATED, ACT, true> : act_backward_kernel<TYPE, GATED, ACT, false>;
    return launch_kernel(kern, grid, dim3(kGradThreads), 0, stream, a.pdl, p);
}

template <int TYPE, bool GATED>
cudaError_t launch_act_switch(const ActBackwardLaunch& a, const ActBackwardParams& p, bool aligned, cudaStream_t stream)
{
    switch (a.act) {
    case kActRelu: return launch_act<TYPE, GATED, kActRelu>(a, p, aligned, stream);
    case kActGelu: return launch_act<TYPE, GATED, kActGelu>(a, p, aligned, stream);
    case kActGeluTanh: return launch_act<TYPE, GATED, kActGeluTanh>(a, p, aligned, stream);
    case kActSilu: return launch_act<TYPE, GATED, kActSilu>(a, p, aligned, stream);
    default: return launch_act<TYPE, GATED, kActNone>(a, p, aligned, stream);
    }
}

}  // namespace

// Chunks of tokens (a row of blocks each): one wave of the three blocks that fit on an SM, with no
// block left for a second (gated backward 1500 x 2731 x 1000: 46.8 us; 48.9 with eight blocks per SM,
// 4096 x 17408 x 5120: 1656 and 1672).  At least two rows per thread.
int act_backward_chunks(int n, int M, int num_sms)
{
    const long long cols = (M + kGradTileCols - 1) / kGradTileCols;
    long long chunks = 3LL * num_sms / cols;
    constexpr long long kLeast = 2 * kGradRowThreads;
    const long long most = (n + kLeast - 1) / kLeast;
    if (chunks > most) chunks = most;
    if (chunks > 512) chunks = 512;
    return static_cast<int>(chunks < 1 ? 1 : chunks);
}

int launch_act_backward(const ActBackwardLaunch& a, cudaStream_t stream, char* msg, size_t msg_len)
{
    ActBackwardParams p = {};
    p.n = a.n;
    p.M = a.M;
    p.rows_per_chunk = (a.n + a.chunks - 1) / a.chunks;
    p.ldz = a.ldz;
    p.dy = static_cast<const uint16_t*>(a.dy);
    p.ld_dy = a.ld_dy;
    p.ld_dz = a.ld_dz;
    p.partial = a.partial;
    // whole 16-byte units, the last one of a row (which may reach past it) included
    auto units = [&](const void* q, long long ld) {
        return q == nullptr || ((reinterpret_cast<uintptr_t>(q) | static_cast<uintptr_t>(ld * 2)) & 15u) == 0;
    };
    bool aligned = units(a.dy, a.ld_dy);
    for (int i = 0; i < 2; ++i) {
        p.z[i] = static_cast<const uint16_t*>(a.z[i]);
        p.dz[i] = static_cast<uint16_t*>(a.dz[i]);
        aligned = aligned && units(a.z[i], a.ldz);
    }
    cudaError_t e;
    if (a.type == kTypeBF16)
        e = a.gated ? launch_act_switch<kTypeBF16, true>(a, p, aligned, stream) : launch_act_switch<kTypeBF16, false>(a, p, aligned, stream);
    else
        e = a.gated ? launch_act_switch<kTypeF16, true>(a, p, aligned, stream) : launch_act_switch<kTypeF16, false>(a, p, aligned, stream);
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "element-wise backward launch failed: %s", cudaGetErrorString(e));
        return 1;
    }
    return 0;
}

int launch_bias_grad(const BiasGradLaunch& a, cudaStream_t stream, char* msg, size_t msg_len)
{
    const long long total = static_cast<long long>(a.parts) * a.M;
    const dim3 grid(static_cast<unsigned>((total + 31) / 32));
    auto kern = a.type == kTypeBF16 ? bias_grad_kernel<kTypeBF16> : bias_grad_kernel<kTypeF16>;
    const cudaError_t e = launch_kernel(kern, grid, dim3(256), 0, stream, a.pdl, a.partial, a.chunks, a.parts, a.M,
                                        a.db[0], a.db[1], a.f32 ? 1 : 0, a.accumulate ? 1 : 0);
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "bias gradient launch failed: %s", cudaGetErrorString(e));
        return 1;
    }
    return 0;
}

}  // namespace bsk
