// linear_grad.cu -- the element-wise part of the feed-forward layers' backward
// passes, and the bias gradients.
//
//   dz = dy act'(z);   gated: dg = dh u act'(g),  du = dh act(g)
//
// One pass over the tokens: every value is read once, FP32 inside, dz rounded
// once to the type, because it is an operand of the tensor cores' products next
// (2^-9 of each term in BF16, 2^-12 in FP16, at random: the gradients' sums see
// about as much as from their own rounding).  A bias gradient is the column sum
// of the unrounded dz: each thread keeps its columns' sums over its tokens, a
// block adds its threads' in a fixed order and leaves one FP32 row, a second
// kernel adds those rows in order.  No atomics: the same call gives the same bits.
// Bound: HBM (6 bytes read and 4 written per value of a gated layer).
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

// A thread's 8 columns of a block's 256: VEC: side by side (16-byte accesses), else 32
// apart, so that a warp's 2-byte accesses are to neighbouring addresses whatever the alignment.
struct GradValues {
    uint4 w;   // 8 values
};
template <bool VEC>
__device__ __forceinline__ GradValues grad_load(const uint16_t* p, int n)
{
    GradValues v;
    if (VEC && n == kGradCols) {
        v.w = *reinterpret_cast<const uint4*>(p);
    } else {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = 2 * i < n ? p[VEC ? 2 * i : 64 * i] : 0u;
            const uint32_t hi = 2 * i + 1 < n ? p[VEC ? 2 * i + 1 : 64 * i + 32] : 0u;
            u[i] = lo | hi << 16;
        }
        v.w = make_uint4(u[0], u[1], u[2], u[3]);
    }
    return v;
}
template <int TYPE>
__device__ __forceinline__ void grad_unpack(float (&f)[kGradCols], const GradValues& v)
{
    const uint32_t u[4] = {v.w.x, v.w.y, v.w.z, v.w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = unpack2<TYPE>(u[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}

template <int TYPE, bool VEC>
__device__ __forceinline__ void grad_store(uint16_t* p, const float (&v)[kGradCols], int n)
{
    if (VEC && n == kGradCols) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack2<TYPE>(v[0], v[1]), pack2<TYPE>(v[2], v[3]),
                                                  pack2<TYPE>(v[4], v[5]), pack2<TYPE>(v[6], v[7]));
    } else {
#pragma unroll
        for (int i = 0; i < kGradCols; ++i)
            if (i < n) p[VEC ? i : 32 * i] = to_16<TYPE>(v[i]);
    }
}

template <int TYPE, bool GATED, int ACT, bool VEC>
__global__ void __launch_bounds__(kGradThreads) act_backward_kernel(const ActBackwardParams p)
{
    constexpr int kParts = GATED ? 2 : 1;
    constexpr bool kNeedZ = ACT != kActNone || GATED;
    __shared__ float sums[kParts][kGradRowThreads][kGradTileCols];
    griddep_wait();
    griddep_launch_dependents();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int first = blockIdx.x * kGradTileCols;
    const int c0 = first + (VEC ? tx * kGradCols : tx);
    const int left = p.M - c0;
    const int n = VEC ? (left < kGradCols ? left : kGradCols) : (left + 31) / 32 < kGradCols ? (left + 31) / 32 : kGradCols;
    const long long r0 = static_cast<long long>(blockIdx.y) * p.rows_per_chunk;
    const long long r1 = r0 + p.rows_per_chunk < p.n ? r0 + p.rows_per_chunk : p.n;
    float sum[kParts][kGradCols] = {};
    if (left > 0) {
        // kAhead rows' values are loaded before the first of them is worked on: three loads a thread
        // in flight left HBM at half its rate.
        constexpr int kAhead = 3;
        for (long long r = r0 + ty; r < r1; r += kAhead * kGradRowThreads) {
            GradValues vy[kAhead], vz[kAhead], vu[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const long long q = r + a * kGradRowThreads;
                if (q < r1) {
                    vy[a] = grad_load<VEC>(p.dy + q * p.ld_dy + c0, n);
                    if (kNeedZ) vz[a] = grad_load<VEC>(p.z[0] + q * p.ldz + c0, n);
                    if (GATED) vu[a] = grad_load<VEC>(p.z[1] + q * p.ldz + c0, n);
                }
            }
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const long long q = r + a * kGradRowThreads;
                if (q >= r1) break;
                float dy[kGradCols], z[kGradCols], u[kGradCols], d0[kGradCols], d1[kGradCols];
                grad_unpack<TYPE>(dy, vy[a]);
                if (kNeedZ) grad_unpack<TYPE>(z, vz[a]);
                if (GATED) grad_unpack<TYPE>(u, vu[a]);
                float slope[kGradCols];
                if (kNeedZ) act_values<ACT, true, kGradCols>(z, slope);   // z becomes act(z)
#pragma unroll
                for (int i = 0; i < kGradCols; ++i) {
                    d0[i] = !kNeedZ ? dy[i] : GATED ? dy[i] * u[i] * slope[i] : dy[i] * slope[i];
                    d1[i] = GATED ? dy[i] * z[i] : 0.f;
                    sum[0][i] += d0[i];
                    if (GATED) sum[kParts - 1][i] += d1[i];
                }
                if (p.dz[0] != nullptr) {
                    grad_store<TYPE, VEC>(p.dz[0] + q * p.ld_dz + c0, d0, n);
                    if (GATED) grad_store<TYPE, VEC>(p.dz[1] + q * p.ld_dz + c0, d1, n);
                }
            }
        }
    }
    if (p.partial != nullptr) {
        // column e of the block's at [e % 8 or e / 32][...]: a thread's i-th column at i * 32 + tx
#pragma unroll
        for (int q = 0; q < kParts; ++q)
#pragma unroll
            for (int i = 0; i < kGradCols; ++i) sums[q][ty][i * 32 + tx] = sum[q][i];
        __syncthreads();
        for (int e = threadIdx.x; e < kParts * kGradTileCols; e += kGradThreads) {
            const int q = e / kGradTileCols, c = e % kGradTileCols;
            if (first + c >= p.M) continue;
            const int at = VEC ? (c % kGradCols) * 32 + c / kGradCols : c;
            float v = 0.f;
#pragma unroll
            for (int y = 0; y < kGradRowThreads; ++y) v += sums[q][y][at];
            p.partial[(static_cast<long long>(blockIdx.y) * kParts + q) * p.M + first + c] = v;
        }
    }
}

template <int TYPE>
__global__ void __launch_bounds__(256)
    bias_grad_kernel(const float* __restrict__ partial, int chunks, int parts, int M, void* db0, void* db1, int f32,
                     int accumulate)
{
    griddep_wait();
    griddep_launch_dependents();
    const long long e = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (e >= static_cast<long long>(parts) * M) return;
    const int q = static_cast<int>(e / M);
    const int c = static_cast<int>(e - static_cast<long long>(q) * M);
    float v = 0.f;
#pragma unroll 8
    for (int i = 0; i < chunks; ++i) v += partial[static_cast<long long>(i) * parts * M + e];
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
cudaError_t launch_act(const ActBackwardLaunch& a, const ActBackwardParams& p, bool vec, cudaStream_t stream)
{
    const dim3 grid((a.M + kGradTileCols - 1) / kGradTileCols, a.chunks);
    auto kern = vec ? act_backward_kernel<TYPE, GATED, ACT, true> : act_backward_kernel<TYPE, GATED, ACT, false>;
    return launch_kernel(kern, grid, dim3(kGradThreads), 0, stream, a.pdl, p);
}

template <int TYPE, bool GATED>
cudaError_t launch_act_switch(const ActBackwardLaunch& a, const ActBackwardParams& p, bool vec, cudaStream_t stream)
{
    switch (a.act) {
    case kActRelu: return launch_act<TYPE, GATED, kActRelu>(a, p, vec, stream);
    case kActGelu: return launch_act<TYPE, GATED, kActGelu>(a, p, vec, stream);
    case kActGeluTanh: return launch_act<TYPE, GATED, kActGeluTanh>(a, p, vec, stream);
    case kActSilu: return launch_act<TYPE, GATED, kActSilu>(a, p, vec, stream);
    default: return launch_act<TYPE, GATED, kActNone>(a, p, vec, stream);
    }
}

bool aligned(const void* p, long long ld)
{
    return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * 2)) & 15u) == 0;
}

}  // namespace

// Chunks of tokens (a row of blocks each): some 24 blocks per SM, so that the last wave counts for
// little, and at least 16 tokens a block.  4096 x 17408 gated: 244 us with 4 blocks per SM, of which 3
// fit at once.
int act_backward_chunks(int n, int M, int num_sms)
{
    const long long cols = (M + kGradTileCols - 1) / kGradTileCols;
    long long chunks = (24LL * num_sms + cols - 1) / cols;
    const long long most = (n + 2LL * kGradRowThreads - 1) / (2LL * kGradRowThreads);
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
    bool vec = aligned(a.dy, a.ld_dy);
    for (int i = 0; i < 2; ++i) {
        p.z[i] = static_cast<const uint16_t*>(a.z[i]);
        p.dz[i] = static_cast<uint16_t*>(a.dz[i]);
        if (a.z[i] != nullptr) vec = vec && aligned(a.z[i], a.ldz);
        if (a.dz[i] != nullptr) vec = vec && aligned(a.dz[i], a.ld_dz);
    }
    cudaError_t e;
    if (a.type == kTypeBF16)
        e = a.gated ? launch_act_switch<kTypeBF16, true>(a, p, vec, stream) : launch_act_switch<kTypeBF16, false>(a, p, vec, stream);
    else
        e = a.gated ? launch_act_switch<kTypeF16, true>(a, p, vec, stream) : launch_act_switch<kTypeF16, false>(a, p, vec, stream);
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "element-wise backward launch failed: %s", cudaGetErrorString(e));
        return 1;
    }
    return 0;
}

int launch_bias_grad(const BiasGradLaunch& a, cudaStream_t stream, char* msg, size_t msg_len)
{
    const long long total = static_cast<long long>(a.parts) * a.M;
    const dim3 grid(static_cast<unsigned>((total + 255) / 256));
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
