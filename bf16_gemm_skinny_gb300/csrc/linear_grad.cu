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
    int act;
    int vec;   // 16-byte accesses allowed everywhere
};

template <int TYPE>
__device__ __forceinline__ void grad_load(float (&v)[kGradCols], const uint16_t* p, int n, bool vec)
{
    if (vec && n == kGradCols) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<TYPE>(u[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kGradCols; ++i) v[i] = i < n ? to_f32<TYPE>(p[i]) : 0.f;
    }
}

template <int TYPE>
__device__ __forceinline__ void grad_store(uint16_t* p, const float (&v)[kGradCols], int n, bool vec)
{
    if (vec && n == kGradCols) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack2<TYPE>(v[0], v[1]), pack2<TYPE>(v[2], v[3]),
                                                  pack2<TYPE>(v[4], v[5]), pack2<TYPE>(v[6], v[7]));
    } else {
#pragma unroll
        for (int i = 0; i < kGradCols; ++i)
            if (i < n) p[i] = to_16<TYPE>(v[i]);
    }
}

template <int TYPE, bool GATED, int ACT>
__global__ void __launch_bounds__(kGradThreads) act_backward_kernel(const ActBackwardParams p)
{
    constexpr int kParts = GATED ? 2 : 1;
    __shared__ float sums[kParts][kGradRowThreads][kGradTileCols];
    griddep_wait();
    griddep_launch_dependents();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c0 = blockIdx.x * kGradTileCols + tx * kGradCols;
    const int n = p.M - c0 < kGradCols ? p.M - c0 : kGradCols;
    const long long r0 = static_cast<long long>(blockIdx.y) * p.rows_per_chunk;
    const long long r1 = r0 + p.rows_per_chunk < p.n ? r0 + p.rows_per_chunk : p.n;
    const bool vec = p.vec != 0;
    float sum[kParts][kGradCols] = {};
    if (n > 0) {
#pragma unroll 2
        for (long long r = r0 + ty; r < r1; r += kGradRowThreads) {
            float dy[kGradCols], z[kGradCols], u[kGradCols];
            grad_load<TYPE>(dy, p.dy + r * p.ld_dy + c0, n, vec);
            if (ACT != kActNone || GATED) grad_load<TYPE>(z, p.z[0] + r * p.ldz + c0, n, vec);
            if (GATED) grad_load<TYPE>(u, p.z[1] + r * p.ldz + c0, n, vec);
            float d0[kGradCols], d1[kGradCols];
#pragma unroll
            for (int i = 0; i < kGradCols; ++i) {
                const float2 f = ACT != kActNone || GATED ? act_value_slope<ACT>(z[i]) : make_float2(0.f, 1.f);
                d0[i] = GATED ? dy[i] * u[i] * f.y : dy[i] * f.y;
                d1[i] = GATED ? dy[i] * f.x : 0.f;
                sum[0][i] += d0[i];
                if (GATED) sum[kParts - 1][i] += d1[i];
            }
            if (p.dz[0] != nullptr) {
                grad_store<TYPE>(p.dz[0] + r * p.ld_dz + c0, d0, n, vec);
                if (GATED) grad_store<TYPE>(p.dz[1] + r * p.ld_dz + c0, d1, n, vec);
            }
        }
    }
    if (p.partial != nullptr) {
#pragma unroll
        for (int q = 0; q < kParts; ++q)
#pragma unroll
            for (int i = 0; i < kGradCols; ++i) sums[q][ty][i * 32 + tx] = sum[q][i];
        __syncthreads();
        for (int e = threadIdx.x; e < kParts * kGradTileCols; e += kGradThreads) {
            const int q = e / kGradTileCols, c = e % kGradTileCols;
            const int col = blockIdx.x * kGradTileCols + c;
            if (col >= p.M) continue;
            float v = 0.f;
#pragma unroll
            for (int y = 0; y < kGradRowThreads; ++y) v += sums[q][y][(c % kGradCols) * 32 + c / kGradCols];
            p.partial[(static_cast<long long>(blockIdx.y) * kParts + q) * p.M + col] = v;
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
cudaError_t launch_act(const ActBackwardLaunch& a, const ActBackwardParams& p, cudaStream_t stream)
{
    const dim3 grid((a.M + kGradTileCols - 1) / kGradTileCols, a.chunks);
    return launch_kernel(act_backward_kernel<TYPE, GATED, ACT>, grid, dim3(kGradThreads), 0, stream, a.pdl, p);
}

template <int TYPE, bool GATED>
cudaError_t launch_act_switch(const ActBackwardLaunch& a, const ActBackwardParams& p, cudaStream_t stream)
{
    switch (a.act) {
    case kActRelu: return launch_act<TYPE, GATED, kActRelu>(a, p, stream);
    case kActGelu: return launch_act<TYPE, GATED, kActGelu>(a, p, stream);
    case kActGeluTanh: return launch_act<TYPE, GATED, kActGeluTanh>(a, p, stream);
    case kActSilu: return launch_act<TYPE, GATED, kActSilu>(a, p, stream);
    default: return launch_act<TYPE, GATED, kActNone>(a, p, stream);
    }
}

bool aligned(const void* p, long long ld)
{
    return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * 2)) & 15u) == 0;
}

}  // namespace

// Chunks of tokens: about four blocks per SM, each with a row per thread at least.
int act_backward_chunks(int n, int M, int num_sms)
{
    const long long cols = (M + kGradTileCols - 1) / kGradTileCols;
    long long chunks = (4LL * num_sms + cols - 1) / cols;
    const long long most = (n + kGradRowThreads - 1LL) / kGradRowThreads;
    if (chunks > most) chunks = most;
    if (chunks > 65535) chunks = 65535;
    return static_cast<int>(chunks < 1 ? 1 : chunks);
}

int launch_act_backward(const ActBackwardLaunch& a, cudaStream_t stream, char* msg, size_t msg_len)
{
    ActBackwardParams p = {};
    p.n = a.n;
    p.M = a.M;
    p.rows_per_chunk = (a.n + a.chunks - 1) / a.chunks;
    p.act = a.act;
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
    p.vec = vec;
    cudaError_t e;
    if (a.type == kTypeBF16)
        e = a.gated ? launch_act_switch<kTypeBF16, true>(a, p, stream) : launch_act_switch<kTypeBF16, false>(a, p, stream);
    else
        e = a.gated ? launch_act_switch<kTypeF16, true>(a, p, stream) : launch_act_switch<kTypeF16, false>(a, p, stream);
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
