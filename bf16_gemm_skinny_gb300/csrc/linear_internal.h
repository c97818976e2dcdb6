// linear_internal.h -- the products of the feed-forward layer calls as their
// kernels see them, and the launchers of the linear_*.cu files (not part of the
// C ABI).
//
// Every product here leaves a row-major result: rows along the accumulator's
// TMEM lanes, columns along its registers.
//   linear   out[t, j] = act(sum_k x[t, k] W[j, k] + b[j]) + r[t, j]
//   gated    out[t, j] = act(g) * u,  g and u two such sums (Wg and Wu)
//   gradients         dx[t, k] = sum over the sources s and features j of dz_s[t, j] W_s[j, k],
//                     dW_s[j, k] (+)= sum_t dz_s[t, j] x[t, k],  one launch for both
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace bsk {

enum ValueType : int { kTypeBF16 = 0, kTypeF16 = 1 };
enum Activation : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };
enum LinearMode : int { kModeLinear = 0, kModeGated = 1, kModeGrad = 2 };

// One launch.  Operands are 16-bit, 16-byte aligned, with leading dimensions
// (elements) that are multiples of 8.
struct LinearLaunch {
    int mode = kModeLinear;
    int type = kTypeBF16;
    int parts = 1;                 // sources: 2 in gated layers
    int n = 0, M = 0, K = 0;       // tokens, output and input features
    const void* x = nullptr;       // [n, K]
    long long ldx = 0;
    const void* W[2] = {nullptr, nullptr};   // [M, K]
    long long ldw = 0;
    // forward
    void* out = nullptr;           // [n, M]
    long long ldo = 0;
    int act = kActNone;
    const void* bias[2] = {nullptr, nullptr};
    const void* residual = nullptr;
    long long ldr = 0;
    void* keep[2] = {nullptr, nullptr};   // pre-activations, rounded
    long long ldk = 0;
    // gradients
    const void* dz[2] = {nullptr, nullptr};   // [n, M]
    long long ldz = 0;
    // rows of the operand may be read up to the next multiple of 64 elements (its values are not used)
    bool x_padded = false, w_padded = false, z_padded = false;
    void* dx = nullptr;            // [n, K], NULL: not wanted
    long long ld_dx = 0;
    void* dW[2] = {nullptr, nullptr};   // [M, K], NULL: not wanted
    long long ld_dw = 0;
    bool grad_f32 = false, accumulate = false;
    const float* db_partial = nullptr;   // chunks x parts x M sums to add up into db, or NULL
    int db_chunks = 0;
    void* db[2] = {nullptr, nullptr};

    int num_sms = 1;
    int* status = nullptr;
    unsigned long long wait_limit_ns = 2000000000ull;
    bool pdl = true;
    // plan_linear()'s choice
    bool pair = false;             // 256-row tiles on CTA pairs, else 128-row tiles
    int bn = 128;                  // accumulator columns per tile (gated: both halves)
    int split = 1;                 // one-CTA tiles: CTAs of a cluster that share a tile's k loop
    int group_m = 16;              // tile rows that neighbouring CTAs go through column by column
};

constexpr int kFewRows = 64;   // tokens up to which the weights' stream is the bound of a forward pass

// Shared memory of a product's kernel: in all, of the barriers and of the staging buffers; of a k-block.
constexpr int kLinSmemBytes = 232448;
constexpr int kLinBarBytes = 512 + 1024;   // barriers, and the bias gradients' sums
constexpr int kLinStageBytes = 32768;
inline int linear_block_bytes(const LinearLaunch& g, bool pair, int bn)
{
    const int a_rows = pair || g.mode == kModeGrad || g.n >= 128 ? 128 : (g.n + 7) / 8 * 8;
    return (a_rows + (pair ? bn / 2 : bn)) * 128;
}
inline int linear_ring_room(bool few, bool staged)
{
    return (few ? kLinSmemBytes / 2 - 1024 : kLinSmemBytes) - 1024 - kLinBarBytes - (staged ? kLinStageBytes : 0);
}
// k-blocks per turn of the MMA warp.  A wait, a commit and the issue of its MMAs cost some 150 ns a
// turn, more than a small tile's MMAs of a k-block take (250 ns a k-block for every width up to 128):
// two or four k-blocks a turn, as far as the ring keeps a few turns.  Forward on pairs of 256 columns one: with
// two, 8192 x 8192 x 1024 took 82.9 us instead of 80.8, and longer k loops the same (4096 x 5120 x 17408 393 us,
// gated 4096 x 17408 x 5120 708).  Gradients there two (8192 x 5120 x 4096 396 us, with one 426).
inline int linear_group(const LinearLaunch& g, bool pair, int bn, bool few, bool staged)
{
    const int fit = linear_ring_room(few, staged) / linear_block_bytes(g, pair, bn);
    return pair && g.mode != kModeGrad && bn == 256 ? 1 : fit >= 16 ? 4 : fit >= 6 ? 2 : 1;
}

// Fills in the plan (tile width, kernel, split) from the sizes; options override it.
void plan_linear(LinearLaunch& g);
int launch_linear(const LinearLaunch& g, cudaStream_t stream, char* msg, size_t msg_len);
int launch_linear_bf16(const LinearLaunch& g, cudaStream_t stream, char* msg, size_t msg_len);
int launch_linear_f16(const LinearLaunch& g, cudaStream_t stream, char* msg, size_t msg_len);

// The element-wise part of the backward passes, and the sums over the tokens:
//   gated:  dz[0] = dy * u * act'(g),  dz[1] = dy * act(g)   (z[0] = g, z[1] = u)
//   else:   dz[0] = dy * act'(z[0])
// rounded to the type ([n, M], ld_dz apart; NULL: not stored).  With `partial`
// (chunks x parts x M floats) the columns' FP32 sums over each chunk of tokens
// go there.
struct ActBackwardLaunch {
    int type = kTypeBF16;
    bool gated = false;
    int act = kActNone;
    int n = 0, M = 0;
    const void* z[2] = {nullptr, nullptr};
    long long ldz = 0;
    const void* dy = nullptr;
    long long ld_dy = 0;
    void* dz[2] = {nullptr, nullptr};
    long long ld_dz = 0;
    float* partial = nullptr;
    int chunks = 1;
    bool pdl = true;
};
int act_backward_chunks(int n, int M, int num_sms);
int launch_act_backward(const ActBackwardLaunch& a, cudaStream_t stream, char* msg, size_t msg_len);

// db[p][j] (+)= sum over the chunks, in order, of partial[chunk][p][j].
struct BiasGradLaunch {
    int type = kTypeBF16;
    int parts = 1, M = 0, chunks = 1;
    const float* partial = nullptr;
    void* db[2] = {nullptr, nullptr};
    bool f32 = false, accumulate = false, pdl = true;
};
int launch_bias_grad(const BiasGradLaunch& a, cudaStream_t stream, char* msg, size_t msg_len);

}  // namespace bsk
