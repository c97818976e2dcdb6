// linear_api.cu -- the C entry points of the feed-forward layer calls: argument
// checks, plan, workspace, launches.  No compute here.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "bsk.h"
#include "bsk_internal.h"
#include "bsk_tuning.h"
#include "kv_internal.h"
#include "linear_internal.h"

namespace {

int fail(int status, const char* fmt, ...)
{
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    bsk::record_error(msg);
    return status;
}

int fail_cuda(cudaError_t e, const char* what)
{
    return fail(BSK_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// Stream-ordered workspace in 256-byte aligned parts, freed in stream order after
// use.  From the library's pool, whose memory stays mapped; a capturing stream
// takes the default pool, whose allocations become nodes of the graph.
class Workspace {
  public:
    explicit Workspace(cudaStream_t stream) : s_(stream) {}
    Workspace(const Workspace&) = delete;
    Workspace& operator=(const Workspace&) = delete;
    ~Workspace()
    {
        if (ptr_ != nullptr) cudaFreeAsync(ptr_, s_);
    }
    // Notes a part; its offset.
    size_t part(size_t bytes)
    {
        const size_t at = bytes_;
        bytes_ += (bytes + 255) / 256 * 256;
        return at;
    }
    int take()
    {
        if (bytes_ == 0) return BSK_OK;
        cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
        cudaError_t e = cudaStreamIsCapturing(s_, &capture);
        cudaMemPool_t pool = nullptr;
        if (e == cudaSuccess) {
            if (capture != cudaStreamCaptureStatusNone || bsk::api_pool(&pool) != BSK_OK)
                e = cudaMallocAsync(&ptr_, bytes_, s_);
            else
                e = cudaMallocFromPoolAsync(&ptr_, bytes_, pool, s_);
        }
        if (e == cudaSuccess) return BSK_OK;
        cudaGetLastError();
        ptr_ = nullptr;
        return fail(BSK_ERR_NO_MEMORY, "cudaMallocAsync(%zu bytes) for a workspace failed: %s", bytes_,
                    cudaGetErrorString(e));
    }
    uint8_t* at(size_t offset) const { return static_cast<uint8_t*>(ptr_) + offset; }

  private:
    void* ptr_ = nullptr;
    size_t bytes_ = 0;
    cudaStream_t s_;
};

// A matrix argument: `rows` rows of `width` elements of `size` bytes, `ld` elements apart.
struct Matrix {
    const char* name;
    const void* p;
    long long rows, width, ld;
    int size;

    long long bytes() const { return p != nullptr && rows > 0 && width > 0 ? ((rows - 1) * ld + width) * size : 0; }
};

// Whether two matrices share a byte.  Parts of the same wider rows (one distance between rows, each
// within its own columns) share none; otherwise what lies between the first and the last row's end counts.
bool overlap(const Matrix& a, const Matrix& b)
{
    const long long ab = a.bytes(), bb = b.bytes();
    if (ab <= 0 || bb <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    if (!(a0 < b0 + static_cast<uintptr_t>(bb) && b0 < a0 + static_cast<uintptr_t>(ab))) return false;
    const long long pitch = a.ld * a.size;
    if (pitch != b.ld * b.size) return true;
    const bool b_first = b0 < a0;
    const long long apart = static_cast<long long>(b_first ? a0 - b0 : b0 - a0) % pitch;
    return !((b_first ? b : a).width * (b_first ? b : a).size <= apart && apart + (b_first ? a : b).width * (b_first ? a : b).size <= pitch);
}

// Outputs overlap neither an input nor each other.  `same`: index of the one input that may be
// the first output itself (same address and stride), or -1.  An index and not an address: another operand
// may lie where that input does, and is read while the output is written.
int check_overlaps(const Matrix* out, int outs, const Matrix* in, int ins, int same = -1)
{
    for (int i = 0; i < outs; ++i) {
        for (int j = 0; j < ins; ++j) {
            if (i == 0 && j == same && in[j].p == out[0].p && in[j].ld == out[0].ld) continue;
            if (overlap(out[i], in[j])) return fail(BSK_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, in[j].name);
        }
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return fail(BSK_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, out[j].name);
    }
    return BSK_OK;
}

// Alignment to the element, and a stride that holds a row.
int check_matrix(const Matrix& m)
{
    if (m.p == nullptr) return BSK_OK;
    if (reinterpret_cast<uintptr_t>(m.p) % static_cast<unsigned>(m.size) != 0)
        return fail(BSK_ERR_INVALID_ARG, "%s is not aligned to its elements (%d bytes)", m.name, m.size);
    if (m.ld < (m.width > 1 ? m.width : 1))
        return fail(BSK_ERR_INVALID_ARG, "the stride of %s (%lld) must be at least %lld", m.name, m.ld,
                    m.width > 1 ? m.width : 1LL);
    return BSK_OK;
}

int check_common(int type, int activation, int M, int K, int n)
{
    if (type != BSK_TYPE_BF16 && type != BSK_TYPE_F16)
        return fail(BSK_ERR_INVALID_ARG, "type must be BSK_TYPE_BF16 or BSK_TYPE_F16 (got %d)", type);
    if (activation < BSK_ACT_NONE || activation > BSK_ACT_SILU)
        return fail(BSK_ERR_INVALID_ARG, "unknown activation %d", activation);
    if (M < 0 || K < 0 || n < 0) return fail(BSK_ERR_INVALID_ARG, "negative size (M=%d K=%d n=%d)", M, K, n);
    const long long big = 0x7FFFFC00LL;   // tile coordinates stay in 32 bits
    if (M > big || K > big || n > big) return fail(BSK_ERR_INVALID_ARG, "sizes must be at most 2^31 - 1024");
    return BSK_OK;
}

bool direct(const void* p, long long ld) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0; }

// Operands that the TMA unit cannot read where they are (base not 16-byte
// aligned, or rows not a multiple of 16 bytes apart), to be copied to padded rows.
class Packer {
  public:
    explicit Packer(Workspace& ws) : ws_(ws) {}
    // Before take(): plans the copy of an operand, if it needs one.
    void plan(const void** p, long long* ld, long long rows, long long width)
    {
        if (!direct(*p, *ld)) force(p, ld, rows, width);
    }
    // Plans the copy of an operand, whether or not it needs one.
    void force(const void** p, long long* ld, long long rows, long long width)
    {
        Item& i = items_[n_++];
        i.p = p;
        i.ld = ld;
        i.rows = rows;
        i.width = width;
        i.padded = (width + 63) / 64 * 64;
        i.offset = ws_.part(static_cast<size_t>(rows) * static_cast<size_t>(i.padded) * 2);
    }
    // After take(): enqueues the copies and points the operands at them.
    int run(int sms, bool pdl, int* status, unsigned long long limit_ns, cudaStream_t s)
    {
        char msg[256] = "";
        bsk::PackCopy c[kMost];
        for (int i = 0; i < n_; ++i) {
            const Item& t = items_[i];
            c[i] = {*t.p, *t.ld * 2, ws_.at(t.offset), t.padded * 2, t.width * 2, t.rows};
        }
        if (n_ > 0 && bsk::launch_pack(c, n_, sms, pdl, status, limit_ns, s, msg, sizeof(msg)))
            return fail(BSK_ERR_CUDA, "%s", msg);
        for (int i = 0; i < n_; ++i) {   // (weights share one stride: set after all were read)
            *items_[i].p = ws_.at(items_[i].offset);
            *items_[i].ld = items_[i].padded;
        }
        return BSK_OK;
    }

  private:
    struct Item {
        const void** p;
        long long* ld;
        long long rows, width, padded;
        size_t offset;
    };
    Workspace& ws_;
    static constexpr int kMost = bsk::kPackJobs;   // x and both weights, or x, W and dy
    Item items_[kMost];
    int n_ = 0;
};

// What every launch of a call needs from the device and the options.
struct Context {
    int sms = 0;
    int* status = nullptr;
    unsigned long long limit_ns = 2000000000ull;
    bool pdl = true;
    cudaStream_t s = nullptr;

    int prepare(void* stream)
    {
        s = static_cast<cudaStream_t>(stream);
        const int st = bsk::api_prepare(&sms, &status);
        if (st != BSK_OK) return st;
        const long long us = bsk_get_option(BSK_OPT_WAIT_LIMIT_US);
        if (us > 0) limit_ns = static_cast<unsigned long long>(us) * 1000ull;
        pdl = bsk_get_option(BSK_OPT_PDL) != 1;
        return BSK_OK;
    }
    int run(bsk::LinearLaunch& g) const
    {
        g.num_sms = sms;
        g.status = status;
        g.wait_limit_ns = limit_ns;
        g.pdl = pdl;
        bsk::plan_linear(g);
        char msg[512] = "";
        if (bsk::launch_linear(g, s, msg, sizeof(msg))) return fail(BSK_ERR_CUDA, "%s", msg);
        return BSK_OK;
    }
};

struct ForwardArgs {
    int type;
    bool gated;
    const uint16_t* W[2];
    long long w_stride;
    const uint16_t* x;
    long long x_stride;
    const uint16_t* bias[2];
    const uint16_t* residual;
    long long r_stride;
    uint16_t* out;
    long long out_stride;
    uint16_t* keep[2];
    long long keep_stride;
    int M, K, n, activation;
};

// *launched: the stream has work of this call.
int enqueue_forward(const ForwardArgs& a, void* stream, bool* launched)
{
    *launched = false;
    int st = check_common(a.type, a.activation, a.M, a.K, a.n);
    if (st != BSK_OK) return st;
    const int parts = a.gated ? 2 : 1;
    const Matrix out[3] = {{a.gated ? "h" : "y", a.out, a.n, a.M, a.out_stride, 2},
                           {a.gated ? "g" : "z", a.keep[0], a.n, a.M, a.keep_stride, 2},
                           {"u", a.gated ? a.keep[1] : nullptr, a.n, a.M, a.keep_stride, 2}};
    const Matrix in[6] = {{"x", a.x, a.n, a.K, a.x_stride, 2},
                          {a.gated ? "Wg" : "W", a.W[0], a.M, a.K, a.w_stride, 2},
                          {"Wu", a.gated ? a.W[1] : nullptr, a.M, a.K, a.w_stride, 2},
                          {a.gated ? "bias_g" : "bias", a.bias[0], 1, a.M, a.M + 1LL, 2},
                          {"bias_u", a.gated ? a.bias[1] : nullptr, 1, a.M, a.M + 1LL, 2},
                          {"residual", a.residual, a.n, a.M, a.r_stride, 2}};
    for (const Matrix& m : out)
        if ((st = check_matrix(m)) != BSK_OK) return st;
    for (const Matrix& m : in)
        if ((st = check_matrix(m)) != BSK_OK) return st;
    if (a.M == 0 || a.n == 0) return BSK_OK;
    if (a.out == nullptr) return fail(BSK_ERR_INVALID_ARG, "%s is NULL", out[0].name);
    if (a.K > 0)
        for (int i = 0; i < parts + 1; ++i)
            if (in[i].p == nullptr) return fail(BSK_ERR_INVALID_ARG, "%s is NULL", in[i].name);
    if (a.gated && (a.keep[0] == nullptr) != (a.keep[1] == nullptr))
        return fail(BSK_ERR_INVALID_ARG, "g and u are kept together: pass both or neither");
    if ((st = check_overlaps(out, 3, in, 6, 5)) != BSK_OK) return st;   // (the residual)
    if (((a.M + 15LL) / 16) * ((a.n + 127LL) / 128) > INT_MAX) return fail(BSK_ERR_INVALID_ARG, "problem too large");

    Context ctx;
    if ((st = ctx.prepare(stream)) != BSK_OK) return st;
    *launched = true;
    bsk::LinearLaunch g;
    g.mode = a.gated ? bsk::kModeGated : bsk::kModeLinear;
    g.type = a.type;
    g.parts = parts;
    g.n = a.n;
    g.M = a.M;
    g.K = a.K;
    g.x = a.x;
    g.ldx = a.x_stride;
    g.ldw = a.w_stride;
    g.out = a.out;
    g.ldo = a.out_stride;
    g.act = a.activation;
    g.residual = a.residual;
    g.ldr = a.r_stride;
    g.ldk = a.keep_stride;
    for (int i = 0; i < parts; ++i) {
        g.W[i] = a.W[i];
        g.bias[i] = a.bias[i];
        g.keep[i] = a.keep[i];
    }
    Workspace ws(ctx.s);
    if (a.K == 0) {
        // an empty sum: the same product over 8 zeros
        const size_t bytes = static_cast<size_t>(a.n > a.M ? a.n : a.M) * 16;
        const size_t at = ws.part(bytes);
        if ((st = ws.take()) != BSK_OK) return st;
        const cudaError_t e = cudaMemsetAsync(ws.at(at), 0, bytes, ctx.s);
        if (e != cudaSuccess) return fail_cuda(e, "cudaMemsetAsync");
        g.x = g.W[0] = ws.at(at);
        if (a.gated) g.W[1] = g.W[0];
        g.ldx = g.ldw = g.K = 8;
        return ctx.run(g);
    }
    Packer pack(ws);
    pack.plan(&g.x, &g.ldx, a.n, a.K);
    // the weights share a stride: if one needs a copy, both get one
    const bool w_direct = direct(g.W[0], g.ldw) && (!a.gated || direct(g.W[1], g.ldw));
    if (!w_direct)
        for (int i = 0; i < parts; ++i) pack.force(&g.W[i], &g.ldw, a.M, a.K);
    if ((st = ws.take()) != BSK_OK) return st;
    if ((st = pack.run(ctx.sms, ctx.pdl, ctx.status, ctx.limit_ns, ctx.s)) != BSK_OK) return st;
    return ctx.run(g);
}

struct BackwardArgs {
    int type;
    bool gated;
    const uint16_t* W[2];
    long long w_stride;
    const uint16_t* x;
    long long x_stride;
    const uint16_t* z[2];
    long long z_stride;
    const uint16_t* dy;
    long long dy_stride;
    uint16_t* dx;
    long long dx_stride;
    void* dW[2];
    long long dw_stride;
    void* db[2];
    int grad_type, accumulate, M, K, n, activation;
};

int enqueue_backward(const BackwardArgs& a, void* stream, bool* launched)
{
    *launched = false;
    int st = check_common(a.type, a.activation, a.M, a.K, a.n);
    if (st != BSK_OK) return st;
    if (a.grad_type != BSK_GRAD_F32 && a.grad_type != BSK_GRAD_16)
        return fail(BSK_ERR_INVALID_ARG, "grad_type must be BSK_GRAD_F32 or BSK_GRAD_16 (got %d)", a.grad_type);
    if (a.accumulate != 0 && a.accumulate != 1)
        return fail(BSK_ERR_INVALID_ARG, "accumulate must be 0 or 1 (got %d)", a.accumulate);
    const int parts = a.gated ? 2 : 1;
    const int gs = a.grad_type == BSK_GRAD_F32 ? 4 : 2;
    const Matrix out[5] = {{"dx", a.dx, a.n, a.K, a.dx_stride, 2},
                           {a.gated ? "dWg" : "dW", a.dW[0], a.M, a.K, a.dw_stride, gs},
                           {"dWu", a.dW[1], a.M, a.K, a.dw_stride, gs},
                           {a.gated ? "dbias_g" : "dbias", a.db[0], 1, a.M, a.M + 1LL, gs},
                           {"dbias_u", a.db[1], 1, a.M, a.M + 1LL, gs}};
    const Matrix in[6] = {{a.gated ? "Wg" : "W", a.W[0], a.M, a.K, a.w_stride, 2},
                          {"Wu", a.W[1], a.M, a.K, a.w_stride, 2},
                          {"x", a.x, a.n, a.K, a.x_stride, 2},
                          {a.gated ? "g" : "z", a.z[0], a.n, a.M, a.z_stride, 2},
                          {"u", a.z[1], a.n, a.M, a.z_stride, 2},
                          {a.gated ? "dh" : "dy", a.dy, a.n, a.M, a.dy_stride, 2}};
    for (const Matrix& m : out)
        if ((st = check_matrix(m)) != BSK_OK) return st;
    for (const Matrix& m : in)
        if ((st = check_matrix(m)) != BSK_OK) return st;
    if (a.gated && (a.dW[0] == nullptr) != (a.dW[1] == nullptr))
        return fail(BSK_ERR_INVALID_ARG, "dWg and dWu are computed together: pass both or neither");
    const bool want_dx = a.dx != nullptr && a.n > 0 && a.K > 0;
    const bool want_dw = a.dW[0] != nullptr && a.M > 0 && a.K > 0;
    const bool want_db = (a.db[0] != nullptr || a.db[1] != nullptr) && a.M > 0;
    if (!want_dx && !want_dw && !want_db) return BSK_OK;
    const bool need_z = a.gated || a.activation != BSK_ACT_NONE;
    if (a.n > 0 && a.M > 0) {
        if (a.dy == nullptr) return fail(BSK_ERR_INVALID_ARG, "%s is NULL", in[5].name);
        if (need_z && a.z[0] == nullptr) return fail(BSK_ERR_INVALID_ARG, "%s is NULL", in[3].name);
        if (a.gated && a.z[1] == nullptr) return fail(BSK_ERR_INVALID_ARG, "u is NULL");
        if (want_dx && (a.W[0] == nullptr || (a.gated && a.W[1] == nullptr)))
            return fail(BSK_ERR_INVALID_ARG, "%s is NULL", a.W[0] == nullptr ? in[0].name : "Wu");
        if (want_dw && a.x == nullptr) return fail(BSK_ERR_INVALID_ARG, "x is NULL");
    }
    if ((st = check_overlaps(out, 5, in, 6)) != BSK_OK) return st;
    const long long most_tiles = 0x7FFFFFFFLL;
    if (((a.n + 127LL) / 128) * ((a.K + 63LL) / 64) > most_tiles || 2 * ((a.M + 127LL) / 128) * ((a.K + 63LL) / 64) > most_tiles)
        return fail(BSK_ERR_INVALID_ARG, "problem too large");

    Context ctx;
    if ((st = ctx.prepare(stream)) != BSK_OK) return st;
    *launched = true;
    cudaError_t e = cudaSuccess;
    if (a.M == 0) {   // dx is an empty sum
        e = cudaMemset2DAsync(a.dx, static_cast<size_t>(a.dx_stride) * 2, 0, static_cast<size_t>(a.K) * 2, a.n, ctx.s);
        return e == cudaSuccess ? BSK_OK : fail_cuda(e, "cudaMemset2DAsync");
    }
    if (a.n == 0) {   // so are the weights' and biases' gradients
        for (int i = 0; i < parts && a.accumulate == 0 && e == cudaSuccess; ++i) {
            if (want_dw)
                e = cudaMemset2DAsync(a.dW[i], static_cast<size_t>(a.dw_stride) * gs, 0, static_cast<size_t>(a.K) * gs, a.M, ctx.s);
            if (a.db[i] != nullptr && e == cudaSuccess) e = cudaMemsetAsync(a.db[i], 0, static_cast<size_t>(a.M) * gs, ctx.s);
        }
        return e == cudaSuccess ? BSK_OK : fail_cuda(e, "cudaMemsetAsync");
    }

    // dz: dy itself without an activation, else computed into the workspace
    Workspace ws(ctx.s);
    const bool products = want_dx || want_dw;
    const bool make_dz = need_z && products;
    const void* dz[2] = {a.dy, nullptr};
    long long ld_dz = a.dy_stride;
    size_t dz_at[2] = {0, 0};
    if (make_dz) {
        ld_dz = (a.M + 63LL) / 64 * 64;
        for (int i = 0; i < parts; ++i) dz_at[i] = ws.part(static_cast<size_t>(a.n) * static_cast<size_t>(ld_dz) * 2);
    }
    const int chunks = bsk::act_backward_chunks(a.n, a.M, ctx.sms);
    const size_t partial_at = want_db ? ws.part(static_cast<size_t>(chunks) * parts * static_cast<size_t>(a.M) * 4) : 0;
    const void* x = a.x;
    long long ldx = a.x_stride;
    const void* W[2] = {a.W[0], a.W[1]};
    long long ldw = a.w_stride;
    Packer pack(ws);
    if (want_dw) pack.plan(&x, &ldx, a.n, a.K);
    if (want_dx && (!direct(W[0], ldw) || (a.gated && !direct(W[1], ldw))))
        for (int i = 0; i < parts; ++i) pack.force(&W[i], &ldw, a.M, a.K);
    if (!make_dz && products) pack.plan(&dz[0], &ld_dz, a.n, a.M);
    if ((st = ws.take()) != BSK_OK) return st;
    char msg[512] = "";
    if (make_dz || want_db) {
        bsk::ActBackwardLaunch l;
        l.type = a.type;
        l.gated = a.gated;
        l.act = a.activation;
        l.n = a.n;
        l.M = a.M;
        l.ldz = a.z_stride;
        l.dy = a.dy;
        l.ld_dy = a.dy_stride;
        l.ld_dz = ld_dz;
        for (int i = 0; i < parts; ++i) {
            l.z[i] = need_z ? a.z[i] : nullptr;
            if (make_dz) dz[i] = l.dz[i] = ws.at(dz_at[i]);
        }
        l.partial = want_db ? reinterpret_cast<float*>(ws.at(partial_at)) : nullptr;
        l.chunks = chunks;
        l.pdl = ctx.pdl;
        if (bsk::launch_act_backward(l, ctx.s, msg, sizeof(msg))) return fail(BSK_ERR_CUDA, "%s", msg);
    }
    const float* partial = want_db ? reinterpret_cast<const float*>(ws.at(partial_at)) : nullptr;
    if (!products) {   // the bias gradients alone
        bsk::BiasGradLaunch b;
        b.type = a.type;
        b.parts = parts;
        b.M = a.M;
        b.chunks = chunks;
        b.partial = partial;
        b.db[0] = a.db[0];
        b.db[1] = a.db[1];
        b.f32 = gs == 4;
        b.accumulate = a.accumulate != 0;
        b.pdl = ctx.pdl;
        if (bsk::launch_bias_grad(b, ctx.s, msg, sizeof(msg))) return fail(BSK_ERR_CUDA, "%s", msg);
        return BSK_OK;
    }
    if ((st = pack.run(ctx.sms, ctx.pdl, ctx.status, ctx.limit_ns, ctx.s)) != BSK_OK) return st;
    bsk::LinearLaunch g;
    g.mode = bsk::kModeGrad;
    g.type = a.type;
    g.parts = parts;
    g.n = a.n;
    g.M = a.M;
    g.K = a.K;
    g.x = x;
    g.ldx = ldx;
    g.ldw = ldw;
    g.ldz = ld_dz;
    g.x_padded = x != a.x;   // copies and dz have rows of whole multiples of 64
    g.w_padded = W[0] != a.W[0];
    g.z_padded = dz[0] != a.dy;
    g.dx = want_dx ? a.dx : nullptr;
    g.ld_dx = a.dx_stride;
    g.ld_dw = a.dw_stride;
    g.grad_f32 = gs == 4;
    g.accumulate = a.accumulate != 0;
    g.db_partial = partial;
    g.db_chunks = chunks;
    for (int i = 0; i < parts; ++i) {
        g.W[i] = W[i];
        g.dz[i] = dz[i];
        g.dW[i] = want_dw ? a.dW[i] : nullptr;
        g.db[i] = a.db[i];
    }
    if ((st = ctx.run(g)) != BSK_OK) return st;
    return BSK_OK;
}

// The blocking form of a call: the stream's work is done, its errors reported.
template <typename Args>
int blocking(int (*enqueue)(const Args&, void*, bool*), const Args& a, void* stream)
{
    bool launched = false;
    const int st = enqueue(a, stream, &launched);
    return st != BSK_OK || !launched ? st : bsk::api_sync_and_check(static_cast<cudaStream_t>(stream));
}
template <typename Args>
int only_enqueue(int (*enqueue)(const Args&, void*, bool*), const Args& a, void* stream)
{
    bool launched = false;
    return enqueue(a, stream, &launched);
}

}  // namespace

namespace bsk {

// The tile, the kernel and the split of a launch: the least estimated time (us).
//
// The estimates are fitted to some 9000 timings on GB300, back to back (forward calls of 1 to 8192 tokens, 64 to
// 17408 features in and out, gradients from 16 tokens on; every tile, split and kernel): over 96 sizes of
// those ranges that it was not fitted to, the plan taken is up to 2% slower than the best one on average
// for each of the four calls, 1.3 times at worst.  A k-block
// costs the MMA warp's turn (shared by the k-blocks of a turn) and its MMAs, or the time its operands take
// on the way from L2, the more the more SMs ask for theirs; a tile's epilogue overlaps the next one's loop.
namespace {

long long div_up(long long a, long long b) { return (a + b - 1) / b; }
double either(double a, double b) { return std::sqrt(std::sqrt(a * a * a * a + b * b * b * b)); }

struct LinearChoice {
    bool pair;
    int bn, split;
};

// Clusters' CTAs that fit on the device at once, of `slots` SMs (152: 76 clusters of 2, 36 of 4, 15 of 8).
long long split_slots(long long slots, int split)
{
    return split <= 2 ? slots : split == 4 ? slots * 36 / 38 : slots * 30 / 38;
}

// Whether a launch of one-CTA tiles of bn columns can split job 0's k loops: two k-blocks for every
// CTA and, beside another job, all its clusters on the device at once.
bool linear_split_fits(const LinearLaunch& g, int bn, int split)
{
    if (split == 1) return true;
    if (g.mode != kModeGrad) return div_up(g.K, 64) >= 2LL * split;
    const long long kx = g.dx != nullptr ? div_up(g.M, 64) * g.parts : 0, kw = g.dW[0] != nullptr ? div_up(g.n, 64) : 0;
    const bool both = kx > 0 && kw > 0;
    const long long tiles = kw > kx ? div_up(g.M, 128) * g.parts * div_up(g.K, bn) : div_up(g.n, 128) * div_up(g.K, bn);
    return (kx > kw ? kx : kw) >= 2LL * split && (!both || tiles * split <= split_slots(g.num_sms, split));
}

double forward_time(const LinearLaunch& g, const LinearChoice& c)
{
    const bool gated = g.mode == kModeGated;
    const int rows = c.pair ? 256 : 128, wcols = gated ? c.bn / 2 : c.bn;
    const long long tiles = div_up(g.n, rows) * div_up(g.M, wcols), kb = div_up(g.K, 64);
    const int a_rows = c.pair || g.n >= 128 ? 128 : static_cast<int>(div_up(g.n, 8)) * 8;
    const bool few = !c.pair && g.n <= kFewRows;
    long long slots = c.pair ? (g.num_sms > 1 ? g.num_sms / 2 : 1) : split_slots(g.num_sms, c.split);
    if (few && (c.split > 1 || c.bn <= 128)) slots *= 2;
    const double waves = static_cast<double>(div_up(tiles * c.split, slots));
    const double filled = static_cast<double>(tiles * c.split) / static_cast<double>(slots);
    const double load = filled < 1.0 ? filled : 1.0;
    const int group = linear_group(g, c.pair, c.bn, few, !few);
    const double turn = c.pair ? (group == 1 ? 0.099 : 0.141) + 0.00056 * c.bn
                               : (group == 4 ? 0.092 : group == 2 ? 0.11 : 0.135) + 0.00108 * c.bn;
    const double mma = turn > 0.00105 * c.bn ? turn : 0.00105 * c.bn;
    double bytes = c.pair ? (128 + c.bn / 2) * 128.0 : (a_rows + c.bn) * 128.0;
    const double per_sm = static_cast<double>(tiles * c.split) / g.num_sms;
    if (few && per_sm > 1.0) bytes *= c.split == 1 || per_sm > 2.0 ? 2.0 : per_sm;
    const double block = either(mma, bytes * 7.0e-6 * (0.4 + 0.6 * load));
    const double part = a_rows / 128.0;
    // a column's share of the epilogue; kept values and rows that are not 16-byte aligned cost more
    // (gated 333 x 2731 x 1024 with both: 13.1 us by tiles of 128, 15.1 by wider ones of CTA pairs)
    const bool keep = g.keep[0] != nullptr;
    const double more = (keep ? 0.011 : 0.0) + (g.ldo % 8 != 0 || (keep && g.ldk % 8 != 0) ? 0.005 : 0.0);
    double t = 4.04 + waves * static_cast<double>(div_up(kb, c.split)) * block + (0.0093 + more) * c.bn * part;
    const double join = c.split > 1 ? 1.36 + 0.0055 * c.bn * part : 0.0;   // (a part of it after the last operands from memory)
    if (c.split > 1) t += 0.7 * join + (waves - 1.0) * (4.1 + 0.0093 * c.bn);
    else t += (waves - 1.0) * (0.0113 + more) * c.bn;
    const double parts = g.parts;
    const double memory = 2.0 * (parts * g.M * g.K + static_cast<double>(g.n) * (g.K + static_cast<double>(g.M))) / 4.87e6;
    return either(t, memory + 2.4) + 0.3 * join;
}

double grad_time(const LinearLaunch& g, const LinearChoice& c)
{
    const int rows = c.pair ? 256 : 128;
    long long tiles[2] = {0, 0}, kb[2] = {0, 0};
    if (g.dx != nullptr) {
        tiles[0] = div_up(g.n, rows) * div_up(g.K, c.bn);
        kb[0] = div_up(g.M, 64) * g.parts;
    }
    if (g.dW[0] != nullptr) {
        tiles[1] = div_up(g.M, rows) * g.parts * div_up(g.K, c.bn);
        kb[1] = div_up(g.n, 64);
    }
    const int first = tiles[0] == 0 || (tiles[1] != 0 && kb[1] > kb[0]) ? 1 : 0;
    const double t0 = static_cast<double>(tiles[first]), t1 = static_cast<double>(tiles[1 - first]);
    const double slots = static_cast<double>(c.pair ? (g.num_sms > 1 ? g.num_sms / 2 : 1) : split_slots(g.num_sms, c.split));
    const int group = linear_group(g, c.pair, c.bn, false, true);
    const double turn = c.pair ? 0.192 + 0.00062 * c.bn : (group >= 2 ? 0.237 : 0.292) + 0.00053 * c.bn;
    const double mma = turn > 0.00105 * c.bn ? turn : 0.00105 * c.bn;
    const double bytes = c.pair ? (128 + c.bn / 2) * 128.0 : (128 + c.bn) * 128.0;
    const double filled = (t0 * c.split + t1) / slots;
    const double block = either(mma, bytes * 6.1e-6 * (0.4 + 0.6 * (filled < 1.0 ? filled : 1.0)));
    // a tile takes its k loop or, overlapped, the epilogue of another
    const double epilogue = 1.57 + 0.0068 * c.bn;
    const double longest = static_cast<double>(div_up(kb[first], c.split)) * block, other = static_cast<double>(kb[1 - first]) * block;
    const double c0 = longest > epilogue ? longest : epilogue, c1 = t1 > 0.0 ? (other > epilogue ? other : epilogue) : 0.0;
    const double mean = (t0 * c.split * c0 + t1 * c1) / slots + 0.77 * c1;
    const double rounds = static_cast<double>(div_up(tiles[first] * c.split, static_cast<long long>(slots))) * c0;
    const double t = 4.25 + (c.split > 1 ? 1.2 + 0.003 * c.bn : 0.0) + (mean > rounds ? mean : rounds) + 0.0064 * c.bn;
    const double parts = g.parts;
    const double memory = 2.0 * (2.0 * parts * g.M * g.K + static_cast<double>(g.n) * (2.0 * g.K + parts * g.M)) / 3.7e6;
    return either(t, memory + 2.5);
}

}  // namespace

void plan_linear(LinearLaunch& g)
{
    const bool grad = g.mode == kModeGrad;
    const long long opt_kernel = bsk_get_option(BSK_OPT_LINEAR_KERNEL);
    const long long opt_tile = bsk_get_option(BSK_OPT_LINEAR_TILE);
    const long long opt_split = bsk_get_option(BSK_OPT_SPLIT_K);
    double best = -1.0;
    for (int pair = 0; pair < 2; ++pair) {
        if ((opt_kernel == 1 && pair) || (opt_kernel == 2 && !pair)) continue;
        const int unit = grad ? (pair ? 128 : 64) : pair ? 32 : g.mode == kModeGated ? 32 : 16;
        for (int bn = unit; bn <= 256; bn += unit) {
            if (opt_tile > 0 ? bn != opt_tile && opt_tile % unit == 0 : bn > 48 && bn % 32 != 0) continue;
            for (int split = 1; split <= (pair ? 1 : 8); split *= 2) {
                if (split > 1 && opt_split == 1) break;
                if (!linear_split_fits(g, bn, split)) break;
                // (a split that was asked for, where there is one)
                if (!pair && opt_split > 1 && opt_split <= 8 && split != opt_split && linear_split_fits(g, bn, static_cast<int>(opt_split)))
                    continue;
                const LinearChoice c{pair != 0, bn, split};
                const double t = grad ? grad_time(g, c) : forward_time(g, c);
                if (best < 0.0 || t < best) {
                    best = t;
                    g.pair = c.pair;
                    g.bn = bn;
                    g.split = split;
                }
            }
        }
    }
    // Rows of tiles that are worked on together, so that their rows of x and columns of W meet in L2: 1, 4, 8, 16,
    // 32 gave 907, 749, 722, 709, 709 us for gated 4096 x 17408 x 5120, 1702, 1695, 1656, 1650, 1704 for its
    // backward pass; linear 4096 x 5120 x 17408 is 1 us better with 8, the others do not care.
    const long long opt_group = bsk_get_option(BSK_OPT_GROUP_M);
    g.group_m = opt_group > 0 ? static_cast<int>(opt_group) : 16;
}

int launch_linear(const LinearLaunch& g, cudaStream_t stream, char* msg, size_t msg_len)
{
    return g.type == kTypeBF16 ? launch_linear_bf16(g, stream, msg, msg_len) : launch_linear_f16(g, stream, msg, msg_len);
}

}  // namespace bsk

extern "C" {

int bsk_linear_act_enqueue(
    int type, const uint16_t* W, int w_stride, const uint16_t* x, int x_stride, const uint16_t* bias,
    const uint16_t* residual, int residual_stride, uint16_t* y, int y_stride, uint16_t* z, int z_stride, int M, int K, int n,
    int activation, void* stream)
{
    return only_enqueue<ForwardArgs>(enqueue_forward,
                         {type, false, {W, nullptr}, w_stride, x, x_stride, {bias, nullptr}, residual, residual_stride, y,
                         y_stride, {z, nullptr}, z_stride, M, K, n, activation},
                         stream);
}

int linear_act(
    int type, const uint16_t* W, int w_stride, const uint16_t* x, int x_stride, const uint16_t* bias,
    const uint16_t* residual, int residual_stride, uint16_t* y, int y_stride, uint16_t* z, int z_stride, int M, int K, int n,
    int activation, void* stream)
{
    return blocking<ForwardArgs>(enqueue_forward,
                         {type, false, {W, nullptr}, w_stride, x, x_stride, {bias, nullptr}, residual, residual_stride, y,
                         y_stride, {z, nullptr}, z_stride, M, K, n, activation},
                         stream);
}

int bsk_gated_linear_enqueue(
    int type, const uint16_t* Wg, const uint16_t* Wu, int w_stride, const uint16_t* x, int x_stride,
    const uint16_t* bias_g, const uint16_t* bias_u, uint16_t* h, int h_stride, uint16_t* g, uint16_t* u, int gu_stride, int M,
    int K, int n, int activation, void* stream)
{
    return only_enqueue<ForwardArgs>(enqueue_forward,
                         {type, true, {Wg, Wu}, w_stride, x, x_stride, {bias_g, bias_u}, nullptr, 0, h, h_stride, {g, u},
                         gu_stride, M, K, n, activation},
                         stream);
}

int gated_linear(
    int type, const uint16_t* Wg, const uint16_t* Wu, int w_stride, const uint16_t* x, int x_stride,
    const uint16_t* bias_g, const uint16_t* bias_u, uint16_t* h, int h_stride, uint16_t* g, uint16_t* u, int gu_stride, int M,
    int K, int n, int activation, void* stream)
{
    return blocking<ForwardArgs>(enqueue_forward,
                         {type, true, {Wg, Wu}, w_stride, x, x_stride, {bias_g, bias_u}, nullptr, 0, h, h_stride, {g, u},
                         gu_stride, M, K, n, activation},
                         stream);
}

int bsk_linear_act_backward_enqueue(
    int type, const uint16_t* W, int w_stride, const uint16_t* x, int x_stride, const uint16_t* z,
    int z_stride, const uint16_t* dy, int dy_stride, uint16_t* dx, int dx_stride, void* dW, int dw_stride, void* dbias,
    int grad_type, int accumulate, int M, int K, int n, int activation, void* stream)
{
    return only_enqueue<BackwardArgs>(enqueue_backward,
                         {type, false, {W, nullptr}, w_stride, x, x_stride, {z, nullptr}, z_stride, dy, dy_stride, dx, dx_stride,
                          {dW, nullptr}, dw_stride, {dbias, nullptr}, grad_type, accumulate, M, K, n, activation},
                         stream);
}

int linear_act_backward(
    int type, const uint16_t* W, int w_stride, const uint16_t* x, int x_stride, const uint16_t* z,
    int z_stride, const uint16_t* dy, int dy_stride, uint16_t* dx, int dx_stride, void* dW, int dw_stride, void* dbias,
    int grad_type, int accumulate, int M, int K, int n, int activation, void* stream)
{
    return blocking<BackwardArgs>(enqueue_backward,
                         {type, false, {W, nullptr}, w_stride, x, x_stride, {z, nullptr}, z_stride, dy, dy_stride, dx, dx_stride,
                          {dW, nullptr}, dw_stride, {dbias, nullptr}, grad_type, accumulate, M, K, n, activation},
                         stream);
}

int bsk_gated_linear_backward_enqueue(
    int type, const uint16_t* Wg, const uint16_t* Wu, int w_stride, const uint16_t* x, int x_stride,
    const uint16_t* g, const uint16_t* u, int gu_stride, const uint16_t* dh, int dh_stride, uint16_t* dx, int dx_stride,
    void* dWg, void* dWu, int dw_stride, void* dbias_g, void* dbias_u, int grad_type, int accumulate, int M, int K, int n,
    int activation, void* stream)
{
    return only_enqueue<BackwardArgs>(enqueue_backward,
                         {type, true, {Wg, Wu}, w_stride, x, x_stride, {g, u}, gu_stride, dh, dh_stride, dx, dx_stride,
                          {dWg, dWu}, dw_stride, {dbias_g, dbias_u}, grad_type, accumulate, M, K, n, activation},
                         stream);
}

int gated_linear_backward(
    int type, const uint16_t* Wg, const uint16_t* Wu, int w_stride, const uint16_t* x, int x_stride,
    const uint16_t* g, const uint16_t* u, int gu_stride, const uint16_t* dh, int dh_stride, uint16_t* dx, int dx_stride,
    void* dWg, void* dWu, int dw_stride, void* dbias_g, void* dbias_u, int grad_type, int accumulate, int M, int K, int n,
    int activation, void* stream)
{
    return blocking<BackwardArgs>(enqueue_backward,
                         {type, true, {Wg, Wu}, w_stride, x, x_stride, {g, u}, gu_stride, dh, dh_stride, dx, dx_stride,
                          {dWg, dWu}, dw_stride, {dbias_g, dbias_u}, grad_type, accumulate, M, K, n, activation},
                         stream);
}

int bsk_plan_linear(int mode, int gated, int M, int K, int n, int sms, int* plan)
{
    if (plan == nullptr || M < 1 || K < 1 || n < 1 || sms < 2 || mode < 0 || mode > 3)
        return fail(BSK_ERR_INVALID_ARG, "plan query: sizes and SM count must be positive (sms >= 2), plan non-NULL");
    static uint16_t some;   // stands for a result; not written
    bsk::LinearLaunch g;
    g.mode = mode == 0 ? (gated ? bsk::kModeGated : bsk::kModeLinear) : bsk::kModeGrad;
    g.parts = gated ? 2 : 1;
    g.n = n;
    g.M = M;
    g.K = K;
    g.num_sms = sms;
    if (mode & 1) g.dx = &some;
    if (mode & 2) g.dW[0] = g.dW[1] = &some;
    bsk::plan_linear(g);
    plan[0] = g.pair ? 1 : 0;
    plan[1] = g.bn;
    plan[2] = g.split;
    return BSK_OK;
}

}  // extern "C"
