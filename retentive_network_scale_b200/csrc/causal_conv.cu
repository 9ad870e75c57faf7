// causal_conv.cu -- ret_causal_conv: the short causal convolution along the
// rows of every channel, y_t = act(bias + sum_k w[k] x_{t-W+1+k}), for prompts
// (any number of rows, a padded batch through `lengths`) and for single tokens
// (L = 1 on a carried state).
//
// Bound by HBM: x is read once and y written once.  A thread owns V adjacent
// channels (16 bytes where rows are aligned) and a run of kRun rows, and keeps
// the last W-1 rows in registers, so a row is read once per run; the W-1 rows
// before a run come from L2, where the neighbouring run has just read them.
#include <cmath>

#include "common.cuh"
#include "launch.h"
#include "retention.h"

namespace ret {
namespace {

constexpr int kThreads = 128;
constexpr int kRun = 32;   // rows per thread
constexpr int kAhead = 4;  // rows of loads in flight

struct ConvArgs {
    int B, L, D, swish;
    int runs, cblocks;
    long long ldx;
    const void *x;
    const float *w, *bias;
    const int *lengths;
    const void *s_in;
    void *s_out, *y;
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T v[V];
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float &d, float v) { d = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16 &d, float v) { d = __float2bfloat16_rn(v); }

// v sigmoid(v); the quotient goes to 0 where exp(-v) overflows
__device__ __forceinline__ float swish(float v) { return __fdividef(v, 1.f + __expf(-v)); }

template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads)
causal_conv_kernel(const ConvArgs a) {
    long long blk = blockIdx.x;
    const int cb = (int)(blk % a.cblocks);
    blk /= a.cblocks;
    const int run = (int)(blk % a.runs), b = (int)(blk / a.runs);
    const int c = (cb * kThreads + threadIdx.x) * V;
    if (c >= a.D) return;
    const int len = a.lengths ? min(max(a.lengths[b], 0), a.L) : a.L;
    const int t0 = run * kRun, t1 = min(t0 + kRun, len);
    using P = Pack<T, V>;
    const T *x = static_cast<const T *>(a.x) + (long long)b * a.L * a.ldx + c;
    const T *s_in = a.s_in ? static_cast<const T *>(a.s_in) + (long long)b * (W - 1) * a.D + c : nullptr;
    // row t of the sequence continued to the left by the state (zeros without)
    auto row = [&](int t) {
        P p;
        if (t >= 0)
            p = *reinterpret_cast<const P *>(x + (long long)t * a.ldx);
        else if (s_in)
            p = *reinterpret_cast<const P *>(s_in + (long long)(t + W - 1) * a.D);
        else
#pragma unroll
            for (int i = 0; i < V; ++i) from_f(p.v[i], 0.f);
        return p;
    };

    if (t0 < t1) {
        float w[W][V], bias[V], win[W - 1][V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            bias[i] = a.bias ? a.bias[c + i] : 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][i] = a.w[(long long)(c + i) * W + k];
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const P p = row(t0 - (W - 1) + j);
#pragma unroll
            for (int i = 0; i < V; ++i) win[j][i] = to_f(p.v[i]);
        }
        T *y = static_cast<T *>(a.y) + ((long long)b * a.L) * a.D + c;
        for (int t = t0; t < t1; t += kAhead) {
            P in[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (t + j < t1) in[j] = *reinterpret_cast<const P *>(x + (long long)(t + j) * a.ldx);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (t + j < t1) {
                    P out;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float now = to_f(in[j].v[i]);
                        float acc = bias[i];
#pragma unroll
                        for (int k = 0; k < W - 1; ++k) acc = fmaf(w[k][i], win[k][i], acc);
                        acc = fmaf(w[W - 1][i], now, acc);
#pragma unroll
                        for (int k = 0; k + 1 < W - 1; ++k) win[k][i] = win[k + 1][i];
                        if (W > 1) win[W - 2][i] = now;
                        from_f(out.v[i], a.swish ? swish(acc) : acc);
                    }
                    *reinterpret_cast<P *>(y + (long long)(t + j) * a.D) = out;
                }
            }
        }
    }
    // The state after the sequence: its last W-1 rows, the entering state's
    // among them when it is shorter.  Only the thread of the first run reads
    // s_in, and it has read all it needs of it before it writes, so s_out may
    // be s_in.
    if (run == 0 && a.s_out) {
        P last[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) last[j] = row(len - (W - 1) + j);
        T *s_out = static_cast<T *>(a.s_out) + (long long)b * (W - 1) * a.D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) *reinterpret_cast<P *>(s_out + (long long)j * a.D) = last[j];
    }
}

template <typename T, int V>
cudaError_t launch_v(ConvArgs a, int W, cudaStream_t st) {
    a.runs = a.L > 0 ? (a.L + kRun - 1) / kRun : 1;
    a.cblocks = ((a.D + V - 1) / V + kThreads - 1) / kThreads;
    const long long blocks = (long long)a.B * a.runs * a.cblocks;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    switch (W) {
        case 2: causal_conv_kernel<T, V, 2><<<(unsigned)blocks, kThreads, 0, st>>>(a); break;
        case 3: causal_conv_kernel<T, V, 3><<<(unsigned)blocks, kThreads, 0, st>>>(a); break;
        default: causal_conv_kernel<T, V, 4><<<(unsigned)blocks, kThreads, 0, st>>>(a); break;
    }
    const cudaError_t err = cudaGetLastError();
    if (err == cudaSuccess) note_launches(1);
    return err;
}

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Widest piece (elements) that every row of x, y and the states starts on.
template <typename T>
int vector_width(const ConvArgs &a) {
    for (int v = 16 / (int)sizeof(T); v > 2; v /= 2)
        if (a.D % v == 0 && a.ldx % v == 0 && aligned(a.x, v * sizeof(T))) return v;
    return a.D % 2 == 0 && a.ldx % 2 == 0 && aligned(a.x, 2 * sizeof(T)) ? 2 : 1;
}

cudaError_t launch_causal_conv(const ConvArgs &a, int W, bool bf16, cudaStream_t st) {
    if (bf16) {
        using T = __nv_bfloat16;
        switch (vector_width<T>(a)) {
            case 8: return launch_v<T, 8>(a, W, st);
            case 4: return launch_v<T, 4>(a, W, st);
            case 2: return launch_v<T, 2>(a, W, st);
            default: return launch_v<T, 1>(a, W, st);
        }
    }
    switch (vector_width<float>(a)) {
        case 4: return launch_v<float, 4>(a, W, st);
        case 2: return launch_v<float, 2>(a, W, st);
        default: return launch_v<float, 1>(a, W, st);
    }
}

}  // namespace
}  // namespace ret

extern "C" ret_status ret_causal_conv(int B, int L, int D, int width, int dtype, const void *X,
                                      long long ldx, const float *W, const float *bias, int swish,
                                      const int *lengths, const void *state_in, void *state_out,
                                      void *Y, void *stream) {
    using namespace ret;
    if (B < 0 || L < 0 || D < 1 || width < 2 || width > RET_MAX_CONV_WIDTH || ldx < D)
        return RET_ERR_SHAPE;
    if (dtype != RET_F32 && dtype != RET_BF16) return RET_ERR_DTYPE;
    if (swish != 0 && swish != 1) return RET_ERR_ARG;
    const bool rows = (long long)B * L > 0;
    if ((rows && (!X || !Y)) || (B > 0 && !W)) return RET_ERR_NULL;
    if (!aligned(X, dtype == RET_BF16 ? 2 : 4) || !aligned(W, 16) || !aligned(bias, 16) ||
        !aligned(lengths, 4) || !aligned(state_in, 16) || !aligned(state_out, 16) || !aligned(Y, 16))
        return RET_ERR_ALIGN;
    const ret_status s = validate_device();
    if (s != RET_OK) return s;
    if (B == 0 || (L == 0 && !state_out)) return RET_OK;
    ConvArgs a{B, L, D, swish, 0, 0, ldx, X, W, bias, lengths, state_in, state_out, Y};
    const cudaError_t e = launch_causal_conv(a, width, dtype == RET_BF16, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RET_OK : RET_ERR_CUDA;
}
