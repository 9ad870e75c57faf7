// causal_conv.cu -- ret_causal_conv: the short causal convolution along the
// rows of every channel, y_t = act(bias + sum_k w[k] x_{t-W+1+k}), for prompts
// (any number of rows, a padded batch through `lengths`) and for single tokens
// (L = 1 on a carried state).
//
// Bound by HBM: x is read once and y written once.  A thread owns V adjacent
// channels and a run of rows, and keeps the last W-1 rows in registers, so a row is
// read once per run; the W-1 rows before a run come from L2, where the
// neighbouring run has just read them.  Rows are taken kAhead at a time, all
// requested before the first is used, as straight-line code on pairs of channels
// (a window shifted row by row costs three register moves per element).
#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "retention.h"
#include "tc_util.cuh"

namespace ret {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 8;  // rows of loads in flight
constexpr int kRunRows = 128;  // rows of a thread, at most

struct ConvArgs {
    int B, L, D, swish;
    int runs, run_rows, cblocks;
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

__device__ __forceinline__ void from_f(float &d, float v) { d = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16 &d, float v) { d = __float2bfloat16_rn(v); }

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint64_t dup(float v) { return tc::f2_make(v, v); }
// v sigmoid(v) of both values of a pair; 0 where exp(-v) overflows
__device__ __forceinline__ uint64_t swish2(uint64_t v) {
    const uint64_t a = tc::f2_mul(v, dup(-1.4426950408889634f));
    const uint64_t q = tc::f2_add(tc::f2_make(exp2_fast(tc::f2_lo(a)), exp2_fast(tc::f2_hi(a))), dup(1.f));
    return tc::f2_mul(v, tc::f2_make(rcp_fast(tc::f2_lo(q)), rcp_fast(tc::f2_hi(q))));
}

// Values 2i and 2i + 1 of a piece (a bf16 is the high half of its fp32); the
// second is 0 in a piece of one.
template <int V>
__device__ __forceinline__ uint64_t pair(const Pack<float, V> &p, int i) {
    return tc::f2_make(p.v[2 * i], 2 * i + 1 < V ? p.v[2 * i + 1] : 0.f);
}
template <int V>
__device__ __forceinline__ uint64_t pair(const Pack<__nv_bfloat16, V> &p, int i) {
    if (V == 1) return tc::f2_make(__bfloat162float(p.v[0]), 0.f);
    const uint32_t u = reinterpret_cast<const uint32_t *>(&p)[i];
    return tc::f2_make(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads)
causal_conv_kernel(const ConvArgs a) {
    constexpr int P2 = (V + 1) / 2;  // channel pairs
    const int cb = blockIdx.x % a.cblocks;
    const int c = (cb * kThreads + threadIdx.x) * V;
    if (c >= a.D) return;
    using P = Pack<T, V>;
    uint64_t w[W][P2], bias[P2];
#pragma unroll
    for (int i = 0; i < P2; ++i) {
        auto of = [&](const float *p, int cc, int n, int k) { return p && cc < a.D ? p[(long long)cc * n + k] : 0.f; };
        bias[i] = tc::f2_make(of(a.bias, c + 2 * i, 1, 0), V > 1 ? of(a.bias, c + 2 * i + 1, 1, 0) : 0.f);
#pragma unroll
        for (int k = 0; k < W; ++k)
            w[k][i] = tc::f2_make(of(a.w, c + 2 * i, W, k), V > 1 ? of(a.w, c + 2 * i + 1, W, k) : 0.f);
    }
    const long long task = blockIdx.x / a.cblocks;
    const int run = (int)(task % a.runs), b = (int)(task / a.runs);
    const int len = a.lengths ? min(max(a.lengths[b], 0), a.L) : a.L;
    const int t0 = run * a.run_rows, t1 = min(t0 + a.run_rows, len);
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
        uint64_t win[W - 1][P2];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const P p = row(t0 - (W - 1) + j);
#pragma unroll
            for (int i = 0; i < P2; ++i) win[j][i] = pair(p, i);
        }
        const T *px = x + (long long)t0 * a.ldx;
        T *py = static_cast<T *>(a.y) + ((long long)b * a.L + t0) * a.D + c;
        // n rows of a batch, and all of the one after it requested before this
        // one is computed (the compiler keeps reads behind the writes before them)
        P in[kAhead];
        auto request = [&](const T *p, int n) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (j < n) in[j] = *reinterpret_cast<const P *>(p + (long long)j * a.ldx);
        };
        request(px, t1 - t0);
        auto rows = [&](auto whole, int n) {
            constexpr bool ALL = decltype(whole)::value;
            uint64_t v[W - 1 + kAhead][P2];
#pragma unroll
            for (int i = 0; i < P2; ++i) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) v[j][i] = win[j][i];
#pragma unroll
                for (int j = 0; j < kAhead; ++j) v[W - 1 + j][i] = pair(in[j], i);
            }
            px += (long long)kAhead * a.ldx;
            request(px, n - kAhead);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (!ALL && j >= n) break;
                P out;
#pragma unroll
                for (int i = 0; i < P2; ++i) {
                    uint64_t acc = bias[i];
#pragma unroll
                    for (int k = 0; k < W; ++k) acc = tc::f2_fma(w[k][i], v[j + k][i], acc);
                    if (a.swish) acc = swish2(acc);
                    from_f(out.v[2 * i], tc::f2_lo(acc));
                    if (V > 1) from_f(out.v[2 * i + (V > 1)], tc::f2_hi(acc));
                }
                *reinterpret_cast<P *>(py + (long long)j * a.D) = out;
            }
#pragma unroll
            for (int i = 0; i < P2; ++i)
#pragma unroll
                for (int j = 0; j < W - 1; ++j) win[j][i] = v[kAhead + j][i];
            py += (long long)kAhead * a.D;
        };
        int t = t0;
#pragma unroll 1
        for (; t + kAhead <= t1; t += kAhead) rows(std::true_type{}, t1 - t);
        if (t < t1) rows(std::false_type{}, t1 - t);
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
    a.cblocks = ((a.D + V - 1) / V + kThreads - 1) / kThreads;
    // long runs read fewer rows twice, short ones make more CTAs
    a.run_rows = kRunRows;
    while (a.run_rows > kAhead && (long long)a.B * a.cblocks * ((a.L + a.run_rows - 1) / a.run_rows) < 148 * 8) a.run_rows /= 2;
    a.runs = a.L > 0 ? (a.L + a.run_rows - 1) / a.run_rows : 1;
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

// Channels per thread: 8 bytes of a row, or 4 where that leaves SMs without
// threads (one token of 64 x 4096 bf16 channels 5.2 us against 4.1), or what the
// rows of x, y and the states start on.  16 bytes cost so many registers that too
// few rows are in flight (8 x 4096 x 4096 bf16: 137 us against 104).
template <typename T>
int vector_width(const ConvArgs &a) {
    const bool few = (long long)a.B * a.D * ((a.L + kRunRows - 1) / kRunRows) * (long long)sizeof(T) / 8 < 148 * 1024;
    for (int v = (few ? 4 : 8) / (int)sizeof(T); v > 1; v /= 2)
        if (a.D % v == 0 && a.ldx % v == 0 && aligned(a.x, v * sizeof(T))) return v;
    return 1;
}

cudaError_t launch_causal_conv(const ConvArgs &a, int W, bool bf16, cudaStream_t st) {
    if (bf16) {
        using T = __nv_bfloat16;
        switch (vector_width<T>(a)) {
            case 4: return launch_v<T, 4>(a, W, st);
            case 2: return launch_v<T, 2>(a, W, st);
            default: return launch_v<T, 1>(a, W, st);
        }
    }
    return vector_width<float>(a) == 2 ? launch_v<float, 2>(a, W, st) : launch_v<float, 1>(a, W, st);
}

}  // namespace
}  // namespace ret

extern "C" ret_status ret_causal_conv(int B, int L, int D, int width, int dtype, const void *X,
                                      long long ldx, const float *W, const float *bias, int swish,
                                      const int *lengths, const void *state_in, void *state_out,
                                      void *Y, void *stream) {
    using namespace ret;
    // (the extents' limit keeps rows and channels rounded up to whole CTAs in an int)
    if (B < 0 || L < 0 || D < 1 || L > RET_MAX_EXTENT || D > RET_MAX_EXTENT || width < 2 ||
        width > RET_MAX_CONV_WIDTH || ldx < D)
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
    ConvArgs a{B, L, D, swish, 0, 0, 0, ldx, X, W, bias, lengths, state_in, state_out, Y};
    const cudaError_t e = launch_causal_conv(a, width, dtype == RET_BF16, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RET_OK : RET_ERR_CUDA;
}
