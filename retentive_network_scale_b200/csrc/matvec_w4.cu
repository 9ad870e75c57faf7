// matvec_w4.cu -- ret_matvec_w4: products of a few rows with 4-bit weights,
//     y[m][n] = sum_g s[n][g] sum_{k in g} (q[n][k] - z[n][g]) x[m][k],
// and ret_quantize_w4, which lays such weights out.
//
// Bound by HBM for few rows: the codes are read once.  The products run on the
// tensor cores' warp-level instruction (m16n8k16, bf16 in, fp32 out): 16 weight
// rows by 8 columns of x.  Nothing is rounded on the way in: q - z is a small
// integer, exact in bf16, x is bf16 already, or 8-bit codes (exact in bf16, their
// scale applied to the sum), or fp32 split into three bf16 parts that add up to
// it (three columns of the instruction, which has columns to spare).  The sum of
// a group of weights is scaled in fp32.
//
// A 32-bit word holds 8 codes of one weight row; masking it at shifts of 0, 4,
// 8 and 12 bits leaves the pairs (k, k+4), (k+1, k+5), ..., each of which one
// OR turns into two bf16 values 128 + q.  The instruction sums over k in any
// order as long as both operands use the same one, so x is kept in shared memory
// in that order and the codes are never moved between lanes.
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "retention.h"

namespace ret {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;

struct W4Args {
    int M, N, K, x_dtype, xg, cols;  // xg: columns of x per x scale; cols: columns of the products
    long long ldx;
    const void *x;
    const float *xs;
    const uint8_t *wq, *zeros;
    const __nv_bfloat16 *s;
    void *y;
    int y_bf16, kc;  // kc: columns of x staged at a time
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Codes (k+j, k+j+4) of the 8 codes in w, as bf16 minus `zero` (both lanes of
// it 128 + z): exact.
template <int J>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, __nv_bfloat162 zero) {
    const uint32_t u = ((w >> (4 * J)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&u), zero);
    return *reinterpret_cast<const uint32_t *>(&d);
}

template <int W>
__device__ __forceinline__ void load_words(uint32_t (&w)[W], const uint8_t *p);
template <>
__device__ __forceinline__ void load_words<1>(uint32_t (&w)[1], const uint8_t *p) {
    w[0] = __ldcs(reinterpret_cast<const unsigned int *>(p));
}
template <>
__device__ __forceinline__ void load_words<2>(uint32_t (&w)[2], const uint8_t *p) {
    const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
    w[0] = v.x; w[1] = v.y;
}
template <>
__device__ __forceinline__ void load_words<4>(uint32_t (&w)[4], const uint8_t *p) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 8 columns of x from column k of product column `col`, as bf16 pairs (j, j+4).
__device__ __forceinline__ uint4 load_x(const W4Args &a, int col, int k) {
    float v[8];
    if (a.x_dtype == RET_F32) {
        const int m = col / 3, part = col - 3 * m;
        const float *p = static_cast<const float *>(a.x) + (long long)m * a.ldx + k;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // parts of 8 bits each: what the parts before it leave
            const float x = p[i];
            float r = x;
            for (int j = 0; j < part; ++j) {
                const float top = __bfloat162float(__float2bfloat16_rn(r));
                r = isfinite(top) ? r - top : 0.f;  // infinities and NaN go with the first part
            }
            v[i] = r;
        }
    } else if (a.x_dtype == RET_BF16) {
        const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(a.x) + (long long)col * a.ldx + k;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __bfloat162float(p[i]);
    } else {
        const uint8_t *p = static_cast<const uint8_t *>(a.x) + (long long)col * a.ldx + k;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = a.x_dtype == RET_I8 ? (float)(int8_t)p[i]
                                       : __half2float(__half(__nv_cvt_fp8_to_halfraw(p[i], __NV_E4M3)));
    }
    return make_uint4(pack_bf16(v[0], v[4]), pack_bf16(v[1], v[5]), pack_bf16(v[2], v[6]), pack_bf16(v[3], v[7]));
}

// One CTA: 16 weight rows, all K; its warps take the groups of the rows in
// turn and their sums meet in shared memory.  WPL: 32-bit words of codes per
// load, a group of weights being 32 WPL columns: the four lanes of a row read
// one group in one load each.  NT: 8-column tiles of x.
template <int WPL, int NT>
__global__ void __launch_bounds__(kThreads)
matvec_w4_kernel(const W4Args a) {
    constexpr int GK = 32 * WPL;
    extern __shared__ __align__(16) uint8_t dsm[];
    uint4 *xs = reinterpret_cast<uint4 *>(dsm);  // [kc / 32][cols][4]
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, q = lane / 4, c = lane % 4;
    const int n0 = blockIdx.x * 16;
    const int col0 = blockIdx.y * NT * 8, ncol = min(NT * 8, a.cols - col0);
    const int groups = a.K / GK;
    const int r0 = min(n0 + q, a.N - 1), r1 = min(n0 + q + 8, a.N - 1);
    const uint8_t *w0 = a.wq + (long long)r0 * (a.K / 2), *w1 = a.wq + (long long)r1 * (a.K / 2);
    const long long s0 = (long long)r0 * groups, s1 = (long long)r1 * groups;

    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;

    for (int k0 = 0; k0 < a.K; k0 += a.kc) {
        const int kn = min(a.kc, a.K - k0);
        if (k0) __syncthreads();
        // x of the chunk: piece (step of 32 columns, product column, c) holds
        // the 8 columns that lane c multiplies in that step
        for (int i = tid; i < kn / 8 * ncol; i += kThreads) {
            const int cc = i % 4, col = i / 4 % ncol, step = i / (4 * ncol);
            const int blk = step / WPL, j = step % WPL;
            xs[i] = load_x(a, col0 + col, k0 + blk * GK + cc * 8 * WPL + 8 * j);
        }
        __syncthreads();
        for (int blk = warp; blk < kn / GK; blk += kWarps) {
            const int gi = k0 / GK + blk;
            uint32_t wa[WPL], wb[WPL];
            load_words<WPL>(wa, w0 + (long long)gi * (GK / 2) + c * 4 * WPL);
            load_words<WPL>(wb, w1 + (long long)gi * (GK / 2) + c * 4 * WPL);
            const float sa = __bfloat162float(a.s[s0 + gi]), sb = __bfloat162float(a.s[s1 + gi]);
            const uint32_t za = a.zeros ? 0x4300u + (a.zeros[s0 + gi] & 15u) : 0x4308u;
            const uint32_t zb = a.zeros ? 0x4300u + (a.zeros[s1 + gi] & 15u) : 0x4308u;
            const uint32_t za2 = za | za << 16, zb2 = zb | zb << 16;
            const __nv_bfloat162 zeroa = *reinterpret_cast<const __nv_bfloat162 *>(&za2);
            const __nv_bfloat162 zerob = *reinterpret_cast<const __nv_bfloat162 *>(&zb2);
            float sum[NT][4];
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[i][j] = 0.f;
#pragma unroll
            for (int j = 0; j < WPL; ++j) {
                const uint32_t fa[4] = {code_pair<0>(wa[j], zeroa), code_pair<0>(wb[j], zerob),
                                        code_pair<1>(wa[j], zeroa), code_pair<1>(wb[j], zerob)};
                const uint32_t fb[4] = {code_pair<2>(wa[j], zeroa), code_pair<2>(wb[j], zerob),
                                        code_pair<3>(wa[j], zeroa), code_pair<3>(wb[j], zerob)};
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int col = 8 * i + q;
                    uint4 b = make_uint4(0, 0, 0, 0);
                    if (col < ncol) b = xs[((blk * WPL + j) * ncol + col) * 4 + c];
                    mma16816(sum[i], fa, b.x, b.y);
                    mma16816(sum[i], fb, b.z, b.w);
                }
            }
            const int per = a.x_dtype == RET_F32 ? 3 : 1;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                float x0 = 1.f, x1 = 1.f;
                if (a.xs && a.xg < a.K) {  // x scales by group of columns
                    const int m0 = col0 + 8 * i + 2 * c, xgs = a.K / a.xg, xi = gi * GK / a.xg;
                    if (m0 < a.cols) x0 = a.xs[(long long)(m0 / per) * xgs + xi];
                    if (m0 + 1 < a.cols) x1 = a.xs[(long long)((m0 + 1) / per) * xgs + xi];
                }
                acc[i][0] = fmaf(sa * x0, sum[i][0], acc[i][0]);
                acc[i][1] = fmaf(sa * x1, sum[i][1], acc[i][1]);
                acc[i][2] = fmaf(sb * x0, sum[i][2], acc[i][2]);
                acc[i][3] = fmaf(sb * x1, sum[i][3], acc[i][3]);
            }
        }
    }
    // join the warps' sums: red[warp][16 rows][NT*8 columns + 1]
    __syncthreads();
    float *red = reinterpret_cast<float *>(dsm);
    constexpr int RS = NT * 8 + 1;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        float *p = red + (warp * 16 + q) * RS + 8 * i + 2 * c;
        p[0] = acc[i][0];
        p[1] = acc[i][1];
        p[8 * RS] = acc[i][2];
        p[8 * RS + 1] = acc[i][3];
    }
    __syncthreads();
    const int per = a.x_dtype == RET_F32 ? 3 : 1;
    for (int i = tid; i < 16 * (ncol / per); i += kThreads) {
        const int r = i % 16, m = i / 16, n = n0 + r;
        if (n >= a.N) continue;
        float y = 0.f;
        for (int p = per - 1; p >= 0; --p)
            for (int w = 0; w < kWarps; ++w) y += red[(w * 16 + r) * RS + m * per + p];
        const int mm = col0 / per + m;
        if (a.xs && a.xg == a.K) y *= a.xs[mm];
        const long long at = (long long)mm * a.N + n;
        if (a.y_bf16)
            static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(y);
        else
            static_cast<float *>(a.y)[at] = y;
    }
}

template <int WPL, int NT>
cudaError_t launch_w4(W4Args a, cudaStream_t st) {
    constexpr int RS = NT * 8 + 1;
    const int ncol = std::min(a.cols, NT * 8);
    const int limit = 96 * 1024 / (2 * ncol) / 128 * 128;
    a.kc = std::min((a.K + 127) / 128 * 128, std::max(limit, 128));
    const size_t smem = std::max((size_t)a.kc * 2 * ncol, sizeof(float) * kWarps * 16 * RS);
    const long long bx = ((long long)a.N + 15) / 16, by = (a.cols + NT * 8 - 1) / (NT * 8);
    auto kern = matvec_w4_kernel<WPL, NT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<dim3((unsigned)bx, (unsigned)by), kThreads, smem, st>>>(a);
    e = cudaGetLastError();
    if (e == cudaSuccess) note_launches(1);
    return e;
}

template <int WPL>
cudaError_t launch_cols(const W4Args &a, cudaStream_t st) {
    // fp32 rows take three product columns: 24 columns (three tiles) hold
    // whole rows
    if (a.cols <= 8) return launch_w4<WPL, 1>(a, st);
    if (a.cols <= 16) return launch_w4<WPL, 2>(a, st);
    return launch_w4<WPL, 3>(a, st);
}

// One thread per (weight row n, group): scale and codes of `group` weights.
template <typename T>
__global__ void quantize_w4_kernel(int K, int N, int group, const T *W, long long ldw, uint8_t *wq,
                                   __nv_bfloat16 *scales, uint8_t *zeros) {
    const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int groups = K / group;
    if (idx >= (long long)N * groups) return;
    const int n = (int)(idx % N), g = (int)(idx / N);
    const T *w = W + (long long)g * group * ldw + n;
    float lo = 0.f, hi = 0.f;
    for (int k = 0; k < group; ++k) {
        const float v = ld(w, (size_t)k * ldw);
        lo = fminf(lo, v);
        hi = fmaxf(hi, v);
    }
    // with zero points [lo, hi] (0 included) to 0..15, else +-max to 8 +- 7
    const __nv_bfloat16 sb = __float2bfloat16_rn(zeros ? (hi - lo) / 15.f : fmaxf(hi, -lo) / 7.f);
    const float s = __bfloat162float(sb), inv = s > 0.f ? 1.f / s : 0.f;
    const float z = zeros ? fminf(fmaxf(rintf(-lo * inv), 0.f), 15.f) : 8.f;
    scales[(long long)n * groups + g] = sb;
    if (zeros) zeros[(long long)n * groups + g] = (uint8_t)z;
    uint8_t *p = wq + (long long)n * (K / 2) + (long long)g * (group / 2);
    for (int k = 0; k < group; k += 2) {
        const float a = fminf(fmaxf(rintf(ld(w, (size_t)k * ldw) * inv) + z, 0.f), 15.f);
        const float b = fminf(fmaxf(rintf(ld(w, (size_t)(k + 1) * ldw) * inv) + z, 0.f), 15.f);
        p[k / 2] = (uint8_t)((uint32_t)a | (uint32_t)b << 4);
    }
}

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace ret

extern "C" ret_status ret_matvec_w4(int M, int N, int K, int group, int x_dtype, const void *X,
                                    long long ldx, const float *x_scales, int x_group,
                                    const void *Wq, const void *scales, const void *zeros,
                                    int y_dtype, void *Y, void *stream) {
    using namespace ret;
    if (M < 0 || M > RET_MAX_MATVEC_ROWS || N < 0 || K < 1 || ldx < K ||
        (group != 32 && group != 64 && group != 128) || K % group)
        return RET_ERR_SHAPE;
    if (x_dtype < RET_F32 || x_dtype > RET_E4M3 || (y_dtype != RET_F32 && y_dtype != RET_BF16))
        return RET_ERR_DTYPE;
    const bool codes = x_dtype == RET_I8 || x_dtype == RET_E4M3;
    // x scales: one per row, or one per x_group columns
    if (codes ? (x_group != 0 && (x_group < group || x_group % group || K % x_group)) : x_group != 0)
        return RET_ERR_SHAPE;
    const bool empty = M == 0 || N == 0;
    if (!empty && (!X || !Wq || !scales || !Y || (codes && !x_scales))) return RET_ERR_NULL;
    const unsigned xsize = codes ? 1 : x_dtype == RET_BF16 ? 2 : 4;
    if (!aligned(X, xsize) || !aligned(x_scales, 16) || !aligned(Wq, 16) || !aligned(scales, 16) ||
        !aligned(zeros, 16) || !aligned(Y, 16))
        return RET_ERR_ALIGN;
    const ret_status s = validate_device();
    if (s != RET_OK) return s;
    if (empty) return RET_OK;
    W4Args a{};
    a.M = M; a.N = N; a.K = K;
    a.x_dtype = x_dtype;
    a.xg = x_group ? x_group : K;
    a.cols = x_dtype == RET_F32 ? 3 * M : M;
    a.ldx = ldx;
    a.x = X;
    a.xs = codes ? x_scales : nullptr;
    a.wq = static_cast<const uint8_t *>(Wq);
    a.zeros = static_cast<const uint8_t *>(zeros);
    a.s = static_cast<const __nv_bfloat16 *>(scales);
    a.y = Y;
    a.y_bf16 = y_dtype == RET_BF16;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = group == 128 ? launch_cols<4>(a, st) : group == 64 ? launch_cols<2>(a, st) : launch_cols<1>(a, st);
    return e == cudaSuccess ? RET_OK : RET_ERR_CUDA;
}

extern "C" ret_status ret_quantize_w4(int K, int N, int group, int w_dtype, const void *W, long long ldw,
                                      void *Wq, void *scales, void *zeros, void *stream) {
    using namespace ret;
    if (K < 1 || N < 0 || ldw < N || (group != 32 && group != 64 && group != 128) || K % group)
        return RET_ERR_SHAPE;
    if (w_dtype != RET_F32 && w_dtype != RET_BF16) return RET_ERR_DTYPE;
    if (N > 0 && (!W || !Wq || !scales)) return RET_ERR_NULL;
    if (!aligned(W, w_dtype == RET_BF16 ? 2 : 4) || !aligned(Wq, 16) || !aligned(scales, 16) || !aligned(zeros, 16))
        return RET_ERR_ALIGN;
    const ret_status s = validate_device();
    if (s != RET_OK) return s;
    if (N == 0) return RET_OK;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const long long blocks = ((long long)N * (K / group) + 127) / 128;
    if (blocks > 0x7fffffffLL) return RET_ERR_CUDA;
    if (w_dtype == RET_BF16)
        quantize_w4_kernel<<<(unsigned)blocks, 128, 0, st>>>(K, N, group, static_cast<const __nv_bfloat16 *>(W), ldw,
                                                             static_cast<uint8_t *>(Wq),
                                                             static_cast<__nv_bfloat16 *>(scales),
                                                             static_cast<uint8_t *>(zeros));
    else
        quantize_w4_kernel<<<(unsigned)blocks, 128, 0, st>>>(K, N, group, static_cast<const float *>(W), ldw,
                                                             static_cast<uint8_t *>(Wq),
                                                             static_cast<__nv_bfloat16 *>(scales),
                                                             static_cast<uint8_t *>(zeros));
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) note_launches(1);
    return e == cudaSuccess ? RET_OK : RET_ERR_CUDA;
}
