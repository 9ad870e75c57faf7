// rms_norm.cu -- ret_rms_norm: the residual's addition and the root-mean-
// square norm of a block's rows, s = x + r, y = w s / sqrt(mean(s^2) + eps),
// with y in fp32, bf16, or in 8 bits (int8 or e4m3) with one fp32 scale per
// group of channels.
//
// Bound by HBM: x and r are read once, r_out and y written once.  A row is
// spread over `tpr` threads (a power of two, one warp or more) that hold it in
// registers between the sum of squares and the output, kVec adjacent channels per
// thread and step, so nothing is read twice; all of x and r is requested before any is
// used, the weights (from L2) step by step.  The arithmetic runs on pairs.  The largest |w s| of a row comes out of the same
// reduction as the sum of squares (|y| = |w s| / rms), so the 8-bit scale of a
// whole row needs no second one, and that of a group of 32, 64 or 128 channels
// only shuffles among 4, 8 or 16 lanes.
//
// With a residual, us (share of the measured copy bandwidth): 32768 bf16 rows of 2048
// to bf16 80 (103%), to e4m3 with groups of 128 94 (78%); 8192 rows of 16384 in bf16
// 202 (82%), in fp32 432 (77%; there 116 bytes a thread are spilled).
#include <cuda_fp8.h>

#include <cmath>

#include "common.cuh"
#include "launch.h"
#include "retention.h"
#include "tc_util.cuh"

namespace ret {
namespace {

constexpr int kVec = 8;

struct NormArgs {
    long long rows, ldx;
    int d, tpr, y_dtype, group;
    float eps;
    const void *x, *r;
    void *r_out, *y;
    const float *w;
    float *scales;
};

// kVec elements as loaded.  VEC: adjacent, all there if n > 0 and 16-byte aligned.
// Otherwise element i is i * stride further on, zero where that is not below n.
template <typename T>
struct Raw8 {
    uint4 q[sizeof(T) * kVec / 16];
};
template <bool VEC, typename T>
__device__ __forceinline__ void load8(Raw8<T> &r, const T *p, int n, int stride) {
    constexpr int Q = sizeof(T) * kVec / 16;
#pragma unroll
    for (int i = 0; i < Q; ++i) r.q[i] = make_uint4(0, 0, 0, 0);
    if (VEC) {
        if (n > 0)
#pragma unroll
            for (int i = 0; i < Q; ++i) r.q[i] = reinterpret_cast<const uint4 *>(p)[i];
    } else {
        T *v = reinterpret_cast<T *>(r.q);
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i * stride < n) v[i] = p[i * stride];
    }
}
// Values 2i and 2i + 1 (a bf16 is the high half of its fp32).
__device__ __forceinline__ uint64_t pair(const Raw8<float> &r, int i) {
    const uint32_t *u = reinterpret_cast<const uint32_t *>(r.q);
    return tc::f2_make(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
}
__device__ __forceinline__ uint64_t pair(const Raw8<__nv_bfloat16> &r, int i) {
    const uint32_t u = reinterpret_cast<const uint32_t *>(r.q)[i];
    return tc::f2_make(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
// The larger of m and |a|, |b|; NaN when one of them is.
__device__ __forceinline__ float max_abs(float m, uint64_t v) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(tc::f2_lo(v))));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(tc::f2_hi(v))));
    return m;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t dup(float v) { return tc::f2_make(v, v); }
__device__ __forceinline__ void unpack(float *v, const uint64_t *p) {
#pragma unroll
    for (int i = 0; i < kVec / 2; ++i) {
        v[2 * i] = tc::f2_lo(p[i]);
        v[2 * i + 1] = tc::f2_hi(p[i]);
    }
}
template <bool VEC>
__device__ __forceinline__ void store8(float *p, const float *v, int n, int stride) {
    if (VEC) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i * stride < n) p[i * stride] = v[i];
    }
}
template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float *v, int n, int stride) {
    if (VEC) {
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            q[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(q[0], q[1], q[2], q[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i * stride < n) p[i * stride] = __float2bfloat16_rn(v[i]);
    }
}
// 8-bit codes of the values v (already divided by the scale)
template <bool VEC>
__device__ __forceinline__ void store8_codes(uint8_t *p, const float *v, int n, int stride, bool e4m3) {
    uint32_t q[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kVec; i += 2) {
        uint32_t c;
        if (e4m3)
            c = __nv_cvt_float2_to_fp8x2(make_float2(v[i], v[i + 1]), __NV_SATFINITE, __NV_E4M3);
        else
            c = ((uint32_t)__float2int_rn(v[i]) & 0xffu) | ((uint32_t)__float2int_rn(v[i + 1]) & 0xffu) << 8;
        q[i / 4] |= c << (8 * (i % 4));
    }
    if (VEC) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(q[0], q[1]);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i * stride < n) p[i * stride] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
    }
}

// The scale of a group whose largest |y| is m, and the factor that takes y to its
// codes.  All-zero group, or a scale below 2^-119: 0 and 0.  A value that is not
// finite: NaN and 0.
__device__ __forceinline__ void group_scale(float m, float top, float &scale, float &factor) {
    if (!(m <= 3.4028235e38f)) {
        scale = __uint_as_float(0x7fc00000u);
        factor = 0.f;
    } else {
        // from 2^-119 on the scale, the factor (at most 2^119) and a code times
        // the scale (e4m3: down to 2^-9 of it) are normal numbers
        scale = m / top;
        factor = scale >= 0x1p-119f ? top / m : 0.f;
        if (factor == 0.f) scale = 0.f;
    }
}

enum { kPlain, kRowCodes, kGroupCodes };  // y as numbers; codes with a scale per row, per group

template <typename TX, typename TR, int ITERS, bool VEC, int MODE>
__global__ void __launch_bounds__(ITERS > 1 ? 512 : 1024)
rms_norm_kernel(const NormArgs a) {
    constexpr int H = kVec / 2;
    __shared__ float s_sum[32], s_max[32];
    const int tpr = a.tpr, rpb = blockDim.x / tpr;
    const int lane = threadIdx.x % tpr;
    const long long row = (long long)blockIdx.x * rpb + threadIdx.x / tpr;
    const bool live = row < a.rows;
    const TX *x = static_cast<const TX *>(a.x) + row * a.ldx;
    const TR *r = static_cast<const TR *>(a.r) + row * a.d;
    TR *ro = static_cast<TR *>(a.r_out) + row * a.d;
    // first channel of a step, and how many from it on are this row's; element by
    // element the threads take every tpr-th channel, so that a warp's accesses are
    // adjacent (a group's channels stay with its lanes)
    constexpr bool ADJACENT = VEC || MODE == kGroupCodes;
    const int stride = ADJACENT ? 1 : tpr;
    auto first = [&](int it) { return ADJACENT ? (it * tpr + lane) * kVec : it * tpr * kVec + lane; };
    auto count = [&](int it) { return live ? a.d - first(it) : 0; };

    Raw8<TX> rx[ITERS];
    Raw8<TR> rr[ITERS];
#pragma unroll
    for (int it = 0; it < ITERS; ++it) load8<VEC>(rx[it], x + first(it), count(it), stride);
    if (a.r)
#pragma unroll
        for (int it = 0; it < ITERS; ++it) load8<VEC>(rr[it], r + first(it), count(it), stride);
    // s = x + r, kept as w s
    uint64_t v[ITERS][H], ss2 = 0;
    float mx = 0.f, gmax[ITERS];
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
        gmax[it] = 0.f;
        if (count(it) > 0) {
            Raw8<float> rw;
            if (a.w) load8<VEC>(rw, a.w + first(it), count(it), stride);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                v[it][i] = pair(rx[it], i);
                if (a.r) v[it][i] = tc::f2_add(v[it][i], pair(rr[it], i));
                ss2 = tc::f2_fma(v[it][i], v[it][i], ss2);
            }
            if (a.r_out) {
                float t[kVec];
                unpack(t, v[it]);
                store8<VEC>(ro + first(it), t, count(it), stride);
            }
#pragma unroll
            for (int i = 0; i < H; ++i) {
                if (a.w) v[it][i] = tc::f2_mul(v[it][i], pair(rw, i));
                if (MODE != kPlain) gmax[it] = max_abs(gmax[it], v[it][i]);
            }
        }
        if (MODE == kRowCodes) mx = max_nan(mx, gmax[it]);
        if (MODE == kGroupCodes)  // every lane of a warp takes part in the shuffles
            for (int m = 1; m < a.group / kVec; m <<= 1)
                gmax[it] = max_nan(gmax[it], __shfl_xor_sync(0xffffffffu, gmax[it], m));
    }
    float ss = tc::f2_lo(ss2) + tc::f2_hi(ss2);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, m);
        if (MODE == kRowCodes) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, m));
    }
    if (tpr > 32) {
        const int warp = threadIdx.x / 32, wpr = tpr / 32, w0 = warp / wpr * wpr;
        if (threadIdx.x % 32 == 0) {
            s_sum[warp] = ss;
            s_max[warp] = mx;
        }
        __syncthreads();
        ss = 0.f;
        for (int i = 0; i < wpr; ++i) {
            ss += s_sum[w0 + i];
            if (MODE == kRowCodes) mx = max_nan(mx, s_max[w0 + i]);
        }
    }
    if (!live) return;

    const float rs = rsqrtf(ss / (float)a.d + a.eps);
    const float top = a.y_dtype == RET_I8 ? 127.f : 448.f;
    float factor = 0.f;  // from y to its codes; 0: the codes are 0
    if (MODE == kRowCodes) {
        float scale;
        group_scale(rs * mx, top, scale, factor);
        if (lane == 0) a.scales[row] = scale;
    }
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
        const int e = first(it), n = count(it);
        if (n <= 0) continue;
        if (MODE == kGroupCodes) {
            float scale;
            group_scale(rs * gmax[it], top, scale, factor);
            if (e % a.group == 0) a.scales[row * (a.d / a.group) + e / a.group] = scale;
        }
        float y[kVec];
#pragma unroll
        for (int i = 0; i < H; ++i) {
            // (two products: rs times the factor may lie outside fp32 where y and
            // its code do not, as for tiny rows and a small eps)
            v[it][i] = tc::f2_mul(v[it][i], dup(rs));
            if (MODE != kPlain) v[it][i] = tc::f2_mul(v[it][i], dup(factor));
        }
        unpack(y, v[it]);
        if (MODE != kPlain && factor == 0.f) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) y[i] = 0.f;  // 0 x NaN is not a code
        }
        const long long at = row * a.d + e;
        if (MODE != kPlain)
            store8_codes<VEC>(static_cast<uint8_t *>(a.y) + at, y, n, stride, a.y_dtype == RET_E4M3);
        else if (a.y_dtype == RET_F32)
            store8<VEC>(static_cast<float *>(a.y) + at, y, n, stride);
        else
            store8<VEC>(static_cast<__nv_bfloat16 *>(a.y) + at, y, n, stride);
    }
}

template <typename TX, typename TR, int ITERS>
void launch_iters(const NormArgs &a, bool vec, unsigned blocks, int threads, cudaStream_t st) {
    const int mode = a.y_dtype < RET_I8 ? kPlain : a.group ? kGroupCodes : kRowCodes;
    auto kern = vec ? mode == kPlain      ? rms_norm_kernel<TX, TR, ITERS, true, kPlain>
                      : mode == kRowCodes ? rms_norm_kernel<TX, TR, ITERS, true, kRowCodes>
                                          : rms_norm_kernel<TX, TR, ITERS, true, kGroupCodes>
                    : mode == kPlain      ? rms_norm_kernel<TX, TR, ITERS, false, kPlain>
                      : mode == kRowCodes ? rms_norm_kernel<TX, TR, ITERS, false, kRowCodes>
                                          : rms_norm_kernel<TX, TR, ITERS, false, kGroupCodes>;
    kern<<<blocks, threads, 0, st>>>(a);
}

template <typename TX, typename TR>
cudaError_t launch_t(NormArgs a, bool vec, cudaStream_t st) {
    const int vecs = (a.d + kVec - 1) / kVec;
    // Steps per thread: one where the rows are few (latency), two where they fill
    // the SMs (32768 bf16 rows of 2048 with a residual, e4m3 out: 94 us, and 122
    // with one step, 98 with four; blocks of 256 threads 103), four for the widest.
    int iters = vecs > 1024 ? 4 : vecs > 32 && a.rows > 148 * 8 ? 2 : 1;
    int tpr = 32;
    while (tpr * iters < vecs) tpr *= 2;
    const int threads = tpr > 128 ? tpr : 128;
    const long long rpb = threads / tpr, blocks = (a.rows + rpb - 1) / rpb;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    a.tpr = tpr;
    switch (iters) {
        case 1: launch_iters<TX, TR, 1>(a, vec, (unsigned)blocks, threads, st); break;
        case 2: launch_iters<TX, TR, 2>(a, vec, (unsigned)blocks, threads, st); break;
        default: launch_iters<TX, TR, 4>(a, vec, (unsigned)blocks, threads, st); break;
    }
    const cudaError_t err = cudaGetLastError();
    if (err == cudaSuccess) note_launches(1);
    return err;
}

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace ret

extern "C" ret_status ret_rms_norm(long long rows, int d, int x_dtype, const void *X, long long ldx,
                                   const float *w, int r_dtype, const void *R, void *R_out,
                                   float eps, int y_dtype, void *Y, int group, float *scales,
                                   void *stream) {
    using namespace ret;
    if (rows < 0 || d < 1 || d > RET_MAX_NORM_WIDTH || ldx < d) return RET_ERR_SHAPE;
    if ((x_dtype != RET_F32 && x_dtype != RET_BF16) || (r_dtype != RET_F32 && r_dtype != RET_BF16) ||
        y_dtype < RET_F32 || y_dtype > RET_E4M3)
        return RET_ERR_DTYPE;
    if (!(eps >= 0.0f && std::isfinite(eps))) return RET_ERR_ARG;
    const bool codes = y_dtype == RET_I8 || y_dtype == RET_E4M3;
    if (codes ? (group != 0 && ((group != 32 && group != 64 && group != 128) || d % group)) : group != 0)
        return RET_ERR_SHAPE;
    if (rows > 0 && (!X || !Y || (codes && !scales))) return RET_ERR_NULL;
    if (R_out && !R) return RET_ERR_NULL;
    const unsigned xsize = x_dtype == RET_BF16 ? 2 : 4;
    if (!aligned(X, xsize) || !aligned(w, 16) || !aligned(R, 16) || !aligned(R_out, 16) ||
        !aligned(Y, 16) || !aligned(scales, 16))
        return RET_ERR_ALIGN;
    const ret_status s = validate_device();
    if (s != RET_OK) return s;
    if (rows == 0) return RET_OK;
    NormArgs a{rows, ldx, d, 0, y_dtype, group, eps, X, R, R_out, Y, w, scales};
    // whole kVec pieces on 16-byte boundaries (8 bytes for codes) in every row
    const bool vec = d % kVec == 0 && aligned(X, 16) && (ldx * xsize) % 16 == 0;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (x_dtype == RET_BF16)
        e = r_dtype == RET_BF16 ? launch_t<__nv_bfloat16, __nv_bfloat16>(a, vec, st)
                                : launch_t<__nv_bfloat16, float>(a, vec, st);
    else
        e = r_dtype == RET_BF16 ? launch_t<float, __nv_bfloat16>(a, vec, st)
                                : launch_t<float, float>(a, vec, st);
    return e == cudaSuccess ? RET_OK : RET_ERR_CUDA;
}
