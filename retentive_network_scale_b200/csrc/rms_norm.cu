// rms_norm.cu -- ret_rms_norm: the residual's addition and the root-mean-
// square norm of a block's rows, s = x + r, y = w s / sqrt(mean(s^2) + eps),
// with y in fp32, bf16, or in 8 bits (int8 or e4m3) with one fp32 scale per
// group of channels.
//
// Bound by HBM: x and r are read once, r_out and y written once.  A row is
// spread over `tpr` threads (a power of two, one warp or more) that hold it
// in fp32 registers between the sum of squares and the output, kVec adjacent
// channels per thread and step, so nothing is read twice.  The row's largest
// |w s| comes out of the same reduction as the sum of squares: |y| = |w s| /
// rms, so the 8-bit scale of a whole row needs no second one, and the scale of
// a group of 32, 64 or 128 channels only shuffles among 4, 8 or 16 lanes.
#include <cuda_fp8.h>

#include <cmath>

#include "common.cuh"
#include "launch.h"
#include "retention.h"

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

// kVec elements starting at p, zero past the first n; VEC: all there and
// 16-byte aligned.
template <bool VEC>
__device__ __forceinline__ void load8(float *v, const float *p, int n) {
    if (VEC) {
        const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = i < n ? p[i] : 0.f;
    }
}
template <bool VEC>
__device__ __forceinline__ void load8(float *v, const __nv_bfloat16 *p, int n) {
    if (VEC) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // a bf16 is the high half of its fp32
            v[2 * i] = __uint_as_float(q[i] << 16);
            v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = i < n ? __bfloat162float(p[i]) : 0.f;
    }
}
template <bool VEC>
__device__ __forceinline__ void store8(float *p, const float *v, int n) {
    if (VEC) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i < n) p[i] = v[i];
    }
}
template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float *v, int n) {
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
            if (i < n) p[i] = __float2bfloat16_rn(v[i]);
    }
}
// 8-bit codes of the values v (already divided by the scale)
template <bool VEC>
__device__ __forceinline__ void store8_codes(uint8_t *p, const float *v, int n, bool e4m3) {
    uint32_t q[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const uint32_t c = e4m3 ? (uint32_t)__nv_cvt_float_to_fp8(v[i], __NV_SATFINITE, __NV_E4M3)
                                : (uint32_t)__float2int_rn(v[i]) & 0xffu;
        q[i / 4] |= c << (8 * (i % 4));
    }
    if (VEC) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(q[0], q[1]);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i < n) p[i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
    }
}

// The scale of a group whose largest |y| has the bits `amax` (as unsigned
// integers the bits of NaN and infinity are the largest, so a maximum over
// them keeps a value that is not finite), and the factor that takes y to its
// codes.  All-zero group: 0 and 0.  A value that is not finite: NaN and 0.
__device__ __forceinline__ void group_scale(uint32_t amax, float top, float &scale, float &factor) {
    const float m = __uint_as_float(amax);
    if (amax >= 0x7f800000u) {
        scale = __uint_as_float(0x7fc00000u);
        factor = 0.f;
    } else {
        scale = m / top;
        // top / m overflows for m below about 2^-119; such codes are lost
        // with the scale's own precision (it is denormal there)
        factor = scale > 1.2e-36f ? top / m : 0.f;
        if (factor == 0.f) scale = 0.f;
    }
}

template <typename TX, typename TR, int ITERS, bool VEC>
__global__ void __launch_bounds__(1024)
rms_norm_kernel(const NormArgs a) {
    __shared__ float s_sum[32];
    __shared__ uint32_t s_max[32];
    const int tpr = a.tpr, rpb = blockDim.x / tpr;
    const int lane = threadIdx.x % tpr;
    const long long row = (long long)blockIdx.x * rpb + threadIdx.x / tpr;
    const bool live = row < a.rows;
    const TX *x = static_cast<const TX *>(a.x) + row * a.ldx;
    const TR *r = static_cast<const TR *>(a.r) + row * a.d;
    TR *ro = static_cast<TR *>(a.r_out) + row * a.d;

    // s = x + r (kept as w s from here on), its squares and its largest |w s|
    float v[ITERS][kVec];
    float ss = 0.f;
    uint32_t mx = 0;
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
        const int e = (it * tpr + lane) * kVec, n = a.d - e;
        if (live && n > 0) {
            load8<VEC>(v[it], x + e, n);
            if (a.r) {
                float t[kVec];
                load8<VEC>(t, r + e, n);
#pragma unroll
                for (int i = 0; i < kVec; ++i) v[it][i] += t[i];
            }
        }
    }
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
        const int e = (it * tpr + lane) * kVec, n = a.d - e;
        if (live && n > 0) {
            float w[kVec];
            if (a.w) load8<VEC>(w, a.w + e, n);
            if (a.r_out) store8<VEC>(ro + e, v[it], n);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                ss = fmaf(v[it][i], v[it][i], ss);
                if (a.w) v[it][i] *= w[i];
                mx = max(mx, __float_as_uint(fabsf(v[it][i])));
            }
        }
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, m);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, m));
    }
    if (tpr > 32) {
        const int warp = threadIdx.x / 32, wpr = tpr / 32, w0 = warp / wpr * wpr;
        if (threadIdx.x % 32 == 0) {
            s_sum[warp] = ss;
            s_max[warp] = mx;
        }
        __syncthreads();
        ss = 0.f;
        mx = 0;
        for (int i = 0; i < wpr; ++i) {
            ss += s_sum[w0 + i];
            mx = max(mx, s_max[w0 + i]);
        }
    }
    if (!live) return;

    const float rs = rsqrtf(ss / (float)a.d + a.eps);
    const bool codes = a.y_dtype >= RET_I8;
    const float top = a.y_dtype == RET_I8 ? 127.f : 448.f;
    const int groups = codes ? (a.group ? a.d / a.group : 1) : 0;
    float factor = rs;
    if (codes && !a.group) {
        float scale;
        group_scale(__float_as_uint(rs * __uint_as_float(mx)), top, scale, factor);
        if (lane == 0) a.scales[row] = scale;
        factor *= rs;
    }
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
        const int e = (it * tpr + lane) * kVec, n = a.d - e;
        const bool in = n > 0;
        if (codes && a.group) {
            // every lane of a warp takes part in the shuffles
            uint32_t g = 0;
            if (in)
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    g = max(g, __float_as_uint(fabsf(rs * v[it][i])));
                }
            for (int m = 1; m < a.group / kVec; m <<= 1) g = max(g, __shfl_xor_sync(0xffffffffu, g, m));
            float scale;
            group_scale(g, top, scale, factor);
            if (in && e % a.group == 0) a.scales[row * groups + e / a.group] = scale;
            factor *= rs;
        }
        if (!in) continue;
        if (codes && factor == 0.f) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) v[it][i] = 0.f;  // 0 x NaN is not a code
        } else {
#pragma unroll
            for (int i = 0; i < kVec; ++i) v[it][i] *= factor;
        }
        const long long at = row * a.d + e;
        switch (a.y_dtype) {
            case RET_F32: store8<VEC>(static_cast<float *>(a.y) + at, v[it], n); break;
            case RET_BF16: store8<VEC>(static_cast<__nv_bfloat16 *>(a.y) + at, v[it], n); break;
            default: store8_codes<VEC>(static_cast<uint8_t *>(a.y) + at, v[it], n, a.y_dtype == RET_E4M3);
        }
    }
}

template <typename TX, typename TR, int ITERS>
void launch_iters(const NormArgs &a, bool vec, unsigned blocks, int threads, cudaStream_t st) {
    if (vec)
        rms_norm_kernel<TX, TR, ITERS, true><<<blocks, threads, 0, st>>>(a);
    else
        rms_norm_kernel<TX, TR, ITERS, false><<<blocks, threads, 0, st>>>(a);
}

template <typename TX, typename TR>
cudaError_t launch_t(NormArgs a, bool vec, cudaStream_t st) {
    const int vecs = (a.d + kVec - 1) / kVec;
    const int iters = vecs > 256 ? 2 : 1;
    int tpr = 32;
    while (tpr * iters < vecs) tpr *= 2;
    const int threads = tpr > 256 ? tpr : 256;
    const long long rpb = threads / tpr, blocks = (a.rows + rpb - 1) / rpb;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    a.tpr = tpr;
    if (iters == 1)
        launch_iters<TX, TR, 1>(a, vec, (unsigned)blocks, threads, st);
    else
        launch_iters<TX, TR, 2>(a, vec, (unsigned)blocks, threads, st);
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
