// selective_scan.cu -- ret_selective_scan: the diagonal recurrence whose decay
// depends on the token,
//     h_t = exp(d_t A) h_{t-1} + d_t u_t B_t,  y_t = (C_t . h_t + skip u_t) swish(z_t),
// per channel with N states, for prompts and for single tokens over an fp32
// state.
#include <cmath>

#include "common.cuh"
#include "launch.h"
#include "retention.h"

namespace ret {
namespace {

struct ScanArgs {
    int B, L, D, N, G, dpg;  // dpg: channels per group
    int softplus, blocks_per_group;
    long long ldu, ldd, ldz, ldb, ldc;
    const void *u, *delta, *z, *bm, *cm;
    const float *A, *skip, *bias;
    const int *lengths;
    const float *s_in;
    float *s_out;
    void *y;
};

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// log(1 + e^x) = max(x, 0) + log1p(e^-|x|).  With e = e^-|x| in (0, 1],
// log1p(e) = 2 artanh(s), s = e / (2 + e) <= 1/3, by the series of artanh up
// to s^15 (the rest is below 2^-27 of the value), which keeps its relative
// accuracy for small e, where log(1 + e) would not.
__device__ __forceinline__ float softplus(float x) {
    const float e = exp2_fast(-fabsf(x) * kLog2e);
    const float s = __fdividef(e, 2.f + e), q = s * s;
    float p = 1.f / 15.f;
    p = fmaf(p, q, 1.f / 13.f);
    p = fmaf(p, q, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    p = fmaf(p, q, 1.f);
    return fmaxf(x, 0.f) + 2.f * s * p;
}
__device__ __forceinline__ float swish(float v) { return __fdividef(v, 1.f + exp2_fast(-v * kLog2e)); }

// E consecutive elements of a row from p, zero past the first n; in one piece
// where the address allows it.
template <typename T, int E>
struct alignas(sizeof(T) * E > 16 ? 16 : sizeof(T) * E) Raw {
    T v[E];
};
template <typename T, int E>
__device__ __forceinline__ Raw<T, E> load_raw(const T *p, int n) {
    Raw<T, E> r;
    constexpr unsigned mask = alignof(Raw<T, E>) - 1;
    if (n >= E && (reinterpret_cast<uintptr_t>(p) & mask) == 0) {
        r = *reinterpret_cast<const Raw<T, E> *>(p);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            r.v[i] = T(0.f);
            if (i < n) r.v[i] = p[i];
        }
    }
    return r;
}
template <typename T, int E>
__device__ __forceinline__ void store_raw(T *p, const Raw<T, E> &r, int n) {
    constexpr unsigned mask = alignof(Raw<T, E>) - 1;
    if (n >= E && (reinterpret_cast<uintptr_t>(p) & mask) == 0) {
        *reinterpret_cast<Raw<T, E> *>(p) = r;
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (i < n) p[i] = r.v[i];
    }
}
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float &d, float v) { d = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16 &d, float v) { d = __float2bfloat16_rn(v); }

// One CTA: kChannels channels of one group of one sequence, all N states, all
// rows.  LANES threads share a channel and hold SPT states each (state
// n = 4 LANES (i / 4) + 4 lane + i % 4 in register i), so that B_t and C_t are
// read from shared memory in 16-byte pieces without bank conflicts.  Rows go in
// tiles: the threads turn a tile's delta into d = softplus(delta + bias) and
// d u once per row and channel, then run the recurrence on it.
template <typename T, int SPT, int LANES, int TT>
__global__ void __launch_bounds__(128)
selective_scan_kernel(const ScanArgs a) {
    constexpr int NT = 128, CH = NT / LANES, NP = SPT * LANES;
    constexpr int E = TT / LANES;           // staged elements per thread and operand
    constexpr int VS = SPT < 4 ? SPT : 4;   // states per 16-byte piece
    constexpr int YS = CH + 32 / LANES;     // row stride of s_y: no bank conflicts
    constexpr int NB = (TT * NP + NT - 1) / NT;
    static_assert(E * LANES == TT && TT % LANES == 0, "tile");
    __shared__ float2 s_du[TT][CH];
    __shared__ __align__(16) float s_b[TT][NP], s_c[TT][NP];
    __shared__ float s_y[TT][YS];

    const int tid = threadIdx.x, lane = tid % LANES, ch = tid / LANES;
    int blk = blockIdx.x;
    const int cb = blk % a.blocks_per_group;
    blk /= a.blocks_per_group;
    const int g = blk % a.G, b = blk / a.G;
    const int c0 = g * a.dpg + cb * CH;                // first channel
    const int nch = min(CH, a.dpg - cb * CH);          // channels of this CTA
    const int len = a.lengths ? min(max(a.lengths[b], 0), a.L) : a.L;

    auto state_of = [&](int i) { return i / VS * (VS * LANES) + lane * VS + i % VS; };
    const bool live = ch < nch;
    float h[SPT], A2[SPT];
#pragma unroll
    for (int i = 0; i < SPT; ++i) {
        const int n = state_of(i);
        const bool in = live && n < a.N;
        A2[i] = in ? a.A[(long long)(c0 + ch) * a.N + n] * kLog2e : 0.f;
        h[i] = in && a.s_in ? a.s_in[((long long)b * a.D + c0 + ch) * a.N + n] : 0.f;
    }

    // staging: thread -> row sr of the tile, channels sc .. sc + E - 1
    constexpr int TPR = CH / E;
    const int sr = tid / TPR, sc = tid % TPR * E;
    const int sn = nch - sc;  // of them live (may be <= 0)
    const long long row0 = (long long)b * a.L;
    const T *pu = static_cast<const T *>(a.u) + row0 * a.ldu + c0 + sc;
    const T *pd = static_cast<const T *>(a.delta) + row0 * a.ldd + c0 + sc;
    const T *pz = a.z ? static_cast<const T *>(a.z) + row0 * a.ldz + c0 + sc : nullptr;
    const T *pb = static_cast<const T *>(a.bm) + row0 * a.ldb + (long long)g * a.N;
    const T *pc = static_cast<const T *>(a.cm) + row0 * a.ldc + (long long)g * a.N;
    T *py = static_cast<T *>(a.y) + row0 * a.D + c0 + sc;
    float bias[E], skip[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        bias[i] = a.bias && i < sn ? a.bias[c0 + sc + i] : 0.f;
        skip[i] = a.skip && i < sn ? a.skip[c0 + sc + i] : 0.f;
    }

    Raw<T, E> ru, rd, rz;
    T rb[NB], rc[NB];
    auto fetch = [&](int t0) {  // the tile's u, delta, B, C
        const int t = t0 + sr, n = t < len ? sn : 0;
        ru = load_raw<T, E>(pu + (long long)t * a.ldu, n);
        rd = load_raw<T, E>(pd + (long long)t * a.ldd, n);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int idx = tid + j * NT, r = idx / NP, n2 = idx % NP;
            const bool in = (TT * NP % NT == 0 || r < TT) && t0 + r < len && n2 < a.N;
            rb[j] = in ? pb[(long long)(t0 + r) * a.ldb + n2] : T(0.f);
            rc[j] = in ? pc[(long long)(t0 + r) * a.ldc + n2] : T(0.f);
        }
    };
    fetch(0);

    for (int t0 = 0; t0 < len; t0 += TT) {
        const bool inside = t0 + sr < len;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float u = to_f(ru.v[i]);
            float d = to_f(rd.v[i]) + bias[i];
            if (a.softplus) d = softplus(d);
            if (!inside) d = 0.f;
            s_du[sr][sc + i] = make_float2(d, d * u);
            s_y[sr][sc + i] = skip[i] * u;
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int idx = tid + j * NT;
            if (TT * NP % NT == 0 || idx < TT * NP) {
                (&s_b[0][0])[idx] = to_f(rb[j]);
                (&s_c[0][0])[idx] = to_f(rc[j]);
            }
        }
        __syncthreads();
        if (pz) rz = load_raw<T, E>(pz + (long long)(t0 + sr) * a.ldz, inside ? sn : 0);
        if (t0 + TT < len) fetch(t0 + TT);

        // LANES rows at a time: lane l of a channel ends up with row l's sum
#pragma unroll 1
        for (int t = 0; t < TT; t += LANES) {
            float part[LANES];
#pragma unroll
            for (int k = 0; k < LANES; ++k) {
                const float2 du = s_du[t + k][ch];
                float acc = 0.f;
#pragma unroll
                for (int i0 = 0; i0 < SPT; i0 += VS) {
                    float bv[VS], cv[VS];
                    const float *qb = &s_b[t + k][i0 * LANES + lane * VS];
                    const float *qc = &s_c[t + k][i0 * LANES + lane * VS];
                    if (VS == 4) {
                        *reinterpret_cast<float4 *>(bv) = *reinterpret_cast<const float4 *>(qb);
                        *reinterpret_cast<float4 *>(cv) = *reinterpret_cast<const float4 *>(qc);
                    } else {
#pragma unroll
                        for (int i = 0; i < VS; ++i) { bv[i] = qb[i]; cv[i] = qc[i]; }
                    }
#pragma unroll
                    for (int i = 0; i < VS; ++i) {
                        const float e = exp2_fast(du.x * A2[i0 + i]);
                        h[i0 + i] = fmaf(e, h[i0 + i], du.y * bv[i]);
                        acc = fmaf(cv[i], h[i0 + i], acc);
                    }
                }
                part[k] = acc;
            }
#pragma unroll
            for (int m = LANES / 2; m > 0; m >>= 1) {
                const bool up = lane & m;
#pragma unroll
                for (int k = 0; k < m; ++k) {
                    const float keep = up ? part[k + m] : part[k], send = up ? part[k] : part[k + m];
                    part[k] = keep + __shfl_xor_sync(0xffffffffu, send, m);
                }
            }
            s_y[t + lane][ch] += part[0];
        }
        __syncthreads();
        if (inside && sn > 0) {
            Raw<T, E> out;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                float y = s_y[sr][sc + i];
                if (pz) y *= swish(to_f(rz.v[i]));
                from_f(out.v[i], y);
            }
            store_raw<T, E>(py + (long long)(t0 + sr) * a.D, out, sn);
        }
    }
    if (a.s_out && live) {
#pragma unroll
        for (int i = 0; i < SPT; ++i) {
            const int n = state_of(i);
            if (n < a.N) a.s_out[((long long)b * a.D + c0 + ch) * a.N + n] = h[i];
        }
    }
}

template <typename T, int SPT, int LANES, int TT>
cudaError_t launch_scan(ScanArgs a, cudaStream_t st) {
    constexpr int CH = 128 / LANES;
    a.blocks_per_group = (a.dpg + CH - 1) / CH;
    const long long blocks = (long long)a.B * a.G * a.blocks_per_group;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    selective_scan_kernel<T, SPT, LANES, TT><<<(unsigned)blocks, 128, 0, st>>>(a);
    const cudaError_t err = cudaGetLastError();
    if (err == cudaSuccess) note_launches(1);
    return err;
}

template <typename T>
cudaError_t launch_n(const ScanArgs &a, cudaStream_t st) {
    if (a.N <= 8) return launch_scan<T, 2, 4, 32>(a, st);
    if (a.N <= 16) return launch_scan<T, 4, 4, 32>(a, st);
    if (a.N <= 32) return launch_scan<T, 8, 4, 32>(a, st);
    if (a.N <= 64) return launch_scan<T, 16, 4, 16>(a, st);
    return launch_scan<T, 32, 4, 8>(a, st);
}

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace ret

extern "C" ret_status ret_selective_scan(const ret_scan_desc *d, const void *U, const void *delta,
                                         const float *delta_bias, const float *A, const void *Bm,
                                         const void *Cm, const float *skip, const void *Z,
                                         const int *lengths, const float *state_in,
                                         float *state_out, void *Y, void *stream) {
    using namespace ret;
    if (!d) return RET_ERR_NULL;
    if (d->B < 0 || d->L < 0 || d->D < 1 || d->N < 1 || d->N > RET_MAX_SCAN_STATES || d->G < 1 ||
        d->D % d->G)
        return RET_ERR_SHAPE;
    if (d->dtype != RET_F32 && d->dtype != RET_BF16) return RET_ERR_DTYPE;
    if (d->softplus != 0 && d->softplus != 1) return RET_ERR_ARG;
    const long long gn = (long long)d->G * d->N;
    if (d->ldu < d->D || d->ldd < d->D || (Z && d->ldz < d->D) || d->ldb < gn || d->ldc < gn)
        return RET_ERR_SHAPE;
    const bool rows = (long long)d->B * d->L > 0;
    if (rows && (!U || !delta || !A || !Bm || !Cm || !Y)) return RET_ERR_NULL;
    const unsigned size = d->dtype == RET_BF16 ? 2 : 4;
    if (!aligned(U, size) || !aligned(delta, size) || !aligned(Bm, size) || !aligned(Cm, size) ||
        !aligned(Z, size) || !aligned(lengths, 4) || !aligned(A, 16) || !aligned(skip, 16) ||
        !aligned(delta_bias, 16) || !aligned(state_in, 16) || !aligned(state_out, 16) || !aligned(Y, 16))
        return RET_ERR_ALIGN;
    const ret_status s = validate_device();
    if (s != RET_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!rows) {
        // no rows: the state passes through unchanged
        const size_t bytes = sizeof(float) * (size_t)d->B * d->D * d->N;
        if (!state_out || state_out == state_in || bytes == 0) return RET_OK;
        const cudaError_t e = state_in ? cudaMemcpyAsync(state_out, state_in, bytes, cudaMemcpyDeviceToDevice, st)
                                       : cudaMemsetAsync(state_out, 0, bytes, st);
        return e == cudaSuccess ? RET_OK : RET_ERR_CUDA;
    }
    ScanArgs a{d->B, d->L, d->D, d->N, d->G, d->D / d->G, d->softplus, 0, d->ldu, d->ldd, d->ldz,
               d->ldb, d->ldc, U, delta, Z, Bm, Cm, A, skip, delta_bias, lengths, state_in, state_out, Y};
    const cudaError_t e = d->dtype == RET_BF16 ? launch_n<__nv_bfloat16>(a, st) : launch_n<float>(a, st);
    return e == cudaSuccess ? RET_OK : RET_ERR_CUDA;
}
