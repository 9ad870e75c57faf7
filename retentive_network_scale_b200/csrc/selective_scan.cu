// selective_scan.cu -- ret_selective_scan: the diagonal recurrence whose decay
// depends on the token,
//     h_t = exp(d_t A) h_{t-1} + d_t u_t B_t,  y_t = (C_t . h_t + skip u_t) swish(z_t),
// per channel with N states, for prompts and for single tokens over an fp32
// state.
#include <cmath>

#include "common.cuh"
#include "launch.h"
#include "retention.h"
#include "tc_util.cuh"

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

// log(1 + e^x) = max(x, 0) + log1p(e^-|x|).  log1p(e) / e for e = e^-|x| in
// (0, 1] is a polynomial of degree 8 fitted by reweighted least squares at
// Chebyshev nodes (relative error 3e-8), which keeps the relative accuracy for
// small e, where log(1 + e) would not, and leaves the special-function unit to
// the decays.
__device__ __forceinline__ float softplus(float x) {
    const float e = exp2_fast(-fabsf(x) * kLog2e);
    float p = 0.005232624709606171f;
    p = fmaf(p, e, -0.029504960402846336f);
    p = fmaf(p, e, 0.0782255008816719f);
    p = fmaf(p, e, -0.1366320699453354f);
    p = fmaf(p, e, 0.1910598874092102f);
    p = fmaf(p, e, -0.2484297752380371f);
    p = fmaf(p, e, 0.3331909477710724f);
    p = fmaf(p, e, -0.4999949336051941f);
    p = fmaf(p, e, 0.9999999403953552f);
    return fmaf(p, e, fmaxf(x, 0.f));
}
__device__ __forceinline__ float swish(float v) { return __fdividef(v, 1.f + exp2_fast(-v * kLog2e)); }

// E consecutive elements.
template <typename T, int E>
struct alignas(sizeof(T) * E > 16 ? 16 : sizeof(T) * E) Raw {
    T v[E];
};
// From shared memory: in one piece (WHOLE) or element by element.
template <bool WHOLE, typename T, int E>
__device__ __forceinline__ Raw<T, E> shared_raw(const T *p) {
    Raw<T, E> r;
    if (WHOLE) {
        r = *reinterpret_cast<const Raw<T, E> *>(p);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) r.v[i] = p[i];
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// Sizes.  A warp owns CPW channels (LANES threads each) and does all the work
// on them itself; the CTA's four warps share the tiles of B and C.
template <typename T, int SPT, int LANES, int TT, bool VEC>
struct ScanTile {
    static constexpr int WARPS = 4, NT = 32 * WARPS, CPW = 32 / LANES, CH = WARPS * CPW, NP = SPT * LANES;
    static constexpr int E = TT / LANES;                 // elements per thread, operand and tile
    static constexpr int GRP = 32 / TT;                  // threads that share a row of the warp's channels
    static constexpr int WORDS = CPW * (int)sizeof(T) / 16 + (VEC ? 0 : 1);  // 16-byte words of a row
    static constexpr int RS = 16 * (WORDS | 1);          // its bytes: an odd number of words, no bank conflicts
    static constexpr int DS = TT + 2;                    // row stride of du (float2)
    static constexpr int YS = TT + 4;                    // row stride of y
    static constexpr int PE = 8;                         // elements of a piece of B or C
    static constexpr int PR = NP / PE;                   // pieces per row
    static constexpr int PIECES = 2 * TT * PR;           // of both
    static constexpr int NB = (PIECES + NT - 1) / NT;    // per thread
    static constexpr int PB = PE * (int)sizeof(T) + (VEC ? 0 : 16);  // bytes a copied piece takes
    static_assert(TT <= 32 && E * LANES == TT && NP % PE == 0, "tile");
    struct Warp {
        uint8_t in[2][3][TT][RS];  // u, delta, z as copied, two tiles
        float2 du[CPW][DS];        // (d, d u), rows of a channel adjacent
        float y[CPW][LANES][YS];   // every lane's part of y
    };
    struct Smem {
        Warp warp[WARPS];
        float bc[2][2][TT][NP];            // two tiles of B and C
        uint8_t bcin[2][NB][NT][PB];       // as copied, by the thread that converts it
    };
};

// The recurrence: LANES threads share a channel and hold SPT states each (state
// n = 4 LANES (i / 4) + 4 lane + i % 4 in register i, so that B_t and C_t are
// read from shared memory in 16-byte pieces without bank conflicts), two states
// to a packed register pair.  Rows go in tiles of TT.  While a tile is computed
// the next one is copied to shared memory as it is; then each warp turns its
// channels' delta into d = softplus(delta + bias) and d u, once per row and
// channel, and the CTA its share of B and C into fp32 (the tile's only barrier);
// the parts of y that the lanes of a channel write are added, gated and rounded
// by the same warp.
//
// VEC: every row of every operand starts on 16 bytes.  Otherwise the aligned
// words that hold a row are copied and the row starts a few elements into its
// place (bytes before an unaligned row are in its first word, so in the same
// allocation; bytes past its end are not read).
template <typename T, int SPT, int LANES, int TT, bool VEC>
__global__ void __launch_bounds__(128, SPT <= 8 ? 4 : 2)
selective_scan_kernel(const ScanArgs a) {
    using C = ScanTile<T, SPT, LANES, TT, VEC>;
    constexpr int NT = C::NT, CPW = C::CPW, NP = C::NP, E = C::E, NB = C::NB, PE = C::PE;
    constexpr int PR = SPT / 2;  // state pairs
    constexpr int SZ = (int)sizeof(T);
    extern __shared__ __align__(16) uint8_t dsm[];
    auto &sm = *reinterpret_cast<typename C::Smem *>(dsm);

    const int tid = threadIdx.x, wl = tid % 32, lane = tid % LANES, ch = wl / LANES;
    auto &sw = sm.warp[tid / 32];
    int blk = blockIdx.x;
    const int cb = blk % a.blocks_per_group;
    blk /= a.blocks_per_group;
    const int g = blk % a.G, b = blk / a.G;
    const int w0 = cb * C::CH + tid / 32 * CPW;        // first channel of the warp in its group
    const int c0 = g * a.dpg + w0;
    const int nch = max(0, min(CPW, a.dpg - w0));      // channels of this warp
    const int len = a.lengths ? min(max(a.lengths[b], 0), a.L) : a.L;
    const long long row0 = (long long)b * a.L;

    // this thread's row of a tile, and its E channels from sc on
    const int sr = wl % TT, sg = wl / TT, sc = sg * E;
    const T *pu = static_cast<const T *>(a.u) + (row0 + sr) * a.ldu + c0;
    const T *pd = static_cast<const T *>(a.delta) + (row0 + sr) * a.ldd + c0;
    const T *pz = a.z ? static_cast<const T *>(a.z) + (row0 + sr) * a.ldz + c0 : nullptr;
    T *py = static_cast<T *>(a.y) + (row0 + sr) * a.D + c0 + sc;
    auto misfit = [](const T *p) { return VEC ? 0 : (int)(reinterpret_cast<uintptr_t>(p) & 15u); };
    auto copy_row = [&](const T *p, bool there, uint8_t *dst) {
        const int head = misfit(p), end = there ? head + nch * SZ : 0;
        const uint8_t *base = there ? reinterpret_cast<const uint8_t *>(p) - head : static_cast<const uint8_t *>(a.u) - misfit(static_cast<const T *>(a.u));
        const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
#pragma unroll
        for (int w = 0; w < C::WORDS; w += C::GRP) {
            if (C::WORDS % C::GRP == 0 || w + sg < C::WORDS) {
                const int at = 16 * (w + sg), n = min(16, max(0, end - at));
                cp_async16(d + at, n ? base + at : base, n);
            }
        }
    };
    // pieces of B and C: this thread's j-th
    auto piece = [&](int j, int &r, int &n0, bool &c) {
        const int p = tid + j * NT;
        r = p / C::PR % TT;
        n0 = p % C::PR * PE;
        c = p >= TT * C::PR;
        return C::PIECES % NT == 0 || p < C::PIECES;
    };
    auto piece_at = [&](int t, int n0, bool c) {
        return static_cast<const T *>(c ? a.cm : a.bm) + (row0 + t) * (c ? a.ldc : a.ldb) + (long long)g * a.N + n0;
    };
    // copies the tile that starts at row t0 into slot k; advances the pointers
    auto copy_tile = [&](int t0, int k) {
        const bool there = t0 + sr < len && nch > 0;
        copy_row(pu, there, sw.in[k][0][sr]);
        copy_row(pd, there, sw.in[k][1][sr]);
        if (pz) copy_row(pz, there, sw.in[k][2][sr]);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            int r, n0;
            bool c;
            if (piece(j, r, n0, c)) {
                const T *p = piece_at(t0 + r, n0, c);
                const int n = t0 + r < len ? min(PE, max(0, a.N - n0)) : 0;
                const int head = n ? misfit(p) : 0, end = head + n * SZ;
                const uint8_t *base = n ? reinterpret_cast<const uint8_t *>(p) - head : static_cast<const uint8_t *>(a.u) - misfit(static_cast<const T *>(a.u));
                const uint32_t d = (uint32_t)__cvta_generic_to_shared(sm.bcin[k][j][tid]);
#pragma unroll
                for (int w = 0; w < C::PB; w += 16) {
                    const int m = n ? min(16, max(0, end - w)) : 0;
                    cp_async16(d + w, m ? base + w : base, m);
                }
            }
        }
        cp_async_commit();
    };
    // B and C of the tile at t0, from slot k to the fp32 tile k
    auto convert_bc = [&](int t0, int k) {
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            int r, n0;
            bool c;
            if (piece(j, r, n0, c)) {
                const bool there = t0 + r < len;
                const int head = VEC || !there ? 0 : misfit(piece_at(t0 + r, n0, c)) / SZ;
                const Raw<T, PE> v = shared_raw<VEC, T, PE>(reinterpret_cast<const T *>(sm.bcin[k][j][tid]) + head);
                float f[PE];
#pragma unroll
                for (int i = 0; i < PE; ++i) f[i] = VEC || (there && n0 + i < a.N) ? to_f(v.v[i]) : 0.f;
                float *dst = &sm.bc[k][c][r][n0];
                *reinterpret_cast<float4 *>(dst) = make_float4(f[0], f[1], f[2], f[3]);
                *reinterpret_cast<float4 *>(dst + 4) = make_float4(f[4], f[5], f[6], f[7]);
            }
        }
    };

    if (len > 0) copy_tile(0, 0);

    auto state_of = [&](int i) { return i / 4 * (4 * LANES) + lane * 4 + i % 4; };
    const bool live = ch < nch;
    const long long hrow = ((long long)b * a.D + c0 + ch) * a.N;
    uint64_t h[PR], A2[PR];
#pragma unroll
    for (int j = 0; j < PR; ++j) {
        float av[2], hv[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = state_of(2 * j + i);
            const bool in = live && n < a.N;
            av[i] = in ? a.A[(long long)(c0 + ch) * a.N + n] * kLog2e : 0.f;
            hv[i] = in && a.s_in ? a.s_in[hrow + n] : 0.f;
        }
        A2[j] = tc::f2_make(av[0], av[1]);
        h[j] = tc::f2_make(hv[0], hv[1]);
    }
    float bias[E], skip[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        bias[i] = a.bias && sc + i < nch ? a.bias[c0 + sc + i] : 0.f;
        skip[i] = a.skip && sc + i < nch ? a.skip[c0 + sc + i] : 0.f;
    }

    for (int t0 = 0, k = 0; t0 < len; t0 += TT, k ^= 1) {
        cp_async_wait();
        convert_bc(t0, k);
        __syncthreads();  // also: every warp is done with the B and C of the tile before last
        const bool inside = t0 + sr < len;
        const Raw<T, E> ru = shared_raw<VEC, T, E>(reinterpret_cast<const T *>(sw.in[k][0][sr] + misfit(pu)) + sc);
        {
            const Raw<T, E> rd = shared_raw<VEC, T, E>(reinterpret_cast<const T *>(sw.in[k][1][sr] + misfit(pd)) + sc);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                float d = to_f(rd.v[i]) + bias[i];
                if (a.softplus) d = softplus(d);
                const bool in1 = inside && (VEC || sc + i < nch);
                sw.du[sc + i][sr] = make_float2(in1 ? d : 0.f, in1 ? d * to_f(ru.v[i]) : 0.f);
            }
        }
        const T *pz_now = pz;
        pu += TT * a.ldu;
        pd += TT * a.ldd;
        if (pz) pz += TT * a.ldz;
        if (t0 + TT < len) copy_tile(t0 + TT, k ^ 1);
        __syncwarp();

        const float *tb = &sm.bc[k][0][0][lane * 4], *tc_ = &sm.bc[k][1][0][lane * 4];
#pragma unroll(SPT <= 8 ? TT / 4 : 1)
        for (int t = 0; t < TT; t += 4) {
            float part[4];
#pragma unroll
            for (int r = 0; r < 4; r += 2) {
                const float4 du2 = *reinterpret_cast<const float4 *>(&sw.du[ch][t + r]);
#pragma unroll
                for (int rr = 0; rr < 2; ++rr) {
                    const float d = rr ? du2.z : du2.x, du = rr ? du2.w : du2.y;
                    const uint64_t dd = tc::f2_make(d, d), dudu = tc::f2_make(du, du);
                    uint64_t acc = 0;
#pragma unroll
                    for (int j = 0; j < PR; j += 2) {
                        const ulonglong2 bv = *reinterpret_cast<const ulonglong2 *>(tb + (t + r + rr) * NP + j * 2 * LANES);
                        const ulonglong2 cv = *reinterpret_cast<const ulonglong2 *>(tc_ + (t + r + rr) * NP + j * 2 * LANES);
                        const uint64_t p0 = tc::f2_mul(dd, A2[j]), p1 = tc::f2_mul(dd, A2[j + 1]);
                        const uint64_t e0 = tc::f2_make(exp2_fast(tc::f2_lo(p0)), exp2_fast(tc::f2_hi(p0)));
                        const uint64_t e1 = tc::f2_make(exp2_fast(tc::f2_lo(p1)), exp2_fast(tc::f2_hi(p1)));
                        h[j] = tc::f2_fma(e0, h[j], tc::f2_mul(dudu, bv.x));
                        h[j + 1] = tc::f2_fma(e1, h[j + 1], tc::f2_mul(dudu, bv.y));
                        acc = j ? tc::f2_fma(cv.x, h[j], acc) : tc::f2_mul(cv.x, h[j]);
                        acc = tc::f2_fma(cv.y, h[j + 1], acc);
                    }
                    part[r + rr] = tc::f2_lo(acc) + tc::f2_hi(acc);
                }
            }
            *reinterpret_cast<float4 *>(&sw.y[ch][lane][t]) = make_float4(part[0], part[1], part[2], part[3]);
        }
        __syncwarp();
        if (inside && sc < nch) {
            float y[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                y[i] = skip[i] * to_f(ru.v[i]);
#pragma unroll
                for (int l = 0; l < LANES; ++l) y[i] += sw.y[sc + i][l][sr];
            }
            if (pz) {
                const Raw<T, E> rz = shared_raw<VEC, T, E>(reinterpret_cast<const T *>(sw.in[k][2][sr] + misfit(pz_now)) + sc);
#pragma unroll
                for (int i = 0; i < E; ++i) y[i] *= swish(to_f(rz.v[i]));
            }
            Raw<T, E> out;
#pragma unroll
            for (int i = 0; i < E; ++i) from_f(out.v[i], y[i]);
            store_raw<T, E>(py, out, nch - sc);
        }
        py += TT * (long long)a.D;
    }
    if (a.s_out && live) {
#pragma unroll
        for (int j = 0; j < PR; ++j) {
            const int n = state_of(2 * j);  // n + 1 is the pair's other state
            if (n < a.N) a.s_out[hrow + n] = tc::f2_lo(h[j]);
            if (n + 1 < a.N) a.s_out[hrow + n + 1] = tc::f2_hi(h[j]);
        }
    }
}

template <typename T, int SPT, int LANES, int TT, bool VEC>
cudaError_t launch_vec(ScanArgs a, cudaStream_t st) {
    using C = ScanTile<T, SPT, LANES, TT, VEC>;
    a.blocks_per_group = (a.dpg + C::CH - 1) / C::CH;
    const long long blocks = (long long)a.B * a.G * a.blocks_per_group;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto kern = selective_scan_kernel<T, SPT, LANES, TT, VEC>;
    constexpr int smem = (int)sizeof(typename C::Smem);
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    kern<<<(unsigned)blocks, C::NT, smem, st>>>(a);
    err = cudaGetLastError();
    if (err == cudaSuccess) note_launches(1);
    return err;
}

template <typename T, int SPT, int LANES, int TT>
cudaError_t launch_scan(const ScanArgs &a, cudaStream_t st) {
    auto fits = [](const void *p, long long ld) {
        return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * (long long)sizeof(T) % 16 == 0;
    };
    const bool vec = fits(a.u, a.ldu) && fits(a.delta, a.ldd) && (!a.z || fits(a.z, a.ldz)) && fits(a.bm, a.ldb) &&
                     fits(a.cm, a.ldc) && fits(a.y, a.D) && (a.G == 1 || (fits(nullptr, a.dpg) && fits(nullptr, a.N)));
    return vec ? launch_vec<T, SPT, LANES, TT, true>(a, st) : launch_vec<T, SPT, LANES, TT, false>(a, st);
}

template <typename T>
cudaError_t launch_n(const ScanArgs &a, cudaStream_t st) {
    if (a.N <= 8) return launch_scan<T, 4, 2, 16>(a, st);
    if (a.N <= 16) return launch_scan<T, 8, 2, 16>(a, st);
    if (a.N <= 32) return launch_scan<T, 16, 2, 16>(a, st);
    if (a.N <= 64) return launch_scan<T, 16, 4, 16>(a, st);
    return launch_scan<T, 32, 4, 16>(a, st);
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
