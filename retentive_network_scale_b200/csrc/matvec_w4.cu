// matvec_w4.cu -- ret_matvec_w4: products of a few rows with 4-bit weights,
//     y[m][n] = sum_g s[n][g] sum_{k in g} (q[n][k] - z[n][g]) x[m][k],
// and ret_quantize_w4, which lays such weights out.
//
// The products run on the tensor cores' warp-level instruction (m16n8k16, bf16 in,
// fp32 out): 16 weight rows by 8 columns of x.  Nothing is rounded on the way in:
// q - z is a small integer, exact in bf16, x is bf16 already, or 8-bit codes (exact
// in bf16, their scale applied to the sum), or fp32 split into three bf16 parts
// that add up to it (three columns of the instruction, which has columns to spare).
// The sum of a group of weights is scaled in fp32.
//
// A 32-bit word holds 8 codes of one weight row; masking it at shifts of 0, 4,
// 8 and 12 bits leaves the pairs (k, k+4), (k+1, k+5), ..., each of which one
// OR turns into two bf16 values 128 + q.  The instruction sums over k in any
// order as long as both operands use the same one, so x is kept in shared memory
// in that order and the codes are never moved between lanes.
//
// What bounds it: the floor is HBM, N K / 2 bytes (18.8 us for 8192 x 28672), but
// turning codes into bf16 takes 11 instructions a word, most of them on the integer
// pipe, and the loop about as many again: 38 us for one row there (50% of HBM), 58 us
// for 16 rows of 8-bit codes.  One row times 2048 x 12288: 6.1 us, of which a launch is
// 2.4.  Beyond 16 columns of x the accumulators leave 8 warps a CTA, and the tiles'
// reads of x and the warp-level products add up: 4096 x 14336 (floor 5) takes 44 us for
// 32 bf16 rows, 76 for 64 (75 of int8, 209 of fp32, whose 192 columns are four blocks
// that unpack every weight anew); with groups of 32 91, with zero points 100 (40 bytes
// a thread are spilled there).  The mask and the OR as one three-input operation, which the
// compiler does not make of them, took the first from 42.7 to 37.5.  Measured and
// not kept: three CTAs an SM at 80 registers (49.6: spills), shifts as
// multiplications (46.9), 16 words ahead (the same, but 6.4 us for the small one).
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "retention.h"

namespace ret {
namespace {


// Threads of a CTA: sixteen warps where the accumulators leave them registers.
__host__ __device__ constexpr int max_threads(int NT) { return NT <= 2 ? 512 : 256; }
constexpr size_t kStage = 64 * 1024;  // bytes of x staged at a time
constexpr int kMaxShared = 2 * kStage;
constexpr int kSms = 148;

struct W4Args {
    int M, N, K, x_dtype, xg, cols;  // xg: columns of x per x scale; cols: columns of the products
    long long ldx;
    const void *x;
    const float *xs;
    const uint8_t *wq, *zeros;
    const __nv_bfloat16 *s;
    void *y;
    int y_bf16, vec;
    int kc;                 // columns of x staged at a time
    int wr, wk, tile_cols;  // row tiles of a CTA, warps to a tile, product columns of a CTA
    int xgrouped;           // x scales by group of columns, not by row
};

// c = a b + (FIRST ? 0 : c)
template <bool FIRST>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    const float c0 = FIRST ? 0.f : c[0], c1 = FIRST ? 0.f : c[1], c2 = FIRST ? 0.f : c[2], c3 = FIRST ? 0.f : c[3];
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
// Codes (k+j, k+j+4) of the 8 codes in w, as bf16 minus `zero` (both lanes of
// it 128 + z): exact.
template <int J>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, __nv_bfloat162 zero) {
    uint32_t u;  // (w >> 4 J & 0x000f000f) | 0x43004300, the last two in one instruction
    asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(u) : "r"(w >> (4 * J)));
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

// bf16 pairs (j, j + 4) of 8 values.
__device__ __forceinline__ uint4 pack_x(const float (&v)[8]) {
    return make_uint4(pack_bf16(v[0], v[4]), pack_bf16(v[1], v[5]), pack_bf16(v[2], v[6]), pack_bf16(v[3], v[7]));
}
// 8 columns of an x row as loaded (16 bytes of bf16, 8 of codes, 32 of fp32).
struct RawX {
    uint4 q[2];
};
// a.vec: rows of x start on the size of 8 elements (16 bytes for fp32).
__device__ __forceinline__ void load_x(const W4Args &a, RawX &r, int m, int k) {
    if (a.x_dtype == RET_BF16) {
        const uint16_t *p = static_cast<const uint16_t *>(a.x) + (long long)m * a.ldx + k;
        r.q[0] = a.vec ? *reinterpret_cast<const uint4 *>(p)
                       : make_uint4(p[0] | (uint32_t)p[1] << 16, p[2] | (uint32_t)p[3] << 16, p[4] | (uint32_t)p[5] << 16,
                                    p[6] | (uint32_t)p[7] << 16);
    } else if (a.x_dtype == RET_F32) {
        const uint32_t *p = static_cast<const uint32_t *>(a.x) + (long long)m * a.ldx + k;
        r.q[0] = a.vec ? *reinterpret_cast<const uint4 *>(p) : make_uint4(p[0], p[1], p[2], p[3]);
        r.q[1] = a.vec ? *reinterpret_cast<const uint4 *>(p + 4) : make_uint4(p[4], p[5], p[6], p[7]);
    } else {
        const uint8_t *p = static_cast<const uint8_t *>(a.x) + (long long)m * a.ldx + k;
        const uint2 u = a.vec ? *reinterpret_cast<const uint2 *>(p)
                              : make_uint2(p[0] | (uint32_t)p[1] << 8 | (uint32_t)p[2] << 16 | (uint32_t)p[3] << 24,
                                           p[4] | (uint32_t)p[5] << 8 | (uint32_t)p[6] << 16 | (uint32_t)p[7] << 24);
        r.q[0].x = u.x;
        r.q[0].y = u.y;
    }
}
// Them as bf16 pairs (j, j + 4): for fp32 rows the three parts that the 24 bits of a
// value are cut into, 8 bits each, dst[0], dst[4] and dst[8].  Cut, not rounded: a
// first part rounded up could be infinite.  (What is below 2^-133, the least bf16,
// is lost.)
__device__ __forceinline__ void stage_x(const W4Args &a, const RawX &r, uint4 *dst) {
    const uint4 u = r.q[0], t = r.q[1];
    if (a.x_dtype == RET_BF16) {
        *dst = make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632), __byte_perm(u.y, u.w, 0x5410),
                          __byte_perm(u.y, u.w, 0x7632));
    } else if (a.x_dtype == RET_F32) {
        const uint32_t bits[8] = {u.x, u.y, u.z, u.w, t.x, t.y, t.z, t.w};
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(bits[i]);
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
            dst[4 * j] = make_uint4(__byte_perm(w[0], w[4], 0x7632), __byte_perm(w[1], w[5], 0x7632),
                                    __byte_perm(w[2], w[6], 0x7632), __byte_perm(w[3], w[7], 0x7632));
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // what this part leaves: of an infinity nothing, of a NaN NaN
                const float top = __uint_as_float(w[i] & 0xffff0000u);
                v[i] = v[i] == top ? 0.f : v[i] - top;
            }
        }
    } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t w = i < 4 ? u.x : u.y;
            if (a.x_dtype == RET_I8)  // 2^23 + 128 + code, minus 2^23 + 128
                v[i] = __uint_as_float(__byte_perm(w ^ 0x80808080u, 0x4b000000u, 0x7650 + i % 4)) - 8388736.f;
            else
                v[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw((uint8_t)(w >> (8 * (i % 4))), __NV_E4M3)));
        }
        *dst = pack_x(v);
    }
}

// One CTA: `wr` tiles of 16 weight rows, `wk` warps to a tile that share its groups,
// their sums meeting in shared memory.  x is staged kc columns at a time; of a
// chunk's groups each of the wk warps takes a stretch.  WPL: 32-bit words of codes
// per load, a group of weights being 32 WPL columns: the four lanes of a row read
// one group in one load each.  NT: 8-column tiles of x.  PF: groups requested ahead,
// across chunks.  ZP: with zero points.  XG: x scales by group of columns.
template <int WPL, int NT, int PF, bool ZP, bool XG>
__global__ void __launch_bounds__(max_threads(NT))
matvec_w4_kernel(const W4Args a) {
    constexpr int GK = 32 * WPL;
    extern __shared__ __align__(16) uint8_t dsm[];
    uint4 *xs = reinterpret_cast<uint4 *>(dsm);  // [kc / 32][columns][4]
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, q = lane / 4, c = lane % 4;
    const int wr = a.wr, wk = a.wk, mr = warp % wr, mk = warp / wr;
    const int n0 = (blockIdx.x * wr + mr) * 16;
    const int per = a.x_dtype == RET_F32 ? 3 : 1;  // product columns of an x row
    const int col0 = blockIdx.y * a.tile_cols, ncol = min(a.tile_cols, a.cols - col0), nrow = ncol / per;
    const int groups = a.K / GK;
    // groups of a chunk, and of it of this warp
    const int gc = a.kc / GK, stretch = (gc + wk - 1) / wk, lo = min(mk * stretch, gc), hi = min(lo + stretch, gc);

    struct Weights {
        uint32_t w[2][WPL];
        uint16_t s[2];
        uint8_t z[2];
    };
    // rows q and q + 8 of the tile (rows past the last repeat it)
    const int r0 = min(n0 + q, a.N - 1), r1 = min(n0 + q + 8, a.N - 1);
    const uint8_t *w0 = a.wq + (long long)r0 * (a.K / 2) + c * 4 * WPL, *w1 = a.wq + (long long)r1 * (a.K / 2) + c * 4 * WPL;
    const unsigned short *s0 = reinterpret_cast<const unsigned short *>(a.s) + (long long)r0 * groups;
    const unsigned short *s1 = reinterpret_cast<const unsigned short *>(a.s) + (long long)r1 * groups;
    const uint8_t *z0 = a.zeros + (ZP ? (long long)r0 * groups : 0), *z1 = a.zeros + (ZP ? (long long)r1 * groups : 0);
    int ahead = lo, ahead_hi = min(hi, groups);  // next group to request; end of the stretch it is of
    auto fetch = [&](Weights &o) {
        if (ahead >= ahead_hi) {  // on to this warp's stretch of the next chunk
            ahead += gc - (hi - lo);
            ahead_hi = min(ahead_hi + gc, groups);
            if (lo >= hi) return;
        }
        if (ahead < ahead_hi) {
            load_words<WPL>(o.w[0], w0 + (unsigned)ahead * (GK / 2));
            load_words<WPL>(o.w[1], w1 + (unsigned)ahead * (GK / 2));
            o.s[0] = __ldg(s0 + ahead);
            o.s[1] = __ldg(s1 + ahead);
            if (ZP) {
                o.z[0] = __ldg(z0 + ahead);
                o.z[1] = __ldg(z1 + ahead);
            }
        }
        ++ahead;
    };
    Weights ring[PF];
#pragma unroll
    for (int i = 0; i < PF; ++i) fetch(ring[i]);

    float acc[NT][4];
    int xat[NT];  // this lane's place in a step's columns (columns past the last repeat it)
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        xat[i] = min(8 * i + q, ncol - 1) * 4 + c;
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    }

    // staging: this thread's first piece of a chunk, and the way to its next ones
    const int row_first = tid / 4 % nrow, step_first = tid / 4 / nrow;
    const int row_next = (int)blockDim.x / 4 % nrow, step_next = (int)blockDim.x / 4 / nrow;
    for (int left = a.K; left > 0; left -= a.kc) {  // (k0 + a.kc may lie past 2^31)
        const int k0 = a.K - left, kn = min(a.kc, left);
        if (k0) __syncthreads();
        // x of the chunk: piece (step of 32 columns, product column, c) holds
        // the 8 columns that lane c multiplies in that step
        constexpr int UX = 2;  // pieces a thread has in flight
        int row = row_first, st = step_first;
        while (st < kn / 32) {
            RawX raw[UX];
            int at[UX];
#pragma unroll
            for (int u = 0; u < UX; ++u) {
                at[u] = st < kn / 32 ? (st * ncol + row * per) * 4 + tid % 4 : -1;
                if (at[u] >= 0) load_x(a, raw[u], col0 / per + row, k0 + st / WPL * GK + tid % 4 * 8 * WPL + 8 * (st % WPL));
                row += row_next;
                st += step_next;
                if (row >= nrow) {
                    row -= nrow;
                    ++st;
                }
            }
#pragma unroll
            for (int u = 0; u < UX; ++u)
                if (at[u] >= 0) stage_x(a, raw[u], xs + at[u]);
        }
        __syncthreads();
        const int g1 = min(hi, kn / GK);
        const uint4 *xp = xs + lo * (WPL * 4) * ncol;
        auto group = [&](Weights &o, int g) {
            float sum[NT][4];
            float more[4];  // one column tile: a second chain of products
            const uint32_t za = ZP ? 0x43004300u + (o.z[0] & 15u) * 0x10001u : 0x43084308u;
            const uint32_t zb = ZP ? 0x43004300u + (o.z[1] & 15u) * 0x10001u : 0x43084308u;
            const __nv_bfloat162 zero0 = *reinterpret_cast<const __nv_bfloat162 *>(&za);
            const __nv_bfloat162 zero1 = *reinterpret_cast<const __nv_bfloat162 *>(&zb);
#pragma unroll
            for (int j = 0; j < WPL; ++j) {
                uint4 b[NT];
#pragma unroll
                for (int i = 0; i < NT; ++i) b[i] = xp[xat[i]];
                xp += 4 * ncol;
                const uint32_t wa = o.w[0][j], wb = o.w[1][j];
                const uint32_t fa[4] = {code_pair<0>(wa, zero0), code_pair<0>(wb, zero1), code_pair<1>(wa, zero0),
                                        code_pair<1>(wb, zero1)};
                const uint32_t fb[4] = {code_pair<2>(wa, zero0), code_pair<2>(wb, zero1), code_pair<3>(wa, zero0),
                                        code_pair<3>(wb, zero1)};
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    if (j == 0) mma16816<true>(sum[i], fa, b[i].x, b[i].y);
                    else mma16816<false>(sum[i], fa, b[i].x, b[i].y);
                    if (NT > 1) mma16816<false>(sum[i], fb, b[i].z, b[i].w);
                    else if (j == 0) mma16816<true>(more, fb, b[i].z, b[i].w);
                    else mma16816<false>(more, fb, b[i].z, b[i].w);
                }
            }
            if (NT == 1)
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[0][j] += more[j];
            const float sa = __uint_as_float((uint32_t)o.s[0] << 16), sb = __uint_as_float((uint32_t)o.s[1] << 16);
            if (XG) {
                const int xgs = a.K / a.xg, xi = (k0 + g * GK) / a.xg;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int m0 = min(col0 + 8 * i + 2 * c, a.cols - 1), m1 = min(col0 + 8 * i + 2 * c + 1, a.cols - 1);
                    const float x0 = a.xs[(long long)m0 * xgs + xi], x1 = a.xs[(long long)m1 * xgs + xi];
                    sum[i][0] *= x0;
                    sum[i][1] *= x1;
                    sum[i][2] *= x0;
                    sum[i][3] *= x1;
                }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                acc[i][0] = fmaf(sa, sum[i][0], acc[i][0]);
                acc[i][1] = fmaf(sa, sum[i][1], acc[i][1]);
                acc[i][2] = fmaf(sb, sum[i][2], acc[i][2]);
                acc[i][3] = fmaf(sb, sum[i][3], acc[i][3]);
            }
            fetch(o);
        };
        int g = lo;
#pragma unroll 1
        for (; g + PF <= g1; g += PF)
#pragma unroll
            for (int p = 0; p < PF; ++p) group(ring[p], g + p);
        // the rest of a stretch (the last one's: whole chunks hold whole rings)
#pragma unroll
        for (int p = 0; p < PF - 1; ++p)
            if (g + p < g1) group(ring[p], g + p);
    }
    // join the warps' sums: red[mk][rows of the CTA][NT*8 columns + 1]
    __syncthreads();
    float *red = reinterpret_cast<float *>(dsm);
    constexpr int RS = NT * 8 + 1;
    const int rows = wr * 16;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        float *p = red + (mk * rows + mr * 16 + q) * RS + 8 * i + 2 * c;
        p[0] = acc[i][0];
        p[1] = acc[i][1];
        p[8 * RS] = acc[i][2];
        p[8 * RS + 1] = acc[i][3];
    }
    __syncthreads();
    for (int i = tid; i < rows * nrow; i += blockDim.x) {
        const int r = i % rows, m = i / rows, n = blockIdx.x * rows + r;
        if (n >= a.N) continue;
        float y = 0.f;
        for (int p = per - 1; p >= 0; --p)
            for (int w = 0; w < wk; ++w) y += red[(w * rows + r) * RS + m * per + p];
        const int mm = col0 / per + m;
        if (a.xs && !a.xgrouped) y *= a.xs[mm];
        const long long at = (long long)mm * a.N + n;
        if (a.y_bf16)
            static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(y);
        else
            static_cast<float *>(a.y)[at] = y;
    }
}

template <int WPL, int NT>
cudaError_t launch_w4(W4Args a, cudaStream_t st) {
    constexpr int PF = 8 / WPL;  // 8 words a row ahead
    const int per = a.x_dtype == RET_F32 ? 3 : 1;
    a.tile_cols = std::min(a.cols, NT * 8 / per * per);  // whole rows of x
    const int groups = a.K / (32 * WPL);
    const long long tiles = ((long long)a.N + 15) / 16, by = (a.cols + a.tile_cols - 1) / a.tile_cols;
    const size_t x_bytes = (size_t)a.K * 2 * a.tile_cols;
    auto unit = [&](int wk) { return 32 * WPL * PF * wk; };  // columns: one ring of each warp
    // The CTA that leaves the fullest SM least to do, counted in instructions (a
    // group's, x's staging and a CTA's own; read off the code, not fitted), each tile
    // of rows shared by as many warps as fit, down to two groups each.  us by tiles of
    // a CTA, * chosen: one bf16 row times 2048 x 12288 9.4 (1), 10.0 (2), 6.6* (6), 9.7
    // (12); times 8192 x 28672 63 (1), 50 (2), 41 (7), 38* (14); 16 int8 rows 180 (1),
    // 120 (2), 71 (7), 58* (13); 64 bf16 rows times 4096 x 14336 378 (1), 144 (2), 76*
    // (7), 70 (8); 64 fp32 rows times 4096 x 4096 201 (1), 95 (2), 60* (7), 61 (8); 48
    // bf16 rows times 2048 x 2048 in groups of 32 26* (1), 22 (2), 48 (8).  Over 16
    // shapes of 1 to 64 rows it is within 10% of the best but for small weights and
    // many rows (16 and 18%).
    const int most = max_threads(NT) / 32;
    double best = 1e300;
    for (int wr = most; wr >= 1; --wr) {
        int wk = std::max(1, std::min(most / wr, groups / 2));
        while (wk > 1 && x_bytes > kStage && (size_t)unit(wk) * 2 * a.tile_cols > 2 * kStage) --wk;
        const double ctas = (double)(((tiles + wr - 1) / wr * by + kSms - 1) / kSms);
        // (a CTA of fewer warps than fit takes as long as a nearly full one)
        const double warps = std::max(wr * wk, most * 7 / 8) + 0.01 * wr * wk;
        const double group = warps * (double)((groups + wk - 1) / wk) * (WPL * (30 + 4 * NT) + 60 + 8 * NT);
        const double cost = ctas * (group + (double)a.K * a.tile_cols / 256 * 20 + 3000);
        if (cost < best) {
            best = cost;
            a.wr = wr;
            a.wk = wk;
        }
    }
    // a chunk holds whole rings of every warp, or all of x
    a.kc = x_bytes <= kStage ? a.K : std::max(1, (int)(kStage / (2 * a.tile_cols) / unit(a.wk))) * unit(a.wk);
    if (a.kc > a.K) a.kc = a.K;
    const size_t smem = std::max((size_t)a.kc * 2 * a.tile_cols, sizeof(float) * a.wk * a.wr * 16 * (NT * 8 + 1));
    const long long bx = (tiles + a.wr - 1) / a.wr;
    auto kern = a.zeros ? a.xgrouped ? matvec_w4_kernel<WPL, NT, PF, true, true> : matvec_w4_kernel<WPL, NT, PF, true, false>
                        : a.xgrouped ? matvec_w4_kernel<WPL, NT, PF, false, true> : matvec_w4_kernel<WPL, NT, PF, false, false>;
    // (the same limit in every call: calls of other sizes may run at once)
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared);
    if (e != cudaSuccess) return e;
    if (smem > (size_t)kMaxShared) return cudaErrorInvalidConfiguration;
    kern<<<dim3((unsigned)bx, (unsigned)by), 32 * a.wr * a.wk, smem, st>>>(a);
    e = cudaGetLastError();
    if (e == cudaSuccess) note_launches(1);
    return e;
}

template <int WPL>
cudaError_t launch_cols(const W4Args &a, cudaStream_t st) {
    if (a.cols <= 8) return launch_w4<WPL, 1>(a, st);
    if (a.cols <= 16) return launch_w4<WPL, 2>(a, st);
    if (a.cols <= 32) return launch_w4<WPL, 4>(a, st);
    return launch_w4<WPL, 8>(a, st);
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
    // with zero points [lo, hi] (0 included) to 0..15, else +-max to 8 +- 7 (halves:
    // hi - lo may pass the largest float)
    const __nv_bfloat16 sb = __float2bfloat16_rn(zeros ? (0.5f * hi - 0.5f * lo) / 7.5f : fmaxf(hi, -lo) / 7.f);
    const float s = __bfloat162float(sb);
    // steps of the scale, to the nearest, exactly: w / s next to k + 1/2 cannot round
    // onto it (s (k + 1/2) has 13 bits, so is itself an fp32 number, and the ones beside
    // it are farther off than a quotient's rounding); 1 / s to multiply by, 8% quicker
    // in 8192 x 28672 bf16 weights in groups of 128 (1.00 ms, and 1.09), decides ties
    // either way and is infinite for subnormal scales
    auto steps = [s](float w) { return s > 0.f ? rintf(w / s) : 0.f; };
    const float z = zeros ? fminf(fmaxf(steps(-lo), 0.f), 15.f) : 8.f;
    scales[(long long)n * groups + g] = sb;
    if (zeros) zeros[(long long)n * groups + g] = (uint8_t)z;
    uint8_t *p = wq + (long long)n * (K / 2) + (long long)g * (group / 2);
    for (int k = 0; k < group; k += 2) {
        const float a = fminf(fmaxf(steps(ld(w, (size_t)k * ldw)) + z, 0.f), 15.f);
        const float b = fminf(fmaxf(steps(ld(w, (size_t)(k + 1) * ldw)) + z, 0.f), 15.f);
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
    if (M < 0 || M > RET_MAX_MATVEC_ROWS || N < 0 || N > RET_MAX_MATVEC_COLUMNS || K < 1 || ldx < K ||
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
    a.xgrouped = codes && a.xg < K;
    a.wq = static_cast<const uint8_t *>(Wq);
    a.zeros = static_cast<const uint8_t *>(zeros);
    a.s = static_cast<const __nv_bfloat16 *>(scales);
    a.y = Y;
    a.y_bf16 = y_dtype == RET_BF16;
    const unsigned piece = codes ? 8 : 16;
    a.vec = aligned(X, piece) && (ldx * xsize) % piece == 0;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = group == 128 ? launch_cols<4>(a, st) : group == 64 ? launch_cols<2>(a, st) : launch_cols<1>(a, st);
    return e == cudaSuccess ? RET_OK : RET_ERR_CUDA;
}

extern "C" ret_status ret_quantize_w4(int K, int N, int group, int w_dtype, const void *W, long long ldw,
                                      void *Wq, void *scales, void *zeros, void *stream) {
    using namespace ret;
    if (K < 1 || N < 0 || N > RET_MAX_MATVEC_COLUMNS || ldw < N || (group != 32 && group != 64 && group != 128) || K % group)
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
