// selective_scan.cu -- ret_selective_scan: the diagonal recurrence whose decay
// depends on the token,
//     h_t = exp(d_t A) h_{t-1} + d_t u_t B_t,  y_t = (C_t . h_t + skip u_t) swish(z_t),
// per channel with N states, for prompts and for single tokens over an fp32
// state.
#include <algorithm>
#include <cmath>
#include <type_traits>

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

__device__ __forceinline__ uint64_t dup(float v) { return tc::f2_make(v, v); }

// log(1 + e^x) = max(x, 0) + log1p(e^-|x|), of both values of a pair.
// log1p(e) / e for e = e^-|x| in (0, 1] is a polynomial of degree 8 fitted by
// reweighted least squares at Chebyshev nodes (relative error 3e-8), which keeps
// the relative accuracy for small e, where log(1 + e) would not, and leaves the
// special-function unit to the decays.
__device__ __forceinline__ uint64_t softplus2(uint64_t x) {
    const float x0 = tc::f2_lo(x), x1 = tc::f2_hi(x);
    const uint64_t a = tc::f2_mul(tc::f2_make(fabsf(x0), fabsf(x1)), dup(-kLog2e));
    const uint64_t e = tc::f2_make(exp2_fast(tc::f2_lo(a)), exp2_fast(tc::f2_hi(a)));
    uint64_t p = dup(0.005232624709606171f);
    p = tc::f2_fma(p, e, dup(-0.029504960402846336f));
    p = tc::f2_fma(p, e, dup(0.0782255008816719f));
    p = tc::f2_fma(p, e, dup(-0.1366320699453354f));
    p = tc::f2_fma(p, e, dup(0.1910598874092102f));
    p = tc::f2_fma(p, e, dup(-0.2484297752380371f));
    p = tc::f2_fma(p, e, dup(0.3331909477710724f));
    p = tc::f2_fma(p, e, dup(-0.4999949336051941f));
    p = tc::f2_fma(p, e, dup(0.9999999403953552f));
    return tc::f2_fma(p, e, tc::f2_make(fmaxf(x0, 0.f), fmaxf(x1, 0.f)));
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

// Sizes.  LANES threads share a channel and hold SPT states each, so a warp owns
// CPW channels and a CTA CH; rows go in tiles of TT.
template <typename T, int SPT, int LANES, bool VEC>
struct ScanTile {
    static constexpr int WARPS = 4, NT = 32 * WARPS, TT = 16;
    static constexpr int CPW = 32 / LANES, CH = WARPS * CPW, NP = SPT * LANES;
    static constexpr int E = CPW * TT / 32;              // elements per thread, operand and tile
    static constexpr int SLOTS = NT / TT;                // threads that copy a row
    static constexpr int WORDS = CH * (int)sizeof(T) / 16 + (VEC ? 0 : 1);  // 16-byte words of a row
    static constexpr int RS = 16 * (WORDS | 1);          // its bytes: an odd number of words, no bank conflicts
    static constexpr int PE = 8;                         // elements of a piece of B or C
    static constexpr int PR = NP / PE;                   // pieces per row
    static constexpr int PIECES = 2 * TT * PR;           // of both
    static constexpr int NB = (PIECES + NT - 1) / NT;    // per thread
    static constexpr int PB = PE * (int)sizeof(T) + (VEC ? 0 : 16);  // bytes a copied piece takes
    static_assert(NP % PE == 0 && E >= 2, "tile");
    struct Smem {
        uint8_t in[2][3][TT][RS];                // u, delta, z as copied, two tiles
        float2 du[CH][TT + 2];                   // (d, d u)
        float y[CH][LANES][TT + 4];              // its threads' parts of y
        float bc[2][2][TT][NP];                  // two tiles of B and C
        uint8_t bcin[2][NB][NT][PB];             // as copied, by the thread that converts it
    };
    // What a segment does to the state: h -> a h + b.
    struct Segment {
        float a[CH][NP], b[CH][NP];
    };
};

// The recurrence: LANES threads share a channel and hold SPT states each (state
// n = 4 LANES (i / 4) + 4 lane + i % 4 in register i, so that B_t and C_t are read
// from shared memory in 16-byte pieces), two states to a packed register pair.
// Rows go in tiles of TT.  While a tile is computed the next one is copied to
// shared memory as it is; then the CTA turns its B and C into fp32 (the tile's only
// barrier) and each warp its channels' delta into d = softplus(delta + bias) and
// d u, once per row and channel; y is gated and rounded by the warp that computed
// it.
//
// What bounds it: N exponentials per row and channel on the special-function
// units (16 a clock and SM), 478 us for 8 x 4096 rows of 4096 channels with 16
// states, next to some 60 instructions a row for a warp's 16 channels and the reads
// of B and C, which return 128 bytes a clock however many lanes read the same.
// Measured 867 us there, 165 us being the floor of its bytes.  Measured and not
// kept: 4 threads a channel (942 us; 1085 with one register pair of du in place of
// two copies), 2 channels a thread (945), a polynomial for a quarter of the
// exponentials (991), unpacked arithmetic (992): what costs is instructions and
// shared memory as much as the exponentials, and 2048 warps are 3.5 a scheduler,
// of which the fullest have 4.  More states, 8 x 2048 rows of 2048 channels, us (their
// exponentials alone): 24 453 (179; computed as 32), 32 450 (239), 64 770 (477), 128
// 1413 (954).
//
// SPLIT (few channels): a cluster of CTAs shares the channels, each CTA one segment
// of the rows.  1 x 16384 rows of 1024 channels: 1462 us in one piece, 443 in 8
// segments, 314 in 16.
//
// VEC: every row of every operand starts on 16 bytes.  Otherwise the aligned
// words that hold a row are copied and the row starts a few elements into its
// place (bytes before an unaligned row are in its first word, so in the same
// allocation; bytes past its end are not read).
template <typename T, int SPT, int LANES, bool VEC, bool SPLIT>
__global__ void __launch_bounds__(128, SPT <= 8 ? 4 : 3)
selective_scan_kernel(const ScanArgs a) {
    using C = ScanTile<T, SPT, LANES, VEC>;
    constexpr int NT = C::NT, TT = C::TT, CPW = C::CPW, NP = C::NP, E = C::E, NB = C::NB, PE = C::PE;
    constexpr int PR = SPT / 2;  // state pairs
    constexpr int SZ = (int)sizeof(T);
    extern __shared__ __align__(16) uint8_t dsm[];
    auto &sm = *reinterpret_cast<typename C::Smem *>(dsm);
    auto &seg = *reinterpret_cast<typename C::Segment *>(dsm + sizeof(typename C::Smem));

    const int tid = threadIdx.x, wl = tid % 32, lane = tid % LANES, ch = tid / LANES;
    const int segments = SPLIT ? (int)gridDim.y : 1, me = SPLIT ? (int)blockIdx.y : 0;
    int blk = blockIdx.x;
    const int cb = blk % a.blocks_per_group;
    blk /= a.blocks_per_group;
    const int g = blk % a.G, b = blk / a.G;
    const int c0 = g * a.dpg + cb * C::CH;             // first channel
    const int nch = min(C::CH, a.dpg - cb * C::CH);    // channels of the CTA
    const int len = a.lengths ? min(max(a.lengths[b], 0), a.L) : a.L;
    const long long row0 = (long long)b * a.L;

    // the CTA's part of an operand's row t
    auto row_of = [&](const void *p, long long ld, int t) { return static_cast<const T *>(p) + (row0 + t) * ld + c0; };
    auto misfit = [](const T *p) { return VEC ? 0 : (int)(reinterpret_cast<uintptr_t>(p) & 15u); };
    const uint8_t *somewhere = static_cast<const uint8_t *>(a.u) - misfit(static_cast<const T *>(a.u));
    auto copy_row = [&](const T *p, bool there, uint8_t *dst, int slot) {
        const int head = misfit(p), end = there ? head + nch * SZ : 0;
        const uint8_t *base = reinterpret_cast<const uint8_t *>(p) - head;
        const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
#pragma unroll
        for (int w = 0; w < C::WORDS; w += C::SLOTS) {
            if (C::WORDS % C::SLOTS == 0 || w + slot < C::WORDS) {
                const int at = 16 * (w + slot), n = min(16, max(0, end - at));
                cp_async16(d + at, n ? base + at : somewhere, n);
            }
        }
    };
    // pieces of B and C: this thread's j-th (the last threads take the first
    // pieces, since the first ones copy more of the rows)
    auto piece = [&](int j, int &r, int &n0, bool &c) {
        const int p = NT - 1 - tid + j * NT;
        r = p / C::PR % TT;
        n0 = p % C::PR * PE;
        c = p >= TT * C::PR;
        return C::PIECES % NT == 0 || p < C::PIECES;
    };
    auto piece_at = [&](int t, int n0, bool c) {
        return static_cast<const T *>(c ? a.cm : a.bm) + (row0 + t) * (c ? a.ldc : a.ldb) + (long long)g * a.N + n0;
    };
    // copies the tile that starts at row t0 into slot k (y: z and C too)
    const int cr = tid / C::SLOTS, slot = tid % C::SLOTS;
    auto copy_tile = [&](int t0, int k, bool y) {
        const int t = t0 + cr;
        if (VEC && nch == C::CH && t0 + TT <= len) {  // nothing to cut
            auto go = [&](const void *p, long long ld, int op) {
                const uint8_t *src = reinterpret_cast<const uint8_t *>(row_of(p, ld, t)) + 16 * slot;
                const uint32_t d = (uint32_t)__cvta_generic_to_shared(sm.in[k][op][cr]) + 16 * slot;
#pragma unroll
                for (int w = 0; w < C::WORDS; w += C::SLOTS)
                    if (C::WORDS % C::SLOTS == 0 || w + slot < C::WORDS) cp_async16(d + 16 * w, src + 16 * w, 16);
            };
            go(a.u, a.ldu, 0);
            go(a.delta, a.ldd, 1);
            if (y && a.z) go(a.z, a.ldz, 2);
        } else {
            const bool there = t < len;
            copy_row(row_of(a.u, a.ldu, t), there, sm.in[k][0][cr], slot);
            copy_row(row_of(a.delta, a.ldd, t), there, sm.in[k][1][cr], slot);
            if (y && a.z) copy_row(row_of(a.z, a.ldz, t), there, sm.in[k][2][cr], slot);
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            int r, n0;
            bool c;
            if (piece(j, r, n0, c) && (y || !c)) {
                const T *p = piece_at(t0 + r, n0, c);
                const int n = t0 + r < len ? min(PE, max(0, a.N - n0)) : 0;
                const int head = misfit(p), end = n ? head + n * SZ : 0;
                const uint8_t *base = reinterpret_cast<const uint8_t *>(p) - head;
                const uint32_t d = (uint32_t)__cvta_generic_to_shared(sm.bcin[k][j][tid]);
#pragma unroll
                for (int w = 0; w < C::PB; w += 16) {
                    const int m = min(16, max(0, end - w));
                    cp_async16(d + w, m ? base + w : somewhere, m);
                }
            }
        }
        cp_async_commit();
    };
    // B and C of the tile at t0, from slot k to the fp32 tile k
    auto convert_bc = [&](int t0, int k, bool y) {
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            int r, n0;
            bool c;
            if (piece(j, r, n0, c) && (y || !c)) {
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

    // this CTA's rows: all, or a whole number of tiles of the sequence
    const int per = SPLIT ? ((len + TT - 1) / TT + segments - 1) / segments * TT : len;
    const int first = me * per, end = min(len, first + per);
    if (first < end) copy_tile(first, 0, !SPLIT);

    auto state_of = [&](int i) { return i / 4 * (4 * LANES) + lane * 4 + i % 4; };
    const long long state_row = ((long long)b * a.D + c0 + ch) * a.N;
    auto entering = [&](int j) {  // states 2j and 2j + 1 before the first row
        const int n = state_of(2 * j);
        const bool in = a.s_in && ch < nch;
        return tc::f2_make(in && n < a.N ? a.s_in[state_row + n] : 0.f, in && n + 1 < a.N ? a.s_in[state_row + n + 1] : 0.f);
    };
    uint64_t h[PR], A2[PR];
#pragma unroll
    for (int j = 0; j < PR; ++j) {
        const int n = state_of(2 * j);
        const float *p = a.A + (long long)(c0 + ch) * a.N + n;
        A2[j] = tc::f2_make(ch < nch && n < a.N ? p[0] * kLog2e : 0.f, ch < nch && n + 1 < a.N ? p[1] * kLog2e : 0.f);
        h[j] = me == 0 ? entering(j) : 0;
    }
    auto sum_parts = [](const float (&y)[LANES][TT + 4], int r) {
        float v = y[0][r];
#pragma unroll
        for (int l = 1; l < LANES; ++l) v += y[l][r];
        return v;
    };
    // conversion and output: this thread's row of a tile and its E channels
    // (of the warp's own)
    const int sr = wl % TT, sc = tid / 32 * CPW + wl / TT * E;
    uint64_t bias[E / 2], skip[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        const int c = sc + 2 * i;
        auto of = [&](const float *p, int cc) { return p && cc < nch ? p[c0 + cc] : 0.f; };
        bias[i] = tc::f2_make(of(a.bias, c), of(a.bias, c + 1));
        skip[i] = tc::f2_make(of(a.skip, c), of(a.skip, c + 1));
    }
    auto copied = [&](int k, int op, const T *row) {
        return shared_raw<VEC, T, E>(reinterpret_cast<const T *>(sm.in[k][op][sr] + misfit(row)) + sc);
    };

    // The recurrence over this CTA's rows.  Y: writes y; else only follows the
    // state, and the sum of d (by tiles, so that long sums stay exact).
    float sum_d = 0.f;
    auto run = [&](auto want_y) {
        constexpr bool Y = decltype(want_y)::value;
        for (int t0 = first, k = 0; t0 < end; t0 += TT, k ^= 1) {
            cp_async_wait();
            convert_bc(t0, k, Y);
            __syncthreads();  // also: every warp is done with the tile before this one
            const int tr = t0 + sr;
            const bool inside = tr < len;
            const Raw<T, E> ru = copied(k, 0, row_of(a.u, a.ldu, tr));
            const Raw<T, E> rd = copied(k, 1, row_of(a.delta, a.ldd, tr));
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                uint64_t d = tc::f2_add(tc::f2_make(to_f(rd.v[2 * i]), to_f(rd.v[2 * i + 1])), bias[i]);
                if (a.softplus) d = softplus2(d);
                // rows past the sequence keep the state (their u reads as 0)
                const float d0 = inside ? tc::f2_lo(d) : 0.f, d1 = inside ? tc::f2_hi(d) : 0.f;
                sm.du[sc + 2 * i][sr] = make_float2(d0, d0 * to_f(ru.v[2 * i]));
                sm.du[sc + 2 * i + 1][sr] = make_float2(d1, d1 * to_f(ru.v[2 * i + 1]));
            }
            if (t0 + TT < end) copy_tile(t0 + TT, k ^ 1, Y);
            __syncwarp();

            // A row's operands are read two rows ahead and its exponentials taken
            // one row ahead of their use.
            struct Ops {
                float2 dx;  // (d, d u)
                uint64_t b[PR], c[PR];
            };
            const float *tb = &sm.bc[k][0][0][lane * 4], *tc_ = &sm.bc[k][1][0][lane * 4];
            auto read = [&](Ops &o, int t) {
                o.dx = sm.du[ch][t];
#pragma unroll
                for (int j = 0; j < PR; j += 2) {
                    const int at = t * NP + j * 2 * LANES;
                    *reinterpret_cast<ulonglong2 *>(&o.b[j]) = *reinterpret_cast<const ulonglong2 *>(tb + at);
                    if (Y) *reinterpret_cast<ulonglong2 *>(&o.c[j]) = *reinterpret_cast<const ulonglong2 *>(tc_ + at);
                }
            };
            auto decay = [&](uint64_t (&e)[PR], const Ops &o) {
#pragma unroll
                for (int j = 0; j < PR; ++j) {
                    const uint64_t p = tc::f2_mul(dup(o.dx.x), A2[j]);
                    e[j] = tc::f2_make(exp2_fast(tc::f2_lo(p)), exp2_fast(tc::f2_hi(p)));
                }
            };
            Ops ops[2];
            uint64_t e[2][PR];
            float part[4], tile_d = 0.f;
            read(ops[0], 0);
            read(ops[1], 1);
            decay(e[0], ops[0]);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const Ops o = ops[t % 2];
                if (t + 1 < TT) decay(e[(t + 1) % 2], ops[(t + 1) % 2]);
                if (t + 2 < TT) read(ops[t % 2], t + 2);
                const uint64_t xx = dup(o.dx.y);
                uint64_t acc = 0;
#pragma unroll
                for (int j = 0; j < PR; ++j) {
                    h[j] = tc::f2_fma(e[t % 2][j], h[j], tc::f2_mul(xx, o.b[j]));
                    if (Y) acc = j ? tc::f2_fma(o.c[j], h[j], acc) : tc::f2_mul(o.c[j], h[j]);
                }
                if (Y) {
                    part[t % 4] = tc::f2_lo(acc) + tc::f2_hi(acc);
                    if (t % 4 == 3)
                        *reinterpret_cast<float4 *>(&sm.y[ch][lane][t - 3]) = make_float4(part[0], part[1], part[2], part[3]);
                } else {
                    tile_d += o.dx.x;
                }
            }
            if (!Y) sum_d += tile_d;
            __syncwarp();
            if (Y && inside && sc < nch) {
                uint64_t y2[E / 2];
#pragma unroll
                for (int i = 0; i < E / 2; ++i)
                    y2[i] = tc::f2_fma(skip[i], tc::f2_make(to_f(ru.v[2 * i]), to_f(ru.v[2 * i + 1])),
                                       tc::f2_make(sum_parts(sm.y[sc + 2 * i], sr), sum_parts(sm.y[sc + 2 * i + 1], sr)));
                if (a.z) {
                    const Raw<T, E> rz = copied(k, 2, row_of(a.z, a.ldz, tr));
#pragma unroll
                    for (int i = 0; i < E / 2; ++i)
                        y2[i] = tc::f2_mul(y2[i], tc::f2_make(swish(to_f(rz.v[2 * i])), swish(to_f(rz.v[2 * i + 1]))));
                }
                Raw<T, E> out;
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    from_f(out.v[2 * i], tc::f2_lo(y2[i]));
                    from_f(out.v[2 * i + 1], tc::f2_hi(y2[i]));
                }
                store_raw<T, E>(static_cast<T *>(a.y) + (row0 + tr) * a.D + c0 + sc, out, nch - sc);
            }
        }
    };

    if (SPLIT) {
        // 1. what each segment but the last does to the state: its own rows from
        //    a zero state (the first one from the entering state), and the decay
        //    over all of them, exp(A sum d)
        if (me + 1 < segments) run(std::false_type{});
#pragma unroll
        for (int j = 0; j < PR; ++j) {
            const uint64_t p = tc::f2_mul(dup(sum_d), A2[j]);
            const int n = state_of(2 * j);
            // (a growth past fp32's range is passed on as its exponent, negated)
            auto factor = [](float e) { return e <= 127.f ? exp2_fast(e) : -e; };
            *reinterpret_cast<float2 *>(&seg.a[ch][n]) = make_float2(factor(tc::f2_lo(p)), factor(tc::f2_hi(p)));
            *reinterpret_cast<uint64_t *>(&seg.b[ch][n]) = h[j];
        }
        __syncthreads();
        if (first < end) copy_tile(first, 0, true);
        tc::cluster_sync();
        // 2. the state that enters this segment, through those before it
        auto join = [&](auto apply) {
#pragma unroll
            for (int j = 0; j < PR; ++j) {
                const uint32_t at_a = (uint32_t)__cvta_generic_to_shared(&seg.a[ch][state_of(2 * j)]);
                const uint32_t at_b = (uint32_t)__cvta_generic_to_shared(&seg.b[ch][state_of(2 * j)]);
                h[j] = me == 0 ? entering(j) : 0;
                for (int i = 0; i < me; ++i) {
                    const float2 ai = tc::ld_cluster_f32x2(tc::map_to_rank(at_a, i));
                    const float2 bi = tc::ld_cluster_f32x2(tc::map_to_rank(at_b, i));
                    const uint64_t b2 = tc::f2_make(bi.x, bi.y);
                    h[j] = i ? apply(ai, h[j], b2) : b2;
                }
            }
        };
        float least = 0.f;
        join([&](float2 a, uint64_t v, uint64_t b) {
            least = fminf(least, fminf(a.x, a.y));
            return tc::f2_fma(tc::f2_make(a.x, a.y), v, b);
        });
        if (least < 0.f)  // a growth 2^-a, in three factors: a small or zero state stays what it is
            join([&](float2 a, uint64_t v, uint64_t b) {
                auto grow = [](float &f, float x) {
                    if (!(f < 0.f)) return x;
                    x *= exp2_fast(fminf(-f - 127.f, 127.f));
                    x *= exp2_fast(fminf(fmaxf(-f - 254.f, 0.f), 127.f));
                    f = 0x1p127f;
                    return x;
                };
                const float lo = grow(a.x, tc::f2_lo(v)), hi = grow(a.y, tc::f2_hi(v));
                return tc::f2_fma(tc::f2_make(a.x, a.y), tc::f2_make(lo, hi), b);
            });
        tc::cluster_sync();  // nothing of this CTA's is read after this; state_out may be state_in
    }
    run(std::true_type{});
    if (SPLIT && me + 1 < segments) return;
    if (a.s_out && ch < nch) {
#pragma unroll
        for (int j = 0; j < PR; ++j) {
            const int n = state_of(2 * j);  // n + 1 is the pair's other state
            if (n < a.N) a.s_out[state_row + n] = tc::f2_lo(h[j]);
            if (n + 1 < a.N) a.s_out[state_row + n + 1] = tc::f2_hi(h[j]);
        }
    }
}

// A few rows per sequence (single tokens): bound by the state, which is read and
// written once.  A thread holds V times four states of a channel; `lanes` threads
// (a power of two, two where N allows, so that a read covers whole 32-byte
// sectors) share the channel, and u, d and the step's softplus are worked out once
// per thread.  Several sequences per thread (A read once for them) measured
// slower, since the registers cost resident warps.  ONE: L = 1, 10.2 us for one bf16
// token of 64 x 4096 x 16 states (floor 5.6), f32 8.9.
constexpr int kTokenThreads = 128;
// Longest L: the rows go one after the other here, while a tile above takes 16 rows in
// the time of one, but has a CTA's start and the reads of whole tiles before it.
// Measured, us here / tiles, for 5 and 8 rows, 16 states if not said:
//    1 x  512 channels, bf16   5.1 / 4.4    7.0 / 4.5
//    8 x 1024           bf16   5.4 / 4.5    7.2 / 4.5      fp32   4.9 / 4.5    6.6 / 4.6
//      64 states        bf16   7.0 / 6.8    9.4 / 6.8      fp32   5.8 / 7.2    7.8 / 7.2
//    8 x 4096           bf16   6.3 / 7.5    8.8 / 7.5      fp32   5.6 / 9.1    7.6 / 9.2
//   16 x 4096           bf16   8.9 / 11.8  12.8 / 11.8     fp32   8.2 / 13.4  11.1 / 13.6
//      128 states       bf16  53.2 / 76.0  79.8 / 75.9     fp32  44.6 / 100   68.4 / 101
//   64 x 4096           bf16  30 / 40      46.6 / 41.2     fp32  29 / 48      45.5 / 49.3
// 9 rows, bf16: 9.5 / 7.7 (8 x 4096), 14.1 / 11.8 (16 x 4096), 53.0 / 41.4 (64 x 4096).
inline int token_rows(long long threads) { return threads < 48 * 1024 ? 5 : 8; }

template <typename T, int V, bool VEC, bool ONE>
__global__ void __launch_bounds__(kTokenThreads)
selective_token_kernel(const ScanArgs a, int lanes) {
    const int idx = blockIdx.x * kTokenThreads + threadIdx.x;
    const int c = idx / lanes, lane = idx % lanes;
    const int b = blockIdx.y;
    const bool live = c < a.D;
    const int cc = live ? c : a.D - 1;  // the other threads of the warp take part in its shuffles
    const int g = cc / a.dpg;
    auto first = [&](int v) { return 4 * (lane + lanes * v); };  // state of piece v
    auto states = [&](int v) { return live ? min(4, a.N - first(v)) : 0; };
    float A2[V][4];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
        const float *p = a.A + (long long)cc * a.N + first(v);
        if (VEC) {
            if (states(v) > 0) r = *reinterpret_cast<const float4 *>(p);
        } else {
            if (states(v) > 0) r.x = p[0];
            if (states(v) > 1) r.y = p[1];
            if (states(v) > 2) r.z = p[2];
            if (states(v) > 3) r.w = p[3];
        }
        A2[v][0] = r.x * kLog2e; A2[v][1] = r.y * kLog2e; A2[v][2] = r.z * kLog2e; A2[v][3] = r.w * kLog2e;
    }
    const float bias = a.bias ? a.bias[cc] : 0.f, skip = a.skip ? a.skip[cc] : 0.f;
    float h[V][4];
    const int len = a.lengths ? min(max(a.lengths[b], 0), a.L) : a.L;
    const long long state_row = ((long long)b * a.D + cc) * a.N;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float *p = a.s_in + state_row + first(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[v][i] = 0.f;
        if (a.s_in && states(v) > 0) {
            if (VEC) {
                *reinterpret_cast<float4 *>(h[v]) = __ldcs(reinterpret_cast<const float4 *>(p));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < states(v)) h[v][i] = p[i];
            }
        }
    }
    for (int t = 0; t < (ONE ? 1 : a.L); ++t) {
        const bool in = t < len;
        const long long row = (long long)b * a.L + t;
        const float u = in ? to_f(static_cast<const T *>(a.u)[row * a.ldu + cc]) : 0.f;
        float d = in ? to_f(static_cast<const T *>(a.delta)[row * a.ldd + cc]) : 0.f;
        const float z = in && a.z ? to_f(static_cast<const T *>(a.z)[row * a.ldz + cc]) : 0.f;
        const T *pb = static_cast<const T *>(a.bm) + row * a.ldb + (long long)g * a.N;
        const T *pc = static_cast<const T *>(a.cm) + row * a.ldc + (long long)g * a.N;
        Raw<T, 4> rb[V], rc[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                from_f(rb[v].v[i], 0.f);
                from_f(rc[v].v[i], 0.f);
            }
            if (VEC) {
                if (in && states(v) > 0) {
                    rb[v] = *reinterpret_cast<const Raw<T, 4> *>(pb + first(v));
                    rc[v] = *reinterpret_cast<const Raw<T, 4> *>(pc + first(v));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (in && i < states(v)) {
                        rb[v].v[i] = pb[first(v) + i];
                        rc[v].v[i] = pc[first(v) + i];
                    }
            }
        }
        d += bias;
        if (a.softplus) d = tc::f2_lo(softplus2(dup(d)));
        if (!in) d = 0.f;
        const float x = d * u;
        float y = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[v][i] = fmaf(exp2_fast(d * A2[v][i]), h[v][i], x * to_f(rb[v].v[i]));
                y = fmaf(to_f(rc[v].v[i]), h[v][i], y);
            }
        for (int m = lanes / 2; m > 0; m >>= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
        if (lane == 0 && live && in) {
            y = fmaf(skip, u, y);
            if (a.z) y *= swish(z);
            from_f(static_cast<T *>(a.y)[row * a.D + c], y);
        }
    }
    if (!a.s_out) return;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float *p = a.s_out + state_row + first(v);
        if (states(v) <= 0) continue;
        if (VEC) {
            __stcs(reinterpret_cast<float4 *>(p), *reinterpret_cast<float4 *>(h[v]));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < states(v)) p[i] = h[v][i];
        }
    }
}

template <typename T, int V>
cudaError_t launch_token_t(const ScanArgs &a, int lanes, cudaStream_t st) {
    const long long bx = ((long long)a.D * lanes + kTokenThreads - 1) / kTokenThreads;
    // whole float4s of states, and 4-element pieces of B and C on their size
    auto fits = [](const void *p, long long ld) {
        return (reinterpret_cast<uintptr_t>(p) & (4 * sizeof(T) - 1)) == 0 && ld % 4 == 0;
    };
    const bool vec = a.N % 4 == 0 && fits(a.bm, a.ldb) && fits(a.cm, a.ldc), one = a.L == 1;
    auto kern = vec ? one ? selective_token_kernel<T, V, true, true> : selective_token_kernel<T, V, true, false>
                    : one ? selective_token_kernel<T, V, false, true> : selective_token_kernel<T, V, false, false>;
    kern<<<dim3((unsigned)bx, (unsigned)a.B), kTokenThreads, 0, st>>>(a, lanes);
    const cudaError_t err = cudaGetLastError();
    if (err == cudaSuccess) note_launches(1);
    return err;
}

// Threads that share a channel's states in the kernel of few rows.
inline int token_lanes(int N) { return N <= 4 ? 1 : N <= 16 ? 2 : N <= 64 ? 4 : 8; }

template <typename T>
cudaError_t launch_tokens(const ScanArgs &a, cudaStream_t st) {
    const int lanes = token_lanes(a.N);
    if (a.N <= 8) return launch_token_t<T, 1>(a, lanes, st);
    if (a.N <= 32) return launch_token_t<T, 2>(a, lanes, st);
    return launch_token_t<T, 4>(a, lanes, st);
}

// Segments that a sequence of L rows is cut into, 1, 4, 8 or 16, by the time that
// each would take, in us.  An SM with one CTA takes `row` for a row; with w CTAs an
// uncut sequence takes 0.38 + 0.53 w of that and a cut one, whose rows run about
// twice, 0.8 + w, where w is what the fullest SM has (at most per_sm at a time;
// clusters of 8 and 16 fill the SMs 10% less evenly).  Joining costs a few us, and
// most for many clusters of 16.
//
// Measured, us, uncut / 4 / 8 / 16 segments, 2048 rows (8192), bf16 if not said, by the
// CTAs of uncut sequences; * is chosen here.  Over 180 shapes (8 to 128 states, fp32 and
// bf16, 4 to 512 CTAs, 512 to 8192 rows) the choice is 0.7% off the best on average,
// 15% at worst; one made from the warps alone, whatever the layout, was 12% and 126% off.
//   16 states,  16 CTAs   173 /  83 /  62 /  56*      (685 /  317 /  227 /  162*)
//               32 CTAs   176 /  86 /  67*/  90       (689 /  318 /  236 /  259*)
//               64 CTAs   176 / 120 / 113*/ 147       (689 /  461 /  427*/  430)
//       fp32    64 CTAs   180 / 125*/ 137 / 181       (705 /  480 /  498 /  514*)
//              128 CTAs   176*/ 212 / 200 / 261       (689*/  826 /  756 /  790)
//    8 states, 128 CTAs   145*/ 130 / 131 / 162       (566*/  504 /  494 /  505)
//   64 states,  32 CTAs   170 /  77 /  62*/  83       (674 /  291 /  229 /  249*)
//  128 states,  32 CTAs   276 / 127 / 112*/ 182      (1097 /  479 /  424*/  513)
//              128 CTAs   278*/ 385 / 410 / 627
int segments_of(long long ctas, size_t smem, int spt, int L, int tile) {
    const double row = spt == 4 ? 0.065 : spt == 8 ? 0.084 : 0.135;
    const int per_sm = std::min<int>(spt <= 8 ? 4 : 3, 227 * 1024 / (int)(smem + 1024));
    auto cost = [&](int s) {
        const double w = (double)(ctas * s) / 148, even = s > 4 ? 1.1 * w : w;
        const double rounds = std::floor(even / per_sm), rest = std::ceil(even - rounds * per_sm - 1e-9);
        auto rows = [s](double v) { return s == 1 ? std::max(1.0, 0.38 + 0.53 * v) : 0.8 + v; };
        const double t = rounds * rows(per_sm) + (rest > 0 ? rows(rest) : 0.0);
        return L * row * t / s + (s == 1 ? 0.0 : s == 4 ? 4 + w : s == 8 ? 4.5 + w : 3 + 5 * w);
    };
    int best = 1;
    for (int s = 4; s <= 16; s *= 2)
        if (L >= s * 4 * tile && cost(s) < cost(best)) best = s;
    return best;
}

template <typename T, int SPT, int LANES, bool VEC>
cudaError_t launch_vec(ScanArgs a, cudaStream_t st) {
    using C = ScanTile<T, SPT, LANES, VEC>;
    a.blocks_per_group = (a.dpg + C::CH - 1) / C::CH;
    const long long blocks = (long long)a.B * a.G * a.blocks_per_group;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const size_t cut_smem = sizeof(typename C::Smem) + sizeof(typename C::Segment);
    const int segments = segments_of(blocks, cut_smem, SPT, a.L, C::TT);
    auto kern = segments > 1 ? selective_scan_kernel<T, SPT, LANES, VEC, true>
                             : selective_scan_kernel<T, SPT, LANES, VEC, false>;
    const size_t smem = segments > 1 ? cut_smem : sizeof(typename C::Smem);
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    if (segments > 8) {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (err != cudaSuccess) return err;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)segments);
    cfg.blockDim = dim3(C::NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = (unsigned)segments;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = segments > 1 ? 1 : 0;
    err = cudaLaunchKernelEx(&cfg, kern, a);
    if (err == cudaSuccess) note_launches(1);
    return err;
}

template <typename T, int SPT, int LANES>
cudaError_t launch_scan(const ScanArgs &a, cudaStream_t st) {
    auto fits = [](const void *p, long long ld) {
        return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * (long long)sizeof(T) % 16 == 0;
    };
    const bool vec = fits(a.u, a.ldu) && fits(a.delta, a.ldd) && (!a.z || fits(a.z, a.ldz)) && fits(a.bm, a.ldb) &&
                     fits(a.cm, a.ldc) && fits(a.y, a.D) && (a.G == 1 || (fits(nullptr, a.dpg) && fits(nullptr, a.N)));
    return vec ? launch_vec<T, SPT, LANES, true>(a, st) : launch_vec<T, SPT, LANES, false>(a, st);
}

template <typename T>
cudaError_t launch_n(const ScanArgs &a, cudaStream_t st) {
    // (its grid: threads of a sequence in an int, sequences in y)
    const long long threads = (long long)a.D * token_lanes(a.N);
    if (a.L <= token_rows(a.B * threads) && threads <= 0x7fffff00LL && a.B <= 65535) return launch_tokens<T>(a, st);
    if (a.N <= 8) return launch_scan<T, 4, 2>(a, st);
    if (a.N <= 16) return launch_scan<T, 8, 2>(a, st);
    if (a.N <= 32) return launch_scan<T, 8, 4>(a, st);
    if (a.N <= 64) return launch_scan<T, 8, 8>(a, st);
    return launch_scan<T, 16, 8>(a, st);
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
    // (the extents' limit keeps rows rounded up to whole tiles of 16 segments, and
    // channels to whole CTAs, in an int)
    if (d->B < 0 || d->L < 0 || d->D < 1 || d->L > RET_MAX_EXTENT || d->D > RET_MAX_EXTENT || d->N < 1 ||
        d->N > RET_MAX_SCAN_STATES || d->G < 1 || d->D % d->G)
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
