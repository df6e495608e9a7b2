// gdn_mm_kernel.h -- the kernels of the matrix products with what follows them
// in their epilogue, and how a product is cut, shared by gdn_linear and
// gdn_gated_linear.
#pragma once
#include "gdn_device.h"
#include "gdn_launch.h"
#include "gdn_mm.h"
#include "gdn_row.h"
#include "gdn_tile.h"

namespace gdn {

constexpr int kCUs = 256;  // compute units of the MI355X

enum { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3 };

__device__ __forceinline__ float sigmoid_fast(float z) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-z * LOG2E));
}

// Phi(z) of the normal distribution, and e = exp(-z^2 / 2).  With a = |z| the
// lower tail is Q(a) = e R(a), R the ratio of the tail to e, which falls like
// 1 / a: R(a) = t P(s) with t = 1 / (a + 2.875), s = a t, and P of degree 8
// fitted to the ratio so that the largest relative error on [0, 13.5] is least
// (2.6e-8), so the tail keeps its accuracy down to where it leaves fp32's
// normal range; evaluated in fp32: 4.3e-7 of Q, 1.8e-7 of Phi for z > 0.
// The exponent's rounding costs 2^-24 z^2 of e relatively (7.5e-6 at -13).
// FULL corrects it by the bits that the square and the product lost (e within
// 1.2e-7); bf16 outputs, which round to 2^-8, do without: 32768 x 4096 x 1024
// with bias takes 319 us to bf16 and 360 to fp32, 311 and 328 with a rational
// form of degree 5 that is accurate absolutely only (1e-2 of the tail at -8).
template <bool FULL>
__device__ __forceinline__ float normal_cdf(float z, float &e) {
    const float a = FULL ? fminf(fabsf(z), 16.f) : fabsf(z);  // a^2 finite for the correction; e is 0 from 14 on
    const float t = __builtin_amdgcn_rcpf(a + 2.875f), s = fmaf(t, -2.875f, 1.f);
    const float h = a * a, m = h * (-0.5f * LOG2E);
    e = __builtin_amdgcn_exp2f(m);
    if constexpr (FULL) {
        float r = fmaf(h, -0.5f * LOG2E, -m);
        r = fmaf(h, -9.62981517e-9f, r);  // -log2(e) / 2 beyond its fp32 value
        r = fmaf(fmaf(a, a, -h), -0.5f * LOG2E, r);
        e = fmaf(e, r * 0.693147182f, e);
    }
    float p = fmaf(s, -0.0829192773f, 0.24741888f);
    p = fmaf(s, p, -0.165203735f);
    p = fmaf(s, p, -0.0536689647f);
    p = fmaf(s, p, -0.192989036f);
    p = fmaf(s, p, 0.285614789f);
    p = fmaf(s, p, 0.783157051f);
    p = fmaf(s, p, -1.8599999f);
    p = fmaf(s, p, 1.4375f);
    const float q = e * (t * p);
    return z < 0.f ? q : 1.f - q;
}

// FULL: for fp32 outputs.
template <bool FULL>
__device__ __forceinline__ float act_fwd(int act, float z) {
    switch (act) {
        case ACT_RELU: return z < 0.f ? 0.f : z;  // NaN stays
        case ACT_SILU: return z * sigmoid_fast(z);
        case ACT_GELU: {
            float e;
            return z * normal_cdf<FULL>(z, e);
        }
    }
    return z;
}

// dy act'(z)
__device__ __forceinline__ float dz_of(int act, float dy, float z) {
    switch (act) {
        case ACT_RELU: return z > 0.f ? dy : 0.f;  // a choice: 0 times an infinity would be NaN
        case ACT_SILU: {
            const float p = sigmoid_fast(z);
            return dy * (p * (1.f + z * (1.f - p)));
        }
        case ACT_GELU: {
            float e;
            const float c = normal_cdf<true>(z, e);
            return dy * (c + z * e * 0.3989422804014327f);
        }
    }
    return dy;
}

// What rounding left of d (nothing of an infinity or NaN: the first plane holds it).
__device__ __forceinline__ float rest(float d, float hi) { return fabsf(hi) < __builtin_inff() ? d - hi : 0.f; }

// The epilogue of eight consecutive columns of one row.
struct Epilogue {
    const float *xs, *ws, *bias;
    const void *residual;
    void *y;
    uint16_t *z;
    long ld;        // columns of y, residual and z
    int act;
    bool y32;
    bool past;      // y is larger than the L2 caches together: it leaves by non-temporal stores
    // What columns j .. j + 7 share over all rows, and what a row adds.
    struct Cols {
        f32x8 s, b;
    };
    struct Row {
        u32x4 r0, r1;  // residual: eight bf16, or eight fp32
    };
    __device__ __forceinline__ Cols cols(int j, int J) const {
        Cols c;
        if (xs) c.s = load8v(ws, j, J);
        if (bias) c.b = load8v(bias, j, J);
        return c;
    }
    // the residual's piece, only for j + 8 <= J
    __device__ __forceinline__ Row row(long i, int j) const {
        Row o;
        if (y32) {
            const u32x4_a2 *p = (const u32x4_a2 *)((const float *)residual + i * ld + j);
            o.r0 = p[0];
            o.r1 = p[1];
        } else {
            o.r0 = *(const u32x4_a2 *)((const uint16_t *)residual + i * ld + j);
        }
        return o;
    }
    __device__ __forceinline__ f32x8 before(f32x8 v, const Cols &c, float a) const {
        if (xs) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] * a * c.s[e];
        }
        if (bias) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += c.b[e];
        }
        return v;
    }
    __device__ __forceinline__ f32x8 activate(f32x8 v) const {
        if (act == ACT_RELU) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = act_fwd<true>(ACT_RELU, v[e]);
        } else if (act == ACT_SILU) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = act_fwd<true>(ACT_SILU, v[e]);
        } else if (act == ACT_GELU && y32) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = act_fwd<true>(ACT_GELU, v[e]);
        } else if (act == ACT_GELU) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = act_fwd<false>(ACT_GELU, v[e]);
        }
        return v;
    }
    // N whole pieces (j + 8 <= J) in rows i, i + step, .., x_scale applied
    // already; with what cols() and, RES, row() fetched.  Each stage runs over
    // all of them, so that the branches on what there is to do are taken
    // once.  Nothing is loaded here: a wait for a load is a wait for every
    // store before it.
    template <bool XS, bool RES, int N>
    __device__ __forceinline__ void whole(f32x8 (&v)[N], const Cols &c, const Row (&o)[N], long i, int step, int j,
                                          int I) const {
        const long at = i * ld + j, hop = (long)step * ld;
        const int n = i < I ? (int)((I - i + step - 1) / step) : 0;  // rows that are there
        if (XS) {
#pragma unroll
            for (int q = 0; q < N; ++q)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[q][e] *= c.s[e];
        }
        if (bias) {
#pragma unroll
            for (int q = 0; q < N; ++q)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[q][e] += c.b[e];
        }
        if (z) {  // read again in the backward only
#pragma unroll
            for (int q = 0; q < N; ++q)
                if (q < n) store8nt(z + at + q * hop, v[q]);
        }
        if (act == ACT_RELU) {
#pragma unroll
            for (int q = 0; q < N; ++q)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[q][e] = act_fwd<true>(ACT_RELU, v[q][e]);
        } else if (act == ACT_SILU) {
#pragma unroll
            for (int q = 0; q < N; ++q)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[q][e] = act_fwd<true>(ACT_SILU, v[q][e]);
        } else if (act == ACT_GELU && y32) {
#pragma unroll
            for (int q = 0; q < N; ++q)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[q][e] = act_fwd<true>(ACT_GELU, v[q][e]);
        } else if (act == ACT_GELU) {
#pragma unroll
            for (int q = 0; q < N; ++q)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[q][e] = act_fwd<false>(ACT_GELU, v[q][e]);
        }
        if (y32) {
            if (RES) {
#pragma unroll
                for (int q = 0; q < N; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[q][e] += __uint_as_float(o[q].r0[e]);
                        v[q][4 + e] += __uint_as_float(o[q].r1[e]);
                    }
            }
#pragma unroll
            for (int q = 0; q < N; ++q)
                if (q < n) store8p((float *)y + at + q * hop, v[q], past);
        } else {
            if (RES) {
#pragma unroll
                for (int q = 0; q < N; ++q) {
                    const f32x8 t = bf16x8_to_f32(o[q].r0);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[q][e] += t[e];
                }
            }
#pragma unroll
            for (int q = 0; q < N; ++q)
                if (q < n) store8p((uint16_t *)y + at + q * hop, v[q], past);
        }
    }
    // any piece that begins in the row
    __device__ __forceinline__ void any(f32x8 v, long i, int j, int J) const {
        v = before(v, cols(j, J), xs ? xs[i] : 0.f);
        if (z) store8v(z + i * ld, v, j, J);
        v = activate(v);
        if (residual) {
            const f32x8 t = y32 ? load8v((const float *)residual + i * ld, j, J)
                                : load8v((const uint16_t *)residual + i * ld, j, J);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += t[e];
        }
        if (y32) store8v((float *)y + i * ld, v, j, J);
        else store8v((uint16_t *)y + i * ld, v, j, J);
    }
};

// The epilogue of a gated product: eight consecutive columns of a row of the
// gate and of the up product, y = act(gate) up.
struct GatedEpilogue {
    const float *xs, *ws, *bias;  // ws and bias: 2 N, the gate's first
    void *y;
    uint16_t *z;    // [M, 2 N]: gate, then up
    long ld;        // N
    int act;
    bool y32;
    bool past;      // as in Epilogue
    struct Cols {
        f32x8 sg, su, bg, bu;
    };
    __device__ __forceinline__ Cols cols(int j, int J) const {
        Cols c;
        if (xs) {
            c.sg = load8v(ws, j, J);
            c.su = load8v(ws + ld, j, J);
        }
        if (bias) {
            c.bg = load8v(bias, j, J);
            c.bu = load8v(bias + ld, j, J);
        }
        return c;
    }
    // y of N pieces, from their gate and up arguments
    template <int N>
    __device__ __forceinline__ void gate(f32x8 (&g)[N], const f32x8 (&u)[N]) const {
        if (act == ACT_SILU) {
#pragma unroll
            for (int q = 0; q < N; ++q)
#pragma unroll
                for (int e = 0; e < 8; ++e) g[q][e] = act_fwd<true>(ACT_SILU, g[q][e]);
        } else if (act == ACT_RELU) {
#pragma unroll
            for (int q = 0; q < N; ++q)
#pragma unroll
                for (int e = 0; e < 8; ++e) g[q][e] = act_fwd<true>(ACT_RELU, g[q][e]);
        } else if (act == ACT_GELU && y32) {
#pragma unroll
            for (int q = 0; q < N; ++q)
#pragma unroll
                for (int e = 0; e < 8; ++e) g[q][e] = act_fwd<true>(ACT_GELU, g[q][e]);
        } else if (act == ACT_GELU) {
#pragma unroll
            for (int q = 0; q < N; ++q)
#pragma unroll
                for (int e = 0; e < 8; ++e) g[q][e] = act_fwd<false>(ACT_GELU, g[q][e]);
        }
#pragma unroll
        for (int q = 0; q < N; ++q)
#pragma unroll
            for (int e = 0; e < 8; ++e) g[q][e] *= u[q][e];
    }
    // N pieces in rows i, i + 1, .., x_scale applied already; whole ones (j + 8 <= ld), or, TAIL, any.  Nothing is
    // loaded here: a wait for a load is a wait for every store before it (1037 x 2731 x 1024 in e4m3 18.4 us with
    // the last tile's bias and scales loaded there, 15.7 so; 4000 x 2731 x 1024 in bf16 78 and 51).
    template <bool XS, bool TAIL, int N>
    __device__ __forceinline__ void pieces(f32x8 (&g)[N], f32x8 (&u)[N], const Cols &c, long i, int j, int I) const {
        const int n = i < I && (!TAIL || j < ld) ? (int)(I - i) : 0;  // rows that are there
        if (XS) {
#pragma unroll
            for (int q = 0; q < N; ++q)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    g[q][e] *= c.sg[e];
                    u[q][e] *= c.su[e];
                }
        }
        if (bias) {
#pragma unroll
            for (int q = 0; q < N; ++q)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    g[q][e] += c.bg[e];
                    u[q][e] += c.bu[e];
                }
        }
        if (z) {  // read again in the backward only
#pragma unroll
            for (int q = 0; q < N; ++q)
                if (q < n) {
                    uint16_t *row = z + (i + q) * 2 * ld;
                    if (TAIL) {
                        store8v(row, g[q], j, (int)ld);
                        store8v(row + ld, u[q], j, (int)ld);
                    } else {
                        store8nt(row + j, g[q]);
                        store8nt(row + ld + j, u[q]);
                    }
                }
        }
        gate(g, u);
        if (y32) {
#pragma unroll
            for (int q = 0; q < N; ++q)
                if (q < n) {
                    float *row = (float *)y + (i + q) * ld;
                    if (TAIL) store8v(row, g[q], j, (int)ld);
                    else store8p(row + j, g[q], past);
                }
        } else {
#pragma unroll
            for (int q = 0; q < N; ++q)
                if (q < n) {
                    uint16_t *row = (uint16_t *)y + (i + q) * ld;
                    if (TAIL) store8v(row, g[q], j, (int)ld);
                    else store8p(row + j, g[q], past);
                }
        }
    }
    // any piece that begins in the row
    __device__ __forceinline__ void any(f32x8 g, f32x8 u, long i, int j, int J) const {
        const Cols c = cols(j, J);
        if (xs) {
            const float a = xs[i];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                g[e] = g[e] * a * c.sg[e];
                u[e] = u[e] * a * c.su[e];
            }
        }
        if (bias) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                g[e] += c.bg[e];
                u[e] += c.bu[e];
            }
        }
        if (z) {
            store8v(z + i * 2 * ld, g, j, J);
            store8v(z + i * 2 * ld + ld, u, j, J);
        }
        f32x8 v[1] = {g};
        const f32x8 w[1] = {u};
        gate(v, w);
        if (y32) store8v((float *)y + i * ld, v[0], j, J);
        else store8v((uint16_t *)y + i * ld, v[0], j, J);
    }
};

// Operand types of a product.  The e4m3 instructions, 128 and 32 deep alike,
// keep fewer bits than fp32 while they add: products go in groups of eight
// consecutive k, each cut off (towards zero) at 2^-13 of 2^(ex + ew), the
// largest sum of exponents in the group (subnormal values count as -6), and
// the groups' sums are added in fp32 (measured on single products).  Of normal
// values at most 7 * 2^-13 = 2^-10.2 of a group's sum of |x w| is lost so; sums
// of 4096 normally distributed values are off by 1e-5 relatively, bf16 ones by
// 7e-8.  A choice for bf16 outputs:
// their rounding is 2^-8 of the value, that of the operands to e4m3 up to 2^-3
// of each product, and the way over bf16 fragments takes twice the time (1500
// TFLOP/s for 2945).  For fp32 outputs the values are converted to bf16, which
// holds them exactly, as they leave LDS.
enum { MM_BF16 = 0, MM_F8 = 1, MM_F8_F32 = 2 };

// LDS of a workgroup: NBUF slabs; bias and w_scale of the tile's columns and
// x_scale of its rows; 256 bytes a wave that touches write to.
template <int BI, int BJ, int WI, int WJ, int NBUF>
constexpr int mm_lds() {
    return NBUF * (BI + BJ) * 128 + (2 * BJ + BI) * 4 + WI * WJ * 256;
}

// One tile of one split of k.  part (nullable): fp32 partial sums [split, I, J]
// instead of the epilogue.  With a GatedEpilogue the tile's BJ rows of U are
// BJ / 2 gate and BJ / 2 up rows, J counts the outputs' columns, and partial
// sums are [split, I, 2 J].
template <int BI, int BJ, int WI, int WJ, int NBUF, bool TV, bool TU, int MODE, class EP>
__device__ __forceinline__ void mm_body(char *smem, const MmArgs &a, const EP &ep, float *part, int tile, int split) {
    constexpr bool GATED = std::is_same_v<EP, GatedEpilogue>;
    constexpr bool F8 = MODE != MM_BF16;
    constexpr int W = WI * WJ, NI = BI / WI / 16, NJ = BJ / WJ / 16;  // 16-wide tiles per wave
    using SV = Stage<BI, W, TV>;
    using SU = Stage<BJ, W, TU>;
    constexpr int SLAB = F8 ? 128 : 64;            // values of k per slab
    constexpr int BUF = SV::kBytes + SU::kBytes;
    constexpr bool AHEAD = BI == 256 && !TV;       // see the epilogue
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int bi, bj;
    mm_tile(tile, a.ti, a.tj, bi, bj);
    const int i0 = bi * BI, j0 = bj * (GATED ? BJ / 2 : BJ);
    SV sv;
    SU su;
    constexpr int ES = F8 ? 1 : 2;
    const int per = (a.K + SLAB - 1) / SLAB;       // slabs of one plane
    const int lastb = (a.K - (per - 1) * SLAB) * ES;  // k bytes of its last slab
    const int s0 = split * a.per_split, s1 = min(s0 + a.per_split, a.slabs);
    const int p0 = s0 / per;
    sv.init(a.V, a.ldv, i0, a.I - i0, a.K, a.part_stride, per, p0, s0 - p0 * per, lane, wave);
    if constexpr (GATED) su.init_pairs(a.U, a.ldu, j0, a.J - j0, a.K, a.pair, per, s0, lane, wave);
    else su.init(a.U, a.ldu, j0, a.J - j0, a.K, 0, per, p0, s0 - p0 * per, lane, wave);
    lds_cchar *lds = (lds_cchar *)smem;
    const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

    // What the epilogue needs of the columns and rows, by way of LDS: loaded
    // there, it would wait for the stores before it.  Issued before the slabs,
    // it has landed when the first of them has.
    const uint32_t aux0 = lds0 + NBUF * BUF, touch0 = aux0 + (2 * BJ + BI) * 4 + wave * 256;
    const float *aux = (const float *)(smem + NBUF * BUF);
    auto fetch = [&](const float *p, int at, int n, int valid) {
        const i32x4 rs = make_rsrc((const char *)p, (uint32_t)min(n, valid) * 4);
        for (int k = wave; k < n / 64; k += W)
            lds_touch(__builtin_amdgcn_readfirstlane(aux0 + at * 4 + k * 256), (k * 64 + lane) * 4, rs);
    };
    if (!part) {
        if constexpr (GATED) {  // the gate's half, then the up half
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (ep.bias) fetch(ep.bias + h * ep.ld + j0, h * (BJ / 2), BJ / 2, a.J - j0);
                if (F8) fetch(ep.ws + h * ep.ld + j0, BJ + h * (BJ / 2), BJ / 2, a.J - j0);
            }
        } else {
            if (ep.bias) fetch(ep.bias + j0, 0, BJ, a.J - j0);
            if (F8) fetch(ep.ws + j0, BJ, BJ, a.J - j0);
        }
        if (F8) fetch(ep.xs + i0, 2 * BJ, BI, a.I - i0);
    }

    f32x4 acc[NJ][NI];
#pragma unroll
    for (int x = 0; x < NJ; ++x)
#pragma unroll
        for (int y = 0; y < NI; ++y) acc[x][y] = zero4();

    // Slab loads: piece() issues the n-th instruction of the slab that is due,
    // V's first, into buffer buf; move() goes on to the next slab, in three
    // steps that the loop spreads out.
    constexpr int LV = SV::kLoads, LU = SU::kLoads;
    int s = s0 - p0 * per, next = s0;
    bool last;
    int left;
    auto bound = [&] {
        last = s == per - 1;
        left = last ? lastb : 128;
        sv.bound(last, next < s1);
        su.bound(last, next < s1);
    };
    auto move = [&](int step) {
        if (step == 0) sv.advance(last);
        if (step == 1) su.advance(last);
        if (step == 2) {
            s = last ? 0 : s + 1;
            ++next;
            bound();
        }
    };
    auto piece = [&](int buf, int n) {
        if (n < LV) sv.load(lds0 + buf * BUF, n, left, wave);
        else su.load(lds0 + buf * BUF + SV::kBytes, n - LV, left, wave);
    };
    auto load = [&](int buf) {
#pragma unroll
        for (int n = 0; n < LV + LU; ++n) piece(buf, n);
    };
    auto move_on = [&] {
        move(0);
        move(1);
        move(2);
    };
    bound();
    const int wi = (wave % WI) * NI * 16, wj = (wave / WI) * NJ * 16;
    if constexpr (MODE == MM_BF16) {
        // Fragments are read half a slab ahead of their products, in two
        // register sets, so the MFMAs only wait where waves meet: in the
        // middle of slab t every wave holds the last of t in registers, slab
        // t + 1 has landed, and the loads of t + NBUF go into t's buffer.
        // Past the end the loads write zeros and the reads are not used,
        // which keeps the loop free of branches.
        u32x4 fv[2][NI], fu[2][NJ];
        // n-th read of a set: the V fragments, which the first products all
        // need, then those of U
        auto read = [&](auto set, int buf, int n) {
            constexpr int h = decltype(set)::value;
            lds_cchar *iv = lds + buf * BUF, *iu = iv + SV::kBytes;
            if (n < NI) fv[h][n] = mm_frag<BI, TV>(iv, wi + 16 * n, h, lane);
            else fu[h][n - NI] = mm_frag<BJ, TU>(iu, wj + 16 * (n - NI), h, lane);
        };
        constexpr int R = NI + NJ, L = LV + LU, MM = NI * NJ;
        // m-th product of a half, and nothing moved across it
        auto mul = [&](auto set, int m) {
            constexpr int h = decltype(set)::value;
            const int x = m / NI, y = m % NI;
            acc[x][y] = mma_bf16_raw(acc[x][y], fu[h][x], fv[h][y]);
            __builtin_amdgcn_sched_barrier(0);
        };
        constexpr std::integral_constant<int, 0> h0;
        constexpr std::integral_constant<int, 1> h1;
        if (s0 < s1) {
#pragma unroll
            for (int n = 0; n < NBUF; ++n) {
                if (n > 0) move_on();
                load(n);
            }
            mm_wait<(NBUF - 1) * (LV + LU)>();
            __builtin_amdgcn_s_barrier();
            mm_fence();
#pragma unroll
            for (int n = 0; n < R; ++n) read(h0, 0, n);
        }
        int buf = 0;
        for (int t = s0; t < s1; ++t) {
            // About one read, or one slab load, after each product: they issue
            // while the matrix cores are busy with it (in groups between
            // groups of products, 1380 against 1430 TFLOP/s at 8192^3).  The
            // last ones leave a few products before the half ends.
            constexpr int E0 = MM * 6 / 8, E1 = MM * 7 / 8, OPS = R + L;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int m = 0; m < MM; ++m) {
                mul(h0, m);
#pragma unroll
                for (int n = m * R / E0; n < (m + 1) * R / E0 && n < R; ++n) read(h1, buf, n);
                if (m == MM / 4) move(0);
                if (m == MM / 2) move(1);
                if (m == MM * 3 / 4) move(2);
                __builtin_amdgcn_sched_barrier(0);
            }
            mm_wait<(NBUF - 2) * L>();
            __builtin_amdgcn_s_barrier();
            mm_fence();
            const int after = buf + 1 < NBUF ? buf + 1 : 0;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int m = 0; m < MM; ++m) {
                mul(h1, m);
#pragma unroll
                for (int k = m * OPS / E1; k < (m + 1) * OPS / E1 && k < OPS; ++k) {
                    // of OPS turns, L go to loads, evenly, the first one first
                    const int before = (k * L + OPS - 1) / OPS, upto = ((k + 1) * L + OPS - 1) / OPS;
                    if (upto > before) piece(buf, before);
                    else read(h0, after, k - before);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            buf = after;
        }
        mm_wait<0>();  // the loads past the end have written before LDS is used again
    } else if constexpr (MODE == MM_F8) {
        // The same with whole-slab fragments: the products of the first half
        // of the U fragments, then those of the second.  Every wave holds the
        // second half's in registers when it comes to the middle; from there
        // on the next slab's first half is read, and each V fragment as soon
        // as its last product of this slab is under way.
        constexpr int H = NJ / 2, MM = NI * H, L = LV + LU;
        i32x8 fv[NI], fa[H], fb[H];
        auto pair_v = [&](int buf, int y) {
            lds_cchar *iv = lds + buf * BUF;
            return mm_pair(mm_frag<BI, TV>(iv, wi + 16 * y, 0, lane), mm_frag<BI, TV>(iv, wi + 16 * y, 1, lane));
        };
        auto pair_u = [&](int buf, int x) {
            lds_cchar *iu = lds + buf * BUF + SV::kBytes;
            return mm_pair(mm_frag<BJ, TU>(iu, wj + 16 * x, 0, lane), mm_frag<BJ, TU>(iu, wj + 16 * x, 1, lane));
        };
        if (s0 < s1) {
#pragma unroll
            for (int n = 0; n < NBUF; ++n) {
                if (n > 0) move_on();
                load(n);
            }
            mm_wait<(NBUF - 1) * L>();
            __builtin_amdgcn_s_barrier();
            mm_fence();
#pragma unroll
            for (int y = 0; y < NI; ++y) fv[y] = pair_v(0, y);
#pragma unroll
            for (int x = 0; x < H; ++x) fa[x] = pair_u(0, x);
        }
        int buf = 0;
        for (int t = s0; t < s1; ++t) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int m = 0; m < MM; ++m) {
                const int y = m / H, x = m % H;
                acc[x][y] = mma_f8_slab(acc[x][y], fa[x], fv[y]);
                __builtin_amdgcn_sched_barrier(0);
                if (m % 2 == 0 && m / 2 < H) fb[m / 2] = pair_u(buf, H + m / 2);
                if (m == MM / 4) move(0);
                if (m == MM / 2) move(1);
                if (m == MM * 3 / 4) move(2);
                __builtin_amdgcn_sched_barrier(0);
            }
            mm_wait<(NBUF - 2) * L>();
            __builtin_amdgcn_s_barrier();
            mm_fence();
            const int after = buf + 1 < NBUF ? buf + 1 : 0;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int m = 0; m < MM; ++m) {
                const int y = m / H, x = m % H;
                acc[H + x][y] = mma_f8_slab(acc[H + x][y], fb[x], fv[y]);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int n = m * L / MM; n < (m + 1) * L / MM; ++n) piece(buf, n);
                if (m % 2 == 1 && m / 2 < H) fa[m / 2] = pair_u(after, m / 2);
                if (x == H - 1) fv[y] = pair_v(after, y);
                __builtin_amdgcn_sched_barrier(0);
            }
            buf = after;
        }
        mm_wait<0>();
    } else {
        if (s0 < s1) {
#pragma unroll
            for (int n = 0; n < NBUF - 1; ++n) {
                load(n);
                move_on();
            }
        }
        int buf = 0;
        for (int t = s0; t < s1; ++t) {
            // this slab's loads have landed (each wave its own), and every
            // wave is done with the buffer that the next ones go to
            mm_wait<(NBUF - 2) * (LV + LU)>();
            __builtin_amdgcn_s_barrier();
            mm_fence();
            load(buf > 0 ? buf - 1 : NBUF - 1);
            move_on();
            lds_cchar *iv = lds + buf * BUF, *iu = iv + SV::kBytes;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 fv[NI][2];
#pragma unroll
                for (int y = 0; y < NI; ++y) f8_to_bf16(fv[y], mm_frag<BI, TV>(iv, wi + 16 * y, h, lane));
#pragma unroll
                for (int x = 0; x < NJ; ++x) {
                    u32x4 fu[2];
                    f8_to_bf16(fu, mm_frag<BJ, TU>(iu, wj + 16 * x, h, lane));
#pragma unroll
                    for (int y = 0; y < NI; ++y) {
                        acc[x][y] = mma_bf16_raw(acc[x][y], fu[0], fv[y][0]);
                        acc[x][y] = mma_bf16_raw(acc[x][y], fu[1], fv[y][1]);
                    }
                }
            }
            buf = buf + 1 < NBUF ? buf + 1 : 0;
        }
        mm_wait<0>();
    }

    // Epilogue, from the accumulators to memory: a lane holds four columns of
    // a row in each 16-wide tile.  Exchanged between lanes 16 apart, two tiles
    // give it eight consecutive ones; exchanged between the lanes of an even
    // row and the next one, four tiles give a row's 64 columns, in bf16 a
    // cache line, to eight lanes.
    // The accumulators are vector registers from here on, and so in the loop:
    // left to choose, the compiler moved those of the 128-tiles between the
    // two register files at every slab (1000 x 4096 x 4096: 47 against 35 us).
#pragma unroll
    for (int x = 0; x < NJ; ++x)
#pragma unroll
        for (int y = 0; y < NI; ++y) asm volatile("" : "+v"(acc[x][y]));
    if constexpr (AHEAD) {
        // The workgroup that follows on this XCD finds its rows of V, where
        // they are no longer than 2 KB, on the way: one touch a cache line,
        // shared among the workgroups that will use them.  They arrive during
        // the epilogue; left to the next tile's own loads, which all miss at
        // once when a band begins, such a tile took 35 us for 27.  32768 x 4096
        // x 1024 in bf16 with x from HBM: 257 against 268 us, to fp32 300
        // against 311, K = 512 166 against 173, e4m3 with K = 2048 258 against
        // 268, with SiLU and pre-activation 311 both; it costs where x is in
        // the caches already (244 against 238, with SiLU 290 against 273), and
        // with rows of 4 KB (32768 x 1024 x 2048: 112 against 104 us).
        if (a.ldv <= 2048 && tile + kCUs < a.ti * a.tj) {
            int ni, nj;
            mm_tile(tile + kCUs, a.ti, a.tj, ni, nj);
            const int shares = min(8, a.tj), rows = (BI + shares - 1) / shares, lines = ((int)a.ldv + 127) / 128;
            const i32x4 rs = make_rsrc(a.V + (long)ni * BI * a.ldv, (uint32_t)min(BI, a.I - ni * BI) * (uint32_t)a.ldv);
            for (int n = 0; n < rows * lines; n += W * 64) {
                const int u = n + wave * 64 + lane, row = (nj % shares) * rows + u / lines;
                lds_touch(__builtin_amdgcn_readfirstlane(touch0),
                          u < rows * lines ? (uint32_t)row * (uint32_t)a.ldv + (u % lines) * 128 : kOutOfRange, rs);
            }
        }
    }
    const int r = lane & 15, g = lane >> 4;
    // Four tiles p, the lane's four columns of row r in each, to v: rows r & ~1
    // and the next one, eight columns (16 (g & 1) + 8 (g >> 1) ..) of the
    // first two tiles for even r, of the last two for odd r.
    auto exchange = [&](f32x8 (&v)[2], const f32x4 (&p)[4]) {
        const bool odd = r & 1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // the odd rows of 16 lanes of the first and the even ones of the second change places
            const auto a0 = __builtin_amdgcn_permlane16_swap(__float_as_uint(p[0][e]), __float_as_uint(p[1][e]), false, false);
            const auto a1 = __builtin_amdgcn_permlane16_swap(__float_as_uint(p[2][e]), __float_as_uint(p[3][e]), false, false);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t got = dpp_u32<0xb1, 0xf>(odd ? a0[h] : a1[h]);  // from the neighbouring lane
                v[0][4 * h + e] = __uint_as_float(odd ? got : a0[h]);
                v[1][4 * h + e] = __uint_as_float(odd ? a1[h] : got);
            }
        }
    };
    if constexpr (GATED) {
        // Of the wave's tiles along j the even ones are gate, the odd ones up.
        // A turn: the 64 columns of a row tile (eight tiles), or the 32 columns
        // of two row tiles (four).
        static_assert(NJ == 8 || (NJ == 4 && NI % 2 == 0), "eight tiles a turn");
        constexpr int TURNS = NJ == 8 ? NI : NI / 2;
        const int jl = wj / 2 + (NJ == 8 ? 32 * (r & 1) : 0) + 16 * (g & 1) + 8 * (g >> 1);
        const int il = wi + (r & ~1) + (NJ == 8 ? 0 : 16 * (r & 1));
        auto pick = [&](f32x8 (&vg)[2], f32x8 (&vu)[2], int t) {
            f32x4 pg[4], pu[4];
#pragma unroll
            for (int k = 0; k < TURNS; ++k) {
                if (k == t) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int x = NJ == 8 ? 2 * q : 2 * (q & 1), y = NJ == 8 ? k : 2 * k + (q >> 1);
                        pg[q] = acc[x][y];
                        pu[q] = acc[x + 1][y];
                    }
                    asm volatile("; gated turn %0" ::"n"(k));  // distinct per case, as below
                }
            }
            exchange(vg, pg);
            exchange(vu, pu);
        };
        const int j = j0 + jl;
        auto row = [&](int t) { return i0 + il + 16 * (NJ == 8 ? t : 2 * t); };
        if (part) {
            part += (long)split * a.I * 2 * a.J;
#pragma unroll 1
            for (int t = 0; t < TURNS; ++t) {
                f32x8 vg[2], vu[2];
                pick(vg, vu, t);
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (row(t) + q < a.I && j < a.J) {
                        float *pr = part + (long)(row(t) + q) * 2 * a.J;
                        store8v(pr, vg[q], j, a.J);
                        store8v(pr + a.J, vu[q], j, a.J);
                    }
            }
        } else {
            GatedEpilogue::Cols c;
            if (ep.bias) {
                c.bg = load8v(aux + jl);
                c.bu = load8v(aux + BJ / 2 + jl);
            }
            if (F8) {
                c.sg = load8v(aux + BJ + jl);
                c.su = load8v(aux + BJ + BJ / 2 + jl);
            }
            auto turns = [&](auto tail) {
#pragma unroll 1
                for (int t = 0; t < TURNS; ++t) {
                    f32x8 vg[2], vu[2];
                    pick(vg, vu, t);
                    if (F8) {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const float s = aux[2 * BJ + row(t) - i0 + q];
                            vg[q] *= s;
                            vu[q] *= s;
                        }
                    }
                    ep.template pieces<F8, decltype(tail)::value>(vg, vu, c, row(t), j, a.I);
                }
            };
            if (j0 + BJ / 2 <= a.J) turns(std::false_type{});
            else turns(std::true_type{});
        }
    } else {
        constexpr int NQ = NJ / 4, TURNS = NQ * NI;  // a turn: 64 columns of a row tile
        const int jl = wj + 32 * (r & 1) + 16 * (g & 1) + 8 * (g >> 1), il = wi + (r & ~1);
        // (the loops over turns stay loops: unrolled, their code is longer than
        // the instruction cache)
        // v: the lane's columns of rows il and il + 1
        auto pick = [&](f32x8 (&v)[2], int t) {
            f32x4 p[4];
#pragma unroll
            for (int k = 0; k < TURNS; ++k) {
                if (k == t) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) p[q] = acc[4 * (k % NQ) + q][k / NQ];
                    // distinct per case: merged, the accumulators would be
                    // indexed at run time, that is, moved to scratch memory
                    asm volatile("; turn %0" ::"n"(k));
                }
            }
            exchange(v, p);
        };
        auto col = [&](int t) { return j0 + jl + 64 * (t % NQ); };
        auto row = [&](int t) { return i0 + il + 16 * (t / NQ); };
        auto turns = [&](auto res) {
            constexpr bool RES = decltype(res)::value;
            Epilogue::Row o[2];
            auto fetch_rows = [&](int t) {
#pragma unroll
                for (int q = 0; q < 2; ++q) o[q] = ep.row(min(row(t) + q, a.I - 1), col(t));
            };
            if (RES) fetch_rows(0);
#pragma unroll 1
            for (int t = 0; t < TURNS; ++t) {
                f32x8 v[2];
                pick(v, t);
                const Epilogue::Row now[2] = {o[0], o[1]};
                if (RES && t + 1 < TURNS) fetch_rows(t + 1);  // ahead of this turn's stores
                const float *ca = aux + jl + 64 * (t % NQ);
                Epilogue::Cols c;
                if (ep.bias) c.b = load8v(ca);
                if (F8) {
                    c.s = load8v(ca + BJ);
#pragma unroll
                    for (int q = 0; q < 2; ++q) v[q] *= aux[2 * BJ + il + 16 * (t / NQ) + q];
                }
                ep.template whole<F8, RES>(v, c, now, row(t), 1, col(t), a.I);
            }
        };
        if (part) {
            part += (long)split * a.I * a.J;
#pragma unroll 1
            for (int t = 0; t < TURNS; ++t) {
                f32x8 v[2];
                pick(v, t);
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (row(t) + q < a.I && col(t) < a.J) store8v(part + (long)(row(t) + q) * a.J, v[q], col(t), a.J);
            }
        } else if (j0 + BJ <= a.J) {
            if (ep.residual) turns(std::true_type{});
            else turns(std::false_type{});
        } else {
#pragma unroll 1
            for (int t = 0; t < TURNS; ++t) {
                f32x8 v[2];
                pick(v, t);
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (row(t) + q < a.I && col(t) < a.J) ep.any(v[q], row(t) + q, col(t), a.J);
            }
        }
    }
    if (AHEAD) mm_wait<0>();  // nothing may reach LDS after the workgroup's end
}

// Grid: x = tiles, y = splits of k.
template <int BI, int BJ, int WI, int WJ, int NBUF, bool TV, bool TU, int MODE, class EP>
__global__ __launch_bounds__(WI *WJ * 64) void mm_kernel(MmArgs a, EP ep, float *part) {
    __shared__ __attribute__((aligned(1024))) char smem[mm_lds<BI, BJ, WI, WJ, NBUF>()];
    mm_body<BI, BJ, WI, WJ, NBUF, TV, TU, MODE>(smem, a, ep, part, blockIdx.x, blockIdx.y);
}

// Few rows (decode) or few columns (gate projections): every weight, or every
// row of x, is read once and used for at most 64 products, so the product is
// bound by that read.  A workgroup owns 16 MT rows and 16 NB columns; its W
// waves take turns along k in pieces of RB bytes per row.  A wave brings its
// piece of the weight rows and of the rows of x into its own part of LDS,
// whole rows' pieces per instruction: fragments loaded directly would touch 16
// rows at once, which a power-of-two row length puts on one memory channel
// (64 x 64 x 4096 in bf16: 19.8 us so, 8.1 us this way).  Waves do not wait
// for each other until their sums meet in LDS, where they are added in order.
// One launch, no workspace.  1 x 4096 x 4096 in bf16: 8.7 us in a graph, 3.9
// TB/s of weights; 1 x 4096 x 16384: 30.9 us, 4.3 TB/s.  e4m3 is converted to
// bf16 fragments for every output type (the conversion hides behind the loads).
// A gated product's 16 rows of w are eight gate and eight up rows (pair bytes
// behind); J then counts the outputs' columns, 8 NB to a workgroup.
template <int NB, int MT, int W, int RB, bool F8, class EP>
__global__ __launch_bounds__(W * 64) void mv_kernel(const char *x, const char *w, int I, int J, int K, long pair, EP ep) {
    constexpr bool GATED = std::is_same_v<EP, GatedEpilogue>;
    constexpr int CB = GATED ? 8 * NB : 16 * NB;  // output columns
    constexpr int ES = F8 ? 1 : 2;
    constexpr int RPL = 1024 / RB;              // rows per load instruction
    constexpr int UNITS = RB / 16;              // 16-byte units per row piece
    constexpr int WB = 16 * NB * RB, XB = 16 * MT * RB;
    constexpr int LDR = 16 * NB + 4;            // floats per row of a wave's sums
    constexpr int SB = W * 16 * MT * LDR * 4;
    constexpr int PPR = CB / 8, PIECES = PPR * 16 * MT;
    __shared__ __attribute__((aligned(1024))) char smem[W * (WB + XB) > SB ? W * (WB + XB) : SB];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int tj = (J + CB - 1) / CB;
    const int j0 = (int)(blockIdx.x % tj) * CB, i0 = (int)(blockIdx.x / tj) * 16 * MT;
    const int rows = min(16 * MT, I - i0);
    const uint32_t row = (uint32_t)K * ES;
    // what the epilogue's threads will need
    const int pi = threadIdx.x / PPR, pj = j0 + 8 * (threadIdx.x % PPR);
    const bool mine = threadIdx.x < PIECES && pi < rows && pj < J, full = pj + 8 <= J;
    typename EP::Cols ec;
    Epilogue::Row er;
    float ea = 1.f;
    if (PIECES <= W * 64 && mine && full) {
        ec = ep.cols(pj, J);
        if (F8) ea = ep.xs[i0 + pi];
        if constexpr (!GATED) {
            if (ep.residual) er = ep.row(i0 + pi, pj);
        }
    }
    f32x4 acc[NB][MT];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[n][m] = zero4();

    lds_cchar *wl = (lds_cchar *)smem + wave * (WB + XB), *xl = wl + WB;
    const uint32_t lw = (uint32_t)(uintptr_t)wl, lx = lw + WB;
    const char *wb = w + (long)j0 * row, *xb = x + (long)i0 * row;
    const uint32_t wr = (uint32_t)min(CB, J - j0) * row, xr = (uint32_t)rows * row;
    // unit c of row k of a piece lies at c ^ (2 swz_col(k)): the rows of a
    // fragment read fall on different banks
    const int lr = lane / UNITS;
    for (int p = wave; p * RB < (int)row; p += W) {
        const int left = (int)row - p * RB;
        const i32x4 rw = make_rsrc(wb + (long)p * RB, wr), rx = make_rsrc(xb + (long)p * RB, xr);
        i32x4 ru;
        if constexpr (GATED) ru = make_rsrc(wb + pair + (long)p * RB, wr);
#pragma unroll
        for (int n = 0; n < 16 * NB / RPL; ++n) {
            const int k = n * RPL + lr, c = ((lane % UNITS) ^ (swz_col(k & 15) << 1)) * 16;
            if constexpr (GATED) {
                const int col = (k >> 4) * 8 + (k & 7);
                lds_load(lw + n * 1024, c < left ? (uint32_t)col * row + c : kOutOfRange, (n * RPL) & 8 ? ru : rw);
            } else {
                lds_load(lw + n * 1024, c < left ? (uint32_t)k * row + c : kOutOfRange, rw);
            }
        }
#pragma unroll
        for (int n = 0; n < 16 * MT / RPL; ++n) {
            const int k = n * RPL + lr, c = ((lane % UNITS) ^ (swz_col(k & 15) << 1)) * 16;
            if (n * RPL < rows)  // rows past I: left as they are, their sums are not used
                lds_load(lx + n * 1024, c < left ? (uint32_t)k * row + c : kOutOfRange, rx);
        }
        mm_wait<0>();
        typedef __attribute__((address_space(3))) const u32x4 lds_v;
#pragma unroll
        for (int u = 0; u < RB / 64; ++u) {
            const int at = r * RB + ((4 * u + g) ^ (swz_col(r) << 1)) * 16;
            u32x4 fw[NB], fx[MT];
#pragma unroll
            for (int n = 0; n < NB; ++n) fw[n] = *(lds_v *)(wl + at + n * 16 * RB);
#pragma unroll
            for (int m = 0; m < MT; ++m) fx[m] = *(lds_v *)(xl + at + m * 16 * RB);
            if constexpr (F8) {
                u32x4 bx[MT][2];
#pragma unroll
                for (int m = 0; m < MT; ++m) f8_to_bf16(bx[m], fx[m]);
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    u32x4 bw[2];
                    f8_to_bf16(bw, fw[n]);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        acc[n][m] = mma_bf16_raw(acc[n][m], bw[0], bx[m][0]);
                        acc[n][m] = mma_bf16_raw(acc[n][m], bw[1], bx[m][1]);
                    }
                }
            } else {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int m = 0; m < MT; ++m) acc[n][m] = mma_bf16_raw(acc[n][m], fw[n], fx[m]);
            }
        }
        mm_wait<0>();  // this piece's reads are done before the next one's loads
    }
    __syncthreads();
    typedef float Sums[16 * MT][LDR];
    Sums *sums = (Sums *)smem;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) *(f32x4 *)&sums[wave][16 * m + r][16 * n + 4 * g] = acc[n][m];
    __syncthreads();
    for (int q = threadIdx.x; q < PIECES; q += W * 64) {
        const int i = q / PPR, c = 8 * (q % PPR), j = j0 + c;
        if (i >= rows || j >= J) continue;
        auto add_up = [&](int at) {
            f32x8 v = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int p = 0; p < W; ++p) {
                const f32x4 lo = *(const f32x4 *)&sums[p][i][at], hi = *(const f32x4 *)&sums[p][i][at + 4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] += lo[e];
                    v[4 + e] += hi[e];
                }
            }
            return v;
        };
        if constexpr (GATED) {
            const f32x8 g = add_up(2 * c), u = add_up(2 * c + 8);
            if (PIECES <= W * 64 && full) {
                f32x8 g1[1] = {F8 ? g * ea : g}, u1[1] = {F8 ? u * ea : u};
                ep.template pieces<F8, false>(g1, u1, ec, i0 + i, j, I);
            } else {
                ep.any(g, u, i0 + i, j, J);
            }
        } else {
            const f32x8 v = add_up(c);
            if (PIECES <= W * 64 && full) {
                f32x8 v1[1] = {F8 ? v * ea : v};
                const Epilogue::Row er1[1] = {er};
                if (ep.residual) ep.template whole<F8, true>(v1, ec, er1, i0 + i, 1, j, I);
                else ep.template whole<F8, false>(v1, ec, er1, i0 + i, 1, j, I);
            } else {
                ep.any(v, i0 + i, j, J);
            }
        }
    }
}

// ---- host side ----------------------------------------------------------------

// How a product of I x J over `slabs` slabs is cut: a tile size and a number
// of splits of k, the pair with the least estimated time.  The estimate is a
// fit to measured launches (bf16 and e4m3, all operand orders, 1 to 2600
// workgroups): 4 us a launch; a slab of the 128-tile takes 0.42 to 0.52 us
// with at most one workgroup in each compute unit (four buffers, 2.5 us more
// to start), 0.94 with two (two buffers), in between proportionally; a slab of
// the 256-tile 1.2 us alone on the card to 1.55 with all compute units at
// work; splits cost a second launch of 3 us and 8 bytes of partial sum per
// output and split at 7 TB/s (they come back from the caches).  Four buffers
// against two at 1024 x 4096 x 4096: 38.9 and 47.3 us.
inline double mm_round_us(int tile, long n, int per) {  // n workgroups, at most one round
    if (tile == 256) return per * (1.2 + 0.35 * n / kCUs);
    return n <= kCUs ? 2.5 + per * (0.42 + 0.1 * n / kCUs) : per * (0.62 + 0.32 * (n - kCUs) / kCUs);
}

inline MmPlan mm_plan(int I, int J, int slabs) {
    MmPlan best{};
    double least = 1e30;
    for (const int tile : {256, 128}) {
        const long tiles = (long)((I + tile - 1) / tile) * ((J + tile - 1) / tile);
        const long at_once = tile == 256 ? kCUs : 2 * kCUs;
        // more splits than fill the card once only add partial sums
        for (int s = 1; s <= 32 && (s == 1 || (s * 2 <= slabs && tiles * s <= at_once)); ++s) {
            const int per = (slabs + s - 1) / s;
            if (s > 1 && (slabs + per - 1) / per != s) continue;  // the same cut as a smaller s
            const long n = tiles * s;
            double us = 4.0;
            if (n <= at_once) {
                us += mm_round_us(tile, n, per);
            } else {
                us += (double)(n / at_once) * (mm_round_us(tile, at_once, per) + 2.0);
                if (n % at_once) us += mm_round_us(tile, n % at_once, per);
            }
            if (s > 1) us += 3.0 + 8.0 * s * I * J / 7e6;
            if (us < least) {
                least = us;
                best = MmPlan{tile, s, per, tile == 128 && n <= kCUs};
            }
        }
    }
    return best;
}

inline size_t mm_part_bytes(const MmPlan &p, int I, int J) {
    return p.splits > 1 ? (size_t)p.splits * I * J * sizeof(float) : 0;
}

// What the kernel for few rows or columns takes.  More columns are faster in
// tiles (32768 x 64 x 4096: 54 us there, 68 here; x 8 x 1024: 18.2 and 16.3).
constexpr int kFewRows = 64, kFewCols = 16;
inline bool mv_takes(int M, int N) {
    return M <= kFewRows || (N <= kFewCols && M < (1 << 27));  // a launch holds fewer than 2^32 threads
}

// N rows of w, of a gated product both kinds: its N / 2 columns are cut like
// the N of another.
template <bool F8, class EP>
hipError_t mv_run(const void *x, const void *w, int M, int N, int K, const EP &ep, hipStream_t st) {
    constexpr bool GATED = std::is_same_v<EP, GatedEpilogue>;
    const long pair = GATED ? (long)(N / 2) * K * (F8 ? 1 : 2) : 0;
#define GDN_MV(NBv, MTv, Wv, RBv)                                                                                  \
    hipLaunchKernelGGL((mv_kernel<NBv, MTv, Wv, RBv, F8, EP>),                                                         \
                       dim3((unsigned)((N + 16 * NBv - 1) / (16 * NBv)) * (unsigned)((M + 16 * MTv - 1) / (16 * MTv))), \
                       dim3(Wv * 64), 0, st, (const char *)x, (const char *)w, M, GATED ? N / 2 : N, K, pair, ep)
    if (M > kFewRows) {  // few columns
        GDN_MV(1, 2, 8, 256);
        return hipGetLastError();
    }
    // 16 columns a workgroup, one of these in each compute unit with its LDS
    // full of pieces in flight.  More columns than that (more) go to
    // workgroups of fewer waves, three of which share a compute unit instead
    // of taking turns (17 rows in e4m3: 4099 x 4096 8.3 against 9.3 us, 8192 x
    // 1024 5.0 against 6.8; 4096 x 4096 8.4 against 6.9 the other way round),
    // and beyond what the card holds of these at once (wide: two to a compute
    // unit for 33 rows and more, three below) 32 to one, which reads x half as
    // often (17 x 16384 x 1024 in bf16: 8.1 against 9.4 us; 17 x 4096 x 4096:
    // 15.9 against 9.7 the other way round; at the bounds, bf16: 64 x 8208 x
    // 4096 29.4 against 35.9 us, x 8192 25.8 against 25.3; 20 x 12304 x 8192
    // 48.8 against 50.0, x 12288 50.5 against 45.9).  Up to 16 rows take so
    // little LDS that two workgroups of eight waves share a compute unit.
    // There rows of 16 KB and more bring pieces of 512 bytes for up to four
    // rows of x (1 x 1024 x 16384 in bf16: 13.3 against 15.5 us, x 24576 20.1
    // against 22.6; 4 x 4096 x 8192 17.0 both; more rows lose: 16 x 4096 x 8192
    // 18.8 against 17.1, x 20480 39.1 against 36.8) and, where the rows lie a
    // multiple of 32 KB apart, on the same memory channels, for all (8 x 4096 x
    // 16384 30.1 against 35.7 us, 16 rows 31.9 against 35.3); beyond 8192
    // columns they gain nothing (1 x 8192 x 16384: 62.4 against 61.6).  Rows of
    // 2 KB, which eight waves read in one turn, go to four (1 x 32768 x 1024 in
    // bf16: 13.8 against 16.3 us, x 8192 5.4 against 5.6; 1 x 16384 x 2048: 16.8
    // against 15.5 the other way round).
    const bool wide = N > 2 * kCUs * 16, more = N > kCUs * 16;
    const long row = (long)K * (F8 ? 1 : 2);
    if (M <= 16) {
        if (row >= 16384 && !wide && (M <= 4 || row % 32768 == 0)) GDN_MV(1, 1, 8, 512);
        else if (row <= 2048 && more) GDN_MV(1, 1, 4, 256);
        else GDN_MV(1, 1, 8, 256);
    } else if (M <= 32) {
        if (N > 3 * kCUs * 16) GDN_MV(2, 2, 4, 256);
        else if (more) GDN_MV(1, 2, 4, 256);
        else GDN_MV(1, 2, 8, 256);
    } else {
        if (wide) GDN_MV(2, 4, 3, 256);
        else if (more) GDN_MV(1, 4, 3, 256);
        else GDN_MV(1, 4, 7, 256);
    }
#undef GDN_MV
    return hipGetLastError();
}

inline int slabs_of(int K, bool f8) { return (K + (f8 ? 127 : 63)) / (f8 ? 128 : 64); }

// Fills in what the plan decides.
inline void mm_set(MmArgs &a, const MmPlan &p, bool f8) {
    a.slabs = a.parts * slabs_of(a.K, f8);
    a.per_split = p.per_split;
    a.ti = (a.I + p.tile - 1) / p.tile;
    a.tj = (a.J + p.tile - 1) / p.tile;
}

// Whether an output of I x J is larger than the eight L2 caches of 4 MB.
// Non-temporal stores then leave them to the operands: 32768 x 4096 x 1024 in
// bf16 260 -> 249 us, 32768 x 1024 x 4096 in e4m3 121 -> 118.
inline bool past_caches(int I, int J, bool f32) { return (size_t)I * J * (f32 ? 4 : 2) > ((size_t)32 << 20); }

}  // namespace gdn
