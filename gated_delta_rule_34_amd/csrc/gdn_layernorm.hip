// gdn_layernorm.hip -- residual addition and layer norm in one pass (with an
// output in the input's type or in e4m3 with one scale per row), and its
// backward.
//   forward   u = x + residual;  r = u in the residual's type
//             m = mean(u), s = (mean((u - m)^2) + eps)^-1/2;  y = (u - m) s w + b
//   8 bits    scale = max|y| / 448,  q = e4m3(y / scale)
//   backward  xhat = (r - m) s,  a = w dy
//             dx = s (a - mean(a) - xhat mean(a xhat)) + dr
//             dw = sum over rows of dy xhat,  db = sum over rows of dy
// Everything is fp32 between the loads and one rounding at the stores.  The
// variance is taken of the differences to the mean, in a second turn over the
// registers that hold the row: the difference of the two moments would lose
// all bits where the mean is large beside the spread.  Bound by HBM: a row is
// read once, held in registers while its sums are formed, and written once:
// 32768 x 1024 from bf16 and a fp32 residual stream to e4m3 72 us, 5.1 TB/s (a
// large copy reaches 5.15); 4096 x 4096 in bf16 25 us; 4 x 1024 3.2 us.
// Rows are laid over threads as in the RMS norm: one wave up to 2048 columns
// in the forward and 1024 in the backward, beyond that 256, 512 or 1024
// threads with one LDS exchange per sum; columns in pieces of eight per
// thread at element alignment.  A row of fewer than 512 columns leaves lanes of
// its wave idle: 131072 x 256 in bf16 with a residual 70 us, its backward with dr
// 117, for 52 of bytes; 262144 x 128 117 and 205, 524288 x 64 215 and 389.
#include "gdn_device.h"
#include "gdn_launch.h"
#include "gdn_row.h"
#include "gdn_tile.h"

namespace gdn {

// A thread's eight columns.  In a row that is no multiple of eight the last ones
// begin that much earlier, over columns that another thread has too: both
// compute and store the same values there, with whole 16-byte accesses, and
// `dup` of them are left out of this thread's sums (8: the row ends before this
// piece, which only reads).  One by one, the last columns cost more than the rest
// of the row: 32800 x 1023 in bf16 70 against 50 us, the backward 99 against 55;
// 8194 x 4095 76 against 61 and 135 against 72 (rows that begin inside a
// 16-byte word; 8200 x 4092 takes 52 and 59).
struct Piece {
    int c, dup;
    __device__ __forceinline__ Piece(int c0, int D) : c(max(min(c0, D - 8), 0)), dup(min(c0 - c, 8)) {}
    __device__ __forceinline__ bool live() const { return dup < 8; }
    __device__ __forceinline__ bool whole(int D) const { return dup == 0 && c + 8 <= D; }
    __device__ __forceinline__ bool counts(int e, int D) const { return e >= dup && c + e < D; }
};

// Two sums over the TPR threads of a row in one exchange; sh holds TPR / 64
// pairs and is written once per call.
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2 *sh) {
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = make_float2(a, b);
        __syncthreads();
        a = b = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) {
            a += sh[i].x;
            b += sh[i].y;
        }
    }
    return make_float2(a, b);
}

template <class XT, class RT, class OT, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void ln_kernel(const XT *x, const RT *res, const float *w,
                                                                   const float *b, OT *y, RT *rout, float *mean,
                                                                   float *rstd, float *yscale, long rows, int D,
                                                                   float eps) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;  // rows per workgroup
    constexpr bool F8 = sizeof(OT) == 1;
    __shared__ float sh[2][TPR / 64 + 1];
    __shared__ float2 sh2[TPR / 64 + 1];
    const int tid = threadIdx.x % TPR;
    const long row = (long)blockIdx.x * RPB + threadIdx.x / TPR;
    if (row >= rows) return;  // whole waves leave, and only where a row is one wave
    const XT *xr = x + row * D;
    const auto piece = [&](int i) { return Piece((tid + i * TPR) * 8, D); };
    float u[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) load_piece(u[i], xr, piece(i).c, D);
    if (res) {
        const RT *rr = res + row * D;
        float t[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) load_piece(t[i], rr, piece(i).c, D);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) u[i][e] += t[i][e];
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const Piece p = piece(i);
        if (p.whole(D)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += u[i][e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += p.counts(e, D) ? u[i][e] : 0.f;
        }
    }
    // The mean's own rounding moves every difference alike: their sum says by
    // how much, and takes it out of the variance and of the differences.
    const float m = row_sum<TPR>(sum, sh[0]) / (float)D;
    if (res && rout) {  // may be res itself: every thread of the row has read by now (each has added to the sum)
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (piece(i).live()) store_piece(rout + row * D, u[i], piece(i).c, D);
    }
    float ss = 0.f, sd = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const Piece p = piece(i);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[i][e] -= m;
        if (F8 && D < 8) {
            // what lies past such a row takes part in its largest magnitude: zero, as -mean rstd may be beyond fp32
#pragma unroll
            for (int e = 0; e < 8; ++e) u[i][e] = e < D ? u[i][e] : 0.f;
        }
        if (p.whole(D)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss = fmaf(u[i][e], u[i][e], ss);
                sd += u[i][e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = p.counts(e, D) ? u[i][e] : 0.f;
                ss = fmaf(v, v, ss);
                sd += v;
            }
        }
    }
    const float2 both = row_sum2<TPR>(ss, sd, sh2);
    const float off = both.y / (float)D;
    const float var = fmaf(-off, off, both.x / (float)D);
    const float s = 1.f / sqrtf((var < 0.f ? 0.f : var) + eps);  // NaN stays
    if (tid == 0) {
        if (mean) mean[row] = m + off;
        if (rstd) rstd[row] = s;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float wv[8], bv[8];
        load_piece(wv, w, piece(i).c, D);
        if (b) load_piece(bv, b, piece(i).c, D);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            u[i][e] = (u[i][e] - off) * s;
            u[i][e] = b ? fmaf(u[i][e], wv[e], bv[e]) : u[i][e] * wv[e];
        }
    }
    if constexpr (F8) {
        // largest magnitude, compared as bits: an infinity or NaN in the row
        // wins, so such a row's scale and codes show it
        uint32_t am = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) am = max(am, __float_as_uint(u[i][e]) & 0x7fffffffu);
        am = row_max<TPR>(am, (uint32_t *)sh[1]);
        float scale = __uint_as_float(am) / 448.f;
        if (scale == 0.f) scale = 1.f;
        if (tid == 0) yscale[row] = scale;
        const QuantRow q(scale);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (piece(i).live()) store_piece_f8((uint8_t *)y + row * D, u[i], q, piece(i).c, D);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (piece(i).live()) store_piece(y + row * D, u[i], piece(i).c, D);
    }
}

constexpr int ln_bwd_waves(int dy_bytes, int TPR, int NV) {
    return NV == 2 && (dy_bytes == 2 || TPR == 64) ? 3 : 1;
}

// Backward.  A workgroup walks rows (its first row, then every RPB * grid rows
// on) and keeps the column sums of dy xhat and dy in registers; they leave as
// one row of 2 D partial sums per workgroup, which ln_colsum_kernel adds up in
// a fixed order (no atomics, so results repeat bit for bit).  The next row's
// loads are issued before this row's sums where the registers hold both
// (AHEAD).  32768 x 1024 in bf16 with dr 51 us, 5.2 TB/s of dy, r, dr and dx;
// 16384 x 5120 in fp32 197 us, 5.1; beyond 8192 columns the two sums a column
// crowd the registers: 4096 x 16384 in bf16 100 us, 4.0; beyond 16384 they do
// not fit, and 145 to 337 registers are spilled: 2048 x 32768 in bf16 with dr
// 318 us, 1.7, with fp32 rows 473, 2.0.
// Two pieces a thread are held to the registers of three waves a SIMD unit
// where that spills little: 43690 x 768 with a fp32 residual 93 us against 131
// at two waves, all in fp32 103 against 139; but 8192 x 4096 all in fp32, which
// spills into its walk, 112 against 104, and keeps two.
// ODD, a width that is no multiple of eight, leaves the columns that come twice
// out of the sums; the others are spared its registers.
template <class DT, class RT, int TPR, int NV, bool ODD>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR, ln_bwd_waves(sizeof(DT), TPR, NV)) void ln_bwd_kernel(
    const DT *dy, const RT *r, const float *w, const float *mean, const float *rstd, const RT *dr, RT *dx, float *part,
    long rows, int D) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    constexpr bool AHEAD = TPR < 1024 && !(NV == 4 && sizeof(RT) == 4);
    using DRaw = typename RawOf<DT>::type;
    using RRaw = typename RawOf<RT>::type;
    __shared__ float2 sh[2][TPR / 64 + 1];
    __shared__ float shw[RPB > 1 ? RPB * TPR * 8 : 1];
    const int tid = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const auto piece = [&](int i) { return Piece((tid + i * TPR) * 8, ODD ? D : 1 << 30); };
    f32x8 aw[NV], ab[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) aw[i] = ab[i] = f32x8{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    DRaw g0[NV];
    RRaw r0[NV], d0[NV];
    float m0 = 0.f, s0 = 0.f;
    auto load = [&](long row) {
        m0 = mean[row];
        s0 = rstd[row];
#pragma unroll
        for (int i = 0; i < NV; ++i) g0[i] = load_raw(dy + row * D, piece(i).c, D);
#pragma unroll
        for (int i = 0; i < NV; ++i) r0[i] = load_raw(r + row * D, piece(i).c, D);
        if (dr) {
#pragma unroll
            for (int i = 0; i < NV; ++i) d0[i] = load_raw(dr + row * D, piece(i).c, D);
        }
    };
    const long step = (long)gridDim.x * RPB;
    long row = (long)blockIdx.x * RPB + grp;
    if (AHEAD && row < rows) load(row);
    for (int turn = 0; row < rows; row += step, turn ^= 1) {
        if (!AHEAD) load(row);
        f32x8 g[NV], xh[NV];
        RRaw d1[NV];
        const float s = s0, m = m0;
        float dot = 0.f, sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Piece p = piece(i);
            const f32x8 wv = load8v(w, p.c, D);
            const float before = dot;
            g[i] = raw_f32(g0[i]);
            xh[i] = raw_f32(r0[i]);
            d1[i] = d0[i];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[i][e] = (xh[i][e] - m) * s;
                aw[i][e] = fmaf(g[i][e], xh[i][e], aw[i][e]);
                ab[i][e] += g[i][e];
                g[i][e] *= wv[e];
                if constexpr (!ODD) {  // past the row's end dy and w are zero
                    sum += g[i][e];
                    dot = fmaf(g[i][e], xh[i][e], dot);
                }
            }
            if constexpr (!ODD) {  // and xhat is -mean rstd there: beyond fp32 it gave NaN
                dot = p.c < D ? dot : before;
                continue;
            }
            if (p.whole(D)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    sum += g[i][e];
                    dot = fmaf(g[i][e], xh[i][e], dot);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = p.counts(e, D) ? g[i][e] : 0.f;
                    sum += v;
                    dot = p.counts(e, D) ? fmaf(v, xh[i][e], dot) : dot;
                }
            }
        }
        if (AHEAD && row + step < rows) load(row + step);
        // the two halves of sh alternate, so a fast wave of the next row does
        // not overwrite sums that a slow one still reads
        const float2 both = row_sum2<TPR>(dot, sum, sh[turn]);
        dot = both.x / (float)D;
        sum = both.y / (float)D;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            f32x8 v;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = s * (g[i][e] - sum - xh[i][e] * dot);
            if (dr) {
                const f32x8 d = raw_f32(d1[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += d[e];
            }
            if (piece(i).live()) store8v(dx + row * D, v, piece(i).c, D);
        }
    }
    if (!part) return;
    float *pr = part + (long)blockIdx.x * 2 * D;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x8(&acc)[NV] = h ? ab : aw;
        if constexpr (RPB > 1) {  // add the workgroup's rows of sums, in order
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < 8; ++e) shw[(grp * 8 + e) * TPR + tid] = acc[i][e];
                __syncthreads();
                if (grp == 0) {
                    f32x8 v;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[e] = 0.f;
#pragma unroll
                        for (int p = 0; p < RPB; ++p) v[e] += shw[(p * 8 + e) * TPR + tid];
                    }
                    if (piece(i).live()) store8v(pr + h * D, v, piece(i).c, D);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (piece(i).live()) store8v(pr + h * D, acc[i], piece(i).c, D);
        }
    }
}

// dw[c], db[c] (nullable) = sums over n rows of part [n, 2 D]: 32 columns and
// 32 row strides per workgroup, so that the loads of a column are in flight
// together.
__global__ __launch_bounds__(1024) void ln_colsum_kernel(const float *part, float *dw, float *db, int n, int D) {
    __shared__ float sh[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int groups = (D + 31) / 32, h = blockIdx.x >= (unsigned)groups;
    float *out = h ? db : dw;
    if (!out) return;
    const int c = ((int)blockIdx.x - h * groups) * 32 + tx;
    float v = 0.f;
    if (c < D) {
        const float *p = part + h * D + c;
#pragma unroll 8
        for (int i = ty; i < n; i += 32) v += p[(long)i * 2 * D];
    }
    sh[ty][tx] = v;
    __syncthreads();
    if (ty == 0 && c < D) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += sh[i][tx];
        out[c] = s;
    }
}

template <class XT, class RT, class OT>
static hipError_t launch_ln_t(const void *x, const void *res, const float *w, const float *b, void *y, void *rout,
                              float *mean, float *rstd, float *yscale, long rows, int D, float eps, hipStream_t st) {
    // a launch holds fewer than 2^32 threads: more rows than 2^21 workgroups
    // take go in several launches
#define GDN_LN(TPRv, NVv)                                                                                       \
    if (D <= TPRv * NVv * 8) {                                                                                  \
        constexpr int rpb = TPRv < 256 ? 256 / TPRv : 1;                                                        \
        constexpr long most = (long)rpb << 21;                                                                  \
        for (long r0 = 0; r0 < rows; r0 += most) {                                                              \
            const long n = rows - r0 < most ? rows - r0 : most;                                                 \
            hipLaunchKernelGGL((ln_kernel<XT, RT, OT, TPRv, NVv>), dim3((unsigned)((n + rpb - 1) / rpb)),       \
                               dim3(TPRv < 256 ? 256 : TPRv), 0, st, (const XT *)x + r0 * D,                    \
                               res ? (const RT *)res + r0 * D : nullptr, w, b, (OT *)y + r0 * D,                \
                               rout ? (RT *)rout + r0 * D : nullptr, mean ? mean + r0 : nullptr,                \
                               rstd ? rstd + r0 : nullptr, yscale ? yscale + r0 : nullptr, n, D, eps);          \
            const hipError_t e = hipGetLastError();                                                             \
            if (e != hipSuccess) return e;                                                                      \
        }                                                                                                       \
        return hipSuccess;                                                                                      \
    }
    GDN_LN(64, 1)
    GDN_LN(64, 2)
    GDN_LN(64, 4)
    GDN_LN(256, 2)
    GDN_LN(256, 4)
    GDN_LN(512, 4)
    GDN_LN(1024, 4)
#undef GDN_LN
    return hipErrorInvalidValue;
}

hipError_t launch_add_layernorm(const void *x, const void *res, const float *w, const float *b, void *y, void *rout,
                                float *mean, float *rstd, float *yscale, long rows, int D, bool x_bf16, bool r_bf16,
                                bool f8, float eps, hipStream_t st) {
#define GDN_LN_T(XT, RT, OT) launch_ln_t<XT, RT, OT>(x, res, w, b, y, rout, mean, rstd, yscale, rows, D, eps, st)
    if (x_bf16 && r_bf16) return f8 ? GDN_LN_T(uint16_t, uint16_t, uint8_t) : GDN_LN_T(uint16_t, uint16_t, uint16_t);
    if (x_bf16) return f8 ? GDN_LN_T(uint16_t, float, uint8_t) : GDN_LN_T(uint16_t, float, uint16_t);
    if (!r_bf16) return f8 ? GDN_LN_T(float, float, uint8_t) : GDN_LN_T(float, float, float);
#undef GDN_LN_T
    return hipErrorInvalidValue;
}

// Workgroups of the backward: enough to fill the card, few enough that their
// partial sums (8 bytes a column and workgroup, written and read) stay small
// beside the rows.  Measured at 128 to 1024 of them: 32768 x 256 in bf16 1024
// best (30 us, 768 32, 512 42), 32768 x 1024 768 (51 us, 384 58, 1024 62),
// 16384 x 5120 in fp32 512 (197 us, 256 244, 768 228), 4096 x 4096 in bf16 512
// (33 us, 1024 42), 4096 x 8192 256 (45 us, 128 62, 512 53), 4096 x 16384 256
// (100 us, 512 112).  Not swept below 4096 rows, where a workgroup has a few
// rows and the partial sums weigh: 3294 x 1080 takes 14.7 + 4.1 us for 4.2 of
// the rows' bytes, 13 MB of sums beside 21 MB.
int ln_bwd_blocks(long rows, int D) {
    const long groups = D <= 1024 ? (rows + 3) / 4 : rows;
    const long most = D <= 512 ? 1024 : D <= 2048 ? 768 : D <= 6144 ? 512 : 256;
    return (int)(groups < most ? groups : most);
}

template <class DT, class RT>
static hipError_t launch_ln_bwd_t(const void *dy, const void *r, const float *w, const float *mean, const float *rstd,
                                  const void *dr, void *dx, float *dw, float *db, float *part, long rows, int D,
                                  hipStream_t st) {
    const int nb = ln_bwd_blocks(rows, D);
    float *pp = dw || db ? part : nullptr;
#define GDN_LNB(MOST, TPRv, NVv)                                                                                      \
    if (D <= MOST) {                                                                                                  \
        const auto k = D % 8 ? ln_bwd_kernel<DT, RT, TPRv, NVv, true> : ln_bwd_kernel<DT, RT, TPRv, NVv, false>;      \
        hipLaunchKernelGGL(k, dim3((unsigned)nb), dim3(TPRv < 256 ? 256 : TPRv), 0, st, (const DT *)dy,               \
                           (const RT *)r, w, mean, rstd, (const RT *)dr, (RT *)dx, pp, rows, D);                      \
    } else
    GDN_LNB(512, 64, 1)
    GDN_LNB(1024, 64, 2)
    GDN_LNB(2048, 256, 1)
    GDN_LNB(4096, 256, 2)
    GDN_LNB(6144, 256, 3)
    GDN_LNB(8192, 512, 2)
    GDN_LNB(16384, 512, 4)
    GDN_LNB(kMaxNormCols, 1024, 4) return hipErrorInvalidValue;
#undef GDN_LNB
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || !pp) return err;
    const int groups = (D + 31) / 32;
    hipLaunchKernelGGL(ln_colsum_kernel, dim3((unsigned)(db ? 2 * groups : groups)), dim3(1024), 0, st, part, dw, db,
                       nb, D);
    return hipGetLastError();
}

hipError_t launch_add_layernorm_bwd(const void *dy, const void *r, const float *w, const float *mean,
                                    const float *rstd, const void *dr, void *dx, float *dw, float *db, float *part,
                                    long rows, int D, bool dy_bf16, bool r_bf16, hipStream_t st) {
    if (dy_bf16 && r_bf16)
        return launch_ln_bwd_t<uint16_t, uint16_t>(dy, r, w, mean, rstd, dr, dx, dw, db, part, rows, D, st);
    if (dy_bf16) return launch_ln_bwd_t<uint16_t, float>(dy, r, w, mean, rstd, dr, dx, dw, db, part, rows, D, st);
    if (!r_bf16) return launch_ln_bwd_t<float, float>(dy, r, w, mean, rstd, dr, dx, dw, db, part, rows, D, st);
    return hipErrorInvalidValue;
}

}  // namespace gdn
