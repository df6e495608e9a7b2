// gdn_norm.hip -- the block's entry: residual addition and RMS norm in one
// pass (with an output in the input's type or in e4m3 with one scale per
// row), its backward, and the row quantiser.
//   forward   u = x + residual;  r = u in the residual's type
//             s = (mean(u^2) + eps)^-1/2;  y = u s w
//   8 bits    scale = max|y| / 448,  q = e4m3(y / scale)
//   backward  xhat = r s;  dx = s (w dy - xhat mean(w dy xhat)) + dr
//             dw = sum over rows of dy xhat
// Everything is fp32 between the loads and one rounding at the stores; the
// norm is taken of the unrounded sum u, so y does not depend on the type the
// residual stream is kept in.  The kernels are bound by HBM: a row is read
// once, held in registers while its sums are formed, and written once.  A row
// belongs to one wave up to 2048 columns in the forward and 1024 in the
// backward (four rows per workgroup, sums on DPP with no LDS), beyond that to
// 256, 512 or 1024 threads with one LDS exchange per sum.  Columns go in
// pieces of eight per lane; rows of a width that is no multiple of eight start
// at any element, so the 16-byte accesses are declared with element alignment
// (the hardware takes them at any address) and the row's last few columns go
// one by one.
#include "gdn_device.h"
#include "gdn_launch.h"
#include "gdn_row.h"
#include "gdn_tile.h"

namespace gdn {

// Threads per row and pieces of eight columns per thread for rows of D.
struct RowPlan {
    int tpr, nv;
};

template <class XT, class RT, class OT, bool NORM, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_kernel(const XT *x, const RT *res, const float *w,
                                                                     OT *y, RT *rout, float *rstd, float *yscale,
                                                                     long rows, int D, float eps) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;  // rows per workgroup
    constexpr bool F8 = sizeof(OT) == 1;
    __shared__ float sh[2][TPR / 64 + 1];
    const int tid = threadIdx.x % TPR;
    const long row = (long)blockIdx.x * RPB + threadIdx.x / TPR;
    if (row >= rows) return;  // whole waves leave, and only where a row is one wave
    const XT *xr = x + row * D;
    float u[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) load_piece(u[i], xr, (tid + i * TPR) * 8, D);
    if (NORM && res) {
        const RT *rr = res + row * D;
        float t[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) load_piece(t[i], rr, (tid + i * TPR) * 8, D);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) u[i][e] += t[i][e];
        if (rout)  // may be res itself: this thread has read what it replaces
#pragma unroll
            for (int i = 0; i < NV; ++i) store_piece(rout + row * D, u[i], (tid + i * TPR) * 8, D);
    }
    if (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(u[i][e], u[i][e], ss);
        ss = row_sum<TPR>(ss, sh[0]);
        const float s = 1.f / sqrtf(ss / (float)D + eps);
        if (rstd && tid == 0) rstd[row] = s;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float wv[8];
            load_piece(wv, w, (tid + i * TPR) * 8, D);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[i][e] = u[i][e] * s * wv[e];
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
        float scale = __uint_as_float(am) * (1.f / 448.f);
        if (scale == 0.f) scale = 1.f;
        if (yscale && tid == 0) yscale[row] = scale;
        const QuantRow q(scale);
#pragma unroll
        for (int i = 0; i < NV; ++i) store_piece_f8((uint8_t *)y + row * D, u[i], q, (tid + i * TPR) * 8, D);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) store_piece(y + row * D, u[i], (tid + i * TPR) * 8, D);
    }
}

// Backward.  A workgroup walks rows (its first row, then every RPB * grid
// rows on) and keeps the column sums of dy xhat in registers; they leave as
// one row of partial sums per workgroup, which colsum_kernel adds up in a
// fixed order (no atomics, so results repeat bit for bit).  A row takes as long
// as its loads, its sum and its stores one after the other, so the next row's
// loads are issued before this row's sum (AHEAD; not at 1024 threads, whose
// registers do not hold two rows): 32768 x 1024 in bf16 43.1 -> 39.6 us, 5.1
// TB/s.  Up to 8192 columns nothing spills and the loads bound it (4.8 to 5.3
// TB/s of dy, r and dx from 32 million elements on).  Beyond, registers spill
// to scratch memory with an fp32 r (80 and 140 bytes a thread), beyond 16384
// columns with any (128 to 232), and the rate falls: 4096 x 16384 86 us in bf16
// (4.7 TB/s), 180 with an fp32 r, 237 in fp32 (3.4); 4096 x 32768 247, 380
// and 409 us (3.3, 3.5 and 3.9 TB/s).
template <class DT, class RT, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_bwd_kernel(const DT *dy, const RT *r, const float *w,
                                                                         const float *rstd, const RT *dr, RT *dx,
                                                                         float *part, long rows, int D) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    constexpr bool AHEAD = TPR < 1024;
    using DRaw = typename RawOf<DT>::type;
    using RRaw = typename RawOf<RT>::type;
    __shared__ float sh[2][TPR / 64 + 1];
    __shared__ float shw[RPB > 1 ? RPB * TPR * 8 : 1];
    const int tid = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    f32x8 acc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] = f32x8{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    DRaw g0[NV];
    RRaw r0[NV], d0[NV];
    float s0 = 0.f;
    auto load = [&](long row) {
        s0 = rstd[row];
#pragma unroll
        for (int i = 0; i < NV; ++i) g0[i] = load_raw(dy + row * D, (tid + i * TPR) * 8, D);
#pragma unroll
        for (int i = 0; i < NV; ++i) r0[i] = load_raw(r + row * D, (tid + i * TPR) * 8, D);
        if (dr) {
#pragma unroll
            for (int i = 0; i < NV; ++i) d0[i] = load_raw(dr + row * D, (tid + i * TPR) * 8, D);
        }
    };
    const long step = (long)gridDim.x * RPB;
    long row = (long)blockIdx.x * RPB + grp;
    if (AHEAD && row < rows) load(row);
    for (int turn = 0; row < rows; row += step, turn ^= 1) {
        if (!AHEAD) load(row);
        f32x8 g[NV], xh[NV];
        RRaw d1[NV];
        const float s = s0;
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const f32x8 wv = load8v(w, (tid + i * TPR) * 8, D);
            g[i] = raw_f32(g0[i]);
            xh[i] = raw_f32(r0[i]);
            d1[i] = d0[i];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[i][e] *= s;
                acc[i][e] = fmaf(g[i][e], xh[i][e], acc[i][e]);
                g[i][e] *= wv[e];
                dot = fmaf(g[i][e], xh[i][e], dot);
            }
        }
        if (AHEAD && row + step < rows) load(row + step);
        // the two halves of sh alternate, so a fast wave of the next row does
        // not overwrite sums that a slow one still reads
        dot = row_sum<TPR>(dot, sh[turn]) / (float)D;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            f32x8 v;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = s * (g[i][e] - xh[i][e] * dot);
            if (dr) {
                const f32x8 d = raw_f32(d1[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += d[e];
            }
            store8v(dx + row * D, v, (tid + i * TPR) * 8, D);
        }
    }
    if (!part) return;
    float *pr = part + (long)blockIdx.x * D;
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
                store8v(pr, v, (tid + i * TPR) * 8, D);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) store8v(pr, acc[i], (tid + i * TPR) * 8, D);
    }
}

// out[c] = sum over n rows of part[.][c]: 32 columns and 32 row strides per
// workgroup, so that the loads of a column are in flight together.
__global__ __launch_bounds__(1024) void colsum_kernel(const float *part, float *out, int n, int D) {
    __shared__ float sh[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + tx;
    float v = 0.f;
    if (c < D) {
#pragma unroll 8
        for (int i = ty; i < n; i += 32) v += part[(long)i * D + c];
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

hipError_t launch_colsum(const float *part, float *out, int n, int D, hipStream_t st) {
    hipLaunchKernelGGL(colsum_kernel, dim3((unsigned)((D + 31) / 32)), dim3(1024), 0, st, part, out, n, D);
    return hipGetLastError();
}

template <class XT, class RT, class OT, bool NORM>
static hipError_t launch_norm_t(const void *x, const void *res, const float *w, void *y, void *rout, float *rstd,
                                float *yscale, long rows, int D, float eps, hipStream_t st) {
    // a launch holds fewer than 2^32 threads: more rows than 2^21 workgroups
    // take go in several launches
#define GDN_NORM(TPRv, NVv)                                                                                        \
    if (D <= TPRv * NVv * 8) {                                                                                     \
        constexpr int rpb = TPRv < 256 ? 256 / TPRv : 1;                                                           \
        constexpr long most = (long)rpb << 21;                                                                     \
        for (long r0 = 0; r0 < rows; r0 += most) {                                                                 \
            const long n = rows - r0 < most ? rows - r0 : most;                                                    \
            hipLaunchKernelGGL((norm_kernel<XT, RT, OT, NORM, TPRv, NVv>), dim3((unsigned)((n + rpb - 1) / rpb)),  \
                               dim3(TPRv < 256 ? 256 : TPRv), 0, st, (const XT *)x + r0 * D,                       \
                               res ? (const RT *)res + r0 * D : nullptr, w, (OT *)y + r0 * D,                      \
                               rout ? (RT *)rout + r0 * D : nullptr, rstd ? rstd + r0 : nullptr,                   \
                               yscale ? yscale + r0 : nullptr, n, D, eps);                                         \
            const hipError_t e = hipGetLastError();                                                                \
            if (e != hipSuccess) return e;                                                                         \
        }                                                                                                          \
        return hipSuccess;                                                                                         \
    }
    GDN_NORM(64, 1)
    GDN_NORM(64, 2)
    GDN_NORM(64, 4)
    GDN_NORM(256, 2)
    GDN_NORM(256, 4)
    GDN_NORM(512, 4)
    GDN_NORM(1024, 4)
#undef GDN_NORM
    return hipErrorInvalidValue;
}

hipError_t launch_add_rmsnorm(const void *x, const void *res, const float *w, void *y, void *rout, float *rstd,
                              float *yscale, long rows, int D, bool x_bf16, bool r_bf16, bool f8, float eps,
                              hipStream_t st) {
    if (x_bf16 && r_bf16)
        return f8 ? launch_norm_t<uint16_t, uint16_t, uint8_t, true>(x, res, w, y, rout, rstd, yscale, rows, D, eps, st)
                  : launch_norm_t<uint16_t, uint16_t, uint16_t, true>(x, res, w, y, rout, rstd, yscale, rows, D, eps, st);
    if (x_bf16)
        return f8 ? launch_norm_t<uint16_t, float, uint8_t, true>(x, res, w, y, rout, rstd, yscale, rows, D, eps, st)
                  : launch_norm_t<uint16_t, float, uint16_t, true>(x, res, w, y, rout, rstd, yscale, rows, D, eps, st);
    if (!r_bf16)
        return f8 ? launch_norm_t<float, float, uint8_t, true>(x, res, w, y, rout, rstd, yscale, rows, D, eps, st)
                  : launch_norm_t<float, float, float, true>(x, res, w, y, rout, rstd, yscale, rows, D, eps, st);
    return hipErrorInvalidValue;
}

hipError_t launch_quantize_rows(const void *x, void *q, float *scale, long rows, int D, bool bf16, hipStream_t st) {
    return bf16 ? launch_norm_t<uint16_t, uint16_t, uint8_t, false>(x, nullptr, nullptr, q, nullptr, nullptr, scale,
                                                                    rows, D, 0.f, st)
                : launch_norm_t<float, float, uint8_t, false>(x, nullptr, nullptr, q, nullptr, nullptr, scale, rows, D,
                                                              0.f, st);
}

static RowPlan bwd_plan(int D) {
    if (D <= 512) return {64, 1};
    if (D <= 1024) return {64, 2};
    if (D <= 2048) return {256, 1};
    if (D <= 4096) return {256, 2};
    if (D <= 6144) return {256, 3};  // fewer lanes past the row's end: 16384 x 5120 in fp32 189 against 214 us
    if (D <= 8192) return {512, 2};
    if (D <= 16384) return {512, 4};
    return {1024, 4};
}

// Workgroups of the backward: enough to fill the card, few enough that their
// partial sums stay small beside the rows.  Measured best counts over 64 to
// 2048: 768 of four waves with a row each (32768 x 1024 in bf16: 39.6 us; 256
// 50, 2048 46), 512, two per compute unit, up to 6144 columns (4096 x 4096
// 22 us; 16384 x 5120 in fp32 189 us, 640 255, 260 292); beyond that one per
// compute unit, two once there are rows for 16 each (5000 x 8000 in bf16 55
// against 66 us, 16384 x 8192 151 against 148, fp32 106 against 103).
int norm_bwd_blocks(long rows, int D) {
    const RowPlan p = bwd_plan(D);
    const int rpb = p.tpr < 256 ? 256 / p.tpr : 1;
    const long groups = (rows + rpb - 1) / rpb;
    const long wide = D <= 8192 && rows >= 4096 ? 512 : 256;
    const long most = D <= 512 ? 1024 : D <= 2048 ? 768 : D <= 6144 ? 512 : wide;
    return (int)(groups < most ? groups : most);
}

template <class DT, class RT>
static hipError_t launch_norm_bwd_t(const void *dy, const void *r, const float *w, const float *rstd, const void *dr,
                                    void *dx, float *dw, float *part, long rows, int D, hipStream_t st) {
    const RowPlan p = bwd_plan(D);
    const int nb = norm_bwd_blocks(rows, D);
    hipError_t err = hipErrorInvalidValue;
#define GDN_NORMB(TPRv, NVv)                                                                                         \
    if (p.tpr == TPRv && p.nv == NVv) {                                                                              \
        hipLaunchKernelGGL((norm_bwd_kernel<DT, RT, TPRv, NVv>), dim3((unsigned)nb), dim3(TPRv < 256 ? 256 : TPRv), 0, \
                           st, (const DT *)dy, (const RT *)r, w, rstd, (const RT *)dr, (RT *)dx,                     \
                           dw ? part : nullptr, rows, D);                                                            \
        err = hipGetLastError();                                                                                     \
    }
    GDN_NORMB(64, 1)
    GDN_NORMB(64, 2)
    GDN_NORMB(256, 1)
    GDN_NORMB(256, 2)
    GDN_NORMB(256, 3)
    GDN_NORMB(512, 2)
    GDN_NORMB(512, 4)
    GDN_NORMB(1024, 4)
#undef GDN_NORMB
    if (err != hipSuccess || !dw) return err;
    return launch_colsum(part, dw, nb, D, st);
}

hipError_t launch_add_rmsnorm_bwd(const void *dy, const void *r, const float *w, const float *rstd, const void *dr,
                                  void *dx, float *dw, float *part, long rows, int D, bool dy_bf16, bool r_bf16,
                                  hipStream_t st) {
    if (dy_bf16 && r_bf16)
        return launch_norm_bwd_t<uint16_t, uint16_t>(dy, r, w, rstd, dr, dx, dw, part, rows, D, st);
    if (dy_bf16) return launch_norm_bwd_t<uint16_t, float>(dy, r, w, rstd, dr, dx, dw, part, rows, D, st);
    if (!r_bf16) return launch_norm_bwd_t<float, float>(dy, r, w, rstd, dr, dx, dw, part, rows, D, st);
    return hipErrorInvalidValue;
}

}  // namespace gdn
