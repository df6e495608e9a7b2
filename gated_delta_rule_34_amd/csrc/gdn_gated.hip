// gdn_gated.hip -- the gated feed-forward projection,
//   (g, u) = (x W^T) x_scale w_scale + bias,   y = act(g) u
// with the N gate rows of W before its N up rows, in one product whose tiles
// hold the gate's and the up columns side by side, so that g and u meet in
// registers and leave for memory only where the backward asks for them; and
// the backward of the bf16 form,
//   dg = dy u act'(g),  du = dy act(g),  dx = (dg du) W,  dW = (dg du)^T x.
// A tile's 256 (128) rows of W are sixteen gate rows and their sixteen up rows
// in turn, read by way of two base addresses (a wave's loads are all of one
// kind), so the products' kernel and its speed are those of a plain product of
// 2 N columns.  Few rows take eight gate and eight up rows to a fragment.
// 32768 x 4096 x 1024 (550 GFLOP) with SiLU 484 us, 1136 TFLOP/s, with both
// arguments kept 537 (their 537 MB take 104 us at the rate of a copy); 16384 x 4096
// x 4096 819 us, 1342; in e4m3 32768 x 4096 x 1024 324 us, 1700.  The epilogue
// (an exponential, a reciprocal and the exchange between lanes for each
// output) is what the matrix units wait for with short K: 5 us a tile of 25;
// starting the workgroups apart in time did not hide it (489 to 497 us).
// 1 x 8192 x 8192: 48 us, 5.5 TB/s of weights; 1 x 4096 x 1024 3.6 us in a graph.
#include "gdn_device.h"
#include "gdn_launch.h"
#include "gdn_mm.h"
#include "gdn_mm_kernel.h"
#include "gdn_row.h"
#include "gdn_tile.h"

namespace gdn {

// Adds the partial sums [split, I, 2 J] of the splits in order and applies the epilogue.
__global__ __launch_bounds__(256) void gated_join_kernel(const float *part, GatedEpilogue ep, int splits, int I, int J) {
    const int pieces = (J + 7) / 8;
    const long n = (long)I * pieces;
    for (long t = (long)blockIdx.x * 256 + threadIdx.x; t < n; t += (long)gridDim.x * 256) {
        const long i = t / pieces;
        const int j = (int)(t - i * pieces) * 8;
        f32x8 g = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, u = g;
        for (int s = 0; s < splits; ++s) {
            const float *p = part + ((long)s * I + i) * 2 * J;
            const f32x8 a = load8v(p, j, J), b = load8v(p + J, j, J);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                g[e] += a[e];
                u[e] += b[e];
            }
        }
        ep.any(g, u, i, j, J);
    }
}

// act(g) and act'(g) together.
__device__ __forceinline__ void act_both(int act, float g, float &f, float &df) {
    switch (act) {
        case ACT_RELU:
            f = g < 0.f ? 0.f : g;
            df = g > 0.f ? 1.f : 0.f;
            return;
        case ACT_SILU: {
            const float p = sigmoid_fast(g);
            f = g * p;
            df = p * (1.f + g * (1.f - p));
            return;
        }
        case ACT_GELU: {
            float e;
            const float c = normal_cdf<true>(g, e);
            f = g * c;
            df = c + g * e * 0.3989422804014327f;
            return;
        }
    }
    f = g;
    df = 1.f;
}

// (dg, du) in `planes` bf16 planes (rounded; what is left of it; what is left
// of that) of Jp columns: dg at 0, du at J, zero from 2 J to Jp; and the column
// sums [block, 2 J] of the unrounded values over this workgroup's rows.
// One plane for bf16 gradients and three for fp32 ones, for the reasons of
// the plain projection's dz.  Bound by HBM: 16384 x 4096 with SiLU 130 us, 5.2
// TB/s of dy, g, u, dg and du.  With RELU dg is chosen, not multiplied: zero
// where g <= 0, whatever dy and u hold there.
template <class DT>
__global__ __launch_bounds__(256) void gated_dz_kernel(const DT *dy, const uint16_t *z, uint16_t *out, long plane,
                                                       int planes, float *part, int I, int J, int Jp, int act,
                                                       int rows) {
    __shared__ float sh[4][64][8];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int j = (blockIdx.x * 64 + lane) * 8;
    const int i0 = blockIdx.y * rows, i1 = min(i0 + rows, I);
    constexpr int AT = 4;  // rows requested together
    f32x8 sg = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, su = sg;
    const bool full = j + 8 <= J;
    if (j < J) {
        for (int i = i0 + wave; i < i1; i += 4 * AT) {
            typename RawOf<DT>::type rd[AT];
            Raw16 rg[AT], ru[AT];
#pragma unroll
            for (int q = 0; q < AT; ++q) {
                const long row = min(i + 4 * q, i1 - 1);
                rd[q] = load_raw(dy + row * J, j, J);
                rg[q] = load_raw(z + row * 2 * J, j, J);
                ru[q] = load_raw(z + row * 2 * J + J, j, J);
            }
#pragma unroll
            for (int q = 0; q < AT; ++q) {
                if (i + 4 * q >= i1) break;
                const f32x8 d = raw_f32(rd[q]), g = raw_f32(rg[q]), u = raw_f32(ru[q]);
                f32x8 dg, du;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float f, df;
                    act_both(act, g[e], f, df);
                    dg[e] = d[e] * u[e] * df;
                    if (act == ACT_RELU && !(g[e] > 0.f)) dg[e] = 0.f;
                    du[e] = d[e] * f;
                    sg[e] += dg[e];
                    su[e] += du[e];
                }
                if (out) {
                    uint16_t *o = out + (long)(i + 4 * q) * Jp;
                    for (int p = 0; p < planes; ++p, o += plane) {
                        u32x4 a, b;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            a[e] = pack2_bf16(dg[2 * e], dg[2 * e + 1]);
                            b[e] = pack2_bf16(du[2 * e], du[2 * e + 1]);
                            dg[2 * e] = rest(dg[2 * e], __uint_as_float(a[e] << 16));
                            dg[2 * e + 1] = rest(dg[2 * e + 1], __uint_as_float(a[e] & 0xffff0000u));
                            du[2 * e] = rest(du[2 * e], __uint_as_float(b[e] << 16));
                            du[2 * e + 1] = rest(du[2 * e + 1], __uint_as_float(b[e] & 0xffff0000u));
                        }
                        if (full) {
                            *(u32x4 *)(o + j) = a;
                            *(u32x4_a2 *)(o + J + j) = b;
                        } else {  // the last columns of each, one by one
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (j + e < J) {
                                    o[j + e] = (uint16_t)(a[e >> 1] >> (16 * (e & 1)));
                                    o[J + j + e] = (uint16_t)(b[e >> 1] >> (16 * (e & 1)));
                                }
                        }
                        if (j + 8 >= J)
                            for (int c = 2 * J; c < Jp; ++c) o[c] = 0;
                    }
                }
            }
        }
    }
    if (!part) return;
    float *pr = part + (long)blockIdx.y * 2 * J;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x8 &s = h ? su : sg;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) sh[wave][lane][e] = s[e];
        __syncthreads();
        if (wave == 0 && j < J) {
            f32x8 v;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = ((sh[0][lane][e] + sh[1][lane][e]) + sh[2][lane][e]) + sh[3][lane][e];
            store8v(pr + h * (long)J, v, j, J);
        }
    }
}

// ---- host side ----------------------------------------------------------------

template <int MODE>
static hipError_t gated_run(MmArgs a, const MmPlan &p, const GatedEpilogue &ep, float *part, hipStream_t st) {
    mm_set(a, p, MODE != MM_BF16);
    a.tj = (a.J + p.tile / 2 - 1) / (p.tile / 2);
    const dim3 grid((unsigned)(a.ti * a.tj), (unsigned)p.splits);
    float *pp = p.splits > 1 ? part : nullptr;
    if (p.tile == 256)
        hipLaunchKernelGGL((mm_kernel<256, 256, 4, 2, 2, false, false, MODE, GatedEpilogue>), grid, dim3(512), 0, st, a,
                           ep, pp);
    else if (p.deep)
        hipLaunchKernelGGL((mm_kernel<128, 128, 2, 2, 4, false, false, MODE, GatedEpilogue>), grid, dim3(256), 0, st, a,
                           ep, pp);
    else
        hipLaunchKernelGGL((mm_kernel<128, 128, 2, 2, 2, false, false, MODE, GatedEpilogue>), grid, dim3(256), 0, st, a,
                           ep, pp);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    const long pieces = (long)a.I * ((a.J + 7) / 8), blocks = (pieces + 255) / 256;
    hipLaunchKernelGGL(gated_join_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, part, ep,
                       p.splits, a.I, a.J);
    return hipGetLastError();
}

hipError_t launch_gated_linear(const MmPlan &p, const void *x, const void *w, const float *xs, const float *ws,
                               const float *bias, void *y, void *z, int M, int N, int K, bool f8, bool y_f32, int act,
                               float *part, hipStream_t st) {
    const long row = (long)K * (f8 ? 1 : 2);
    const GatedEpilogue ep{xs, ws, bias, y, (uint16_t *)z, N, act, y_f32, past_caches(M, N, y_f32)};
    if (p.tile == 0)
        return f8 ? mv_run<true>(x, w, M, 2 * N, K, ep, st) : mv_run<false>(x, w, M, 2 * N, K, ep, st);
    MmArgs a{};
    a.V = (const char *)x; a.U = (const char *)w;
    a.ldv = a.ldu = row;
    a.I = M; a.J = N; a.K = K; a.parts = 1;
    a.pair = (long)N * row;
    if (!f8) return gated_run<MM_BF16>(a, p, ep, part, st);
    return y_f32 ? gated_run<MM_F8_F32>(a, p, ep, part, st) : gated_run<MM_F8>(a, p, ep, part, st);
}

LinearBwdPlan gated_linear_bwd_plan(int M, int N, int K, bool grad_f32, bool dx, bool dw, bool dbias) {
    // (dg, du) is computed, never dy itself: planned like an activation that changes every value
    return linear_bwd_plan(M, 2 * N, K, true, grad_f32, ACT_SILU, dx, dw, dbias);
}

hipError_t launch_gated_linear_bwd(const LinearBwdPlan &p, const void *dy, const void *x, const void *w, const void *z,
                                   void *dx, void *dw, float *dbias, int M, int N, int K, bool dy_f32, bool grad_f32,
                                   int act, char *ws, hipStream_t st) {
    const int rows = dz_rows(M, 2 * N);
    const dim3 grid((unsigned)((N + 511) / 512), (unsigned)p.blocks);
    uint16_t *out = p.copy ? (uint16_t *)ws : nullptr;
    float *sums = dbias ? (float *)(ws + p.sums_off) : nullptr;
    if (dy_f32)
        hipLaunchKernelGGL((gated_dz_kernel<float>), grid, dim3(256), 0, st, (const float *)dy, (const uint16_t *)z, out,
                           (long)(p.plane / 2), p.planes, sums, M, N, p.Np, act, rows);
    else
        hipLaunchKernelGGL((gated_dz_kernel<uint16_t>), grid, dim3(256), 0, st, (const uint16_t *)dy,
                           (const uint16_t *)z, out, (long)(p.plane / 2), p.planes, sums, M, N, p.Np, act, rows);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return launch_linear_grads(p, ws, x, w, dx, dw, dbias, M, 2 * N, K, grad_f32, ws, st);
}

}  // namespace gdn
