// gdn_linear.hip -- the layer's matrix products with their epilogue,
//   z = (x W^T) x_scale w_scale + bias,   y = act(z) + residual
// and the backward of the bf16 form,
//   dz = dy act'(z),  dx = dz W,  dW = dz^T x,  dbias = sum over rows of dz.
// Products of bf16 values are exact and summed in fp32 by the MFMA; those of
// e4m3 values lose bits on the way to bf16 outputs (see MM_F8).  Everything
// after the sum is fp32 with one rounding per output.
// Measured at 8192^3: bf16 1430 TFLOP/s, its gradients 1465 (dx) and 1505
// (dw), e4m3 2945 (1500 for fp32 outputs).
#include "gdn_device.h"
#include "gdn_launch.h"
#include "gdn_mm.h"
#include "gdn_mm_kernel.h"
#include "gdn_row.h"
#include "gdn_tile.h"

namespace gdn {

// dbias from n rows of partial column sums [n, J], 32 columns a workgroup.
struct ColSums {
    const float *sums;
    float *out;
    int n, J;
};

__device__ __forceinline__ void colsum_body(char *smem, const ColSums &c, int group) {
    float(*sh)[33] = (float(*)[33])smem;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, j = group * 32 + tx;
    float v = 0.f;
    if (j < c.J) {
#pragma unroll 8
        for (int i = ty; i < c.n; i += 8) v += c.sums[(long)i * c.J + j];
    }
    sh[ty][tx] = v;
    __syncthreads();
    if (ty == 0 && j < c.J) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sh[i][tx];
        c.out[j] = s;
    }
}

// Both products of the backward in one launch, where they fit the card
// together: workgroups 0 .. na - 1 are dx's tiles and splits, the next nb dw's,
// those after them add up dbias.
template <int NBUF>
__global__ __launch_bounds__(256) void mm_pair_kernel(MmArgs a, Epilogue ea, float *pa, int na, MmArgs b, Epilogue eb,
                                                      float *pb, int nb, ColSums c) {
    __shared__ __attribute__((aligned(1024))) char smem[mm_lds<128, 128, 2, 2, NBUF>()];
    const int g = blockIdx.x, ta = a.ti * a.tj, tb = b.ti * b.tj;
    if (g >= na + nb) colsum_body(smem, c, g - na - nb);
    else if (g < na) mm_body<128, 128, 2, 2, NBUF, false, true, MM_BF16>(smem, a, ea, pa, g % ta, g / ta);
    else mm_body<128, 128, 2, 2, NBUF, true, true, MM_BF16>(smem, b, eb, pb, (g - na) % tb, (g - na) / tb);
}

// Adds the partial sums of the splits in order and applies the epilogue.
__global__ __launch_bounds__(256) void mm_join_kernel(const float *part, Epilogue ep, int splits, int I, int J) {
    const int pieces = (J + 7) / 8;
    const long n = (long)I * pieces;
    for (long u = (long)blockIdx.x * 256 + threadIdx.x; u < n; u += (long)gridDim.x * 256) {
        const long i = u / pieces;
        const int j = (int)(u - i * pieces) * 8;
        f32x8 v = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < splits; ++s) {
            const f32x8 t = load8v(part + ((long)s * I + i) * J, j, J);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += t[e];
        }
        ep.any(v, i, j, J);
    }
}

// dz = dy act'(z) in `planes` bf16 planes (rounded; what is left of it; what
// is left of that) of Jp columns, Jp a multiple of 8, zero past J; and the
// column sums of the unrounded dz over this workgroup's rows.
// One plane for bf16 gradients is a choice: they round to 2^-8 themselves, the
// operands of their products are bf16, and each plane more costs the products
// once more.  16384 x 4096 x 1024 with SiLU: gradients 2.35e-3 off in the
// 2-norm for the 1.66e-3 of their own rounding, in 320 us; with three planes
// and fp32 gradients 800 us.
// Bound by HBM: 16384 x 4096 with SiLU 85 us, 4.7 TB/s (97 with a row's loads
// awaited before the next one's).
template <class DT>
__global__ __launch_bounds__(256) void dz_kernel(const DT *dy, const uint16_t *z, uint16_t *out, long plane,
                                                 int planes, float *part, int I, int J, int Jp, int act, int rows) {
    __shared__ float sh[4][64][8];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int j = (blockIdx.x * 64 + lane) * 8;
    const int i0 = blockIdx.y * rows, i1 = min(i0 + rows, I);
    constexpr int AT = 4;  // rows requested together
    f32x8 sum = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (j < Jp) {
        for (int i = i0 + wave; i < i1; i += 4 * AT) {
            typename RawOf<DT>::type rd[AT];
            Raw16 rz[AT];
#pragma unroll
            for (int q = 0; q < AT; ++q) rd[q] = load_raw(dy + (long)min(i + 4 * q, i1 - 1) * J, j, J);
            if (z) {
#pragma unroll
                for (int q = 0; q < AT; ++q) rz[q] = load_raw(z + (long)min(i + 4 * q, i1 - 1) * J, j, J);
            }
#pragma unroll
            for (int q = 0; q < AT; ++q) {
                if (i + 4 * q >= i1) break;
                f32x8 d = raw_f32(rd[q]);
                if (z) {
                    const f32x8 t = raw_f32(rz[q]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) d[e] = dz_of(act, d[e], t[e]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += d[e];
                if (out) {
                    for (int p = 0; p < planes; ++p) {
                        u32x4 u;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            u[e] = pack2_bf16(d[2 * e], d[2 * e + 1]);
                            d[2 * e] = rest(d[2 * e], __uint_as_float(u[e] << 16));
                            d[2 * e + 1] = rest(d[2 * e + 1], __uint_as_float(u[e] & 0xffff0000u));
                        }
                        *(u32x4 *)(out + p * plane + (long)(i + 4 * q) * Jp + j) = u;
                    }
                }
            }
        }
    }
    if (!part) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) sh[wave][lane][e] = sum[e];
    __syncthreads();
    if (wave == 0 && j < J) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = ((sh[0][lane][e] + sh[1][lane][e]) + sh[2][lane][e]) + sh[3][lane][e];
        store8v(part + (long)blockIdx.y * J, sum, j, J);
    }
}

// ---- host side ----------------------------------------------------------------

static hipError_t mm_join(const MmArgs &a, const MmPlan &p, const Epilogue &ep, const float *part, hipStream_t st) {
    if (p.splits == 1) return hipSuccess;
    const long pieces = (long)a.I * ((a.J + 7) / 8);
    const long blocks = (pieces + 255) / 256;
    hipLaunchKernelGGL(mm_join_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, part, ep,
                       p.splits, a.I, a.J);
    return hipGetLastError();
}

template <bool TV, bool TU, int MODE>
static hipError_t mm_run(MmArgs a, const MmPlan &p, const Epilogue &ep, float *part, hipStream_t st) {
    mm_set(a, p, MODE != MM_BF16);
    const dim3 grid((unsigned)(a.ti * a.tj), (unsigned)p.splits);
    float *pp = p.splits > 1 ? part : nullptr;
    if (p.tile == 256)
        hipLaunchKernelGGL((mm_kernel<256, 256, 4, 2, 2, TV, TU, MODE, Epilogue>), grid, dim3(512), 0, st, a, ep, pp);
    else if (p.deep)
        hipLaunchKernelGGL((mm_kernel<128, 128, 2, 2, 4, TV, TU, MODE, Epilogue>), grid, dim3(256), 0, st, a, ep, pp);
    else
        hipLaunchKernelGGL((mm_kernel<128, 128, 2, 2, 2, TV, TU, MODE, Epilogue>), grid, dim3(256), 0, st, a, ep, pp);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : mm_join(a, p, ep, part, st);
}


MmPlan linear_plan(int M, int N, int K, bool f8) {
    return mv_takes(M, N) ? MmPlan{0, 1, 0, false} : mm_plan(M, N, slabs_of(K, f8));
}

size_t linear_ws_bytes(const MmPlan &p, int M, int N) { return mm_part_bytes(p, M, N); }

hipError_t launch_linear(const MmPlan &p, const void *x, const void *w, const float *xs, const float *ws,
                         const float *bias, const void *residual, void *y, void *z, int M, int N, int K, bool f8,
                         bool y_f32, int act, float *part, hipStream_t st) {
    MmArgs a{};
    const long es = f8 ? 1 : 2;
    a.V = (const char *)x; a.U = (const char *)w;
    a.ldv = a.ldu = K * es;
    a.I = M; a.J = N; a.K = K; a.parts = 1;
    const Epilogue ep{xs, ws, bias, residual, y, (uint16_t *)z, N, act, y_f32, past_caches(M, N, y_f32)};
    if (p.tile == 0)
        return f8 ? mv_run<true>(x, w, M, N, K, ep, st) : mv_run<false>(x, w, M, N, K, ep, st);
    if (!f8) return mm_run<false, false, MM_BF16>(a, p, ep, part, st);
    return y_f32 ? mm_run<false, false, MM_F8_F32>(a, p, ep, part, st)
                 : mm_run<false, false, MM_F8>(a, p, ep, part, st);
}

// Rows of dz per workgroup of dz_kernel: about 2048 workgroups, whole groups of
// four rows for each of its waves.
int dz_rows(int M, int N) {
    const int cols = (N + 511) / 512;
    const int want = (2048 + cols - 1) / cols;
    int rows = (M + want - 1) / want;
    return (rows + 15) / 16 * 16;
}

LinearBwdPlan linear_bwd_plan(int M, int N, int K, bool dy_f32, bool grad_f32, int act, bool dx, bool dw, bool dbias) {
    LinearBwdPlan p{};
    const bool direct = !dy_f32 && act == ACT_NONE;        // dz is dy
    p.Np = (N + 7) / 8 * 8;
    p.copy = (dx || dw) && !(direct && p.Np == N);
    const bool exact = !dy_f32 && act <= ACT_RELU;         // dz is dy or zero: bf16 holds it
    p.planes = exact || !grad_f32 ? 1 : 3;
    auto up = [](size_t b) { return (b + 255) / 256 * 256; };
    p.plane = up((size_t)M * p.Np * 2);
    size_t off = p.copy ? p.plane * p.planes : 0;
    p.sums_off = off;
    const int rows = dz_rows(M, N);
    p.blocks = (M + rows - 1) / rows;
    if (dbias) off += up((size_t)p.blocks * N * 4);
    p.part_off = off;
    MmPlan &a = p.dx, &b = p.dw;
    if (dx) a = mm_plan(M, K, p.planes * slabs_of(N, false));
    if (dw) b = mm_plan(N, K, p.planes * slabs_of(M, false));
    const size_t pa = dx ? up(mm_part_bytes(a, M, K)) : 0, pb = dw ? up(mm_part_bytes(b, N, K)) : 0;
    // both products at once where they fit the card together
    auto groups = [&](const MmPlan &m, int I) {
        return (long)((I + m.tile - 1) / m.tile) * ((K + m.tile - 1) / m.tile) * m.splits;
    };
    p.pair = dx && dw && a.tile == 128 && b.tile == 128 && groups(a, M) + groups(b, N) <= 2 * kCUs;
    p.deep = p.pair && groups(a, M) + groups(b, N) <= kCUs;
    p.part2_off = p.part_off + (p.pair ? pa : 0);
    p.total = p.pair ? p.part2_off + pb : off + (pa > pb ? pa : pb);
    return p;
}

hipError_t launch_linear_bwd(const LinearBwdPlan &p, const void *dy, const void *x, const void *w, const void *z,
                             void *dx, void *dw, float *dbias, int M, int N, int K, bool dy_f32, bool grad_f32, int act,
                             char *ws, hipStream_t st) {
    const uint16_t *dz = (const uint16_t *)dy;
    hipError_t e = hipSuccess;
    if (p.copy || dbias) {
        const int rows = dz_rows(M, N);
        const dim3 grid((unsigned)((p.Np + 511) / 512), (unsigned)p.blocks);
        uint16_t *out = p.copy ? (uint16_t *)ws : nullptr;
        float *sums = dbias ? (float *)(ws + p.sums_off) : nullptr;
        if (dy_f32)
            hipLaunchKernelGGL((dz_kernel<float>), grid, dim3(256), 0, st, (const float *)dy,
                               act ? (const uint16_t *)z : nullptr, out, (long)(p.plane / 2), p.planes, sums, M, N, p.Np,
                               act, rows);
        else
            hipLaunchKernelGGL((dz_kernel<uint16_t>), grid, dim3(256), 0, st, (const uint16_t *)dy,
                               act ? (const uint16_t *)z : nullptr, out, (long)(p.plane / 2), p.planes, sums, M, N, p.Np,
                               act, rows);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (out) dz = out;
    }
    return launch_linear_grads(p, dz, x, w, dx, dw, dbias, M, N, K, grad_f32, ws, st);
}

hipError_t launch_linear_grads(const LinearBwdPlan &p, const void *dz, const void *x, const void *w, void *dx, void *dw,
                               float *dbias, int M, int N, int K, bool grad_f32, char *ws, hipStream_t st) {
    hipError_t e = hipSuccess;
    if (dbias && !p.pair) {
        e = launch_colsum((const float *)(ws + p.sums_off), dbias, p.blocks, N, st);
        if (e != hipSuccess) return e;
    }
    float *pa = (float *)(ws + p.part_off), *pb = (float *)(ws + p.part2_off);
    // dx: V = dz [M, N] along n, U = W [N, K] with n as its rows; dw: V = dz with m as its rows, U = x [M, K]
    MmArgs a{}, b{};
    a.V = b.V = (const char *)dz;
    a.ldv = b.ldv = (long)p.Np * 2;
    a.parts = b.parts = p.planes;
    a.part_stride = b.part_stride = (long)p.plane;
    a.U = (const char *)w;
    b.U = (const char *)x;
    a.ldu = b.ldu = (long)K * 2;
    a.I = M; a.J = K; a.K = N;
    b.I = N; b.J = K; b.K = M;
    const Epilogue ea{nullptr, nullptr, nullptr, nullptr, dx, nullptr, K, ACT_NONE, grad_f32, past_caches(M, K, grad_f32)};
    const Epilogue eb{nullptr, nullptr, nullptr, nullptr, dw, nullptr, K, ACT_NONE, grad_f32, past_caches(N, K, grad_f32)};
    if (p.pair) {
        const MmPlan &qa = p.dx, &qb = p.dw;
        mm_set(a, qa, false);
        mm_set(b, qb, false);
        const int na = a.ti * a.tj * qa.splits, nb = b.ti * b.tj * qb.splits;
        float *sa = qa.splits > 1 ? pa : nullptr, *sb = qb.splits > 1 ? pb : nullptr;
        const ColSums c{(const float *)(ws + p.sums_off), dbias, p.blocks, N};
        const dim3 grid((unsigned)(na + nb + (dbias ? (N + 31) / 32 : 0)));
        if (p.deep)
            hipLaunchKernelGGL((mm_pair_kernel<4>), grid, dim3(256), 0, st, a, ea, sa, na, b, eb, sb, nb, c);
        else
            hipLaunchKernelGGL((mm_pair_kernel<2>), grid, dim3(256), 0, st, a, ea, sa, na, b, eb, sb, nb, c);
        e = hipGetLastError();
        if (e == hipSuccess) e = mm_join(a, qa, ea, pa, st);
        return e != hipSuccess ? e : mm_join(b, qb, eb, pb, st);
    }
    if (dx) e = mm_run<false, true, MM_BF16>(a, p.dx, ea, pa, st);
    if (dw && e == hipSuccess) e = mm_run<true, true, MM_BF16>(b, p.dw, eb, pb, st);
    return e;
}

}  // namespace gdn
