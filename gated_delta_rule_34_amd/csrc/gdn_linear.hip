// gdn_linear.hip -- the layer's matrix products with their epilogue,
//   z = (x W^T) x_scale w_scale + bias,   y = act(z) + residual
// and the backward of the bf16 form,
//   dz = dy act'(z),  dx = dz W,  dW = dz^T x,  dbias = sum over rows of dz.
// Products of bf16 and e4m3 values are exact and summed in fp32 by the MFMA;
// everything after the sum is fp32 with one rounding per output.
#include "gdn_device.h"
#include "gdn_launch.h"
#include "gdn_mm.h"
#include "gdn_row.h"
#include "gdn_tile.h"

namespace gdn {

enum { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3 };

__device__ __forceinline__ float sigmoid_fast(float z) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-z * LOG2E));
}

__device__ __forceinline__ float act_fwd(int act, float z) {
    switch (act) {
        case ACT_RELU: return z < 0.f ? 0.f : z;  // NaN stays
        case ACT_SILU: return z * sigmoid_fast(z);
        case ACT_GELU: return z * (0.5f * (1.f + erff(z * 0.70710678118654752f)));
    }
    return z;
}

__device__ __forceinline__ float act_bwd(int act, float z) {
    switch (act) {
        case ACT_RELU: return z > 0.f ? 1.f : 0.f;
        case ACT_SILU: {
            const float p = sigmoid_fast(z);
            return p * (1.f + z * (1.f - p));
        }
        case ACT_GELU:
            return 0.5f * (1.f + erff(z * 0.70710678118654752f)) +
                   z * __builtin_amdgcn_exp2f(-0.5f * LOG2E * z * z) * 0.3989422804014327f;
    }
    return 1.f;
}

// The epilogue of eight consecutive columns of one row.
struct Epilogue {
    const float *xs, *ws, *bias;
    const void *residual;
    void *y;
    uint16_t *z;
    long ld;        // columns of y, residual and z
    int act;
    bool y32;
    __device__ __forceinline__ void operator()(float (&v)[8], long i, int j, int J) const {
        if (xs) {
            float s[8];
            load_piece(s, ws, j, J);
            const float a = xs[i];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= a * s[e];
        }
        if (bias) {
            float b[8];
            load_piece(b, bias, j, J);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += b[e];
        }
        if (z) store_piece(z + i * ld, v, j, J);
        if (act != ACT_NONE) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = act_fwd(act, v[e]);
        }
        if (residual) {
            float t[8];
            if (y32) load_piece(t, (const float *)residual + i * ld, j, J);
            else load_piece(t, (const uint16_t *)residual + i * ld, j, J);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += t[e];
        }
        if (y32) store_piece((float *)y + i * ld, v, j, J);
        else store_piece((uint16_t *)y + i * ld, v, j, J);
    }
};

// Operand types of a product.  The e4m3 instructions, 128 and 32 deep alike,
// keep fewer bits than fp32 while they add their products (measured: sums of
// 4096 are off by 1e-5 relatively; bf16 ones by 7e-8).  They serve bf16
// outputs, whose rounding is 2^-8; for fp32 outputs the values are converted
// to bf16, which holds them exactly, as they leave LDS.
enum { MM_BF16 = 0, MM_F8 = 1, MM_F8_F32 = 2 };

// Grid: x = tiles, y = splits of k.  part (nullable): fp32 partial sums
// [split, I, J] instead of the epilogue.
template <int BI, int BJ, int WI, int WJ, bool TV, bool TU, int MODE>
__global__ __launch_bounds__(WI *WJ * 64) void mm_kernel(MmArgs a, Epilogue ep, float *part) {
    constexpr bool F8 = MODE != MM_BF16;
    constexpr int W = WI * WJ, NI = BI / WI / 16, NJ = BJ / WJ / 16;  // 16-wide tiles per wave
    using SV = Stage<BI, W, TV>;
    using SU = Stage<BJ, W, TU>;
    constexpr int SLAB = F8 ? 128 : 64;            // values of k per slab
    constexpr int BUF = SV::kBytes + SU::kBytes;
    constexpr int LDJ = BJ / WJ + 4;               // floats per row of the epilogue's image
    constexpr int EPI = W * 16 * LDJ * 4;
    __shared__ __attribute__((aligned(1024))) char smem[2 * BUF > EPI ? 2 * BUF : EPI];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int bi, bj;
    mm_tile(blockIdx.x, a.ti, a.tj, bi, bj);
    const int i0 = bi * BI, j0 = bj * BJ;
    SV sv;
    SU su;
    constexpr int ES = F8 ? 1 : 2;
    sv.init(a.V, a.ldv, i0, a.I - i0, a.K, lane, wave);
    su.init(a.U, a.ldu, j0, a.J - j0, a.K, lane, wave);
    const int per = (a.K + SLAB - 1) / SLAB;       // slabs of one plane
    const int lastb = (a.K - (per - 1) * SLAB) * ES;  // k bytes of its last slab
    const int s0 = blockIdx.y * a.per_split, s1 = min(s0 + a.per_split, a.slabs);
    lds_cchar *lds = (lds_cchar *)smem;
    const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

    f32x4 acc[NJ][NI];
#pragma unroll
    for (int x = 0; x < NJ; ++x)
#pragma unroll
        for (int y = 0; y < NI; ++y) acc[x][y] = zero4();

    // Slab loads: begin() takes the next slab's descriptors, piece() issues its
    // n-th instruction of V, then of U, into buffer buf.
    constexpr int LV = SV::kLoads, LU = SU::kLoads;
    int p = s0 / per, s = s0 - p * per, next = s0;  // plane and slab of the next load
    i32x4 rv, ru;
    int left;
    auto begin = [&] {
        const bool last = s == per - 1, live = next < s1;
        rv = sv.slab(p * a.part_stride, s, last, live);
        ru = su.slab(0, s, last, live);
        left = last ? lastb : 128;
        ++next;
        p += last;
        s = last ? 0 : s + 1;
    };
    auto piece = [&](int buf, int n) {
        if (n < LV) sv.load(rv, lds0 + buf * BUF, n, left, wave);
        else su.load(ru, lds0 + buf * BUF + SV::kBytes, n - LV, left, wave);
    };
    auto load = [&](int buf) {
        begin();
#pragma unroll
        for (int n = 0; n < LV + LU; ++n) piece(buf, n);
    };
    const int wi = (wave % WI) * NI * 16, wj = (wave / WI) * NJ * 16;
    if constexpr (MODE == MM_BF16) {
        // Fragments are read half a slab ahead of their products, in two
        // register sets, so the MFMAs only wait where waves meet: in the
        // middle of slab t every wave holds the last of t in registers, slab
        // t + 1 has landed, and the loads of t + 2 go into t's buffer.  Past
        // the end the loads write zeros and the reads are not used, which
        // keeps the loop free of branches.
        u32x4 fv[2][NI], fu[2][NJ];
        auto read = [&](auto set, int buf, int x) {  // x-th share of a set's reads
            constexpr int h = decltype(set)::value;
            lds_cchar *iv = lds + buf * BUF, *iu = iv + SV::kBytes;
            if (x < NI) fv[h][x] = mm_frag<BI, TV>(iv, wi + 16 * x, h, lane);
            fu[h][x] = mm_frag<BJ, TU>(iu, wj + 16 * x, h, lane);
        };
        auto mul = [&](auto set, int x) {
            constexpr int h = decltype(set)::value;
#pragma unroll
            for (int y = 0; y < NI; ++y) acc[x][y] = mma_bf16_raw(acc[x][y], fu[h][x], fv[h][y]);
        };
        static_assert(NI <= NJ && (LV + LU) % NJ == 0, "shares");
        constexpr int PER = (LV + LU) / NJ;
        constexpr std::integral_constant<int, 0> h0;
        constexpr std::integral_constant<int, 1> h1;
        if (s0 < s1) {
            load(0);
            load(1);
            mm_wait<LV + LU>();
            __builtin_amdgcn_s_barrier();
            mm_fence();
#pragma unroll
            for (int x = 0; x < NJ; ++x) read(h0, 0, x);
        }
        for (int t = s0; t < s1; ++t) {
            const int buf = (t - s0) & 1;
#pragma unroll
            for (int x = 0; x < NJ; ++x) {
                // (the first products go first: the wait for their operands,
                // read before the loop's jump, is for all reads)
                __builtin_amdgcn_sched_barrier(0);
                if (x == 0) mul(h0, x);
                __builtin_amdgcn_sched_barrier(0);
                read(h1, buf, x);
                __builtin_amdgcn_sched_barrier(0);
                if (x > 0) mul(h0, x);
            }
            __builtin_amdgcn_sched_barrier(0);
            begin();
            mm_wait<0>();
            __builtin_amdgcn_s_barrier();
            mm_fence();
#pragma unroll
            for (int x = 0; x < NJ; ++x) {
                __builtin_amdgcn_sched_barrier(0);
                read(h0, buf ^ 1, x);
#pragma unroll
                for (int n = 0; n < PER; ++n) piece(buf, x * PER + n);
                __builtin_amdgcn_sched_barrier(0);
                mul(h1, x);
            }
        }
        mm_wait<0>();  // the loads past the end have written before LDS is used again
    } else {
        if (s0 < s1) load(0);
        for (int t = s0; t < s1; ++t) {
            // this slab's loads have landed (each wave its own), and every
            // wave is done with the other buffer
            mm_wait<0>();
            __builtin_amdgcn_s_barrier();
            mm_fence();
            const int buf = (t - s0) & 1;
            load(buf ^ 1);
            lds_cchar *iv = lds + buf * BUF, *iu = iv + SV::kBytes;
            if constexpr (MODE == MM_F8) {
                i32x8 fv[NI];
#pragma unroll
                for (int y = 0; y < NI; ++y)
                    fv[y] = mm_pair(mm_frag<BI, TV>(iv, wi + 16 * y, 0, lane), mm_frag<BI, TV>(iv, wi + 16 * y, 1, lane));
#pragma unroll
                for (int x = 0; x < NJ; ++x) {
                    const i32x8 fu =
                        mm_pair(mm_frag<BJ, TU>(iu, wj + 16 * x, 0, lane), mm_frag<BJ, TU>(iu, wj + 16 * x, 1, lane));
#pragma unroll
                    for (int y = 0; y < NI; ++y)
                        acc[x][y] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fu, fv[y], acc[x][y], 0, 0, 0, 0, 0, 0);
                }
            } else {
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
            }
        }
        mm_wait<0>();
    }

    // Epilogue: 16 rows of the wave's part of the tile at a time through LDS
    // (its own region), so that a lane holds eight consecutive columns and a
    // row's stores are contiguous.
    __syncthreads();
    float *img = (float *)smem + wave * 16 * LDJ;
    constexpr int LPR = NJ * 2, RPP = 64 / LPR;    // lanes per row, rows per pass
    const int r = lane & 15, g = lane >> 4, c8 = (lane % LPR) * 8, rr = lane / LPR;
    const int j = j0 + wj + c8;
#pragma unroll
    for (int y = 0; y < NI; ++y) {
#pragma unroll
        for (int x = 0; x < NJ; ++x) *(f32x4 *)(img + r * LDJ + 16 * x + 4 * g) = acc[x][y];
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int q = 0; q < 16 / RPP; ++q) {
            const int i = i0 + wi + 16 * y + q * RPP + rr;
            const float *src = img + (q * RPP + rr) * LDJ + c8;
            const f32x4 lo = *(const f32x4 *)src, hi = *(const f32x4 *)(src + 4);
            float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            if (i < a.I && j < a.J) {
                if (part) store_piece(part + ((long)blockIdx.y * a.I + i) * a.J, v, j, a.J);
                else ep(v, i, j, a.J);
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Adds the partial sums of the splits in order and applies the epilogue.
__global__ __launch_bounds__(256) void mm_join_kernel(const float *part, Epilogue ep, int splits, int I, int J) {
    const int pieces = (J + 7) / 8;
    const long n = (long)I * pieces;
    for (long u = (long)blockIdx.x * 256 + threadIdx.x; u < n; u += (long)gridDim.x * 256) {
        const long i = u / pieces;
        const int j = (int)(u - i * pieces) * 8;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < splits; ++s) {
            float t[8];
            load_piece(t, part + ((long)s * I + i) * J, j, J);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += t[e];
        }
        ep(v, i, j, J);
    }
}

// What rounding left of d (nothing of an infinity or NaN: the first plane holds it).
__device__ __forceinline__ float rest(float d, float hi) { return fabsf(hi) < __builtin_inff() ? d - hi : 0.f; }

// dz = dy act'(z) in `planes` bf16 planes (rounded; what is left of it; what
// is left of that) of Jp columns, Jp a multiple of 8, zero past J; and the
// column sums of the unrounded dz over this workgroup's rows.
template <class DT>
__global__ __launch_bounds__(256) void dz_kernel(const DT *dy, const uint16_t *z, uint16_t *out, long plane,
                                                 int planes, float *part, int I, int J, int Jp, int act, int rows) {
    __shared__ float sh[4][64][8];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int j = (blockIdx.x * 64 + lane) * 8;
    const int i0 = blockIdx.y * rows, i1 = min(i0 + rows, I);
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (j < Jp) {
#pragma unroll 2
        for (int i = i0 + wave; i < i1; i += 4) {
            float d[8];
            load_piece(d, dy + (long)i * J, j, J);
            if (z) {
                float t[8];
                load_piece(t, z + (long)i * J, j, J);
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] *= act_bwd(act, t[e]);
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
                    *(u32x4 *)(out + p * plane + (long)i * Jp + j) = u;
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
        store_piece(part + (long)blockIdx.y * J, sum, j, J);
    }
}

// ---- host side ----------------------------------------------------------------

constexpr int kCUs = 256;

// How a product of I x J over `slabs` slabs is cut: a tile size and a number
// of splits of k.  With fewer tiles than compute units the sum is split so
// that they fill the card once, as long as a split keeps 4 slabs.
struct MmPlan {
    int tile, splits, per_split;
};

static MmPlan mm_plan(int I, int J, int slabs) {
    MmPlan p;
    const long big = (long)((I + 255) / 256) * ((J + 255) / 256);
    p.tile = big >= kCUs ? 256 : 128;
    const long tiles = (long)((I + p.tile - 1) / p.tile) * ((J + p.tile - 1) / p.tile);
    int s = 1;
    const long fill = 2 * kCUs;  // two workgroups of the small tile share a compute unit
    if (p.tile == 128 && tiles * 2 <= fill) s = (int)(fill / tiles);
    if (s > slabs / 4) s = slabs / 4;
    if (s > 32) s = 32;
    if (s < 1) s = 1;
    p.per_split = (slabs + s - 1) / s;
    p.splits = (slabs + p.per_split - 1) / p.per_split;
    return p;
}

static size_t mm_part_bytes(const MmPlan &p, int I, int J) {
    return p.splits > 1 ? (size_t)p.splits * I * J * sizeof(float) : 0;
}

template <bool TV, bool TU, int MODE>
static hipError_t mm_run(MmArgs a, const Epilogue &ep, float *part, hipStream_t st) {
    const int slab = MODE == MM_BF16 ? 64 : 128;
    a.slabs = a.parts * ((a.K + slab - 1) / slab);
    const MmPlan p = mm_plan(a.I, a.J, a.slabs);
    a.per_split = p.per_split;
    a.ti = (a.I + p.tile - 1) / p.tile;
    a.tj = (a.J + p.tile - 1) / p.tile;
    const dim3 grid((unsigned)(a.ti * a.tj), (unsigned)p.splits);
    float *pp = p.splits > 1 ? part : nullptr;
    if (p.tile == 256)
        hipLaunchKernelGGL((mm_kernel<256, 256, 4, 2, TV, TU, MODE>), grid, dim3(512), 0, st, a, ep, pp);
    else
        hipLaunchKernelGGL((mm_kernel<128, 128, 2, 2, TV, TU, MODE>), grid, dim3(256), 0, st, a, ep, pp);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    const long pieces = (long)a.I * ((a.J + 7) / 8);
    const long blocks = (pieces + 255) / 256;
    hipLaunchKernelGGL(mm_join_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, part, ep,
                       p.splits, a.I, a.J);
    return hipGetLastError();
}

static int slabs_of(int K, bool f8) { return (K + (f8 ? 127 : 63)) / (f8 ? 128 : 64); }

size_t linear_ws_bytes(int M, int N, int K, bool f8) { return mm_part_bytes(mm_plan(M, N, slabs_of(K, f8)), M, N); }

hipError_t launch_linear(const void *x, const void *w, const float *xs, const float *ws, const float *bias,
                         const void *residual, void *y, void *z, int M, int N, int K, bool f8, bool y_f32, int act,
                         float *part, hipStream_t st) {
    MmArgs a{};
    const long es = f8 ? 1 : 2;
    a.V = (const char *)x; a.U = (const char *)w;
    a.ldv = a.ldu = K * es;
    a.I = M; a.J = N; a.K = K; a.parts = 1;
    const Epilogue ep{xs, ws, bias, residual, y, (uint16_t *)z, N, act, y_f32};
    if (!f8) return mm_run<false, false, MM_BF16>(a, ep, part, st);
    return y_f32 ? mm_run<false, false, MM_F8_F32>(a, ep, part, st) : mm_run<false, false, MM_F8>(a, ep, part, st);
}

// Rows of dz per workgroup of dz_kernel: about 512 workgroups, whole groups of
// four rows.
static int dz_rows(int M, int N) {
    const int cols = (N + 511) / 512;
    const int want = (512 + cols - 1) / cols;
    int rows = (M + want - 1) / want;
    return (rows + 15) / 16 * 16;
}

LinearBwdPlan linear_bwd_plan(int M, int N, int K, bool dy_f32, bool grad_f32, int act, bool dx, bool dw, bool dbias) {
    LinearBwdPlan p{};
    const bool direct = !dy_f32 && act == ACT_NONE;        // dz is dy
    p.Np = (N + 7) / 8 * 8;
    p.copy = (dx || dw) && !(direct && p.Np == N);
    p.planes = direct || !grad_f32 ? 1 : 3;
    auto up = [](size_t b) { return (b + 255) / 256 * 256; };
    p.plane = up((size_t)M * p.Np * 2);
    size_t off = p.copy ? p.plane * p.planes : 0;
    p.sums_off = off;
    const int rows = dz_rows(M, N);
    p.blocks = (M + rows - 1) / rows;
    if (dbias) off += up((size_t)p.blocks * N * 4);
    p.part_off = off;
    size_t part = 0;
    if (dx) part = mm_part_bytes(mm_plan(M, K, p.planes * slabs_of(N, false)), M, K);
    if (dw) {
        const size_t b = mm_part_bytes(mm_plan(N, K, p.planes * slabs_of(M, false)), N, K);
        if (b > part) part = b;
    }
    p.total = off + up(part);
    return p;
}

hipError_t launch_linear_bwd(const void *dy, const void *x, const void *w, const void *z, void *dx, void *dw,
                             float *dbias, int M, int N, int K, bool dy_f32, bool grad_f32, int act, char *ws,
                             hipStream_t st) {
    const LinearBwdPlan p = linear_bwd_plan(M, N, K, dy_f32, grad_f32, act, dx, dw, dbias);
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
        if (dbias) {
            e = launch_colsum(sums, dbias, p.blocks, N, st);
            if (e != hipSuccess) return e;
        }
    }
    float *part = (float *)(ws + p.part_off);
    if (dx) {  // V = dz [M, N] along n, U = W [N, K] with n as its rows
        MmArgs a{};
        a.V = (const char *)dz; a.ldv = (long)p.Np * 2; a.parts = p.planes; a.part_stride = (long)p.plane;
        a.U = (const char *)w; a.ldu = (long)K * 2;
        a.I = M; a.J = K; a.K = N;
        const Epilogue ep{nullptr, nullptr, nullptr, nullptr, dx, nullptr, K, ACT_NONE, grad_f32};
        e = mm_run<false, true, MM_BF16>(a, ep, part, st);
        if (e != hipSuccess) return e;
    }
    if (dw) {  // V = dz [M, N] with m as its rows, U = x [M, K]
        MmArgs a{};
        a.V = (const char *)dz; a.ldv = (long)p.Np * 2; a.parts = p.planes; a.part_stride = (long)p.plane;
        a.U = (const char *)x; a.ldu = (long)K * 2;
        a.I = N; a.J = K; a.K = M;
        const Epilogue ep{nullptr, nullptr, nullptr, nullptr, dw, nullptr, K, ACT_NONE, grad_f32};
        e = mm_run<true, true, MM_BF16>(a, ep, part, st);
    }
    return e;
}

}  // namespace gdn
