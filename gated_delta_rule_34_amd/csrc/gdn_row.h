// gdn_row.h -- row-wise pieces shared by the norm, quantiser and linear
// kernels: eight columns per lane at any element alignment, sums and maxima
// over a wave (DPP) or a workgroup, and the e4m3 rounding of a scaled row.
#pragma once
#include "gdn_device.h"
#include "gdn_tile.h"

namespace gdn {

// 16- and 8-byte accesses at element alignment (rows of odd width start
// anywhere; global memory accesses need no alignment on this target).
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));

__device__ __forceinline__ uint32_t pack2_bf16(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}
__device__ __forceinline__ uint16_t to_bf16(float a) { return (uint16_t)pack2_bf16(a, 0.f); }

// Columns c .. c + 7 of a row of D as fp32, zero past its end.
__device__ __forceinline__ void load_piece(float (&v)[8], const uint16_t *p, int c, int D) {
    if (c + 8 <= D) {
        const u32x4_a2 u = *(const u32x4_a2 *)(p + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(u[e] << 16);
            v[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c + e < D ? bf16_to_f32(p[c + e]) : 0.f;
    }
}
__device__ __forceinline__ void load_piece(float (&v)[8], const float *p, int c, int D) {
    if (c + 8 <= D) {
        const f32x4_a4 a = *(const f32x4_a4 *)(p + c), b = *(const f32x4_a4 *)(p + c + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = a[e];
            v[4 + e] = b[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c + e < D ? p[c + e] : 0.f;
    }
}
__device__ __forceinline__ void store_piece(uint16_t *p, const float (&v)[8], int c, int D) {
    if (c + 8 <= D) {
        u32x4_a2 u;
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = pack2_bf16(v[2 * e], v[2 * e + 1]);
        *(u32x4_a2 *)(p + c) = u;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < D) p[c + e] = to_bf16(v[e]);
    }
}
__device__ __forceinline__ void store_piece(float *p, const float (&v)[8], int c, int D) {
    if (c + 8 <= D) {
        *(f32x4_a4 *)(p + c) = f32x4_a4{v[0], v[1], v[2], v[3]};
        *(f32x4_a4 *)(p + c + 4) = f32x4_a4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < D) p[c + e] = v[e];
    }
}

// The same on a native vector (kept in registers where an array that is passed
// around can end up in scratch memory), whole pieces and any piece.
typedef float f32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x8 bf16x8_to_f32(const u32x4 &u) {
    f32x8 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(u[e] << 16);
        v[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
    }
    return v;
}
__device__ __forceinline__ f32x8 load8v(const float *p) {
    const f32x4_a4 a = *(const f32x4_a4 *)p, b = *(const f32x4_a4 *)(p + 4);
    return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
__device__ __forceinline__ f32x8 load8v(const uint16_t *p) { return bf16x8_to_f32(*(const u32x4_a2 *)p); }
__device__ __forceinline__ void store8v(uint16_t *p, const f32x8 &v) {
    u32x4_a2 u;
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = pack2_bf16(v[2 * e], v[2 * e + 1]);
    *(u32x4_a2 *)p = u;
}
__device__ __forceinline__ void store8v(float *p, const f32x8 &v) {
    *(f32x4_a4 *)p = f32x4_a4{v[0], v[1], v[2], v[3]};
    *(f32x4_a4 *)(p + 4) = f32x4_a4{v[4], v[5], v[6], v[7]};
}
// Non-temporal: for what this pass and the next one do not read.
__device__ __forceinline__ void store8nt(uint16_t *p, const f32x8 &v) {
    u32x4_a2 u;
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = pack2_bf16(v[2 * e], v[2 * e + 1]);
    __builtin_nontemporal_store(u, (u32x4_a2 *)p);
}
__device__ __forceinline__ void store8nt(float *p, const f32x8 &v) {
    __builtin_nontemporal_store(f32x4_a4{v[0], v[1], v[2], v[3]}, (f32x4_a4 *)p);
    __builtin_nontemporal_store(f32x4_a4{v[4], v[5], v[6], v[7]}, (f32x4_a4 *)(p + 4));
}
template <class T>
__device__ __forceinline__ void store8p(T *p, const f32x8 &v, bool nt) {
    if (nt) store8nt(p, v);
    else store8v(p, v);
}
template <class T>
__device__ __forceinline__ f32x8 load8v(const T *p, int c, int D) {
    if (c + 8 <= D) return load8v(p + c);
    f32x8 v = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (c + e < D) v[e] = load_elem(p + c + e);
    return v;
}
__device__ __forceinline__ void store_elem(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_elem(uint16_t *p, float v) { *p = to_bf16(v); }
template <class T>
__device__ __forceinline__ void store8v(T *p, const f32x8 &v, int c, int D) {
    if (c + 8 <= D) {
        store8v(p + c, v);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (c + e < D) store_elem(p + c + e, v[e]);
}

// Eight columns as they lie in memory (zero past D), for loads that are
// issued long before their values are used.
struct Raw16 {
    u32x4 a;
};
struct Raw32 {
    u32x4 a, b;
};
template <class T> struct RawOf;
template <> struct RawOf<uint16_t> { using type = Raw16; };
template <> struct RawOf<float> { using type = Raw32; };

__device__ __forceinline__ Raw16 load_raw(const uint16_t *p, int c, int D) {
    Raw16 o;
    if (c + 8 <= D) {
        o.a = *(const u32x4_a2 *)(p + c);
    } else {
        uint32_t t[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = c + e < D ? p[c + e] : 0;
        o.a = u32x4{t[0] | t[1] << 16, t[2] | t[3] << 16, t[4] | t[5] << 16, t[6] | t[7] << 16};
    }
    return o;
}
__device__ __forceinline__ Raw32 load_raw(const float *p, int c, int D) {
    Raw32 o;
    const uint32_t *u = (const uint32_t *)p;
    typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
    if (c + 8 <= D) {
        o.a = *(const u32x4_a4 *)(u + c);
        o.b = *(const u32x4_a4 *)(u + c + 4);
    } else {
        uint32_t t[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = c + e < D ? u[c + e] : 0;
        o.a = u32x4{t[0], t[1], t[2], t[3]};
        o.b = u32x4{t[4], t[5], t[6], t[7]};
    }
    return o;
}
__device__ __forceinline__ f32x8 raw_f32(const Raw16 &r) { return bf16x8_to_f32(r.a); }
__device__ __forceinline__ f32x8 raw_f32(const Raw32 &r) {
    f32x8 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = __uint_as_float(r.a[e]);
        v[4 + e] = __uint_as_float(r.b[e]);
    }
    return v;
}

// v / scale for one row: a reciprocal and one correction step, which gives the
// correctly rounded quotient that a division would (codes are compared with
// it, and quotients of bf16 values fall on e4m3's midpoints often); scales
// whose reciprocal leaves the normal range are divided by, and clamped, since
// a denormal scale may have rounded down.
struct QuantRow {
    float scale, inv;
    bool plain;
    __device__ __forceinline__ explicit QuantRow(float s) : scale(s), inv(1.f / s), plain(s > 1e-30f && s < 1e30f) {}
    __device__ __forceinline__ float operator()(float v) const {
        if (plain) {
            const float q = v * inv;
            return fmaf(fmaf(-q, scale, v), inv, q);
        }
        const float q = v / scale;
        return fabsf(q) > 448.f ? copysignf(448.f, q) : q;  // NaN passes through
    }
};

__device__ __forceinline__ uint32_t pack4_f8(float a, float b, float c, float d) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

__device__ __forceinline__ void store_piece_f8(uint8_t *p, const float (&v)[8], const QuantRow &q, int c, int D) {
    if (c >= D) return;
    u32x2_a1 u = {pack4_f8(q(v[0]), q(v[1]), q(v[2]), q(v[3])), pack4_f8(q(v[4]), q(v[5]), q(v[6]), q(v[7]))};
    if (c + 8 <= D) {
        *(u32x2_a1 *)(p + c) = u;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < D) p[c + e] = (uint8_t)(u[e >> 2] >> (8 * (e & 3)));
    }
}

template <int CTRL, int ROWMASK>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWMASK, 0xf, false);
}

// Sum and maximum over the wave, the same in every lane: shifts 1, 2, 4, 8
// within rows of 16 lanes, the row totals by the lane-15 and lane-31
// broadcasts, and lane 63 read back.
__device__ __forceinline__ float wave_sum(float x) {
    x += dpp_f32<0x111, 0xf>(x);
    x += dpp_f32<0x112, 0xf>(x);
    x += dpp_f32<0x114, 0xf>(x);
    x += dpp_f32<0x118, 0xf>(x);
    x += dpp_f32<0x142, 0xa>(x);
    x += dpp_f32<0x143, 0xc>(x);
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), 63));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    x = max(x, dpp_u32<0x111, 0xf>(x));
    x = max(x, dpp_u32<0x112, 0xf>(x));
    x = max(x, dpp_u32<0x114, 0xf>(x));
    x = max(x, dpp_u32<0x118, 0xf>(x));
    x = max(x, dpp_u32<0x142, 0xa>(x));
    x = max(x, dpp_u32<0x143, 0xc>(x));
    return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

// The same over the TPR threads of a row; sh holds TPR / 64 words and is
// written once per call (callers that call in a loop alternate two of them).
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float *sh) {
    x = wave_sum(x);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
        __syncthreads();
        x = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) x += sh[i];
    }
    return x;
}
template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t x, uint32_t *sh) {
    x = wave_max(x);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
        __syncthreads();
        x = 0;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) x = max(x, sh[i]);
    }
    return x;
}

}  // namespace gdn
