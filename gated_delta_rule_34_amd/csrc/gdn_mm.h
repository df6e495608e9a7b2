// gdn_mm.h -- the tiled matrix product of the layer's projections on gfx950,
// shared by gdn_linear and its backward:
//   C[i][j] = sum_k V(i, k) U(j, k),   j contiguous in C
// with V either [I, K] (k contiguous) or [K, I], U either [J, K] or [K, J],
// in bf16, or e4m3 for the k-contiguous forms.
//
// A workgroup owns a BI x BJ tile of C and steps through k in slabs of 128
// bytes (64 bf16 or 128 e4m3 values).  Slabs go from HBM/L2 straight into LDS
// (buffer loads with LDS destination, no registers in between), two or four
// of them ahead of the products.  The buffer descriptors carry the range of
// the tile's valid rows, so rows past the end, and k past the end (lanes sent
// out of range in the last slab), arrive as zeros with no branch.
// U is the A operand of the MFMA and V the B operand, so a lane's four
// accumulator values are four consecutive j of one row i.
//
// LDS images.  A load instruction writes 1024 consecutive LDS bytes, 16 per
// lane, so swizzles are applied to the global side: a lane fetches the 16-byte
// unit that belongs at its place.
//   k contiguous: rows of 128 bytes, unit c of row r at c ^ (2 (r>>1 & 1) +
//     4 (r>>3 & 1)).  A fragment read takes unit 4 s + g of 16 rows; the 16
//     lanes of each of its four passes then cover all 64 banks once.
//   k strided: rows of BJ (BI) values, the 32-byte pair of units p of row k at
//     p ^ ((k & 3) + 4 (k>>3 & 1)).  The transpose load takes 4 x 4 blocks;
//     the 8 rows of each of its two passes fall on different bank groups.
// Both forms give lane g of a 32-deep MFMA the values k = 8 g .. 8 g + 7, so
// they combine freely.
#pragma once
#include <type_traits>

#include "gdn_device.h"
#include "gdn_tile.h"

namespace gdn {

typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(4))) int i32x4;

struct MmArgs {
    const char *V, *U;
    long ldv, ldu;      // bytes from row to row as stored
    int I, J, K;        // sizes, K in values
    int parts;          // V in this many planes whose products add up
    long part_stride;   // bytes from plane to plane
    int slabs;          // slabs of the whole sum: parts * ceil(K / slab)
    int per_split;      // slabs per split; splits = gridDim.y
    int ti, tj;         // tiles along i and j
    long pair;          // gated products: bytes from a gate row of U to its up row
};

// Sixteen e4m3 values as two bf16 fragments (exact).
__device__ __forceinline__ void f8_to_bf16(u32x4 (&o)[2], const u32x4 &a) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a[e], 1.f, false);
        const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a[e], 1.f, true);
        o[e >> 1][2 * (e & 1)] = __builtin_bit_cast(uint32_t, lo);
        o[e >> 1][2 * (e & 1) + 1] = __builtin_bit_cast(uint32_t, hi);
    }
}

__device__ __forceinline__ i32x8 mm_pair(const u32x4 &lo, const u32x4 &hi) {
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

__device__ __forceinline__ f32x4 mma_f8_slab(f32x4 acc, const i32x8 &a, const i32x8 &b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 0, 0, 0, 0, 0, 0);
}

// Waits until at most N of this wave's slab loads are in flight and its LDS
// reads are done; nothing moves across.
template <int N>
__device__ __forceinline__ void mm_wait() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"(N) : "memory");
}
__device__ __forceinline__ void mm_fence() { asm volatile("" ::: "memory"); }

constexpr uint32_t kOutOfRange = 0xfffffff0u;  // beyond every descriptor's range

// One 1024-byte piece into LDS at byte address lds (same in every lane).
__device__ __forceinline__ void lds_load(uint32_t lds, uint32_t voff, i32x4 rsrc) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc)
                 : "m0", "memory");
}

// The same with 4 bytes a lane: for what it brings into the caches.
__device__ __forceinline__ void lds_touch(uint32_t lds, uint32_t voff, i32x4 rsrc) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc)
                 : "m0", "memory");
}

__device__ __forceinline__ i32x4 make_rsrc(const char *base, uint32_t bytes) {
    const uint64_t b = (uint64_t)base;
    i32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)b);
    r[1] = __builtin_amdgcn_readfirstlane((int)((uint32_t)(b >> 32) & 0xffffu));
    r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
    r[3] = 0x00020000;
    return r;
}

__device__ __forceinline__ int swz_row(int r) { return (r & 2) | ((r >> 1) & 4); }        // k contiguous
__device__ __forceinline__ int swz_col(int k) { return (k & 3) | ((k >> 1) & 4); }        // k strided, pairs

// Staging of one operand: R rows of the tile (R = BI or BJ), and the
// descriptor of the slab that is loaded next.
template <int R, int W, bool T>
struct Stage {
    static constexpr int kBytes = R * 128;
    static constexpr int kLoads = R / 8 / W;  // instructions per wave and slab
    static_assert(R % (8 * W) == 0, "whole instructions per wave");
    uint32_t off[kLoads];   // byte offsets of this lane's units, from the slab's base
    int chunk[kLoads];      // k contiguous: first k byte of the unit within the slab
    i32x4 rsrc;
    long step, wrap;        // bytes to the next slab, and from a plane's last slab to the next plane's first
    uint32_t range, range_last;

    // rows: valid rows from this tile's first on; K: bytes (k contiguous) or rows (k strided) of the sum;
    // plane, s: plane and slab of the first load, per slabs a plane, planes part bytes apart
    __device__ __forceinline__ void init(const char *p, long ld, int row0, int rows, int Kb, long part, int per, int plane,
                                         int s, int lane, int wave) {
        if (!T) {
            p += (long)row0 * ld;
            step = 128;
            range = range_last = (uint32_t)min(rows, R) * (uint32_t)ld;
#pragma unroll
            for (int n = 0; n < kLoads; ++n) {
                const int row = (wave + W * n) * 8 + (lane >> 3);
                chunk[n] = ((lane & 7) ^ swz_row(row & 15)) * 16;
                off[n] = (uint32_t)row * (uint32_t)ld + chunk[n];
            }
        } else {
            constexpr int UPR = R / 8;        // units per k row
            p += (long)row0 * 2;
            step = 64 * ld;
            range = (uint32_t)(64 * ld - (long)row0 * 2);
            const int left = Kb & 63;
            range_last = (uint32_t)((left ? left : 64) * ld - (long)row0 * 2);
#pragma unroll
            for (int n = 0; n < kLoads; ++n) {
                const int u = (wave + W * n) * 64 + lane, k = u / UPR, c = u % UPR;
                off[n] = (uint32_t)k * (uint32_t)ld + (uint32_t)((c ^ (swz_col(k) << 1)) * 16);
                chunk[n] = 0;
            }
        }
        wrap = part - (long)(per - 1) * step;
        rsrc = make_rsrc(p + plane * part + s * step, 0);
    }
    // The rows of a gated product: sixteen gate rows and the sixteen up rows
    // `pair` bytes behind them in turn, so that the wave that holds a gate
    // column's products holds those of its up column.  A wave's instructions
    // are all of one kind.
    __device__ __forceinline__ void init_pairs(const char *p, long ld, int row0, int rows, int Kb, long pair, int per, int s,
                                               int lane, int wave) {
        static_assert(!T && W % 4 == 0, "eight rows an instruction, four instructions a pair of sixteens");
        init(p + (wave & 2 ? pair : 0), ld, row0, min(rows, R / 2), Kb, 0, per, 0, s, lane, wave);
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
            const int row = (wave + W * n) * 8 + (lane >> 3);
            off[n] = (uint32_t)((row >> 5) * 16 + (row & 15)) * (uint32_t)ld + chunk[n];
        }
    }
    // A slab past the end (live false) has no range: its loads write zeros and read nothing.
    __device__ __forceinline__ void bound(bool last, bool live) { rsrc[2] = (int)(live ? (last ? range_last : range) : 0u); }
    __device__ __forceinline__ void advance(bool last) {
        const uint64_t at = ((uint64_t)(uint32_t)rsrc[1] << 32 | (uint32_t)rsrc[0]) + (uint64_t)(last ? wrap : step);
        rsrc[0] = (int)(uint32_t)at;
        rsrc[1] = (int)(uint32_t)(at >> 32);
    }
    // Instruction n of the slab into LDS at lds; left: bytes of k in the slab
    // (128 but for a k-contiguous operand's last one)
    __device__ __forceinline__ void load(uint32_t lds, int n, int left, int wave) const {
        const uint32_t o = T || chunk[n] < left ? off[n] : kOutOfRange;
        lds_load(__builtin_amdgcn_readfirstlane(lds + (uint32_t)(wave + W * n) * 1024), o, rsrc);
    }
};

typedef __attribute__((address_space(3))) const char lds_cchar;

// Fragment (half slab s, 16 rows from row0) of a k-contiguous image.
__device__ __forceinline__ u32x4 mm_frag_rows(lds_cchar *img, int row0, int s, int lane) {
    typedef __attribute__((address_space(3))) const u32x4 lds_v;
    const int r = lane & 15, g = lane >> 4;
    return *(lds_v *)(img + r * 128 + (((4 * s + g) ^ swz_row(r)) << 4) + row0 * 128);
}

// Fragment (k = 32 s .. 32 s + 31, 16 columns from col0) of a k-strided image of R columns.
template <int R>
__device__ __forceinline__ u32x4 mm_frag_cols(lds_cchar *img, int col0, int s, int lane) {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const int r = lane & 15, g = lane >> 4;
    const int f = (r >> 2) | ((g & 1) << 2);
    const int row = 8 * g + (r >> 2);
    lds_cchar *p = img + row * (R * 2) + (((col0 >> 4) ^ f) << 5) + ((r & 3) << 3) + s * 32 * (R * 2);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * (R * 2)));
    const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
    return u32x4{a.x, a.y, b.x, b.y};
}

template <int R, bool T>
__device__ __forceinline__ u32x4 mm_frag(lds_cchar *img, int row0, int s, int lane) {
    if constexpr (T) return mm_frag_cols<R>(img, row0, s, lane);
    else return mm_frag_rows(img, row0, s, lane);
}

// The tile (bi, bj) of workgroup b of n.  Workgroup b runs on XCD b % 8: each
// XCD gets a contiguous run of tiles, walked in bands of 4 tile rows, so that
// the tiles an XCD works on at a time (8 columns of a band) share their
// operand rows in its L2.  Bands of 2, 8 and 16 were up to 4 % slower.
__device__ __forceinline__ void mm_tile(int b, int ti, int tj, int &bi, int &bj) {
    const int n = ti * tj, q = n / 8, rem = n % 8, x = b % 8;
    const int id = x * q + min(x, rem) + b / 8;
    constexpr int BAND = 4;
    const int band = id / (BAND * tj), first = band * BAND, h = min(BAND, ti - first);
    const int in = id - band * BAND * tj;
    bi = first + in % h;
    bj = in / h;
}

}  // namespace gdn
