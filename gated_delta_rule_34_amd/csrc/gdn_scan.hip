// gdn_scan.hip -- the selective state space scan and the short causal
// convolution in front of it.
//   convolution  y_t = act(b + sum_j w_j x_{t-W+1+j}) per channel
//   scan         d = softplus(dt + dt_bias), per channel and state n
//                h_n = exp(d A_n) h_n + d x B_n
//                y = (sum_n C_n h_n + D x) silu(z)
// The decay differs in every channel and state, so there is no matrix product
// in it: a state costs one exponential, two products and two multiply-adds a
// token, on the vector unit.
#include <limits.h>

#include "gdn_device.h"
#include "gdn_launch.h"
#include "gdn_row.h"
#include "gdn_tile.h"

namespace gdn {

__device__ __forceinline__ float silu_of(float z) {
    return z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-z * LOG2E));
}

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|).  log1p(e) = 2 atanh(s)
// with s = e / (2 + e) <= 1/3, atanh(s) = s P(s^2) with P of degree 4 fitted so
// that the largest relative error is least (8e-9 with its coefficients in
// fp32): small steps keep their relative accuracy, which the logarithm of
// 1 + e would lose.  The exponent's rounding costs 2^-24 |v| of e relatively
// (3.8e-6 at -80): exp(-a) = 2^m exp(-(a + m ln 2)) takes it out, up to 3e-9 a
// of the rounding of ln 2 (8 x 4096 x 2048 channels with 16 states take 306 us
// for 302 without).
__device__ __forceinline__ float softplus(float v) {
    const float a = fminf(fabsf(v), 160.f);  // finite for the correction; e is zero there
    const float m = a * -LOG2E;
    float e = __builtin_amdgcn_exp2f(m);
    e = fmaf(e, fmaf(m, -0.693147182f, -a), e);
    const float s = e * __builtin_amdgcn_rcpf(2.f + e), q = s * s;
    float p = 0.14089167f;
    p = fmaf(p, q, 0.139803f);
    p = fmaf(p, q, 0.20012455f);
    p = fmaf(p, q, 0.33333158f);
    p = fmaf(p, q, 1.f);
    return fmaf(s + s, p, v < 0.f ? 0.f : v);  // NaN stays
}

// Sequence offsets, clamped so that malformed ones stay in range.
__device__ __forceinline__ int seq_at(const int *cu, int n, int total) { return min(max(cu[n], 0), total); }

// ---- the convolution ------------------------------------------------------------

struct ConvArgs {
    const void *x;
    const float *w, *bias, *state_in;
    void *y;
    float *state_out;   // null where the state is written by conv_state_kernel
    const int *cu;      // null: seqs sequences of T tokens
    int seqs, T, total; // total: tokens
    int C, octets, last; // the last octet's first channel
    int run;            // tokens a thread walks
    int runs;           // runs of a sequence (dense) or of all tokens (packed)
    bool silu;
};

// A thread owns eight channels over a run of tokens: the window slides through
// its registers, every input is read once a run (and W - 1 before it again).
// Four tokens' loads are in flight while the four before them are computed.
// Where the channels are no multiple of eight, the last octet begins that much
// earlier and computes some of the one before it again, with the same results
// (not in place, where that one's new state may be written already; there its
// channels go one by one): 8 x 4096 x 2047 62 us against 87.
// Bound by HBM: 8 x 4096 x 2048 channels in bf16 55 us, 4.8 TB/s (110 with each
// four awaited first); one token of 64 sequences 4 us in a graph.
template <class ET, int W, bool PACKED>
__global__ __launch_bounds__(256) void conv_kernel(ConvArgs a) {
    constexpr int AT = 4, H = W - 1;
    const long id = (long)blockIdx.x * 256 + threadIdx.x;
    const long u = id / a.octets;
    const int c = min((int)(id - u * a.octets) * 8, a.last);
    const f32x8 zero = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    int n, start, end, t0, t1;
    if constexpr (PACKED) {
        if (u >= a.runs) return;
        t0 = (int)u * a.run;
        t1 = min(t0 + a.run, a.total);
        int lo = 0, hi = a.seqs;  // the first sequence that ends behind t0
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (seq_at(a.cu, mid + 1, a.total) > t0) hi = mid;
            else lo = mid + 1;
        }
        n = lo - 1;
        start = end = t0;         // the walk below enters sequence lo
        if (a.state_out) {  // sequences without tokens, shared among the runs
            for (int k = (int)u; k < a.seqs; k += a.runs) {
                if (seq_at(a.cu, k + 1, a.total) > seq_at(a.cu, k, a.total)) continue;
                for (int j = 0; j < H; ++j) {
                    const long at = ((long)k * H + j) * a.C;
                    store8v(a.state_out + at, a.state_in ? load8v(a.state_in + at, c, a.C) : zero, c, a.C);
                }
            }
        }
    } else {
        n = (int)(u / a.runs);
        if (n >= a.seqs) return;
        start = n * a.T;
        end = start + a.T;
        t0 = start + (int)(u - (long)n * a.runs) * a.run;
        t1 = min(t0 + a.run, end);
    }
    const ET *x = (const ET *)a.x;
    ET *y = (ET *)a.y;
    using Raw = typename RawOf<ET>::type;
    Raw ahead[AT];
    auto fetch = [&](int t) {
#pragma unroll
        for (int k = 0; k < AT; ++k) ahead[k] = load_raw(x + (long)min(t + k, t1 - 1) * a.C, c, a.C);
    };
    fetch(t0);
    f32x8 hist[H];  // the H inputs before t, oldest first
    auto enter = [&](int t) {
#pragma unroll
        for (int j = 0; j < H; ++j) {
            const int p = t - H + j;
            if (p >= start) hist[j] = raw_f32(load_raw(x + (long)p * a.C, c, a.C));
            else if (a.state_in) hist[j] = load8v(a.state_in + ((long)n * H + (p - start + H)) * a.C, c, a.C);
            else hist[j] = zero;
        }
    };
    if (!PACKED) enter(t0);
    f32x8 w[W], bias = zero;
    if (a.bias) bias = load8v(a.bias, c, a.C);
    if (c + 8 <= a.C) {
        float v[8 * W];
#pragma unroll
        for (int e = 0; e < 8 * W; e += 4) *(f32x4 *)&v[e] = *(const f32x4_a4 *)(a.w + (long)c * W + e);
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][e] = v[e * W + j];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][e] = c + e < a.C ? a.w[(long)(c + e) * W + j] : 0.f;
    }
    bool in = !PACKED;  // hist holds what comes before t
    for (int t = t0; t < t1; t += AT) {
        Raw raw[AT];
#pragma unroll
        for (int k = 0; k < AT; ++k) raw[k] = ahead[k];
        if (t + AT < t1) fetch(t + AT);
#pragma unroll
        for (int k = 0; k < AT; ++k) {
            const int now = t + k;
            if (now >= t1) break;
            if constexpr (PACKED) {
                if (now >= end) {  // on to the sequence of this token
                    do {
                        ++n;
                        if (n >= a.seqs) return;  // behind the last one
                        start = seq_at(a.cu, n, a.total);
                        end = seq_at(a.cu, n + 1, a.total);
                    } while (end <= now);
                    in = false;
                }
                if (now < start) continue;
                if (!in) enter(now);
                in = true;
            }
            const f32x8 v = raw_f32(raw[k]);
            f32x8 o = bias;
#pragma unroll
            for (int j = 0; j < H; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = fmaf(w[j][e], hist[j][e], o[e]);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = fmaf(w[H][e], v[e], o[e]);
            if (a.silu) {
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = silu_of(o[e]);
            }
            store8v(y + (long)now * a.C, o, c, a.C);
#pragma unroll
            for (int j = 0; j + 1 < H; ++j) hist[j] = hist[j + 1];
            hist[H - 1] = v;
            if (now + 1 == end && a.state_out) {
#pragma unroll
                for (int j = 0; j < H; ++j) store8v(a.state_out + ((long)n * H + j) * a.C, hist[j], c, a.C);
            }
        }
    }
}

// The carried inputs after each sequence, in place: a thread reads all that its
// eight channels need before it writes them.
template <class ET, int W>
__global__ __launch_bounds__(256) void conv_state_kernel(ConvArgs a, float *out) {
    constexpr int H = W - 1;
    const long id = (long)blockIdx.x * 256 + threadIdx.x;
    const int n = (int)(id / a.octets), c = (int)(id - (long)n * a.octets) * 8;
    if (n >= a.seqs) return;
    const int start = a.cu ? seq_at(a.cu, n, a.total) : n * a.T;
    const int end = a.cu ? max(seq_at(a.cu, n + 1, a.total), start) : start + a.T;
    f32x8 hist[H];
#pragma unroll
    for (int j = 0; j < H; ++j) {
        const int p = end - H + j;
        if (p >= start) hist[j] = raw_f32(load_raw((const ET *)a.x + (long)p * a.C, c, a.C));
        else hist[j] = load8v(a.state_in + ((long)n * H + (p - start + H)) * a.C, c, a.C);
    }
#pragma unroll
    for (int j = 0; j < H; ++j) store8v(out + ((long)n * H + j) * a.C, hist[j], c, a.C);
}

template <class ET, int W>
static hipError_t conv_run(ConvArgs a, float *state_out, bool apart, hipStream_t st) {
    a.state_out = apart ? nullptr : state_out;
    const long threads = (long)(a.cu ? 1 : a.seqs) * a.runs * a.octets;
    const dim3 grid((unsigned)((threads + 255) / 256));
    if (a.cu) hipLaunchKernelGGL((conv_kernel<ET, W, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((conv_kernel<ET, W, false>), grid, dim3(256), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !apart || !state_out) return e;
    const long n = (long)a.seqs * a.octets;
    hipLaunchKernelGGL((conv_state_kernel<ET, W>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, a, state_out);
    return hipGetLastError();
}

hipError_t launch_causal_conv(const void *x, const float *w, const float *bias, const float *state_in, void *y,
                              float *state_out, const int *cu, int seqs, int T, int total, int C, int W, bool bf16,
                              bool silu, hipStream_t st) {
    const int octets = (C + 7) / 8;
    const int last = C < 8 || (state_in && state_in == state_out) ? (octets - 1) * 8 : C - 8;
    ConvArgs a{x, w, bias, state_in, y, nullptr, cu, seqs, T, total, C, octets, last, 0, 0, silu};
    const int per = cu ? total : T;
    a.run = 16;
    while (a.run > 4 && (long)total * a.octets / a.run < 64 * 2048) a.run /= 2;
    a.runs = (per + a.run - 1) / a.run;
    // in place, a run at a sequence's end would overwrite what one at its start reads
    const bool apart = state_in && state_in == state_out && (cu || T > a.run);
#define GDN_CONV(Wv)                                                              \
    if (W == Wv)                                                                  \
        return bf16 ? conv_run<uint16_t, Wv>(a, state_out, apart, st) : conv_run<float, Wv>(a, state_out, apart, st);
    GDN_CONV(2)
    GDN_CONV(3)
    GDN_CONV(4)
#undef GDN_CONV
    return hipErrorInvalidValue;
}

// ---- the scan -------------------------------------------------------------------

// Four consecutive values of a row of D as they lie in memory, zero past its end.
template <class ET> struct Four;
template <> struct Four<uint16_t> {
    uint2 u;
    __device__ __forceinline__ void load(const uint16_t *p) {
        typedef uint32_t v2 __attribute__((ext_vector_type(2), aligned(2)));
        const v2 t = *(const v2 *)p;
        u = make_uint2(t[0], t[1]);
    }
    // value e becomes value e + n (n < 4), zero past the last
    __device__ __forceinline__ Four shifted(int n) const {
        const uint64_t v = ((uint64_t)u.y << 32 | u.x) >> (16 * n);
        Four o;
        o.u = make_uint2((uint32_t)v, (uint32_t)(v >> 32));
        return o;
    }
    __device__ __forceinline__ float operator[](int e) const {
        const uint32_t v = e < 2 ? u.x : u.y;
        return __uint_as_float(e & 1 ? v & 0xffff0000u : v << 16);
    }
    static __device__ __forceinline__ void store(uint16_t *p, const f32x4 &v, int c, int D) {
        typedef uint32_t v2 __attribute__((ext_vector_type(2), aligned(2)));
        if (c <= D - 4) {
            *(v2 *)(p + c) = v2{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])};
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < D) p[c + e] = to_bf16(v[e]);
        }
    }
};
template <> struct Four<float> {
    f32x4 u;
    __device__ __forceinline__ void load(const float *p) { u = *(const f32x4_a4 *)p; }
    __device__ __forceinline__ Four shifted(int n) const {
        Four o;
        o.u = n == 0 ? u : n == 1 ? f32x4{u[1], u[2], u[3], 0.f} : n == 2 ? f32x4{u[2], u[3], 0.f, 0.f} : f32x4{u[3], 0.f, 0.f, 0.f};
        return o;
    }
    __device__ __forceinline__ float operator[](int e) const { return u[e]; }
    static __device__ __forceinline__ void store(float *p, const f32x4 &v, int c, int D) {
        if (c <= D - 4) {
            *(f32x4_a4 *)(p + c) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < D) p[c + e] = v[e];
        }
    }
};

__device__ __forceinline__ float value_of(uint16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ float value_of(float v) { return v; }

constexpr int kTT = 16;   // tokens a tile
constexpr int kCH = 64;   // channels a workgroup

struct ScanArgs {
    const void *x, *dt, *B, *C, *z;
    const float *A, *D, *dt_bias, *h0;
    void *y;
    float *ht;
    const int *cu;         // null: seqs sequences of T tokens
    int seqs, T, total;
    int ch, L;             // channels; tokens a segment
    int per_seq;           // dense: segments a sequence
    float *E, *F;          // [segment, ch, N] state at a segment's end from zero (or its sequence's start); [segment, ch] sum of d
};

struct Tile {
    int t, len, seq;  // first token, tokens (0: none left), sequence
    bool first, last; // it begins, ends its sequence
};

// Tiles of a segment in order, none across a sequence's end.  Every wave of a
// workgroup walks the same ones; all of it is uniform, kept in scalar registers.
template <bool PACKED>
struct Walk {
    int pos, n, start, end, stop;
    __device__ __forceinline__ void init(const ScanArgs &a, int seg, int lane) {
        if constexpr (PACKED) {
            pos = seg * a.L;
            stop = min(pos + a.L, a.total);
            // sequences that end at or before pos, 64 offsets a look
            int lo = 0, hi = a.seqs;
            while (lo < hi) {
                const int step = (hi - lo + 63) / 64, k = lo + lane * step;
                const int ended = __popcll(__ballot(k < hi && seq_at(a.cu, k + 1, a.total) <= pos));
                hi = min(lo + ended * step, hi);
                lo = ended ? lo + (ended - 1) * step + 1 : lo;
            }
            n = __builtin_amdgcn_readfirstlane(lo);
            bounds(a);
        } else {
            n = seg / a.per_seq;
            start = n * a.T;
            end = start + a.T;
            pos = start + (seg - n * a.per_seq) * a.L;
            stop = min(pos + a.L, end);
        }
    }
    __device__ __forceinline__ void bounds(const ScanArgs &a) {
        const int k = min(n, a.seqs - 1);
        start = __builtin_amdgcn_readfirstlane(seq_at(a.cu, k, a.total));
        end = __builtin_amdgcn_readfirstlane(seq_at(a.cu, k + 1, a.total));
    }
    // On to the first sequence that ends behind token at; false: there is none.
    __device__ __forceinline__ bool reach(const ScanArgs &a, int at) {
        while (n < a.seqs && at >= end) {
            ++n;
            bounds(a);
        }
        return n < a.seqs;
    }
    // The tile at pos; moves on.
    __device__ __forceinline__ Tile next(const ScanArgs &a) {
        Tile r{0, 0, 0, false, false};
        if constexpr (PACKED) {
            if (!reach(a, pos)) return r;
            pos = max(pos, start);
        }
        if (pos >= stop) return r;
        r.t = pos;
        r.seq = n;
        r.len = min(min(kTT, end - pos), stop - pos);
        r.first = pos == start;
        pos += r.len;
        r.last = pos == end;
        return r;
    }
};

// A workgroup owns 64 channels of a segment.  SW waves scan: a lane holds N / SW
// of a channel's states, so that what a token costs them is its arithmetic and
// four LDS accesses, and leaves its part of y in LDS.  Four waves work beside
// them: they compute d and d x once per token and channel a tile ahead, and turn
// the parts of y into outputs a tile behind.  One barrier a tile.
// Bound by the vector unit: a state costs a token four instructions and an
// exponential (4.2 and 8.4 clocks each, measured), the rest of a channel and
// token 37 instructions, two exponentials and two reciprocals (counted).
// 8 x 4096 x 2048 channels, 16 states, bf16 with skip and gate: that is 253 us
// at 2.4 GHz, and takes 306 with 256 workgroups, whose two waves a SIMD leave
// gaps (vector unit busy 76 %; a single wave issues one instruction in 5.6
// clocks), 260 with two workgroups to a compute unit (16 x 2048 tokens).  HBM
// would take 105 us.  With 8 states the rest weighs as much as the states: 8 x
// 4096 x 2048 245 us for 166 of instructions.
// Tried and not kept, for 302 us then: the 4x4x1 matrix products for B (d x)
// and for y (362 us; for the first alone 310, and 250 with two workgroups),
// decays computed a group of tokens ahead (310), staging two tiles ahead (313).
// A tile never crosses a sequence's end and a sequence's entry state is asked
// for when its first tile comes: 2000 sequences of 4 tokens of 2048 channels
// 276 us, 256 of one token beside one of 2000 154 (that one alone takes 42, 256
// steps 15).  Sequences without tokens are walked one by one, about 0.2 us each:
// 4000 of them around one of 300 tokens of 256 channels 790 us for 16.
// CARRY: only the state at the segment's end, and the sum of d, for the
// segments that follow (E, F); with several segments a sequence's state enters
// a segment as E of the last, plus exp(A F) times what entered that, and so on
// back to the segment where the sequence starts.
template <class ET, int N, int SW, bool PACKED, bool CARRY>
__global__ __launch_bounds__((SW + 4) * 64, SW == 8 ? 3 : N == 64 ? 2 : 4) void scan_kernel(ScanArgs a) {
    constexpr int SPL = N / SW, PB = N / 8;
    constexpr int G = SPL == 16 ? 1 : SPL == 8 ? 2 : 4;
    typedef float sv __attribute__((ext_vector_type(SPL)));
    struct Token {
        float2 d;
        sv b, c;
    };
    __shared__ __attribute__((aligned(16))) float2 dd[2][kTT][kCH];
    __shared__ __attribute__((aligned(16))) float bc[2][2][kTT][N];
    __shared__ __attribute__((aligned(16))) float part[CARRY ? 1 : 2][CARRY ? 1 : kTT][SW][kCH];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int groups = (a.ch + kCH - 1) / kCH, seg = blockIdx.x / groups, c0 = (blockIdx.x % groups) * kCH;
    const bool whole = c0 + kCH <= a.ch;
    Walk<PACKED> walk;
    walk.init(a, seg, lane);
    if constexpr (CARRY) {
        // needed only where the sequence of the last token goes on; from its start
        if constexpr (PACKED) {
            if (!walk.reach(a, walk.stop - 1) || walk.end <= walk.stop) return;
            walk.pos = max(walk.pos, walk.start);
        } else if (walk.stop == walk.end) {
            return;
        }
    }
    if (wave < SW) {
        const int c = c0 + lane, n0 = wave * SPL;
        const bool live = c < a.ch;
        sv A, h;
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
            A[s] = live ? a.A[(long)c * N + n0 + s] * LOG2E : 0.f;
            h[s] = 0.f;
        }
        float sum = 0.f;
        if (!CARRY) {
            if (PACKED && a.ht) {  // sequences without tokens pass their state on
                for (int k = seg * 64; k < a.seqs; k += gridDim.x / groups * 64) {
                    const bool none = k + lane < a.seqs &&
                                      seq_at(a.cu, k + lane + 1, a.total) <= seq_at(a.cu, k + lane, a.total);
                    for (uint64_t m = __ballot(none); m; m &= m - 1) {
                        const long at = ((long)(k + __builtin_ctzll(m)) * a.ch + c) * N + n0;
                        sv v;
#pragma unroll
                        for (int s = 0; s < SPL; ++s) v[s] = 0.f;
                        if (live && a.h0) v = *(const sv *)(a.h0 + at);
                        if (live) *(sv *)(a.ht + at) = v;
                    }
                }
            }
            if (walk.pos > walk.start && walk.n < a.seqs) {  // the sequence comes from segments before
                const int q0 = PACKED ? walk.start / a.L : walk.n * a.per_seq;
                // four segments' values are asked for together: one after the other, their latencies would add up
                constexpr int AT = 4;
                if (live)
                    for (int q = q0; q < seg; q += AT) {
                        sv e[AT];
                        float f[AT];
#pragma unroll
                        for (int i = 0; i < AT; ++i) {
                            const long at = (long)min(q + i, seg - 1) * a.ch + c;
                            e[i] = *(const sv *)(a.E + at * N + n0);
                            f[i] = a.F[at];
                        }
#pragma unroll
                        for (int i = 0; i < AT; ++i) {
                            if (q + i >= seg) break;
#pragma unroll
                            for (int s = 0; s < SPL; ++s)
                                h[s] = q + i == q0 ? e[i][s] : fmaf(__builtin_amdgcn_exp2f(f[i] * A[s]), h[s], e[i][s]);
                        }
                    }
            }
        }
        __builtin_amdgcn_s_setprio(3);  // the others fill the gaps these waves leave
        auto fetch = [&](Token &o, int in, int k) {
            o.d = dd[in][k][lane];
            o.b = *(const sv *)&bc[in][0][k][n0];
            if (!CARRY) o.c = *(const sv *)&bc[in][1][k][n0];
        };
        auto token = [&](const Token &o, int out, int k) {
            if (CARRY) sum += o.d.x;
            float y = 0.f;
#pragma unroll
            for (int s = 0; s < SPL; ++s) {
                h[s] = fmaf(__builtin_amdgcn_exp2f(o.d.x * A[s]), h[s], o.d.y * o.b[s]);
                if (!CARRY) y = s ? fmaf(o.c[s], h[s], y) : o.c[s] * h[s];
            }
            if (!CARRY) part[out][k][wave][lane] = y;
        };
        __syncthreads();
        for (int buf = 0;; buf ^= 1) {
            const Tile tile = walk.next(a);
            if (tile.len == 0) break;
            if (tile.first) {
#pragma unroll
                for (int s = 0; s < SPL; ++s) h[s] = 0.f;
                if (a.h0 && live) h = *(const sv *)(a.h0 + ((long)tile.seq * a.ch + c) * N + n0);
            }
            if (tile.len == kTT) {
                // what G tokens need leaves LDS while the G before them are computed
                Token g[2][G];
#pragma unroll
                for (int k = 0; k < G; ++k) fetch(g[0][k], buf, k);
#pragma unroll
                for (int k0 = 0; k0 < kTT; k0 += G) {
                    const int now = k0 / G & 1;
                    if (k0 + G < kTT) {
#pragma unroll
                        for (int k = 0; k < G; ++k) fetch(g[now ^ 1][k], buf, k0 + G + k);
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int k = 0; k < G; ++k) token(g[now][k], buf, k0 + k);
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
                for (int k = 0; k < tile.len; ++k) {
                    Token o;
                    fetch(o, buf, k);
                    token(o, buf, k);
                }
            }
            if (!CARRY && tile.last && a.ht && live) *(sv *)(a.ht + ((long)tile.seq * a.ch + c) * N + n0) = h;
            __syncthreads();
        }
        __syncthreads();  // the turn in which the others finish the last tile
        if constexpr (CARRY) {
            if (live) {
                *(sv *)(a.E + ((long)seg * a.ch + c) * N + n0) = h;
                if (wave == 0) a.F[(long)seg * a.ch + c] = sum;
            }
        }
    } else {
        const int id = threadIdx.x - SW * 64, k = id >> 4, cc = (id & 15) * 4, c = c0 + cc;
        const int side = id >> 7, bt = (id & 127) * PB / N, bn = (id & 127) * PB % N;
        f32x4 bias, skip;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            bias[e] = a.dt_bias && c + e < a.ch ? a.dt_bias[c + e] : 0.f;
            skip[e] = a.D && c + e < a.ch ? a.D[c + e] : 0.f;
        }
        typedef ET bv __attribute__((ext_vector_type(PB)));
        struct In {
            Four<ET> x, dt, z;
            bv b;
            int t, len;
        };
        // Loads are issued for every thread and every tile, so that the wait
        // for one is not a wait for all: a thread whose token or channels the
        // tile lacks reads what another one does (its values are not used).
        // Channels past the last are reached by a shift.
        const int cl = min(c, a.ch - 4), shift = min(c - cl, 3);
        const void *const zp = a.z ? a.z : a.x;
        const char *const bp = (const char *)(side ? a.C : a.B);
        auto load = [&](In &in) {
            const Tile tile = walk.next(a);
            in.t = tile.t;
            in.len = tile.len;
            const int row = min(k, max(tile.len - 1, 0)), brow = min(bt, max(tile.len - 1, 0));
            const long first = (long)tile.t * a.ch * (long)sizeof(ET);
            const uint32_t at = ((uint32_t)row * (uint32_t)a.ch + (uint32_t)cl) * (uint32_t)sizeof(ET);
            in.x.load((const ET *)((const char *)a.x + first + at));
            in.dt.load((const ET *)((const char *)a.dt + first + at));
            if (!CARRY) in.z.load((const ET *)((const char *)zp + first + at));
            in.b = *(const bv *)(bp + (long)tile.t * (N * (long)sizeof(ET)) + ((uint32_t)brow * N + bn) * (uint32_t)sizeof(ET));
        };
        auto stage = [&](In in, int buf) {
            if (!whole) {
                in.x = in.x.shifted(shift);
                in.dt = in.dt.shifted(shift);
            }
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const float d0 = softplus(in.dt[e] + bias[e]), d1 = softplus(in.dt[e + 1] + bias[e + 1]);
                *(f32x4 *)&dd[buf][k][cc + e] = f32x4{d0, d0 * in.x[e], d1, d1 * in.x[e + 1]};
            }
#pragma unroll
            for (int e = 0; e < PB; ++e) bc[buf][side][bt][bn + e] = value_of(in.b[e]);
        };
        auto finish = [&](In in, int buf) {
            if (!whole) {
                in.x = in.x.shifted(shift);
                in.z = in.z.shifted(shift);
            }
            f32x4 v = *(const f32x4 *)&part[buf][k][0][cc];
#pragma unroll
            for (int w = 1; w < SW; ++w) v += *(const f32x4 *)&part[buf][k][w][cc];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = fmaf(skip[e], in.x[e], v[e]);
            if (a.z) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] *= silu_of(in.z[e]);
            }
            if (k < in.len) {
                ET *row = (ET *)a.y + (long)(in.t + k) * a.ch;
                if (whole) Four<ET>::store(row, v, c, INT_MAX);
                else Four<ET>::store(row, v, c, a.ch);
            }
        };
        // Turn j, on which the others scan tile j: tile j + 2 is asked for,
        // tile j - 1 finished and tile j + 1 staged.  The turn after the last
        // tile's is one like the others, so that the sets in flight stay where
        // they are.
        In i0, i1, i2, i3{};
        load(i0);
        load(i1);
        stage(i0, 0);
        auto turn = [&](const In &before, const In &now, const In &after, In &far, int buf) {
            load(far);
            if (!CARRY) finish(before, buf ^ 1);
            stage(after, buf ^ 1);
            __syncthreads();
            return now.len != 0;
        };
        __syncthreads();
        for (;;) {
            if (!turn(i3, i0, i1, i2, 0)) break;
            if (!turn(i0, i1, i2, i3, 1)) break;
            if (!turn(i1, i2, i3, i0, 0)) break;
            if (!turn(i2, i3, i0, i1, 1)) break;
        }
    }
}

__global__ __launch_bounds__(256) void scan_copy_kernel(const float *src, float *dst, long n) {
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256) dst[i] = src[i];
}

// How a scan is cut along its tokens.  In one part a workgroup takes T tokens at
// the pace of one alone in its compute unit; in parts their work is divided by
// the compute units, two workgroups in each, but every token is scanned twice
// (the states between the parts).  4096 tokens, 16 states, 2048 channels: 4
// sequences (128 groups of channels) 231 us in four parts, 302 in one; 5 (160)
// 334 in four parts, which are more than two workgroups to a compute unit, and
// 302 in one; 7 (224) 392 and 304.  Twice or half as many parts: 8192 tokens
// of 2048 channels 128 and 142 us for 123.  A second launch and parts that
// begin and end do not pay for few tokens: with 16 states 200 of them take 18 us
// in one part and 21 in parts of 64, 300 25 and 21; with 64 states 150 take 35,
// and 24 in parts of 32 (in parts of 64 36).  64 states, of which a compute unit
// holds one workgroup, are cut for two like the others.
ScanPlan scan_plan(int seqs, int T, int total, int ch, int N, bool packed) {
    const long groups = (ch + kCH - 1) / kCH;
    ScanPlan p{};
    const long base = packed ? groups : groups * seqs;
    const long len = packed ? total : T;
    long k = base > 128 || len * (N + 16) <= 8192 ? 1 : 512 / base;
    const long most = N >= 32 ? (len + 31) / 32 : (len + 63) / 64;
    if (k > most) k = most;
    long L = (len + k - 1) / k;
    L = (L + kTT - 1) / kTT * kTT;
    p.L = (int)L;
    p.per_seq = (int)((len + L - 1) / L);
    p.segs = packed ? p.per_seq : p.per_seq * seqs;
    if (p.per_seq > 1) {
        auto up = [](size_t b) { return (b + 255) / 256 * 256; };
        p.f_off = up((size_t)p.segs * ch * N * 4);
        p.h_off = p.f_off + up((size_t)p.segs * ch * 4);
        p.total = p.h_off + up((size_t)seqs * ch * N * 4);
    }
    return p;
}

template <class ET, int N>
static hipError_t scan_run(const ScanArgs &a, const ScanPlan &p, hipStream_t st) {
    const dim3 grid((unsigned)((a.ch + kCH - 1) / kCH) * (unsigned)p.segs);
    if (p.per_seq > 1) {
        if (a.cu) hipLaunchKernelGGL((scan_kernel<ET, N, 4, true, true>), grid, dim3(512), 0, st, a);
        else hipLaunchKernelGGL((scan_kernel<ET, N, 4, false, true>), grid, dim3(512), 0, st, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if constexpr (N >= 32) {
        // at most one workgroup to each compute unit: eight scanning waves, so
        // that each SIMD has three waves to choose from (8 x 2048 x 2048
        // channels with 32 states 237 us against 269 with four, 8 x 1024 x 2048
        // with 64 205 against 230; with 16, two to a lane, the reads from LDS
        // outweigh it: 8 x 4096 x 2048 358 against 302).  More workgroups take
        // four, two of which share a compute unit with 32 states.  With 64 the
        // four-wave form takes 140 registers, three waves a SIMD, and so runs
        // alone, too; eight waves would serve there as well: 16 x 1024 x 2048
        // 457 us so and 408 with eight, 1 x 8192 x 2048 in parts 398 and 375.
        if (grid.x <= 256) {
            if (a.cu) hipLaunchKernelGGL((scan_kernel<ET, N, 8, true, false>), grid, dim3(768), 0, st, a);
            else hipLaunchKernelGGL((scan_kernel<ET, N, 8, false, false>), grid, dim3(768), 0, st, a);
            return hipGetLastError();
        }
    }
    if (a.cu) hipLaunchKernelGGL((scan_kernel<ET, N, 4, true, false>), grid, dim3(512), 0, st, a);
    else hipLaunchKernelGGL((scan_kernel<ET, N, 4, false, false>), grid, dim3(512), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_selective_scan(const ScanPlan &p, const void *x, const void *dt, const float *A, const void *B,
                                 const void *C, const float *D, const void *z, const float *dt_bias, const float *h0,
                                 void *y, float *ht, const int *cu, int seqs, int T, int total, int ch, int N, bool bf16,
                                 char *ws, hipStream_t st) {
    ScanArgs a{x, dt, B, C, z, A, D, dt_bias, h0, y, ht, cu, seqs, T, total, ch, p.L, p.per_seq, nullptr, nullptr};
    if (p.per_seq > 1) {
        a.E = (float *)ws;
        a.F = (float *)(ws + p.f_off);
        if (h0 && h0 == ht) {  // a segment at a sequence's end would overwrite what one at its start reads
            const long n = (long)seqs * ch * N, blocks = (n + 255) / 256;
            float *copy = (float *)(ws + p.h_off);
            hipLaunchKernelGGL(scan_copy_kernel, dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, st, h0, copy,
                               n);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            a.h0 = copy;
        }
    }
#define GDN_SCAN(Nv) \
    if (N == Nv) return bf16 ? scan_run<uint16_t, Nv>(a, p, st) : scan_run<float, Nv>(a, p, st);
    GDN_SCAN(8)
    GDN_SCAN(16)
    GDN_SCAN(32)
    GDN_SCAN(64)
#undef GDN_SCAN
    return hipErrorInvalidValue;
}

// ---- one token --------------------------------------------------------------------

// A lane holds four states of a channel (16 bytes in, 16 out), N / 4 lanes a
// channel; y is summed over them on DPP.  Bound by the states' traffic: 256 x
// 2048 channels with 16 states 15 us, 4.75 TB/s; 64 sequences 4.8 us in a graph.
template <class ET, int N>
__global__ __launch_bounds__(256) void scan_step_kernel(const ET *x, const ET *dt, const float *A, const ET *B,
                                                        const ET *C, const float *D, const ET *z,
                                                        const float *dt_bias, const float *h0, float *h1, ET *y,
                                                        int seqs, int ch) {
    constexpr int LPC = N / 4;
    const long id = (long)blockIdx.x * 256 + threadIdx.x;
    const long u = id / LPC;  // (sequence, channel)
    const int q = (int)(id % LPC) * 4;
    if (u >= (long)seqs * ch) return;  // whole groups of LPC lanes
    const long b = u / ch;
    const int c = (int)(u - b * ch);
    const f32x4 h = *(const f32x4 *)(h0 + u * N + q);
    const f32x4 A4 = *(const f32x4 *)(A + (long)c * N + q);
    Four<ET> bv, cv;
    bv.load(B + b * N + q);
    cv.load(C + b * N + q);
    const float xv = load_elem(x + u);
    const float d = softplus(load_elem(dt + u) + (dt_bias ? dt_bias[c] : 0.f));
    f32x4 o;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        o[e] = fmaf(__builtin_amdgcn_exp2f(d * LOG2E * A4[e]), h[e], d * xv * bv[e]);
        s = fmaf(cv[e], o[e], s);
    }
    *(f32x4 *)(h1 + u * N + q) = o;
    s += dpp_f32<0xB1, 0xf>(s);                      // quad_perm [1, 0, 3, 2]
    if (LPC >= 4) s += dpp_f32<0x4E, 0xf>(s);        // quad_perm [2, 3, 0, 1]
    if (LPC >= 8) s += dpp_f32<0x141, 0xf>(s);       // row_half_mirror
    if (LPC >= 16) s += dpp_f32<0x140, 0xf>(s);      // row_mirror
    if (q == 0) {
        if (D) s = fmaf(D[c], xv, s);
        if (z) s *= silu_of(load_elem(z + u));
        store_elem(y + u, s);
    }
}

hipError_t launch_selective_step(const void *x, const void *dt, const float *A, const void *B, const void *C,
                                 const float *D, const void *z, const float *dt_bias, const float *h0, float *h1,
                                 void *y, int seqs, int ch, int N, bool bf16, hipStream_t st) {
    const long threads = (long)seqs * ch * (N / 4);
    const dim3 grid((unsigned)((threads + 255) / 256));
#define GDN_STEP(ET, Nv)                                                                                            \
    hipLaunchKernelGGL((scan_step_kernel<ET, Nv>), grid, dim3(256), 0, st, (const ET *)x, (const ET *)dt, A,        \
                       (const ET *)B, (const ET *)C, D, (const ET *)z, dt_bias, h0, h1, (ET *)y, seqs, ch)
#define GDN_STEP_N(Nv)                      \
    if (N == Nv) {                          \
        if (bf16) GDN_STEP(uint16_t, Nv);   \
        else GDN_STEP(float, Nv);           \
        return hipGetLastError();           \
    }
    GDN_STEP_N(8)
    GDN_STEP_N(16)
    GDN_STEP_N(32)
    GDN_STEP_N(64)
#undef GDN_STEP_N
#undef GDN_STEP
    return hipErrorInvalidValue;
}

}  // namespace gdn
