// gdn_api.hip -- the C ABI declared in include/gdn.h: argument validation,
// workspace layout and kernel sequencing on the caller's stream.  No device
// memory is allocated here; every buffer belongs to the caller.
#include <limits.h>
#include <stdint.h>

#include "../../include/gdn.h"
#include "gdn_launch.h"

namespace {

constexpr int kBT = 64;
constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool head_ok(int d) { return d == 64 || d == 128; }
bool dtype_ok(gdn_dtype dt) { return dt == GDN_F32 || dt == GDN_BF16; }
size_t esize(gdn_dtype dt) { return dt == GDN_BF16 ? 2 : 4; }

struct Range {
    const void *p;
    size_t n;
};

bool overlap(Range a, Range b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.n && b0 < a0 + a.n;
}

// No output may overlap an input, another output or the workspace.
template <int NI, int NO>
static bool disjoint(const Range (&ins)[NI], const Range (&outs)[NO]) {
    for (int a = 0; a < NO; ++a) {
        for (Range in : ins)
            if (overlap(outs[a], in)) return false;
        for (int c = a + 1; c < NO; ++c)
            if (overlap(outs[a], outs[c])) return false;
    }
    return true;
}

// Workspace of the chunked forward: G2 [B,H,NT,64] fp32, then (T - I)
// [B,H,NT,64,64] fp32, each section 256-byte aligned.
struct ChunkWs {
    size_t g2_off, t_off, total;
};

ChunkWs chunk_ws(int B, int T, int H) {
    const size_t NT = (size_t)(T + kBT - 1) / kBT;
    const size_t chunks = (size_t)B * H * NT;
    ChunkWs w;
    w.g2_off = 0;
    w.t_off = align_up(chunks * kBT * sizeof(float));
    w.total = w.t_off + align_up(chunks * kBT * kBT * sizeof(float));
    return w;
}

bool sizes_ok(int B, int T, int H) {
    if (B < 1 || T < 1 || H < 1) return false;
    const long long NT = (T + kBT - 1) / kBT;
    return (long long)B * H * NT < (1LL << 31);
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Chunk-parallel plan for the bf16 forward of a dense batch (gdn_fused.hip,
// SegArgs).  The single kernel runs (Dv / 32) workgroups per head, one per
// compute unit, each walking every chunk in order; when that fills less than
// half of the 256 compute units, each sequence is cut into NS segments of L
// chunks.  The walk launch runs 2 NS - 3 workgroup sets per head (one for
// segment 0's end state, two per middle segment), so NS is the largest count
// for which they fit the compute units in one round; the single kernel then
// runs the NS segments of every head together.  NS = 0: no plan.
struct SegPlan {
    int NS, L;
};

constexpr int kPlanCUs = 256;  // compute units of the MI355X

SegPlan seg_plan(int B, int T, int H, int Dk, int Dv) {
    SegPlan p{0, 0};
    if (Dk != Dv) return p;
    const long sets = (long)B * H * (Dv / 32);   // workgroups of the single kernel
    if (sets * 2 > kPlanCUs) return p;
    const int NT = (T + kBT - 1) / kBT;
    int ns = (int)((kPlanCUs / sets + 3) / 2);
    if (ns > 16) ns = 16;
    for (; ns >= 3; --ns) {
        const int L = (NT + ns - 1) / ns;
        if (L >= 8 && (ns - 1) * L < NT) {
            p = SegPlan{ns, L};
            return p;
        }
    }
    return p;
}

// Workspace of the plan: Hin, Hout, M [B NS, H, D, D] fp32, then the B NS + 1
// segment offsets (int32); each section 256-byte aligned.
struct SegWs {
    size_t hin, hout, m, cu, total;
};

SegWs seg_ws(int B, int H, int D, const SegPlan &p) {
    const size_t st = align_up((size_t)B * p.NS * H * D * D * sizeof(float));
    SegWs w;
    w.hin = 0;
    w.hout = st;
    w.m = 2 * st;
    w.cu = 3 * st;
    w.total = w.cu + align_up(((size_t)B * p.NS + 1) * sizeof(int));
    return w;
}

gdn_status from_hip(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_HIP; }

}  // namespace

extern "C" {

const char *gdn_status_string(gdn_status s) {
    switch (s) {
        case GDN_OK: return "ok";
        case GDN_ERR_INVALID_ARG: return "invalid argument";
        case GDN_ERR_UNSUPPORTED: return "unsupported head size or dtype";
        case GDN_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
        case GDN_ERR_HIP: return "HIP launch failed";
    }
    return "unknown status";
}

// bf16 inputs take the single-kernel path, which needs no workspace; fp32
// inputs take the two-stage path (intra-chunk stage, then the state walk).
size_t gdn_chunk_fwd_workspace(int B, int T, int H, int Dk, int Dv, gdn_dtype dtype) {
    if (!sizes_ok(B, T, H) || !head_ok(Dk) || !head_ok(Dv) || !dtype_ok(dtype)) return 0;
    if (dtype == GDN_BF16) {
        const SegPlan p = seg_plan(B, T, H, Dk, Dv);
        return p.NS ? seg_ws(B, H, Dk, p).total : kAlign;
    }
    return chunk_ws(B, T, H).total;
}

gdn_status gdn_chunk_intra(const void *k, const float *g, const float *beta, float *G2, float *Tinv, int B,
                           int T, int H, int Dk, gdn_dtype dtype, void *stream) {
    if (!k || !g || !beta || !G2 || !Tinv) return GDN_ERR_INVALID_ARG;
    if (!sizes_ok(B, T, H)) return GDN_ERR_INVALID_ARG;
    if (!head_ok(Dk) || !dtype_ok(dtype)) return GDN_ERR_UNSUPPORTED;
    return from_hip(gdn::launch_intra(k, g, beta, G2, Tinv, B, T, H, Dk, dtype == GDN_BF16,
                                      (hipStream_t)stream));
}

gdn_status gdn_chunk_fwd(const void *q, const void *k, const void *v, const float *g, const float *beta,
                         const float *h0, float *o, float *ht, int B, int T, int H, int Dk, int Dv,
                         gdn_dtype dtype, float scale, void *ws, size_t ws_bytes, void *stream) {
    if (!q || !k || !v || !g || !beta || !o) return GDN_ERR_INVALID_ARG;
    if (!sizes_ok(B, T, H)) return GDN_ERR_INVALID_ARG;
    if (!head_ok(Dk) || !head_ok(Dv) || !dtype_ok(dtype)) return GDN_ERR_UNSUPPORTED;
    const size_t es = esize(dtype);
    const size_t ntok = (size_t)B * T * H;
    const size_t nstate = (size_t)B * H * Dk * Dv * sizeof(float);
    const Range rq{q, ntok * Dk * es}, rk{k, ntok * Dk * es}, rv{v, ntok * Dv * es};
    const Range rg{g, ntok * 4}, rb{beta, ntok * 4}, rh0{h0, h0 ? nstate : 0};
    const Range ro{o, ntok * Dv * 4}, rht{ht, ht ? nstate : 0};
    const bool fused = dtype == GDN_BF16;
    // the fused kernel moves q, k, v rows and output rows in 16-byte pieces
    if (fused && (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16)))
        return GDN_ERR_INVALID_ARG;
    const ChunkWs lay = chunk_ws(B, T, H);
    // bf16: the chunk-parallel scan when planned and the workspace holds it
    const SegPlan plan = fused ? seg_plan(B, T, H, Dk, Dv) : SegPlan{0, 0};
    const SegWs slay = plan.NS ? seg_ws(B, H, Dk, plan) : SegWs{0, 0, 0, 0, 0};
    const size_t seg_bytes = slay.total;
    const bool seg = plan.NS && ws && aligned(ws, kAlign) && ws_bytes >= seg_bytes;
    const Range rws{fused ? (seg ? ws : nullptr) : ws, fused ? seg_bytes : lay.total};
    // Outputs may not overlap inputs, each other or the workspace; ht may be exactly h0.
    for (Range in : {rq, rk, rv, rg, rb, rh0, rws})
        if (overlap(ro, in)) return GDN_ERR_INVALID_ARG;
    if (ht) {
        if (overlap(rht, rh0) && ht != h0) return GDN_ERR_INVALID_ARG;
        for (Range in : {rq, rk, rv, rg, rb, ro, rws})
            if (overlap(rht, in)) return GDN_ERR_INVALID_ARG;
    }
    hipStream_t st = (hipStream_t)stream;
    if (seg) {
        for (Range in : {rq, rk, rv, rg, rb, rh0})
            if (overlap(rws, in)) return GDN_ERR_INVALID_ARG;
        char *base = (char *)ws;
        return from_hip(gdn::launch_fused_seg_bf16(q, k, v, g, beta, h0, o, ht, B, T, H, Dk, scale, plan.NS, plan.L,
                                                   (float *)(base + slay.hin), (float *)(base + slay.hout),
                                                   (float *)(base + slay.m), (int *)(base + slay.cu), st));
    }
    if (fused)
        return from_hip(gdn::launch_fused_bf16(q, k, v, g, beta, h0, o, ht, nullptr, B, T, H, Dk, Dv, scale, st));
    if (!ws || ((uintptr_t)ws % kAlign) != 0 || ws_bytes < lay.total) return GDN_ERR_WORKSPACE;
    for (Range in : {rq, rk, rv, rg, rb, rh0})
        if (overlap(rws, in)) return GDN_ERR_INVALID_ARG;

    float *G2 = (float *)((char *)ws + lay.g2_off);
    float *Tinv = (float *)((char *)ws + lay.t_off);
    gdn_status s = from_hip(gdn::launch_intra(k, g, beta, G2, Tinv, B, T, H, Dk, dtype == GDN_BF16, st));
    if (s != GDN_OK) return s;
    return from_hip(gdn::launch_walk(q, k, v, beta, G2, Tinv, h0, o, ht, nullptr, B, T, H, Dk, Dv, dtype == GDN_BF16,
                                     scale, st));
}

gdn_status gdn_chunk_walk(const void *q, const void *k, const void *v, const float *beta, const float *G2,
                          const float *Tinv, const float *h0, float *o, float *ht, int B, int T, int H, int Dk,
                          int Dv, gdn_dtype dtype, float scale, void *stream) {
    if (!q || !k || !v || !beta || !G2 || !Tinv || !o) return GDN_ERR_INVALID_ARG;
    if (!sizes_ok(B, T, H)) return GDN_ERR_INVALID_ARG;
    if (!head_ok(Dk) || !head_ok(Dv) || !dtype_ok(dtype)) return GDN_ERR_UNSUPPORTED;
    const size_t es = esize(dtype);
    const size_t ntok = (size_t)B * T * H;
    const size_t nstate = (size_t)B * H * Dk * Dv * sizeof(float);
    const size_t nchunk = (size_t)B * H * ((T + kBT - 1) / kBT);
    const Range rq{q, ntok * Dk * es}, rk{k, ntok * Dk * es}, rv{v, ntok * Dv * es}, rb{beta, ntok * 4};
    const Range rg2{G2, nchunk * kBT * 4}, rt{Tinv, nchunk * kBT * kBT * 4}, rh0{h0, h0 ? nstate : 0};
    const Range ro{o, ntok * Dv * 4}, rht{ht, ht ? nstate : 0};
    for (Range in : {rq, rk, rv, rb, rg2, rt, rh0})
        if (overlap(ro, in)) return GDN_ERR_INVALID_ARG;
    if (ht) {
        if (overlap(rht, rh0) && ht != h0) return GDN_ERR_INVALID_ARG;
        for (Range in : {rq, rk, rv, rb, rg2, rt, ro})
            if (overlap(rht, in)) return GDN_ERR_INVALID_ARG;
    }
    return from_hip(gdn::launch_walk(q, k, v, beta, G2, Tinv, h0, o, ht, nullptr, B, T, H, Dk, Dv, dtype == GDN_BF16,
                                     scale, (hipStream_t)stream));
}

// Workspace of the GDN-2 forward, per chunk of each head: Ehat, Qhat, Khat
// [64, Dk] in the MFMA operand type (fp16 for bf16 inputs, else fp32),
// Gamma_C [Dk], T - I and strict P [64, 64], diag P [64], all fp32; each
// array 256-byte aligned.
struct Gdn2Ws {
    size_t e_off, q_off, k_off, gam_off, t_off, p_off, d_off, total;
};

static Gdn2Ws gdn2_ws(int B, int T, int H, int Dk, int Dv, gdn_dtype dt) {
    const size_t NT = (size_t)(T + kBT - 1) / kBT;
    const size_t chunks = (size_t)B * H * NT;
    const size_t mts = dt == GDN_BF16 ? 2 : 4;
    Gdn2Ws w;
    size_t off = 0;
    if (dt == GDN_BF16) {  // per-chunk blocks of prepared operands and a state carry (gdn2_fused.hip)
        w = Gdn2Ws{};
        w.total = align_up(gdn::gdn2_fused_ws_bytes(B, T, H, Dk, Dv));
        return w;
    }
    w.e_off = off; off += align_up(chunks * kBT * Dk * mts);
    w.q_off = off; off += align_up(chunks * kBT * Dk * mts);
    w.k_off = off; off += align_up(chunks * kBT * Dk * mts);
    w.gam_off = off; off += align_up(chunks * Dk * 4);
    w.t_off = off; off += align_up(chunks * kBT * kBT * 4);
    w.p_off = off; off += align_up(chunks * kBT * kBT * 4);
    w.d_off = off; off += align_up(chunks * kBT * 4);
    w.total = off;
    return w;
}

size_t gdn2_chunk_fwd_workspace(int B, int T, int H, int Dk, int Dv, gdn_dtype dtype) {
    if (!sizes_ok(B, T, H) || !head_ok(Dk) || !head_ok(Dv) || !dtype_ok(dtype)) return 0;
    return gdn2_ws(B, T, H, Dk, Dv, dtype).total;
}

gdn_status gdn2_chunk_fwd(const void *q, const void *k, const void *v, const float *log_alpha, const void *b,
                          const void *w, const float *h0, float *o, float *ht, int B, int T, int H, int Dk,
                          int Dv, gdn_dtype dtype, float scale, void *ws, size_t ws_bytes, void *stream) {
    if (!q || !k || !v || !log_alpha || !b || !w || !o) return GDN_ERR_INVALID_ARG;
    if (!sizes_ok(B, T, H)) return GDN_ERR_INVALID_ARG;
    if (!head_ok(Dk) || !head_ok(Dv) || !dtype_ok(dtype)) return GDN_ERR_UNSUPPORTED;
    // the bf16 kernels move q, k, v, b, w rows and output rows in 16-byte pieces
    if (dtype == GDN_BF16 && (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(b, 16) ||
                              !aligned(w, 16) || !aligned(o, 16)))
        return GDN_ERR_INVALID_ARG;
    const size_t es = esize(dtype);
    const size_t ntok = (size_t)B * T * H;
    const size_t nstate = (size_t)B * H * Dk * Dv * sizeof(float);
    const Gdn2Ws lay = gdn2_ws(B, T, H, Dk, Dv, dtype);
    const Range rq{q, ntok * Dk * es}, rk{k, ntok * Dk * es}, rv{v, ntok * Dv * es};
    const Range rla{log_alpha, ntok * Dk * 4}, rb{b, ntok * Dk * es}, rw{w, ntok * Dv * es};
    const Range rh0{h0, h0 ? nstate : 0}, ro{o, ntok * Dv * 4}, rht{ht, ht ? nstate : 0}, rws{ws, lay.total};
    for (Range in : {rq, rk, rv, rla, rb, rw, rh0, rws})
        if (overlap(ro, in)) return GDN_ERR_INVALID_ARG;
    if (ht) {
        if (overlap(rht, rh0) && ht != h0) return GDN_ERR_INVALID_ARG;
        for (Range in : {rq, rk, rv, rla, rb, rw, ro, rws})
            if (overlap(rht, in)) return GDN_ERR_INVALID_ARG;
    }
    if (!ws || ((uintptr_t)ws % kAlign) != 0 || ws_bytes < lay.total) return GDN_ERR_WORKSPACE;
    for (Range in : {rq, rk, rv, rla, rb, rw, rh0})
        if (overlap(rws, in)) return GDN_ERR_INVALID_ARG;
    hipStream_t st = (hipStream_t)stream;
    if (dtype == GDN_BF16)
        return from_hip(gdn::launch_gdn2_fused_bf16(q, k, log_alpha, b, v, w, h0, o, ht, ws, B, T, H, Dk, Dv, scale, st));
    char *base = (char *)ws;
    void *E = base + lay.e_off, *Qh = base + lay.q_off, *Kh = base + lay.k_off;
    float *Gam = (float *)(base + lay.gam_off), *Tinv = (float *)(base + lay.t_off);
    float *P = (float *)(base + lay.p_off), *D = (float *)(base + lay.d_off);
    const bool bf = dtype == GDN_BF16;
    gdn_status s = from_hip(gdn::launch_gdn2_intra(q, k, log_alpha, b, E, Qh, Kh, Gam, Tinv, P, D, B, T, H, Dk, bf, st));
    if (s != GDN_OK) return s;
    return from_hip(gdn::launch_gdn2_walk(E, Qh, Kh, Gam, Tinv, P, D, v, w, h0, o, ht, B, T, H, Dk, Dv, bf, scale, st));
}

// Packed sequences for GDN-2: sizes the chunk numbering can hold (every
// prep index h NC + g and every walk workgroup id fits in 32 bits).
static bool var2_sizes_ok(int N, int total_T, int H, int Dv) {
    if (N < 1 || total_T < 1 || H < 1) return false;
    const long long NC = ((long long)total_T + kBT - 1) / kBT + N;
    return (long long)H * NC < (1LL << 31) && (long long)N * H * (Dv / 32 > 0 ? Dv / 32 : 1) < (1LL << 31);
}

size_t gdn2_chunk_fwd_varlen_workspace(int N, int total_T, int H, int Dk, int Dv, gdn_dtype dtype) {
    if (!var2_sizes_ok(N, total_T, H, Dv) || !head_ok(Dk) || !head_ok(Dv) || dtype != GDN_BF16) return 0;
    return gdn::gdn2_var_ws(N, total_T, H, Dk).total;
}

gdn_status gdn2_chunk_fwd_varlen(const void *q, const void *k, const void *v, const float *log_alpha, const void *b,
                                 const void *w, const int *cu_seqlens, const float *h0, float *o, float *ht, int N,
                                 int total_T, int H, int Dk, int Dv, gdn_dtype dtype, float scale, void *ws,
                                 size_t ws_bytes, void *stream) {
    if (!q || !k || !v || !log_alpha || !b || !w || !cu_seqlens || !o) return GDN_ERR_INVALID_ARG;
    if (!var2_sizes_ok(N, total_T, H, Dv)) return GDN_ERR_INVALID_ARG;
    if (!head_ok(Dk) || !head_ok(Dv) || !dtype_ok(dtype)) return GDN_ERR_UNSUPPORTED;
    if (dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(b, 16) || !aligned(w, 16) ||
        !aligned(o, 16))
        return GDN_ERR_INVALID_ARG;
    const size_t es = esize(dtype);
    const size_t ntok = (size_t)total_T * H;
    const size_t nstate = (size_t)N * H * Dk * Dv * sizeof(float);
    const gdn::Gdn2VarWs lay = gdn::gdn2_var_ws(N, total_T, H, Dk);
    const Range rq{q, ntok * Dk * es}, rk{k, ntok * Dk * es}, rv{v, ntok * Dv * es};
    const Range rla{log_alpha, ntok * Dk * 4}, rb{b, ntok * Dk * es}, rw{w, ntok * Dv * es};
    const Range rcu{cu_seqlens, (size_t)(N + 1) * sizeof(int)}, rh0{h0, h0 ? nstate : 0};
    const Range ro{o, ntok * Dv * 4}, rht{ht, ht ? nstate : 0}, rws{ws, lay.total};
    for (Range in : {rq, rk, rv, rla, rb, rw, rcu, rh0, rws})
        if (overlap(ro, in)) return GDN_ERR_INVALID_ARG;
    if (ht) {
        if (overlap(rht, rh0) && ht != h0) return GDN_ERR_INVALID_ARG;
        for (Range in : {rq, rk, rv, rla, rb, rw, rcu, ro, rws})
            if (overlap(rht, in)) return GDN_ERR_INVALID_ARG;
    }
    if (!ws || ((uintptr_t)ws % kAlign) != 0 || ws_bytes < lay.total) return GDN_ERR_WORKSPACE;
    for (Range in : {rq, rk, rv, rla, rb, rw, rcu, rh0})
        if (overlap(rws, in)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_gdn2_fused_varlen_bf16(q, k, log_alpha, b, v, w, cu_seqlens, h0, o, ht, ws, N,
                                                       total_T, H, Dk, Dv, scale, (hipStream_t)stream));
}

gdn_status gdn_recurrent_step(const void *q, const void *k, const void *v, const float *g, const float *beta,
                              float *S, float *o, int B, int H, int Dk, int Dv, gdn_dtype dtype, float scale,
                              void *stream) {
    if (!q || !k || !v || !g || !beta || !S || !o) return GDN_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || (long long)B * H * (Dv / 64 > 0 ? Dv / 64 : 1) >= (1LL << 31))
        return GDN_ERR_INVALID_ARG;
    if (!head_ok(Dk) || !head_ok(Dv) || !dtype_ok(dtype)) return GDN_ERR_UNSUPPORTED;
    const size_t es = esize(dtype);
    const size_t nh = (size_t)B * H;
    const Range rS{S, nh * Dk * Dv * 4}, ro{o, nh * Dv * 4};
    const Range rq{q, nh * Dk * es}, rk{k, nh * Dk * es}, rv{v, nh * Dv * es}, rg{g, nh * 4}, rb{beta, nh * 4};
    for (Range in : {rq, rk, rv, rg, rb, ro})
        if (overlap(rS, in)) return GDN_ERR_INVALID_ARG;
    for (Range in : {rq, rk, rv, rg, rb})
        if (overlap(ro, in)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_step(q, k, v, g, beta, S, o, B, H, Dk, Dv, dtype == GDN_BF16, scale,
                                     (hipStream_t)stream));
}

gdn_status gdn2_recurrent_step(const void *q, const void *k, const void *v, const float *log_alpha, const void *b,
                               const void *w, float *S, float *o, int B, int H, int Dk, int Dv, gdn_dtype dtype,
                               float scale, void *stream) {
    if (!q || !k || !v || !log_alpha || !b || !w || !S || !o) return GDN_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || (long long)B * H * (Dv / 64 > 0 ? Dv / 64 : 1) >= (1LL << 31))
        return GDN_ERR_INVALID_ARG;
    if (!head_ok(Dk) || !head_ok(Dv) || !dtype_ok(dtype)) return GDN_ERR_UNSUPPORTED;
    const size_t es = esize(dtype);
    const size_t nh = (size_t)B * H;
    const Range rS{S, nh * Dk * Dv * 4}, ro{o, nh * Dv * 4};
    const Range rq{q, nh * Dk * es}, rk{k, nh * Dk * es}, rv{v, nh * Dv * es};
    const Range rla{log_alpha, nh * Dk * 4}, rb{b, nh * Dk * es}, rw{w, nh * Dv * es};
    for (Range in : {rq, rk, rv, rla, rb, rw, ro})
        if (overlap(rS, in)) return GDN_ERR_INVALID_ARG;
    for (Range in : {rq, rk, rv, rla, rb, rw})
        if (overlap(ro, in)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_step2(q, k, v, log_alpha, b, w, S, o, B, H, Dk, Dv, dtype == GDN_BF16, scale,
                                      (hipStream_t)stream));
}

gdn_status gdn_chunk_fwd_varlen(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                const int *cu_seqlens, const float *h0, float *o, float *ht, int N, int total_T,
                                int H, int Dk, int Dv, gdn_dtype dtype, float scale, void *stream) {
    if (!q || !k || !v || !g || !beta || !cu_seqlens || !o) return GDN_ERR_INVALID_ARG;
    if (N < 1 || total_T < 1 || H < 1 || (long long)N * H * (Dv / 32 > 0 ? Dv / 32 : 1) >= (1LL << 31))
        return GDN_ERR_INVALID_ARG;
    if (!head_ok(Dk) || !head_ok(Dv) || !dtype_ok(dtype)) return GDN_ERR_UNSUPPORTED;
    if (dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16)) return GDN_ERR_INVALID_ARG;
    const size_t es = esize(dtype);
    const size_t ntok = (size_t)total_T * H;
    const size_t nstate = (size_t)N * H * Dk * Dv * sizeof(float);
    const Range rq{q, ntok * Dk * es}, rk{k, ntok * Dk * es}, rv{v, ntok * Dv * es}, rg{g, ntok * 4},
        rb{beta, ntok * 4}, rcu{cu_seqlens, (size_t)(N + 1) * sizeof(int)}, rh0{h0, h0 ? nstate : 0},
        ro{o, ntok * Dv * 4}, rht{ht, ht ? nstate : 0};
    for (Range in : {rq, rk, rv, rg, rb, rcu, rh0})
        if (overlap(ro, in)) return GDN_ERR_INVALID_ARG;
    if (ht) {
        if (overlap(rht, rh0) && ht != h0) return GDN_ERR_INVALID_ARG;
        for (Range in : {rq, rk, rv, rg, rb, rcu, ro})
            if (overlap(rht, in)) return GDN_ERR_INVALID_ARG;
    }
    return from_hip(gdn::launch_fused_bf16(q, k, v, g, beta, h0, o, ht, cu_seqlens, N, total_T, H, Dk, Dv, scale,
                                           (hipStream_t)stream));
}

// Workspace of the backward: the forward's intra stage (G2, T - I), then the
// entry state and the leaving-state gradient of every chunk, fp32
// [B, H, NT, Dk, Dv] each.
struct BwdWs {
    size_t ck_off, dck_off, g2d_off, total;
};

static BwdWs bwd_ws(int B, int T, int H, int Dk, int Dv) {
    const size_t NT = (size_t)(T + kBT - 1) / kBT;
    const size_t st = align_up((size_t)B * H * NT * Dk * Dv * sizeof(float));
    BwdWs w;
    w.ck_off = chunk_ws(B, T, H).total;
    w.dck_off = w.ck_off + st;
    w.g2d_off = w.dck_off + st;  // fp64 gate sums [B, H, NT, 64]
    w.total = w.g2d_off + align_up((size_t)B * H * NT * kBT * sizeof(double));
    return w;
}

size_t gdn_chunk_bwd_workspace(int B, int T, int H, int Dk, int Dv, gdn_dtype dtype) {
    if (!sizes_ok(B, T, H) || !head_ok(Dk) || !head_ok(Dv) || !dtype_ok(dtype)) return 0;
    return bwd_ws(B, T, H, Dk, Dv).total;
}

gdn_status gdn_chunk_bwd(const void *q, const void *k, const void *v, const float *g, const float *beta,
                         const float *h0, const float *dO, const float *dht, float *dq, float *dk, float *dv,
                         float *dg, float *dbeta, float *dh0, int B, int T, int H, int Dk, int Dv, gdn_dtype dtype,
                         float scale, void *ws, size_t ws_bytes, void *stream) {
    if (!q || !k || !v || !g || !beta || !dO || !dq || !dk || !dv || !dg || !dbeta) return GDN_ERR_INVALID_ARG;
    if (!sizes_ok(B, T, H)) return GDN_ERR_INVALID_ARG;
    if (!head_ok(Dk) || !head_ok(Dv) || !dtype_ok(dtype)) return GDN_ERR_UNSUPPORTED;
    // the bf16 recompute walk reads q, k, v rows in 16-byte pieces
    if (dtype == GDN_BF16 && (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16))) return GDN_ERR_INVALID_ARG;
    const BwdWs lay = bwd_ws(B, T, H, Dk, Dv);
    if (!ws || ((uintptr_t)ws % kAlign) != 0 || ws_bytes < lay.total) return GDN_ERR_WORKSPACE;
    const size_t es = esize(dtype);
    const size_t ntok = (size_t)B * T * H;
    const size_t nstate = (size_t)B * H * Dk * Dv * sizeof(float);
    const Range ins[] = {{q, ntok * Dk * es}, {k, ntok * Dk * es}, {v, ntok * Dv * es}, {g, ntok * 4},
                         {beta, ntok * 4}, {h0, h0 ? nstate : 0}, {dO, ntok * Dv * 4}, {dht, dht ? nstate : 0}};
    const Range outs[] = {{dq, ntok * Dk * 4}, {dk, ntok * Dk * 4}, {dv, ntok * Dv * 4}, {dg, ntok * 4},
                          {dbeta, ntok * 4}, {dh0, dh0 ? nstate : 0}, {ws, lay.total}};
    const int nouts = sizeof(outs) / sizeof(outs[0]);
    for (int a = 0; a < nouts; ++a) {
        for (Range in : ins)
            if (overlap(outs[a], in)) return GDN_ERR_INVALID_ARG;
        for (int c = a + 1; c < nouts; ++c)
            if (overlap(outs[a], outs[c])) return GDN_ERR_INVALID_ARG;
    }
    hipStream_t st = (hipStream_t)stream;
    const ChunkWs cw = chunk_ws(B, T, H);
    char *base = (char *)ws;
    float *G2 = (float *)(base + cw.g2_off), *Tinv = (float *)(base + cw.t_off);
    float *Sck = (float *)(base + lay.ck_off), *dSck = (float *)(base + lay.dck_off);
    const bool bf = dtype == GDN_BF16;
    double *G2d = (double *)(base + lay.g2d_off);
    gdn_status s = from_hip(gdn::launch_intra(k, g, beta, G2, Tinv, B, T, H, Dk, bf, st, true, G2d));
    if (s != GDN_OK) return s;
    // entry state of every chunk: for bf16 inputs the fused forward's walk
    // (bf16 hi + lo state products, T - I and the residuals as fp16 hi + lo),
    // else the staged fp32 walk
    if (bf)
        s = from_hip(gdn::launch_fused_states_bf16(q, k, v, g, beta, Tinv, h0, Sck, B, T, H, Dk, Dv, st));
    else
        s = from_hip(
            gdn::launch_walk(q, k, v, beta, G2, Tinv, h0, nullptr, nullptr, Sck, B, T, H, Dk, Dv, bf, scale, st, true));
    if (s != GDN_OK) return s;
    return from_hip(gdn::launch_bwd(q, k, v, beta, dO, dht, G2d, Tinv, Sck, dSck, dq, dk, dv, dg, dbeta, dh0, B, T, H,
                                    Dk, Dv, bf, scale, st));
}

// Workspace of the GDN-2 backward, fp32 sections each 256-byte aligned:
// Ehat, Qhat, Khat [B,H,NT,64,Dk]; Gamma_C [B,H,NT,Dk]; T - I, P
// [B,H,NT,64,64]; diag(P) [B,H,NT,64]; chunk entry states and leaving-state
// gradients [B,H,NT,Dk,Dv].
struct Bwd2Ws {
    size_t e_off, q_off, k_off, gam_off, t_off, p_off, d_off, ck_off, dck_off, total;
};

static Bwd2Ws bwd2_ws(int B, int T, int H, int Dk, int Dv) {
    const size_t chunks = (size_t)B * H * ((T + kBT - 1) / kBT);
    Bwd2Ws w;
    size_t off = 0;
    w.e_off = off; off += align_up(chunks * kBT * Dk * 4);
    w.q_off = off; off += align_up(chunks * kBT * Dk * 4);
    w.k_off = off; off += align_up(chunks * kBT * Dk * 4);
    w.gam_off = off; off += align_up(chunks * Dk * 4);
    w.t_off = off; off += align_up(chunks * kBT * kBT * 4);
    w.p_off = off; off += align_up(chunks * kBT * kBT * 4);
    w.d_off = off; off += align_up(chunks * kBT * 4);
    w.ck_off = off; off += align_up(chunks * (size_t)Dk * Dv * 4);
    w.dck_off = off; off += align_up(chunks * (size_t)Dk * Dv * 4);
    w.total = off;
    return w;
}

size_t gdn2_chunk_bwd_workspace(int B, int T, int H, int Dk, int Dv, gdn_dtype dtype) {
    if (!sizes_ok(B, T, H) || !head_ok(Dk) || !head_ok(Dv) || !dtype_ok(dtype)) return 0;
    return bwd2_ws(B, T, H, Dk, Dv).total;
}

gdn_status gdn2_chunk_bwd(const void *q, const void *k, const void *v, const float *log_alpha, const void *b,
                          const void *w, const float *h0, const float *dO, const float *dht, float *dq, float *dk,
                          float *dv, float *dlog_alpha, float *db, float *dw, float *dh0, int B, int T, int H, int Dk,
                          int Dv, gdn_dtype dtype, float scale, void *ws, size_t ws_bytes, void *stream) {
    if (!q || !k || !v || !log_alpha || !b || !w || !dO || !dq || !dk || !dv || !dlog_alpha || !db || !dw)
        return GDN_ERR_INVALID_ARG;
    if (!sizes_ok(B, T, H)) return GDN_ERR_INVALID_ARG;
    if (!head_ok(Dk) || !head_ok(Dv) || !dtype_ok(dtype)) return GDN_ERR_UNSUPPORTED;
    // the bf16 path moves q, k, b, log_alpha, v and w rows in 16-byte pieces
    if (dtype == GDN_BF16 && (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(b, 16) ||
                              !aligned(w, 16) || !aligned(log_alpha, 16)))
        return GDN_ERR_INVALID_ARG;
    const Bwd2Ws lay = bwd2_ws(B, T, H, Dk, Dv);
    if (!ws || ((uintptr_t)ws % kAlign) != 0 || ws_bytes < lay.total) return GDN_ERR_WORKSPACE;
    const size_t es = esize(dtype);
    const size_t ntok = (size_t)B * T * H;
    const size_t nstate = (size_t)B * H * Dk * Dv * sizeof(float);
    const Range ins[] = {{q, ntok * Dk * es}, {k, ntok * Dk * es}, {v, ntok * Dv * es}, {log_alpha, ntok * Dk * 4},
                         {b, ntok * Dk * es}, {w, ntok * Dv * es}, {h0, h0 ? nstate : 0}, {dO, ntok * Dv * 4},
                         {dht, dht ? nstate : 0}};
    const Range outs[] = {{dq, ntok * Dk * 4}, {dk, ntok * Dk * 4}, {dv, ntok * Dv * 4}, {dlog_alpha, ntok * Dk * 4},
                          {db, ntok * Dk * 4}, {dw, ntok * Dv * 4}, {dh0, dh0 ? nstate : 0}, {ws, lay.total}};
    const int nouts = sizeof(outs) / sizeof(outs[0]);
    for (int a = 0; a < nouts; ++a) {
        for (Range in : ins)
            if (overlap(outs[a], in)) return GDN_ERR_INVALID_ARG;
        for (int c = a + 1; c < nouts; ++c)
            if (overlap(outs[a], outs[c])) return GDN_ERR_INVALID_ARG;
    }
    hipStream_t st = (hipStream_t)stream;
    char *base = (char *)ws;
    float *Eh = (float *)(base + lay.e_off), *Qh = (float *)(base + lay.q_off), *Kh = (float *)(base + lay.k_off);
    float *Gam = (float *)(base + lay.gam_off), *Tm = (float *)(base + lay.t_off), *P = (float *)(base + lay.p_off);
    float *D = (float *)(base + lay.d_off), *Sck = (float *)(base + lay.ck_off), *dSck = (float *)(base + lay.dck_off);
    const bool bf = dtype == GDN_BF16;
    gdn_status s = from_hip(gdn::launch_gdn2_recompute(q, k, log_alpha, b, v, w, h0, Eh, Qh, Kh, Gam, Tm, P, D, Sck,
                                                       B, T, H, Dk, Dv, bf, st));
    if (s != GDN_OK) return s;
    return from_hip(gdn::launch_gdn2_bwd(q, k, v, log_alpha, b, w, dO, dht, Eh, Qh, Kh, Gam, Tm, P, D, Sck, dSck, dq,
                                         dk, dv, dlog_alpha, db, dw, dh0, B, T, H, Dk, Dv, bf, scale, st));
}

gdn_status gdn_prologue(const void *xq, const void *xk, const void *xv, const float *a, const float *b,
                        const float *wq, const float *wk, const float *wv, const float *A_log, const float *dt_bias,
                        const float *conv_in, void *q, void *k, void *v, float *g, float *beta, float *conv_out,
                        int B, int T, int H, int Dk, int Dv, void *stream) {
    if (!xq || !xk || !xv || !a || !b || !wq || !wk || !wv || !A_log || !dt_bias || !q || !k || !v || !g || !beta)
        return GDN_ERR_INVALID_ARG;
    if (B < 1 || T < 1 || H < 1 || (long long)B * T * H >= (1LL << 33)) return GDN_ERR_INVALID_ARG;
    if (!head_ok(Dk) || !head_ok(Dv)) return GDN_ERR_UNSUPPORTED;
    for (const void *p : {xq, xk, xv, (const void *)q, (const void *)k, (const void *)v, (const void *)wq,
                          (const void *)wk, (const void *)wv, (const void *)conv_in})
        if (!aligned(p, 16)) return GDN_ERR_INVALID_ARG;
    if (!aligned(conv_out, 4)) return GDN_ERR_INVALID_ARG;
    const size_t ntok = (size_t)B * T * H, C = (size_t)H * (2 * Dk + Dv);
    const size_t nstate = (size_t)B * 3 * C * sizeof(float);
    const Range rxq{xq, ntok * Dk * 2}, rxk{xk, ntok * Dk * 2}, rxv{xv, ntok * Dv * 2}, ra{a, ntok * 4},
        rb{b, ntok * 4}, rwq{wq, (size_t)H * Dk * 16}, rwk{wk, (size_t)H * Dk * 16}, rwv{wv, (size_t)H * Dv * 16},
        rA{A_log, (size_t)H * 4}, rdt{dt_bias, (size_t)H * 4}, rci{conv_in, conv_in ? nstate : 0},
        rq{q, ntok * Dk * 2}, rk{k, ntok * Dk * 2}, rv{v, ntok * Dv * 2}, rg{g, ntok * 4}, rbe{beta, ntok * 4},
        rco{conv_out, conv_out ? nstate : 0};
    const Range ins[] = {rxq, rxk, rxv, ra, rb, rwq, rwk, rwv, rA, rdt, rci};
    const Range outs[] = {rq, rk, rv, rg, rbe};
    for (int i = 0; i < 5; ++i) {
        for (Range in : ins)
            if (overlap(outs[i], in)) return GDN_ERR_INVALID_ARG;
        for (int j = i + 1; j < 5; ++j)
            if (overlap(outs[i], outs[j])) return GDN_ERR_INVALID_ARG;
        if (overlap(outs[i], rco)) return GDN_ERR_INVALID_ARG;
    }
    if (conv_out) {
        if (overlap(rco, rci) && conv_out != conv_in) return GDN_ERR_INVALID_ARG;
        for (int i = 0; i < 10; ++i)
            if (overlap(rco, ins[i])) return GDN_ERR_INVALID_ARG;
    }
    return from_hip(gdn::launch_prologue(xq, xk, xv, a, b, wq, wk, wv, A_log, dt_bias, conv_in, q, k, v, g, beta,
                                         conv_out, B, T, H, Dk, Dv, (hipStream_t)stream));
}

gdn_status gdn_gated_rmsnorm(const float *o, const void *z, const float *weight, void *y, long long rows, int Dv,
                             float eps, void *stream) {
    if (!o || !z || !weight || !y || rows < 1 || rows >= (1LL << 33) || !(eps > 0.f)) return GDN_ERR_INVALID_ARG;
    if (!head_ok(Dv)) return GDN_ERR_UNSUPPORTED;
    if (!aligned(o, 16) || !aligned(z, 16) || !aligned(weight, 16) || !aligned(y, 16)) return GDN_ERR_INVALID_ARG;
    const Range ry{y, (size_t)rows * Dv * 2};
    for (Range in : {Range{o, (size_t)rows * Dv * 4}, Range{z, (size_t)rows * Dv * 2}, Range{weight, (size_t)Dv * 4}})
        if (overlap(ry, in)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_gated_rmsnorm(o, z, weight, y, (long)rows, Dv, eps, (hipStream_t)stream));
}

// Element size of the types the norm and linear entry points take.
static size_t esize3(gdn_dtype dt) { return dt == GDN_F32 ? 4 : dt == GDN_BF16 ? 2 : 1; }

static bool norm_types_ok(gdn_dtype dtype, gdn_dtype rdtype) {
    return dtype_ok(dtype) && dtype_ok(rdtype) && (rdtype == GDN_F32 || dtype == GDN_BF16);
}

// rows * D elements of 4 bytes must stay within an address range
static bool rows_ok(long long rows, int D) { return rows >= 1 && D >= 1 && rows < (1LL << 40); }

gdn_status gdn_add_rmsnorm(const void *x, const void *residual, const float *weight, void *y, void *r, float *rstd,
                           float *y_scale, long long rows, int D, gdn_dtype dtype, gdn_dtype rdtype,
                           gdn_dtype out_dtype, float eps, void *stream) {
    if (!x || !weight || !y || !rows_ok(rows, D) || !(eps > 0.f)) return GDN_ERR_INVALID_ARG;
    if (!norm_types_ok(dtype, rdtype) || D > gdn::kMaxNormCols) return GDN_ERR_UNSUPPORTED;
    const bool f8 = out_dtype == GDN_F8E4M3;
    if (!f8 && out_dtype != dtype) return GDN_ERR_UNSUPPORTED;
    if (f8 != (y_scale != nullptr) || (r && !residual)) return GDN_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(r, 16) || !aligned(y, f8 ? 8 : 16) || !aligned(weight, 4) ||
        !aligned(rstd, 4) || !aligned(y_scale, 4))
        return GDN_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * D;
    const Range ins[] = {{x, n * esize3(dtype)}, {weight, (size_t)D * 4}, {residual, n * esize3(rdtype)}};
    const Range outs[] = {{y, n * esize3(out_dtype)}, {rstd, (size_t)rows * 4}, {y_scale, (size_t)rows * 4},
                          {r, n * esize3(rdtype)}};
    for (int a = 0; a < 4; ++a) {
        for (int c = 0; c < 3; ++c)
            if (overlap(outs[a], ins[c]) && !(a == 3 && c == 2 && r == residual)) return GDN_ERR_INVALID_ARG;
        for (int c = a + 1; c < 4; ++c)
            if (overlap(outs[a], outs[c])) return GDN_ERR_INVALID_ARG;
    }
    return from_hip(gdn::launch_add_rmsnorm(x, residual, weight, y, r, rstd, y_scale, (long)rows, D,
                                            dtype == GDN_BF16, rdtype == GDN_BF16, f8, eps, (hipStream_t)stream));
}

size_t gdn_add_rmsnorm_bwd_workspace(long long rows, int D) {
    if (!rows_ok(rows, D) || D > gdn::kMaxNormCols) return 0;
    return align_up((size_t)gdn::norm_bwd_blocks((long)rows, D) * D * sizeof(float));
}

gdn_status gdn_add_rmsnorm_bwd(const void *dy, const void *r, const float *weight, const float *rstd, const void *dr,
                               void *dx, float *dweight, long long rows, int D, gdn_dtype dtype, gdn_dtype rdtype,
                               void *ws, size_t ws_bytes, void *stream) {
    if (!dy || !r || !weight || !rstd || !dx || !rows_ok(rows, D)) return GDN_ERR_INVALID_ARG;
    if (!norm_types_ok(dtype, rdtype) || D > gdn::kMaxNormCols) return GDN_ERR_UNSUPPORTED;
    if (!aligned(dy, 16) || !aligned(r, 16) || !aligned(dr, 16) || !aligned(dx, 16) || !aligned(weight, 4) ||
        !aligned(rstd, 4) || !aligned(dweight, 4))
        return GDN_ERR_INVALID_ARG;
    const size_t need = dweight ? gdn_add_rmsnorm_bwd_workspace(rows, D) : 0;
    if (dweight && (!ws || !aligned(ws, kAlign) || ws_bytes < need)) return GDN_ERR_WORKSPACE;
    const size_t n = (size_t)rows * D;
    const Range ins[] = {{dy, n * esize3(dtype)}, {r, n * esize3(rdtype)}, {weight, (size_t)D * 4},
                         {rstd, (size_t)rows * 4}, {dr, n * esize3(rdtype)}};
    const Range outs[] = {{dx, n * esize3(rdtype)}, {dweight, (size_t)D * 4}, {dweight ? ws : nullptr, need}};
    for (int a = 0; a < 3; ++a) {
        for (Range in : ins)
            if (overlap(outs[a], in)) return GDN_ERR_INVALID_ARG;
        for (int c = a + 1; c < 3; ++c)
            if (overlap(outs[a], outs[c])) return GDN_ERR_INVALID_ARG;
    }
    return from_hip(gdn::launch_add_rmsnorm_bwd(dy, r, weight, rstd, dr, dx, dweight, (float *)ws, (long)rows, D,
                                                dtype == GDN_BF16, rdtype == GDN_BF16, (hipStream_t)stream));
}

gdn_status gdn_quantize_rows(const void *x, void *q, float *scale, long long rows, int D, gdn_dtype dtype,
                             void *stream) {
    if (!x || !q || !scale || !rows_ok(rows, D)) return GDN_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || D > gdn::kMaxNormCols) return GDN_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(q, 8) || !aligned(scale, 4)) return GDN_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * D;
    const Range rx{x, n * esize3(dtype)}, rq{q, n}, rs{scale, (size_t)rows * 4};
    if (overlap(rq, rx) || overlap(rs, rx) || overlap(rq, rs)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_quantize_rows(x, q, scale, (long)rows, D, dtype == GDN_BF16, (hipStream_t)stream));
}

gdn_status gdn_add_layernorm(const void *x, const void *residual, const float *weight, const float *bias, void *y,
                             void *r, float *mean, float *rstd, float *y_scale, long long rows, int D,
                             gdn_dtype dtype, gdn_dtype rdtype, gdn_dtype out_dtype, float eps, void *stream) {
    if (!x || !weight || !y || !rows_ok(rows, D) || !(eps > 0.f)) return GDN_ERR_INVALID_ARG;
    if (!norm_types_ok(dtype, rdtype) || D > gdn::kMaxNormCols) return GDN_ERR_UNSUPPORTED;
    const bool f8 = out_dtype == GDN_F8E4M3;
    if (!f8 && out_dtype != dtype) return GDN_ERR_UNSUPPORTED;
    if (f8 != (y_scale != nullptr) || (r && !residual)) return GDN_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(r, 16) || !aligned(y, f8 ? 8 : 16) || !aligned(weight, 4) ||
        !aligned(bias, 4) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(y_scale, 4))
        return GDN_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * D;
    const Range ins[] = {{x, n * esize3(dtype)}, {weight, (size_t)D * 4}, {bias, (size_t)D * 4},
                         {r == residual ? nullptr : residual, n * esize3(rdtype)}};
    const Range outs[] = {{y, n * esize3(out_dtype)}, {mean, (size_t)rows * 4}, {rstd, (size_t)rows * 4},
                          {y_scale, (size_t)rows * 4}, {r, n * esize3(rdtype)}};
    if (!disjoint(ins, outs)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_add_layernorm(x, residual, weight, bias, y, r, mean, rstd, y_scale, (long)rows, D,
                                              dtype == GDN_BF16, rdtype == GDN_BF16, f8, eps, (hipStream_t)stream));
}

size_t gdn_add_layernorm_bwd_workspace(long long rows, int D) {
    if (!rows_ok(rows, D) || D > gdn::kMaxNormCols) return 0;
    return align_up((size_t)gdn::ln_bwd_blocks((long)rows, D) * 2 * D * sizeof(float));
}

gdn_status gdn_add_layernorm_bwd(const void *dy, const void *r, const float *weight, const float *mean,
                                 const float *rstd, const void *dr, void *dx, float *dweight, float *dbias,
                                 long long rows, int D, gdn_dtype dtype, gdn_dtype rdtype, void *ws, size_t ws_bytes,
                                 void *stream) {
    if (!dy || !r || !weight || !mean || !rstd || !dx || !rows_ok(rows, D)) return GDN_ERR_INVALID_ARG;
    if (!norm_types_ok(dtype, rdtype) || D > gdn::kMaxNormCols) return GDN_ERR_UNSUPPORTED;
    if (!aligned(dy, 16) || !aligned(r, 16) || !aligned(dr, 16) || !aligned(dx, 16) || !aligned(weight, 4) ||
        !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dbias, 4))
        return GDN_ERR_INVALID_ARG;
    const bool sums = dweight || dbias;
    const size_t need = sums ? gdn_add_layernorm_bwd_workspace(rows, D) : 0;
    if (sums && (!ws || !aligned(ws, kAlign) || ws_bytes < need)) return GDN_ERR_WORKSPACE;
    const size_t n = (size_t)rows * D;
    const Range ins[] = {{dy, n * esize3(dtype)}, {r, n * esize3(rdtype)}, {weight, (size_t)D * 4},
                         {mean, (size_t)rows * 4}, {rstd, (size_t)rows * 4}, {dr, n * esize3(rdtype)}};
    const Range outs[] = {{dx, n * esize3(rdtype)}, {dweight, (size_t)D * 4}, {dbias, (size_t)D * 4},
                          {sums ? ws : nullptr, need}};
    if (!disjoint(ins, outs)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_add_layernorm_bwd(dy, r, weight, mean, rstd, dr, dx, dweight, dbias, (float *)ws,
                                                  (long)rows, D, dtype == GDN_BF16, rdtype == GDN_BF16,
                                                  (hipStream_t)stream));
}

// Sizes of a product the kernels index: 32-bit offsets within a tile of 256
// rows (N, K), a grid of fewer than 2^32 threads (the tiles of each output:
// M x N in the forward, M x K and N x K in the backward, which reads M x N).
static bool mm_sizes_ok(int M, int N, int K, bool bwd) {
    auto tiles = [](long long a, long long b) { return ((a + 255) / 256) * ((b + 255) / 256) < (1LL << 21); };
    return N <= (1 << 22) && K <= (1 << 22) && tiles(M, N) && (!bwd || (tiles(M, K) && tiles(N, K)));
}

static bool act_ok(gdn_act a) { return a >= GDN_ACT_NONE && a <= GDN_ACT_GELU; }

static gdn_status linear_check(int M, int N, int K, gdn_dtype dtype, bool bwd) {
    if (M < 1 || N < 1 || K < 1) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_F8E4M3) return GDN_ERR_UNSUPPORTED;
    if (K % (dtype == GDN_BF16 ? 8 : 16) || !mm_sizes_ok(M, N, K, bwd)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

size_t gdn_linear_workspace(int M, int N, int K, gdn_dtype dtype) {
    if (linear_check(M, N, K, dtype, false) != GDN_OK) return 0;
    return align_up(gdn::linear_ws_bytes(gdn::linear_plan(M, N, K, dtype == GDN_F8E4M3), M, N));
}

gdn_status gdn_linear(const void *x, const void *w, const float *x_scale, const float *w_scale, const float *bias,
                      const void *residual, void *y, void *z, int M, int N, int K, gdn_dtype dtype,
                      gdn_dtype out_dtype, gdn_act act, void *ws, size_t ws_bytes, void *stream) {
    if (!x || !w || !y) return GDN_ERR_INVALID_ARG;
    const gdn_status st = linear_check(M, N, K, dtype, false);
    if (st != GDN_OK) return st;
    if (!dtype_ok(out_dtype) || !act_ok(act)) return GDN_ERR_UNSUPPORTED;
    const bool f8 = dtype == GDN_F8E4M3;
    if (f8 != (x_scale != nullptr) || f8 != (w_scale != nullptr)) return GDN_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(residual, 16) || !aligned(y, 16) || !aligned(z, 16) ||
        !aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4))
        return GDN_ERR_INVALID_ARG;
    const gdn::MmPlan plan = gdn::linear_plan(M, N, K, f8);
    const size_t need = align_up(gdn::linear_ws_bytes(plan, M, N));
    if (need && (!ws || !aligned(ws, kAlign) || ws_bytes < need)) return GDN_ERR_WORKSPACE;
    const size_t mn = (size_t)M * N;
    const Range ins[] = {{x, (size_t)M * K * esize3(dtype)}, {w, (size_t)N * K * esize3(dtype)},
                         {x_scale, (size_t)M * 4}, {w_scale, (size_t)N * 4}, {bias, (size_t)N * 4},
                         {residual == y ? nullptr : residual, mn * esize3(out_dtype)}};
    const Range outs[] = {{y, mn * esize3(out_dtype)}, {z, mn * 2}, {need ? ws : nullptr, need}};
    if (!disjoint(ins, outs)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_linear(plan, x, w, x_scale, w_scale, bias, residual, y, z, M, N, K, f8, out_dtype == GDN_F32,
                                       (int)act, (float *)ws, (hipStream_t)stream));
}

size_t gdn_linear_bwd_workspace(int M, int N, int K, gdn_dtype dy_dtype, gdn_dtype grad_dtype, gdn_act act,
                                int need_dx, int need_dw, int need_dbias) {
    if (linear_check(M, N, K, GDN_BF16, true) != GDN_OK || !dtype_ok(dy_dtype) || !dtype_ok(grad_dtype) || !act_ok(act))
        return 0;
    return gdn::linear_bwd_plan(M, N, K, dy_dtype == GDN_F32, grad_dtype == GDN_F32, (int)act, need_dx != 0,
                                need_dw != 0, need_dbias != 0)
        .total;
}

gdn_status gdn_linear_bwd(const void *dy, const void *x, const void *w, const void *z, void *dx, void *dw,
                          float *dbias, int M, int N, int K, gdn_dtype dy_dtype, gdn_dtype grad_dtype, gdn_act act,
                          void *ws, size_t ws_bytes, void *stream) {
    if (!dy || !x || !w || (!dx && !dw && !dbias)) return GDN_ERR_INVALID_ARG;
    const gdn_status st = linear_check(M, N, K, GDN_BF16, true);
    if (st != GDN_OK) return st;
    if (!dtype_ok(dy_dtype) || !dtype_ok(grad_dtype) || !act_ok(act)) return GDN_ERR_UNSUPPORTED;
    if ((act != GDN_ACT_NONE) != (z != nullptr)) return GDN_ERR_INVALID_ARG;
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(w, 16) || !aligned(z, 16) || !aligned(dx, 16) ||
        !aligned(dw, 16) || !aligned(dbias, 4))
        return GDN_ERR_INVALID_ARG;
    const gdn::LinearBwdPlan plan = gdn::linear_bwd_plan(M, N, K, dy_dtype == GDN_F32, grad_dtype == GDN_F32, (int)act,
                                                         dx != nullptr, dw != nullptr, dbias != nullptr);
    const size_t need = plan.total;
    if (need && (!ws || !aligned(ws, kAlign) || ws_bytes < need)) return GDN_ERR_WORKSPACE;
    const size_t mn = (size_t)M * N, mk = (size_t)M * K, nk = (size_t)N * K;
    const Range ins[] = {{dy, mn * esize3(dy_dtype)}, {x, mk * 2}, {w, nk * 2}, {z, mn * 2}};
    const Range outs[] = {{dx, mk * esize3(grad_dtype)}, {dw, nk * esize3(grad_dtype)}, {dbias, (size_t)N * 4},
                          {need ? ws : nullptr, need}};
    if (!disjoint(ins, outs)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_linear_bwd(plan, dy, x, w, z, dx, dw, dbias, M, N, K, dy_dtype == GDN_F32,
                                           grad_dtype == GDN_F32, (int)act, (char *)ws, (hipStream_t)stream));
}

// A gated product is one of 2 N columns.
static gdn_status gated_check(int M, int N, int K, gdn_dtype dtype, bool bwd) {
    if (N < 1) return GDN_ERR_INVALID_ARG;
    return linear_check(M, N > (1 << 21) ? (1 << 22) + 1 : 2 * N, K, dtype, bwd);  // too many columns either way
}

size_t gdn_gated_linear_workspace(int M, int N, int K, gdn_dtype dtype) {
    if (gated_check(M, N, K, dtype, false) != GDN_OK) return 0;
    return align_up(gdn::linear_ws_bytes(gdn::linear_plan(M, 2 * N, K, dtype == GDN_F8E4M3), M, 2 * N));
}

gdn_status gdn_gated_linear(const void *x, const void *w, const float *x_scale, const float *w_scale,
                            const float *bias, void *y, void *z, int M, int N, int K, gdn_dtype dtype,
                            gdn_dtype out_dtype, gdn_act act, void *ws, size_t ws_bytes, void *stream) {
    if (!x || !w || !y) return GDN_ERR_INVALID_ARG;
    const gdn_status st = gated_check(M, N, K, dtype, false);
    if (st != GDN_OK) return st;
    if (!dtype_ok(out_dtype) || !act_ok(act)) return GDN_ERR_UNSUPPORTED;
    const bool f8 = dtype == GDN_F8E4M3;
    if (f8 != (x_scale != nullptr) || f8 != (w_scale != nullptr)) return GDN_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16) || !aligned(z, 16) || !aligned(x_scale, 4) ||
        !aligned(w_scale, 4) || !aligned(bias, 4))
        return GDN_ERR_INVALID_ARG;
    const gdn::MmPlan plan = gdn::linear_plan(M, 2 * N, K, f8);
    const size_t need = align_up(gdn::linear_ws_bytes(plan, M, 2 * N));
    if (need && (!ws || !aligned(ws, kAlign) || ws_bytes < need)) return GDN_ERR_WORKSPACE;
    const size_t mn = (size_t)M * N;
    const Range ins[] = {{x, (size_t)M * K * esize3(dtype)}, {w, (size_t)2 * N * K * esize3(dtype)},
                         {x_scale, (size_t)M * 4}, {w_scale, (size_t)N * 8}, {bias, (size_t)N * 8}};
    const Range outs[] = {{y, mn * esize3(out_dtype)}, {z, mn * 4}, {need ? ws : nullptr, need}};
    if (!disjoint(ins, outs)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_gated_linear(plan, x, w, x_scale, w_scale, bias, y, z, M, N, K, f8, out_dtype == GDN_F32,
                                             (int)act, (float *)ws, (hipStream_t)stream));
}

size_t gdn_gated_linear_bwd_workspace(int M, int N, int K, gdn_dtype dy_dtype, gdn_dtype grad_dtype, gdn_act act,
                                      int need_dx, int need_dw, int need_dbias) {
    if (gated_check(M, N, K, GDN_BF16, true) != GDN_OK || !dtype_ok(dy_dtype) || !dtype_ok(grad_dtype) || !act_ok(act))
        return 0;
    return gdn::gated_linear_bwd_plan(M, N, K, grad_dtype == GDN_F32, need_dx != 0, need_dw != 0, need_dbias != 0).total;
}

gdn_status gdn_gated_linear_bwd(const void *dy, const void *x, const void *w, const void *z, void *dx, void *dw,
                                float *dbias, int M, int N, int K, gdn_dtype dy_dtype, gdn_dtype grad_dtype,
                                gdn_act act, void *ws, size_t ws_bytes, void *stream) {
    if (!dy || !x || !w || !z || (!dx && !dw && !dbias)) return GDN_ERR_INVALID_ARG;
    const gdn_status st = gated_check(M, N, K, GDN_BF16, true);
    if (st != GDN_OK) return st;
    if (!dtype_ok(dy_dtype) || !dtype_ok(grad_dtype) || !act_ok(act)) return GDN_ERR_UNSUPPORTED;
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(w, 16) || !aligned(z, 16) || !aligned(dx, 16) ||
        !aligned(dw, 16) || !aligned(dbias, 4))
        return GDN_ERR_INVALID_ARG;
    const gdn::LinearBwdPlan plan = gdn::gated_linear_bwd_plan(M, N, K, grad_dtype == GDN_F32, dx != nullptr,
                                                               dw != nullptr, dbias != nullptr);
    const size_t need = plan.total;
    if (!ws || !aligned(ws, kAlign) || ws_bytes < need) return GDN_ERR_WORKSPACE;
    const size_t mn = (size_t)M * N, mk = (size_t)M * K, nk = (size_t)2 * N * K;
    const Range ins[] = {{dy, mn * esize3(dy_dtype)}, {x, mk * 2}, {w, nk * 2}, {z, mn * 4}};
    const Range outs[] = {{dx, mk * esize3(grad_dtype)}, {dw, nk * esize3(grad_dtype)}, {dbias, (size_t)N * 8},
                          {ws, need}};
    if (!disjoint(ins, outs)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_gated_linear_bwd(plan, dy, x, w, z, dx, dw, dbias, M, N, K, dy_dtype == GDN_F32,
                                                 grad_dtype == GDN_F32, (int)act, (char *)ws, (hipStream_t)stream));
}

static void plan_ints(const gdn::MmPlan &p, int *out) {
    out[0] = p.tile;
    out[1] = p.splits;
    out[2] = p.per_split;
    out[3] = p.tile ? (p.deep ? 4 : 2) : 0;
}

gdn_status gdn_linear_plan(int M, int N, int K, gdn_dtype dtype, int *plan) {
    if (!plan) return GDN_ERR_INVALID_ARG;
    const gdn_status st = linear_check(M, N, K, dtype, false);
    if (st != GDN_OK) return st;
    plan_ints(gdn::linear_plan(M, N, K, dtype == GDN_F8E4M3), plan);
    return GDN_OK;
}

gdn_status gdn_linear_bwd_plan(int M, int N, int K, gdn_dtype dy_dtype, gdn_dtype grad_dtype, gdn_act act, int need_dx,
                               int need_dw, int need_dbias, int *plan) {
    if (!plan) return GDN_ERR_INVALID_ARG;
    const gdn_status st = linear_check(M, N, K, GDN_BF16, true);
    if (st != GDN_OK) return st;
    if (!dtype_ok(dy_dtype) || !dtype_ok(grad_dtype) || !act_ok(act)) return GDN_ERR_UNSUPPORTED;
    const gdn::LinearBwdPlan p = gdn::linear_bwd_plan(M, N, K, dy_dtype == GDN_F32, grad_dtype == GDN_F32, (int)act,
                                                      need_dx != 0, need_dw != 0, need_dbias != 0);
    plan[0] = p.planes;
    plan[1] = p.pair ? (p.deep ? 4 : 2) : 0;
    plan_ints(p.dx, plan + 2);
    plan_ints(p.dw, plan + 6);
    return GDN_OK;
}

static gdn_status conv_call(const void *x, const float *w, const float *bias, const int *cu, const float *state_in,
                            void *y, float *state_out, int seqs, int T, long long total, int C, int W,
                            gdn_dtype dtype, gdn_act act, void *stream) {
    if (!x || !w || !y || seqs < 1 || T < 1 || C < 1) return GDN_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || W < 2 || W > 4 || (act != GDN_ACT_NONE && act != GDN_ACT_SILU)) return GDN_ERR_UNSUPPORTED;
    const long long octets = ((long long)C + 7) / 8;
    // the kernels count channels past the last octet's end in 32 bits
    if (C > INT_MAX - 16 || total > (1 << 30) || total * octets >= (1LL << 32) - 256 || seqs * octets >= (1LL << 32) - 256)
        return GDN_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(w, 4) || !aligned(bias, 4) || !aligned(cu, 4) ||
        !aligned(state_in, 4) || !aligned(state_out, 4))
        return GDN_ERR_INVALID_ARG;
    const size_t n = (size_t)total * C * esize(dtype), ns = (size_t)seqs * (W - 1) * C * 4;
    const Range ins[] = {{x, n}, {w, (size_t)C * W * 4}, {bias, (size_t)C * 4}, {cu, cu ? (size_t)(seqs + 1) * 4 : 0},
                         {state_in == state_out ? nullptr : state_in, ns}};
    const Range outs[] = {{y, n}, {state_out, ns}};
    if (!disjoint(ins, outs) || overlap({y, n}, {state_in, ns})) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_causal_conv(x, w, bias, state_in, y, state_out, cu, seqs, T, (int)total, C, W,
                                            dtype == GDN_BF16, act == GDN_ACT_SILU, (hipStream_t)stream));
}

gdn_status gdn_causal_conv(const void *x, const float *w, const float *bias, const float *state_in, void *y,
                           float *state_out, int B, int T, int C, int W, gdn_dtype dtype, gdn_act act, void *stream) {
    return conv_call(x, w, bias, nullptr, state_in, y, state_out, B, T, (long long)B * T, C, W, dtype, act, stream);
}

gdn_status gdn_causal_conv_varlen(const void *x, const float *w, const float *bias, const int *cu_seqlens,
                                  const float *state_in, void *y, float *state_out, int N, int total_T, int C, int W,
                                  gdn_dtype dtype, gdn_act act, void *stream) {
    if (!cu_seqlens) return GDN_ERR_INVALID_ARG;
    return conv_call(x, w, bias, cu_seqlens, state_in, y, state_out, N, total_T, total_T, C, W, dtype, act, stream);
}

// Sizes of a scan: 32-bit token numbers, a grid of fewer than 2^32 threads.
static gdn_status scan_check(int seqs, int T, long long total, int ch, int N, bool packed) {
    if (seqs < 1 || T < 1 || ch < 1 || N < 1) return GDN_ERR_INVALID_ARG;
    if ((N != 8 && N != 16 && N != 32 && N != 64) || total > (1 << 30) || ch < 4 || ch > (1 << 24))
        return GDN_ERR_UNSUPPORTED;
    const gdn::ScanPlan p = gdn::scan_plan(seqs, T, (int)total, ch, N, packed);
    return (long long)p.segs * ((ch + 63) / 64) < (1LL << 23) ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

size_t gdn_selective_scan_workspace(int B, int T, int ch, int N) {
    if (scan_check(B, T, (long long)B * T, ch, N, false) != GDN_OK) return 0;
    return gdn::scan_plan(B, T, B * T, ch, N, false).total;
}

size_t gdn_selective_scan_varlen_workspace(int seqs, int total_T, int ch, int N) {
    if (scan_check(seqs, total_T, total_T, ch, N, true) != GDN_OK) return 0;
    return gdn::scan_plan(seqs, total_T, total_T, ch, N, true).total;
}

static gdn_status scan_call(const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                            const int *cu, const float *D, const void *z, const float *dt_bias, const float *h0, void *y,
                            float *ht, int seqs, int T, long long total, int ch, int N, gdn_dtype dtype, void *ws,
                            size_t ws_bytes, void *stream) {
    if (!x || !dt || !A || !Bm || !Cm || !y) return GDN_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return GDN_ERR_UNSUPPORTED;
    const gdn_status st = scan_check(seqs, T, total, ch, N, cu != nullptr);
    if (st != GDN_OK) return st;
    for (const void *p : {x, dt, (const void *)A, Bm, Cm, z, (const void *)h0, (const void *)y, (const void *)ht})
        if (!aligned(p, 16)) return GDN_ERR_INVALID_ARG;
    if (!aligned(D, 4) || !aligned(dt_bias, 4) || !aligned(cu, 4)) return GDN_ERR_INVALID_ARG;
    const gdn::ScanPlan plan = gdn::scan_plan(seqs, T, (int)total, ch, N, cu != nullptr);
    const size_t need = plan.total;
    if (need && (!ws || !aligned(ws, kAlign) || ws_bytes < need)) return GDN_ERR_WORKSPACE;
    const size_t es = esize(dtype), n = (size_t)total * ch * es, nb = (size_t)total * N * es;
    const size_t ns = (size_t)seqs * ch * N * 4;
    const Range ins[] = {{x, n}, {dt, n}, {A, (size_t)ch * N * 4}, {Bm, nb}, {Cm, nb}, {D, (size_t)ch * 4}, {z, n},
                         {dt_bias, (size_t)ch * 4}, {cu, cu ? (size_t)(seqs + 1) * 4 : 0},
                         {h0 == ht ? nullptr : h0, ns}};
    const Range outs[] = {{y, n}, {ht, ns}, {need ? ws : nullptr, need}};
    if (!disjoint(ins, outs)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_selective_scan(plan, x, dt, A, Bm, Cm, D, z, dt_bias, h0, y, ht, cu, seqs, T, (int)total,
                                               ch, N, dtype == GDN_BF16, (char *)ws, (hipStream_t)stream));
}

gdn_status gdn_selective_scan(const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                              const float *D, const void *z, const float *dt_bias, const float *h0, void *y, float *ht,
                              int B, int T, int ch, int N, gdn_dtype dtype, void *ws, size_t ws_bytes, void *stream) {
    return scan_call(x, dt, A, Bm, Cm, nullptr, D, z, dt_bias, h0, y, ht, B, T, (long long)B * T, ch, N, dtype, ws,
                     ws_bytes, stream);
}

gdn_status gdn_selective_scan_varlen(const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                                     const int *cu_seqlens, const float *D, const void *z, const float *dt_bias,
                                     const float *h0, void *y, float *ht, int seqs, int total_T, int ch, int N,
                                     gdn_dtype dtype, void *ws, size_t ws_bytes, void *stream) {
    if (!cu_seqlens) return GDN_ERR_INVALID_ARG;
    return scan_call(x, dt, A, Bm, Cm, cu_seqlens, D, z, dt_bias, h0, y, ht, seqs, total_T, total_T, ch, N, dtype, ws,
                     ws_bytes, stream);
}

gdn_status gdn_selective_step(const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                              const float *D, const void *z, const float *dt_bias, const float *h_in, float *h_out,
                              void *y, int B, int ch, int N, gdn_dtype dtype, void *stream) {
    if (!x || !dt || !A || !Bm || !Cm || !h_in || !h_out || !y || B < 1 || ch < 1 || N < 1) return GDN_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || (N != 8 && N != 16 && N != 32 && N != 64)) return GDN_ERR_UNSUPPORTED;
    if ((long long)B * ch >= ((1LL << 32) - 256) / (N / 4)) return GDN_ERR_UNSUPPORTED;
    for (const void *p : {x, dt, (const void *)A, Bm, Cm, z, (const void *)h_in, (const void *)h_out, (const void *)y})
        if (!aligned(p, 16)) return GDN_ERR_INVALID_ARG;
    if (!aligned(D, 4) || !aligned(dt_bias, 4)) return GDN_ERR_INVALID_ARG;
    const size_t es = esize(dtype), n = (size_t)B * ch * es, nb = (size_t)B * N * es, ns = (size_t)B * ch * N * 4;
    const Range ins[] = {{x, n}, {dt, n}, {A, (size_t)ch * N * 4}, {Bm, nb}, {Cm, nb}, {D, (size_t)ch * 4}, {z, n},
                         {dt_bias, (size_t)ch * 4}, {h_in == h_out ? nullptr : h_in, ns}};
    const Range outs[] = {{y, n}, {h_out, ns}};
    if (!disjoint(ins, outs)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_selective_step(x, dt, A, Bm, Cm, D, z, dt_bias, h_in, h_out, y, B, ch, N,
                                               dtype == GDN_BF16, (hipStream_t)stream));
}

}  // extern "C"
