// gdn_launch.h -- host-side launch functions of the gfx950 kernels (internal;
// the public boundary is include/gdn.h).  Each returns the launch status.
#pragma once

#include <hip/hip_runtime.h>

namespace gdn {

// exact: fp32 operands also for bf16 inputs (used by the backward's recompute).
// G2d (nullable): the gate sums also in fp64 [B, H, NT, 64] (for the backward).
hipError_t launch_intra(const void *k, const float *g, const float *beta, float *G2, float *Tinv, int B,
                        int T, int H, int Dk, bool bf16, hipStream_t st, bool exact = false,
                        double *G2d = nullptr);

// ck (nullable): entry state of every chunk, [B, H, NT, Dk, Dv] fp32; o may
// then be null to skip the output.
hipError_t launch_walk(const void *q, const void *k, const void *v, const float *beta, const float *G2,
                       const float *Tinv, const float *h0, float *o, float *ht, float *ck, int B, int T, int H,
                       int Dk, int Dv, bool bf16, float scale, hipStream_t st, bool exact = false);

// Single-kernel chunked forward for bf16 inputs (no workspace).  With
// cu_seqlens (device, B + 1 int32 offsets) the tensors hold B packed
// sequences of T tokens in total; otherwise a dense [B, T, H, D] batch.
// The forward walk of bf16 inputs storing only the state that enters every
// chunk: states [B, H, ceil(T / 64), Dk, Dv] fp32 (a backward's recompute),
// with T - I of every chunk from Tws (fp32 [B, H, ceil(T / 64), 64, 64]).
hipError_t launch_fused_states_bf16(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                    const float *Tws, const float *h0, float *states, int B, int T, int H, int Dk,
                                    int Dv, hipStream_t st);
hipError_t launch_fused_bf16(const void *q, const void *k, const void *v, const float *g, const float *beta,
                             const float *h0, float *o, float *ht, const int *cu_seqlens, int B, int T, int H, int Dk,
                             int Dv, float scale, hipStream_t st);

// The same forward over a dense batch as a chunk-parallel state scan (Dk =
// Dv = D): each sequence in NS segments of L chunks; output-free walks give
// every segment but the last its end state from its entry (segment 0) or from
// zero, and its transfer matrix (middle segments); a scan gives every
// segment's true entry state; then the single kernel runs all segments as
// packed sequences.  Hin, Hout, M: [B NS, H, D, D] fp32, cu: B NS + 1 int32
// (the caller's workspace).
hipError_t launch_fused_seg_bf16(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                 const float *h0, float *o, float *ht, int B, int T, int H, int D, float scale,
                                 int NS, int L, float *Hin, float *Hout, float *M, int *cu, hipStream_t st);

// Gated DeltaNet-2, two stages: per-chunk prepared operands (decayed e, q
// and k; Gamma_C; T - I; strict P; diag P), then the state walk.
hipError_t launch_gdn2_intra(const void *q, const void *k, const float *la, const void *bg, void *Ehat, void *Qhat,
                             void *Khat, float *GamC, float *Tinv, float *P, float *D, int B, int T, int H, int Dk,
                             bool bf16, hipStream_t st);

hipError_t launch_gdn2_walk(const void *Ehat, const void *Qhat, const void *Khat, const float *GamC,
                            const float *Tinv, const float *P, const float *D, const void *v, const void *wg,
                            const float *h0, float *o, float *ht, int B, int T, int H, int Dk, int Dv, bool bf16,
                            float scale, hipStream_t st);

// Gated DeltaNet-2 for bf16 inputs: a parallel prep kernel writes one block
// of prepared operands per chunk into ws (gdn2_fused_block_bytes(Dk) each),
// then the walk kernel carries the state through the chunks; when the walk
// leaves compute units idle, the sequence runs in time parts and the prep of
// one part shares a launch with the walk of the previous one.  ws holds
// gdn2_fused_ws_bytes() bytes.
size_t gdn2_fused_block_bytes(int Dk);
size_t gdn2_fused_ws_bytes(int B, int T, int H, int Dk, int Dv);
hipError_t launch_gdn2_fused_bf16(const void *q, const void *k, const float *la, const void *bg, const void *v,
                                  const void *wg, const float *h0, float *o, float *ht, void *ws, int B, int T,
                                  int H, int Dk, int Dv, float scale, hipStream_t st);

// The same kernels over packed variable-length sequences (cu_seqlens on the
// device, N + 1 offsets into total_T tokens): two small kernels number the
// chunks of every sequence into NC = ceil(total_T / 64) + N chunk numbers,
// the prep fills block (head, number) of each, and one walk workgroup per
// (sequence, head, 32 value columns) carries the state.  ws layout in
// Gdn2VarWs (total bytes, offsets of the sequence and chunk tables).
struct Gdn2VarWs {
    long long NC;
    size_t seq_off, tab_off, total;
};
Gdn2VarWs gdn2_var_ws(int N, int total_T, int H, int Dk);
hipError_t launch_gdn2_fused_varlen_bf16(const void *q, const void *k, const float *la, const void *bg,
                                         const void *v, const void *wg, const int *cu, const float *h0, float *o,
                                         float *ht, void *ws, int N, int total_T, int H, int Dk, int Dv, float scale,
                                         hipStream_t st);

hipError_t launch_step(const void *q, const void *k, const void *v, const float *g, const float *beta,
                       float *S, float *o, int B, int H, int Dk, int Dv, bool bf16, float scale,
                       hipStream_t st);

hipError_t launch_step2(const void *q, const void *k, const void *v, const float *la, const void *bg,
                        const void *wg, float *S, float *o, int B, int H, int Dk, int Dv, bool bf16, float scale,
                        hipStream_t st);

// The reverse state walk of the GDN backward for bf16 inputs in one fused
// kernel (gdn_bwd_fused.hip): dS' of every chunk into dSck, dh0 (nullable).
hipError_t launch_bwd_walk_fused(const void *q, const void *k, const float *beta, const float *dO, const float *dht,
                                 const double *G2, const float *Tinv, float *dSck, float *dh0, int B, int T, int H,
                                 int Dk, int Dv, float scale, hipStream_t st);

// Backward of the chunked GDN forward (gdn_bwd.hip): the reverse state walk
// (dS' of every chunk into dSck, dh0) and the per-chunk gradients, given the
// intra stage (G2, T - I) and the entry state of every chunk (Sck).
hipError_t launch_bwd(const void *q, const void *k, const void *v, const float *beta, const float *dO,
                      const float *dht, const double *G2, const float *Tinv, const float *Sck, float *dSck, float *dq,
                      float *dk, float *dv, float *dg, float *dbeta, float *dh0, int B, int T, int H, int Dk, int Dv,
                      bool bf16, float scale, hipStream_t st);

// Backward of the chunked GDN-2 forward: the fp32 forward recompute
// (gdn2_chunk.hip; intra operands into Eh .. D, chunk entry states into ck),
// then the reverse walk and the per-chunk gradients (gdn2_bwd.hip), which
// overwrite Eh, Qh, Kh, GamC, Tinv and P with their gradients.
// Entry state of every chunk of the GDN-2 forward from the intra stage's
// fp32 operands (bf16 v and w), on split 16-bit MFMA operands.
hipError_t launch_gdn2_states_bf16(const float *Eh, const float *Kh, const float *Tws, const float *GamC,
                                   const void *v, const void *w, const float *h0, float *ck, int B, int T, int H,
                                   int Dk, int Dv, hipStream_t st);
hipError_t launch_gdn2_recompute(const void *q, const void *k, const float *la, const void *bg, const void *v,
                                 const void *wg, const float *h0, float *Eh, float *Qh, float *Kh, float *GamC,
                                 float *Tinv, float *P, float *D, float *ck, int B, int T, int H, int Dk, int Dv,
                                 bool bf16, hipStream_t st);
hipError_t launch_gdn2_bwd(const void *q, const void *k, const void *v, const float *la, const void *bg,
                           const void *wg, const float *dO, const float *dht, float *Eh, float *Qh, float *Kh,
                           float *GamC, float *Tws, float *Pws, const float *Dws, const float *Sck, float *dSck,
                           float *dq, float *dk, float *dv, float *dla, float *db, float *dw, float *dh0, int B, int T,
                           int H, int Dk, int Dv, bool bf16, float scale, hipStream_t st);

// Prologue and epilogue around the rule (gdn_prologue.hip).
hipError_t launch_prologue(const void *xq, const void *xk, const void *xv, const float *a, const float *b,
                           const float *wq, const float *wk, const float *wv, const float *A_log,
                           const float *dt_bias, const float *state_in, void *q, void *k, void *v, float *g,
                           float *beta, float *state_out, int B, int T, int H, int Dk, int Dv, hipStream_t st);
hipError_t launch_gated_rmsnorm(const float *o, const void *z, const float *w, void *y, long rows, int Dv, float eps,
                                hipStream_t st);

// The block's entry (gdn_norm.hip): u = x + res (res nullable), rout = u,
// y = u s w with s = (mean(u^2) + eps)^-1/2 into rstd; y in the type of x, or
// (f8) e4m3 with one scale per row.  Types (x, res): (bf16, bf16),
// (bf16, fp32), (fp32, fp32).  D <= kMaxNormCols.
constexpr int kMaxNormCols = 32768;
hipError_t launch_add_rmsnorm(const void *x, const void *res, const float *w, void *y, void *rout, float *rstd,
                              float *yscale, long rows, int D, bool x_bf16, bool r_bf16, bool f8, float eps,
                              hipStream_t st);
hipError_t launch_quantize_rows(const void *x, void *q, float *scale, long rows, int D, bool bf16, hipStream_t st);
// Backward; part holds norm_bwd_blocks(rows, D) rows of D partial column sums
// (used when dw is wanted).
int norm_bwd_blocks(long rows, int D);
hipError_t launch_add_rmsnorm_bwd(const void *dy, const void *r, const float *w, const float *rstd, const void *dr,
                                  void *dx, float *dw, float *part, long rows, int D, bool dy_bf16, bool r_bf16,
                                  hipStream_t st);
// out[c] = sum of n rows of part [n, D], in a fixed order.
hipError_t launch_colsum(const float *part, float *out, int n, int D, hipStream_t st);

// How a product is cut: tile edge (0: the kernel for few rows or columns),
// splits of k and slabs in each, four buffers or two.
struct MmPlan {
    int tile, splits, per_split;
    bool deep;
};
// The layer's matrix products (gdn_linear.hip): y = act((x w^T) xs ws + bias)
// + residual, z = the activation's argument; x [M, K], w [N, K] in bf16 or
// (f8) e4m3, y and residual bf16 or (y_f32) fp32, z bf16.  part:
// linear_ws_bytes() bytes of partial sums (0: none needed).  act: 0 none,
// 1 relu, 2 silu, 3 gelu.
MmPlan linear_plan(int M, int N, int K, bool f8);
size_t linear_ws_bytes(const MmPlan &p, int M, int N);
hipError_t launch_linear(const MmPlan &p, const void *x, const void *w, const float *xs, const float *ws,
                         const float *bias, const void *residual, void *y, void *z, int M, int N, int K, bool f8,
                         bool y_f32, int act, float *part, hipStream_t st);
// Its backward (bf16 x and w): dz = dy act'(z) in bf16 planes (one, or three
// for fp32 gradients of an inexact dz) where it is not dy itself; dx, dw
// (nullable) in bf16 or (grad_f32) fp32; dbias (nullable) fp32.
struct LinearBwdPlan {
    int Np, planes, blocks;   // columns of a plane; planes; partial rows of dbias
    bool copy;                // dz is written to the workspace
    bool pair, deep;          // both products in one launch; four buffers each
    MmPlan dx, dw;
    size_t plane, sums_off, part_off, part2_off, total;
};
LinearBwdPlan linear_bwd_plan(int M, int N, int K, bool dy_f32, bool grad_f32, int act, bool dx, bool dw, bool dbias);
hipError_t launch_linear_bwd(const LinearBwdPlan &p, const void *dy, const void *x, const void *w, const void *z,
                             void *dx, void *dw, float *dbias, int M, int N, int K, bool dy_f32, bool grad_f32, int act,
                             char *ws, hipStream_t st);
// The second half of it, from the planes of dz (p.Np columns each) and, with
// dbias, the p.blocks rows of its partial sums in ws: a row for every
// dz_rows(M, N) rows of dz.
int dz_rows(int M, int N);
hipError_t launch_linear_grads(const LinearBwdPlan &p, const void *dz, const void *x, const void *w, void *dx, void *dw,
                               float *dbias, int M, int N, int K, bool grad_f32, char *ws, hipStream_t st);

// The gated projection (gdn_gated.hip): w [2 N, K], N gate rows, then N up
// rows; y = act(gate) up [M, N], z [M, 2 N] the arguments.  Cut like a product
// of 2 N columns.
hipError_t launch_gated_linear(const MmPlan &p, const void *x, const void *w, const float *xs, const float *ws,
                               const float *bias, void *y, void *z, int M, int N, int K, bool f8, bool y_f32, int act,
                               float *part, hipStream_t st);
// Its backward.
LinearBwdPlan gated_linear_bwd_plan(int M, int N, int K, bool grad_f32, bool dx, bool dw, bool dbias);
hipError_t launch_gated_linear_bwd(const LinearBwdPlan &p, const void *dy, const void *x, const void *w, const void *z,
                                   void *dx, void *dw, float *dbias, int M, int N, int K, bool dy_f32, bool grad_f32,
                                   int act, char *ws, hipStream_t st);

// Residual layer norm (gdn_layernorm.hip); arguments as the RMS norm's, b and
// mean nullable.  Backward: part holds ln_bwd_blocks(rows, D) rows of 2 D
// partial column sums (used when dw or db is wanted).
hipError_t launch_add_layernorm(const void *x, const void *res, const float *w, const float *b, void *y, void *rout,
                                float *mean, float *rstd, float *yscale, long rows, int D, bool x_bf16, bool r_bf16,
                                bool f8, float eps, hipStream_t st);
int ln_bwd_blocks(long rows, int D);
hipError_t launch_add_layernorm_bwd(const void *dy, const void *r, const float *w, const float *mean,
                                    const float *rstd, const void *dr, void *dx, float *dw, float *db, float *part,
                                    long rows, int D, bool dy_bf16, bool r_bf16, hipStream_t st);

// The selective scan and its convolution (gdn_scan.hip).  cu (nullable): seqs
// sequences packed into total tokens, else seqs of T tokens; bf16 or fp32.
hipError_t launch_causal_conv(const void *x, const float *w, const float *bias, const float *state_in, void *y,
                              float *state_out, const int *cu, int seqs, int T, int total, int C, int W, bool bf16,
                              bool silu, hipStream_t st);
// How a scan is cut along its tokens: segments of L tokens, per_seq to a
// sequence (packed: to all tokens), and the offsets of what passes between
// them (total 0: one segment each, nothing does).
struct ScanPlan {
    int L, per_seq, segs;
    size_t f_off, h_off, total;
};
ScanPlan scan_plan(int seqs, int T, int total, int ch, int N, bool packed);
hipError_t launch_selective_scan(const ScanPlan &p, const void *x, const void *dt, const float *A, const void *B,
                                 const void *C, const float *D, const void *z, const float *dt_bias, const float *h0,
                                 void *y, float *ht, const int *cu, int seqs, int T, int total, int ch, int N, bool bf16,
                                 char *ws, hipStream_t st);
hipError_t launch_selective_step(const void *x, const void *dt, const float *A, const void *B, const void *C,
                                 const float *D, const void *z, const float *dt_bias, const float *h0, float *h1,
                                 void *y, int seqs, int ch, int N, bool bf16, hipStream_t st);

}  // namespace gdn
