// internal.h -- declarations shared by the library's translation units (host side).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "nf4.h"

namespace nf4 {

// Device status codes written by kernels into the status word (same values as
// nf4_status).
constexpr int kStatusTimeout = NF4_ERR_TIMEOUT;
constexpr int kStatusBadOffsets = NF4_ERR_BAD_OFFSETS;

// Checked debug build (-DNF4_CHECKED=1, libnf4_checked.so): the kernels test the
// index of each computed global or shared-memory access with in_bounds() before
// it; a false test records NF4_ERR_BOUNDS in the status word (first error wins)
// and the caller skips the access.  In the normal build in_bounds() is the
// constant true and the tests compile to nothing.
#ifndef NF4_CHECKED
#define NF4_CHECKED 0
#endif

#ifdef __CUDACC__
__device__ __forceinline__ bool in_bounds(bool ok, int* status) {
#if NF4_CHECKED
  if (!ok && status) atomicCAS(status, 0, NF4_ERR_BOUNDS);
  return ok;
#else
  (void)ok;
  (void)status;
  return true;
#endif
}
#endif

// Upper bound of experts the grouped kernels accept.
constexpr int kMaxExperts = 512;

// Tile geometry of the fused products.
constexpr int kTileW = 128;  // rows of the dequantised operand per tile (MMA M)
constexpr int kTileK = 64;   // contraction per pipeline stage (one 64-value block)

// Top-k combine of the grouped experts and its backward (nf4_moe_combine,
// nf4_moe_combine_bwd).  Forward: rows = the grouped output [R, H], out = [tokens,
// H]; backward: rows = the gradient of the combined output [tokens, H], out = the
// rows' gradient [R, H].  token_rows [tokens, k]: row of each (token, route), -1
// for none.
struct MoeArgs {
  const __nv_bfloat16* rows;
  int64_t ld_rows;
  const int32_t* token_rows;
  int32_t k;
  int64_t tokens, R, H;
  __nv_bfloat16* out;
  int64_t ld_out;
  int* status;
};
cudaError_t launch_moe(bool backward, const MoeArgs& a, cudaStream_t s);

// The gated residual norm and its backward (nf4_norm_residual_fwd / _bwd).  Rows of
// width H with their own pitches in elements; a null pointer leaves that input or
// output out.
struct NormArgs {
  const void *y, *residual, *gate, *gz, *gh;
  void *z, *h, *gy, *gr, *ggate;
  int64_t ld_y, ld_r, ld_gate, ld_gz, ld_gh, ld_z, ld_h, ld_gy, ld_gr, ld_ggate;
  const float *w_post, *w_pre;
  float *gw_post, *gw_pre;
  float* stats;  // [2][T]: rstd of y, rstd of z
  float* part;   // backward: partial sums over tokens [CTAs][3][H] (gw_pre, gw_post, ggate)
  int64_t T, H;
  int gate_kind;
  float scale, eps;
  int* status;
  int starve;  // failure-path test hook: row 0's copies never complete
};
// CTAs of the backward, each with its own partial sums.
int norm_bwd_ctas(int64_t T, int64_t H, int sms);
cudaError_t launch_norm(bool backward, int dtype, const NormArgs& a, int sms, cudaStream_t s);

// AdamW over many tensors.  The table travels in the kernel's parameters (no copy to
// the device): tensor i holds blocks blk0[i] .. blk0[i + 1] - 1 of kAdamBlock values.
constexpr int kAdamBlock = NF4_ADAMW_BLOCK;
constexpr int kAdamMaxTensors = 400;  // of one launch
struct AdamTensor {
  void* param;
  const void* grad;
  void *m, *v;
  float *m_absmax, *v_absmax;
  int64_t n;
  int64_t vec;  // set by the launcher: vector accesses to every array
};
struct AdamTable {
  AdamTensor t[kAdamMaxTensors];
  int64_t blk0[kAdamMaxTensors + 1];
  int count;
};
static_assert(sizeof(AdamTable) < 30000, "kernel parameters hold 32764 bytes");
struct AdamArgs {
  float beta1, one_minus_beta1, beta2, one_minus_beta2, eps, decay, step_size, inv_sqrt_c2;
  const float* grad_scale;
  const float *levels_m, *levels_v;
};
cudaError_t launch_adamw(int dtype, int bits, AdamTable& tab, const AdamArgs& a, int sms, cudaStream_t s);
struct AdamValuesArgs {
  const uint8_t *m, *v;
  const float *m_absmax, *v_absmax, *levels_m, *levels_v;
  float *out_m, *out_v;
  int64_t n;
  int vec;  // set by the launcher
};
cudaError_t launch_adamw_values(AdamValuesArgs a, int sms, cudaStream_t s);

// Causal attention over packed sequences and its backward (nf4_attention_fwd / _bwd):
// tensors [T, heads, D] with token and head strides in elements, unit stride within
// a head.
struct AttnArgs {
  const void *q, *k, *v, *go;
  void *o, *gq, *gk, *gv;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h, go_t, go_h, gq_t, gq_h, gk_t, gk_h, gv_t, gv_h;
  void* o_rest;  // [T][Hq][D] or null: o before its rounding, less o
  float* lse;    // [Hq][T]
  float* delta;  // [Hq][T], backward
  // Backward in fp16: [Hq][T], [Hk][T], [Hk][T].  shift_q holds the rows' |go| until the
  // exponents of the queries' scales replace them; |v|; the exponents of the keys' scales.
  float *shift_q, *v_norm, *shift_k;
  const int32_t* cu_seqlens;  // [nseq + 1], or null: one sequence of T rows
  int64_t T, nseq;
  int Hq, Hk, D;
  float scale;
  int* status;
};
// Most tiles of `rows` rows that any offsets within [0, T] give.
inline int64_t attn_tiles(const AttnArgs& a, int rows) {
  const int64_t most = a.nseq < a.T ? a.nseq : a.T;  // sequences that can hold a row
  return a.T / rows + most;
}
// Tensor-core kernels: [T][heads][D] tensors as 3-D maps with a box of 64 columns x 1
// head x 128 rows, 128-byte swizzle.
struct AttnMaps {
  CUtensorMap q, k, v, go;
};
cudaError_t launch_attn_fwd(bool f16, const AttnMaps& m, const AttnArgs& a, cudaStream_t s);
cudaError_t launch_attn_bwd(bool f16, const AttnMaps& m, const AttnArgs& a, int sms, cudaStream_t s);
cudaError_t launch_attn_any(bool backward, int dtype, const AttnArgs& a, int sms, cudaStream_t s);

// The paged key-value cache: writing new tokens into it (nf4_paged_append) and attention of
// one query token a sequence over it (nf4_paged_attention).
struct PagedArgs {
  const void *q, *k_new, *v_new;
  void *k, *v, *o;  // pages; outputs
  float* lse;       // [nseq][Hq] or null
  int64_t k_page, k_token, k_head, v_page, v_token, v_head;  // strides of the pages in elements
  int64_t q_s, q_h, o_s, o_h, kn_t, kn_h, vn_t, vn_h;
  int64_t pages, nseq, ld_table, T;
  const int32_t *table, *lengths, *cu_seqlens;
  int max_pages, page_size, Hq, Hk, D;
  unsigned page_mul, page_shift;  // p / page_size = p * page_mul >> page_shift for p < 2^31
  float scale;
  float* part;  // partial results [CTAs][2][query heads of a set][paged_part_stride(D)]
  struct PagedRec* rec;  // [CTAs]
  int* status;
};
// What a CTA left in the partial results: slot 1 holds a run of units that begins a (sequence,
// head set) and goes on in a later CTA, slot 0 one that began in an earlier CTA.
struct PagedRec {
  int64_t seq;
  int32_t set;    // of slot 1
  int32_t flags;  // 1: slot 1 is in use; 2: slot 0 is; 4: slot 0 ends its (sequence, head set)
};
// floats of one head's partial result: D sums, maximum (base 2), sum of weights
inline __host__ __device__ int paged_part_stride(int D) { return (D + 3) / 4 * 4 + 4; }
// How a kernel shares out the heads: groups of `group` query heads, `wh` of them a CTA.
struct PagedShape {
  int group, groups, wh, ctas;  // ctas: a SM
};
// Several heads a CTA where a token's heads lie together (`together`; ragged batch of 463,000
// tokens, 8 heads of 128: 275 us against 297 with all warps on one head), else one, whose tokens do (24
// sequences, 32 heads of 64: 76 us against 67).
inline PagedShape paged_shape(int G, int Hk, int group, int warps, int ctas, bool together) {
  PagedShape s{group, (G + group - 1) / group, 1, ctas};
  while (together && s.wh < warps && Hk * s.groups % (2 * s.wh) == 0) s.wh *= 2;
  return s;
}
inline int log2_of(int n) {
  int l = 0;
  while (n >> (l + 1)) ++l;
  return l;
}
inline size_t paged_part_bytes(const PagedShape& s, int D) {  // of a SM
  return static_cast<size_t>(s.ctas) * (2 * s.wh * s.group * paged_part_stride(D) * sizeof(float) + sizeof(PagedRec));
}
PagedShape paged_shape_mma(int G, int Hk, int D, bool together);
PagedShape paged_shape_f32(int G, int Hk, int D, bool together);
PagedShape paged_shape_any(int G, int Hk);
constexpr int kPagedCtas = 4;  // CTAs a SM at most
// enough for whichever kernel takes the call
inline size_t paged_ws_bytes(int Hq, int Hk, int D, int sms) {
  const int G = Hq / Hk;
  size_t most = paged_part_bytes(paged_shape_any(G, Hk), D);
  for (const PagedShape& s : {paged_shape_mma(G, Hk, D, true), paged_shape_f32(G, Hk, D, true)})
    if (paged_part_bytes(s, D) > most) most = paged_part_bytes(s, D);
  return static_cast<size_t>(sms) * (most + kPagedCtas * sizeof(PagedRec));
}
cudaError_t launch_paged_append(int dtype, const PagedArgs& a, int sms, cudaStream_t s);
cudaError_t launch_paged_mma(bool f16, const PagedArgs& a, int sms, cudaStream_t s);
cudaError_t launch_paged_f32(const PagedArgs& a, int sms, cudaStream_t s);
cudaError_t launch_paged_any(int dtype, const PagedArgs& a, int sms, cudaStream_t s);

// The router of the experts (nf4_route_fwd / nf4_route_bwd).
struct RouteArgs {
  const void* logits;  // [T][E], pitch ld
  int64_t ld, T;
  const float* bias;     // [E] or null
  const uint8_t* live;   // [T] or null
  int E, k, sigmoid, groups, top_groups, group_top, renorm;
  float scale;
  int32_t *experts, *offsets, *row_token, *token_rows;  // [T][k], [E + 1], [T k], [T][k]; tables null: not wanted
  float *weights, *row_weight;                          // [T][k], [T k]
  int32_t* counts;  // [CTAs][route_pitch(E)] values, or bytes where a CTA has few tokens; workspace
  // backward
  const float *g_weights, *g_rows;  // [T][k], [T k]; either may be null
  void* g_logits;
  int64_t ld_g;
  int* status;
};
constexpr int kRouteMaxK = 32;
inline __host__ __device__ int route_pitch(int E) { return (E + 15) / 16 * 16; }
int route_ctas(int64_t T, int sms);
// workspace of the forward with tables
inline size_t route_ws_bytes(int64_t T, int E, int sms) {
  const int n = route_ctas(T, sms);
  return n > 1 ? static_cast<size_t>(n) * route_pitch(E) * sizeof(int32_t) : 0;
}
cudaError_t launch_route(bool backward, int dtype, const RouteArgs& a, int sms, cudaStream_t s);

// Multi-product launches (nf4_linear_fwd_multi / nf4_linear_dgrad_multi): up to
// kMaxProds independent products with the same M and in-features K, each with its
// own weight, activation and output, whose work items share one grid.
constexpr int kMaxProds = 4;

// One product of a multi-product launch.
struct ProdArgs {
  const float* absmax;
  const uint8_t* absmax_q;
  const float* nested_absmax;
  const float* nested_offset;
  __nv_bfloat16* out;
  int64_t ld_out;
  int64_t N_total;  // rows of this weight
  int64_t ncols;    // output columns (forward: this weight's rows; input gradient: K)
  int ksteps;       // contraction steps of an item
  int wtiles;       // tiles over the output columns
  int64_t item0;    // first item of this product in the launch's item order
};

// Tensor maps of a launch: activations, packed codes and output, one per product
// (N = 1 for single-product launches).
template <int N>
struct MapSet {
  CUtensorMap act[N];
  CUtensorMap pk[N];
  CUtensorMap out[N];
};

// Parameters of the fused product kernel (everything but the tensor maps).
struct GemmArgs {
  int64_t M;        // activation rows (dense) or T (grouped)
  int64_t ncols;    // output columns: N (fwd), N_e (grouped fwd), K (dgrad)
  int64_t N_total;  // rows of the packed weight tensor
  int64_t K;        // in-features
  int64_t KB;       // K / 64
  int64_t N_e;      // rows per expert (grouped); N for dense
  int ksteps;       // contraction steps of a full item
  int wtiles;       // tiles over the output columns
  int ttiles;       // token tiles (dense)
  int splits;       // contraction splits (dense, small M)
  int64_t total_items;  // dense only; grouped computes it on the device
  int grouped;
  int E;
  const int32_t* offsets;
  const float* absmax;
  const uint8_t* absmax_q;
  const float* nested_absmax;
  const float* nested_offset;
  const float* code4;
  const float* code8;
  int dq;
  __nv_bfloat16* out;
  int64_t ld_out;
  float* ws;  // split-K partials [splits][M][ncols]
  int* status;
  int prefetch;  // dense: the weight may be read before the preceding grid has finished
  int tma_out;  // dense bf16 output written by bulk tensor stores (aligned out and ld_out)
  // Cluster split (dense, tma_out): cs > 1 CTAs, one cluster, share each tile, one
  // contraction slice each (items = tiles x cs, one per CTA, splits == cs); token
  // slice p of the tile (bt / cs tokens) is summed and stored by cluster rank p from
  // the partials the other ranks write into its activation ring.
  int cs;
  // Grouped forward epilogue (nf4_grouped_fwd_ep): fp32 bias per weight row, fp32
  // scale per output row (routing weights), SwiGLU of interleaved gate/up rows.
  const float* ep_bias;
  const float* ep_scale;
  int ep_swiglu;
  // Grouped: columns of `out` to set to zero in the rows behind the last expert's (0: those
  // rows are left as they were).
  int64_t rest_cols;
  // Backward of the SwiGLU epilogue (ep_swiglu and ep_bwd set): the recomputed
  // gate g and up u meet the upstream gradient dh [T, N_e / 2] (bf16, row pitch
  // ep_ld_dh) and, instead of h, the kernel writes dg = dh r u silu'(g) and
  // du = dh r silu(g) in bf16 at the weight rows' own columns of `out` ([T, N_e]),
  // and, when ep_drw is set, per 32 gate columns the fp32 partial sum over those
  // columns of silu(g) u dh into ep_drw[(N_e / 64) partials][T].
  int ep_bwd;
  const __nv_bfloat16* ep_dh;
  int64_t ep_ld_dh;
  float* ep_drw;
  // Stream-K schedule (dense, splits == 1): the items * ksteps
  // contraction steps are cut into sk_ctas equal contiguous runs, one per CTA, and
  // each CTA walks the tiles of its run in reverse.  A tile cut between CTAs is
  // finished by the highest-index CTA holding part of it (the one with its last
  // steps), which adds the lower CTAs' fp32 partials in a fixed order; a CTA thus
  // only ever waits for CTAs of lower index, which are dispatched before it.
  int sk;
  int64_t sk_units;     // items * ksteps
  int sk_ctas;          // CTAs (= grid)
  float* sk_ws;         // partial tiles [sk_ctas][4 row quarters][bt tokens][32 rows] fp32
  uint64_t* sk_flags;   // [sk_ctas][4] in the caller's workspace: partial of (CTA,
                        // row quarter) published; cleared by the finishing CTA
  uint64_t sk_epoch;    // value this launch publishes (never 0)
  uint64_t sk_wait_xor; // the finishing CTA waits for sk_epoch ^ sk_wait_xor (0; the
                        // failure-path test sets a bit no contributor publishes)
  int chk_inject;       // checked build: fail the statistics-load index check (test hook)
  // Multi-product launches: nprod products (items of product p from prod[p].item0),
  // classic schedule, no splits; the single-product fields above are unused for
  // the per-product quantities.
  int nprod;
  ProdArgs prod[kMaxProds];
};

// Stream-K workspace: partial tiles, then the ready flags (8 bytes per CTA and row
// quarter).
constexpr int kSkMaxCtas = 1024;
inline size_t stream_k_ws_bytes(int ctas, int bt) {
  return static_cast<size_t>(ctas) * kTileW * bt * sizeof(float) + static_cast<size_t>(ctas) * 4 * 8;
}

// Parameters of the small-M GEMV kernels.
struct GemvArgs {
  const __nv_bfloat16* act;  // x [M, K] (forward) or grad_y [M, N] (input gradient)
  int64_t ld_act;
  const uint8_t* packed;
  int64_t N, K, KB;
  const float* absmax;
  const uint8_t* absmax_q;
  const float* nested_absmax;
  const float* nested_offset;
  const float* code4;
  const float* code8;
  int dq;
  __nv_bfloat16* out;
  int64_t ld_out;
  float* ws;  // input gradient: per-row-group partials [groups][M][K]
  int64_t M;
  int64_t m0;  // first activation row of a launch (set by the launcher)
  int kseg;    // forward: contraction segments per row group
  int* status;
};

// Parameters of the small-M tensor-core kernels (mma.sync m16n8k16).  The grid
// is C clusters of S CTAs; cluster c owns the output tiles c*T/C .. (c+1)*T/C - 1
// (forward: 16 weight rows; input gradient: 64 in-features), and CTA rank r of a
// cluster owns the contraction slice r*cc .. (r+1)*cc - 1; the S partial sums of
// a tile are reduced through distributed shared memory in rank order.
// Shared-memory layout of a small-M CTA (byte offsets).
struct SkinnyLayout {
  int table, ring, gy, first, recv, scales, code8, bars, act, total;
};

struct SkinnyArgs {
  // x [M, K] (forward) or grad_y [M, N] (input gradient); like `out`, bf16, or
  // IEEE fp16 bits when f16 is set.
  const __nv_bfloat16* act;
  int64_t ld_act;
  const uint8_t* packed;
  int64_t N, K, KB;
  const float* absmax;
  const uint8_t* absmax_q;
  const float* nested_absmax;
  const float* nested_offset;
  const float* code4;
  const float* code8;
  int dq;
  int f16;        // fp16 operands and output
  __nv_bfloat16* out;
  int64_t ld_out;
  int64_t M;
  int S;          // CTAs per cluster (contraction split)
  int C;          // clusters
  int64_t T;      // output tiles
  int64_t cc;     // contraction per CTA (forward: multiple of 64; input gradient: of 16)
  int prefetch;   // the weight may be read before the preceding grid has finished
  int* status;    // device status word (NF4_ERR_TIMEOUT from a bounded wait)
  // Derived on the host by launch_skinny (no 64-bit divisions in the kernels):
  SkinnyLayout lay;  // the CTA's shared-memory layout
  int64_t nt_max;    // most tiles of a cluster, ceil(T / C)
  int64_t tq;        // T / C
  int tr;            // T % C
  int log2S;         // S = 1 << log2S
};

constexpr int kSkinnyMaxM = 16;

struct SkinnyPlan {
  int S = 0, C = 0;
  int64_t T = 0, cc = 0;
  size_t smem = 0;
};

// Plans and launches (S CTAs per cluster along the contraction).
bool skinny_plan(int mode, int64_t M, int64_t N, int64_t K, int sms, SkinnyPlan* p, bool f16 = false);
// tmap: the packed codes [N rows, K/2 bytes] as a uint8 tensor with a box of
// 128 bytes x 16 rows and 128B swizzle (forward) or 32 bytes x 64 rows and 32B
// swizzle (input gradient).
cudaError_t launch_skinny(int mode, const SkinnyArgs& a, const SkinnyPlan& p, const CUtensorMap& tmap,
                          cudaStream_t s);

// Largest M each product sends to the GEMV kernels.
constexpr int kGemvMaxMFwd = 4;
constexpr int kGemvMaxMDgrad = 4;

// Launchers (return cudaSuccess or the launch error).
cudaError_t launch_gemv_fwd(const GemvArgs& a, cudaStream_t s);
cudaError_t launch_gemv_dgrad(const GemvArgs& a, cudaStream_t s);
int gemv_fwd_kseg(int64_t K);
int64_t gemv_dgrad_row_groups(int64_t N);
// tmap_out: 16-bit output [M, ncols] with a 32 x 32 box, used when a.tma_out is set.
// bits: code width of the weight (4, or 8 with bt <= 128).  f16: fp16 activations,
// operand and output instead of bf16 (4-bit codes).
// Multi-product launch (a.nprod products, bf16, 4-bit codes, bt 128 or 256,
// classic schedule); maps.act/pk/out[p] are product p's tensor maps.
cudaError_t launch_gemm_multi(int mode, int bt, const GemmArgs& a, const MapSet<kMaxProds>& maps, int grid,
                              cudaStream_t s);
cudaError_t launch_gemm(int mode, int bt, int bits, bool f16, const GemmArgs& a,
                        const CUtensorMap& tmap_act, const CUtensorMap& tmap_packed,
                        const CUtensorMap& tmap_out, int grid, cudaStream_t s);
cudaError_t launch_gemm_8bit(int mode, int bt, const GemmArgs& a, const CUtensorMap& tmap_act,
                             const CUtensorMap& tmap_packed, const CUtensorMap& tmap_out, int grid,
                             cudaStream_t s);
cudaError_t launch_gemm_f16(int mode, int bt, const GemmArgs& a, const CUtensorMap& tmap_act,
                            const CUtensorMap& tmap_packed, const CUtensorMap& tmap_out, int grid,
                            cudaStream_t s);
cudaError_t launch_splitk_reduce(const float* ws, int splits, int64_t M, int64_t ncols,
                                 void* out, int64_t ld, bool f16, cudaStream_t s);
// Bytes of the fused kernel's rings (decoded, activation and code tiles) for a
// token tile and code width: the exchange area of a cluster split (receive and
// outgoing blocks), idle once a CTA's single tile is done.
size_t gemm_exchange_bytes(int bt, int bits);
// Clusters of `cs` CTAs of the fused kernel (4-bit bf16 instance of `bt`) that can
// be resident at once on the current device; 0 when it cannot be queried.
int gemm_cluster_capacity(int mode, int bt, int cs);
// out[t] = sum over p = 0 .. P-1 in order of part[p][t] for rows inside the expert
// ranges (offsets[0] <= t < offsets[E]), 0 for the other rows of [0, T).
cudaError_t launch_row_partial_sum(const float* part, int P, int64_t T, const int32_t* offsets,
                                   int E, float* out, cudaStream_t s);

cudaError_t launch_quantize(const void* W, int w_dtype, int64_t numel, const float* code4,
                            uint8_t* packed, float* absmax, cudaStream_t s);
cudaError_t launch_quantize8(const void* W, int w_dtype, int64_t numel, const float* code,
                             uint8_t* codes, float* absmax, cudaStream_t s);
cudaError_t launch_double_quant(const float* absmax, int64_t nblocks, const float* code8,
                                uint8_t* absmax_q, float* nested_absmax, float* nested_offset,
                                double* chunk_ws, cudaStream_t s);
cudaError_t launch_dequantize(const nf4_weight& w, void* out, int out_dtype, cudaStream_t s);

constexpr int kMeanChunk = 1024;    // fixed summation order of the mean offset
constexpr int kNestedBlock = 256;   // nested blocksize

}  // namespace nf4
