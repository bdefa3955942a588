// nf4_attn_bwd.cu -- backward of causal attention over packed sequences on the tensor
// cores (fp16 or bf16, head width a multiple of 8 up to 128).
//
// A first kernel forms delta_i = do_i . o_i (o with the rest of its rounding, where the
// forward left it).  A second launch holds two kinds of CTAs,
// the longer ones first:
//  - keys: 128 keys of one key head, over every query tile that sees them and every
//    query head of the group.  Transposed, so that P and dS stay in tensor memory as the
//    left operands:
//      S' = K Q^T,  dP' = V dO^T,  P' = exp2(S' c - lse log2 e),  dV += P' dO,
//      dS' = P' (dP' - delta),  dK += dS' Q
//  - queries: 128 queries of one head, over the key tiles they see:
//      S = Q K^T,  dP = dO V^T,  dS = P (dP - delta),  dQ += dS K
// Seven products against the five that the definition needs: the scores and their
// gradient are formed twice so that each sum stays with one CTA in one order, without
// atomics on dQ or partial sums through memory.  P and dS are rounded to the operands'
// type for their products; sums are fp32.
//
// In fp16 each query's (for dK each key's) dS is held times a power of two, divided out of
// the sum at the end, that brings a bound of the row's |dS| just below 2^15: what the range
// of fp16 loses then lies 2^-29 below the largest that a row may hold, whatever the size of
// dO and V.  The bound is (|do_i| |v_j| + |delta_i|) with the largest |v_j| that query i
// sees, or the largest |do_i| and |delta_i| that see key j: two more passes over the rows'
// norms (attn_shift_kernel), and nothing of a masked pair.
//
// The MMA warp keeps the tensor cores on one of a step's products while the two
// compute groups (each half of a tile's columns, one thread a row) work on the other:
// in the keys' CTAs dV and the next S' run during dS, dK and the next dP' during P; in
// the queries' CTAs dQ and the scores after next run while dS is formed.
//
// What bounds it: the products, 7/5 of the definition's (12289 rows, 40 heads over 8 of
// width 128, fp16: 3.7 to 3.9 ms with the passes before it, 1000 TFLOP/s of the definition's,
// 1400 executed, at 1905 MHz under the power limit), two of four
// (three) of them with both operands in shared memory at its full read rate.  A step of the
// keys' CTAs spends 2250 of 3070 cycles issuing MMAs at the tensor cores' rate; with the
// loads of Q and dO in two joint stages instead of three and two of their own it waited 730
// cycles more for them.  Four compute groups of 32 columns instead of two of 64 were slower
// (4.6 against 4.4 ms) while an MMA still took 100 cycles to issue; not tried since.  Short tiles pay for a CTA's start and end: about 4000 cycles before
// its first step and as many after the last, of 28000 (8192 rows in 9 sequences).  Short
// sequences are bound by the longest chain of steps of a key tile: 512 rows take 30 us with
// the row sums.  The scale of dS costs fp16 a multiplication a pair in the keys' CTAs and the
// shift kernel: 8192 rows 503 us against 473 in bf16, 512 rows 38 against 32.
//
// Masked pairs: P and dS are set to 0 by index.  Where that 0 would still meet an
// infinity or a NaN as a factor -- rows of another sequence in a ragged tile, and rows
// of the diagonal tile -- the tile is cleaned in shared memory first.  A row whose lse
// is not finite has P = NaN wherever it is seen, and non-finite values of dO taken out
// of a diagonal tile are added to dV at the end.  The queries' diagonal tile of K is
// cleaned for dQ only, after its scores (a key of -inf scores has P = 0, not what its
// other columns give); a query that sees a non-finite value of it gets NaN there, as its
// dS is 0 or NaN.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "attn_mma.cuh"
#include "elem.cuh"
#include "smem_limit.h"

namespace nf4 {
namespace {

constexpr int kThreads = 384;
constexpr int kWarpMma = 8, kWarpLoad = 9, kWarpPrep = 10;  // the last one and the next
constexpr int kCompute = 8;  // warps of the two compute groups
constexpr float kLog2e = 1.4426950408889634f;
// fp16 keeps 11 bits down to 2^-14 only: the keys' CTAs hold P' times 2^14 (P' <= 1), and
// divide dV by it at the end.  dS has a scale of its own (attn_shift_kernel).
constexpr float kShift = 14.0f, kUnshift = 1.0f / 16384.0f;

template <int PANELS>
struct Geo {
  static constexpr int kTileBytes = PANELS * kPanelBytes;
  // keys: K, V, three Q, two dO.  queries: Q, dO, three K, two V.
  static constexpr int kSmem = 7 * kTileBytes;
};

// Row statistics of the keys' CTAs, negated (they are only subtracted).
struct alignas(16) Rows {
  float lse2[2][kAttnTile];
  float delta[2][kAttnTile];
};

struct Shared {
  Rows rows;
  AttnTile tile;
  uint32_t tmem;
  int abort_flag;
  int dirty;
  uint64_t own_full, full[3], vfull[2], empty[3], vempty[2], ready[2], gready[2], diag, scored, clean;
  uint64_t s_full[2], dp_full, dp_free, p_full, ds_full, out_full, drain;
};

// delta[h][t] = do . (o + what its rounding left over): 16 bytes a lane, rows of a head
// side by side.  In fp16 also the rows' |do| and |v|, 0 where they are not finite (every
// gradient that such a row reaches is not finite either).  Bound by HBM.
template <typename T>
__global__ void __launch_bounds__(256) attn_delta_kernel(const __grid_constant__ AttnArgs a) {
  constexpr bool f16 = std::is_same<T, __half>::value;
  const int per = a.D / 8;                          // lanes with work in a row
  const int width = per <= 8 ? 8 : 16;              // lanes of a row
  const int lane = threadIdx.x & (width - 1);
  const int64_t nq = a.T * a.Hq, n = f16 ? nq + a.T * a.Hk : nq, rows = static_cast<int64_t>(gridDim.x) * 256 / width;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / width;
  for (int64_t i0 = 0; i0 < n; i0 += rows) {  // the same trips for all lanes of a warp
    const int64_t i = i0 + first;
    const bool value = f16 && i >= nq;
    const int64_t row = value ? i - nq : i;
    const int heads = value ? a.Hk : a.Hq;
    const int64_t t = row / heads;
    const int h = static_cast<int>(row - t * heads);
    float s = 0.0f, sq = 0.0f;
    if (i < n && lane < per) {
      const T* yp = value ? static_cast<const T*>(a.v) + t * a.v_t + h * a.v_h : static_cast<const T*>(a.go) + t * a.go_t + h * a.go_h;
      const uint4 y = *reinterpret_cast<const uint4*>(yp + lane * 8);
      uint4 x = make_uint4(0u, 0u, 0u, 0u), z = x;
      if (!value) {
        x = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.o) + t * a.o_t + h * a.o_h + lane * 8);
        if (a.o_rest) z = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.o_rest) + i * a.D + lane * 8);
      }
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w}, zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s = fmaf(lo16<f16>(xs[e]) + lo16<f16>(zs[e]), lo16<f16>(ys[e]), s);
        s = fmaf(hi16<f16>(xs[e]) + hi16<f16>(zs[e]), hi16<f16>(ys[e]), s);
        if (f16) {
          sq = fmaf(lo16<f16>(ys[e]), lo16<f16>(ys[e]), sq);
          sq = fmaf(hi16<f16>(ys[e]), hi16<f16>(ys[e]), sq);
        }
      }
    }
    for (int o = width / 2; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      if (f16) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    }
    if (i < n && lane == 0) {
      const int64_t at = h * a.T + t;
      if (!value) a.delta[at] = s;
      if (f16) (value ? a.v_norm : a.shift_q)[at] = sq < INFINITY ? sqrtf(sq) : 0.0f;
    }
  }
}

constexpr int kScanThreads = 1024;

// Running maxima of N rows of values over the threads of a CTA, from thread 0 on, carried
// from call to call.  Ends with a CTA barrier.
template <int N>
__device__ __forceinline__ void scan_max(float (&x)[N], float (&carry)[N], float (&totals)[2][32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float up = __shfl_up_sync(0xffffffffu, x[k], o);
      if (lane >= o) x[k] = fmaxf(x[k], up);
    }
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (lane == 31) totals[k][warp] = x[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float all = totals[k][lane];
    x[k] = fmaxf(x[k], fmaxf(carry[k], warp_max(lane < warp ? all : 0.0f)));
    carry[k] = fmaxf(carry[k], warp_max(all));
  }
  __syncthreads();
}

// The exponent of the scale for score gradients of at most `bound`: below 2^15 with it.
__device__ __forceinline__ float shift_of(float bound) {
  const int e = static_cast<int>(__float_as_uint(bound) >> 23) - 127;
  return bound > 0.0f ? static_cast<float>(max(-64, min(64, 14 - e))) : 0.0f;
}

__device__ __forceinline__ float pow2(float e) { return __int_as_float((127 + static_cast<int>(e)) << 23); }

// The exponents of the scales that fp16 score gradients are held at (see the head of the
// file): one CTA a sequence and key head.  First the keys, from the last row back, then the
// queries.  A row sum that is not finite bounds nothing: its row's gradients are not finite.
// Bound by the latency of its loads, a chunk of rows after the other (8192 rows in 9 sequences,
// 32 heads over 8: 11 us, beside 450 for the products; one sequence of 12289: 54 of 3660).
__global__ void __launch_bounds__(kScanThreads) attn_shift_kernel(const __grid_constant__ AttnArgs a) {
  __shared__ float totals[2][32];
  const int hk = blockIdx.y, group = a.Hq / a.Hk;
  int64_t first, last;
  seq_bounds(a, blockIdx.x, &first, &last);
  auto finite = [](float x) { return fabsf(x) < INFINITY ? fabsf(x) : 0.0f; };
  float seen[2] = {0.0f, 0.0f}, value[1] = {0.0f};
  for (int64_t end = last; end > first; end -= kScanThreads) {
    const int64_t t = end - 1 - threadIdx.x;
    float m[2] = {0.0f, 0.0f};
    if (t >= first)
#pragma unroll 4
      for (int h = hk * group; h < (hk + 1) * group; ++h) {
        m[0] = fmaxf(m[0], a.shift_q[h * a.T + t]);
        m[1] = fmaxf(m[1], finite(a.delta[h * a.T + t]));
      }
    scan_max(m, seen, totals);
    if (t >= first) a.shift_k[hk * a.T + t] = shift_of(fmaf(m[0], a.v_norm[hk * a.T + t], m[1]));
  }
  for (int64_t at = first; at < last; at += kScanThreads) {
    const int64_t t = at + threadIdx.x;
    float v[1] = {t < last ? a.v_norm[hk * a.T + t] : 0.0f};
    scan_max(v, value, totals);
    if (t < last)
#pragma unroll 4
      for (int h = hk * group; h < (hk + 1) * group; ++h)
        a.shift_q[h * a.T + t] = shift_of(fmaf(a.shift_q[h * a.T + t], v[0], finite(a.delta[h * a.T + t])));
  }
}

// lse in units of log2, as the weights need it: +inf (weight 0) past the sequence, NaN
// for a row of it whose sum of exponentials is not a positive number.
__device__ __forceinline__ float lse2_of(const AttnArgs& a, int64_t at, bool in) {
  if (!in) return INFINITY;
  const float l = a.lse[at];
  return fabsf(l) < INFINITY ? l * kLog2e : __int_as_float(0x7fffffff);
}

// Writes 32 columns of a row that this thread holds.
template <bool F16, typename T>
__device__ __forceinline__ void store32(T* out, const uint32_t* r, float f, int from, int D) {
#pragma unroll
  for (int e = 0; e < 32; e += 8)
    if (from + e < D)
      *reinterpret_cast<uint4*>(out + from + e) =
          make_uint4(pack16<F16>(__uint_as_float(r[e]) * f, __uint_as_float(r[e + 1]) * f),
                     pack16<F16>(__uint_as_float(r[e + 2]) * f, __uint_as_float(r[e + 3]) * f),
                     pack16<F16>(__uint_as_float(r[e + 4]) * f, __uint_as_float(r[e + 5]) * f),
                     pack16<F16>(__uint_as_float(r[e + 6]) * f, __uint_as_float(r[e + 7]) * f));
}

template <bool F16, int PANELS, bool FULL>
struct Ctx {
  using G = Geo<PANELS>;
  const AttnArgs& a;
  Shared& sh;
  AttnGuard guard;
  uint8_t* smem;
  uint32_t sbase, tmem;
  int warp, lane;
  AttnTile w;
  int ksteps, boxes;

  __device__ __forceinline__ uint32_t bar(const uint64_t& b) const { return smem_addr(&b); }
  __device__ __forceinline__ uint32_t tile(int i) const { return sbase + i * G::kTileBytes; }
  // Every role's warp stays converged: all lanes walk its loop, one lane issues.
  __device__ __forceinline__ bool wait(const uint64_t& b, uint32_t parity) const {
    return attn_wait_warp(bar(b), parity, guard);
  }
  __device__ __forceinline__ void expect(const uint64_t& b, uint32_t n) const {
    if (elect_one()) mbar_arrive_expect_tx(bar(b), n);
    __syncwarp();
  }
  __device__ __forceinline__ void commit(const uint64_t& b) const {
    if (elect_one()) mma_commit(bar(b));
    __syncwarp();
  }
  __device__ __forceinline__ void load(const CUtensorMap* m, int to, const uint64_t& b, int head, int row) const {
    if (elect_one())
      for (int x = 0; x < boxes; ++x) tma_load_3d(tile(to) + x * kPanelBytes, m, bar(b), x * 64, head, row);
    __syncwarp();
  }
  __device__ __forceinline__ uint32_t bytes() const { return boxes * kPanelBytes; }
  // D = A B^T over the head's columns, both operands in shared memory.
  __device__ __forceinline__ void over_columns(uint32_t d, int ta, int tb, uint32_t idesc) const {
    if (elect_one()) mma_over_columns<FULL, PANELS>(d, tile(ta), tile(tb), idesc, ksteps);
    __syncwarp();
  }
  // D += A B over the tile's 128 rows, A in tensor memory in two halves 64 columns apart.
  __device__ __forceinline__ void over_rows(uint32_t d, uint32_t at, int tb, uint32_t idesc, bool more) const {
    if (elect_one()) mma_over_rows(d, at, 64, tile(tb), idesc, more);
    __syncwarp();
  }
};

// ------------------------------------------------------------------------- keys --
// Tiles in shared memory: 0 K, 1 V, 2 + it % 3 Q, 5 + it % 2 dO (dO of a step is free after
// dV, Q only after dK).  Tensor memory: S' and P' from 0, dP' and dS' from 128, dV from 256,
// dK from 384.
template <bool COMPUTE, bool F16, int PANELS, bool FULL, typename T>
__device__ __forceinline__ void keys_cta(const Ctx<F16, PANELS, FULL>& x, const CUtensorMap* mq, const CUtensorMap* mk,
                                         const CUtensorMap* mv, const CUtensorMap* mg, int hk) {
  const AttnArgs& a = x.a;
  Shared& sh = x.sh;
  const AttnTile& w = x.w;
  Rows& rs = sh.rows;
  const int jt = w.tile, nt = (w.len + kAttnTile - 1) / kAttnTile, nq = nt - jt;
  const int group = a.Hq / a.Hk, n = group * nq;
  const int row0 = static_cast<int>(w.row0), lane = x.lane, warp = x.warp;
  if constexpr (!COMPUTE) {
  if (warp == kWarpLoad) {
    int loads_q = 0, loads_g = 0, g = 0, i = jt;
    for (int it = 0; it < n; ++it) {
      if (!x.wait(sh.empty[it % 3], ((it / 3) & 1) ^ 1)) break;
      x.expect(sh.full[it % 3], x.bytes());
      x.load(mq, 2 + it % 3, sh.full[it % 3], hk * group + g, row0 + i * kAttnTile);
      loads_q = it + 1;
      if (!x.wait(sh.vempty[it & 1], ((it >> 1) & 1) ^ 1)) break;
      x.expect(sh.vfull[it & 1], x.bytes());
      x.load(mg, 5 + (it & 1), sh.vfull[it & 1], hk * group + g, row0 + i * kAttnTile);
      loads_g = it + 1;
      if (++i == nt) {
        i = jt;
        ++g;
      }
    }
    attn_drain(x.bar(sh.own_full), 0, x.guard);
    for (int it = loads_q < 3 ? 0 : loads_q - 3; it < loads_q; ++it) attn_drain(x.bar(sh.full[it % 3]), (it / 3) & 1, x.guard);
    for (int it = loads_g < 2 ? 0 : loads_g - 2; it < loads_g; ++it) attn_drain(x.bar(sh.vfull[it & 1]), (it >> 1) & 1, x.guard);
    __syncwarp();
  } else if (warp >= kWarpPrep) {
    int g = 0, i = jt;
    for (int it = 0; it < n; ++it) {
      const int st = it & 1, rows = min(kAttnTile, w.len - i * kAttnTile);
      const int64_t at = static_cast<int64_t>(hk * group + g) * a.T + w.row0 + i * kAttnTile;
      float l[2], d[2];  // two rows a lane, the second warp the upper half
      const int r0 = (warp - kWarpPrep) * 64 + lane * 2;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[e] = (F16 ? kShift : 0.0f) - lse2_of(a, at + r0 + e, r0 + e < rows);
        d[e] = r0 + e < rows ? -a.delta[at + r0 + e] : 0.0f;
      }
      // the statistics of two steps ago have been read once that step's dK is done
      if (it >= 2 && !x.wait(sh.empty[(it - 2) % 3], ((it - 2) / 3) & 1)) break;
      *reinterpret_cast<float2*>(&rs.lse2[st][r0]) = make_float2(l[0], l[1]);
      *reinterpret_cast<float2*>(&rs.delta[st][r0]) = make_float2(d[0], d[1]);
      const bool clean = i == jt || rows < kAttnTile;
      if (!x.wait(sh.full[it % 3], (it / 3) & 1)) break;
      if (clean) clean_tile<F16, PANELS>(x.smem + (2 + it % 3) * Geo<PANELS>::kTileBytes, rows, i == jt, warp - kWarpPrep, 2);
      mbar_arrive(x.bar(sh.ready[st]));
      if (!x.wait(sh.vfull[st], (it >> 1) & 1)) break;
      if (clean && clean_tile<F16, PANELS>(x.smem + (5 + st) * Geo<PANELS>::kTileBytes, rows, i == jt, warp - kWarpPrep, 2) &&
          lane == 0)
        sh.dirty = 1;
      mbar_arrive(x.bar(sh.gready[st]));
      if (++i == nt) {
        i = jt;
        ++g;
      }
    }
  } else if (warp == kWarpMma) {
    const uint32_t id_s = F16 ? idesc_f16_f32(128, 128, false, false) : idesc_bf16_f32(128, 128, false, false);
    const uint32_t id_o = F16 ? idesc_f16_f32(128, x.ksteps * 16, false, true) : idesc_bf16_f32(128, x.ksteps * 16, false, true);
    const uint32_t S = x.tmem, P = x.tmem + 128, DV = x.tmem + 256, DK = x.tmem + 384;
    bool ok = x.wait(sh.own_full, 0) && x.wait(sh.ready[0], 0);
    if (ok) {
      x.over_columns(S, 0, 2, id_s);
      x.commit(sh.s_full[0]);
      if ((ok = x.wait(sh.gready[0], 0))) {
        x.over_columns(P, 1, 5, id_s);
        x.commit(sh.dp_full);
      }
    }
    for (int it = 0; ok && it < n; ++it) {
      const int st = it & 1, st1 = st ^ 1, next = ((it + 1) >> 1) & 1;
      const bool more = it + 1 < n;
      if (!(ok = x.wait(sh.p_full, it & 1))) break;
      tc_fence_after();
      x.over_rows(DV, S, 5 + st, id_o, it > 0);
      x.commit(sh.vempty[st]);
      if (more) {
        if (!(ok = x.wait(sh.ready[st1], next))) break;
        x.over_columns(S, 0, 2 + (it + 1) % 3, id_s);
        x.commit(sh.s_full[0]);
      }
      if (!(ok = x.wait(sh.ds_full, it & 1))) break;
      tc_fence_after();
      x.over_rows(DK, P, 2 + it % 3, id_o, it > 0);
      x.commit(sh.empty[it % 3]);
      if (more) {
        if (!(ok = x.wait(sh.gready[st1], next))) break;
        x.over_columns(P, 1, 5 + st1, id_s);
        x.commit(sh.dp_full);
      } else {
        x.commit(sh.out_full);
      }
    }
    // no MMA and no arrival of a commit may be in flight when the CTA exits
    x.commit(sh.drain);
    attn_drain(x.bar(sh.drain), 0, x.guard);
    __syncwarp();
  }
  } else {
    const int wg = warp >> 2, kv = (warp & 3) * 32 + lane;  // this thread's key within the tile
    const uint32_t lanes = ((warp & 3) * 32u) << 16;
    const uint32_t ts = x.tmem + lanes + wg * 64, tp = ts + 128;
    const float c = a.scale * kLog2e;
    const float2 c2 = make_float2(c, c);
    // fp16: the exponent of dS' (read again at the end: a register less); P' holds 2^14 already
    auto shift = [&] { return jt * kAttnTile + kv < w.len ? a.shift_k[hk * a.T + w.row0 + jt * kAttnTile + kv] : 0.0f; };
    const float more = F16 ? pow2(shift() - kShift) : 1.0f;
    bool ok = true;
    int i = jt;
    for (int it = 0; it < n; ++it) {
      const int st = it & 1;
      const bool diag = i == jt;
      if (!(ok = x.wait(sh.ready[st], (it >> 1) & 1) && x.wait(sh.s_full[0], it & 1))) break;
      tc_fence_after();
      uint32_t s[64];
      tmem_ld<32>(ts, s);
      tmem_ld<32>(ts + 32, s + 32);
      tmem_wait_ld<64>(s);
#pragma unroll
      for (int q = 0; q < 64; q += 4) {
        const float4 l = *reinterpret_cast<const float4*>(&rs.lse2[st][wg * 64 + q]);
        const float2 u = fma2(make_float2(__uint_as_float(s[q]), __uint_as_float(s[q + 1])), c2, make_float2(l.x, l.y));
        const float2 v = fma2(make_float2(__uint_as_float(s[q + 2]), __uint_as_float(s[q + 3])), c2, make_float2(l.z, l.w));
        s[q] = __float_as_uint(exp2_approx(u.x));
        s[q + 1] = __float_as_uint(exp2_approx(u.y));
        s[q + 2] = __float_as_uint(exp2_approx(v.x));
        s[q + 3] = __float_as_uint(exp2_approx(v.y));
      }
      if (diag) {
#pragma unroll
        for (int q = 0; q < 64; ++q)
          if (wg * 64 + q < kv) s[q] = 0u;  // queries before this key
      }
      if (const int rows = w.len - i * kAttnTile - wg * 64; rows < 64) {
        // queries past the sequence: a key of infinite values and their cleared rows make NaN, not a weight of 0
#pragma unroll
        for (int q = 0; q < 64; ++q)
          if (q >= rows) s[q] = 0u;
      }
#pragma unroll
      for (int q = 0; q < 64; q += 32) {
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) p[e] = pack16<F16>(__uint_as_float(s[q + 2 * e]), __uint_as_float(s[q + 2 * e + 1]));
        tmem_st16(ts + q / 2, p);
      }
      tmem_wait_st();
      arrive_warp(x.bar(sh.p_full));
      if (F16) {
#pragma unroll
        for (int q = 0; q < 64; q += 2) {
          const float2 u = mul2(make_float2(__uint_as_float(s[q]), __uint_as_float(s[q + 1])), make_float2(more, more));
          s[q] = __float_as_uint(u.x);
          s[q + 1] = __float_as_uint(u.y);
        }
      }
      if (!(ok = x.wait(sh.dp_full, it & 1))) break;
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 64; q += 32) {
        uint32_t d[32], p[16];
        tmem_ld<32>(tp + q, d);
        tmem_wait_ld<32>(d);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 dl = *reinterpret_cast<const float4*>(&rs.delta[st][wg * 64 + q + e]);
          float2 u = make_float2(__uint_as_float(d[e]), __uint_as_float(d[e + 1]));
          float2 v = make_float2(__uint_as_float(d[e + 2]), __uint_as_float(d[e + 3]));
          u = add2(u, make_float2(dl.x, dl.y));
          v = add2(v, make_float2(dl.z, dl.w));
          u = mul2(u, make_float2(__uint_as_float(s[q + e]), __uint_as_float(s[q + e + 1])));
          v = mul2(v, make_float2(__uint_as_float(s[q + e + 2]), __uint_as_float(s[q + e + 3])));
          if (diag) {
            u.x = wg * 64 + q + e < kv ? 0.0f : u.x;
            u.y = wg * 64 + q + e + 1 < kv ? 0.0f : u.y;
            v.x = wg * 64 + q + e + 2 < kv ? 0.0f : v.x;
            v.y = wg * 64 + q + e + 3 < kv ? 0.0f : v.y;
          }
          p[e / 2] = pack16<F16>(u.x, u.y);
          p[e / 2 + 1] = pack16<F16>(v.x, v.y);
        }
        // dS' of columns q .. q + 31 goes to q / 2 ..: columns already read
        tmem_st16(tp + q / 2, p);
      }
      tmem_wait_st();
      arrive_warp(x.bar(sh.ds_full));
      if (++i == nt) i = jt;
    }
    if (ok && x.wait(sh.out_full, 0)) {
      tc_fence_after();
      // the first group writes dV, the second dK
      const bool live = jt * kAttnTile + kv < w.len;
      const int64_t r = w.row0 + jt * kAttnTile + kv;
      const uint32_t from = x.tmem + lanes + 256 + wg * 128;
      T* out = wg == 0 ? static_cast<T*>(a.gv) + r * a.gv_t + hk * a.gv_h : static_cast<T*>(a.gk) + r * a.gk_t + hk * a.gk_h;
      const float f = wg == 0 ? (F16 ? kUnshift : 1.0f) : a.scale * (F16 ? pow2(-shift()) : 1.0f);
      const bool dirty = wg == 0 && sh.dirty;
      for (int q = 0; q < a.D; q += 32) {
        uint32_t o[32];
        tmem_ld<32>(from + q, o);
        tmem_wait_ld<32>(o);
        if (dirty && live) {
          // the non-finite values taken out of dO's diagonal tiles, for the keys that they see
          const int end = min(w.len, (jt + 1) * kAttnTile);
#pragma unroll 1
          for (int g = 0; g < group; ++g)
#pragma unroll 1
            for (int t = jt * kAttnTile + kv; t < end; ++t) {
              const T* go = static_cast<const T*>(a.go) + (w.row0 + t) * a.go_t + (hk * group + g) * a.go_h;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                if (q + e >= a.D) continue;
                const float y = to_f32(go[q + e]);
                if (!(fabsf(y) < INFINITY)) o[e] = __float_as_uint(__uint_as_float(o[e]) + y);
              }
            }
        }
        if (live) store32<F16>(out, o, f, q, a.D);
        __syncwarp();
      }
    }
  }
}

// ---------------------------------------------------------------------- queries --
// Tiles in shared memory: 0 Q, 1 dO, 2 + j % 3 K, 5 + j % 2 V.  Tensor memory: S and dS
// of even steps from 0, of odd steps from 128, dP from 256, dQ from 384.
template <bool COMPUTE, bool F16, int PANELS, bool FULL, typename T>
__device__ __forceinline__ void queries_cta(const Ctx<F16, PANELS, FULL>& x, const CUtensorMap* mq, const CUtensorMap* mk,
                                            const CUtensorMap* mv, const CUtensorMap* mg, int h) {
  const AttnArgs& a = x.a;
  Shared& sh = x.sh;
  const AttnTile& w = x.w;
  const int it = w.tile, n = it + 1, hk = h / (a.Hq / a.Hk);
  const int row0 = static_cast<int>(w.row0), lane = x.lane, warp = x.warp;
  if constexpr (!COMPUTE) {
  if (warp == kWarpLoad) {
    int nk = 0, nv = 0;
    bool diag = false;
    for (int j = 0; j < n; ++j) {
      if (!x.wait(sh.empty[j % 3], ((j / 3) & 1) ^ 1)) break;
      const uint64_t& b = j + 1 == n ? sh.diag : sh.full[j % 3];  // the last one is cleaned
      x.expect(b, x.bytes());
      x.load(mk, 2 + j % 3, b, hk, row0 + j * kAttnTile);
      if (j + 1 == n) diag = true; else nk = j + 1;
      if (!x.wait(sh.vempty[j & 1], ((j >> 1) & 1) ^ 1)) break;
      x.expect(sh.vfull[j & 1], x.bytes());
      x.load(mv, 5 + (j & 1), sh.vfull[j & 1], hk, row0 + j * kAttnTile);
      nv = j + 1;
    }
    attn_drain(x.bar(sh.own_full), 0, x.guard);
    if (diag) attn_drain(x.bar(sh.diag), 0, x.guard);
    for (int j = nk < 3 ? 0 : nk - 3; j < nk; ++j) attn_drain(x.bar(sh.full[j % 3]), (j / 3) & 1, x.guard);
    for (int j = nv < 2 ? 0 : nv - 2; j < nv; ++j) attn_drain(x.bar(sh.vfull[j & 1]), (j >> 1) & 1, x.guard);
    __syncwarp();
  } else if (warp >= kWarpPrep) {
    // the diagonal's K, between its scores and dQ
    if (x.wait(sh.diag, 0) && x.wait(sh.scored, 0)) {
      if (clean_tile<F16, PANELS>(x.smem + (2 + it % 3) * Geo<PANELS>::kTileBytes, min(kAttnTile, w.len - it * kAttnTile), true,
                                  warp - kWarpPrep, 2) &&
          lane == 0)
        sh.dirty = 1;
      mbar_arrive(x.bar(sh.clean));
    }
  } else if (warp == kWarpMma) {
    const uint32_t id_s = F16 ? idesc_f16_f32(128, 128, false, false) : idesc_bf16_f32(128, 128, false, false);
    const uint32_t id_o = F16 ? idesc_f16_f32(128, x.ksteps * 16, false, true) : idesc_bf16_f32(128, x.ksteps * 16, false, true);
    const uint32_t S = x.tmem, P = x.tmem + 256, DQ = x.tmem + 384;
    auto key = [&](int j) { return j + 1 == n ? x.wait(sh.diag, 0) : x.wait(sh.full[j % 3], (j / 3) & 1); };
    auto scores = [&](int j) {
      x.over_columns(S + (j & 1) * 128, 0, 2 + j % 3, id_s);
      x.commit(sh.s_full[j & 1]);
      if (j + 1 == n) x.commit(sh.scored);
    };
    auto grads = [&](int j) {
      x.over_columns(P, 1, 5 + (j & 1), id_s);
      x.commit(sh.dp_full);
      x.commit(sh.vempty[j & 1]);
    };
    bool ok = x.wait(sh.own_full, 0) && key(0);
    if (ok) {
      scores(0);
      if ((ok = x.wait(sh.vfull[0], 0))) grads(0);
      if (ok && n > 1 && (ok = key(1))) scores(1);
    }
    for (int j = 0; ok && j < n; ++j) {
      if (j + 1 < n) {
        if (!(ok = x.wait(sh.vfull[(j + 1) & 1], ((j + 1) >> 1) & 1) && x.wait(sh.dp_free, j & 1))) break;
        tc_fence_after();
        grads(j + 1);
      }
      if (!(ok = x.wait(sh.ds_full, j & 1) && (j + 1 < n || x.wait(sh.clean, 0)))) break;
      tc_fence_after();
      x.over_rows(DQ, S + (j & 1) * 128, 2 + j % 3, id_o, j > 0);
      x.commit(sh.empty[j % 3]);
      if (j + 2 < n) {
        if (!(ok = key(j + 2))) break;
        scores(j + 2);
      }
    }
    if (ok) x.commit(sh.out_full);
    // no MMA and no arrival of a commit may be in flight when the CTA exits
    x.commit(sh.drain);
    attn_drain(x.bar(sh.drain), 0, x.guard);
    __syncwarp();
  }
  } else {
    const int wg = warp >> 2, row = (warp & 3) * 32 + lane, i = it * kAttnTile + row;
    const uint32_t lanes = ((warp & 3) * 32u) << 16;
    const uint32_t tp = x.tmem + lanes + 256 + wg * 64;
    const float c = a.scale * kLog2e;
    const bool live = i < w.len;
    const int64_t at = static_cast<int64_t>(h) * a.T + w.row0 + i;
    auto shift = [&] { return F16 && live ? a.shift_q[at] : 0.0f; };  // P comes times 2^shift
    const float l = lse2_of(a, at, live) - shift(), dl = live ? a.delta[at] : 0.0f;
    const float2 c2 = make_float2(c, c), l2 = make_float2(-l, -l), d2 = make_float2(-dl, -dl);
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const uint32_t ts = x.tmem + lanes + (j & 1) * 128 + wg * 64;
      const bool diag = j + 1 == n;
      if (!(ok = x.wait(sh.s_full[j & 1], (j >> 1) & 1) && x.wait(sh.dp_full, j & 1))) break;
      tc_fence_after();
      uint32_t s[64], d[64];
      tmem_ld<32>(ts, s);
      tmem_ld<32>(ts + 32, s + 32);
      tmem_ld<32>(tp, d);
      tmem_ld<32>(tp + 32, d + 32);
      tmem_wait_ld<64>(s);
      tmem_wait_ld<64>(d);
      arrive_warp(x.bar(sh.dp_free));
#pragma unroll
      for (int q = 0; q < 64; q += 32) {
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float2 u = fma2(make_float2(__uint_as_float(s[q + 2 * e]), __uint_as_float(s[q + 2 * e + 1])), c2, l2);
          u.x = exp2_approx(u.x);
          u.y = exp2_approx(u.y);
          u = mul2(u, add2(make_float2(__uint_as_float(d[q + 2 * e]), __uint_as_float(d[q + 2 * e + 1])), d2));
          if (diag) {
            u.x = wg * 64 + q + 2 * e > row ? 0.0f : u.x;  // keys after this query
            u.y = wg * 64 + q + 2 * e + 1 > row ? 0.0f : u.y;
          }
          p[e] = pack16<F16>(u.x, u.y);
        }
        tmem_st16(ts + q / 2, p);
      }
      tmem_wait_st();
      arrive_warp(x.bar(sh.ds_full));
    }
    if (ok && x.wait(sh.out_full, 0)) {
      tc_fence_after();
      T* out = static_cast<T*>(a.gq) + (w.row0 + i) * a.gq_t + h * a.gq_h;
      for (int q = wg * 32; q < a.D; q += 64) {  // the groups take 32 columns in turn
        uint32_t o[32];
        tmem_ld<32>(x.tmem + lanes + 384 + q, o);
        tmem_wait_ld<32>(o);
        if (sh.dirty && live) {
          const T* k = static_cast<const T*>(a.k) + hk * a.k_h + q;
#pragma unroll 1
          for (int t = it * kAttnTile; t <= i; ++t)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (q + e < a.D && !(fabsf(to_f32(k[(w.row0 + t) * a.k_t + e])) < INFINITY)) o[e] = 0x7fffffffu;
        }
        if (live) store32<F16>(out, o, a.scale * pow2(-shift()), q, a.D);
        __syncwarp();
      }
    }
  }
}

template <bool F16, int PANELS, bool FULL>
__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mg,
                    const __grid_constant__ AttnArgs a, const int64_t key_ctas) {
  using T = typename std::conditional<F16, __half, __nv_bfloat16>::type;
  // the tiles' swizzle counts from multiples of 1024 bytes, and nothing is left to round up to one
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool keys = blockIdx.x < key_ctas;
  const uint32_t id = keys ? blockIdx.x : blockIdx.x - static_cast<uint32_t>(key_ctas);
  const uint32_t heads = keys ? a.Hk : a.Hq, tile_id = id / heads;
  const int h = static_cast<int>(id - tile_id * heads);

  // The load warp finds the CTA's tile and issues the loads of the tiles that it owns, the
  // MMA warp allocates tensor memory, and another sets up the barriers.
  if (warp == kWarpLoad) {
    if (lane == 0) {
      prefetch_tensormap(&mq);
      prefetch_tensormap(&mk);
      prefetch_tensormap(&mv);
      prefetch_tensormap(&mg);
      mbar_init(smem_addr(&sh.own_full), 1);
      fence_mbar_init();
    }
    __syncwarp();
    const AttnTile w = find_tile(a, tile_id, kAttnTile, !keys);
    if (lane == 0) sh.tile = w;
    if (w.tile >= 0 && elect_one()) {
      const int boxes = (a.D + 63) / 64, r = static_cast<int>(w.row0) + w.tile * kAttnTile;
      const uint32_t bar = smem_addr(&sh.own_full), to = smem_addr(smem);
      mbar_arrive_expect_tx(bar, 2 * boxes * kPanelBytes);
      for (int x = 0; x < boxes; ++x) {
        tma_load_3d(to + x * kPanelBytes, keys ? &mk : &mq, bar, x * 64, h, r);
        tma_load_3d(to + Geo<PANELS>::kTileBytes + x * kPanelBytes, keys ? &mv : &mg, bar, x * 64, h, r);
      }
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    tmem_alloc(smem_addr(&sh.tmem), 512);
    tmem_relinquish();
  } else if (warp >= kWarpPrep) {
    if (warp == kWarpPrep && lane == 0) {
      sh.abort_flag = 0;
      sh.dirty = 0;
      uint64_t* one[] = {&sh.full[0], &sh.full[1], &sh.full[2], &sh.vfull[0], &sh.vfull[1], &sh.empty[0], &sh.empty[1],
                         &sh.empty[2], &sh.vempty[0], &sh.vempty[1], &sh.diag, &sh.scored, &sh.s_full[0], &sh.s_full[1], &sh.dp_full,
                         &sh.out_full, &sh.drain};
      for (uint64_t* b : one) mbar_init(smem_addr(b), 1);
      uint64_t* prep[] = {&sh.ready[0], &sh.ready[1], &sh.gready[0], &sh.gready[1], &sh.clean};
      for (uint64_t* b : prep) mbar_init(smem_addr(b), 64);
      uint64_t* groups[] = {&sh.p_full, &sh.ds_full, &sh.dp_free};
      for (uint64_t* b : groups) mbar_init(smem_addr(b), kCompute);
      fence_mbar_init();
    }
    __syncwarp();
    int64_t g0, g1;
    gap_rows(a, &g0, &g1);
    if (g0 > 0 || g1 < a.T) {
      const int me = threadIdx.x - 32 * kWarpPrep;
      zero_rows(static_cast<T*>(a.gq), a.gq_t, a.gq_h, a.Hq, a.D, 0, g0, me, 64);
      zero_rows(static_cast<T*>(a.gq), a.gq_t, a.gq_h, a.Hq, a.D, g1, a.T, me, 64);
      zero_rows(static_cast<T*>(a.gk), a.gk_t, a.gk_h, a.Hk, a.D, 0, g0, me, 64);
      zero_rows(static_cast<T*>(a.gk), a.gk_t, a.gk_h, a.Hk, a.D, g1, a.T, me, 64);
      zero_rows(static_cast<T*>(a.gv), a.gv_t, a.gv_h, a.Hk, a.D, 0, g0, me, 64);
      zero_rows(static_cast<T*>(a.gv), a.gv_t, a.gv_h, a.Hk, a.D, g1, a.T, me, 64);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  {
    const Ctx<F16, PANELS, FULL> x{a, sh, AttnGuard{&sh.abort_flag, a.status}, smem, smem_addr(smem), sh.tmem, warp, lane,
                             sh.tile, (a.D + 15) / 16, (a.D + 63) / 64};
    const bool work = x.w.tile >= 0;
    if (warp < 8) {
      if (work && keys) keys_cta<true, F16, PANELS, FULL, T>(x, &mq, &mk, &mv, &mg, h);
      if (work && !keys) queries_cta<true, F16, PANELS, FULL, T>(x, &mq, &mk, &mv, &mg, h);
    } else {
      if (work && keys) keys_cta<false, F16, PANELS, FULL, T>(x, &mq, &mk, &mv, &mg, h);
      if (work && !keys) queries_cta<false, F16, PANELS, FULL, T>(x, &mq, &mk, &mv, &mg, h);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) tmem_dealloc(sh.tmem, 512);
}

template <bool F16, int PANELS, bool FULL>
cudaError_t launch_one(const AttnMaps& m, const AttnArgs& a, int sms, cudaStream_t s) {
  static SmemLimit limit;
  using T = typename std::conditional<F16, __half, __nv_bfloat16>::type;
  auto kern = attn_bwd_kernel<F16, PANELS, FULL>;
  if (cudaError_t e = limit.allow(kern, Geo<PANELS>::kSmem)) return e;
  const int width = a.D <= 64 ? 8 : 16;
  const int64_t want = (a.T * (a.Hq + (F16 ? a.Hk : 0)) * width + 255) / 256, most = 32 * static_cast<int64_t>(sms);
  attn_delta_kernel<T><<<static_cast<unsigned>(want < most ? want : most), 256, 0, s>>>(a);
  if (cudaError_t e = cudaGetLastError()) return e;
  if (F16) {
    attn_shift_kernel<<<dim3(static_cast<unsigned>(a.nseq), a.Hk, 1), kScanThreads, 0, s>>>(a);
    if (cudaError_t e = cudaGetLastError()) return e;
  }
  const int64_t tiles = attn_tiles(a, kAttnTile), key_ctas = tiles * a.Hk;
  kern<<<static_cast<unsigned>(key_ctas + tiles * a.Hq), kThreads, Geo<PANELS>::kSmem, s>>>(m.q, m.k, m.v, m.go, a, key_ctas);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_bwd(bool f16, const AttnMaps& m, const AttnArgs& a, int sms, cudaStream_t s) {
  if (a.D == 128) return f16 ? launch_one<true, 2, true>(m, a, sms, s) : launch_one<false, 2, true>(m, a, sms, s);
  if (a.D == 64) return f16 ? launch_one<true, 1, true>(m, a, sms, s) : launch_one<false, 1, true>(m, a, sms, s);
  if (a.D > 64) return f16 ? launch_one<true, 2, false>(m, a, sms, s) : launch_one<false, 2, false>(m, a, sms, s);
  return f16 ? launch_one<true, 1, false>(m, a, sms, s) : launch_one<false, 1, false>(m, a, sms, s);
}

}  // namespace nf4
