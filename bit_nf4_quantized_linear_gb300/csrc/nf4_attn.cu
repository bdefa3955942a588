// nf4_attn.cu -- forward of causal attention over packed sequences on the tensor
// cores (fp16 or bf16, head width a multiple of 8 up to 128).
//
// One CTA owns 256 query rows of one head: two tiles of 128 rows that share every key
// and value tile.  Per 128 keys and tile
//   S = Q K^T                (tcgen05.mma, operands from shared memory)
//   P = exp2(S c - m c)      (one thread a row; c = scale log2 e, m the running maximum)
//   O = O + P V              (tcgen05.mma, P from tensor memory, V from shared memory)
// with l = sum of P in fp32 and, at the end, o = O / l and lse = m scale + ln l.
// Tensor memory: the two tiles' S (128 columns each, P written over S) and O (128
// columns each).  The running maximum is only raised, and O and l only rescaled, when a
// row's maximum grew by more than 2^8 in the weights: until then P stays below 2^8 and
// nothing is lost (the same factor divides out of O and l).  P is rounded to the
// operands' type; l sums the unrounded values.
//
// Roles: warps 0-3 and 4-7 the softmax of the two tiles, warp 8 issues every MMA, warp
// 9 every TMA load, warps 10 and 11 clean the value tiles that the causal mask cuts.  The MMA
// warp alternates between the tiles (P V of one, then its next S), so the tensor cores
// work on one tile while the other's softmax runs.
//
// What bounds it: for a long prompt the products at the clock that the power limit leaves
// (12289 rows, 40 heads over 8 of width 128, fp16: 1.18 ms, 1310 TFLOP/s of 1702 that a
// library product sustains; 1957 MHz of 2070 at 1370 W); S has both operands in shared
// memory, which its 128 x 128 products read at the full 128 bytes a clock.  Shorter ones
// wait for tensor memory on either side of the softmax (two sequences of 4096: the tensor
// pipe is active 44% of the cycles).  Issued under a lane test instead of an elected lane the
// MMAs took 1.37 ms.  256 rows a CTA halve the key and value traffic against 128; two tiles
// fill tensor memory.  While the MMAs were still issued under a lane test, splitting a row
// between two threads (1.63 against 1.34 ms) and forming a quarter of the exponentials by a
// polynomial (1.56 against 1.37 ms) were slower; neither was tried since.  Ragged batches pay
// about 4 us a CTA for its start and end on top (8192 rows in sequences of 1 to 3001: 163 us,
// 830 TFLOP/s).  With heads of 64 the products halve (4095 rows, 32 heads: 71 us, 480 TFLOP/s).
//
// Masked pairs: S is replaced before the exponential, so nothing of a masked key enters
// P.  In P V the weight 0 of a masked row would still turn an infinite or NaN value into
// NaN, so in the tiles cut by the mask the rows past the sequence are cleared and
// non-finite values replaced by zero; when there were any, the epilogue adds them
// to the rows that do see them.
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
constexpr int kWarpMma = 8, kWarpLoad = 9, kWarpClean = 10;  // the last one and the next
constexpr float kRaise = 8.0f;  // log2 of the growth that makes the maximum move
// fp16 keeps 11 bits down to 2^-14 only: P is held times 2^7, which with the growth above
// still ends below 2^15.  The factor divides out of O and l.
constexpr float kShift = 7.0f;

template <int PANELS>
struct Geo {
  static constexpr int kTileBytes = PANELS * kPanelBytes;
  static constexpr int kStages = PANELS == 2 ? 4 : 8;
  static constexpr int kOffQ = 0;
  static constexpr int kOffRing = 2 * kTileBytes;
  static constexpr int kSmem = kOffRing + kStages * kTileBytes + 1024;  // and room to align
};

struct Shared {
  AttnTile tile;
  uint32_t tmem;
  int abort_flag;
  int dirty[2];        // the value tiles at the two diagonals held non-finite values
  uint64_t q_full[2];
  uint64_t full[8], empty[8];
  uint64_t s_full[2], p_full[2], o_full[2], diag[2], clean[2], drain;
};

template <bool F16, int PANELS, bool FULL>
__global__ void __launch_bounds__(kThreads, 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const __grid_constant__ AttnArgs a) {
  using G = Geo<PANELS>;
  using T = typename std::conditional<F16, __half, __nv_bfloat16>::type;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_addr(smem);
  const int h = blockIdx.x % a.Hq, hk = h / (a.Hq / a.Hk);

  // The load warp sets the CTA up on its own -- barriers, its tile, the first loads -- while
  // the MMA warp allocates tensor memory.
  auto load = [&](const CUtensorMap* m, uint32_t dst, uint32_t bar, int head, int r) {
    const int boxes = (a.D + 63) / 64;
    if (elect_one()) {
      mbar_arrive_expect_tx(bar, boxes * kPanelBytes);
      for (int b = 0; b < boxes; ++b) tma_load_3d(dst + b * kPanelBytes, m, bar, b * 64, head, r);
    }
    __syncwarp();
  };
  if (warp == kWarpLoad) {
    if (lane == 0) {
      prefetch_tensormap(&mq);
      prefetch_tensormap(&mk);
      prefetch_tensormap(&mv);
      sh.abort_flag = 0;
      for (int i = 0; i < 2; ++i) {
        sh.dirty[i] = 0;
        mbar_init(smem_addr(&sh.q_full[i]), 1);
        mbar_init(smem_addr(&sh.s_full[i]), 1);
        mbar_init(smem_addr(&sh.p_full[i]), 4);
        mbar_init(smem_addr(&sh.o_full[i]), 1);
        mbar_init(smem_addr(&sh.diag[i]), 1);
        mbar_init(smem_addr(&sh.clean[i]), 64);
      }
      mbar_init(smem_addr(&sh.drain), 1);
      for (int i = 0; i < G::kStages; ++i) {
        mbar_init(smem_addr(&sh.full[i]), 1);
        mbar_init(smem_addr(&sh.empty[i]), 1);
      }
      fence_mbar_init();
    }
    __syncwarp();
    const AttnTile w = find_tile(a, blockIdx.x / a.Hq, 2 * kAttnTile);
    if (lane == 0) sh.tile = w;
    if (w.tile >= 0) {
      const int r = static_cast<int>(w.row0) + 2 * w.tile * kAttnTile;
      load(&mq, sbase + G::kOffQ, smem_addr(&sh.q_full[0]), h, r);
      load(&mk, sbase + G::kOffRing, smem_addr(&sh.full[0]), hk, static_cast<int>(w.row0));
      if ((2 * w.tile + 1) * kAttnTile < w.len)
        load(&mq, sbase + G::kOffQ + G::kTileBytes, smem_addr(&sh.q_full[1]), h, r + kAttnTile);
    }
  } else if (warp == kWarpMma) {
    tmem_alloc(smem_addr(&sh.tmem), 512);
    tmem_relinquish();
  } else if (warp >= kWarpClean) {
    int64_t g0, g1;
    gap_rows(a, &g0, &g1);
    if (g0 > 0 || g1 < a.T) {
      const int me = threadIdx.x - 32 * kWarpClean;
      zero_rows(static_cast<T*>(a.o), a.o_t, a.o_h, a.Hq, a.D, 0, g0, me, 64);
      zero_rows(static_cast<T*>(a.o), a.o_t, a.o_h, a.Hq, a.D, g1, a.T, me, 64);
      if (blockIdx.x < a.Hq) {
        for (int64_t t = me; t < g0; t += 64) a.lse[h * a.T + t] = -INFINITY;
        for (int64_t t = g1 + me; t < a.T; t += 64) a.lse[h * a.T + t] = -INFINITY;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const AttnTile w = sh.tile;
  const AttnGuard guard{&sh.abort_flag, a.status};
  const uint32_t tmem = sh.tmem;
  // Key tiles that each query tile sees: tile i of the sequence sees 0 .. i.
  const int i0 = w.tile * 2;
  const int na = w.tile < 0 ? 0 : i0 + 1;
  const int nb = w.tile < 0 || (i0 + 1) * kAttnTile >= w.len ? 0 : i0 + 2;
  const int nkv = na > nb ? na : nb;
  const int row0 = static_cast<int>(w.row0);
  const int ksteps = (a.D + 15) / 16;

  if (warp >= 8) {
    if (na == 0) {
      // no tile: nothing but the deallocation below
    } else if (warp == kWarpLoad) {
      // The load and MMA warps stay converged: all lanes walk the loop, one lane issues.
      // (the first queries and keys are on their way)
      uint32_t st = 1, ph = 0, issued = 1, par = 0, diag = 0;
      for (int j = 1; j < 2 * nkv; ++j) {  // K0 V0 K1 V1 ...
        if (!attn_wait_warp(smem_addr(&sh.empty[st]), ph ^ 1u, guard)) break;
        // the value tiles at the diagonals, the last ones, go to the cleaning warps first
        const int d = (j & 1) ? (j >> 1) - i0 : -1;
        load((j & 1) ? &mv : &mk, sbase + G::kOffRing + st * G::kTileBytes,
             d >= 0 ? smem_addr(&sh.diag[d]) : smem_addr(&sh.full[st]), hk, row0 + (j >> 1) * kAttnTile);
        if (d >= 0) {
          diag |= 1u << d;
        } else {
          issued |= 1u << st;
          par = (par & ~(1u << st)) | (ph << st);
        }
        if (++st == G::kStages) {
          st = 0;
          ph ^= 1u;
        }
      }
      // every load must have landed before the CTA may exit
      attn_drain(smem_addr(&sh.q_full[0]), 0, guard);
      if (nb > 0) attn_drain(smem_addr(&sh.q_full[1]), 0, guard);
      for (int d = 0; d < 2; ++d)
        if (diag & (1u << d)) attn_drain(smem_addr(&sh.diag[d]), 0, guard);
      for (int q = 0; q < G::kStages; ++q)
        if (issued & (1u << q)) attn_drain(smem_addr(&sh.full[q]), (par >> q) & 1u, guard);
      __syncwarp();
    } else if (warp >= kWarpClean) {
      // The value tiles at the two diagonals (the last one of each query tile).
      for (int d = 0; d < (nb > 0 ? 2 : 1); ++d) {
        const int jt = i0 + d, st = (2 * jt + 1) % G::kStages;
        if (!attn_wait_warp(smem_addr(&sh.diag[d]), 0, guard)) break;
        const int rows = min(kAttnTile, w.len - jt * kAttnTile);
        if (clean_tile<F16, PANELS>(smem + G::kOffRing + st * G::kTileBytes, rows, true, warp - kWarpClean, 2) && lane == 0)
          sh.dirty[d] = 1;
        mbar_arrive(smem_addr(&sh.clean[d]));
      }
    } else if (warp == kWarpMma) {
      const uint32_t id_s = F16 ? idesc_f16_f32(128, 128, false, false) : idesc_bf16_f32(128, 128, false, false);
      const uint32_t id_o = F16 ? idesc_f16_f32(128, ksteps * 16, false, true) : idesc_bf16_f32(128, ksteps * 16, false, true);
      auto wait = [&](uint64_t& b, uint32_t parity) { return attn_wait_warp(smem_addr(&b), parity, guard); };
      auto commit = [&](uint64_t& b) {
        if (elect_one()) mma_commit(smem_addr(&b));
        __syncwarp();
      };
      auto scores = [&](int t, uint32_t kaddr) {
        if (elect_one()) {
          mma_over_columns<FULL, PANELS>(tmem + t * 128, sbase + G::kOffQ + t * G::kTileBytes, kaddr, id_s, ksteps);
          mma_commit(smem_addr(&sh.s_full[t]));
        }
        __syncwarp();
      };
      bool ok = wait(sh.q_full[0], 0) && wait(sh.full[0], 0);
      if (ok) {
        scores(0, sbase + G::kOffRing);
        if (nb > 0) {
          ok = wait(sh.q_full[1], 0);
          if (ok) scores(1, sbase + G::kOffRing);
        }
        commit(sh.empty[0]);
      }
      for (int j = 0; ok && j < nkv; ++j) {
        const int lv = 2 * j + 1, lk = 2 * j + 2;  // loads of V_j and K_{j+1}
        const int sv = lv % G::kStages, sk = lk % G::kStages;
        const uint32_t vaddr = sbase + G::kOffRing + sv * G::kTileBytes, kaddr = sbase + G::kOffRing + sk * G::kTileBytes;
        ok = j >= i0 ? wait(sh.clean[j - i0], 0) : wait(sh.full[sv], (lv / G::kStages) & 1);
        if (!ok) break;
        bool have_k = false;
        for (int t = 0; t < 2; ++t) {
          const int n = t ? nb : na;
          if (j >= n) continue;
          if (!(ok = wait(sh.p_full[t], j & 1))) break;
          tc_fence_after();
          if (elect_one()) {
            mma_over_rows(tmem + 256 + t * 128, tmem + t * 128, 32, vaddr, id_o, j > 0);
            if (j + 1 == n) mma_commit(smem_addr(&sh.o_full[t]));
          }
          __syncwarp();
          if (j + 1 < n) {
            if (!have_k && !(ok = wait(sh.full[sk], (lk / G::kStages) & 1))) break;
            have_k = true;
            scores(t, kaddr);
          }
        }
        if (!ok) break;
        commit(sh.empty[sv]);
        if (have_k) commit(sh.empty[sk]);
      }
      // no MMA and no arrival of a commit may be in flight when the CTA exits
      commit(sh.drain);
      attn_drain(smem_addr(&sh.drain), 0, guard);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------- softmax --
    const int t = warp >> 2;
    const int n = t ? nb : na;
    const int i = (i0 + t) * kAttnTile + (warp & 3) * 32 + lane;  // row within the sequence
    const uint32_t ts = tmem + ((warp & 3) * 32u << 16) + t * 128, to = ts + 256;
    const float c = a.scale * 1.4426950408889634f;
    float m = -INFINITY, mc = 0.0f, l = 0.0f;  // mc: m c (less the shift), or 0 while m is -inf
    bool ok = n > 0;
    for (int j = 0; ok && j < n; ++j) {
      if (!(ok = attn_wait_warp(smem_addr(&sh.s_full[t]), j & 1, guard))) break;
      tc_fence_after();
      // The maximum first, over the upper half of the columns, then over the lower half,
      // which stays in registers; the upper half is read again for its exponentials.
      const int last = j + 1 == n ? i - j * kAttnTile : kAttnTile;  // keys past row i are hidden
      uint32_t s[64];
      auto fetch = [&](int from) {
        tmem_ld<32>(ts + from, s);
        tmem_ld<32>(ts + from + 32, s + 32);
        tmem_wait_ld<64>(s);
        if (j + 1 == n) {  // the diagonal
#pragma unroll
          for (int q = 0; q < 64; ++q)
            if (from + q > last) s[q] = 0xff800000u;
        }
      };
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      auto raise_to = [&] {
#pragma unroll
        for (int q = 0; q < 64; q += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx[e] = fmaxf(mx[e], fmaxf(__uint_as_float(s[q + e]), __uint_as_float(s[q + e + 4])));
      };
      fetch(64);
      raise_to();
      fetch(0);
      raise_to();
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      if (j == 0) {
        m = top;
        mc = m == -INFINITY ? 0.0f : m * c - (F16 ? kShift : 0.0f);
      } else if (const bool raise = (top - m) * c > kRaise; __any_sync(0xffffffffu, raise)) {
        // P V of the step before is complete: s_full was committed after it.  Each row
        // decides by its own scores, so that no row depends on its neighbours.
        const float f = raise ? exp2_approx((m - top) * c) : 1.0f;
        if (raise) {
          m = top;
          mc = m * c - (F16 ? kShift : 0.0f);
        }
        l *= f;
        for (int q = 0; q < ksteps; q += 2) {
          uint32_t o[32];
          tmem_ld<32>(to + q * 16, o);
          tmem_wait_ld<32>(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
          tmem_st32(to + q * 16, o);
        }
      }
      const float2 c2 = make_float2(c, c), m2 = make_float2(-mc, -mc);
      float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
      auto weigh = [&](int from) {  // P of 64 columns goes to 32, behind the scores still to be read
#pragma unroll
        for (int q = 0; q < 64; q += 32) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 x = make_float2(__uint_as_float(s[q + 2 * e]), __uint_as_float(s[q + 2 * e + 1]));
            x = fma2(x, c2, m2);
            x.x = exp2_approx(x.x);
            x.y = exp2_approx(x.y);
            sum[e & 1] = add2(sum[e & 1], x);
            p[e] = pack16<F16>(x.x, x.y);
          }
          tmem_st16(ts + (from + q) / 2, p);
        }
      };
      weigh(0);
      fetch(64);
      weigh(64);
      l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      tmem_wait_st();
      arrive_warp(smem_addr(&sh.p_full[t]));
    }
    if (ok && attn_wait_warp(smem_addr(&sh.o_full[t]), 0, guard)) {
      tc_fence_after();
      const bool live = i < w.len;
      const float inv = 1.0f / l;
      const int64_t r = w.row0 + i;
      T* out = static_cast<T*>(a.o) + r * a.o_t + h * a.o_h;
      T* rest = a.o_rest ? static_cast<T*>(a.o_rest) + (r * a.Hq + h) * a.D : nullptr;
      const bool dirty = sh.dirty[0] || sh.dirty[1];
      for (int q = 0; q < ksteps; q += 2) {
        uint32_t o[32];
        tmem_ld<32>(to + q * 16, o);
        tmem_wait_ld<32>(o);
        float f[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]) * inv;
        if (dirty && live) {
          // the non-finite values taken out of the diagonal tiles, for the rows that see them
          const T* v = static_cast<const T*>(a.v) + hk * a.v_h;
          const int from = i0 * kAttnTile;
#pragma unroll 1
          for (int key = from; key <= i; ++key) {
            if (!sh.dirty[(key - from) / kAttnTile]) continue;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (q * 16 + e >= a.D) continue;
              const float x = to_f32(v[(w.row0 + key) * a.v_t + q * 16 + e]);
              if (!(fabsf(x) < INFINITY)) f[e] += x;
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 32; e += 8)
          if (live && q * 16 + e < a.D) {
            uint32_t x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = pack16<F16>(f[e + 2 * k], f[e + 2 * k + 1]);
            *reinterpret_cast<uint4*>(out + q * 16 + e) = make_uint4(x[0], x[1], x[2], x[3]);
            if (rest) {  // what the rounding left over
#pragma unroll
              for (int k = 0; k < 4; ++k) x[k] = pack16<F16>(f[e + 2 * k] - lo16<F16>(x[k]), f[e + 2 * k + 1] - hi16<F16>(x[k]));
              *reinterpret_cast<uint4*>(rest + q * 16 + e) = make_uint4(x[0], x[1], x[2], x[3]);
            }
          }
        __syncwarp();
      }
      if (live) a.lse[h * a.T + r] = (mc + log2f(l)) * 0.6931471805599453f;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

template <bool F16, int PANELS, bool FULL>
cudaError_t launch_one(const AttnMaps& m, const AttnArgs& a, cudaStream_t s) {
  static SmemLimit limit;
  auto kern = attn_fwd_kernel<F16, PANELS, FULL>;
  if (cudaError_t e = limit.allow(kern, Geo<PANELS>::kSmem)) return e;
  const int64_t grid = attn_tiles(a, 2 * kAttnTile) * a.Hq;
  kern<<<static_cast<unsigned>(grid), kThreads, Geo<PANELS>::kSmem, s>>>(m.q, m.k, m.v, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_fwd(bool f16, const AttnMaps& m, const AttnArgs& a, cudaStream_t s) {
  if (a.D == 128) return f16 ? launch_one<true, 2, true>(m, a, s) : launch_one<false, 2, true>(m, a, s);
  if (a.D == 64) return f16 ? launch_one<true, 1, true>(m, a, s) : launch_one<false, 1, true>(m, a, s);
  if (a.D > 64) return f16 ? launch_one<true, 2, false>(m, a, s) : launch_one<false, 2, false>(m, a, s);
  return f16 ? launch_one<true, 1, false>(m, a, s) : launch_one<false, 1, false>(m, a, s);
}

}  // namespace nf4
