// paged_common.cuh -- what the kernels of attention over a paged cache share: the cut of
// all sequences' work into equal runs, one a CTA, and the partial results that a cut leaves.
//
// A CTA's warps share out `wh` heads (a head: a key head, or one group of its query heads) and
// kWarps / wh token tiles; a unit is such a tile of tokens of one sequence for one set of wh
// heads.  Neighbouring key heads lie beside each other in a token's row, so a CTA reads longer
// pieces of memory, and a warp that has a head to itself ends it without the others.  Units in
// the order (head set, sequence, tile) are dealt in contiguous runs of equal cost, from the
// lengths on the device, so that ragged batches load every SM alike, a captured graph follows
// its lengths, and the sets of one token are read at about the same time.  A run that covers a
// (sequence, head set) whole writes its outputs; of the others each CTA leaves at most two, its
// first and its last, and paged_join adds them in CTA order: no atomics, the same bits in every
// run.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "early_launch.cuh"
#include "elem.cuh"
#include "internal.h"

namespace nf4 {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Tokens of sequence s, forced into what its table row can hold; a length outside is recorded.
__device__ __forceinline__ int paged_len(const PagedArgs& a, int64_t s) {
  const int n = a.lengths[s];
  const int64_t most = static_cast<int64_t>(a.max_pages) * a.page_size;
  if ((n < 0 || n > most) && a.status) atomicCAS(a.status, 0, kStatusBadOffsets);
  return n < 0 ? 0 : (n > most ? static_cast<int>(most) : n);
}

__device__ __forceinline__ int paged_tiles(int len, int log2_tile) {
  return static_cast<int>((static_cast<unsigned>(len) + (1u << log2_tile) - 1u) >> log2_tile);
}

__device__ __forceinline__ unsigned paged_index(const PagedArgs& a, int pos) {
  return static_cast<unsigned>(static_cast<uint64_t>(static_cast<unsigned>(pos)) * a.page_mul >> a.page_shift);
}

// The page and slot of token `pos` of sequence s, or page -1 where the table names none.
__device__ __forceinline__ int paged_slot(const PagedArgs& a, int64_t s, int pos, int* slot) {
  const unsigned p = paged_index(a, pos);
  *slot = pos - static_cast<int>(p) * a.page_size;
  const int id = a.table[s * a.ld_table + p];
  if (id >= 0 && id < a.pages) return id;
  if (a.status) atomicCAS(a.status, 0, kStatusBadOffsets);
  return -1;
}

__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {  // of values >= 0; most fit 32 bits, where it is quick
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// A CTA's run of units, one after another.
struct Walk {
  int64_t seq;
  int left;  // units left in the run, this one among them (2^31 would be days of work)
  int len, tiles, set, tile, log2_tile;

  // To a sequence with tokens, from `seq` on.
  __device__ __forceinline__ void settle(const PagedArgs& a) {
    for (int64_t i = 0; i <= a.nseq; ++i, ++seq) {
      if (seq >= a.nseq) {
        seq = 0;
        ++set;
      }
      len = paged_len(a, seq);
      tiles = paged_tiles(len, log2_tile);
      if (tiles > 0) return;
    }
    left = 0;
  }

  __device__ __forceinline__ void next(const PagedArgs& a) {
    --left;
    if (++tile < tiles || left <= 0) return;
    tile = 0;
    ++seq;
    settle(a);
  }
};

// This CTA's run of the units of `sets` head sets.  Equal shares of cost: what a (sequence,
// head set) takes beside its tiles (queries, its end) is about half a tile's, so one of n tiles
// counts 2 n + 1.  Called by all threads of the CTA; `red` holds 68 values and is free again
// when the call returns.
__device__ __forceinline__ Walk paged_run(const PagedArgs& a, int sets, int log2_tile, int64_t* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int64_t each = a.nseq <= blockDim.x ? 1 : (a.nseq + blockDim.x - 1) / blockDim.x;
  const int64_t s0 = threadIdx.x * each, s1 = s0 + each < a.nseq ? s0 + each : a.nseq;
  int64_t own = 0, live = 0;  // tiles, and sequences that have some
  for (int64_t s = s0; s < s1; ++s) {
    const int n = paged_tiles(paged_len(a, s), log2_tile);
    own += n;
    live += n > 0;
  }
  int64_t tiles = own, seqs = live;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, tiles, o), q = __shfl_up_sync(0xffffffffu, seqs, o);
    if (lane >= o) {
      tiles += t;
      seqs += q;
    }
  }
  if (lane == 31) {
    red[warp] = tiles;
    red[32 + warp] = seqs;
  }
  __syncthreads();
  int64_t tiles0 = 0, seqs0 = 0, all_tiles = 0, all_seqs = 0;
  for (int w = 0; w < nw; ++w) {
    if (w == warp) {
      tiles0 = all_tiles;
      seqs0 = all_seqs;
    }
    all_tiles += red[w];
    all_seqs += red[32 + w];
  }
  tiles0 += tiles - own;
  seqs0 += seqs - live;
  // shares of the whole, in halves of a tile
  const int64_t span = 2 * all_tiles + all_seqs, total = span * sets, share = divide(total, gridDim.x), rest = total - share * gridDim.x;
  const int64_t c = blockIdx.x, v0 = c * share + (c < rest ? c : rest), v1 = v0 + share + (c < rest);
  const int64_t first = 2 * tiles0 + seqs0, past = first + 2 * own + live;
  __syncthreads();
  if (threadIdx.x == 0) red[0] = red[1] = all_tiles * sets;  // the end of all units, which no thread's sequences hold
  __syncthreads();
  for (int end = 0; end < 2; ++end) {
    const int64_t v = end ? v1 : v0;
    if (v >= total) continue;
    const int64_t set = divide(v, span), in = v - set * span;
    if (in < first || in >= past) continue;
    int64_t before = tiles0, at = first;
    for (int64_t s = s0; s < s1; ++s) {
      const int n = paged_tiles(paged_len(a, s), log2_tile);
      if (n == 0) continue;
      if (in >= at + 2 * static_cast<int64_t>(n) + 1) {
        at += 2 * static_cast<int64_t>(n) + 1;
        before += n;
        continue;
      }
      const int64_t tile = (in - at) >> 1;  // n: the half behind its last tile, so the next sequence's first
      red[end] = set * all_tiles + before + tile;
      if (end == 0) {
        red[2] = tile < n ? s : s + 1;
        red[3] = tile < n ? tile : 0;
        red[4] = set;
      }
      break;
    }
  }
  __syncthreads();
  Walk w;
  const int64_t units = red[1] - red[0];
  w.left = static_cast<int>(units < INT32_MAX ? units : INT32_MAX);
  w.seq = red[2];
  w.tile = static_cast<int>(red[3]);
  w.set = static_cast<int>(red[4]);
  w.log2_tile = log2_tile;
  if (w.left > 0) w.settle(a);
  __syncthreads();
  return w;
}

__device__ __forceinline__ float exp2_fast(float x) {  // relative error 2^-22
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Types of fp32's range: the sums of weighted values are formed of weights times 2^-20, so that a
// million tokens of the largest finite value do not overflow before they are divided (2^-20 is
// exact, but for sums near the bottom of that range).  fp16's values cannot get there.
template <typename T>
struct PagedSums {
  static constexpr bool kHalf = sizeof(T) == 2 && !std::is_same<T, __nv_bfloat16>::value;
  static constexpr float kDown = kHalf ? 1.0f : 0x1p-20f, kUp = kHalf ? 1.0f : 0x1p20f;
};

// A weighted mean from such a sum and the sum of the weights themselves; 0 where no token has a
// weight (all scores -inf, or no page in the table).
template <typename T>
__device__ __forceinline__ float paged_mean(float v, float sum) { return sum == 0.0f ? 0.0f : v / sum * PagedSums<T>::kUp; }

// Sequences of no tokens: zeros, and -inf for the logarithm of their sum.
template <typename T>
__device__ __forceinline__ void paged_empty(const PagedArgs& a) {
  for (int64_t s = blockIdx.x; s < a.nseq; s += gridDim.x) {
    if (paged_len(a, s) > 0) continue;
    for (int i = threadIdx.x; i < a.Hq * a.D; i += blockDim.x)
      static_cast<T*>(a.o)[s * a.o_s + static_cast<int64_t>(i / a.D) * a.o_h + i % a.D] = T(0.0f);
    for (int h = threadIdx.x; a.lse && h < a.Hq; h += blockDim.x) a.lse[s * a.Hq + h] = -INFINITY;
  }
}

// Adds the partial results of each (sequence, head set) that was cut, in CTA order; `heads` query
// heads a group, `wh` groups a set.  WIDE: a CTA for each such pair that there can be (blockIdx.x,
// which finds the pair's first CTA) and query head, the warps sharing the parts out: for few
// pairs, which are cut into many.  Else a CTA for each CTA of the attention kernel, which may
// begin one, a warp for each query head.  The time is that of a few dependent loads, so what a
// load needs not wait for it does not: flags and sums of several parts are read at once, and
// those of no use are dropped.  3 to 6 us of a call, most of it the wait for the attention
// kernel's last write and the start of CTAs that found no room beside it.
constexpr int kJoinWarps = 16;
constexpr int kJoinCtas = 1024;  // of the attention kernel at most

template <typename T, int DV, bool WIDE>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_join_kernel(PagedArgs a, int ctas, int heads, int groups, int wh) {
  // A cut of many pairs leaves most of them two parts.  (With four at once 200 sequences of 64 to
  // 1024 tokens, 40 heads over 8 of 128 in fp16, take 82.0 us in place of 83.7; most batches the same.)
  constexpr int kAtOnce = WIDE && DV <= 4 ? 4 : 2;
  __shared__ float s_acc[WIDE ? kJoinWarps : 1][DV * 32], s_ml[WIDE ? kJoinWarps : 1][2];
  constexpr int kMost = kJoinCtas;
  __shared__ unsigned s_begin[kMost / 32], s_end[kMost / 32], s_used[kMost / 32];  // flags 1, 4 and 2
  __shared__ PagedRec s_me;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = ctas;
  const int st = paged_part_stride(a.D), G = a.Hq / a.Hk, each = G < heads ? G : heads, step = WIDE ? kJoinWarps : 1;
  // kAtOnce parts from CTA p0 on of query head y of the set, that of CTA c in slot 1.
  float pm[kAtOnce], pl[kAtOnce], pv[kAtOnce][DV];
  auto read = [&](int y, int p0, int c) {
    const int sub = y / each, h = sub * heads + y - sub * each;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int p = min(p0 + step * i, n - 1);
      const float* part = a.part + (static_cast<int64_t>(p * 2 + (p == c)) * (wh * heads) + h) * st;
      pm[i] = part[st - 4];
      pl[i] = part[st - 3];
#pragma unroll
      for (int j = 0; j < DV; ++j) pv[i][j] = lane + 32 * j < a.D ? part[lane + 32 * j] : 0.0f;
    }
  };
  grid_wait();  // (no grid_allow: the attention of the next step would take the room of this one's last CTAs)
  if (!WIDE && warp < wh * each) read(warp, blockIdx.x, blockIdx.x);  // before it is known what they are worth: there 84.6 -> 83.7 us
  // which CTAs begin a cut pair, and which end one
  constexpr int kEach = kMost / (kJoinWarps * 32);
  PagedRec rec[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int p = (i * kJoinWarps + warp) * 32 + lane;
    rec[i] = p < n ? a.rec[p] : PagedRec{0, 0, 0};
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int f = rec[i].flags;
    const unsigned begin = __ballot_sync(0xffffffffu, f & 1), end = __ballot_sync(0xffffffffu, f & 4), used = __ballot_sync(0xffffffffu, f & 2);
    if (lane == 0) {
      s_used[i * kJoinWarps + warp] = used;
      s_begin[i * kJoinWarps + warp] = begin;
      s_end[i * kJoinWarps + warp] = end;
    }
  }
  __syncthreads();
  int c = blockIdx.x;
  if (WIDE) {  // the (c + 1)-th that begins one
    const unsigned begin = s_begin[lane];
    int upto = __popc(begin);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += up;
    }
    const unsigned past = __ballot_sync(0xffffffffu, upto > c);
    if (past == 0) return;
    const int word = __ffs(past) - 1;
    unsigned rest = __shfl_sync(0xffffffffu, begin, word);
    for (int i = c - (__shfl_sync(0xffffffffu, upto, word) - __popc(rest)); i > 0; --i) rest &= rest - 1;
    c = word * 32 + __ffs(rest) - 1;
  } else if (!(s_begin[c >> 5] >> (c & 31) & 1)) {
    return;
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if ((i * kJoinWarps + warp) * 32 + lane == c) s_me = rec[i];
  __syncthreads();
  const PagedRec me = s_me;
  int last;  // the first after c that ends one ends this one
  {
    const int word = c >> 5;
    const unsigned after = (c & 31) == 31 ? 0u : ~0u << ((c & 31) + 1);
    const unsigned end = lane < word ? 0 : lane > word ? s_end[lane] : s_end[lane] & after;
    const unsigned some = __ballot_sync(0xffffffffu, end != 0);
    if (some == 0) return;
    const int at = __ffs(some) - 1;
    last = at * 32 + __ffs(__shfl_sync(0xffffffffu, end, at)) - 1;
  }
  for (int y = WIDE ? blockIdx.y : warp; y < wh * each; y += WIDE ? wh * each : kJoinWarps) {
    const int sub = y / each, head = me.set * wh + sub, hk = head / groups;
    const int g = (head - hk * groups) * heads + y - sub * each;
    if (g >= G) continue;
    float m = -INFINITY, l = 0.0f, acc[DV] = {};
    for (int p0 = c + (WIDE ? warp : 0); p0 <= last; p0 += step * kAtOnce) {
      if (WIDE || y != warp || p0 != c) read(y, p0, c);
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int p = p0 + step * i;
        const bool in = p <= last && (p == c || (s_used[p >> 5] >> (p & 31) & 1));
        pm[i] = in ? pm[i] : -INFINITY;
        pl[i] = in ? pl[i] : 0.0f;
#pragma unroll
        for (int j = 0; j < DV; ++j) pv[i][j] = in ? pv[i][j] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const float top = fmaxf(m, pm[i]), mm = top == -INFINITY ? 0.0f : top;
        const float f0 = exp2_fast(m - mm), f1 = exp2_fast(pm[i] - mm);
        m = top;
        l = l * f0 + pl[i] * f1;
#pragma unroll
        for (int j = 0; j < DV; ++j) acc[j] = acc[j] * f0 + pv[i][j] * f1;
      }
    }
    const int hq = hk * G + g;
    T* o = static_cast<T*>(a.o) + me.seq * a.o_s + hq * a.o_h;
    if constexpr (!WIDE) {
#pragma unroll
      for (int j = 0; j < DV; ++j)
        if (lane + 32 * j < a.D) o[lane + 32 * j] = from_f32<T>(paged_mean<T>(acc[j], l));
      if (lane == 0 && a.lse) a.lse[me.seq * a.Hq + hq] = m * kLn2 + logf(l);
    } else {
#pragma unroll
      for (int i = 0; i < DV; ++i) s_acc[warp][lane + 32 * i] = acc[i];
      if (lane == 0) {
        s_ml[warp][0] = m;
        s_ml[warp][1] = l;
      }
      __syncthreads();
      float top = -INFINITY;
      for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, s_ml[w][0]);
      const float mm = top == -INFINITY ? 0.0f : top;
      for (int d = threadIdx.x; d < a.D; d += kJoinWarps * 32) {
        float v = 0.0f, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
          const float f = exp2_fast(s_ml[w][0] - mm);
          sum += s_ml[w][1] * f;
          v += s_acc[w][d] * f;
        }
        o[d] = from_f32<T>(paged_mean<T>(v, sum));
        if (d == 0 && a.lse) a.lse[me.seq * a.Hq + hq] = top * kLn2 + logf(sum);
      }
    }
  }
}

// The wide form for up to a quarter as many pairs as CTAs.  Us of a call with the narrow and with
// the wide form, in brackets the pairs as a share of the CTAs:
//   32 heads over 8 of 128, bf16: one sequence of 131072 tokens [1/152] 124, 89; of 1 to 2048, 4
//   sequences [1/38] 28, 13; 16 [1/10] 23, 21; 24 [1/6] 24.8, 25.3; 38 [1/4] 36, 41; 100 [2/3] 72, 92
//   12 heads over 4 of 80, fp32, of 1 to 2000: 16 [1/10] 25, 21; 32 [1/5] 33.4, 33.2; 64 [2/5] 53, 56
//   32 unshared heads of 64, of 500 to 3000: 2 [1/7] 15.2, 13.6; 4 [2/7] 17.7, 16.9; 8 [4/7] 32.4, 32.6
// They cross between a seventh (sets of four heads) and a half (single heads) of the CTAs.
template <typename T, int DV>
cudaError_t launch_paged_join_width(const PagedArgs& a, int ctas, int heads, int groups, int wh, cudaStream_t s) {
  if (ctas > kJoinCtas) return cudaErrorInvalidConfiguration;
  const int G = a.Hq / a.Hk;
  const int64_t pairs = a.nseq * (static_cast<int64_t>(a.Hk) * groups / wh);
  if (pairs <= ctas / 4)
    return launch_early(paged_join_kernel<T, DV, true>, dim3(static_cast<unsigned>(pairs), static_cast<unsigned>(wh * (G < heads ? G : heads))),
                        kJoinWarps * 32, 0, s, a, ctas, heads, groups, wh);
  return launch_early(paged_join_kernel<T, DV, false>, dim3(static_cast<unsigned>(ctas)), kJoinWarps * 32, 0, s, a, ctas, heads, groups, wh);
}

template <typename T>
cudaError_t launch_paged_join(const PagedArgs& a, int ctas, int heads, int groups, int wh, cudaStream_t s) {
  if (a.D <= 64) return launch_paged_join_width<T, 2>(a, ctas, heads, groups, wh, s);
  if (a.D <= 128) return launch_paged_join_width<T, 4>(a, ctas, heads, groups, wh, s);
  return launch_paged_join_width<T, 8>(a, ctas, heads, groups, wh, s);
}

}  // namespace nf4
