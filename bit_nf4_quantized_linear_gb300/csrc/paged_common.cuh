// paged_common.cuh -- what the kernels of attention over a paged cache share: the cut of
// all sequences' work into equal runs, one a CTA, and the partial results that a cut leaves.
//
// A unit is kPagedTile tokens of one sequence for one key head (and one group of its query
// heads).  Units in the order (sequence, key head and group, tile) are dealt in contiguous
// runs of equal length, from the lengths on the device, so that ragged batches load every SM
// alike and a captured graph follows its lengths.  A run that covers a (sequence, head group)
// whole writes its outputs; of the others each CTA leaves at most two, its first and its
// last, and paged_join adds them in CTA order: no atomics, the same bits in every run.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "early_launch.cuh"
#include "elem.cuh"
#include "internal.h"

namespace nf4 {

constexpr int kPagedTile = 64;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Tokens of sequence s, forced into what its table row can hold; a length outside is recorded.
__device__ __forceinline__ int paged_len(const PagedArgs& a, int64_t s) {
  const int n = a.lengths[s];
  const int64_t most = static_cast<int64_t>(a.max_pages) * a.page_size;
  if ((n < 0 || n > most) && a.status) atomicCAS(a.status, 0, kStatusBadOffsets);
  return n < 0 ? 0 : (n > most ? static_cast<int>(most) : n);
}

__device__ __forceinline__ int paged_tiles(int len) { return static_cast<int>((static_cast<int64_t>(len) + kPagedTile - 1) / kPagedTile); }

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

struct PagedRun {
  int64_t u0, u1;  // units of this CTA
  int64_t seq;     // sequence of u0
  int64_t before;  // tiles of the sequences before it
};

__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {  // of values >= 0; most fit 32 bits, where it is quick
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// This CTA's run of the units, `heads` a tile.  Equal shares of time, not of units: what a
// (sequence, head group) costs beside its tiles (queries, and the warps' sums at its end) is
// about half a tile's, so one of n tiles counts 2 n + 1.  Called by all threads of the CTA;
// `red` holds 68 values and is free again when the call returns.
__device__ __forceinline__ PagedRun paged_run(const PagedArgs& a, int heads, int64_t* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int64_t each = a.nseq <= blockDim.x ? 1 : (a.nseq + blockDim.x - 1) / blockDim.x;
  const int64_t s0 = threadIdx.x * each, s1 = s0 + each < a.nseq ? s0 + each : a.nseq;
  int64_t own = 0, live = 0;  // tiles, and sequences that have some
  for (int64_t s = s0; s < s1; ++s) {
    const int n = paged_tiles(paged_len(a, s));
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
  const int64_t total = (2 * all_tiles + all_seqs) * heads, share = divide(total, gridDim.x), rest = total - share * gridDim.x;
  const int64_t c = blockIdx.x, v0 = c * share + (c < rest ? c : rest), v1 = v0 + share + (c < rest);
  const int64_t first = (2 * tiles0 + seqs0) * heads, past = first + (2 * own + live) * heads;
  __syncthreads();
  if (threadIdx.x == 0) {  // where no thread's sequences hold an end of the run
    red[0] = red[1] = all_tiles * heads;
    red[2] = a.nseq;
  }
  __syncthreads();
  for (int end = 0; end < 2; ++end) {
    const int64_t v = end ? v1 : v0;
    if (v < first || v >= past) continue;
    int64_t s = s0, before = tiles0, at = first;
    for (; s < s1; ++s) {
      const int n = paged_tiles(paged_len(a, s));
      if (n == 0) continue;
      const int64_t span = static_cast<int64_t>(2 * static_cast<int64_t>(n) + 1) * heads;
      if (v >= at + span) {
        at += span;
        before += n;
        continue;
      }
      const int64_t head = divide(v - at, 2 * static_cast<int64_t>(n) + 1), tile = (v - at - head * (2 * static_cast<int64_t>(n) + 1)) >> 1;
      red[end] = before * heads + head * n + tile;
      if (end == 0) {
        if (head * n + tile == static_cast<int64_t>(heads) * n) {  // the half behind its last tile: the run begins with the next
          before += n;
          do ++s;
          while (s < a.nseq && paged_len(a, s) == 0);
        }
        red[2] = s;
        red[3] = before;
      }
      break;
    }
  }
  __syncthreads();
  PagedRun r;
  r.u0 = red[0];
  r.u1 = red[1];
  r.seq = red[2];
  r.before = red[3];
  __syncthreads();
  return r;
}

// Sequences of no tokens: zeros, and -inf for the logarithm of their sum.
template <typename T>
__device__ __forceinline__ void paged_empty(const PagedArgs& a) {
  for (int64_t s = blockIdx.x; s < a.nseq; s += gridDim.x) {
    if (a.lengths[s] > 0) continue;
    for (int i = threadIdx.x; i < a.Hq * a.D; i += blockDim.x)
      static_cast<T*>(a.o)[s * a.o_s + static_cast<int64_t>(i / a.D) * a.o_h + i % a.D] = T(0.0f);
    for (int h = threadIdx.x; a.lse && h < a.Hq; h += blockDim.x) a.lse[s * a.Hq + h] = -INFINITY;
  }
}

// Adds the partial results of each (sequence, head group) that was cut, in CTA order.  A CTA
// for each CTA of the attention kernel whose run may begin one (blockIdx.x) and each head of
// a group (blockIdx.y); `heads` a group.  Its time is that of a few dependent loads, so what a
// load needs not wait for it does not: flags and sums of all parts are read at once, and those
// of no use are dropped.
template <typename T, int DV>
__global__ void __launch_bounds__(128) paged_join_kernel(PagedArgs a, int heads, int groups) {
  constexpr int kAtOnce = DV <= 4 ? 4 : 2;
  __shared__ float s_acc[4][DV * 32], s_ml[4][2];
  __shared__ int s_last[4];
  const int c = blockIdx.x, n = gridDim.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_wait();
  const PagedRec me = a.rec[c];
  // the CTA that ends it: the first after c with that flag
  int last = n;
  for (int p = n - 1 - threadIdx.x; p > c; p -= 128) last = a.rec[p].flags & 4 ? p : last;
  if (!(me.flags & 1)) return;
  const int G = a.Hq / a.Hk, hk = me.head / groups, g = (me.head - hk * groups) * heads + h;
  if (g >= G) return;
  last = static_cast<int>(__reduce_min_sync(0xffffffffu, static_cast<unsigned>(last)));
  if (lane == 0) s_last[warp] = last;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) last = min(last, s_last[w]);
  const int st = paged_part_stride(a.D);
  float m = -INFINITY, l = 0.0f, acc[DV] = {};
  for (int p0 = c + warp; p0 <= last; p0 += 4 * kAtOnce) {
    float pm[kAtOnce], pl[kAtOnce], pv[kAtOnce][DV];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int p = min(p0 + 4 * i, n - 1);
      const float* part = a.part + (static_cast<int64_t>(p * 2 + (p == c)) * heads + h) * st;
      const bool in = p0 + 4 * i <= last && (p == c || (a.rec[p].flags & 2));
      const float m0 = part[st - 4], l0 = part[st - 3];
      pm[i] = in ? m0 : -INFINITY;
      pl[i] = in ? l0 : 0.0f;
#pragma unroll
      for (int j = 0; j < DV; ++j) {
        const float v = lane + 32 * j < a.D ? part[lane + 32 * j] : 0.0f;
        pv[i][j] = in ? v : 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float top = fmaxf(m, pm[i]), mm = top == -INFINITY ? 0.0f : top;
      const float f0 = exp2f(m - mm), f1 = exp2f(pm[i] - mm);
      m = top;
      l = l * f0 + pl[i] * f1;
#pragma unroll
      for (int j = 0; j < DV; ++j) acc[j] = acc[j] * f0 + pv[i][j] * f1;
    }
  }
#pragma unroll
  for (int i = 0; i < DV; ++i) s_acc[warp][lane + 32 * i] = acc[i];
  if (lane == 0) {
    s_ml[warp][0] = m;
    s_ml[warp][1] = l;
  }
  __syncthreads();
  float top = -INFINITY;
#pragma unroll
  for (int w = 0; w < 4; ++w) top = fmaxf(top, s_ml[w][0]);
  const float mm = top == -INFINITY ? 0.0f : top;
  float f[4], sum = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = exp2f(s_ml[w][0] - mm);
    sum += s_ml[w][1] * f[w];
  }
  const int hq = hk * G + g;
  T* o = static_cast<T*>(a.o) + me.seq * a.o_s + hq * a.o_h;
  for (int d = threadIdx.x; d < a.D; d += 128) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) v += s_acc[w][d] * f[w];
    o[d] = from_f32<T>(v / sum);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[me.seq * a.Hq + hq] = top * kLn2 + logf(sum);
}

template <typename T>
cudaError_t launch_paged_join(const PagedArgs& a, int ctas, int heads, int groups, cudaStream_t s) {
  const int G = a.Hq / a.Hk;
  const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>(G < heads ? G : heads), 1);
  if (a.D <= 64) return launch_early(paged_join_kernel<T, 2>, grid, 128, 0, s, a, heads, groups);
  if (a.D <= 128) return launch_early(paged_join_kernel<T, 4>, grid, 128, 0, s, a, heads, groups);
  return launch_early(paged_join_kernel<T, 8>, grid, 128, 0, s, a, heads, groups);
}

}  // namespace nf4
