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

// The page and slot of token `pos` of sequence s, or page -1 where the table names none.
__device__ __forceinline__ int paged_slot(const PagedArgs& a, int64_t s, int pos, int* slot) {
  const unsigned p = static_cast<unsigned>(pos) / static_cast<unsigned>(a.page_size);
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

// This CTA's run of the units, `heads` a tile.  Called by all threads of the CTA; `red` holds
// 34 values and is free again when the call returns.
__device__ __forceinline__ PagedRun paged_run(const PagedArgs& a, int heads, int64_t* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int64_t each = (a.nseq + blockDim.x - 1) / blockDim.x;
  const int64_t s0 = threadIdx.x * each, s1 = s0 + each < a.nseq ? s0 + each : a.nseq;
  int64_t own = 0;
  for (int64_t s = s0; s < s1; ++s) own += paged_tiles(paged_len(a, s));
  int64_t incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) red[warp] = incl;
  __syncthreads();
  int64_t base = 0, total = 0;
  for (int w = 0; w < nw; ++w) {
    if (w == warp) base = total;
    total += red[w];
  }
  base += incl - own;
  PagedRun r;
  r.u0 = blockIdx.x * (total * heads) / gridDim.x;
  r.u1 = (blockIdx.x + 1) * (total * heads) / gridDim.x;
  if (r.u0 < r.u1 && r.u0 >= base * heads && r.u0 < (base + own) * heads) {
    int64_t s = s0, at = base;
    for (;; ++s) {
      const int n = paged_tiles(paged_len(a, s));
      if (r.u0 < (at + n) * heads || s + 1 >= s1) break;
      at += n;
    }
    red[32] = s;
    red[33] = at;
  }
  __syncthreads();
  r.seq = red[32];
  r.before = red[33];
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

__device__ __forceinline__ void paged_allow_join() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Adds the partial results of each (sequence, head group) that was cut, in CTA order.  A CTA
// for each CTA of the attention kernel whose run may begin one (blockIdx.x) and each head of
// a group (blockIdx.y); `heads` a group.
template <typename T>
__global__ void __launch_bounds__(128) paged_join_kernel(PagedArgs a, int heads, int groups) {
  __shared__ float s_acc[4][256], s_ml[4][2];
  __shared__ int s_n;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, n = gridDim.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const PagedRec me = a.rec[c];
  if (!(me.flags & 1)) return;
  const int G = a.Hq / a.Hk, hk = me.head / groups, g = me.head % groups * heads + h;
  if (g >= G) return;
  if (warp == 0) {  // the CTA that ends it
    int last = n - 1;
    for (int c0 = c + 1; c0 < n; c0 += 32) {
      const int f = c0 + lane < n ? a.rec[c0 + lane].flags : 0;
      const unsigned hit = __ballot_sync(0xffffffffu, (f & 4) != 0);
      if (hit) {
        last = c0 + __ffs(hit) - 1;
        break;
      }
    }
    if (lane == 0) s_n = last;
  }
  __syncthreads();
  const int last = s_n, st = paged_part_stride(a.D);
  float m = -INFINITY, l = 0.0f, acc[8] = {};
  for (int p = c + warp; p <= last; p += 4) {
    if (p > c && !(a.rec[p].flags & 2)) continue;
    const float* part = a.part + (static_cast<int64_t>(p * 2 + (p == c)) * heads + h) * st;
    const float pm = part[st - 4], pl = part[st - 3];
    const float top = fmaxf(m, pm), mm = top == -INFINITY ? 0.0f : top;
    const float f0 = exp2f(m - mm), f1 = exp2f(pm - mm);
    m = top;
    l = l * f0 + pl * f1;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < a.D) acc[i] = acc[i] * f0 + part[lane + 32 * i] * f1;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (lane + 32 * i < a.D) s_acc[warp][lane + 32 * i] = acc[i];
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(heads), 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<T>, a, heads, groups);
}

}  // namespace nf4
