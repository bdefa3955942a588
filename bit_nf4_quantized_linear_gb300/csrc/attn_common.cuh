// attn_common.cuh -- what the attention kernels share: which sequence and tile a CTA
// works on, and the rows that belong to no sequence.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"

namespace nf4 {

struct AttnTile {
  int64_t row0;  // first row of the sequence in the packed tensors
  int len;       // rows of the sequence
  int tile;      // tile within the sequence; -1: the id is past the last tile
};

// Bounds of sequence b, forced into 0 <= start <= end <= T: bad offsets cannot lead
// outside the tensors, and are recorded.
__device__ __forceinline__ void seq_bounds(const AttnArgs& a, int64_t b, int64_t* start, int64_t* end) {
  if (!a.cu_seqlens) {
    *start = 0;
    *end = a.T;
    return;
  }
  const int64_t s = a.cu_seqlens[b], e = a.cu_seqlens[b + 1];
  if ((s < 0 || e < s || e > a.T) && a.status) atomicCAS(a.status, 0, kStatusBadOffsets);
  *start = s < 0 ? 0 : (s > a.T ? a.T : s);
  *end = e < *start ? *start : (e > a.T ? a.T : e);
}

// The sequence and tile of tile number `id` of ceil(len / rows) tiles in each sequence.
// Under the causal mask the last query tile, or the first key tile, has the most work,
// and a grid deals its CTAs in order, so the longest come first: over all sequences where
// there are at most 32 of them, else sequence by sequence.  Called by one full warp; all
// lanes get the answer.
__device__ __forceinline__ AttnTile find_tile(const AttnArgs& a, int64_t id, int rows, bool last_first = true) {
  const int lane = threadIdx.x & 31;
  AttnTile r{0, 0, -1};
  if (a.nseq <= 32) {
    int64_t s = 0, e = 0;
    if (lane < a.nseq) seq_bounds(a, lane, &s, &e);
    const int tiles = static_cast<int>((e - s + rows - 1) / rows);  // its tiles have 1 .. tiles steps of work
    // tiles of at least `steps` steps in all sequences
    auto at_least = [&](int steps) { return __reduce_add_sync(0xffffffffu, max(0, tiles - steps + 1)); };
    int lo = 1, hi = __reduce_max_sync(0xffffffffu, tiles) + 1;  // the largest `steps` with more than id such tiles
    if (id >= at_least(1)) return r;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (at_least(mid) > id) lo = mid; else hi = mid;
    }
    const int rank = static_cast<int>(id) - at_least(lo + 1);  // among the sequences with a tile of lo steps
    const unsigned have = __ballot_sync(0xffffffffu, tiles >= lo);
    // the (rank + 1)-th sequence with one
    const int before = __popc(have & ((1u << lane) - 1u));
    const int src = __ffs(__ballot_sync(0xffffffffu, (have >> lane & 1u) && before == rank)) - 1;
    r.row0 = __shfl_sync(0xffffffffu, s, src);
    r.len = static_cast<int>(__shfl_sync(0xffffffffu, e - s, src));
    r.tile = last_first ? lo - 1 : __shfl_sync(0xffffffffu, tiles, src) - lo;
    return r;
  }
  int64_t base = 0;
  for (int64_t b0 = 0; b0 < a.nseq; b0 += 32) {
    int64_t s = 0, e = 0;
    if (b0 + lane < a.nseq) seq_bounds(a, b0 + lane, &s, &e);
    const int64_t tiles = (e - s + rows - 1) / rows;
    int64_t incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + incl > id);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int64_t before = base + incl - tiles;
      r.row0 = __shfl_sync(0xffffffffu, s, src);
      r.len = static_cast<int>(__shfl_sync(0xffffffffu, e - s, src));
      r.tile = static_cast<int>(__shfl_sync(0xffffffffu, last_first ? tiles - 1 - (id - before) : id - before, src));
      return r;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return r;
}

// Rows before the first sequence and after the last.
__device__ __forceinline__ void gap_rows(const AttnArgs& a, int64_t* head_end, int64_t* tail_start) {
  *head_end = 0;
  *tail_start = a.T;
  if (a.cu_seqlens) {
    const int64_t h = a.cu_seqlens[0], t = a.cu_seqlens[a.nseq];
    *head_end = h < 0 ? 0 : (h > a.T ? a.T : h);
    *tail_start = t < *head_end ? *head_end : (t > a.T ? a.T : t);
  }
}

// Zeros in rows [lo, hi) of every head of `p`, spread over the whole grid; this thread is
// number `me` of the `of` that take part in each CTA.
template <typename T>
__device__ __forceinline__ void zero_rows(T* p, int64_t ld_t, int64_t ld_h, int heads, int D, int64_t lo, int64_t hi, int me,
                                          int of) {
  const int64_t n = (hi - lo) * heads * D;
  const int64_t cta = blockIdx.x + static_cast<int64_t>(gridDim.x) * blockIdx.y;
  const int64_t step = static_cast<int64_t>(gridDim.x) * gridDim.y * of;
  for (int64_t i = cta * of + me; i < n; i += step) {
    const int64_t d = i % D, h = (i / D) % heads, t = lo + i / (static_cast<int64_t>(D) * heads);
    p[t * ld_t + h * ld_h + d] = T(0.0f);
  }
}

}  // namespace nf4
