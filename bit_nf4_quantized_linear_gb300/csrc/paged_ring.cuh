// paged_ring.cuh -- a warp's stream of cache rows through shared memory: 16-byte asynchronous
// copies of one tile of tokens after another, over the borders of sequences and heads, some
// tiles ahead of their use.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "paged_common.cuh"

namespace nf4 {

// Pieces of 16 bytes lie XOR-swizzled by row, so that eight rows' pieces of one column lie in
// different banks.
template <int ROW_BYTES>
__device__ __forceinline__ uint32_t at_chunk(int row, int chunk) {
  return static_cast<uint32_t>(row * ROW_BYTES + ((chunk ^ (row & 7)) << 4));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {  // zeros past `bytes`
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The copies of a tile of ROWS tokens, keys and then values, rows of W values; columns past D
// and rows past a length or without a page are zeros that nothing reads.  Lane i copies column
// piece i % kPieces (and the 32nd after it, of rows that long) of rows i / kPieces and every
// kPer-th after it.
template <typename T, int W, int ROWS>
struct TileCopies {
  static constexpr int kRowBytes = W * static_cast<int>(sizeof(T)), kAll = kRowBytes / 16;
  static constexpr int kPieces = kAll < 32 ? kAll : 32, kPer = 32 / kPieces, kTurns = kAll / kPieces;  // turns of a warp a row
  static constexpr int kTurn = 512 / static_cast<int>(sizeof(T));  // columns between turns
  static constexpr int kHalf = ROWS * kRowBytes, kStage = 2 * kHalf;
  static_assert(kPieces >= 1 && kPer >= 1 && ROWS % 8 == 0 && ROWS <= 16, "a row a warp's copy at least");

  uint32_t dst0;
  uint32_t* s_valid;  // [ring slots]: which rows of a tile are tokens
  int row0, col;
  bool in, one_page;
  int page, slot;  // of the tile that is copied next, where one page holds it: looked up a tile ahead

  __device__ __forceinline__ TileCopies(const PagedArgs& a, uint32_t ring, uint32_t* valid) {
    const int lane = threadIdx.x & 31;
    row0 = lane / kPieces;
    col = lane % kPieces * (16 / static_cast<int>(sizeof(T)));
    in = col < a.D;
    one_page = a.page_size % ROWS == 0;  // a tile lies in one page
    dst0 = ring + at_chunk<kRowBytes>(row0, lane % kPieces);
    s_valid = valid;
  }

  // Looks up the page of the tokens from tok0 on of the unit `load`; before its start().
  __device__ __forceinline__ void look_up(const PagedArgs& a, const Walk& load, int tok0) {
    if (one_page && load.left > 0 && tok0 < load.len) {
      const unsigned p = paged_index(a, tok0);
      slot = tok0 - static_cast<int>(p) * a.page_size;
      page = a.table[load.seq * a.ld_table + p];
    }
  }

  // Starts the copies of the tokens from tok0 on of the unit `load`, key head hk, into ring slot `st`.
  __device__ __forceinline__ void start(const PagedArgs& a, const Walk& load, int tok0, int hk, int st) const {
    const int lane = threadIdx.x & 31, rows = load.len - tok0;
    if (load.left > 0 && rows > 0) {
      const uint32_t to = dst0 + st * kStage;
      // a row's swizzle repeats after eight rows
      auto dst = [&](int i) { return (i * kPer % 8 == 0 ? to : to ^ (i * kPer % 8 << 4)) + i * kPer * kRowBytes; };
      const T* none = static_cast<const T*>(a.q);
      constexpr unsigned kFull = (1u << ROWS) - 1u;
      unsigned valid;
      if (one_page) {
        const bool known = page >= 0 && page < a.pages;
        if (!known && a.status) atomicCAS(a.status, 0, kStatusBadOffsets);
        const int n = known ? rows : 0;
        valid = n >= ROWS ? kFull : (1u << n) - 1u;
        const T *kp = none, *vp = none;
        int64_t ks = 0, vs = 0;
        if (in && known) {
          kp = static_cast<const T*>(a.k) + (page * a.k_page + (slot + row0) * a.k_token + hk * a.k_head + col);
          vp = static_cast<const T*>(a.v) + (page * a.v_page + (slot + row0) * a.v_token + hk * a.v_head + col);
          ks = kPer * a.k_token;
          vs = kPer * a.v_token;
        }
        if (n >= ROWS && kTurns == 1) {
          const int bytes = in ? 16 : 0;
#pragma unroll
          for (int i = 0; i < ROWS / kPer; ++i) {
            copy16(dst(i), kp, bytes);
            copy16(dst(i) + kHalf, vp, bytes);
            kp += ks;
            vp += vs;
          }
        } else {
#pragma unroll
          for (int i = 0; i < ROWS / kPer; ++i) {
#pragma unroll
            for (int t = 0; t < kTurns; ++t) {
              const bool row = col + t * kTurn < a.D && i * kPer + row0 < n;
              copy16(dst(i) + t * 512, row ? kp + t * kTurn : none, row ? 16 : 0);
              copy16(dst(i) + kHalf + t * 512, row ? vp + t * kTurn : none, row ? 16 : 0);
            }
            kp += ks;
            vp += vs;
          }
        }
      } else {
        // lane i < 16 looks up the key row of token i, lane 16 + i its value row
        const int tok = tok0 + (lane & (ROWS - 1));
        int64_t at = 0;
        bool ok = false;
        if (tok < load.len) {
          int slot;
          const int64_t page = paged_slot(a, load.seq, tok, &slot);
          ok = page >= 0;
          if (ok)
            at = lane < 16 ? page * a.k_page + slot * a.k_token + hk * a.k_head
                           : page * a.v_page + slot * a.v_token + hk * a.v_head;
        }
        valid = __ballot_sync(0xffffffffu, ok) & kFull;
#pragma unroll
        for (int i = 0; i < ROWS / kPer; ++i) {
          const int r = i * kPer + row0;
          const int64_t ak = __shfl_sync(0xffffffffu, at, r), av = __shfl_sync(0xffffffffu, at, r + 16);
#pragma unroll
          for (int t = 0; t < kTurns; ++t) {
            const int c = col + t * kTurn, bytes = (valid >> r & 1) && c < a.D ? 16 : 0;
            copy16(dst(i) + t * 512, bytes ? static_cast<const T*>(a.k) + ak + c : none, bytes);
            copy16(dst(i) + kHalf + t * 512, bytes ? static_cast<const T*>(a.v) + av + c : none, bytes);
          }
        }
      }
      if (lane == 0) s_valid[st] = valid;
    }
    copies_commit();
  }
};

}  // namespace nf4
