// attn_mma.cuh -- tcgen05 / TMA pieces of the attention kernels: operands from tensor
// memory, wide tensor-memory loads and stores, packed fp32 arithmetic, bounded waits.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_common.cuh"
#include "elem.cuh"
#include "sm100_ptx.cuh"

namespace nf4 {

using namespace nf4ptx;

constexpr int kAttnTile = 128;                  // rows of a tile (MMA M, and N of the scores)
constexpr int kPanelBytes = kAttnTile * 128;    // a [128 rows][64 columns] 16-bit panel, 128-byte swizzled
constexpr uint64_t kAttnTimeoutNs = 2000000000; // bound of every wait

// What the roles of a CTA share about giving up.
struct AttnGuard {
  volatile int* abort_flag;
  int* status;
};

static __device__ __noinline__ bool attn_wait_slow(uint32_t bar, uint32_t parity, const AttnGuard& g) {
  if (mbar_try_wait_sleep(bar, parity, 100000)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait_sleep(bar, parity, 100000)) return true;
    if (*g.abort_flag) return false;
    if (globaltimer_ns() - t0 > kAttnTimeoutNs) {
      *g.abort_flag = 1;
      if (g.status) atomicCAS(g.status, 0, kStatusTimeout);
      return false;
    }
  }
}

// Bounded wait for a barrier phase; false: this role gives up (a timeout is recorded).
__device__ __forceinline__ bool attn_wait(uint32_t bar, uint32_t parity, const AttnGuard& g) {
  if (mbar_test_wait(bar, parity)) return true;
  return attn_wait_slow(bar, parity, g);
}

// The same for copies and MMAs in flight that must land before the CTA may exit.
static __device__ __noinline__ void attn_drain(uint32_t bar, uint32_t parity, const AttnGuard& g) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_sleep(bar, parity, 20000)) {
    if (globaltimer_ns() - t0 > kAttnTimeoutNs) {
      if (g.status) atomicCAS(g.status, 0, kStatusTimeout);
      return;
    }
  }
}

// True in one lane of a converged warp, the same each time.  Asynchronous operations (MMAs,
// commits, copies) are issued under it and not under `lane == 0`: their operands lie in
// registers of the warp, and only here does the compiler know that one lane is active (an
// MMA took about 100 cycles to issue under the other).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// Tile of 128 rows x 64 columns of one head of a [T][heads][D] tensor.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// D(tmem) (+)= A(tmem) * B(smem): A's row is the lane, two 16-bit values a column.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Operand tile [128 rows][64-column panels], 128-byte swizzled rows.  Rows are M / N
// and columns the contraction (K-major): 16 columns further is 32 bytes, the next
// panel kPanelBytes.  Or columns are M / N and rows the contraction (MN-major): 16 rows
// further is 2 KB.  Steps only change the descriptor's address field (in 16-byte units),
// so one thread issues an MMA every few instructions.
__device__ __forceinline__ uint64_t desc_k_major(uint32_t saddr) { return smem_desc_sw128(saddr, 16, 1024); }
__device__ __forceinline__ uint64_t desc_mn_major(uint32_t saddr) { return smem_desc_sw128(saddr, kPanelBytes, 1024); }

// D = A B^T over the head's columns in steps of 16, both operands in shared memory.  With
// FULL the panels are full: a fixed number of steps, unrolled.  Else `ksteps` steps in a
// rolled loop; no MMA stands under a condition of its own (unrolled MMAs guarded by
// `k < ksteps` came out wrong).
template <bool FULL, int PANELS>
__device__ __forceinline__ void mma_over_columns(uint32_t d, uint32_t a_tile, uint32_t b_tile, uint32_t idesc, int ksteps) {
  uint64_t da = desc_k_major(a_tile), db = desc_k_major(b_tile);
  if constexpr (FULL) {
#pragma unroll
    for (int k = 0; k < 4 * PANELS; ++k) {
      const uint64_t off = (k >> 2) * (kPanelBytes >> 4) + (k & 3) * 2;
      mma_bf16_ss(d, da + off, db + off, idesc, k > 0);
    }
  } else {
#pragma unroll 1
    for (int k = 0; k < ksteps; ++k) {
      const uint64_t off = (k >> 2) * (kPanelBytes >> 4) + (k & 3) * 2;
      mma_bf16_ss(d, da + off, db + off, idesc, k > 0);
    }
  }
}

// D (+)= A B over a tile's 128 rows: A in tensor memory, 16 rows to 8 columns, its second
// half `half` columns after the first; B in shared memory.
__device__ __forceinline__ void mma_over_rows(uint32_t d, uint32_t a_tmem, int half, uint32_t b_tile, uint32_t idesc,
                                              bool more) {
  const uint64_t db = desc_mn_major(b_tile);
#pragma unroll
  for (int k = 0; k < 8; ++k)
    mma_f16_ts(d, a_tmem + (k >> 2) * half + (k & 3) * 8, db + k * 128, idesc, more || k > 0);
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t* r);
template <>
__device__ __forceinline__ void tmem_ld<32>(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23,"
      " %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// Waits for this thread's tensor-memory loads, into `r` among others.  The loads write
// their registers asynchronously, and nothing but this ties the registers to the wait: the
// empty statements keep the compiler from using them before it.
template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                      "+r"(r[i + 6]), "+r"(r[i + 7])::"memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24,"
      " %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// This warp's tensor-memory accesses are done: one arrival for all its lanes.
__device__ __forceinline__ void arrive_warp(uint32_t bar) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
  __syncwarp();
}

// Bounded wait of a converged warp: one answer for all lanes.
__device__ __forceinline__ bool attn_wait_warp(uint32_t bar, uint32_t parity, const AttnGuard& g) {
  const bool ok = __all_sync(0xffffffffu, attn_wait(bar, parity, g));
  __syncwarp();
  return ok;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two values rounded to 16 bits, the first in the low half.
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <bool F16>
__device__ __forceinline__ float lo16(uint32_t w) {
  return F16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(w))) : __uint_as_float(w << 16);
}
template <bool F16>
__device__ __forceinline__ float hi16(uint32_t w) {
  return F16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(w >> 16))) : __uint_as_float(w & 0xffff0000u);
}

// Whether either half of w is an infinity or a NaN (its exponent bits all ones).
template <bool F16>
__device__ __forceinline__ bool nonfinite16(uint32_t w) {
  constexpr uint32_t e = F16 ? 0x7c00u : 0x7f80u;
  return (w & e) == e || ((w >> 16) & e) == e;
}

// `warps` warps (this one the `me`-th) clear rows >= `rows` of an operand tile in shared
// memory and, with `values`, replace the infinities and NaNs of the others by zero; true
// (in every lane of the warp) when it met any.  Ends with the fence that lets the tensor
// cores see the stores.  The scan costs one fused multiply-add a word: x * 0 + acc stays
// 0 until an x is not finite.
template <bool F16, int PANELS>
__device__ __forceinline__ bool clean_tile(uint8_t* tile, int rows, bool values, int me, int warps) {
  const int lane = threadIdx.x & 31;
  constexpr int kPieces = PANELS * kAttnTile * 8;  // of 16 bytes; a row is 8 of a panel
  bool any = false;
  if (rows < kAttnTile) {
    const int dead = (kAttnTile - rows) * 8;
#pragma unroll
    for (int p = 0; p < PANELS; ++p)
      for (int i = me * 32 + lane; i < dead; i += warps * 32)
        *reinterpret_cast<uint4*>(tile + p * kPanelBytes + rows * 128 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  if (values) {
    // the cleared rows may be read before or after: what they held does not matter
    for (int i0 = me * 256 + lane; i0 < kPieces; i0 += warps * 256) {
      uint4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = reinterpret_cast<const uint4*>(tile)[i0 + k * 32];
      uint32_t acc = 0u;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (F16)
            asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w[e]), "r"(0u));
          else
            asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w[e]), "r"(0u));
        }
      }
      if ((acc & 0x7fff7fffu) == 0u) continue;
      for (int k = 0; k < 8; ++k) {
        const int i = i0 + k * 32;
        if (((i >> 3) & (kAttnTile - 1)) >= rows) continue;
        uint32_t* w = reinterpret_cast<uint32_t*>(tile) + i * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          constexpr uint32_t x = F16 ? 0x7c00u : 0x7f80u;
          uint32_t u = w[e];
          if (!nonfinite16<F16>(u)) continue;
          if ((u & x) == x) u &= 0xffff0000u;
          if (((u >> 16) & x) == x) u &= 0x0000ffffu;
          w[e] = u;
          any = true;
        }
      }
    }
  }
  fence_proxy_async_smem();
  return __any_sync(0xffffffffu, any);
}

}  // namespace nf4
