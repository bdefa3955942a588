// nf4_adamw.cu -- one AdamW step over many tensors in one launch, with fp32 states
// or with states in 8 bits.
//
// Per value, the moments by single fp32 operations rounded to nearest (no FMA), so that
// the states do not depend on how the compiler contracts the expression:
//   m = m b1 + g (1 - b1),  v = v b2 + (g g)(1 - b2),  g = grad * grad_scale
//   p = p - (lr wd p + (lr / c1) (m / (sqrt(v) / sqrt(c2) + eps))),  c_i = 1 - b_i^step
// 8-bit states (Dettmers et al. 2022, "8-bit Optimizers via Block-wise
// Quantization"): blocks of 256 values of a tensor share an fp32 scale, the block's
// max |x|; a value is the nearest level of x / scale in the dynamic map (signed for
// m, unsigned for v), ties to the lower index; the update of p uses the m and v
// from before they are rounded.  A block whose values are all zero gets scale 0.  A
// NaN in a block makes its scale NaN, so the whole block reads as NaN.
#include <cuda_runtime.h>

#include <cstdint>

#include "elem.cuh"
#include "internal.h"

namespace nf4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = kAdamBlock / 32;  // values of a block per lane

// max that keeps a NaN of either side.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Count of midpoints below r (ascending), each rounded down to fp32: r > mid is the
// same as r > floor32(mid) for an fp32 r.
__device__ __forceinline__ int nearest(const float* mid, float r) {
  int lo = 0, hi = 255;
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (mid[m] < r) lo = m + 1; else hi = m;
  }
  return lo;
}

// The tensor that holds global block b: first index with blk0[i + 1] > b.
__device__ __forceinline__ int find_tensor(const AdamTable& tab, int64_t b) {
  int lo = 0, hi = tab.count - 1;
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (tab.blk0[m + 1] > b) hi = m; else lo = m + 1;
  }
  return lo;
}

// One warp per block of 256 values.
template <typename T, int BITS>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ AdamTable tab, AdamArgs a) {
  __shared__ float lev[2][256], mid[2][255];
  if (BITS == 8) {
    for (int i = threadIdx.x; i < 256; i += kThreads) {
      for (int k = 0; k < 2; ++k) {
        const float* L = k ? a.levels_v : a.levels_m;
        lev[k][i] = L[i];
        if (i < 255)
          mid[k][i] = __double2float_rd((static_cast<double>(L[i]) + static_cast<double>(L[i + 1])) * 0.5);
      }
    }
    __syncthreads();
  }
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  const int lane = threadIdx.x & 31;
  const int64_t nw = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); b < tab.blk0[tab.count]; b += nw) {
    const int ti = find_tensor(tab, b);
    const AdamTensor& t = tab.t[ti];
    const int64_t blk = b - tab.blk0[ti], base = blk * kAdamBlock;
    T* p = static_cast<T*>(t.param);
    const T* g = static_cast<const T*>(t.grad);
    const float sm = BITS == 8 ? t.m_absmax[blk] : 0.0f, sv = BITS == 8 ? t.v_absmax[blk] : 0.0f;
    float m[kPer], v[kPer];
    float top_m = 0.0f, top_v = 0.0f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int64_t i = base + k * 32 + lane;
      m[k] = v[k] = 0.0f;
      if (i >= t.n) continue;
      const float gr = a.grad_scale ? __fmul_rn(to_f32(g[i]), gs) : to_f32(g[i]);
      float m0, v0;
      if (BITS == 8) {
        m0 = __fmul_rn(lev[0][static_cast<const uint8_t*>(t.m)[i]], sm);
        v0 = __fmul_rn(lev[1][static_cast<const uint8_t*>(t.v)[i]], sv);
      } else {
        m0 = static_cast<const float*>(t.m)[i];
        v0 = static_cast<const float*>(t.v)[i];
      }
      m[k] = __fadd_rn(__fmul_rn(m0, a.beta1), __fmul_rn(gr, a.one_minus_beta1));
      v[k] = __fadd_rn(__fmul_rn(v0, a.beta2), __fmul_rn(__fmul_rn(gr, gr), a.one_minus_beta2));
      const float den = __fadd_rn(__fmul_rn(__fsqrt_rn(v[k]), a.inv_sqrt_c2), a.eps);
      const float q = __fdiv_rn(m[k], den);
      // p - (lr wd p + step q): the rounding of the small bracket does not show in p
      const float p0 = to_f32(p[i]);
      p[i] = from_f32<T>(__fsub_rn(p0, __fmaf_rn(a.decay, p0, __fmul_rn(a.step_size, q))));
      top_m = max_nan(top_m, fabsf(m[k]));
      top_v = max_nan(top_v, fabsf(v[k]));
    }
    if (BITS == 8) {
      top_m = warp_max_nan(top_m);
      top_v = warp_max_nan(top_v);
      const float dm = top_m > 0.0f ? top_m : 1.0f, dv = top_v > 0.0f ? top_v : 1.0f;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int64_t i = base + k * 32 + lane;
        if (i >= t.n) continue;
        static_cast<uint8_t*>(t.m)[i] = static_cast<uint8_t>(nearest(mid[0], __fdiv_rn(m[k], dm)));
        static_cast<uint8_t*>(t.v)[i] = static_cast<uint8_t>(nearest(mid[1], __fdiv_rn(v[k], dv)));
      }
      if (lane == 0) {
        t.m_absmax[blk] = top_m;
        t.v_absmax[blk] = top_v;
      }
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int64_t i = base + k * 32 + lane;
        if (i >= t.n) continue;
        static_cast<float*>(t.m)[i] = m[k];
        static_cast<float*>(t.v)[i] = v[k];
      }
    }
  }
}

// out[i] = levels[codes[i]] * absmax[i / 256] for both states.
__global__ void __launch_bounds__(kThreads) adamw_values_kernel(AdamValuesArgs a) {
  __shared__ float lev[2][256];
  for (int i = threadIdx.x; i < 256; i += kThreads) {
    lev[0][i] = a.levels_m[i];
    lev[1][i] = a.levels_v[i];
  }
  __syncthreads();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < a.n;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    a.out_m[i] = __fmul_rn(lev[0][a.m[i]], a.m_absmax[i / kAdamBlock]);
    a.out_v[i] = __fmul_rn(lev[1][a.v[i]], a.v_absmax[i / kAdamBlock]);
  }
}

int grid_of(int64_t blocks, int sms) {
  const int64_t want = (blocks + kWarps - 1) / kWarps, most = 8 * static_cast<int64_t>(sms);
  return static_cast<int>(want < most ? want : most);
}

template <typename T>
cudaError_t launch_typed(int bits, const AdamTable& tab, const AdamArgs& a, int sms, cudaStream_t s) {
  const int grid = grid_of(tab.blk0[tab.count], sms);
  if (bits == 8)
    adamw_kernel<T, 8><<<grid, kThreads, 0, s>>>(tab, a);
  else
    adamw_kernel<T, 32><<<grid, kThreads, 0, s>>>(tab, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adamw(int dtype, int bits, const AdamTable& tab, const AdamArgs& a, int sms, cudaStream_t s) {
  if (tab.count == 0 || tab.blk0[tab.count] == 0) return cudaSuccess;
  if (dtype == NF4_DTYPE_F32) return launch_typed<float>(bits, tab, a, sms, s);
  if (dtype == NF4_DTYPE_BF16) return launch_typed<__nv_bfloat16>(bits, tab, a, sms, s);
  return launch_typed<__half>(bits, tab, a, sms, s);
}

cudaError_t launch_adamw_values(const AdamValuesArgs& a, int sms, cudaStream_t s) {
  const int64_t want = (a.n + kThreads - 1) / kThreads, most = 8 * static_cast<int64_t>(sms);
  adamw_values_kernel<<<static_cast<unsigned>(want < most ? want : most), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace nf4
