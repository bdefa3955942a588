// nf4_attn_any.cu -- causal attention over packed sequences for any layout: every
// type (fp32, bf16, fp16), head widths up to 256, any strides and alignment.
//
//   o_i = sum_{j <= i} p_ij v_j,   p_ij = exp(scale q_i . k_j - lse_i)
//   dv_j = sum_i p_ij do_i,  ds_ij = p_ij (do_i . v_j - delta_i),  delta_i = do_i . o_i
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i
// over the rows of one sequence; dk and dv also over the query heads that share the
// key head.  All arithmetic is fp32, masked pairs are never touched (so a NaN in one
// reaches nobody), and each sum has one order: no atomics.  The warp holds a tile of
// 32 keys (or queries) across its lanes for the scores, then a strip of the head's
// columns across its lanes for the products.  Bound by shared-memory reads (about 9 TFLOP/s
// forward at 12289 rows): it serves the layouts that the tensor-core kernels cannot load.
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_common.cuh"
#include "elem.cuh"

namespace nf4 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kOwn = 4;               // rows a warp owns
constexpr int kRows = kWarps * kOwn;  // rows a CTA owns
constexpr int kStep = 32;             // rows of the other side per step, one per lane

// rows [r0, r0 + n) of head h of a packed tensor into dst [kStep or kRows][D + 1], zeros beyond n.
template <typename T>
__device__ __forceinline__ void stage(float* dst, const void* src, int64_t ld_t, int64_t ld_h, int h, int64_t r0,
                                      int n, int rows, int D) {
  const T* p = static_cast<const T*>(src) + h * ld_h;
  for (int i = threadIdx.x; i < rows * D; i += kThreads) {
    const int r = i / D, d = i % D;
    dst[r * (D + 1) + d] = r < n ? to_f32(p[(r0 + r) * ld_t + d]) : 0.0f;
  }
}

struct Smem {
  AttnTile tile;
};

template <int NC>
__device__ __forceinline__ void clear(float (&acc)[kOwn][NC]) {
#pragma unroll
  for (int r = 0; r < kOwn; ++r)
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[r][c] = 0.0f;
}

// dot products of the warp's kOwn rows (row-major, pitch D + 1) with this lane's row.
__device__ __forceinline__ void dots(const float* own, const float* mine, int D, float (&s)[kOwn]) {
#pragma unroll
  for (int r = 0; r < kOwn; ++r) s[r] = 0.0f;
  for (int d = 0; d < D; ++d) {
    const float x = mine[d];
#pragma unroll
    for (int r = 0; r < kOwn; ++r) s[r] = fmaf(own[r * (D + 1) + d], x, s[r]);
  }
}

// acc[c] += w * row[lane + 32 c]
template <int NC>
__device__ __forceinline__ void axpy(float (&acc)[NC], float w, const float* row, int D, int lane) {
#pragma unroll
  for (int c = 0; c < NC; ++c)
    if (lane + 32 * c < D) acc[c] = fmaf(w, row[lane + 32 * c], acc[c]);
}

template <typename T, int NC>
__device__ __forceinline__ void store_row(void* dst, int64_t ld_t, int64_t ld_h, int h, int64_t t, const float (&acc)[NC],
                                          float f, int D, int lane) {
  T* p = static_cast<T*>(dst) + t * ld_t + h * ld_h;
#pragma unroll
  for (int c = 0; c < NC; ++c)
    if (lane + 32 * c < D) p[lane + 32 * c] = from_f32<T>(acc[c] * f);
}

// Forward: grid (tiles of kRows rows, query heads).
template <typename T, int NC>
__global__ void __launch_bounds__(kThreads) attn_any_fwd_kernel(AttnArgs a) {
  extern __shared__ float smem[];
  __shared__ Smem sh;
  const int D = a.D, pitch = D + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
  float *qs = smem, *ks = qs + kRows * pitch, *vs = ks + kStep * pitch;
  int64_t g0, g1;
  gap_rows(a, &g0, &g1);
  zero_rows(static_cast<T*>(a.o), a.o_t, a.o_h, a.Hq, D, 0, g0, threadIdx.x, kThreads);
  zero_rows(static_cast<T*>(a.o), a.o_t, a.o_h, a.Hq, D, g1, a.T, threadIdx.x, kThreads);
  if (blockIdx.x == 0)
    for (int64_t t = threadIdx.x; t < a.T; t += kThreads)
      if (t < g0 || t >= g1) a.lse[h * a.T + t] = -INFINITY;
  if (warp == 0) {
    const AttnTile w = find_tile(a, blockIdx.x, kRows);
    if (lane == 0) sh.tile = w;
  }
  __syncthreads();
  const AttnTile w = sh.tile;
  if (w.tile < 0) return;
  const int i0 = w.tile * kRows, n = min(kRows, w.len - i0);
  stage<T>(qs, a.q, a.q_t, a.q_h, h, w.row0 + i0, n, kRows, D);
  const int hk = h / (a.Hq / a.Hk);
  float acc[kOwn][NC], mx[kOwn], sum[kOwn];
  clear(acc);
#pragma unroll
  for (int r = 0; r < kOwn; ++r) {
    mx[r] = -INFINITY;
    sum[r] = 0.0f;
  }
  for (int j0 = 0; j0 < i0 + n; j0 += kStep) {
    const int nk = min(kStep, w.len - j0);
    __syncthreads();
    stage<T>(ks, a.k, a.k_t, a.k_h, hk, w.row0 + j0, nk, kStep, D);
    stage<T>(vs, a.v, a.v_t, a.v_h, hk, w.row0 + j0, nk, kStep, D);
    __syncthreads();
    float s[kOwn];
    dots(qs + warp * kOwn * pitch, ks + lane * pitch, D, s);
#pragma unroll
    for (int r = 0; r < kOwn; ++r) {
      const int i = i0 + warp * kOwn + r;
      const int seen = min(nk, i - j0 + 1);  // keys of this step that row i sees
      if (i >= w.len || seen <= 0) continue;
      const float x = lane < seen ? s[r] * a.scale : -INFINITY;
      const float m = fmaxf(mx[r], warp_max(x));
      // scores that are all -inf so far weigh nothing (a row of nothing else ends as 0 / 0)
      const float mm = m == -INFINITY ? 0.0f : m;
      const float p = lane < seen ? expf(x - mm) : 0.0f;
      const float f = expf(mx[r] - mm);
      sum[r] = sum[r] * f + warp_sum(p);
      mx[r] = m;
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[r][c] *= f;
      for (int j = 0; j < seen; ++j) axpy(acc[r], __shfl_sync(0xffffffffu, p, j), vs + j * pitch, D, lane);
    }
  }
#pragma unroll
  for (int r = 0; r < kOwn; ++r) {
    const int i = i0 + warp * kOwn + r;
    if (i >= w.len) continue;
    store_row<T>(a.o, a.o_t, a.o_h, h, w.row0 + i, acc[r], 1.0f / sum[r], D, lane);
    if (a.o_rest) {  // what the rounding left over
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float x = acc[r][c] * (1.0f / sum[r]);
        acc[r][c] = x - to_f32(from_f32<T>(x));
      }
      store_row<T>(a.o_rest, static_cast<int64_t>(a.Hq) * D, D, h, w.row0 + i, acc[r], 1.0f, D, lane);
    }
    if (lane == 0) a.lse[h * a.T + w.row0 + i] = mx[r] + logf(sum[r]);
  }
}

// delta[h][t] = do . o, one warp per (t, h).
template <typename T>
__global__ void __launch_bounds__(kThreads) attn_any_delta_kernel(AttnArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t n = a.T * a.Hq, nw = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < n; i += nw) {
    const int64_t t = i / a.Hq;
    const int h = static_cast<int>(i % a.Hq);
    const T* o = static_cast<const T*>(a.o) + t * a.o_t + h * a.o_h;
    const T* g = static_cast<const T*>(a.go) + t * a.go_t + h * a.go_h;
    float s = 0.0f;
    const T* rest = a.o_rest ? static_cast<const T*>(a.o_rest) + i * a.D : nullptr;
    for (int d = lane; d < a.D; d += 32) s = fmaf(to_f32(o[d]) + (rest ? to_f32(rest[d]) : 0.0f), to_f32(g[d]), s);
    s = warp_sum(s);
    if (lane == 0) a.delta[h * a.T + t] = s;
  }
}

// dq: grid (tiles of kRows rows, query heads).
template <typename T, int NC>
__global__ void __launch_bounds__(kThreads) attn_any_dq_kernel(AttnArgs a) {
  extern __shared__ float smem[];
  __shared__ Smem sh;
  const int D = a.D, pitch = D + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
  float *qs = smem, *gs = qs + kRows * pitch, *ks = gs + kRows * pitch, *vs = ks + kStep * pitch;
  int64_t g0, g1;
  gap_rows(a, &g0, &g1);
  zero_rows(static_cast<T*>(a.gq), a.gq_t, a.gq_h, a.Hq, D, 0, g0, threadIdx.x, kThreads);
  zero_rows(static_cast<T*>(a.gq), a.gq_t, a.gq_h, a.Hq, D, g1, a.T, threadIdx.x, kThreads);
  if (warp == 0) {
    const AttnTile w = find_tile(a, blockIdx.x, kRows);
    if (lane == 0) sh.tile = w;
  }
  __syncthreads();
  const AttnTile w = sh.tile;
  if (w.tile < 0) return;
  const int i0 = w.tile * kRows, n = min(kRows, w.len - i0);
  stage<T>(qs, a.q, a.q_t, a.q_h, h, w.row0 + i0, n, kRows, D);
  stage<T>(gs, a.go, a.go_t, a.go_h, h, w.row0 + i0, n, kRows, D);
  const int hk = h / (a.Hq / a.Hk);
  float acc[kOwn][NC];
  clear(acc);
  for (int j0 = 0; j0 < i0 + n; j0 += kStep) {
    const int nk = min(kStep, w.len - j0);
    __syncthreads();
    stage<T>(ks, a.k, a.k_t, a.k_h, hk, w.row0 + j0, nk, kStep, D);
    stage<T>(vs, a.v, a.v_t, a.v_h, hk, w.row0 + j0, nk, kStep, D);
    __syncthreads();
    float s[kOwn], dp[kOwn];
    dots(qs + warp * kOwn * pitch, ks + lane * pitch, D, s);
    dots(gs + warp * kOwn * pitch, vs + lane * pitch, D, dp);
#pragma unroll
    for (int r = 0; r < kOwn; ++r) {
      const int i = i0 + warp * kOwn + r;
      const int seen = min(nk, i - j0 + 1);
      if (i >= w.len || seen <= 0) continue;
      const int64_t at = h * a.T + w.row0 + i;
      const float ds = lane < seen ? expf(s[r] * a.scale - a.lse[at]) * (dp[r] - a.delta[at]) : 0.0f;
      for (int j = 0; j < seen; ++j) axpy(acc[r], __shfl_sync(0xffffffffu, ds, j), ks + j * pitch, D, lane);
    }
  }
#pragma unroll
  for (int r = 0; r < kOwn; ++r) {
    const int i = i0 + warp * kOwn + r;
    if (i < w.len) store_row<T>(a.gq, a.gq_t, a.gq_h, h, w.row0 + i, acc[r], a.scale, D, lane);
  }
}

// dk and dv: grid (tiles of kRows keys, key heads); the query heads that share the
// key head one after another.
template <typename T, int NC>
__global__ void __launch_bounds__(kThreads) attn_any_dkv_kernel(AttnArgs a) {
  extern __shared__ float smem[];
  __shared__ Smem sh;
  const int D = a.D, pitch = D + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, hk = blockIdx.y;
  float *ks = smem, *vs = ks + kRows * pitch, *qs = vs + kRows * pitch, *gs = qs + kStep * pitch;
  int64_t g0, g1;
  gap_rows(a, &g0, &g1);
  zero_rows(static_cast<T*>(a.gk), a.gk_t, a.gk_h, a.Hk, D, 0, g0, threadIdx.x, kThreads);
  zero_rows(static_cast<T*>(a.gk), a.gk_t, a.gk_h, a.Hk, D, g1, a.T, threadIdx.x, kThreads);
  zero_rows(static_cast<T*>(a.gv), a.gv_t, a.gv_h, a.Hk, D, 0, g0, threadIdx.x, kThreads);
  zero_rows(static_cast<T*>(a.gv), a.gv_t, a.gv_h, a.Hk, D, g1, a.T, threadIdx.x, kThreads);
  if (warp == 0) {
    const AttnTile w = find_tile(a, blockIdx.x, kRows);
    if (lane == 0) sh.tile = w;
  }
  __syncthreads();
  const AttnTile w = sh.tile;
  if (w.tile < 0) return;
  const int j0 = w.tile * kRows, n = min(kRows, w.len - j0);
  stage<T>(ks, a.k, a.k_t, a.k_h, hk, w.row0 + j0, n, kRows, D);
  stage<T>(vs, a.v, a.v_t, a.v_h, hk, w.row0 + j0, n, kRows, D);
  float dk[kOwn][NC], dv[kOwn][NC];
  clear(dk);
  clear(dv);
  const int G = a.Hq / a.Hk;
  for (int g = 0; g < G; ++g) {
    const int h = hk * G + g;
    for (int i0 = j0; i0 < w.len; i0 += kStep) {
      const int nq = min(kStep, w.len - i0);
      __syncthreads();
      stage<T>(qs, a.q, a.q_t, a.q_h, h, w.row0 + i0, nq, kStep, D);
      stage<T>(gs, a.go, a.go_t, a.go_h, h, w.row0 + i0, nq, kStep, D);
      __syncthreads();
      float s[kOwn], dp[kOwn];
      dots(ks + warp * kOwn * pitch, qs + lane * pitch, D, s);
      dots(vs + warp * kOwn * pitch, gs + lane * pitch, D, dp);
      float lse = 0.0f, delta = 0.0f;
      if (lane < nq) {
        lse = a.lse[h * a.T + w.row0 + i0 + lane];
        delta = a.delta[h * a.T + w.row0 + i0 + lane];
      }
#pragma unroll
      for (int r = 0; r < kOwn; ++r) {
        const int j = j0 + warp * kOwn + r;
        const int from = max(0, j - i0);  // first query of this step that sees key j
        if (j >= w.len || from >= nq) continue;
        const bool on = lane >= from && lane < nq;
        const float p = on ? expf(s[r] * a.scale - lse) : 0.0f;
        const float ds = on ? p * (dp[r] - delta) : 0.0f;
        for (int i = from; i < nq; ++i) {
          axpy(dv[r], __shfl_sync(0xffffffffu, p, i), gs + i * pitch, D, lane);
          axpy(dk[r], __shfl_sync(0xffffffffu, ds, i), qs + i * pitch, D, lane);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kOwn; ++r) {
    const int j = j0 + warp * kOwn + r;
    if (j >= w.len) continue;
    store_row<T>(a.gk, a.gk_t, a.gk_h, hk, w.row0 + j, dk[r], a.scale, D, lane);
    store_row<T>(a.gv, a.gv_t, a.gv_h, hk, w.row0 + j, dv[r], 1.0f, D, lane);
  }
}

template <typename K>
cudaError_t with_smem(K kern, size_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

template <typename T, int NC>
cudaError_t launch_nc(bool backward, const AttnArgs& a, int sms, cudaStream_t s) {
  const size_t pitch = static_cast<size_t>(a.D + 1) * sizeof(float);
  const dim3 gq(static_cast<unsigned>(attn_tiles(a, kRows)), a.Hq, 1), gk(gq.x, a.Hk, 1);
  cudaError_t e;
  if (!backward) {
    const size_t bytes = (kRows + 2 * kStep) * pitch;
    if ((e = with_smem(attn_any_fwd_kernel<T, NC>, bytes)) != cudaSuccess) return e;
    attn_any_fwd_kernel<T, NC><<<gq, kThreads, bytes, s>>>(a);
    return cudaGetLastError();
  }
  const size_t bytes = (2 * kRows + 2 * kStep) * pitch;
  if ((e = with_smem(attn_any_dq_kernel<T, NC>, bytes)) != cudaSuccess) return e;
  if ((e = with_smem(attn_any_dkv_kernel<T, NC>, bytes)) != cudaSuccess) return e;
  const int64_t want = (a.T * a.Hq + kWarps - 1) / kWarps, most = 16 * static_cast<int64_t>(sms);
  attn_any_delta_kernel<T><<<static_cast<unsigned>(want < most ? want : most), kThreads, 0, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  attn_any_dq_kernel<T, NC><<<gq, kThreads, bytes, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  attn_any_dkv_kernel<T, NC><<<gk, kThreads, bytes, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(bool backward, const AttnArgs& a, int sms, cudaStream_t s) {
  if (a.D <= 64) return launch_nc<T, 2>(backward, a, sms, s);
  if (a.D <= 128) return launch_nc<T, 4>(backward, a, sms, s);
  return launch_nc<T, 8>(backward, a, sms, s);
}

}  // namespace

cudaError_t launch_attn_any(bool backward, int dtype, const AttnArgs& a, int sms, cudaStream_t s) {
  if (dtype == NF4_DTYPE_F32) return launch_typed<float>(backward, a, sms, s);
  if (dtype == NF4_DTYPE_BF16) return launch_typed<__nv_bfloat16>(backward, a, sms, s);
  return launch_typed<__half>(backward, a, sms, s);
}

}  // namespace nf4
