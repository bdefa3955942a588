// nf4_norm.cu -- the norms before and after a block, fused with the block's gate,
// the residual scale and the residual sum, and their backward.
//
// Per row (token) of width H, all in fp32 from the inputs' own type:
//   n = y rstd(y) w_post          (no w_post: n = y)
//   z = r + s g n                 (the residual stream after the block)
//   h = z rstd(z) w_pre           (the next block's input)
// with rstd(x) = 1 / sqrt(mean(x^2) + eps), g one value per channel (fp32), one per
// token and channel (the activations' type), or 1.  z and h are each rounded once;
// h comes from the unrounded z.  The backward takes gz, gh and recomputes z from y
// and r, so that its sums see the unrounded values too:
//   a  = gh w_pre,  dz = gz + rstd_z (a - zhat mean(zhat a)),  zhat = z rstd_z
//   gr = dz,        u  = s g dz,   ggate = s dz n
//   b  = u w_post,  gy = rstd_y (b - yhat mean(yhat b)),       yhat = y rstd_y
//   gw_pre = sum_t gh zhat,  gw_post = sum_t u yhat  (and ggate summed over t for a
//   channel gate).
// The sums over tokens are made without atomics: each CTA of the backward adds its
// rows in order into its own partial vectors, and a second kernel adds the CTAs'
// partials in order.
#include <cuda_runtime.h>

#include <cstdint>

#include "elem.cuh"
#include "internal.h"

namespace nf4 {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float gate_at(const NormArgs& a, int64_t t, int64_t c) {
  if (a.gate_kind == NF4_GATE_CHANNEL) return static_cast<const float*>(a.gate)[c];
  if (a.gate_kind == NF4_GATE_TOKEN) return to_f32(static_cast<const T*>(a.gate)[t * a.ld_gate + c]);
  return 1.0f;
}

// n and z of one element, from the row's rstd_y.
template <typename T>
__device__ __forceinline__ float z_at(const NormArgs& a, int64_t t, int64_t c, float rstd_y, float* n_out) {
  const float y = to_f32(static_cast<const T*>(a.y)[t * a.ld_y + c]);
  const float n = a.w_post ? y * rstd_y * a.w_post[c] : y;
  *n_out = n;
  const float r = a.residual ? to_f32(static_cast<const T*>(a.residual)[t * a.ld_r + c]) : 0.0f;
  return r + a.scale * gate_at<T>(a, t, c) * n;
}

// Any width, stride and alignment: one CTA per row, one element per thread and step.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_fwd_any_kernel(NormArgs a) {
  __shared__ float red[64];
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    float rstd_y = 1.0f;
    if (a.w_post) {
      float s = 0.0f;
      for (int64_t c = threadIdx.x; c < a.H; c += kThreads) {
        const float y = to_f32(static_cast<const T*>(a.y)[t * a.ld_y + c]);
        s += y * y;
      }
      rstd_y = rsqrtf(block_sum(s, red) / static_cast<float>(a.H) + a.eps);
    }
    float s = 0.0f, n;
    for (int64_t c = threadIdx.x; c < a.H; c += kThreads) {
      const float z = z_at<T>(a, t, c, rstd_y, &n);
      s += z * z;
      if (a.z) static_cast<T*>(a.z)[t * a.ld_z + c] = from_f32<T>(z);
    }
    const float rstd_z = rsqrtf(block_sum(s, red + 32) / static_cast<float>(a.H) + a.eps);
    if (a.h)
      for (int64_t c = threadIdx.x; c < a.H; c += kThreads)
        static_cast<T*>(a.h)[t * a.ld_h + c] = from_f32<T>(z_at<T>(a, t, c, rstd_y, &n) * rstd_z * a.w_pre[c]);
    if (a.stats && threadIdx.x == 0) {
      a.stats[t] = rstd_y;
      a.stats[a.T + t] = rstd_z;
    }
    __syncthreads();
  }
}

// The backward for any width, stride and alignment.  part [CTAs][3][H].
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_bwd_any_kernel(NormArgs a) {
  __shared__ float red[64];
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 3 * a.H;
  bool first = true;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const float rstd_y = a.stats[t], rstd_z = a.stats[a.T + t];
    const float inv_h = 1.0f / static_cast<float>(a.H);
    float s = 0.0f, n;
    if (a.gh) {
      for (int64_t c = threadIdx.x; c < a.H; c += kThreads) {
        const float zhat = z_at<T>(a, t, c, rstd_y, &n) * rstd_z;
        s += zhat * to_f32(static_cast<const T*>(a.gh)[t * a.ld_gh + c]) * a.w_pre[c];
      }
    }
    const float mz = block_sum(s, red) * inv_h;
    s = 0.0f;
    for (int64_t c = threadIdx.x; c < a.H; c += kThreads) {
      const float zhat = z_at<T>(a, t, c, rstd_y, &n) * rstd_z;
      float dz = a.gz ? to_f32(static_cast<const T*>(a.gz)[t * a.ld_gz + c]) : 0.0f;
      float gwp = 0.0f;
      if (a.gh) {
        const float gh = to_f32(static_cast<const T*>(a.gh)[t * a.ld_gh + c]);
        dz += rstd_z * (gh * a.w_pre[c] - zhat * mz);
        gwp = gh * zhat;
      }
      const float g = gate_at<T>(a, t, c);
      const float u = a.scale * g * dz;
      const float yhat = a.w_post ? to_f32(static_cast<const T*>(a.y)[t * a.ld_y + c]) * rstd_y : 0.0f;
      if (a.w_post) s += yhat * u * a.w_post[c];
      if (a.gr) static_cast<T*>(a.gr)[t * a.ld_gr + c] = from_f32<T>(dz);
      const float gg = a.scale * dz * n;
      if (a.gate_kind == NF4_GATE_TOKEN && a.ggate)
        static_cast<T*>(a.ggate)[t * a.ld_ggate + c] = from_f32<T>(gg);
      if (a.part) {
        part[c] = first ? gwp : part[c] + gwp;
        part[a.H + c] = first ? u * yhat : part[a.H + c] + u * yhat;
        part[2 * a.H + c] = first ? gg : part[2 * a.H + c] + gg;
      }
    }
    const float my = block_sum(s, red + 32) * inv_h;
    if (a.gy)
      for (int64_t c = threadIdx.x; c < a.H; c += kThreads) {
        const float zhat = z_at<T>(a, t, c, rstd_y, &n) * rstd_z;
        float dz = a.gz ? to_f32(static_cast<const T*>(a.gz)[t * a.ld_gz + c]) : 0.0f;
        if (a.gh) dz += rstd_z * (to_f32(static_cast<const T*>(a.gh)[t * a.ld_gh + c]) * a.w_pre[c] - zhat * mz);
        float gy = a.scale * gate_at<T>(a, t, c) * dz;
        if (a.w_post) {
          const float yhat = to_f32(static_cast<const T*>(a.y)[t * a.ld_y + c]) * rstd_y;
          gy = rstd_y * (gy * a.w_post[c] - yhat * my);
        }
        static_cast<T*>(a.gy)[t * a.ld_gy + c] = from_f32<T>(gy);
      }
    first = false;
    __syncthreads();
  }
}

// out[v][c] = sum over p = 0 .. P-1 in order of part[p][v][c], v = gw_pre, gw_post, ggate.
__global__ void __launch_bounds__(kThreads) norm_partials_kernel(NormArgs a, int P) {
  float* outs[3] = {a.gw_pre, a.gw_post, a.gate_kind == NF4_GATE_CHANNEL ? static_cast<float*>(a.ggate) : nullptr};
  float* out = outs[blockIdx.y];
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (!out || c >= a.H) return;
  const float* p = a.part + blockIdx.y * a.H + c;
  float s = 0.0f;
  for (int i = 0; i < P; ++i) s += p[static_cast<int64_t>(i) * 3 * a.H];
  out[c] = s;
}

template <typename T>
cudaError_t launch_typed(bool backward, const NormArgs& a, int sms, cudaStream_t s) {
  if (!backward) {
    const int64_t grid = a.T < 8 * static_cast<int64_t>(sms) ? a.T : 8 * static_cast<int64_t>(sms);
    norm_fwd_any_kernel<T><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  const int P = norm_bwd_ctas(a.T, sms);
  norm_bwd_any_kernel<T><<<P, kThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.part) return e;
  norm_partials_kernel<<<dim3(static_cast<unsigned>((a.H + kThreads - 1) / kThreads), 3, 1), kThreads, 0, s>>>(a, P);
  return cudaGetLastError();
}

}  // namespace

int norm_bwd_ctas(int64_t T, int sms) {
  return static_cast<int>(T < 2 * static_cast<int64_t>(sms) ? T : 2 * static_cast<int64_t>(sms));
}

cudaError_t launch_norm(bool backward, int dtype, const NormArgs& a, int sms, cudaStream_t s) {
  if (dtype == NF4_DTYPE_F32) return launch_typed<float>(backward, a, sms, s);
  if (dtype == NF4_DTYPE_BF16) return launch_typed<__nv_bfloat16>(backward, a, sms, s);
  return launch_typed<__half>(backward, a, sms, s);
}

}  // namespace nf4
