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
// Three forms, by what the rows allow:
//  - rows streamed through shared memory (16-byte rows, more rows than CTAs): 8192 x 5120
//    bf16 with a gate per token 74 us forward (5.7 TB/s of 6.8 measured by a copy) and 134 us
//    backward with the token sums (5.0 TB/s); bound by HBM with the issue slots at 55 to 60%
//  - a row in a CTA's registers (any alignment; few rows): one token of 4096 in 4 us, mostly
//    the latency of one load and two sums; 1023 x 2047 fp16 10 us
//  - rows wider than a CTA's registers (8192 forward, 5120 backward): three passes over the
//    row, from cache where it fits
// The sums over tokens are made without atomics: each CTA of the backward adds its
// rows in order into its own partial vectors, and a second kernel adds the CTAs'
// partials in order.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "elem.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"
#include "smem_limit.h"

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

// Any width: one CTA per row, one element per thread and step, each pass over the row from
// memory.  For rows too wide for the registers of a CTA.
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

// The backward for any width.  part [CTAs][3][H].
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

// ------------------------------------------------------- a row in registers --
// Both directions are bound by HBM (about 12 fp32 operations a value forward, 40
// backward), so the kernels below read each value once: a CTA holds a whole row, eight
// values a thread, and every load of a row is in flight before its first sum.
//   VEC values are one load: 16 bytes where the width, pitches and pointers allow, else
//   single values, neighbours in neighbouring threads (thread i holds columns i, i + n, ...),
//   which costs more instructions but the same memory traffic.

constexpr int kHold = 8;                 // values of a row per thread
constexpr int kMaxThreadsFwd = 1024;     // rows up to 8192 wide
constexpr int kMaxThreadsBwd = 640;      // rows up to 5120 wide: 24 sums a thread in registers

template <typename T, int VEC>
struct Frag {
  static constexpr int kVecs = kHold / VEC;
  using Raw = typename std::conditional<VEC == 1, T, uint4>::type;
  Raw v[kVecs];

  // column of value i, for a CTA of n threads
  static __device__ __forceinline__ int64_t column(int i, int n) {
    return (static_cast<int64_t>(i / VEC) * n + threadIdx.x) * VEC + i % VEC;
  }
  __device__ __forceinline__ void load(const void* row, int64_t H, int n) {
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int64_t c = column(k * VEC, n);
      if (c < H)
        v[k] = *reinterpret_cast<const Raw*>(static_cast<const T*>(row) + c);
      else
        v[k] = Raw{};
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < kVecs; ++k) v[k] = Raw{};
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (VEC == 1)
      return to_f32(v[i]);
    else
      return to_f32(reinterpret_cast<const T*>(&v[i / VEC])[i % VEC]);
  }
  // values 2 i and 2 i + 1
  __device__ __forceinline__ float2 pair(int i) const {
    if constexpr (VEC > 1 && std::is_same<T, __nv_bfloat16>::value) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(&v[0])[i];
      return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else if constexpr (VEC > 1 && std::is_same<T, __half>::value) {
      return __half22float2(reinterpret_cast<const __half2*>(&v[0])[i]);
    } else {
      return make_float2(at(2 * i), at(2 * i + 1));
    }
  }
  __device__ __forceinline__ void set_pair(int i, float2 x) {
    if constexpr (VEC > 1 && std::is_same<T, __nv_bfloat16>::value) {
      reinterpret_cast<__nv_bfloat162*>(&v[0])[i] = __floats2bfloat162_rn(x.x, x.y);
    } else if constexpr (VEC > 1 && std::is_same<T, __half>::value) {
      reinterpret_cast<__half2*>(&v[0])[i] = __floats2half2_rn(x.x, x.y);
    } else {
      set(2 * i, x.x);
      set(2 * i + 1, x.y);
    }
  }
  __device__ __forceinline__ void set(int i, float x) {
    if constexpr (VEC == 1)
      v[i] = from_f32<T>(x);
    else
      reinterpret_cast<T*>(&v[i / VEC])[i % VEC] = from_f32<T>(x);
  }
  __device__ __forceinline__ void store(void* row, int64_t H, int n) const {
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int64_t c = column(k * VEC, n);
      if (c < H) *reinterpret_cast<Raw*>(static_cast<T*>(row) + c) = v[k];
    }
  }
};

// fp32 values (gains, channel gate) at the columns of Frag<T, VEC>.
template <typename T, int VEC>
__device__ __forceinline__ void load_gain(float (&g)[kHold], const float* p, int64_t H, int n, float none) {
#pragma unroll
  for (int k = 0; k < kHold / VEC; ++k) {
    const int64_t c = Frag<T, VEC>::column(k * VEC, n);
    if (!p || c >= H) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) g[k * VEC + e] = none;
    } else if constexpr (VEC == 1) {
      g[k] = p[c];
    } else {
#pragma unroll
      for (int e = 0; e < VEC; e += 4) {
        const float4 f = *reinterpret_cast<const float4*>(p + c + e);
        g[k * VEC + e] = f.x;
        g[k * VEC + e + 1] = f.y;
        g[k * VEC + e + 2] = f.z;
        g[k * VEC + e + 3] = f.w;
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ const void* row_of(const void* p, int64_t t, int64_t ld) {
  return static_cast<const T*>(p) + t * ld;
}
template <typename T>
__device__ __forceinline__ void* row_of(void* p, int64_t t, int64_t ld) {
  return static_cast<T*>(p) + t * ld;
}

// One CTA per row.
template <typename T, int VEC>
__global__ void __launch_bounds__(kMaxThreadsFwd) norm_fwd_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float red[64];
  const int n = blockDim.x;
  const int64_t t = blockIdx.x;
  using F = Frag<T, VEC>;
  F y, r, gt;
  float wp[kHold], wn[kHold], gc[kHold];
  y.load(row_of<T>(a.y, t, a.ld_y), a.H, n);
  if (a.residual) r.load(row_of<T>(a.residual, t, a.ld_r), a.H, n); else r.clear();
  if (a.gate_kind == NF4_GATE_TOKEN) gt.load(row_of<T>(a.gate, t, a.ld_gate), a.H, n);
  load_gain<T, VEC>(wp, a.w_post, a.H, n, 1.0f);
  load_gain<T, VEC>(gc, a.gate_kind == NF4_GATE_CHANNEL ? static_cast<const float*>(a.gate) : nullptr, a.H, n, 1.0f);
  load_gain<T, VEC>(wn, a.w_pre, a.H, n, 1.0f);
  const float inv_h = 1.0f / static_cast<float>(a.H);
  float rstd_y = 1.0f;
  if (a.w_post) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kHold; ++i) s = fmaf(y.at(i), y.at(i), s);
    rstd_y = rsqrtf(block_sum(s, red) * inv_h + a.eps);
  }
  float z[kHold], s = 0.0f;
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const float g = a.gate_kind == NF4_GATE_TOKEN ? gt.at(i) : gc[i];
    z[i] = r.at(i) + a.scale * g * (y.at(i) * rstd_y * wp[i]);
    s = fmaf(z[i], z[i], s);
  }
  if (a.z) {
    F o;
#pragma unroll
    for (int i = 0; i < kHold; ++i) o.set(i, z[i]);
    o.store(row_of<T>(a.z, t, a.ld_z), a.H, n);
  }
  float rstd_z = 1.0f;
  if (a.h || a.stats) rstd_z = rsqrtf(block_sum(s, red + 32) * inv_h + a.eps);
  if (a.h) {
    F o;
#pragma unroll
    for (int i = 0; i < kHold; ++i) o.set(i, z[i] * rstd_z * wn[i]);
    o.store(row_of<T>(a.h, t, a.ld_h), a.H, n);
  }
  if (a.stats && threadIdx.x == 0) {
    a.stats[t] = rstd_y;
    a.stats[a.T + t] = rstd_z;
  }
}

// The inputs of a row of the backward.
template <typename T, int VEC>
struct BwdRow {
  Frag<T, VEC> y, r, gz, gh, gt;
  float rstd_y, rstd_z;
  __device__ __forceinline__ void load(const NormArgs& a, int64_t t, int n) {
    y.load(row_of<T>(a.y, t, a.ld_y), a.H, n);
    if (a.residual) r.load(row_of<T>(a.residual, t, a.ld_r), a.H, n); else r.clear();
    if (a.gz) gz.load(row_of<T>(a.gz, t, a.ld_gz), a.H, n); else gz.clear();
    if (a.gh) gh.load(row_of<T>(a.gh, t, a.ld_gh), a.H, n); else gh.clear();
    if (a.gate_kind == NF4_GATE_TOKEN) gt.load(row_of<T>(a.gate, t, a.ld_gate), a.H, n); else gt.clear();
    rstd_y = a.stats[t];
    rstd_z = a.stats[a.T + t];
  }
};

// The sums over tokens of a CTA's rows, at the thread's columns.
struct Sums {
  float pre[kHold], post[kHold], gate[kHold];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kHold; ++i) pre[i] = post[i] = gate[i] = 0.0f;
  }
};

// One row of the backward.  gains(k, g) fetches w_post, the channel gate or w_pre (k = 0,
// 1, 2) at this thread's columns; it is asked twice, to leave the registers to the sums.
// `red` [64]: CTA barriers separate its reads from the next call's writes.
template <typename T, int VEC, typename Gains>
__device__ __forceinline__ void bwd_row(const NormArgs& a, const BwdRow<T, VEC>& x, int64_t t, int n, float inv_h,
                                        Gains gains, float* red, Sums& sum) {
  using F = Frag<T, VEC>;
  const bool token = a.gate_kind == NF4_GATE_TOKEN;
  {
    float g[kHold], wp[kHold], wn[kHold];
    gains(0, wp);
    gains(1, g);
    gains(2, wn);
    float zhat[kHold], s = 0.0f;
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      if (token) g[i] = x.gt.at(i);
      const float nn = x.y.at(i) * x.rstd_y * wp[i];
      zhat[i] = (x.r.at(i) + a.scale * g[i] * nn) * x.rstd_z;
      s = fmaf(zhat[i], x.gh.at(i) * wn[i], s);
    }
    const float mz = block_sum(s, red) * inv_h;
    gains(0, wp);
    gains(1, g);
    gains(2, wn);
    float b[kHold];
    F gr, gg;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      const float gh = x.gh.at(i);
      const float dz = x.gz.at(i) + x.rstd_z * (gh * wn[i] - zhat[i] * mz);
      const float yhat = x.y.at(i) * x.rstd_y;
      if (token) g[i] = x.gt.at(i);
      const float u = a.scale * g[i] * dz, gate_grad = a.scale * dz * (yhat * wp[i]);
      gr.set(i, dz);
      gg.set(i, gate_grad);
      sum.pre[i] = fmaf(gh, zhat[i], sum.pre[i]);
      sum.post[i] = fmaf(u, yhat, sum.post[i]);
      if (!token) sum.gate[i] += gate_grad;
      b[i] = u * wp[i];
      s = fmaf(yhat, b[i], s);
    }
    if (a.gr) gr.store(row_of<T>(a.gr, t, a.ld_gr), a.H, n);
    if (token && a.ggate) gg.store(row_of<T>(a.ggate, t, a.ld_ggate), a.H, n);
    // without w_post, n is y itself: no norm to go back through
    const float my = a.w_post ? block_sum(s, red + 32) * inv_h : 0.0f;
    if (!a.w_post) __syncthreads();
    if (a.gy) {
      F gy;
#pragma unroll
      for (int i = 0; i < kHold; ++i) gy.set(i, x.rstd_y * (b[i] - x.y.at(i) * x.rstd_y * my));
      gy.store(row_of<T>(a.gy, t, a.ld_gy), a.H, n);
    }
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_sums(const NormArgs& a, const Sums& sum, int n) {
  if (!a.part) return;
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 3 * a.H;
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const int64_t c = Frag<T, VEC>::column(i, n);
    if (c >= a.H) continue;
    part[c] = sum.pre[i];
    part[a.H + c] = sum.post[i];
    part[2 * a.H + c] = sum.gate[i];
  }
}

// CTAs walk the rows with the grid's stride; single-value loads.
template <typename T>
__global__ void __launch_bounds__(kMaxThreadsBwd) norm_bwd_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float red[64];
  const int n = blockDim.x;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  Sums sum;
  sum.clear();
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    BwdRow<T, 1> x;
    x.load(a, t, n);
    auto gains = [&](int k, float (&g)[kHold]) {
      const float* p = k == 0 ? a.w_post : k == 2 ? a.w_pre
                       : a.gate_kind == NF4_GATE_CHANNEL ? static_cast<const float*>(a.gate) : nullptr;
      load_gain<T, 1>(g, p, a.H, n, k == 2 ? 0.0f : 1.0f);
    };
    bwd_row<T, 1>(a, x, t, n, inv_h, gains, red, sum);
  }
  store_sums<T, 1>(a, sum, n);
}

// ------------------------------------------------------------ rows by bulk copy --
// Where rows are whole 16-byte pieces, one thread streams the CTA's rows into a ring in
// shared memory by bulk copies, several rows ahead of the arithmetic, so that the loads
// never wait for a row's two sums; the gains stay in shared memory for all rows.

constexpr int kMaxStages = 4;
struct Ring {
  uint64_t full[kMaxStages];
  volatile int gave_up;
  int64_t unissued;  // the first row that was not copied after that, or T
};

// Bounded: after a timeout (recorded) every later wait returns at once, no further copy is
// issued, and the kernel runs out on whatever the buffers hold.
static __device__ __noinline__ void ring_wait_slow(Ring& r, uint32_t bar, uint32_t parity, uint64_t limit_ns, int* status) {
  const uint64_t t0 = nf4ptx::globaltimer_ns();
  while (!nf4ptx::mbar_try_wait_sleep(bar, parity, 20000)) {
    if (r.gave_up) return;
    if (nf4ptx::globaltimer_ns() - t0 > limit_ns) {
      r.gave_up = 1;
      if (status) atomicCAS(status, 0, kStatusTimeout);
      return;
    }
  }
}

// Thread 0, once a wait ran out: the copies in flight land, or are given up too, before the
// CTA's shared memory can be another's.
static __device__ __noinline__ void ring_drain(Ring& r, int stages, uint64_t limit_ns) {
  const int64_t rows = (r.unissued - blockIdx.x + gridDim.x - 1) / gridDim.x;  // copied ones, in turn to the stages
  const uint64_t t0 = nf4ptx::globaltimer_ns();
  for (int64_t k = rows < stages ? 0 : rows - stages; k < rows; ++k)
    while (!nf4ptx::mbar_try_wait_sleep(nf4ptx::smem_addr(&r.full[k % stages]), (k / stages) & 1, 20000))
      if (nf4ptx::globaltimer_ns() - t0 > limit_ns) break;
}

constexpr int kPairs = kHold / 2;

// This thread's vectors of a row: their first columns, and whether they lie in the row.
template <int VEC>
struct Cols {
  static constexpr int kVecs = kHold / VEC;
  uint32_t col[kVecs];
  bool in[kVecs];
  __device__ __forceinline__ explicit Cols(const NormArgs& a, int n) {
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      col[k] = (k * n + threadIdx.x) * VEC;
      in[k] = col[k] < a.H;
    }
  }
};

// The shared memory of a ring CTA: gains [3][H] fp32 (w_post, scale times the channel
// gate, w_pre; 1, scale and 0 where there is none), then the stages.  A thread's eight
// gains lie four and four, half a row apart: neighbouring threads then read neighbouring
// 16-byte pieces, without bank conflicts.
template <typename T, int VEC, bool BWD>
struct RowRing {
  using F = Frag<T, VEC>;
  const NormArgs& a;
  Ring& ring;
  const Cols<VEC> cols;
  float* gains;
  uint8_t* stage0;
  uint32_t row_bytes, stage_bytes;
  int stages;

  __device__ __forceinline__ RowRing(const NormArgs& a_, Ring& r, uint8_t* smem, int stages_, int n)
      : a(a_), ring(r), cols(a_, n), gains(reinterpret_cast<float*>(smem)), stages(stages_) {
    row_bytes = static_cast<uint32_t>(a.H * sizeof(T));
    stage_bytes = row_bytes * (1 + (a.residual != nullptr) + (a.gate_kind == NF4_GATE_TOKEN) + (BWD && a.gz) + (BWD && a.gh));
    stage0 = smem + 3 * a.H * sizeof(float);
  }
  // Thread 0: the copies of row t into a stage, which waits for `missing` bytes more than they are.
  __device__ __forceinline__ void issue(int st, int64_t t, uint32_t missing) const {
    const uint32_t bar = nf4ptx::smem_addr(&ring.full[st]);
    nf4ptx::mbar_arrive_expect_tx(bar, stage_bytes + missing);
    uint32_t to = nf4ptx::smem_addr(stage0) + st * stage_bytes;
    auto copy = [&](const void* p, int64_t ld) {
      nf4ptx::bulk_load_g2s(to, row_of<T>(p, t, ld), row_bytes, bar);
      to += row_bytes;
    };
    copy(a.y, a.ld_y);
    if (a.residual) copy(a.residual, a.ld_r);
    if (a.gate_kind == NF4_GATE_TOKEN) copy(a.gate, a.ld_gate);
    if (BWD && a.gz) copy(a.gz, a.ld_gz);
    if (BWD && a.gh) copy(a.gh, a.ld_gh);
  }
  __device__ __forceinline__ void wait(int st, uint32_t parity, int* status) const {
    const uint32_t bar = nf4ptx::smem_addr(&ring.full[st]);
    if (!nf4ptx::mbar_test_wait(bar, parity)) ring_wait_slow(ring, bar, parity, limit_ns(), status);
  }
  __device__ __forceinline__ uint64_t limit_ns() const { return a.starve ? 100000000 : 2000000000; }
  // Thread 0: row t, where there is one, into a stage that has been read.  A barrier whose
  // wait ran out is not armed again.
  __device__ __forceinline__ void refill(int st, int64_t t) const {
    if (t >= a.T) return;
    if (!ring.gave_up)
      issue(st, t, 0);
    else if (t < ring.unissued)
      ring.unissued = t;
  }
  __device__ __forceinline__ void take(F& f, bool have, const uint8_t* row) const {
    f.clear();
    if (!have) return;
#pragma unroll
    for (int k = 0; k < F::kVecs; ++k)
      if (cols.in[k]) f.v[k] = *reinterpret_cast<const typename F::Raw*>(row + cols.col[k] * sizeof(T));
  }
  __device__ __forceinline__ void put(const F& f, void* row) const {
#pragma unroll
    for (int k = 0; k < F::kVecs; ++k)
      if (cols.in[k]) *reinterpret_cast<typename F::Raw*>(static_cast<T*>(row) + cols.col[k]) = f.v[k];
  }
  __device__ __forceinline__ uint32_t gain_at(uint32_t c) const {  // c a multiple of 4
    return VEC == 8 ? (c >> 3) * 4 + (c & 4 ? static_cast<uint32_t>(a.H) / 2 : 0u) : c;
  }
  __device__ __forceinline__ void gain(float2 (&g)[kPairs], int which) const {
    const float* p = gains + which * a.H;
#pragma unroll
    for (int k = 0; k < F::kVecs; ++k)
#pragma unroll
      for (int e = 0; e < VEC; e += 4) {
        float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (cols.in[k]) f = *reinterpret_cast<const float4*>(p + gain_at(cols.col[k] + e));
        g[(k * VEC + e) / 2] = make_float2(f.x, f.y);
        g[(k * VEC + e) / 2 + 1] = make_float2(f.z, f.w);
      }
  }
  // Barriers, the first copies and the gains; ends with a CTA barrier.
  __device__ __forceinline__ void start(int n) const {
    if (threadIdx.x == 0) {
      ring.gave_up = 0;
      ring.unissued = a.T;
      for (int i = 0; i < stages; ++i) nf4ptx::mbar_init(nf4ptx::smem_addr(&ring.full[i]), 1);
      nf4ptx::fence_mbar_init();
      for (int i = 0; i < stages; ++i) {
        const int64_t t = blockIdx.x + static_cast<int64_t>(i) * gridDim.x;
        if (t < a.T) issue(i, t, a.starve && t == 0 ? 16 : 0);
      }
    }
    const float* src[3] = {a.w_post, a.gate_kind == NF4_GATE_CHANNEL ? static_cast<const float*>(a.gate) : nullptr, a.w_pre};
    const float none[3] = {1.0f, a.scale, 0.0f};
#pragma unroll
    for (int k = 0; k < 3; ++k)
      for (int64_t c = threadIdx.x * 4; c < a.H; c += n * 4) {
        float4 f = make_float4(none[k], none[k], none[k], none[k]);
        if (src[k]) f = *reinterpret_cast<const float4*>(src[k] + c);
        if (k == 1 && src[k]) f = make_float4(f.x * a.scale, f.y * a.scale, f.z * a.scale, f.w * a.scale);
        *reinterpret_cast<float4*>(gains + k * a.H + gain_at(static_cast<uint32_t>(c))) = f;
      }
    __syncthreads();
  }
};

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The rows' sums overlap: while row t's second sum is formed, so is row t + 1's first, and
// one CTA barrier serves both.
template <typename T, int VEC>
__global__ void __launch_bounds__(kMaxThreadsFwd) norm_fwd_ring_kernel(const __grid_constant__ NormArgs a, int stages) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 red[2][32];
  __shared__ Ring ring;
  const int n = blockDim.x;
  const RowRing<T, VEC, false> rr(a, ring, smem, stages, n);
  rr.start(n);
  using F = Frag<T, VEC>;
  const bool token = a.gate_kind == NF4_GATE_TOKEN;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  int st = 0, buf = 0;
  uint32_t ph = 0;
  auto squares = [&](int stage) {  // of this thread's part of y
    float2 s = both(0.0f);
    if (a.w_post) {
      F y;
      rr.take(y, true, rr.stage0 + stage * rr.stage_bytes);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) s = fma2(y.pair(i), y.pair(i), s);
    }
    return s.x + s.y;
  };
  rr.wait(0, 0, a.status);
  float ss_y = block_sum2(make_float2(squares(0), 0.0f), red[1]).x;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const float rstd_y = a.w_post ? rsqrtf(ss_y * inv_h + a.eps) : 1.0f;
    const uint8_t* p = rr.stage0 + st * rr.stage_bytes;
    F y, r, gt, o;
    rr.take(y, true, p);
    rr.take(r, a.residual != nullptr, p + rr.row_bytes);
    rr.take(gt, token, p + (a.residual ? 2 : 1) * rr.row_bytes);
    float2 g[kPairs], z[kPairs], s = both(0.0f);
    rr.gain(z, 0);
    rr.gain(g, 1);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const float2 nn = mul2(mul2(y.pair(i), both(rstd_y)), z[i]);
      z[i] = fma2(token ? mul2(gt.pair(i), both(a.scale)) : g[i], nn, r.pair(i));
      s = fma2(z[i], z[i], s);
      o.set_pair(i, z[i]);
    }
    if (a.z) rr.put(o, row_of<T>(a.z, t, a.ld_z));
    const int st1 = st + 1 == stages ? 0 : st + 1;
    const uint32_t ph1 = st1 == 0 ? ph ^ 1u : ph;
    float s1 = 0.0f;
    if (t + gridDim.x < a.T) {
      rr.wait(st1, ph1, a.status);
      s1 = squares(st1);
    }
    const float2 sums = block_sum2(make_float2(s.x + s.y, s1), red[buf]);
    buf ^= 1;
    ss_y = sums.y;
    const float rstd_z = rsqrtf(sums.x * inv_h + a.eps);
    // every thread has read its part of row t
    if (threadIdx.x == 0) rr.refill(st, t + static_cast<int64_t>(stages) * gridDim.x);
    if (a.h) {
      rr.gain(g, 2);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) o.set_pair(i, mul2(mul2(z[i], both(rstd_z)), g[i]));
      rr.put(o, row_of<T>(a.h, t, a.ld_h));
    }
    if (a.stats && threadIdx.x == 0) {
      a.stats[t] = rstd_y;
      a.stats[a.T + t] = rstd_z;
    }
    st = st1;
    ph = ph1;
  }
  if (threadIdx.x == 0 && ring.gave_up) ring_drain(ring, stages, rr.limit_ns());
}

// As in the forward, row t's second sum and row t + 1's first share a barrier.  What a row
// needs after its first sum is read from shared memory again, which leaves the registers
// to the sums over tokens.
template <typename T, int VEC>
__global__ void __launch_bounds__(kMaxThreadsBwd) norm_bwd_ring_kernel(const __grid_constant__ NormArgs a, int stages) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 red[2][32];
  __shared__ Ring ring;
  const int n = blockDim.x;
  const RowRing<T, VEC, true> rr(a, ring, smem, stages, n);
  rr.start(n);
  using F = Frag<T, VEC>;
  const bool token = a.gate_kind == NF4_GATE_TOKEN;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  // places of the arrays in a stage
  const uint32_t at_r = rr.row_bytes, at_t = at_r + (a.residual ? rr.row_bytes : 0), at_z = at_t + (token ? rr.row_bytes : 0),
                 at_h = at_z + (a.gz ? rr.row_bytes : 0);
  // z of this thread's columns, with y, n = y rstd_y w_post and scale times the gate
  auto forward = [&](const uint8_t* row, float rstd_y, F& y, float2 (&nn)[kPairs], float2 (&sg)[kPairs], float2 (&z)[kPairs]) {
    F r, gt;
    rr.take(y, true, row);
    rr.take(r, a.residual != nullptr, row + at_r);
    rr.take(gt, token, row + at_t);
    rr.gain(nn, 0);
    rr.gain(sg, 1);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      nn[i] = mul2(nn[i], mul2(y.pair(i), both(rstd_y)));
      if (token) sg[i] = mul2(gt.pair(i), both(a.scale));
      z[i] = fma2(sg[i], nn[i], r.pair(i));
    }
  };
  auto first_sum = [&](int stage, float rstd_y) {  // of z gh w_pre
    float2 s = both(0.0f);
    if (a.gh) {
      const uint8_t* row = rr.stage0 + stage * rr.stage_bytes;
      F y, gh;
      float2 nn[kPairs], sg[kPairs], z[kPairs];
      forward(row, rstd_y, y, nn, sg, z);
      rr.take(gh, true, row + at_h);
      rr.gain(nn, 2);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) s = fma2(z[i], mul2(gh.pair(i), nn[i]), s);
    }
    return s.x + s.y;
  };
  float2 sum_pre[kPairs], sum_post[kPairs], sum_gate[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) sum_pre[i] = sum_post[i] = sum_gate[i] = both(0.0f);
  int st = 0, buf = 0;
  uint32_t ph = 0;
  float rstd_y = a.stats[blockIdx.x], rstd_z = a.stats[a.T + blockIdx.x];
  rr.wait(0, 0, a.status);
  float dot = block_sum2(make_float2(first_sum(0, rstd_y), 0.0f), red[1]).x;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const bool more = t + gridDim.x < a.T;
    const float rstd_y1 = more ? a.stats[t + gridDim.x] : 0.0f, rstd_z1 = more ? a.stats[a.T + t + gridDim.x] : 0.0f;
    // dz = gz + rstd_z gh w_pre - z rstd_z^3 mean(z gh w_pre), without forming the power alone:
    // with a small eps it leaves fp32 long before the product does
    const float pull = rstd_z * dot * inv_h * rstd_z * rstd_z;
    F y;
    float2 b[kPairs], s = both(0.0f);
    {
      const uint8_t* row = rr.stage0 + st * rr.stage_bytes;
      F gz, gh, gr, gg;
      float2 nn[kPairs], z[kPairs], w[kPairs];
      forward(row, rstd_y, y, nn, b, z);
      rr.take(gz, a.gz != nullptr, row + at_z);
      rr.take(gh, a.gh != nullptr, row + at_h);
      rr.gain(w, 2);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float2 ghz = mul2(gh.pair(i), both(rstd_z));
        const float2 dz = fma2(both(-pull), z[i], fma2(ghz, w[i], gz.pair(i)));
        gr.set_pair(i, dz);
        if (token) gg.set_pair(i, mul2(mul2(dz, both(a.scale)), nn[i]));
        b[i] = mul2(b[i], dz);
        sum_pre[i] = fma2(ghz, z[i], sum_pre[i]);
        if (!token) sum_gate[i] = fma2(dz, nn[i], sum_gate[i]);
      }
      if (a.gr) rr.put(gr, row_of<T>(a.gr, t, a.ld_gr));
      if (token && a.ggate) rr.put(gg, row_of<T>(a.ggate, t, a.ld_ggate));
      rr.gain(w, 0);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float2 yhat = mul2(y.pair(i), both(rstd_y));
        sum_post[i] = fma2(b[i], yhat, sum_post[i]);
        b[i] = mul2(b[i], w[i]);
        s = fma2(yhat, b[i], s);
      }
    }
    const int st1 = st + 1 == stages ? 0 : st + 1;
    const uint32_t ph1 = st1 == 0 ? ph ^ 1u : ph;
    float s1 = 0.0f;
    if (more) {
      rr.wait(st1, ph1, a.status);
      s1 = first_sum(st1, rstd_y1);
    }
    const float2 sums = block_sum2(make_float2(s.x + s.y, s1), red[buf]);
    buf ^= 1;
    // every thread has read its part of row t
    if (threadIdx.x == 0) rr.refill(st, t + static_cast<int64_t>(stages) * gridDim.x);
    if (a.gy) {
      // without w_post, n is y itself: no norm to go back through
      const float back = a.w_post ? rstd_y * (sums.x * inv_h) : 0.0f;
      F gy;
#pragma unroll
      for (int i = 0; i < kPairs; ++i) gy.set_pair(i, mul2(both(rstd_y), fma2(both(-back), y.pair(i), b[i])));
      rr.put(gy, row_of<T>(a.gy, t, a.ld_gy));
    }
    dot = sums.y;
    rstd_y = rstd_y1;
    rstd_z = rstd_z1;
    st = st1;
    ph = ph1;
  }
  if (threadIdx.x == 0 && ring.gave_up) ring_drain(ring, stages, rr.limit_ns());
  Sums sum;
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    sum.pre[2 * i] = sum_pre[i].x;
    sum.pre[2 * i + 1] = sum_pre[i].y;
    sum.post[2 * i] = sum_post[i].x;
    sum.post[2 * i + 1] = sum_post[i].y;
    sum.gate[2 * i] = sum_gate[i].x * a.scale;
    sum.gate[2 * i + 1] = sum_gate[i].y * a.scale;
  }
  store_sums<T, VEC>(a, sum, n);
}

// out[v][c] = sum over p of part[p][v][c], v = gw_pre, gw_post, ggate.  A CTA takes 32
// columns; its eight warps each add every eighth partial in order, then the warps' sums
// are added in order.
__global__ void __launch_bounds__(kThreads) norm_partials_kernel(const __grid_constant__ NormArgs a, int P) {
  __shared__ float sums[kThreads / 32][32];
  float* outs[3] = {a.gw_pre, a.gw_post, a.gate_kind == NF4_GATE_CHANNEL ? static_cast<float*>(a.ggate) : nullptr};
  float* out = outs[blockIdx.y];
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const float* p = a.part + blockIdx.y * a.H + c;
  float s = 0.0f;
  if (c < a.H) {
#pragma unroll 8
    for (int i = warp; i < P; i += kThreads / 32) s += p[static_cast<int64_t>(i) * 3 * a.H];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < a.H) {
    for (int k = 1; k < kThreads / 32; ++k) s += sums[k][lane];
    out[c] = s;
  }
}

// Whether every row of the tensors in use can be read and written 16 bytes at a time.
bool vectors(const NormArgs& a, size_t elem) {
  const int64_t vec = static_cast<int64_t>(16 / elem);
  if (a.H % vec != 0) return false;
  const struct { const void* p; int64_t ld; } rows[] = {
      {a.y, a.ld_y}, {a.residual, a.ld_r}, {a.gz, a.ld_gz}, {a.gh, a.ld_gh}, {a.z, a.ld_z}, {a.h, a.ld_h},
      {a.gy, a.ld_gy}, {a.gr, a.ld_gr}, {a.gate_kind == NF4_GATE_TOKEN ? a.gate : nullptr, a.ld_gate},
      {a.gate_kind == NF4_GATE_TOKEN ? a.ggate : nullptr, a.ld_ggate}};
  for (const auto& r : rows)
    if (r.p && (reinterpret_cast<uintptr_t>(r.p) % 16 != 0 || r.ld % vec != 0)) return false;
  const void* gains[] = {a.w_post, a.w_pre, a.gate_kind == NF4_GATE_CHANNEL ? a.gate : nullptr};
  for (const void* g : gains)
    if (reinterpret_cast<uintptr_t>(g) % 16 != 0) return false;
  return true;
}

int threads_of(int64_t H) { return static_cast<int>((H + kHold * 32 - 1) / (kHold * 32)) * 32; }

// Ring CTAs on an SM: narrow rows want several, whose sums overlap.
int ring_ctas(int64_t H, bool backward) {
  const int n = threads_of(H), k = (backward ? kMaxThreadsBwd : kMaxThreadsFwd) / n;
  return k > 8 ? 8 : k;
}

// Shared memory of one: gains and as many stages as its share of the SM holds.
int ring_smem(const NormArgs& a, size_t elem, bool backward, int* stages) {
  const int arrays = 1 + (a.residual != nullptr) + (a.gate_kind == NF4_GATE_TOKEN) + (backward && a.gz) + (backward && a.gh);
  const int64_t gains = 12 * a.H, stage = static_cast<int64_t>(arrays) * a.H * static_cast<int64_t>(elem);
  const int64_t share = 220 * 1024 / ring_ctas(a.H, backward) - 2048;
  int64_t k = (share - gains) / stage;
  *stages = static_cast<int>(k > kMaxStages ? kMaxStages : k);
  return static_cast<int>(gains + *stages * stage);
}

// KERN's own, so that the limit is not set with every launch.
template <auto KERN>
cudaError_t ring_launch(unsigned grid, int n, int smem, const NormArgs& a, int stages, cudaStream_t s) {
  static SmemLimit limit;
  if (cudaError_t e = limit.allow(KERN, 220 * 1024)) return e;
  KERN<<<grid, n, smem, s>>>(a, stages);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(bool backward, const NormArgs& a, int sms, cudaStream_t s) {
  constexpr int kVec = 16 / sizeof(T);
  const bool vec = vectors(a, sizeof(T));
  const int n = threads_of(a.H);
  int stages = 0;
  if (!backward) {
    const int64_t most = static_cast<int64_t>(sms) * (a.H <= kMaxThreadsFwd * kHold ? ring_ctas(a.H, false) : 8);
    if (a.H > kMaxThreadsFwd * kHold) {
      norm_fwd_any_kernel<T><<<static_cast<unsigned>(a.T < most ? a.T : most), kThreads, 0, s>>>(a);
      return cudaGetLastError();
    }
    if (!vec) {
      norm_fwd_kernel<T, 1><<<static_cast<unsigned>(a.T), n, 0, s>>>(a);
      return cudaGetLastError();
    }
    // a row for each CTA at most, or rows too wide for two stages: no ring to fill
    const int smem = ring_smem(a, sizeof(T), false, &stages);
    if (a.T <= most || stages < 2) {
      norm_fwd_kernel<T, kVec><<<static_cast<unsigned>(a.T), n, 0, s>>>(a);
      return cudaGetLastError();
    }
    return ring_launch<norm_fwd_ring_kernel<T, kVec>>(static_cast<unsigned>(most), n, smem, a, stages, s);
  }
  const int P = norm_bwd_ctas(a.T, a.H, sms);
  cudaError_t e = cudaSuccess;
  if (a.H > kMaxThreadsBwd * kHold) {
    norm_bwd_any_kernel<T><<<P, kThreads, 0, s>>>(a);
    e = cudaGetLastError();
  } else {
    const int smem = vec ? ring_smem(a, sizeof(T), true, &stages) : 0;
    if (stages >= 2) {
      e = ring_launch<norm_bwd_ring_kernel<T, kVec>>(static_cast<unsigned>(P), n, smem, a, stages, s);
    } else {
      norm_bwd_kernel<T><<<P, n, 0, s>>>(a);
      e = cudaGetLastError();
    }
  }
  if (e != cudaSuccess || !a.part) return e;
  norm_partials_kernel<<<dim3(static_cast<unsigned>((a.H + 31) / 32), 3, 1), kThreads, 0, s>>>(a, P);
  return cudaGetLastError();
}

}  // namespace

// CTAs of the backward, each with partial sums of its own.
int norm_bwd_ctas(int64_t T, int64_t H, int sms) {
  const int64_t most = static_cast<int64_t>(H > kMaxThreadsBwd * kHold ? 2 : ring_ctas(H, true)) * sms;
  return static_cast<int>(T < most ? T : most);
}

cudaError_t launch_norm(bool backward, int dtype, const NormArgs& a, int sms, cudaStream_t s) {
  if (dtype == NF4_DTYPE_F32) return launch_typed<float>(backward, a, sms, s);
  if (dtype == NF4_DTYPE_BF16) return launch_typed<__nv_bfloat16>(backward, a, sms, s);
  return launch_typed<__half>(backward, a, sms, s);
}

}  // namespace nf4
