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

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = kAdamBlock / 32;  // values of a block per lane

// max that keeps a NaN of either side.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The warp's largest |v|, NaN if any lane's is.
__device__ __forceinline__ float warp_absmax_nan(float v) {
  float r;
  asm volatile("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// ---------------------------------------------------------- nearest level --
// The code of r is the count of midpoints below it.  Each midpoint is rounded down to
// fp32 first: r > mid is the same as r > floor32(mid) for an fp32 r.  A binary search
// takes eight dependent loads; instead the top 16 bits of |r| (sign apart, exponent and
// seven bits) select a bucket that holds one midpoint at most, as the dynamic maps do
// everywhere from 2^-23 up, and one comparison of the low 16 bits decides.  An entry is
//   bits 31..16  low half of the bucket's midpoint (0xffff: none, nothing is above it)
//   bits 15..0   code below the midpoint (r >= 0), or, in the second half of the table,
//                code of an |r| below it (r < 0, where the code falls as |r| grows)
// Levels that do not fit the scheme are searched.
constexpr int kBucket0 = 104 << 7;                        // of 2^-23
constexpr int kBuckets = (127 << 7) - kBucket0 + 1;       // up to that of 1.0

struct Map {
  float level[256];
  float mid[255];
  int searched;
  uint32_t entry[2 * kBuckets];
};

__device__ __forceinline__ int search(const Map& mp, float r) {
  int lo = 0, hi = 255;
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (mp.mid[m] < r) lo = m + 1; else hi = m;
  }
  return lo;
}

__device__ __forceinline__ int bucket_of(float x) { return static_cast<int>((__float_as_uint(x) >> 16) & 0x7fffu) - kBucket0; }

// Levels, midpoints and buckets of both maps, by the whole CTA.
__device__ void build_maps(Map* maps, const float* levels_m, const float* levels_v) {
  for (int i = threadIdx.x; i < 512; i += kThreads) {
    const float* L = i < 256 ? levels_m : levels_v;
    Map& mp = maps[i >> 8];
    const int k = i & 255;
    mp.level[k] = L[k];
    if (k < 255) mp.mid[k] = __double2float_rd((static_cast<double>(L[k]) + static_cast<double>(L[k + 1])) * 0.5);
    if (k == 255) mp.searched = 0;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int k = 0; k < 2; ++k) {
    Map& mp = maps[k];
    int zero = 0;  // midpoints below zero: 0 .. zero - 1
    for (int i = lane; i < 255; i += 32) zero += mp.mid[i] < 0.0f;
    zero = __reduce_add_sync(0xffffffffu, zero);
    // midpoint i of the positive ones fills the buckets after its predecessor's, up to its
    // own; the last stretch, past the last midpoint, is item 255
    for (int i = zero + warp; i <= 255; i += kWarps) {
      const int from = i == zero ? 0 : bucket_of(mp.mid[i - 1]) + 1;
      const int own = i == 255 ? kBuckets : bucket_of(mp.mid[i]);
      if (i < 255 && (own <= 0 || own >= kBuckets || own < from)) mp.searched = 1;
      for (int b = max(from, 0) + lane; b < min(own, kBuckets); b += 32) mp.entry[b] = 0xffff0000u | i;
      if (lane == 0 && i < 255 && own >= 0 && own < kBuckets)
        mp.entry[own] = (__float_as_uint(mp.mid[i]) << 16) | i;
    }
    // the negative ones by |mid|, i falling: code i + 1 below |mid[i]|, i from it on.  The
    // comparison is |r| >= |mid|, so the entry holds the low half of the fp32 before it.
    for (int i = zero - 1 - warp; i >= -1; i -= kWarps) {
      const int from = i == zero - 1 ? 0 : bucket_of(mp.mid[i + 1]) + 1;
      const int own = i < 0 ? kBuckets : bucket_of(mp.mid[i]);
      if (i >= 0 && (own <= 0 || own >= kBuckets || own < from)) mp.searched = 1;
      uint32_t* e = mp.entry + kBuckets;
      for (int b = max(from, 0) + lane; b < min(own, kBuckets); b += 32) e[b] = 0xffff0000u | (i + 1);
      if (lane == 0 && i >= 0 && own >= 0 && own < kBuckets) {
        const uint32_t low = __float_as_uint(mp.mid[i]) & 0xffffu;
        e[own] = low == 0u ? 0xffff0000u | i : ((low - 1) << 16) | (i + 1);
      }
    }
    // no negative midpoints: codes of r < 0 do not occur, entries stay readable
    if (zero == 0)
      for (int b = threadIdx.x; b < kBuckets; b += kThreads) mp.entry[kBuckets + b] = 0xffff0000u;
  }
  __syncthreads();
}

template <bool SIGNED>
__device__ __forceinline__ uint32_t code_of(const Map& mp, float r) {
  const uint32_t u = __float_as_uint(r);
  int b = static_cast<int>((u >> 16) & 0x7fffu) - kBucket0;
  b = min(max(b, 0), kBuckets - 1);
  const bool neg = SIGNED && (u >> 31);
  const uint32_t e = mp.entry[neg ? b + kBuckets : b];
  const uint32_t above = (u & 0xffffu) > (e >> 16) ? 1u : 0u;
  return (neg ? e - above : e + above) & 0xffu;
}

// Exact quotients x / top of |x| <= top by multiplication: with y the correctly rounded
// reciprocal and q within an ulp of the quotient, q + (x - q top) y rounded once is the
// correctly rounded quotient (Markstein 1990); a first step of the same form brings q
// that near.  Both sides are scaled by the power of two that makes top lie in [1, 2), so
// that the residual x - q top is exact.  Only for a normal top below 2^126.
struct Quotient {
  float scale, top, y;
  bool plain;  // outside that range: divide
  __device__ __forceinline__ explicit Quotient(float t) {
    const int e = static_cast<int>(__float_as_uint(t) >> 23);
    plain = e < 1 || e > 252;
    scale = __uint_as_float(static_cast<uint32_t>(254 - (plain ? 127 : e)) << 23);
    top = t * scale;
    y = __frcp_rn(top);
  }
  __device__ __forceinline__ float of(float x) const {
    x *= scale;
    float q = x * y;
    q = __fmaf_rn(__fmaf_rn(-q, top, x), y, q);
    return __fmaf_rn(__fmaf_rn(-q, top, x), y, q);
  }
};

// The tensor that holds global block b: first index with blk0[i + 1] > b.
__device__ __forceinline__ int find_tensor(const AdamTable& tab, int64_t b) {
  int lo = 0, hi = tab.count - 1;
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (tab.blk0[m + 1] > b) hi = m; else lo = m + 1;
  }
  return lo;
}

// Eight neighbouring values of a lane.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[kPer]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = to_f32(e[k]);
  } else {
    const float4 u = reinterpret_cast<const float4*>(p)[0], v = reinterpret_cast<const float4*>(p)[1];
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[kPer]) {
  if constexpr (sizeof(T) == 2) {
    uint4 v;
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = from_f32<T>(x[k]);
    *reinterpret_cast<uint4*>(p) = v;
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// New moments and parameter of one value; the square root and the quotient, which only
// the parameter sees, are the hardware's approximations (errors near 2^-23).
__device__ __forceinline__ void update(const AdamArgs& a, float g, float& m, float& v, float& p) {
  m = __fadd_rn(__fmul_rn(m, a.beta1), __fmul_rn(g, a.one_minus_beta1));
  v = __fadd_rn(__fmul_rn(v, a.beta2), __fmul_rn(__fmul_rn(g, g), a.one_minus_beta2));
  const float den = __fadd_rn(__fmul_rn(sqrt_approx(v), a.inv_sqrt_c2), a.eps);
  // p - (lr wd p + step q): the rounding of the small bracket does not show in p
  p = __fsub_rn(p, __fmaf_rn(a.decay, p, __fmul_rn(a.step_size, __fdividef(m, den))));
}

// One warp per block of 256 values; a lane owns eight neighbours.  Bound by HBM (10 bytes
// a value in and out for 16-bit parameters with 8-bit states) with the integer pipe close
// behind: the codes cost about 20 of its instructions a value.
template <typename T, int BITS>
__global__ void __launch_bounds__(kThreads, 2) adamw_kernel(const __grid_constant__ AdamTable tab,
                                                            const __grid_constant__ AdamArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  Map* maps = reinterpret_cast<Map*>(smem);
  if (BITS == 8) build_maps(maps, a.levels_m, a.levels_v);
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  const int lane = threadIdx.x & 31;
  const int64_t nw = static_cast<int64_t>(gridDim.x) * kWarps, blocks = tab.blk0[tab.count];
  int ti = -1;
  int64_t first = 0, last = 0;
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); b < blocks; b += nw) {
    if (b >= last) {
      ti = find_tensor(tab, b);
      first = tab.blk0[ti];
      last = tab.blk0[ti + 1];
    }
    const AdamTensor& t = tab.t[ti];
    const int64_t blk = b - first, base = blk * kAdamBlock + lane * kPer;
    T* p = static_cast<T*>(t.param) + base;
    const T* g = static_cast<const T*>(t.grad) + base;
    const int have = t.n - base >= kPer ? kPer : t.n > base ? static_cast<int>(t.n - base) : 0;
    // the same for a whole warp but in a tensor's last block
    const bool wide = t.vec && have == kPer;
    float pv[kPer], gv[kPer], m[kPer], v[kPer];
    uint8_t *mc = static_cast<uint8_t*>(t.m) + base, *vc = static_cast<uint8_t*>(t.v) + base;
    float *mf = static_cast<float*>(t.m) + base, *vf = static_cast<float*>(t.v) + base;
    uint8_t cm[kPer], cv[kPer];
    if (wide) {
      load8(g, gv);
      load8(p, pv);
      if (BITS == 8) {
        *reinterpret_cast<uint2*>(cm) = *reinterpret_cast<const uint2*>(mc);
        *reinterpret_cast<uint2*>(cv) = *reinterpret_cast<const uint2*>(vc);
      } else {
        load8(mf, m);
        load8(vf, v);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const bool in = k < have;
        gv[k] = in ? to_f32(g[k]) : 0.0f;
        pv[k] = in ? to_f32(p[k]) : 0.0f;
        if (BITS == 8) {
          cm[k] = in ? mc[k] : 0;
          cv[k] = in ? vc[k] : 0;
        } else {
          m[k] = in ? mf[k] : 0.0f;
          v[k] = in ? vf[k] : 0.0f;
        }
      }
    }
    if (BITS == 8) {
      const float sm = t.m_absmax[blk], sv = t.v_absmax[blk];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        m[k] = __fmul_rn(maps[0].level[cm[k]], sm);
        v[k] = __fmul_rn(maps[1].level[cv[k]], sv);
      }
    }
    if (a.grad_scale)
#pragma unroll
      for (int k = 0; k < kPer; ++k) gv[k] = __fmul_rn(gv[k], gs);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      update(a, gv[k], m[k], v[k], pv[k]);
      if (BITS == 8 && k >= have) m[k] = v[k] = 0.0f;  // past the tensor: no part of the scale
    }
    if (BITS == 8) {
      float top_m = fabsf(m[0]), top_v = fabsf(v[0]);
#pragma unroll
      for (int k = 1; k < kPer; ++k) {
        top_m = max_nan(top_m, fabsf(m[k]));
        top_v = max_nan(top_v, fabsf(v[k]));
      }
      top_m = warp_absmax_nan(top_m);
      top_v = warp_absmax_nan(top_v);
      const Quotient qm(top_m), qv(top_v);
      if (qm.plain || qv.plain || maps[0].searched || maps[1].searched) {
        const float dm = top_m > 0.0f ? top_m : 1.0f, dv = top_v > 0.0f ? top_v : 1.0f;
#pragma unroll 1
        for (int k = 0; k < kPer; ++k) {
          // no indexing of registers: rotate the values through the first place
          const uint32_t x = search(maps[0], __fdiv_rn(m[0], dm)), y = search(maps[1], __fdiv_rn(v[0], dv));
#pragma unroll
          for (int e = 0; e + 1 < kPer; ++e) {
            m[e] = m[e + 1];
            v[e] = v[e + 1];
            cm[e] = cm[e + 1];
            cv[e] = cv[e + 1];
          }
          cm[kPer - 1] = static_cast<uint8_t>(x);
          cv[kPer - 1] = static_cast<uint8_t>(y);
        }
      } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          cm[k] = static_cast<uint8_t>(code_of<true>(maps[0], qm.of(m[k])));
          cv[k] = static_cast<uint8_t>(code_of<false>(maps[1], qv.of(v[k])));
        }
      }
      if (lane == 0) {
        t.m_absmax[blk] = top_m;
        t.v_absmax[blk] = top_v;
      }
    }
    if (wide) {
      store8(p, pv);
      if (BITS == 8) {
        *reinterpret_cast<uint2*>(mc) = *reinterpret_cast<const uint2*>(cm);
        *reinterpret_cast<uint2*>(vc) = *reinterpret_cast<const uint2*>(cv);
      } else {
        store8(mf, m);
        store8(vf, v);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (k >= have) continue;
        p[k] = from_f32<T>(pv[k]);
        if (BITS == 8) {
          mc[k] = cm[k];
          vc[k] = cv[k];
        } else {
          mf[k] = m[k];
          vf[k] = v[k];
        }
      }
    }
  }
}

// out[i] = levels[codes[i]] * absmax[i / 256] for both states, eight values a thread
// where the pointers allow (18 bytes a value in and out: bound by HBM).
__global__ void __launch_bounds__(kThreads) adamw_values_kernel(const __grid_constant__ AdamValuesArgs a) {
  __shared__ float lev[2][256];
  for (int i = threadIdx.x; i < 512; i += kThreads) lev[i >> 8][i & 255] = (i < 256 ? a.levels_m : a.levels_v)[i & 255];
  __syncthreads();
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, nt = static_cast<int64_t>(gridDim.x) * kThreads;
  int64_t done = 0;
  if (a.vec) {
    done = a.n / 8 * 8;
    for (int64_t i = id * 8; i < done; i += nt * 8) {
      const uint2 m = *reinterpret_cast<const uint2*>(a.m + i), v = *reinterpret_cast<const uint2*>(a.v + i);
      const float sm = a.m_absmax[i / kAdamBlock], sv = a.v_absmax[i / kAdamBlock];
      const uint8_t *cm = reinterpret_cast<const uint8_t*>(&m), *cv = reinterpret_cast<const uint8_t*>(&v);
      float x[kPer], y[kPer];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[k] = __fmul_rn(lev[0][cm[k]], sm);
        y[k] = __fmul_rn(lev[1][cv[k]], sv);
      }
      store8(a.out_m + i, x);
      store8(a.out_v + i, y);
    }
  }
  for (int64_t i = done + id; i < a.n; i += nt) {
    a.out_m[i] = __fmul_rn(lev[0][a.m[i]], a.m_absmax[i / kAdamBlock]);
    a.out_v[i] = __fmul_rn(lev[1][a.v[i]], a.v_absmax[i / kAdamBlock]);
  }
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <typename T, int BITS>
cudaError_t launch_one(const AdamTable& tab, const AdamArgs& a, int sms, cudaStream_t s) {
  constexpr int kSmem = BITS == 8 ? 2 * static_cast<int>(sizeof(Map)) : 0;
  static bool configured = false;
  if (!configured && kSmem > 0) {
    if (cudaError_t e = cudaFuncSetAttribute(adamw_kernel<T, BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem))
      return e;
    configured = true;
  }
  const int64_t want = (tab.blk0[tab.count] + kWarps - 1) / kWarps, most = 2 * static_cast<int64_t>(sms);
  adamw_kernel<T, BITS><<<static_cast<unsigned>(want < most ? want : most), kThreads, kSmem, s>>>(tab, a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(int bits, AdamTable& tab, const AdamArgs& a, int sms, cudaStream_t s) {
  for (int i = 0; i < tab.count; ++i) {
    AdamTensor& t = tab.t[i];
    const size_t state = bits == 8 ? 8 : 16;
    t.vec = aligned(t.param, 16) && aligned(t.grad, 16) && aligned(t.m, state) && aligned(t.v, state);
  }
  return bits == 8 ? launch_one<T, 8>(tab, a, sms, s) : launch_one<T, 32>(tab, a, sms, s);
}

}  // namespace

cudaError_t launch_adamw(int dtype, int bits, AdamTable& tab, const AdamArgs& a, int sms, cudaStream_t s) {
  if (tab.count == 0 || tab.blk0[tab.count] == 0) return cudaSuccess;
  if (dtype == NF4_DTYPE_F32) return launch_typed<float>(bits, tab, a, sms, s);
  if (dtype == NF4_DTYPE_BF16) return launch_typed<__nv_bfloat16>(bits, tab, a, sms, s);
  return launch_typed<__half>(bits, tab, a, sms, s);
}

cudaError_t launch_adamw_values(AdamValuesArgs a, int sms, cudaStream_t s) {
  a.vec = aligned(a.m, 8) && aligned(a.v, 8) && aligned(a.out_m, 16) && aligned(a.out_v, 16);
  const int64_t want = (a.n + kThreads * 8 - 1) / (kThreads * 8), most = 4 * static_cast<int64_t>(sms);
  adamw_values_kernel<<<static_cast<unsigned>(want < most ? want : most), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace nf4
