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
//
// A warp takes a block, a lane eight neighbours, all tensors of a launch in one grid (the
// table of tensors travels in the kernel's parameters).  fp32 states are bound by HBM (67 M
// bf16 values: 222 us, 6.6 TB/s of 6.8 measured by a copy).  8-bit states move 10 bytes a
// value instead of 22 but cost about 70 instructions, most of them for the codes: a warp's
// next block is copied to shared memory while it codes the present one, with one CTA of 32
// warps an SM, so that the look-up tables leave room for it (134 M bf16 values: 322 us, 4.2
// TB/s; 385 us with two CTAs of 16 warps and loads as they are needed; 425 us with 24 warps
// of more registers).  The read-out of 8-bit states is bound by HBM (224 us, 6.0 TB/s).
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "elem.cuh"
#include "internal.h"
#include "smem_limit.h"

namespace nf4 {
namespace {

constexpr int kThreads = 512;  // of the read-out
// 8-bit states: one CTA an SM, so that its look-up tables are there once and leave room for
// the next blocks' data.
constexpr int threads(int bits) { return bits == 8 ? 1024 : 512; }
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
// takes eight dependent loads; instead the sign, exponent and seven bits of r select a
// bucket that holds one midpoint at most, as the dynamic maps do everywhere from 2^-23
// up, and one comparison of the low halves picks one of two codes.  Levels that do not
// fit the scheme are searched.
constexpr int kBucket0 = 104 << 7;                        // of 2^-23
constexpr int kBuckets = (127 << 7) - kBucket0 + 1;       // up to that of 1.0
constexpr uint32_t kNoMid = 0xffff0000u;

// Levels are held 32 times over, one copy a bank, so that the lanes' look-ups do not
// collide; bucket entries once (neighbouring values mostly share a few buckets).
//   entry: low half of the bucket's threshold on |r| (bits 16-31; 0xffff: nothing is above
//   it), code above it (8-15), code at or below it (0-7); r >= 0, then r < 0
template <bool SIGNED>
struct Map {
  float level[256 * 32];
  float once[256];
  float mid[255];
  int searched;
  uint32_t entry[(SIGNED ? 2 : 1) * kBuckets];
};
struct Maps {
  Map<true> m;
  Map<false> v;
};

template <bool SIGNED>
__device__ __forceinline__ int search(const Map<SIGNED>& mp, float r) {
  int lo = 0, hi = 255;
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (mp.mid[m] < r) lo = m + 1; else hi = m;
  }
  return lo;
}

__device__ __forceinline__ int bucket_of(float x) { return static_cast<int>((__float_as_uint(x) >> 16) & 0x7fffu) - kBucket0; }

// Buckets of a map by `warps` warps, this one being number `warp` of them.
template <bool SIGNED>
__device__ __forceinline__ void build_buckets(Map<SIGNED>& mp, int warp, int warps) {
  const int lane = threadIdx.x & 31;
  int zero = 0;  // midpoints below zero: 0 .. zero - 1
  for (int i = lane; i < 255; i += 32) zero += mp.mid[i] < 0.0f;
  zero = __reduce_add_sync(0xffffffffu, zero);
  if (!SIGNED && zero > 0) mp.searched = 1;
  // midpoint i of the positive ones fills the buckets after its predecessor's, up to its
  // own; the last stretch, past the last midpoint, is item 255
  for (int i = zero + warp; i <= 255; i += warps) {
    const int from = i == zero ? 0 : bucket_of(mp.mid[i - 1]) + 1;
    const int own = i == 255 ? kBuckets : bucket_of(mp.mid[i]);
    if (i < 255 && (own <= 0 || own >= kBuckets || own < from)) mp.searched = 1;
    for (int b = max(from, 0) + lane; b < min(own, kBuckets); b += 32) mp.entry[b] = kNoMid | i * 0x101u;
    if (lane == 0 && i < 255 && own >= 0 && own < kBuckets)
      mp.entry[own] = __float_as_uint(mp.mid[i]) << 16 | (i + 1) << 8 | i;
  }
  if (SIGNED) {
    // the negative ones by |mid|, i falling: code i + 1 below |mid[i]|, i from it on; the
    // comparison is |r| >= |mid|, so the threshold is the fp32 before it (where that lies
    // in the bucket before, every value here is above it)
    uint32_t* e = mp.entry + kBuckets;
    for (int i = zero - 1 - warp; i >= -1; i -= warps) {
      const int from = i == zero - 1 ? 0 : bucket_of(mp.mid[i + 1]) + 1;
      const int own = i < 0 ? kBuckets : bucket_of(mp.mid[i]);
      if (i >= 0 && (own <= 0 || own >= kBuckets || own < from)) mp.searched = 1;
      for (int b = max(from, 0) + lane; b < min(own, kBuckets); b += 32) e[b] = kNoMid | (i + 1) * 0x101u;
      if (lane == 0 && i >= 0 && own >= 0 && own < kBuckets) {
        const uint32_t low = __float_as_uint(mp.mid[i]) & 0xffffu;
        e[own] = low == 0u ? kNoMid | i * 0x101u : (low - 1u) << 16 | i << 8 | (i + 1);
      }
    }
    if (zero == 0)
      for (int b = warp * 32 + lane; b < kBuckets; b += warps * 32) e[b] = kNoMid;
  }
}

// Levels, midpoints and buckets of both maps, by the whole CTA, each by a half of it.
__device__ __forceinline__ void build_maps(Maps& maps, const float* levels_m, const float* levels_v) {
  constexpr int kHalf = threads(8) / 2, kWarps = kHalf / 32;
  const int lane = threadIdx.x & 31, half = threadIdx.x / kHalf, at = threadIdx.x % kHalf, warp = at / 32;
  float* once = half ? maps.v.once : maps.m.once;
  float* copies = half ? maps.v.level : maps.m.level;
  if (at < 256) once[at] = (half ? levels_v : levels_m)[at];
  if (at == 0) (half ? maps.v.searched : maps.m.searched) = 0;
  __syncthreads();
  for (int i = warp; i < 256; i += kWarps) copies[i * 32 + lane] = once[i];
  // half the sum rounded down: the halving is exact
  if (at < 255) (half ? maps.v.mid : maps.m.mid)[at] = 0.5f * __fadd_rd(once[at], once[at + 1]);
  __syncthreads();
  if (half) build_buckets(maps.v, warp, kWarps); else build_buckets(maps.m, warp, kWarps);
  __syncthreads();
}

// The code in bits 0-7; the bits above are not cleared.  |r| <= 1.
template <bool SIGNED>
__device__ __forceinline__ uint32_t code_of(const Map<SIGNED>& mp, float r) {
  // values below the first bucket have no midpoint between zero and them: they read it
  const uint32_t mag = __float_as_uint(fmaxf(SIGNED ? fabsf(r) : r, 1.1920928955078125e-7f));
  const uint32_t at = (mag >> 14) & ~3u;  // four bytes an entry
  const char* base = reinterpret_cast<const char*>(mp.entry) - static_cast<ptrdiff_t>(kBucket0) * 4;
  if (SIGNED) base += (__float_as_uint(r) >> 31) * (kBuckets * 4);
  const uint32_t e = *reinterpret_cast<const uint32_t*>(base + at);
  // equal low halves give mag << 16 <= e: not above
  return mag << 16 > e ? e >> 8 : e;
}

// Exact quotients x / top of |x| <= top by multiplication: with y the correctly rounded
// reciprocal and q within an ulp of the quotient, q + (x - q top) y rounded once is the
// correctly rounded quotient (Markstein 1990).  q comes from the reciprocal in two words,
// y + rest.  The residual x - q top is exact while top is neither tiny nor huge; outside
// [2^-75, 2^100] the values are divided.
struct Quotient {
  float2 top, y, rest;
  bool plain;
  __device__ __forceinline__ explicit Quotient(float t) {
    plain = !(t >= 2.6469779601696886e-23f && t <= 1.2676506002282294e30f);
    const float d = plain ? 1.0f : t, r = __frcp_rn(d), w = __fmaf_rn(-d, r, 1.0f) * r;
    top = make_float2(-d, -d);
    y = make_float2(r, r);
    rest = make_float2(w, w);
  }
  __device__ __forceinline__ float2 of(float2 x) const {
    const float2 q = fma2(x, y, mul2(x, rest));  // contracted or not
    return fma2(fma2(q, top, x), y, q);
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

// Eight neighbouring values of a lane: one access of 16 or 32 bytes, so that a lane always
// covers whole 32-byte sectors of fp32 data.
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[kPer]) {
  if constexpr (sizeof(T) == 2) {
    uint4 v;
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = from_f32<T>(x[k]);
    *reinterpret_cast<uint4*>(p) = v;
  } else {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
                 "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
  }
}

__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float sqrt_approx_ftz(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// New moments and parameters of two values; the square root and the quotient, which only
// the parameter sees, are the hardware's approximations (errors near 2^-23).  With an eps
// from 1e-12 up (EPS), subnormal second moments may count as zero (their root is below
// 1.1e-19) and the denominator is normal: two plain approximations do.
template <bool EPS>
__device__ __forceinline__ void update(const AdamArgs& a, float2 g, float2& m, float2& v, float2& p) {
  auto both = [](float x) { return make_float2(x, x); };
  // single operations: the packed ones may be contracted into one rounding
  m.x = __fadd_rn(__fmul_rn(m.x, a.beta1), __fmul_rn(g.x, a.one_minus_beta1));
  m.y = __fadd_rn(__fmul_rn(m.y, a.beta1), __fmul_rn(g.y, a.one_minus_beta1));
  v.x = __fadd_rn(__fmul_rn(v.x, a.beta2), __fmul_rn(__fmul_rn(g.x, g.x), a.one_minus_beta2));
  v.y = __fadd_rn(__fmul_rn(v.y, a.beta2), __fmul_rn(__fmul_rn(g.y, g.y), a.one_minus_beta2));
  float2 q;
  if (EPS) {
    const float2 den = fma2(make_float2(sqrt_approx_ftz(v.x), sqrt_approx_ftz(v.y)), both(a.inv_sqrt_c2), both(a.eps));
    q = mul2(m, make_float2(rcp_approx_ftz(den.x), rcp_approx_ftz(den.y)));
  } else {
    q.x = __fdividef(m.x, fmaf(sqrt_approx(v.x), a.inv_sqrt_c2, a.eps));
    q.y = __fdividef(m.y, fmaf(sqrt_approx(v.y), a.inv_sqrt_c2, a.eps));
  }
  // p - (lr wd p + step q): the rounding of the small bracket does not show in p
  const float2 d = fma2(both(a.decay), p, mul2(both(a.step_size), q));
  p = fma2(d, both(-1.0f), p);
}

// Codes of eight values of a block with the scale `top`.
template <bool SIGNED, bool WIDE>
__device__ __forceinline__ void store_codes(const Map<SIGNED>& mp, float (&x)[kPer], float top, uint8_t* to, int have) {
  const Quotient q(top);
  uint32_t w[2] = {0u, 0u};
  if (q.plain || mp.searched) {
    const float d = top > 0.0f ? top : 1.0f;
#pragma unroll 1
    for (int k = 0; k < kPer; ++k) {  // no indexing of registers: values and codes rotate
      const uint32_t c = search(mp, __fdiv_rn(x[0], d));
#pragma unroll
      for (int e = 0; e + 1 < kPer; ++e) x[e] = x[e + 1];
      w[0] = __funnelshift_r(w[0], w[1], 8);
      w[1] = w[1] >> 8 | c << 24;
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 a = q.of(make_float2(x[4 * h], x[4 * h + 1])), b = q.of(make_float2(x[4 * h + 2], x[4 * h + 3]));
      const uint32_t lo = __byte_perm(code_of<SIGNED>(mp, a.x), code_of<SIGNED>(mp, a.y), 0x0040);
      const uint32_t hi = __byte_perm(code_of<SIGNED>(mp, b.x), code_of<SIGNED>(mp, b.y), 0x0040);
      w[h] = __byte_perm(lo, hi, 0x5410);
    }
  }
  if (WIDE) {
    *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (k < have) to[k] = static_cast<uint8_t>(w[k >> 2] >> (8 * (k & 3)));
  }
}

// The level of byte `k` of w, from this lane's copy.
template <bool SIGNED>
__device__ __forceinline__ float level(const Map<SIGNED>& mp, uint32_t w, int k) {
  const uint32_t at = (k == 0 ? w << 7 : w >> (8 * k - 7)) & (255u << 7);
  return *reinterpret_cast<const float*>(reinterpret_cast<const char*>(mp.level + (threadIdx.x & 31)) + at);
}

// Where a warp's block lies: its tensor and its number in it.
struct Place {
  const AdamTensor* t;
  int64_t blk;
};

// A warp's next block on its way through shared memory: a lane copies and later reads only
// its own eight values of each array, in pieces of 16 bytes (8 of the codes), so that its own
// wait suffices.
template <typename T>
struct Slot {
  uint4 g[sizeof(T) / 2][32], p[sizeof(T) / 2][32];
  uint2 m[32], v[32];
  template <int N>
  static __device__ __forceinline__ void copy(void* to, const void* from) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    if (N == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at), "l"(from) : "memory");
  }
  __device__ __forceinline__ void fetch(const Place& at, int lane) {
    const int64_t base = at.blk * kAdamBlock + lane * kPer;
    const T *gr = static_cast<const T*>(at.t->grad) + base, *pa = static_cast<const T*>(at.t->param) + base;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
      copy<16>(&g[i][lane], gr + 4 * i);
      copy<16>(&p[i][lane], pa + 4 * i);
    }
    copy<8>(&m[lane], static_cast<const uint8_t*>(at.t->m) + base);
    copy<8>(&v[lane], static_cast<const uint8_t*>(at.t->v) + base);
  }
};
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A lane's eight values of a block as they lie in memory.
template <typename T, int BITS>
struct Raw {
  uint32_t g[2 * sizeof(T)], p[2 * sizeof(T)];
  uint32_t m[BITS == 8 ? 2 : 8], v[BITS == 8 ? 2 : 8];
  float sm, sv;
  template <int N>
  static __device__ __forceinline__ void get(const void* from, uint32_t (&to)[N]) {
    if constexpr (N == 8) {
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(to[0]), "=r"(to[1]), "=r"(to[2]), "=r"(to[3]), "=r"(to[4]), "=r"(to[5]), "=r"(to[6]), "=r"(to[7])
                   : "l"(from)
                   : "memory");
    } else {
      const uint4 x = *static_cast<const uint4*>(from);
      to[0] = x.x; to[1] = x.y; to[2] = x.z; to[3] = x.w;
    }
  }
  __device__ __forceinline__ void load(const Place& at, int lane) {
    const int64_t base = at.blk * kAdamBlock + lane * kPer;
    get(static_cast<const T*>(at.t->grad) + base, g);
    get(static_cast<const T*>(at.t->param) + base, p);
    get(static_cast<const float*>(at.t->m) + base, m);
    get(static_cast<const float*>(at.t->v) + base, v);
  }
  __device__ __forceinline__ void take(const Slot<T>& s, int lane) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
      const uint4 a = s.g[i][lane], b = s.p[i][lane];
      g[4 * i] = a.x; g[4 * i + 1] = a.y; g[4 * i + 2] = a.z; g[4 * i + 3] = a.w;
      p[4 * i] = b.x; p[4 * i + 1] = b.y; p[4 * i + 2] = b.z; p[4 * i + 3] = b.w;
    }
    const uint2 a = s.m[lane], b = s.v[lane];
    m[0] = a.x; m[1] = a.y;
    v[0] = b.x; v[1] = b.y;
  }
  static __device__ __forceinline__ void widen(const uint32_t (&w)[2 * sizeof(T)], float (&x)[kPer]) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) x[k] = to_f32(reinterpret_cast<const T*>(w)[k]);
  }
};

// A block of 256 values by one warp, a lane owning eight neighbours: from `raw` (WIDE), or
// value by value.  `used()` runs once nothing of `raw` is needed any more.
template <typename T, int BITS, bool WIDE, typename F>
__device__ __forceinline__ void block_step(const AdamArgs& a, const Maps& maps, const Place& at, const Raw<T, BITS>& raw,
                                           int lane, float gs, F used) {
  const AdamTensor& t = *at.t;
  const int64_t blk = at.blk, base = blk * kAdamBlock + lane * kPer;
  T* p = static_cast<T*>(t.param) + base;
  const T* g = static_cast<const T*>(t.grad) + base;
  const int have = WIDE ? kPer : t.n - base >= kPer ? kPer : t.n > base ? static_cast<int>(t.n - base) : 0;
  uint8_t *mc = static_cast<uint8_t*>(t.m) + base, *vc = static_cast<uint8_t*>(t.v) + base;
  float *mf = static_cast<float*>(t.m) + base, *vf = static_cast<float*>(t.v) + base;
  float pv[kPer], gv[kPer], m[kPer], v[kPer];
  if (WIDE) {
    raw.widen(raw.g, gv);
    raw.widen(raw.p, pv);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (BITS == 8) {
        m[k] = __fmul_rn(level(maps.m, raw.m[k >> 2], k & 3), raw.sm);
        v[k] = __fmul_rn(level(maps.v, raw.v[k >> 2], k & 3), raw.sv);
      } else {
        m[k] = __uint_as_float(raw.m[k]);
        v[k] = __uint_as_float(raw.v[k]);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const bool in = k < have;
      gv[k] = in ? to_f32(g[k]) : 0.0f;
      pv[k] = in ? to_f32(p[k]) : 0.0f;
      if (BITS == 8) {
        m[k] = in ? __fmul_rn(level(maps.m, mc[k], 0), t.m_absmax[blk]) : 0.0f;
        v[k] = in ? __fmul_rn(level(maps.v, vc[k], 0), t.v_absmax[blk]) : 0.0f;
      } else {
        m[k] = in ? mf[k] : 0.0f;
        v[k] = in ? vf[k] : 0.0f;
      }
    }
  }
  if (a.grad_scale)
#pragma unroll
    for (int k = 0; k < kPer; ++k) gv[k] = __fmul_rn(gv[k], gs);
  auto all = [&](auto eps) {
#pragma unroll
    for (int k = 0; k < kPer; k += 2) {
      float2 m2 = make_float2(m[k], m[k + 1]), v2 = make_float2(v[k], v[k + 1]), p2 = make_float2(pv[k], pv[k + 1]);
      update<decltype(eps)::value>(a, make_float2(gv[k], gv[k + 1]), m2, v2, p2);
      m[k] = m2.x;
      m[k + 1] = m2.y;
      v[k] = v2.x;
      v[k + 1] = v2.y;
      pv[k] = p2.x;
      pv[k + 1] = p2.y;
    }
  };
  if (a.eps >= 1e-12f) all(std::true_type{}); else all(std::false_type{});
  if (WIDE) {
    store8(p, pv);
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (k < have) p[k] = from_f32<T>(pv[k]);
  }
  if (BITS == 32) {
    if (WIDE) {
      store8(mf, m);
      store8(vf, v);
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (k >= have) continue;
        mf[k] = m[k];
        vf[k] = v[k];
      }
    }
    return;
  }
  float top_m = 0.0f, top_v = 0.0f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (!WIDE && k >= have) continue;  // past the tensor: no part of the scale
    top_m = max_nan(top_m, fabsf(m[k]));
    top_v = max_nan(top_v, fabsf(v[k]));
  }
  top_m = warp_absmax_nan(top_m);
  top_v = warp_absmax_nan(top_v);
  used();
  if (lane == 0) {
    t.m_absmax[blk] = top_m;
    t.v_absmax[blk] = top_v;
  }
  store_codes<true, WIDE>(maps.m, m, top_m, mc, have);
  store_codes<false, WIDE>(maps.v, v, top_v, vc, have);
}

// Finds the places of rising blocks: the tensor is searched for where the last one ends.
struct Finder {
  int ti = 0;
  int64_t first = 0, last = 0;
  __device__ __forceinline__ Place at(const AdamTable& tab, int64_t b) {
    if (b >= last) {
      ti = find_tensor(tab, b);
      first = tab.blk0[ti];
      last = tab.blk0[ti + 1];
    }
    return Place{&tab.t[ti], b - first};
  }
};

// All of the block inside, every array fit for vectors.
__device__ __forceinline__ bool wide(const Place& at) { return at.t->vec && (at.blk + 1) * kAdamBlock <= at.t->n; }

template <typename T, int BITS>
constexpr int smem_bytes() { return BITS == 8 ? sizeof(Maps) + threads(8) / 32 * sizeof(Slot<T>) : 0; }

template <typename T, int BITS>
__global__ void __launch_bounds__(threads(BITS), BITS == 8 ? 1 : 2) adamw_kernel(const __grid_constant__ AdamTable tab,
                                                                                 const __grid_constant__ AdamArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kWarps = threads(BITS) / 32;
  Slot<T>& slot = reinterpret_cast<Slot<T>*>(smem)[BITS == 8 ? threadIdx.x / 32 : 0];
  Maps& maps = *reinterpret_cast<Maps*>(smem + (BITS == 8 ? kWarps * sizeof(Slot<T>) : 0));
  const int lane = threadIdx.x & 31;
  const int64_t blocks = tab.blk0[tab.count];
  // A CTA takes one stretch of blocks, its warps in turn: a stretch lies in few tensors.
  const int64_t per = (blocks + gridDim.x - 1) / gridDim.x, end = min(blocks, (blockIdx.x + 1) * per);
  int64_t b = blockIdx.x * per + threadIdx.x / 32;
  Finder find;
  Raw<T, BITS> raw;
  if constexpr (BITS == 32) {
    const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
    for (; b < end; b += kWarps) {
      const Place at = find.at(tab, b);
      if (wide(at)) {
        raw.load(at, lane);
        block_step<T, BITS, true>(a, maps, at, raw, lane, gs, [] {});
      } else {
        block_step<T, BITS, false>(a, maps, at, raw, lane, gs, [] {});
      }
    }
  } else {
    Place at{}, next{};
    bool full = false;
    float sm = 0.0f, sv = 0.0f;  // scales of the block on its way
    auto fetch = [&](int64_t i) {
      full = false;
      if (i >= end) return;
      next = find.at(tab, i);
      full = wide(next);
      if (!full) return;
      slot.fetch(next, lane);
      sm = next.t->m_absmax[next.blk];
      sv = next.t->v_absmax[next.blk];
    };
    fetch(b);
    build_maps(maps, a.levels_m, a.levels_v);
    const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
    for (; b < end; b += kWarps) {
      at = next;
      if (full) {
        wait_copies();
        raw.take(slot, lane);
        raw.sm = sm;
        raw.sv = sv;
        block_step<T, BITS, true>(a, maps, at, raw, lane, gs, [&] { fetch(b + kWarps); });
      } else {
        block_step<T, BITS, false>(a, maps, at, raw, lane, gs, [&] { fetch(b + kWarps); });
      }
    }
  }
}

// out[i] = levels[codes[i]] * absmax[i / 256] for both states, eight values a thread
// where the pointers allow (10 bytes a value, two in and eight out: bound by HBM).
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
  constexpr int kSmem = smem_bytes<T, BITS>(), kWarps = threads(BITS) / 32;
  if constexpr (kSmem > 0) {
    static SmemLimit limit;
    if (cudaError_t e = limit.allow(adamw_kernel<T, BITS>, kSmem)) return e;
  }
  const int64_t want = (tab.blk0[tab.count] + kWarps - 1) / kWarps, most = (BITS == 8 ? 1 : 2) * static_cast<int64_t>(sms);
  adamw_kernel<T, BITS><<<static_cast<unsigned>(want < most ? want : most), threads(BITS), kSmem, s>>>(tab, a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(int bits, AdamTable& tab, const AdamArgs& a, int sms, cudaStream_t s) {
  for (int i = 0; i < tab.count; ++i) {
    AdamTensor& t = tab.t[i];
    const size_t state = bits == 8 ? 8 : 32;
    t.vec = aligned(t.param, 8 * sizeof(T)) && aligned(t.grad, 8 * sizeof(T)) && aligned(t.m, state) && aligned(t.v, state);
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
  a.vec = aligned(a.m, 8) && aligned(a.v, 8) && aligned(a.out_m, 32) && aligned(a.out_v, 32);
  const int64_t want = (a.n + kThreads * 8 - 1) / (kThreads * 8), most = 4 * static_cast<int64_t>(sms);
  adamw_values_kernel<<<static_cast<unsigned>(want < most ? want : most), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace nf4
