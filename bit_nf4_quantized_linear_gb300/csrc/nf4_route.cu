// nf4_route.cu -- the router of the experts (nf4_route_fwd, nf4_route_bwd): which k experts
// each token goes to, with what weights, the tables that sort the (token, expert) pairs by
// expert for the grouped products, and the gradient of the logits.
//
// With s = softmax(x) or 1 / (1 + exp(-x)) of a token's logits x:
//   c = x (no bias; the order of s), or s + bias; c = -inf where x is (hidden experts);
//   a group's worth is its largest c, or the sum of its two largest s + bias;
//   the best groups are kept, and of their experts the k of largest c are chosen, equal ones
//   by the lower index;
//   w = scale s, or scale s / (sum of the chosen s).
// Two candidates whose fp32 values of c lie nearer than twice their error bound may stand in
// the wrong order, so such tokens are chosen again in fp64: the choice is that of the
// definition, whatever fp32 rounds.
//
// A warp holds a token's row in registers (expert i * 32 + lane) as order-preserving integer
// keys.  The k-th largest of the lanes' largest keys is a lower bound of the k-th largest of
// all (k redux instructions), which few others reach; those that do are packed one a lane, in
// index order, and the smallest are dropped until k are left.  The tables are a counting sort:
// each CTA counts its tokens' pairs, and a second kernel adds the counts of the CTAs before it
// and places its pairs by token, ranks among the CTA's tokens by bit masks: the same rows in
// every run.
//
// Measured (device time): one token over 64 experts 3.8 us; 512 tokens over 64, eight each, 6.5
// us and 2.8 for the gradient; 8192 over 256 in 8 groups, sigmoid with bias, 22.5 us (choice 15,
// tables 7.5) and 5.2, against 2.7 us of bytes: bound by the instructions of the choice, some
// 1500 a warp and token, 59% of the issue slots.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "early_launch.cuh"
#include "elem.cuh"
#include "internal.h"
#include "smem_limit.h"

namespace nf4 {
namespace {

constexpr int kRouteSingle = 32;  // tokens that one CTA routes and sorts alone
// Whether a CTA's counts fit bytes, and the sums of all CTAs' 16 bits.
__host__ __device__ __forceinline__ bool route_bytes(int per, int ctas) { return per <= 255 && per * ctas <= 65535; }
constexpr int kPlaceThreads = 512;
constexpr unsigned kAll = 0xffffffffu;

// Integers in the order of the values: -0 as 0, NaN above all, 0 below all.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  if (v != v) return 0xffffffffu;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  if (v != v) return ~uint64_t{0};
  return u >> 63 ? ~u : u | uint64_t{1} << 63;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

__device__ __forceinline__ uint32_t warp_key_max(uint32_t k) { return __reduce_max_sync(kAll, k); }
__device__ __forceinline__ uint64_t warp_key_max(uint64_t k) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t up = __shfl_xor_sync(kAll, k, o);
    k = up > k ? up : k;
  }
  return k;
}

__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// The `take` largest keys of a warp, equal ones by the lower index i * 32 + lane: bit i of the
// result is set where this lane's key i is among them.  *last: the smallest one taken.  Each
// round one lane gives its largest away and looks for its next.
template <int V, typename K>
__device__ __forceinline__ unsigned take_largest(K (&key)[V], int take, K* last) {
  const int lane = threadIdx.x & 31;
  unsigned chosen = 0;
  K top = 0, own = 0;
  int at = 0;
  auto find = [&]() {
    own = key[0];
    at = 0;
#pragma unroll
    for (int i = 1; i < V; ++i) {
      at = key[i] > own ? i : at;
      own = key[i] > own ? key[i] : own;
    }
  };
  find();
  for (int j = 0; j < take; ++j) {
    top = warp_key_max(own);
    const unsigned first = __reduce_min_sync(kAll, own == top ? at * 32 + lane : 0xffffffffu);
    if (first == static_cast<unsigned>(at * 32 + lane)) {
      chosen |= 1u << at;
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = i == at ? 0 : key[i];
      find();
    }
  }
  *last = top;
  return chosen;
}

// As take_largest where the candidates fit a warp: lane j < take gets the j-th chosen index,
// in ascending order.  False, with nothing done, where more than 32 keys reach the bound.
template <int V>
__device__ __forceinline__ bool pick_largest(const uint32_t (&key)[V], int take, uint16_t* list, int* index, uint32_t* last) {
  const int lane = threadIdx.x & 31;
  uint32_t own = key[0], bound = 0;
#pragma unroll
  for (int i = 1; i < V; ++i) own = max(own, key[i]);
  for (int j = 0; j < take; ++j) {
    bound = __reduce_max_sync(kAll, own);
    own = own == bound ? 0 : own;
  }
  bound = max(bound, 1u);
  int n = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) n += key[i] >= bound;
  if (__reduce_add_sync(kAll, n) > 32) return false;
  n = 0;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool in = key[i] >= bound;
    const unsigned all = __ballot_sync(kAll, in);
    if (in) list[n + __popc(all & ((1u << lane) - 1u))] = static_cast<uint16_t>(i);
    if (in) list[32 + n + __popc(all & ((1u << lane) - 1u))] = static_cast<uint16_t>(lane);
    n += __popc(all);
  }
  __syncwarp();
  const int i = lane < n ? list[lane] : 0, src = lane < n ? list[32 + lane] : 0;
  uint32_t k = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t v = __shfl_sync(kAll, key[j], src);
    k = i == j ? v : k;
  }
  bool in = lane < n;
  for (; n > take; --n) {  // the smallest, of equal ones the last
    const uint32_t low = __reduce_min_sync(kAll, in ? k : 0xffffffffu);
    const unsigned at = __ballot_sync(kAll, in && k == low);
    if (lane == 31 - __clz(at)) in = false;
  }
  *last = __reduce_min_sync(kAll, in ? k : 0xffffffffu);
  const unsigned all = __ballot_sync(kAll, in);
  __syncwarp();
  if (in) list[__popc(all & ((1u << lane) - 1u))] = static_cast<uint16_t>(i * 32 + src);
  __syncwarp();
  *index = lane < take ? list[lane] : -1;
  return true;
}

__device__ __forceinline__ int group_of(int e, float inv) { return static_cast<int>((e + 0.5f) * inv); }

// What group lane / lanes is worth, in its `lanes` lanes (a power of two; 32 / lanes groups or
// more): the largest, or the sum of the two largest, of its `size` values; -inf counts nothing
// beside another.  *least: the smallest that counts.  The groups start at different values
// (bank conflicts).
template <typename F>
__device__ __forceinline__ F group_worth(const F* v, int groups, int size, int top, int lanes, F* least) {
  const int lane = threadIdx.x & 31, g = lane / lanes, sub = lane & (lanes - 1), rounds = (size + lanes - 1) / lanes;
  F a = -INFINITY, b = -INFINITY;
  bool nan = false;
  if (g < groups) {
    int j = g % rounds;
    for (int i = 0; i < rounds; ++i) {
      const int at = j * lanes + sub;
      const F x = at < size ? v[g * size + at] : static_cast<F>(-INFINITY);
      nan |= x != x;
      b = x > a ? a : (x > b ? x : b);
      a = x > a ? x : a;
      j = j + 1 == rounds ? 0 : j + 1;
    }
  }
  for (int o = 1; o < lanes; o <<= 1) {
    const F c = __shfl_xor_sync(kAll, a, o), d = __shfl_xor_sync(kAll, b, o);
    nan |= static_cast<bool>(__shfl_xor_sync(kAll, static_cast<int>(nan), o));
    b = c > a ? (a > d ? a : d) : (c > b ? c : b);
    a = c > a ? c : a;
  }
  *least = top == 2 ? b : a;
  if (nan) return static_cast<F>(NAN);
  return top == 2 && b > -INFINITY ? a + b : a;
}

__device__ __forceinline__ int lanes_of(int groups) {  // a group
  int lanes = 32;
  while (lanes * groups > 32) lanes >>= 1;
  return lanes;
}

// One bit a group from the lanes' bits, of which each group's first counts.
__device__ __forceinline__ unsigned group_bits(bool bit, int lanes) {
  const unsigned all = __ballot_sync(kAll, bit);
  if (lanes == 1) return all;
  const int lane = threadIdx.x & 31;
  return __ballot_sync(kAll, lane * lanes < 32 && (all >> (lane * lanes & 31) & 1));
}

// fp64 values, in row[e], of the experts whose bit i (expert i * 32 + lane) is set: s + bias
// for sigmoid scores; for softmax without bias exp(x - top), in the order of s and of sums of s.
// Their indices are listed in `list`; returns how many they are.
template <typename T, int V>
__device__ __noinline__ int evaluate(const RouteArgs& a, int64_t t, unsigned mask, float top, double* row, uint16_t* list) {
  const int lane = threadIdx.x & 31;
  int n = 0;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const unsigned all = __ballot_sync(kAll, mask >> i & 1);
    if (mask >> i & 1) list[n + __popc(all & ((1u << lane) - 1u))] = static_cast<uint16_t>(i * 32 + lane);
    n += __popc(all);
  }
  __syncwarp();
  for (int i = lane; i < n; i += 32) {
    const int e = list[i];
    const double x = to_f32(static_cast<const T*>(a.logits)[t * a.ld + e]);
    row[e] = a.sigmoid ? 1.0 / (1.0 + exp(-x)) + (a.bias ? static_cast<double>(a.bias[e]) : 0.0) : exp(x - static_cast<double>(top));
  }
  __syncwarp();
  return n;
}

// The choice of token t in fp64.
template <typename T, int V>
__device__ __noinline__ unsigned choose_exactly(const RouteArgs& a, int64_t t, double* row) {
  const int lane = threadIdx.x & 31;
  const T* x = static_cast<const T*>(a.logits) + t * a.ld;
  const bool scores = a.bias || (a.groups > 1 && a.group_top == 2);
  double top = -INFINITY, sum = 0.0;
  if (scores && !a.sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 32 + lane;
      if (e < a.E) top = fmax(top, static_cast<double>(to_f32(x[e])));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(kAll, top, o));
  }
  uint64_t key[V];
  __syncwarp();
  for (int e = lane; e < a.E; e += 32) {
    const double xe = to_f32(x[e]);
    row[e] = !scores ? xe : a.sigmoid ? 1.0 / (1.0 + exp(-xe)) : exp(xe - top);
    sum += row[e];
  }
  if (scores) {
    sum = warp_sum64(sum);
    for (int e = lane; e < a.E; e += 32) {
      const double c = (a.sigmoid ? row[e] : row[e] / sum) + (a.bias ? static_cast<double>(a.bias[e]) : 0.0);
      row[e] = to_f32(x[e]) == -INFINITY ? -INFINITY : c;
    }
  }
  __syncwarp();
  unsigned kept = kAll;
  const int size = a.E / a.groups;
  if (a.groups > 1) {
    const int lanes = lanes_of(a.groups);
    double least;
    const double f = group_worth(row, a.groups, size, a.group_top, lanes, &least);
    uint64_t best[1] = {lane % lanes == 0 && lane / lanes < a.groups ? key_of(f) : 0}, last;
    kept = group_bits(take_largest(best, a.top_groups, &last), lanes);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 32 + lane;
    key[i] = 0;
    if (e < a.E && (kept >> (a.groups > 1 ? e / size : 0) & 1)) key[i] = key_of(a.bias ? row[e] : static_cast<double>(to_f32(x[e])));
  }
  __syncwarp();
  uint64_t last;
  return take_largest(key, a.k, &last);
}

// Whether all experts whose bit i (expert i * 32 + lane) is set, in any lane, have one logit and
// one bias: then what fp32 finds equal is, and goes by the index.
template <typename T, int V>
__device__ __noinline__ bool all_alike(const RouteArgs& a, int64_t t, unsigned mask) {
  const int lane = threadIdx.x & 31;
  uint32_t lo[2] = {0xffffffffu, 0xffffffffu}, hi[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (mask >> i & 1) {
      const int e = i * 32 + lane;
      const uint32_t k[2] = {key_of(to_f32(static_cast<const T*>(a.logits)[t * a.ld + e])), a.bias ? key_of(a.bias[e]) : 0u};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        lo[j] = min(lo[j], k[j]);
        hi[j] = max(hi[j], k[j]);
      }
    }
  return __reduce_min_sync(kAll, lo[0]) == __reduce_max_sync(kAll, hi[0]) && __reduce_min_sync(kAll, lo[1]) == __reduce_max_sync(kAll, hi[1]);
}

__device__ __forceinline__ float ex2_fast(float x) {  // relative error 2^-22
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {  // relative error 2^-23
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Routes token t: lane j < k gets its route's expert, in ascending order, and weight.
template <typename T, int V>
__device__ __forceinline__ int route_token(const RouteArgs& a, int64_t t, double* row, uint16_t* list, float* weight) {
  constexpr float kLog2e = 1.4426950408889634f, u = 5.9604645e-8f;  // u = 2^-24
  const int lane = threadIdx.x & 31;
  const T* xr = static_cast<const T*>(a.logits) + t * a.ld;
  float c[V];  // what the choice goes by
  uint32_t key[V], high = 0;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 32 + lane;
    c[i] = e < a.E ? to_f32(xr[e]) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    nan |= c[i] != c[i];
    key[i] = i * 32 + lane < a.E ? key_of(c[i]) : 0;
    high = max(high, key[i]);
  }
  const bool grouped = a.groups > 1, sums = grouped && a.group_top == 2, inexact = a.bias || sums;
  float top = 0.0f, norm = 0.0f;  // softmax: the largest logit, 1 / sum
  if (!a.sigmoid && (inexact || !a.renorm)) {
    top = value_of(warp_key_max(high));
    const float mm = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    if (a.renorm) {
#pragma unroll
      for (int i = 0; i < V; ++i) sum += ex2_fast((c[i] - mm) * kLog2e);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) sum += expf(c[i] - mm);
    }
    sum = warp_sum(sum);
    norm = top == -INFINITY ? 0.0f : 1.0f / sum;
  }
  unsigned chosen = 0;
  int e = -1;
  bool unsure = __any_sync(kAll, nan), picked = false;
  if (!unsure) {
    float cmax = 0.0f;
    if (inexact) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        const float s = a.sigmoid ? rcp_fast(1.0f + ex2_fast(-c[i] * kLog2e)) : ex2_fast((c[i] - top) * kLog2e) * norm;
        if (c[i] > -INFINITY) c[i] = s + (a.bias ? a.bias[e] : 0.0f);
        if (fabsf(c[i]) < INFINITY) cmax = fmaxf(cmax, fabsf(c[i]));  // an infinite bias is exact
        nan |= c[i] != c[i];
      }
      unsure = __any_sync(kAll, nan);
    }
    // Bounds on the error of c, in units of u = 2^-24.  Sigmoid: an exponential of relative error
    // 4 + 1.5 |x| in 1 / (1 + e), so (4 + 1.5 |x|) s (1 - s) < 1.4, and 3 s of the sum and the
    // reciprocal: less than 4.5.  Softmax: an argument d = top - x is off by 2.3 d (difference,
    // constant, product), which beside exp(-d) / sum is less than 1.  Relative to s: 4 of its own
    // exponential; of the sum 4 of its terms', 2.3 of their mean d (at most the root of w exp(w) =
    // (E - 1) / e: 3.9 for 512 experts), V - 1 + 5 additions; a reciprocal and a product: less than
    // V + 24, and s is at most 1 / sum.  And c's own rounding.
    const float off = a.sigmoid || !inexact ? 4.5f * u + u * __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(cmax)))
                                            : u * (1.0f + (V + 24.0f) * norm) + u * __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(cmax)));
    const int size = a.E / a.groups;
    const float inv = 1.0f / size;
    if (grouped && !unsure) {
      float* r32 = reinterpret_cast<float*>(row);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i * 32 + lane < a.E) r32[i * 32 + lane] = c[i];
      __syncwarp();
      const int lanes = lanes_of(a.groups);
      const bool mine = lane % lanes == 0 && lane / lanes < a.groups;
      float least;
      const float f = group_worth(r32, a.groups, size, a.group_top, lanes, &least);
      uint32_t best[1] = {mine ? key_of(f) : 0}, last;
      unsigned kept = group_bits(take_largest(best, a.top_groups, &last), lanes);
      if (inexact) {  // two values a group: twice the bound each way, and the roundings of the sum and of low - far
        const float low = value_of(last), far = 10.0f * off;
        const bool sure = mine && f > low + far;
        const unsigned near = group_bits(mine && !sure && !(f < low - far), lanes), safe = group_bits(sure, lanes);
        if (__popc(near) + __popc(safe) != a.top_groups) {
          // the values that can count in the groups near the border
          unsigned mask = 0;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int g = group_of(min(i * 32 + lane, a.E - 1), inv);
            const float from = __shfl_sync(kAll, least, g * lanes) - 4.0f * off;
            mask |= (i * 32 + lane < a.E && c[i] > -INFINITY && (near >> g & 1) && !(c[i] < from)) << i;
          }
          const bool alike = low > -INFINITY && all_alike<T, V>(a, t, mask) && !__any_sync(kAll, mine && (near >> (lane / lanes) & 1) && f != low);
          if (alike) {
            // equal sums of equal values: the choice by fp32 stands
          } else if (!a.sigmoid && a.bias) {
            unsure = true;
          } else {
            const int n = evaluate<T, V>(a, t, mask, top, row, list);
            double one = -INFINITY, two = -INFINITY;
            for (int j = 0; j < n; ++j) {
              const double v = row[list[j]];
              if (group_of(list[j], inv) != lane) continue;
              two = v > one ? one : (v > two ? v : two);
              one = v > one ? v : one;
            }
            const double worth = a.group_top == 2 && two > -INFINITY ? one + two : one;
            uint64_t wide[1] = {near >> lane & 1 ? key_of(worth) : 0}, border;
            kept = safe | __ballot_sync(kAll, take_largest(wide, a.top_groups - __popc(safe), &border));
          }
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (!(kept >> group_of(min(i * 32 + lane, a.E - 1), inv) & 1)) key[i] = 0;
    }
    if (!unsure) {
      if (a.bias) {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = key[i] ? key_of(c[i]) : 0;
      }
      uint32_t last;
      picked = pick_largest(key, a.k, list, &e, &last);
      if (a.bias) {
        uint32_t rest[V];
        if (!picked) {
#pragma unroll
          for (int i = 0; i < V; ++i) rest[i] = key[i];
          chosen = take_largest(rest, a.k, &last);
        }
        const float low = value_of(last), far = 3.0f * off;  // the bound each way, and the rounding of low - far
        const uint32_t reach = key_of(low - far);
        int n = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) n += key[i] >= reach;
        if (__reduce_add_sync(kAll, n) != a.k) {
          const bool was_picked = picked;
          picked = false;
          const uint32_t above = key_of(low + far);
          unsigned near = 0, safe = 0;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            safe |= (key[i] > above) << i;
            near |= (key[i] >= reach && key[i] <= above) << i;
          }
          const bool alike = low > -INFINITY && all_alike<T, V>(a, t, near);
          unsure = !alike && (!a.sigmoid || low == -INFINITY);
          if (alike) {
            picked = was_picked;
          } else if (!unsure) {
            evaluate<T, V>(a, t, near, top, row, list);
            uint64_t wide[V], border;
#pragma unroll
            for (int i = 0; i < V; ++i) wide[i] = near >> i & 1 ? key_of(row[i * 32 + lane]) : 0;
            chosen = safe | take_largest(wide, a.k - __reduce_add_sync(kAll, __popc(safe)), &border);
          }
        }
      } else if (!picked) {
        chosen = take_largest(key, a.k, &last);
      }
    }
  }
  if (unsure) chosen = choose_exactly<T, V>(a, t, row);
  if (unsure || !picked) {  // route j to lane j
    int n = 0;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const unsigned all = __ballot_sync(kAll, chosen >> i & 1);
      if (chosen >> i & 1) list[n + __popc(all & ((1u << lane) - 1u))] = static_cast<uint16_t>(i * 32 + lane);
      n += __popc(all);
    }
    __syncwarp();
    e = lane < a.k ? list[lane] : -1;
  }
  const float x = e >= 0 ? to_f32(xr[e]) : -INFINITY;
  if (!a.renorm) {
    const float s = a.sigmoid ? 1.0f / (1.0f + expf(-x)) : top == -INFINITY ? 0.0f : expf(x - top) * norm;
    *weight = a.scale * s;
    return e;
  }
  // s / sum of the chosen s, both times a power of e that keeps them from underflow: softmax
  // relative to the largest chosen logit m, sigmoid times exp(-m) where m < 0.
  const float m = warp_max(x), c0 = a.sigmoid ? fminf(m, 0.0f) : m;
  float p = 0.0f;
  if (e >= 0 && m > -INFINITY) {
    if (!a.sigmoid) p = expf(x - c0);
    else if (x > 0.0f) p = 1.0f / (1.0f + expf(-x));
    else p = expf(x - c0) / (1.0f + expf(x));
  }
  if (x != x) p = x;
  const float sum = warp_sum(p);
  *weight = m == -INFINITY && sum == 0.0f ? 0.0f : a.scale * (p / sum);  // 0: no expert of this row has a score
  return e;
}

// Places the (token, expert) pairs of a CTA's tokens, kPlaceTokens at a time.  fetch() reads
// their experts and weights, mark() sets the masks of which tokens chose an expert; finish()
// needs the first row of each expert in base[], which it moves on.  Called by the whole CTA; mask holds
// kPlaceWords x E values.
constexpr int kPlaceWords = 4, kPlaceTokens = 32 * kPlaceWords;

template <int THREADS>
struct Placer {
  static constexpr int kEach = kPlaceTokens * kRouteMaxK / THREADS;  // pairs of a thread at most
  int e[kEach];
  float w[kEach];

  __device__ __forceinline__ void fetch(const RouteArgs& a, int64_t tb, int64_t t1) {
    const int pairs = static_cast<int>((t1 - tb < kPlaceTokens ? t1 - tb : kPlaceTokens) * a.k);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int p = i * THREADS + threadIdx.x;
      e[i] = -1;
      if (p < pairs) {
        e[i] = a.experts[tb * a.k + p];
        w[i] = a.weights[tb * a.k + p];
      }
    }
  }

  __device__ __forceinline__ void mark(const RouteArgs& a, unsigned* mask) {
    for (int i = threadIdx.x; i < kPlaceWords * a.E; i += THREADS) mask[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int tl = (i * THREADS + threadIdx.x) / a.k;
      if (e[i] >= 0) atomicOr(mask + (tl >> 5) * a.E + e[i], 1u << (tl & 31));
    }
    __syncthreads();
  }

  __device__ __forceinline__ void finish(const RouteArgs& a, int64_t tb, int64_t t1, int* base, const unsigned* mask) {
    const int pairs = static_cast<int>((t1 - tb < kPlaceTokens ? t1 - tb : kPlaceTokens) * a.k);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int p = i * THREADS + threadIdx.x, tl = p / a.k;
      if (p >= pairs) break;
      int r = -1;
      if (e[i] >= 0) {
        r = base[e[i]] + __popc(mask[(tl >> 5) * a.E + e[i]] & ((1u << (tl & 31)) - 1u));
        for (int j = 0; j < tl >> 5; ++j) r += __popc(mask[j * a.E + e[i]]);
        a.row_token[r] = static_cast<int32_t>(tb + tl);
        a.row_weight[r] = w[i];
      }
      a.token_rows[tb * a.k + p] = r;
    }
    __syncthreads();
    for (int x = threadIdx.x; x < a.E; x += THREADS)
#pragma unroll
      for (int j = 0; j < kPlaceWords; ++j) base[x] += __popc(mask[j * a.E + x]);
    __syncthreads();
  }
};

// First row of each expert from the experts' counts (in `base`), which it replaces; returns
// the number of rows.  `red` holds 32 values.
template <int THREADS>
__device__ __forceinline__ int scan_counts(int E, int* base, int* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  static_assert(kMaxExperts <= THREADS, "an expert a thread");
  const int own = threadIdx.x < E ? base[threadIdx.x] : 0;
  int incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(kAll, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) red[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    before += w < warp ? red[w] : 0;
    total += red[w];
  }
  if (threadIdx.x < E) base[threadIdx.x] = before + incl - own;
  __syncthreads();
  return total;
}

__device__ __forceinline__ void write_rest(const RouteArgs& a, int64_t rows, int64_t me, int64_t of) {
  for (int64_t r = rows + me; r < a.T * a.k; r += of) {
    a.row_token[r] = -1;
    a.row_weight[r] = 0.0f;
  }
}

template <typename T, int V, int kWarps>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(RouteArgs a, int per) {
  constexpr int kThreads = kWarps * 32;
  extern __shared__ double s_rows[];  // [kWarps][E], then the lists [kWarps][max(E, 64)]
  uint16_t* s_list = reinterpret_cast<uint16_t*>(s_rows + kWarps * a.E);
  __shared__ int s_base[kMaxExperts], s_red[32];
  __shared__ unsigned s_mask[kPlaceWords * kMaxExperts];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_allow();
  for (int e = threadIdx.x; e < a.E; e += kThreads) s_base[e] = 0;
  __syncthreads();
  grid_wait();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * per, t1 = t0 + per < a.T ? t0 + per : a.T;
  for (int64_t t = t0 + warp; t < t1; t += kWarps) {
    if (a.live && !a.live[t]) {
      if (lane < a.k) {
        a.experts[t * a.k + lane] = -1;
        a.weights[t * a.k + lane] = 0.0f;
      }
      continue;
    }
    float w;
    const int e = route_token<T, V>(a, t, s_rows + warp * a.E, s_list + warp * max(a.E, 64), &w);
    if (lane < a.k) {
      a.experts[t * a.k + lane] = e;
      a.weights[t * a.k + lane] = w;
      if (a.offsets) atomicAdd(s_base + e, 1);
    }
  }
  if (!a.offsets) return;
  __syncthreads();
  if (gridDim.x > 1) {
    const int pitch = route_pitch(a.E);
    for (int e = threadIdx.x; e < pitch; e += kThreads) {
      const int64_t at = static_cast<int64_t>(blockIdx.x) * pitch + e;
      const int n = e < a.E ? s_base[e] : 0;
      if (route_bytes(per, gridDim.x)) reinterpret_cast<uint8_t*>(a.counts)[at] = static_cast<uint8_t>(n);
      else a.counts[at] = n;
    }
    return;
  }
  const int rows = scan_counts<kThreads>(a.E, s_base, s_red);
  for (int e = threadIdx.x; e < a.E; e += kThreads) a.offsets[e] = s_base[e];
  if (threadIdx.x == 0) a.offsets[a.E] = rows;
  Placer<kThreads> place;
  for (int64_t tb = t0; tb < t1; tb += kPlaceTokens) {
    place.fetch(a, tb, t1);
    place.mark(a, s_mask);
    place.finish(a, tb, t1, s_base, s_mask);
  }
  write_rest(a, rows, threadIdx.x, kThreads);
}

// The second pass: a CTA for each CTA of the first, with the same tokens.  Each adds the counts
// of all CTAs, and of those before it, 16 experts a thread.  BYTES: as route_bytes() says, so
// that two sums are added at once.
template <bool BYTES>
__global__ void __launch_bounds__(kPlaceThreads) route_place_kernel(RouteArgs a, int per) {
  __shared__ int s_all[kMaxExperts], s_below[kMaxExperts], s_red[32];
  __shared__ unsigned s_mask[kPlaceWords * kMaxExperts];
  for (int e = threadIdx.x; e < kMaxExperts; e += kPlaceThreads) s_all[e] = s_below[e] = 0;
  __syncthreads();
  grid_wait();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * per, t1 = t0 + per < a.T ? t0 + per : a.T;
  const int me = blockIdx.x, of = gridDim.x, e = threadIdx.x;
  Placer<kPlaceThreads> place;
  place.fetch(a, t0, t1);
  int total = 0, below = 0;  // of expert e
  if constexpr (BYTES) {
    const int runs = route_pitch(a.E) / 16, parts = kPlaceThreads / runs, part = threadIdx.x / runs, q = threadIdx.x - part * runs;
    unsigned all[8] = {}, low[8] = {};
    if (part < parts) {
#pragma unroll 8
      for (int c = part; c < of; c += parts) {
        const uint4 n = reinterpret_cast<const uint4*>(a.counts)[static_cast<int64_t>(c) * runs + q];
        const unsigned v[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const unsigned even = v[j] & 0x00ff00ffu, odd = v[j] >> 8 & 0x00ff00ffu;
          all[2 * j] += even;
          all[2 * j + 1] += odd;
          if (c < me) {
            low[2 * j] += even;
            low[2 * j + 1] += odd;
          }
        }
      }
    }
    place.mark(a, s_mask);
    if (part < parts)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        atomicAdd(reinterpret_cast<unsigned*>(s_all) + q * 8 + j, all[j]);
        atomicAdd(reinterpret_cast<unsigned*>(s_below) + q * 8 + j, low[j]);
      }
    __syncthreads();
    if (e < a.E) {
      const int at = e / 4 * 2 + (e & 1), shift = e & 2 ? 16 : 0;
      total = s_all[at] >> shift & 0xffff;
      below = s_below[at] >> shift & 0xffff;
    }
    __syncthreads();
  } else {
    place.mark(a, s_mask);
    if (e < a.E)
#pragma unroll 16
      for (int c = 0; c < of; ++c) {
        const int n = a.counts[static_cast<int64_t>(c) * route_pitch(a.E) + e];
        total += n;
        below += c < me ? n : 0;
      }
  }
  if (e < a.E) s_all[e] = total;
  __syncthreads();
  const int rows = scan_counts<kPlaceThreads>(a.E, s_all, s_red);
  if (e < a.E) {
    if (me == 0) a.offsets[e] = s_all[e];
    s_all[e] += below;
  }
  if (me == 0 && threadIdx.x == 0) a.offsets[a.E] = rows;
  __syncthreads();
  for (int64_t tb = t0; tb < t1; tb += kPlaceTokens) {
    if (tb > t0) {
      place.fetch(a, tb, t1);
      place.mark(a, s_mask);
    }
    place.finish(a, tb, t1, s_all, s_mask);
  }
  write_rest(a, rows, static_cast<int64_t>(me) * kPlaceThreads + threadIdx.x, static_cast<int64_t>(of) * kPlaceThreads);
}

// -------------------------------------------------------------------- backward --

// A warp a token; lane j holds route j.  With g_j the gradient of weight j, p the weights
// before the scale:
//   renormalised: scale p_j (g_j - sum g p), for sigmoid scores times 1 - s_j;
//   else: softmax scale s_e (g_e - sum g s) over all experts (g_e = 0 off the route), sigmoid
//   scale g_j s_j (1 - s_j).
constexpr int kRouteBwdWarps = 8;

template <typename T>
__global__ void __launch_bounds__(kRouteBwdWarps * 32) route_bwd_kernel(RouteArgs a) {
  extern __shared__ float s_row[];  // [kRouteBwdWarps][E]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = s_row + warp * a.E;
  grid_allow();
  grid_wait();
  const bool whole = !a.renorm && !a.sigmoid;  // every expert of the row has a gradient
  const bool vec = reinterpret_cast<uintptr_t>(a.g_logits) % 16 == 0 && a.ld_g * sizeof(T) % 16 == 0 && a.E * sizeof(T) % 16 == 0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteBwdWarps + warp; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * kRouteBwdWarps) {
    const T* xr = static_cast<const T*>(a.logits) + t * a.ld;
    T* gr = static_cast<T*>(a.g_logits) + t * a.ld_g;
    int e = -1;
    float g = 0.0f, x = -INFINITY;
    if (lane < a.k) {
      e = a.experts[t * a.k + lane];
      if (e >= a.E) {
        if (a.status) atomicCAS(a.status, 0, kStatusBadOffsets);
        e = -1;
      }
      if (e >= 0) {
        x = to_f32(xr[e]);
        if (a.g_weights) g = a.g_weights[t * a.k + lane];
        if (a.g_rows) {
          const int64_t r = a.token_rows[t * a.k + lane];
          if (r >= 0 && r < a.T * a.k) g += a.g_rows[r];
          else if (r >= 0 && a.status) atomicCAS(a.status, 0, kStatusBadOffsets);
        }
      }
    }
    const bool any = __any_sync(kAll, e >= 0);
    float top = -INFINITY, norm = 0.0f, base = 0.0f;
    if (whole && any) {
      float sum = 0.0f;
      for (int i = lane; i < a.E; i += 32) top = fmaxf(top, to_f32(xr[i]));
      top = warp_max(top);
      for (int i = lane; i < a.E; i += 32) sum += expf(to_f32(xr[i]) - top);
      sum = warp_sum(sum);
      norm = top == -INFINITY ? 0.0f : 1.0f / sum;
      const float s = e >= 0 && top > -INFINITY ? expf(x - top) * norm : 0.0f;
      base = warp_sum(g * s);
    } else if (any) {
      float p = 0.0f;
      const float up = 1.0f / (1.0f + expf(x)), s = 1.0f / (1.0f + expf(-x));  // 1 - s, s
      if (a.renorm) {
        const float m = warp_max(x), c0 = a.sigmoid ? fminf(m, 0.0f) : m;
        if (e >= 0 && m > -INFINITY) p = !a.sigmoid ? expf(x - c0) : x > 0.0f ? s : expf(x - c0) / (1.0f + expf(x));
        const float sum = warp_sum(p);
        p = m > -INFINITY ? p / sum : 0.0f;
        g = a.scale * p * (g - warp_sum(g * p));
        if (a.sigmoid) g *= up;
      } else {
        g = a.scale * g * s * up;
      }
      if (e < 0) g = 0.0f;
    }
    if (whole) {
      __syncwarp();
      for (int i = lane; i < a.E; i += 32) row[i] = 0.0f;
      __syncwarp();
      if (e >= 0) row[e] = g;
      __syncwarp();
      for (int i = lane; i < a.E; i += 32)
        gr[i] = from_f32<T>(any && norm != 0.0f ? a.scale * (expf(to_f32(xr[i]) - top) * norm) * (row[i] - base) : 0.0f);
    } else {  // zeros, and the k values on top
      if (vec) {
        constexpr int kEach = 16 / sizeof(T);
        for (int i = lane; i < a.E / kEach; i += 32) reinterpret_cast<uint4*>(gr)[i] = make_uint4(0u, 0u, 0u, 0u);
      } else {
        for (int i = lane; i < a.E; i += 32) gr[i] = from_f32<T>(0.0f);
      }
      __syncwarp();
      if (e >= 0) gr[e] = from_f32<T>(g);
    }
  }
}

template <typename T, int V, int kWarps>
cudaError_t launch_fwd(const RouteArgs& a, int ctas, int per, cudaStream_t s) {
  static SmemLimit limit;
  auto kern = route_kernel<T, V, kWarps>;
  const int each = a.E * 8 + (a.E < 64 ? 64 : a.E) * 2;  // of a warp
  if (cudaError_t e = limit.allow(kern, kWarps * V * 32 * 10)) return e;
  if (cudaError_t e = launch_early(kern, dim3(static_cast<unsigned>(ctas)), kWarps * 32, kWarps * each, s, a, per)) return e;
  if (!a.offsets || ctas == 1) return cudaSuccess;
  return launch_early(route_bytes(per, ctas) ? route_place_kernel<true> : route_place_kernel<false>, dim3(static_cast<unsigned>(ctas)),
                      kPlaceThreads, 0, s, a, per);
}

// 32 warps a CTA where each has more than 16 tokens and the registers suffice (8192 tokens over
// 256 experts: 29 -> 23 us), else 16 (512 tokens: 5.6 us against 6.6 with 32).
template <typename T, int V>
cudaError_t launch_warps(const RouteArgs& a, int sms, cudaStream_t s) {
  const int ctas = route_ctas(a.T, sms), per = static_cast<int>((a.T + ctas - 1) / ctas);
  if constexpr (V <= 8)
    if (ctas > 1 && per > 16) return launch_fwd<T, V, 32>(a, ctas, per, s);
  return launch_fwd<T, V, 16>(a, ctas, per, s);
}

template <typename T>
cudaError_t launch_typed(bool backward, const RouteArgs& a, int sms, cudaStream_t s) {
  if (backward) {
    const int64_t most = static_cast<int64_t>(sms) * 8, want = (a.T + kRouteBwdWarps - 1) / kRouteBwdWarps;
    return launch_early(route_bwd_kernel<T>, dim3(static_cast<unsigned>(want < most ? want : most)), kRouteBwdWarps * 32,
                        kRouteBwdWarps * a.E * 4, s, a);
  }
  if (a.E <= 64) return launch_warps<T, 2>(a, sms, s);
  if (a.E <= 128) return launch_warps<T, 4>(a, sms, s);
  if (a.E <= 256) return launch_warps<T, 8>(a, sms, s);
  return launch_warps<T, 16>(a, sms, s);
}

}  // namespace

// CTAs of the forward, a contiguous run of tokens each.
int route_ctas(int64_t T, int sms) {
  if (T <= kRouteSingle) return 1;
  const int64_t want = (T + 15) / 16;
  return static_cast<int>(want < sms ? want : sms);
}

cudaError_t launch_route(bool backward, int dtype, const RouteArgs& a, int sms, cudaStream_t s) {
  if (dtype == NF4_DTYPE_F32) return launch_typed<float>(backward, a, sms, s);
  if (dtype == NF4_DTYPE_F16) return launch_typed<__half>(backward, a, sms, s);
  return launch_typed<__nv_bfloat16>(backward, a, sms, s);
}

}  // namespace nf4
