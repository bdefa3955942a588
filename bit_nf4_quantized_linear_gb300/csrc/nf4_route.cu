// nf4_route.cu -- the router of the experts (nf4_route_fwd, nf4_route_bwd): which k experts
// each token goes to, with what weights, the tables that sort the (token, expert) pairs by
// expert for the grouped products, and the gradient of the logits.
//
// With s = softmax(x) or 1 / (1 + exp(-x)) of a token's logits x:
//   c = x (no bias; the order of s), or s + bias; experts of logit -inf come after all others;
//   a group's worth is its largest c, or the sum of its two largest s + bias;
//   the best groups are kept, and of their experts the k of largest c are chosen, equal ones
//   by the lower index;
//   w = scale s, or scale s / (sum of the chosen s).
// Two candidates whose fp32 values of c lie nearer than twice their error bound may stand in
// the wrong order, so such tokens are chosen again in fp64: the choice is that of the
// definition, whatever fp32 rounds.
//
// A warp holds a token's row in registers (expert i * 32 + lane); k rounds of a maximum over
// order-preserving integer keys (one redux instruction each) give the choice.  The tables are
// a counting sort: each CTA counts its tokens' pairs, and a second kernel adds the counts of
// the CTAs before it and places its pairs by token, ranks within 32 tokens by bit masks: the
// same rows in every run.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "elem.cuh"
#include "internal.h"
#include "smem_limit.h"

namespace nf4 {
namespace {

constexpr int kRouteWarps = 16;
constexpr int kRouteThreads = kRouteWarps * 32;
constexpr int kRouteSingle = 32;  // tokens that one CTA routes and sorts alone
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
// result is set where this lane's key i is among them.  *last: the smallest one taken.
template <int V, typename K>
__device__ __forceinline__ unsigned take_largest(K (&key)[V], int take, K* last) {
  const int lane = threadIdx.x & 31;
  unsigned chosen = 0;
  K top = 0;
  for (int j = 0; j < take; ++j) {
    K own = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) own = key[i] > own ? key[i] : own;
    top = warp_key_max(own);
    unsigned at = 0xffffffffu;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) at = key[i] == top ? i * 32 + lane : at;
    at = __reduce_min_sync(kAll, at);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * 32 + lane == at) {
        key[i] = 0;
        chosen |= 1u << i;
      }
  }
  *last = top;
  return chosen;
}

__device__ __forceinline__ int group_of(int e, float inv) { return static_cast<int>((e + 0.5f) * inv); }

// The largest, or the sum of the two largest, of a group's `size` values; -inf counts nothing
// beside another.  Lanes start at different values of their groups (bank conflicts).
template <typename F>
__device__ __forceinline__ F group_worth(const F* v, int size, int top, int lane, F* least) {
  F a = -INFINITY, b = -INFINITY;
  bool nan = false;
  int j = lane % size;
  for (int i = 0; i < size; ++i) {
    const F x = v[j];
    nan |= x != x;
    b = x > a ? a : (x > b ? x : b);
    a = x > a ? x : a;
    j = j + 1 == size ? 0 : j + 1;
  }
  *least = top == 2 ? b : a;  // the smallest that counts
  if (nan) return static_cast<F>(NAN);
  return top == 2 && b > -INFINITY ? a + b : a;
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
    double least;
    uint64_t best[1] = {lane < a.groups ? key_of(group_worth(row + lane * size, size, a.group_top, lane, &least)) : 0};
    uint64_t last;
    kept = __ballot_sync(kAll, take_largest(best, a.top_groups, &last));
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

// Routes token t: bit i of the result is set where this lane's expert i * 32 + lane is chosen,
// and w[i] is its weight.
template <typename T, int V>
__device__ __forceinline__ unsigned route_token(const RouteArgs& a, int64_t t, double* row, uint16_t* list, float (&w)[V]) {
  const int lane = threadIdx.x & 31;
  const T* xr = static_cast<const T*>(a.logits) + t * a.ld;
  float x[V], s[V];
  uint32_t key[V];
  bool nan = false;
  uint32_t high = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 32 + lane;
    x[i] = e < a.E ? to_f32(xr[e]) : -INFINITY;
    nan |= x[i] != x[i];
    key[i] = e < a.E ? key_of(x[i]) : 0;
    high = max(high, key[i]);
  }
  const bool any_nan = __any_sync(kAll, nan);
  const float top = value_of(warp_key_max(high));
  // Scores, where they are weights or decide the choice.
  const bool grouped = a.groups > 1, sums = grouped && a.group_top == 2;
  float norm = 1.0f;
  if (!a.renorm || a.bias || sums) {
    float sum = 0.0f;
    const float mm = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = a.sigmoid ? 1.0f / (1.0f + expf(-x[i])) : expf(x[i] - mm);
      sum += s[i];
    }
    if (!a.sigmoid) {
      sum = warp_sum(sum);
      norm = sum > 0.0f ? 1.0f / sum : sum != sum ? sum : 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] *= norm;
    }
  }
  unsigned chosen = 0;
  bool unsure = any_nan;
  if (!unsure) {
    const bool inexact = a.bias || sums;
    float c[V], cmax = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 32 + lane;
      c[i] = x[i];
      if (inexact && x[i] > -INFINITY) {
        c[i] = s[i] + (a.bias ? a.bias[e] : 0.0f);
        cmax = fmaxf(cmax, fabsf(c[i]));
        nan |= c[i] != c[i];
      }
    }
    unsure = __any_sync(kAll, nan);
    // Bounds on the error of c.  Sigmoid: with an exponential of two roundings' error, a sum and
    // a quotient, (4 s (1 - s) + 2 s) units of 2^-24, less than 4.  Softmax: the rounding of x - top (as d exp(-d) <= 0.4 units), and 24
    // units of s for exponential, row sum and quotient; s is at most 1 / sum.  And c's own
    // rounding.
    constexpr float u = 5.9604645e-8f;
    const float off = (a.sigmoid ? 4.0f * u : u * (1.0f + 24.0f * norm)) + u * __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(cmax)));
    const int size = a.E / a.groups;
    if (grouped && !unsure) {
      float* r32 = reinterpret_cast<float*>(row);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i * 32 + lane < a.E) r32[i * 32 + lane] = c[i];
      __syncwarp();
      float least = -INFINITY;
      const float f = lane < a.groups ? group_worth(r32 + lane * size, size, a.group_top, lane, &least) : -INFINITY;
      uint32_t best[1] = {lane < a.groups ? key_of(f) : 0}, last;
      unsigned kept = __ballot_sync(kAll, take_largest(best, a.top_groups, &last));
      if (inexact) {  // two values a group: twice the bound each way, and the roundings of the sum and of low - far
        const float low = value_of(last), far = 10.0f * off;
        const bool sure = lane < a.groups && f > low + far;
        const unsigned near = __ballot_sync(kAll, lane < a.groups && !sure && !(f < low - far)), safe = __ballot_sync(kAll, sure);
        if (__popc(near) + __popc(safe) != a.top_groups) {
          if (!a.sigmoid && a.bias) {
            unsure = true;
          } else {  // the values that can count in the groups near the border
            const float inv = 1.0f / size;
            unsigned mask = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const int g = group_of(min(i * 32 + lane, a.E - 1), inv);
              const float from = __shfl_sync(kAll, least, g) - 4.0f * off;
              mask |= (i * 32 + lane < a.E && x[i] > -INFINITY && (near >> g & 1) && !(c[i] < from)) << i;
            }
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
      const float inv = 1.0f / size;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (!(kept >> group_of(min(i * 32 + lane, a.E - 1), inv) & 1)) key[i] = 0;
    }
    if (!unsure) {
      if (a.bias) {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = key[i] ? key_of(c[i]) : 0;
      }
      unsigned open = 0;  // what may still be chosen
#pragma unroll
      for (int i = 0; i < V; ++i) open |= (key[i] != 0) << i;
      uint32_t last;
      chosen = take_largest(key, a.k, &last);
      if (a.bias) {
        const float low = value_of(last), far = 3.0f * off;  // the bound each way, and the rounding of low - far
        unsigned near = 0, safe = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const bool sure = c[i] > low + far;
          safe |= ((open >> i & 1) && sure) << i;
          near |= ((open >> i & 1) && !sure && !(c[i] < low - far)) << i;
        }
        const int fixed = __reduce_add_sync(kAll, __popc(safe));
        if (fixed + __reduce_add_sync(kAll, __popc(near)) != a.k) {
          // experts of logit -inf are equal to each other and below all else, as their keys are
          unsure = !a.sigmoid || low == -INFINITY;
          if (!unsure) {
            evaluate<T, V>(a, t, near, top, row, list);
            uint64_t wide[V], border;
#pragma unroll
            for (int i = 0; i < V; ++i) wide[i] = near >> i & 1 ? key_of(row[i * 32 + lane]) : 0;
            chosen = safe | take_largest(wide, a.k - fixed, &border);
          }
        }
      }
    }
  }
  if (unsure) chosen = choose_exactly<T, V>(a, t, row);
  if (!a.renorm) {
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = a.scale * s[i];
    return chosen;
  }
  // s / sum of the chosen s, both times a power of e that keeps them from underflow: softmax
  // relative to the largest chosen logit m, sigmoid times exp(-m) where m < 0.
  float m = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (chosen >> i & 1) m = fmaxf(m, x[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
  const float c0 = a.sigmoid ? fminf(m, 0.0f) : m;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    w[i] = 0.0f;
    if (chosen >> i & 1) {
      if (!a.sigmoid) w[i] = expf(x[i] - c0);
      else if (x[i] > 0.0f) w[i] = 1.0f / (1.0f + expf(-x[i]));
      else w[i] = expf(x[i] - c0) / (1.0f + expf(x[i]));
      if (m == -INFINITY) w[i] = 0.0f;  // no expert of this row has a score
    }
    sum += w[i];
  }
  sum = warp_sum(sum);
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (chosen >> i & 1) w[i] = m == -INFINITY ? 0.0f : a.scale * (w[i] / sum);
  return chosen;
}

// Places the pairs of tokens [t0, t1) in the rows that start at base[e] for each expert.
// Called by the whole CTA; base and mask hold E values each, base filled and a barrier passed.
__device__ __forceinline__ void place_pairs(const RouteArgs& a, int64_t t0, int64_t t1, int* base, unsigned* mask) {
  for (int e = threadIdx.x; e < a.E; e += kRouteThreads) mask[e] = 0;
  for (int64_t tb = t0; tb < t1; tb += 32) {
    const int pairs = static_cast<int>((t1 - tb < 32 ? t1 - tb : 32) * a.k);
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += kRouteThreads) {
      const int e = a.experts[tb * a.k + p];
      if (e >= 0) atomicOr(mask + e, 1u << (p / a.k));
    }
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += kRouteThreads) {
      const int64_t at = tb * a.k + p;
      const int e = a.experts[at], tl = p / a.k;
      int r = -1;
      if (e >= 0) {
        r = base[e] + __popc(mask[e] & ((1u << tl) - 1u));
        a.row_token[r] = static_cast<int32_t>(tb + tl);
        a.row_weight[r] = a.weights[at];
      }
      a.token_rows[at] = r;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) {
      base[e] += __popc(mask[e]);
      mask[e] = 0;
    }
  }
}

// First row of each expert from the experts' counts (in `base`), which it replaces; returns
// the number of rows.  `red` holds kRouteWarps + 1 values.
__device__ __forceinline__ int scan_counts(int E, int* base, int* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  static_assert(kMaxExperts <= kRouteThreads, "an expert a thread");
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
  for (int w = 0; w < kRouteWarps; ++w) {
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

template <typename T, int V>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(RouteArgs a, int per) {
  extern __shared__ double s_rows[];  // [kRouteWarps][E], then the lists [kRouteWarps][E]
  uint16_t* s_list = reinterpret_cast<uint16_t*>(s_rows + kRouteWarps * a.E);
  __shared__ int s_base[kMaxExperts];
  __shared__ unsigned s_mask[kMaxExperts];
  __shared__ int s_red[kRouteWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int e = threadIdx.x; e < a.E; e += kRouteThreads) s_base[e] = 0;
  __syncthreads();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * per, t1 = t0 + per < a.T ? t0 + per : a.T;
  for (int64_t t = t0 + warp; t < t1; t += kRouteWarps) {
    if (a.live && !a.live[t]) {
      if (lane < a.k) {
        a.experts[t * a.k + lane] = -1;
        a.weights[t * a.k + lane] = 0.0f;
      }
      continue;
    }
    float w[V];
    const unsigned chosen = route_token<T, V>(a, t, s_rows + warp * a.E, s_list + warp * a.E, w);
    int at = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool mine = chosen >> i & 1;
      const unsigned all = __ballot_sync(kAll, mine);
      if (mine) {
        const int64_t p = t * a.k + at + __popc(all & ((1u << lane) - 1u));
        a.experts[p] = i * 32 + lane;
        a.weights[p] = w[i];
        if (a.offsets) atomicAdd(s_base + i * 32 + lane, 1);
      }
      at += __popc(all);
    }
  }
  if (!a.offsets) return;
  __syncthreads();
  if (gridDim.x > 1) {
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) a.counts[static_cast<int64_t>(blockIdx.x) * a.E + e] = s_base[e];
    return;
  }
  const int rows = scan_counts(a.E, s_base, s_red);
  for (int e = threadIdx.x; e < a.E; e += kRouteThreads) a.offsets[e] = s_base[e];
  if (threadIdx.x == 0) a.offsets[a.E] = rows;
  place_pairs(a, t0, t1, s_base, s_mask);
  write_rest(a, rows, threadIdx.x, kRouteThreads);
}

// The second pass: a CTA for each CTA of the first, with the same tokens.
__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(RouteArgs a, int per) {
  __shared__ int s_base[kMaxExperts], s_below[kMaxExperts];
  __shared__ unsigned s_mask[kMaxExperts];
  __shared__ int s_red[kRouteWarps];
  for (int e = threadIdx.x; e < a.E; e += kRouteThreads) s_base[e] = s_below[e] = 0;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the counts of all CTAs, and of those before this one
  const int parts = kRouteThreads / a.E, part = threadIdx.x / a.E, e = threadIdx.x - part * a.E;
  if (part < parts) {
    int all = 0, below = 0;
#pragma unroll 8
    for (int c = part; c < static_cast<int>(gridDim.x); c += parts) {
      const int n = a.counts[static_cast<int64_t>(c) * a.E + e];
      all += n;
      below += c < static_cast<int>(blockIdx.x) ? n : 0;
    }
    atomicAdd(s_base + e, all);
    atomicAdd(s_below + e, below);
  }
  __syncthreads();
  const int rows = scan_counts(a.E, s_base, s_red);
  if (threadIdx.x < a.E) {
    if (blockIdx.x == 0) a.offsets[threadIdx.x] = s_base[threadIdx.x];
    s_base[threadIdx.x] += s_below[threadIdx.x];
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.E] = rows;
  __syncthreads();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * per, t1 = t0 + per < a.T ? t0 + per : a.T;
  place_pairs(a, t0, t1, s_base, s_mask);
  write_rest(a, rows, static_cast<int64_t>(blockIdx.x) * kRouteThreads + threadIdx.x, static_cast<int64_t>(gridDim.x) * kRouteThreads);
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
  const bool whole = !a.renorm && !a.sigmoid;  // every expert of the row has a gradient
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
    __syncwarp();
    for (int i = lane; i < a.E; i += 32) row[i] = 0.0f;
    __syncwarp();
    if (e >= 0) row[e] = g;
    __syncwarp();
    for (int i = lane; i < a.E; i += 32) {
      float v = row[i];
      if (whole) v = any && norm != 0.0f ? a.scale * (expf(to_f32(xr[i]) - top) * norm) * (v - base) : 0.0f;
      gr[i] = from_f32<T>(v);
    }
  }
}

template <typename T, int V>
cudaError_t launch_fwd(const RouteArgs& a, int sms, cudaStream_t s) {
  static SmemLimit limit;
  auto kern = route_kernel<T, V>;
  const int ctas = route_ctas(a.T, sms), per = static_cast<int>((a.T + ctas - 1) / ctas);
  if (cudaError_t e = limit.allow(kern, kRouteWarps * kMaxExperts * 10)) return e;
  kern<<<ctas, kRouteThreads, kRouteWarps * a.E * 10, s>>>(a, per);
  if (cudaError_t e = cudaGetLastError()) return e;
  if (!a.offsets || ctas == 1) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(kRouteThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, route_place_kernel, a, per);
}

template <typename T>
cudaError_t launch_typed(bool backward, const RouteArgs& a, int sms, cudaStream_t s) {
  if (backward) {
    const int64_t most = static_cast<int64_t>(sms) * 8, want = (a.T + kRouteBwdWarps - 1) / kRouteBwdWarps;
    route_bwd_kernel<T><<<static_cast<unsigned>(want < most ? want : most), kRouteBwdWarps * 32, kRouteBwdWarps * a.E * 4, s>>>(a);
    return cudaGetLastError();
  }
  if (a.E <= 64) return launch_fwd<T, 2>(a, sms, s);
  if (a.E <= 128) return launch_fwd<T, 4>(a, sms, s);
  if (a.E <= 256) return launch_fwd<T, 8>(a, sms, s);
  return launch_fwd<T, 16>(a, sms, s);
}

}  // namespace

// CTAs of the forward, a contiguous run of tokens each.
int route_ctas(int64_t T, int sms) {
  if (T <= kRouteSingle) return 1;
  const int64_t want = (T + kRouteWarps - 1) / kRouteWarps;
  return static_cast<int>(want < sms ? want : sms);
}

cudaError_t launch_route(bool backward, int dtype, const RouteArgs& a, int sms, cudaStream_t s) {
  if (dtype == NF4_DTYPE_F32) return launch_typed<float>(backward, a, sms, s);
  if (dtype == NF4_DTYPE_F16) return launch_typed<__half>(backward, a, sms, s);
  return launch_typed<__nv_bfloat16>(backward, a, sms, s);
}

}  // namespace nf4
