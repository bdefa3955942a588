// nf4_paged.cu -- the paged key-value cache: new tokens written into their pages
// (nf4_paged_append), and attention of one query token a sequence for every type, width and
// alignment (nf4_paged_attention; 16-bit types of whole 16-byte rows run on the tensor cores).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "elem.cuh"
#include "internal.h"
#include "paged_common.cuh"
#include "smem_limit.h"

namespace nf4 {
namespace {

// ---------------------------------------------------------------------- append --

constexpr int kAppendThreads = 256;

// The place of new row r: its page and slot, or page -1 for none.  Row r of sequence i, the
// last with cu[i] <= r, goes to position lengths[i] - cu[i + 1] + r; without cu_seqlens row r
// is the newest token of sequence r.  The length is taken as it is given: a position that the
// table's row cannot name has no page, and no other token makes room for it.
__device__ __forceinline__ int append_place(const PagedArgs& a, int64_t r, int* slot) {
  int64_t seq = r, end = r + 1;
  if (a.cu_seqlens) {
    int64_t lo = 0, hi = a.nseq;  // cu[lo] <= r < cu[hi], as far as the offsets ascend
    if (r < a.cu_seqlens[0] || r >= a.cu_seqlens[a.nseq]) return -1;
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if (a.cu_seqlens[mid] <= r) lo = mid; else hi = mid;
    }
    seq = lo;
    end = a.cu_seqlens[lo + 1];
  }
  const int64_t len = a.lengths[seq], pos = len - end + r;
  if (len == 0) return -1;  // an idle sequence
  if (pos < 0 || pos >= len || pos >= static_cast<int64_t>(a.max_pages) * a.page_size) {
    if (a.status) atomicCAS(a.status, 0, kStatusBadOffsets);
    return -1;
  }
  return paged_slot(a, seq, static_cast<int>(pos), slot);
}

// Copies `V`-wide pieces of ROWS new rows a CTA.  Bound by HBM: each value is read and
// written once.  8192 rows of 8 heads of 128, bf16: 11.7 us, 5.7 TB/s (18.3 us before a thread
// held one column of eight rows); 64 rows 2.5 us.
template <typename V, int ROWS>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(PagedArgs a, int per_head, int elems) {
  __shared__ int64_t s_k[ROWS], s_v[ROWS];
  grid_allow();
  grid_wait();
  if (a.cu_seqlens && blockIdx.x == 0 && a.status) {
    bool bad = threadIdx.x == 0 && (a.cu_seqlens[0] < 0 || a.cu_seqlens[a.nseq] > a.T);
    for (int64_t i = threadIdx.x; i < a.nseq; i += kAppendThreads) bad |= a.cu_seqlens[i + 1] < a.cu_seqlens[i];
    if (bad) atomicCAS(a.status, 0, kStatusBadOffsets);
  }
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * ROWS;
  if (threadIdx.x < ROWS) {
    int slot = 0;
    const int64_t r = r0 + threadIdx.x;
    const int64_t page = r < a.T ? append_place(a, r, &slot) : -1;
    s_k[threadIdx.x] = page < 0 ? -1 : page * a.k_page + slot * a.k_token;
    s_v[threadIdx.x] = page < 0 ? -1 : page * a.v_page + slot * a.v_token;
  }
  __syncthreads();
  // A thread copies one piece of a row's keys or values, of all rows.
  constexpr int64_t e = sizeof(V);
  const int row = 2 * a.Hk * per_head;
  for (int j = threadIdx.x; j < row; j += kAppendThreads) {
    const int h = j / per_head, hk = h < a.Hk ? h : h - a.Hk;
    const int64_t d = static_cast<int64_t>(j - h * per_head) * elems;
    const bool keys = h < a.Hk;
    const int64_t *at = keys ? s_k : s_v, step = (keys ? a.kn_t : a.vn_t) * e / elems;
    char* to = static_cast<char*>(keys ? a.k : a.v) + (hk * (keys ? a.k_head : a.v_head) + d) * e / elems;
    const char* from = static_cast<const char*>(keys ? a.k_new : a.v_new) + (r0 * (keys ? a.kn_t : a.vn_t) + hk * (keys ? a.kn_h : a.vn_h) + d) * e / elems;
    V v[ROWS];
#pragma unroll
    for (int t = 0; t < ROWS; ++t)
      if (at[t] >= 0) v[t] = *reinterpret_cast<const V*>(from + t * step);
#pragma unroll
    for (int t = 0; t < ROWS; ++t)
      if (at[t] >= 0) *reinterpret_cast<V*>(to + at[t] * e / elems) = v[t];
  }
}

// ------------------------------------------------------- attention, any layout --

// fp32 arithmetic throughout, for rows that no 16-byte copy can take: right for everything, at
// an eighth of the others' rate (64 sequences of 1 to 4096 tokens, 120,000 in all, 32 heads over 8
// of 127, bf16: 570 us, 0.9 TB/s).  A warp takes 32 / HC tokens at a time: its lanes hold the
// tokens' rows 32 columns apart, form the partial products with HC query heads, and reduce the
// 32 sums of (token, head) so that lane i ends with sum i, in 31 shuffles.
constexpr int kAnyWarps = 8;
constexpr int kAnyTile = 6;  // log2 of the tokens of a unit, all warps on one head

template <typename T, int HC, int DV>
__global__ void __launch_bounds__(kAnyWarps * 32) paged_any_kernel(PagedArgs a, int groups) {
  constexpr int NT = 32 / HC;
  extern __shared__ float dyn[];
  float* s_q = dyn;                     // [HC][DV * 32]
  float* s_acc = dyn + HC * DV * 32;    // [4][HC][DV * 32]
  __shared__ int64_t s_red[68];
  __shared__ float s_ml[kAnyWarps][HC][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_allow();
  grid_wait();
  paged_empty<T>(a);
  const int G = a.Hq / a.Hk;
  Walk use = paged_run(a, a.Hk * groups, kAnyTile, s_red);
  PagedRec rec{0, 0, 0};
  const T* kp = static_cast<const T*>(a.k);
  const T* vp = static_cast<const T*>(a.v);

  while (use.left > 0) {
    const int64_t seq = use.seq;
    const int len = use.len, n = use.tiles, t0 = use.tile, t1 = n - t0 < use.left ? n : t0 + use.left;
    const int hk = use.set / groups, g0 = use.set % groups * HC, nh = G - g0 < HC ? G - g0 : HC;
    const int64_t hq = static_cast<int64_t>(hk) * G + g0;

    __syncthreads();  // the last run's readers are done
    for (int i = threadIdx.x; i < HC * DV * 32; i += kAnyWarps * 32) {
      const int h = i / (DV * 32), d = i % (DV * 32);
      s_q[i] = h < nh && d < a.D ? to_f32(static_cast<const T*>(a.q)[seq * a.q_s + (hq + h) * a.q_h + d]) : 0.0f;
    }
    __syncthreads();

    float m = -INFINITY, l = 0.0f, acc[HC][DV];
#pragma unroll
    for (int h = 0; h < HC; ++h)
#pragma unroll
      for (int i = 0; i < DV; ++i) acc[h][i] = 0.0f;
    const int64_t end = (static_cast<int64_t>(t1) << kAnyTile) < len ? static_cast<int64_t>(t1) << kAnyTile : len;
    for (int64_t tb = (static_cast<int64_t>(t0) << kAnyTile) + warp * NT; tb < end; tb += kAnyWarps * NT) {
      int64_t at_k = -1, at_v = -1;
      if (lane < NT && tb + lane < end) {
        int slot;
        const int64_t page = paged_slot(a, seq, static_cast<int>(tb + lane), &slot);
        if (page >= 0) {
          at_k = page * a.k_page + slot * a.k_token + hk * a.k_head;
          at_v = page * a.v_page + slot * a.v_token + hk * a.v_head;
        }
      }
      float kr[NT][DV], vr[NT][DV];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int64_t ok = __shfl_sync(0xffffffffu, at_k, j), ov = __shfl_sync(0xffffffffu, at_v, j);
#pragma unroll
        for (int i = 0; i < DV; ++i) {
          const bool in = ok >= 0 && lane + 32 * i < a.D;
          kr[j][i] = in ? to_f32(kp[ok + lane + 32 * i]) : 0.0f;
          vr[j][i] = in ? to_f32(vp[ov + lane + 32 * i]) : 0.0f;
        }
      }
      float s[32];
#pragma unroll
      for (int h = 0; h < HC; ++h) {
#pragma unroll
        for (int j = 0; j < NT; ++j) s[j * HC + h] = 0.0f;
#pragma unroll
        for (int i = 0; i < DV; ++i) {
          const float qv = s_q[(h * DV + i) * 32 + lane];
#pragma unroll
          for (int j = 0; j < NT; ++j) s[j * HC + h] = fmaf(kr[j][i], qv, s[j * HC + h]);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) {
          const bool up = lane & o;
          const float send = up ? s[i] : s[i + o], keep = up ? s[i + o] : s[i];
          s[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
      const bool live = __shfl_sync(0xffffffffu, at_k, lane / HC) >= 0;
      const float x = live ? s[0] * (a.scale * kLog2e) : -INFINITY;
      float top = x;
#pragma unroll
      for (int o = HC; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      top = fmaxf(top, m);
      const float mm = top == -INFINITY ? 0.0f : top;
      const float p = exp2f(x - mm), down = exp2f(m - mm);
      if (__any_sync(0xffffffffu, down != 1.0f)) {
#pragma unroll
        for (int h = 0; h < HC; ++h) {
          const float f = __shfl_sync(0xffffffffu, down, h);
#pragma unroll
          for (int i = 0; i < DV; ++i) acc[h][i] *= f;
        }
      }
      m = top;
      l = l * down + p;
      const float pv = p * PagedSums<T>::kDown;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int h = 0; h < HC; ++h) {
          const float w = __shfl_sync(0xffffffffu, pv, j * HC + h);
#pragma unroll
          for (int i = 0; i < DV; ++i) acc[h][i] = fmaf(w, vr[j][i], acc[h][i]);
        }
    }
#pragma unroll
    for (int o = HC; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane < HC) {
      s_ml[warp][lane][0] = m;
      s_ml[warp][lane][1] = l;
    }
    __syncthreads();
    float top = -INFINITY, sum = 0.0f;
    const int mine = lane % HC;
#pragma unroll
    for (int w = 0; w < kAnyWarps; ++w) top = fmaxf(top, s_ml[w][mine][0]);
    const float mm = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int w = 0; w < kAnyWarps; ++w) sum += s_ml[w][mine][1] * exp2f(s_ml[w][mine][0] - mm);
    const float f = exp2f(m - mm);
#pragma unroll
    for (int h = 0; h < HC; ++h) {
      const float fh = __shfl_sync(0xffffffffu, f, h);
#pragma unroll
      for (int i = 0; i < DV; ++i) acc[h][i] *= fh;
    }
    // the warps' sums in a tree
#pragma unroll
    for (int half = kAnyWarps / 2; half > 0; half >>= 1) {
      if (warp >= half && warp < 2 * half)
#pragma unroll
        for (int h = 0; h < HC; ++h)
#pragma unroll
          for (int i = 0; i < DV; ++i) s_acc[(((warp - half) * HC + h) * DV + i) * 32 + lane] = acc[h][i];
      __syncthreads();
      if (warp < half)
#pragma unroll
        for (int h = 0; h < HC; ++h)
#pragma unroll
          for (int i = 0; i < DV; ++i) acc[h][i] += s_acc[((warp * HC + h) * DV + i) * 32 + lane];
      __syncthreads();
    }
    if (warp == 0) {
      const bool whole = t0 == 0 && t1 == n;
      const int st = paged_part_stride(a.D);
      float* part = a.part + static_cast<int64_t>(blockIdx.x * 2 + (t0 == 0)) * HC * st;
#pragma unroll
      for (int h = 0; h < HC; ++h) {
        const float lh = __shfl_sync(0xffffffffu, sum, h), th = __shfl_sync(0xffffffffu, top, h);
        if (h < nh) {
          T* o = static_cast<T*>(a.o) + seq * a.o_s + (hq + h) * a.o_h;
#pragma unroll
          for (int i = 0; i < DV; ++i)
            if (lane + 32 * i < a.D) {
              if (whole) o[lane + 32 * i] = from_f32<T>(paged_mean<T>(acc[h][i], lh));
              else part[h * st + lane + 32 * i] = acc[h][i];
            }
          if (lane == 0) {
            if (whole) {
              if (a.lse) a.lse[seq * a.Hq + hq + h] = th * kLn2 + logf(lh);
            } else {
              part[h * st + st - 4] = th;
              part[h * st + st - 3] = lh;
            }
          }
        }
      }
    }
    if (t0 > 0) rec.flags |= t1 == n ? 6 : 2;
    if (t0 == 0 && t1 < n) {
      rec.flags |= 1;
      rec.seq = seq;
      rec.set = use.set;
    }
    use.left -= t1 - t0 - 1;
    use.tile = t1 - 1;
    use.next(a);
  }
  if (threadIdx.x == 0) a.rec[blockIdx.x] = rec;
}

constexpr int kAnyCtas = 2;  // a SM: what the registers leave room for

template <typename T, int HC, int DV>
cudaError_t launch_any(const PagedArgs& a, int sms, cudaStream_t s) {
  static SmemLimit limit;
  auto kern = paged_any_kernel<T, HC, DV>;
  const int smem = 5 * HC * DV * 32 * static_cast<int>(sizeof(float));
  if (cudaError_t e = limit.allow(kern, smem)) return e;
  const int groups = (a.Hq / a.Hk + HC - 1) / HC;
  if (cudaError_t e = launch_early(kern, dim3(static_cast<unsigned>(kAnyCtas * sms)), kAnyWarps * 32, smem, s, a, groups)) return e;
  return launch_paged_join<T>(a, kAnyCtas * sms, HC, groups, 1, s);
}

template <typename T, int HC>
cudaError_t launch_any_width(const PagedArgs& a, int sms, cudaStream_t s) {
  if (a.D <= 64) return launch_any<T, HC, 2>(a, sms, s);
  if (a.D <= 128) return launch_any<T, HC, 4>(a, sms, s);
  return launch_any<T, HC, 8>(a, sms, s);
}

template <typename T>
cudaError_t launch_any_heads(const PagedArgs& a, int sms, cudaStream_t s) {
  return a.Hq / a.Hk <= 4 ? launch_any_width<T, 4>(a, sms, s) : launch_any_width<T, 8>(a, sms, s);
}

}  // namespace

PagedShape paged_shape_any(int G, int Hk) { return paged_shape(G, Hk, G <= 4 ? 4 : 8, 1, kAnyCtas, false); }

cudaError_t launch_paged_any(int dtype, const PagedArgs& a, int sms, cudaStream_t s) {
  if (dtype == NF4_DTYPE_F32) return launch_any_heads<float>(a, sms, s);
  if (dtype == NF4_DTYPE_F16) return launch_any_heads<__half>(a, sms, s);
  return launch_any_heads<__nv_bfloat16>(a, sms, s);
}

namespace {

template <typename V>
cudaError_t launch_append(const PagedArgs& a, int per_head, int elems, int sms, cudaStream_t s) {
  if (a.T < 32 * static_cast<int64_t>(sms))  // few rows: a CTA each
    return launch_early(paged_append_kernel<V, 1>, dim3(static_cast<unsigned>(a.T)), kAppendThreads, 0, s, a, per_head, elems);
  return launch_early(paged_append_kernel<V, 8>, dim3(static_cast<unsigned>((a.T + 7) / 8)), kAppendThreads, 0, s, a, per_head, elems);
}

}  // namespace

cudaError_t launch_paged_append(int dtype, const PagedArgs& a, int sms, cudaStream_t s) {
  const int e = dtype == NF4_DTYPE_F32 ? 4 : 2, wide = 16 / e;
  const int64_t ld[] = {a.k_page, a.k_token, a.k_head, a.v_page, a.v_token, a.v_head, a.kn_t, a.kn_h, a.vn_t, a.vn_h, a.D};
  const void* p[] = {a.k, a.v, a.k_new, a.v_new};
  bool vec = true;
  for (int64_t x : ld) vec = vec && x % wide == 0;
  for (const void* x : p) vec = vec && reinterpret_cast<uintptr_t>(x) % 16 == 0;
  if (vec) return launch_append<uint4>(a, a.D / wide, wide, sms, s);
  if (e == 4) return launch_append<uint32_t>(a, a.D, 1, sms, s);
  return launch_append<uint16_t>(a, a.D, 1, sms, s);
}

}  // namespace nf4
