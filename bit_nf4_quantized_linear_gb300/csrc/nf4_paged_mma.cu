// nf4_paged_mma.cu -- attention of one query token a sequence over the paged cache, 16-bit
// types, on the tensor cores (nf4_paged_attention).
//
// The query heads of one key head are the narrow side of two products: S' = K Q' (16 tokens x
// 8 heads an MMA) and O' += V' P' (16 columns x 8 heads), so a group of up to 8 heads wastes
// nothing of the key and value rows, which are read once.  Bound by HBM: 2 D values a token
// and key head against 4 D operations a query head; mma.sync's rate is some ten times what
// that needs, and its operands come from shared memory as the copies left them.
//
// A CTA's four warps share out heads or tokens (paged_common.cuh), 16 tokens a warp's tile.  Each
// warp streams its tokens' rows through a ring of its own (paged_ring.cuh), over the borders of
// sequences and head sets, with no barrier in the loop; where several warps share a head they meet
// as it ends, to add their sums.
// S is fp32; P is held as two values of the operands' type, what the type holds of p and the
// rest (a second MMA that costs nothing here: with both in one the times are the same), so the
// result sees one rounding, its own.  fp16 weights are held times 2^7, out of the subnormal
// range.
//
// Measured, bf16, 32 heads over 8 of 128 unless said (device time with the join; 6.70 TB/s is a
// plain copy's rate; bytes: keys and values once): 64 sequences of 1 to 16384 tokens (480,000 in
// all) 286 us, 6.9 TB/s; one of 131072 tokens 89 us, 6.0 TB/s; 200 of 64 to 1024 (111,000) in
// fp16, 40 heads over 8, 84 us, 5.4 TB/s; 24 of 500 to 3000 (48,000), 32 unshared heads of 64, 66
// us, 5.9 TB/s; one sequence of 37 tokens, 9 us.  Other widths, 32 of 1 to 8192 (146,300): 136
// columns 145 us, 4.4 TB/s, 192 153 us, 5.9, 256 187 us, 6.4.  Groups, 64 of 1 to 8192 (266,600;
// 163 us of bytes): 4 heads 168 us, 8 177, 16 206; from there on the rows are read once for each
// 16: 20 heads 280 us, 32 290, 40 408.  Of a call some 9 us are fixed: launch and cut 3.5, a
// tile's chain of loads and products 2, the join 3.5.  In a long run HBM's order counts: fewer bytes in flight (two ring stages instead of
// three: -4%) and longer pieces a CTA (its warps on neighbouring heads: -7%) beat more of them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "elem.cuh"
#include "internal.h"
#include "paged_common.cuh"
#include "paged_ring.cuh"
#include "sm100_ptx.cuh"
#include "smem_limit.h"

namespace nf4 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;  // tokens of a warp's tile: the MMA's rows

template <int DM>
struct Geo {
  static constexpr int kStages = DM == 128 ? 2 : 3;
  static constexpr int kHalf = kRows * DM * 2;      // bytes of a tile's keys
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kPitch = DM + 4;             // floats between heads of a warp's sums
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kSums = kWarps * 4 * kPitch * 4;  // four heads at a time
  static constexpr int kSmem = kRing + kSums + kWarps * 8 * 8 + kWarps * kStages * 4;
};

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Weights a and b as two values each of the operands' type: what the type holds of them (cut,
// not rounded), and the rest, never negative and never 0 beside a first part, so that an
// infinite value times the weight is that infinity and not 0 x inf.  Both parts of a weight of 0
// are 0: its token adds nothing, however large its finite value.
template <bool F16>
__device__ __forceinline__ void split2(float a, float b, uint32_t* hi, uint32_t* lo) {
  if constexpr (F16) {
    constexpr float least = 5.9604645e-8f;  // 2^-24, of weights up to 2^7
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(*hi) : "f"(b), "f"(a));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(hi));
    const float ra = f.x > 0.0f ? fmaxf(a - f.x, least) : a - f.x, rb = f.y > 0.0f ? fmaxf(b - f.y, least) : b - f.y;
    const __half2 l = __floats2half2_rn(ra, rb);
    *lo = *reinterpret_cast<const uint32_t*>(&l);
  } else {
    constexpr float least = 1.1754944e-38f;
    const uint32_t ua = __float_as_uint(a) & 0xffff0000u, ub = __float_as_uint(b) & 0xffff0000u;
    *hi = ua >> 16 | ub;
    const float ra = a - __uint_as_float(ua), rb = b - __uint_as_float(ub);
    const __nv_bfloat162 l = __floats2bfloat162_rn(ua ? fmaxf(ra, least) : ra, ub ? fmaxf(rb, least) : rb);
    *lo = *reinterpret_cast<const uint32_t*>(&l);
  }
}

template <bool F16, int DM, int NT, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) paged_mma_kernel(PagedArgs a, int groups, int log2_wh) {
  using G = Geo<DM>;
  using T = typename std::conditional<F16, __half, __nv_bfloat16>::type;
  constexpr int HC = 8 * NT, KS = DM / 16;
  constexpr float kShift = F16 ? 7.0f : 0.0f;
  extern __shared__ __align__(128) unsigned char dyn[];
  float* s_sum = reinterpret_cast<float*>(dyn + G::kRing);                          // [kWarps][4][kPitch]
  float2* s_ml = reinterpret_cast<float2*>(dyn + G::kRing + G::kSums);              // [kWarps][8]
  uint32_t* s_valid = reinterpret_cast<uint32_t*>(s_ml + kWarps * 8);               // [kWarps][kStages]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wh = 1 << log2_wh, wt = kWarps >> log2_wh, my_head = warp & (wh - 1), my_tile = warp >> log2_wh;
  const uint32_t ring = nf4ptx::smem_addr(dyn) + warp * G::kStages * G::kStage;
  s_valid += warp * G::kStages;
  grid_allow();
  grid_wait();
  const int GQ = a.Hq / a.Hk;
  Walk load = paged_run(a, a.Hk * groups >> log2_wh, 6 - log2_wh, reinterpret_cast<int64_t*>(s_sum));  // 16 wt tokens a unit
  Walk use = load;
  PagedRec rec{0, 0, 0};

  if (use.left > 0) {
    TileCopies<T, DM, kRows> copies(a, ring, s_valid);
    // The key head of this warp in a head set, and its first query head's place in the group.
    auto place = [&](int set, int* g0) {
      const int head = (set << log2_wh) + my_head, hk = groups == 1 ? head : head / groups;
      *g0 = (head - hk * groups) * HC;
      return hk;
    };
    auto first_token = [&](const Walk& w) { return (w.tile << w.log2_tile) + my_tile * kRows; };
    auto start_copies = [&](int st) {
      int g0;
      copies.start(a, load, first_token(load), place(load.set, &g0), st);
      if (load.left > 0) load.next(a);
      copies.look_up(a, load, first_token(load));
    };

    uint32_t qf[NT][KS][2];
    float acc[NT][KS][4], m[NT][2], l[NT][2];
    const float c = a.scale * kLog2e;
    // Offsets of the ldmatrix rows in a tile: the swizzle repeats after four steps of two chunks.
    constexpr int KO = KS < 4 ? KS : 4;
    uint32_t k_off[KO], v_off[KO];
#pragma unroll
    for (int s = 0; s < KO; ++s) {
      k_off[s] = ring + at_chunk<DM * 2>(lane & 15, 2 * s + (lane >> 4));
      v_off[s] = ring + G::kHalf + at_chunk<DM * 2>((lane & 7) + (lane >> 4 << 3), 2 * s + (lane >> 3 & 1));
    }
    int tile0 = use.tile;  // where the part of this (sequence, head set) begins
    // The queries of the unit `use` as the right operand, 16 columns a step.
    auto fetch_queries = [&]() {
      int g0;
      const int hk = place(use.set, &g0);
      const T* q = static_cast<const T*>(a.q) + use.seq * a.q_s + (static_cast<int64_t>(hk) * GQ + g0 + lane / 4) * a.q_h + (lane & 3) * 2;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int d = s * 16 + j * 8;
            qf[n][s][j] = g0 + n * 8 + lane / 4 < GQ && d < a.D ? *reinterpret_cast<const uint32_t*>(q + n * 8 * a.q_h + d) : 0u;
          }
    };
    auto clear_sums = [&]() {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[n][s][j] = 0.0f;
      }
    };
    copies.look_up(a, load, first_token(load));
#pragma unroll
    for (int i = 0; i < G::kStages; ++i) start_copies(i);
    fetch_queries();
    clear_sums();
    paged_empty<T>(a);
    int st = 0;
    while (use.left > 0) {
      copies_wait<G::kStages - 1>();
      __syncwarp();
      if (first_token(use) < use.len) {
        const uint32_t from = st * G::kStage;
        const unsigned valid = s_valid[st];
        float x[NT][4], x2[NT][4];  // two chains of MMAs
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) x[n][j] = x2[n][j] = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          uint32_t kf[4];
          ldsm(kf, k_off[s % KO] + from + s / KO * 128);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma<F16>(s & 1 ? x2[n] : x[n], kf, qf[n][s][0], qf[n][s][1]);
        }
        uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          // x: tokens lane / 4 and lane / 4 + 8, heads 2 (lane % 4) and the next
#pragma unroll
          for (int j = 0; j < 4; ++j) x[n][j] = (x[n][j] + x2[n][j]) * c;
          if (valid != 0xffffu)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (!(valid >> (lane / 4 + (j & 2) * 4) & 1)) x[n][j] = -INFINITY;
          float t0 = fmaxf(x[n][0], x[n][2]), t1 = fmaxf(x[n][1], x[n][3]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, o));
            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, o));
          }
          if (__any_sync(0xffffffffu, t0 > m[n][0] || t1 > m[n][1])) {
            t0 = fmaxf(t0, m[n][0]);
            t1 = fmaxf(t1, m[n][1]);
            const float f0 = t0 == -INFINITY ? 1.0f : exp2_fast(m[n][0] - t0), f1 = t1 == -INFINITY ? 1.0f : exp2_fast(m[n][1] - t1);
            m[n][0] = t0;
            m[n][1] = t1;
            l[n][0] *= f0;
            l[n][1] *= f1;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
              acc[n][s][0] *= f0;
              acc[n][s][1] *= f1;
              acc[n][s][2] *= f0;
              acc[n][s][3] *= f1;
            }
          }
          const float b0 = m[n][0] == -INFINITY ? 0.0f : m[n][0] - kShift, b1 = m[n][1] == -INFINITY ? 0.0f : m[n][1] - kShift;
#pragma unroll
          for (int j = 0; j < 4; ++j) x[n][j] = exp2_fast(x[n][j] - (j & 1 ? b1 : b0));
          l[n][0] += x[n][0] + x[n][2];
          l[n][1] += x[n][1] + x[n][3];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            split2<F16>(x[n][2 * j] * PagedSums<T>::kDown, x[n][2 * j + 1] * PagedSums<T>::kDown, &hi[n][j], &lo[n][j]);
            hi[n][j] = transpose8(hi[n][j]);
            lo[n][j] = transpose8(lo[n][j]);
          }
        }
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          uint32_t vf[4];
          ldsm_t(vf, v_off[s % KO] + from + s / KO * 128);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma<F16>(acc[n][s], vf, hi[n][0], hi[n][1]);
            mma<F16>(acc[n][s], vf, lo[n][0], lo[n][1]);
          }
        }
      }
      __syncwarp();
      start_copies(st);
      st = st + 1 == G::kStages ? 0 : st + 1;

      const bool ends = use.tile + 1 == use.tiles;
      if (!ends && use.left > 1) {
        use.next(a);
        continue;
      }
      // The part of this (sequence, head set) is done: its outputs, or its sums.  The next one's
      // queries are fetched meanwhile.
      int g0;
      const int hk = place(use.set, &g0);
      const int64_t seq = use.seq;
      const bool whole = ends && tile0 == 0;
      const int stride = paged_part_stride(a.D);
      if (tile0 > 0) rec.flags |= ends ? 6 : 2;
      if (tile0 == 0 && !ends) {
        rec.flags |= 1;
        rec.seq = seq;
        rec.set = use.set;
      }
      float* part = a.part + (static_cast<int64_t>(blockIdx.x * 2 + (tile0 == 0)) * (HC << log2_wh) + my_head * HC) * stride;
      use.next(a);
      if (use.left > 0) fetch_queries();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          l[n][0] += __shfl_xor_sync(0xffffffffu, l[n][0], o);
          l[n][1] += __shfl_xor_sync(0xffffffffu, l[n][1], o);
        }
        if (lane < 4)
#pragma unroll
          for (int j = 0; j < 2; ++j) s_ml[warp * 8 + lane * 2 + j] = make_float2(m[n][j] - kShift, l[n][j]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // four heads at a time, which lie in lanes 0, 1 or 2, 3 of four
          if ((lane >> 1 & 1) == half) {
            float* own = s_sum + (warp * 4 + (lane & 1) * 2) * G::kPitch + lane / 4;
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
              for (int j = 0; j < 4; ++j) own[(j & 1) * G::kPitch + s * 16 + (j & 2) * 4] = acc[n][s][j];
          }
          if (wt > 1) __syncthreads();
          else __syncwarp();
          // the warps of a head take its query heads in turn, a lane four columns
#pragma unroll 2
          for (int i = lane; i < (4 / wt) * (DM / 4); i += 32) {
            const int h4 = my_tile + wt * (i / (DM / 4)), h = half * 4 + h4, d = i % (DM / 4) * 4, hn = n * 8 + h;
            if (g0 + hn >= GQ) break;
            float top = -INFINITY, sum = 0.0f;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (wt == 1) {
              const float2 ml = s_ml[warp * 8 + h];
              top = ml.x;
              sum = ml.y;
              v = *reinterpret_cast<const float4*>(s_sum + (warp * 4 + h4) * G::kPitch + d);
            } else {
              for (int w = my_head; w < kWarps; w += wh) top = fmaxf(top, s_ml[w * 8 + h].x);
              const float mm = top == -INFINITY ? 0.0f : top;
              for (int w = my_head; w < kWarps; w += wh) {
                const float2 ml = s_ml[w * 8 + h];
                const float f = exp2_fast(ml.x - mm);
                const float4 x = *reinterpret_cast<const float4*>(s_sum + (w * 4 + h4) * G::kPitch + d);
                sum += ml.y * f;
                v.x += x.x * f;
                v.y += x.y * f;
                v.z += x.z * f;
                v.w += x.w * f;
              }
            }
            const int64_t hq = static_cast<int64_t>(hk) * GQ + g0 + hn;
            if (d < a.D) {  // D is a multiple of 8
              if (whole) {
                const float inv = paged_mean<T>(1.0f, sum);
                __align__(8) T r[4] = {from_f32<T>(v.x * inv), from_f32<T>(v.y * inv), from_f32<T>(v.z * inv), from_f32<T>(v.w * inv)};
                *reinterpret_cast<uint2*>(static_cast<T*>(a.o) + seq * a.o_s + hq * a.o_h + d) = *reinterpret_cast<const uint2*>(r);
              } else {
                *reinterpret_cast<float4*>(part + hn * stride + d) = v;
              }
            }
            if (d == 0) {
              if (!whole) {
                part[hn * stride + stride - 4] = top;
                part[hn * stride + stride - 3] = sum;
              } else if (a.lse) {
                a.lse[seq * a.Hq + hq] = top * kLn2 + logf(sum);
              }
            }
          }
          if (wt > 1) __syncthreads();
          else __syncwarp();
        }
      }
      tile0 = use.tile;
      clear_sums();
    }
    copies_wait<0>();
  } else {
    paged_empty<T>(a);
  }
  if (threadIdx.x == 0) a.rec[blockIdx.x] = rec;
}

template <bool F16, int DM, int NT, int CTAS>
cudaError_t launch(const PagedArgs& a, const PagedShape& p, int sms, cudaStream_t s) {
  using G = Geo<DM>;
  static SmemLimit limit;
  auto kern = paged_mma_kernel<F16, DM, NT, CTAS>;
  if (cudaError_t e = limit.allow(kern, G::kSmem)) return e;
  const int ctas = p.ctas * sms;
  if (cudaError_t e = launch_early(kern, dim3(static_cast<unsigned>(ctas)), kThreads, G::kSmem, s, a, p.groups, log2_of(p.wh))) return e;
  return launch_paged_join<typename std::conditional<F16, __half, __nv_bfloat16>::type>(a, ctas, p.group, p.groups, p.wh, s);
}

template <bool F16>
cudaError_t launch_width(const PagedArgs& a, int sms, cudaStream_t s) {
  const PagedShape p = paged_shape_mma(a.Hq / a.Hk, a.Hk, a.D, a.k_head < a.k_token);
  const bool wide = p.group == 16;
  if (a.D <= 64) return wide ? launch<F16, 64, 2, 3>(a, p, sms, s) : launch<F16, 64, 1, 3>(a, p, sms, s);
  if (a.D > 128) return launch<F16, 256, 1, 1>(a, p, sms, s);
  if (wide) return launch<F16, 128, 2, 3>(a, p, sms, s);
  return p.ctas == 3 ? launch<F16, 128, 1, 3>(a, p, sms, s) : launch<F16, 128, 1, 2>(a, p, sms, s);
}

}  // namespace

// Groups of 16 query heads from 9 on, so that the rows are read half as often (not beside the
// registers that 256 columns take: 64 heads over 8 of 256 run at the bytes' rate, 333 us for 326,
// 128 over 8 at 499).  Three CTAs a SM where a tile's arithmetic takes longer than its bytes, two
// where HBM is busy with fewer, whose order it minds.  64 sequences of 1 to 8192 tokens (266,600
// in all), 32 heads over 8, us with two and with three, in pages of 16 and of 24 (which no tile
// fits):
//   columns   72        80        88        96        104       112       120       128
//   of 16  125, 121  125, 120  138, 148  138, 138  161, 171  158, 160  180, 187  168, 172
//   of 24  149, 124  148, 124  151, 149  149, 139  157, 168  160, 160  179, 186  172, 176
// (The cut at 112 gives 104 columns, and 88 in pages of 16, 6 to 7% too much.)
PagedShape paged_shape_mma(int G, int Hk, int D, bool together) {
  const int group = G > 8 && D <= 128 ? 16 : 8, ctas = D > 128 ? 1 : D > 112 && group == 8 ? 2 : 3;
  return paged_shape(G, Hk, group, kWarps, ctas, together);
}

cudaError_t launch_paged_mma(bool f16, const PagedArgs& a, int sms, cudaStream_t s) {
  return f16 ? launch_width<true>(a, sms, s) : launch_width<false>(a, sms, s);
}

}  // namespace nf4
