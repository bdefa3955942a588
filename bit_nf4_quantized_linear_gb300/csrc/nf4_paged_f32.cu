// nf4_paged_f32.cu -- attention of one query token a sequence over the paged cache in fp32
// (nf4_paged_attention): rows of whole 16-byte pieces.
//
// The arithmetic is fp32 on the ordinary cores, 4 D operations a query head and token against
// 8 D bytes a key head and token: up to a group of some eight heads HBM would bound it, if the
// rows come in time and few instructions move them about.  They stream through per-warp rings as in
// the tensor-core kernel (paged_ring.cuh), 8 tokens a warp's tile.  Scores: a lane takes one
// token and a quarter of its columns; every 16 bytes of a key meet 16 of each head's query
// (a broadcast); the quarters are added so that a quarter's lanes end with its heads.  Sums: a
// lane takes 16 bytes of columns of all tokens, the weights come back through shared memory.
// Packed fp32 pairs halve the multiply-adds.
//
// Measured (device time with the join; bytes: keys and values once): 32 sequences of 1 to 16384
// tokens (269,000 in all), 32 heads over 8 of 128, 329 us, 6.7 TB/s.  64 of 500 to 3000 (119,600),
// 8 key heads of 64: 32 heads 84 us, 5.9 TB/s; 64 heads 112 us, 4.4 TB/s, where no unit is full
// (issue slots 59%, shared memory's wavefronts 54%, HBM 56%): 16 warps an SM, each with one tile's
// chain of shared-memory reads, multiply-adds and exponentials, and a 16-byte read of a query for
// two packed multiply-adds.  32 of 1 to 4096 (64,600), 32 heads over 8 of 200, 178 us, 4.6 TB/s:
// the same with four warps an SM (issue slots 26%, wavefronts 51%).  Seven of 1 to 2000, 12 heads
// over 4 of 80, 16 us (launches, cut and join).
#include <cuda_runtime.h>

#include <cstdint>

#include "elem.cuh"
#include "internal.h"
#include "paged_common.cuh"
#include "paged_ring.cuh"
#include "sm100_ptx.cuh"
#include "smem_limit.h"

namespace nf4 {
namespace {

constexpr int kRows = 8;  // tokens of a warp's tile: a lane a token and quarter of its columns

template <int DM, int HC>
struct Geo {
  static constexpr int kWarps = DM <= 128 ? 8 : 4, kThreads = kWarps * 32;
  static constexpr int kStages = 2;
  static constexpr int kCtas = DM == 64 ? 2 : 1;  // a SM
  static constexpr int kPitch = DM + 4;           // floats between heads of a warp's sums
  static constexpr int kRing = kWarps * kStages * TileCopies<float, DM, kRows>::kStage;
  static constexpr int kSums = kWarps * 4 * kPitch * 4;  // four heads at a time
  static constexpr int kQ = kWarps * HC * DM * 4;
  static constexpr int kP = kWarps * kRows * HC * 4;
  static constexpr int kMl = kWarps * HC * 8;
  static constexpr int kSmem = kRing + kSums + kQ + kP + kMl + kWarps * kStages * 4;
};

template <int DM, int HC>
__global__ void __launch_bounds__(Geo<DM, HC>::kThreads, Geo<DM, HC>::kCtas) paged_f32_kernel(PagedArgs a, int groups, int log2_wh) {
  using G = Geo<DM, HC>;
  using Copies = TileCopies<float, DM, kRows>;
  constexpr int kWarps = G::kWarps;
  constexpr int HL = HC / 4;                    // heads of a quarter's lanes
  constexpr int PQ = DM / 16;                   // 16-byte pieces of a quarter row
  constexpr int TP = DM == 64 ? 2 : 1;          // tokens that a warp's read of one piece a lane covers
  constexpr int PL = DM <= 128 ? 1 : DM / 128;  // pieces of a row that a lane sums
  extern __shared__ __align__(128) unsigned char dyn[];
  float* s_sum = reinterpret_cast<float*>(dyn + G::kRing);          // [kWarps][4][kPitch]
  float* s_q = reinterpret_cast<float*>(dyn + G::kRing + G::kSums); // [kWarps][HC][DM]
  float* s_p = s_q + kWarps * HC * DM;                              // [kWarps][kRows][HC]
  float2* s_ml = reinterpret_cast<float2*>(s_p + kWarps * kRows * HC);  // [kWarps][HC]
  uint32_t* s_valid = reinterpret_cast<uint32_t*>(s_ml + kWarps * HC);  // [kWarps][kStages]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wh = 1 << log2_wh, wt = kWarps >> log2_wh, my_head = warp & (wh - 1), my_tile = warp >> log2_wh;
  const unsigned char* ring = dyn + warp * G::kStages * Copies::kStage;
  s_q += warp * HC * DM;
  s_p += warp * kRows * HC;
  s_valid += warp * G::kStages;
  grid_allow();
  grid_wait();
  const int GQ = a.Hq / a.Hk;
  Walk load = paged_run(a, a.Hk * groups >> log2_wh, (kWarps == 8 ? 6 : 5) - log2_wh, reinterpret_cast<int64_t*>(s_sum));  // 8 wt tokens a unit
  Walk use = load;
  PagedRec rec{0, 0, 0};

  if (use.left > 0) {
    Copies copies(a, nf4ptx::smem_addr(ring), s_valid);
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
    auto fetch_queries = [&]() {
      int g0;
      const int hk = place(use.set, &g0);
      const float* q = static_cast<const float*>(a.q) + use.seq * a.q_s + (static_cast<int64_t>(hk) * GQ + g0) * a.q_h;
#pragma unroll
      for (int i = 0; i < HC * DM / 32; ++i) {
        const int h = i * 32 / DM, d = (i * 32 + lane) % DM;
        s_q[i * 32 + lane] = g0 + h < GQ && d < a.D ? q[h * a.q_h + d] : 0.0f;
      }
    };
    // lane (t, r): token t = lane % 8; as quarter r = lane / 8 it keeps heads r HL .. r HL + HL - 1
    const int t = lane & 7, r = lane >> 3;
    float2 acc[HC][2 * PL];
    float m[HL], l[HL];
    auto clear_sums = [&]() {
#pragma unroll
      for (int h = 0; h < HC; ++h)
#pragma unroll
        for (int i = 0; i < 2 * PL; ++i) acc[h][i] = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int j = 0; j < HL; ++j) {
        m[j] = -INFINITY;
        l[j] = 0.0f;
      }
    };
    const float c = a.scale * kLog2e;
    copies.look_up(a, load, first_token(load));
#pragma unroll
    for (int i = 0; i < G::kStages; ++i) start_copies(i);
    fetch_queries();
    clear_sums();
    paged_empty<float>(a);
    int st = 0, tile0 = use.tile;  // where the part of this (sequence, head set) begins
    while (use.left > 0) {
      copies_wait<G::kStages - 1>();
      __syncwarp();
      if (first_token(use) < use.len) {
        const unsigned char* keys = ring + st * Copies::kStage;
        const unsigned char* values = keys + Copies::kHalf;
        float2 s2[HC];
#pragma unroll
        for (int h = 0; h < HC; ++h) s2[h] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < PQ; ++i) {
          const float4 k = *reinterpret_cast<const float4*>(keys + at_chunk<DM * 4>(t, r * PQ + i));
#pragma unroll
          for (int h = 0; h < HC; ++h) {
            const float4 q = *reinterpret_cast<const float4*>(s_q + h * DM + (r * PQ + i) * 4);
            s2[h] = fma2(make_float2(k.x, k.y), make_float2(q.x, q.y), s2[h]);
            s2[h] = fma2(make_float2(k.z, k.w), make_float2(q.z, q.w), s2[h]);
          }
        }
        // the quarters' sums, halved twice: heads of the upper half to the lanes of quarters 2 and 3, and so on
        float s[HC];
#pragma unroll
        for (int h = 0; h < HC; ++h) s[h] = s2[h].x + s2[h].y;
#pragma unroll
        for (int h = 0; h < HC / 2; ++h) {
          const bool up = r & 2;
          const float send = up ? s[h] : s[h + HC / 2], keep = up ? s[h + HC / 2] : s[h];
          s[h] = keep + __shfl_xor_sync(0xffffffffu, send, 16);
        }
#pragma unroll
        for (int h = 0; h < HL; ++h) {
          const bool up = r & 1;
          const float send = up ? s[h] : s[h + HL], keep = up ? s[h + HL] : s[h];
          s[h] = keep + __shfl_xor_sync(0xffffffffu, send, 8);
        }
        const bool live = s_valid[st] >> t & 1;
        float down[HL];
        bool moved = false;
#pragma unroll
        for (int j = 0; j < HL; ++j) {
          s[j] = live ? s[j] * c : -INFINITY;
          float top = s[j];
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          top = fmaxf(top, m[j]);
          const float mm = top == -INFINITY ? 0.0f : top;
          down[j] = exp2_fast(m[j] - mm);
          moved |= top != m[j];
          m[j] = top;
          const float p = exp2_fast(s[j] - mm);
          l[j] = l[j] * down[j] + p;
          s_p[t * HC + r * HL + j] = p * PagedSums<float>::kDown;
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int h = 0; h < HC; ++h) {
            const float f = __shfl_sync(0xffffffffu, down[h % HL], h / HL * 8);
#pragma unroll
            for (int i = 0; i < 2 * PL; ++i) acc[h][i] = mul2(acc[h][i], make_float2(f, f));
          }
        }
        __syncwarp();
        const int piece = TP == 2 ? lane & 15 : lane, sub = TP == 2 ? lane >> 4 : 0;
#pragma unroll
        for (int i = 0; i < kRows / TP; ++i) {
          const int tok = i * TP + sub;
          float4 v[PL];
#pragma unroll
          for (int j = 0; j < PL; ++j) v[j] = *reinterpret_cast<const float4*>(values + at_chunk<DM * 4>(tok, piece + 32 * j));
#pragma unroll
          for (int h = 0; h < HC; h += 4) {
            const float4 p = *reinterpret_cast<const float4*>(s_p + tok * HC + h);
            const float w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int j = 0; j < PL; ++j) {
                acc[h + k][2 * j] = fma2(make_float2(w[k], w[k]), make_float2(v[j].x, v[j].y), acc[h + k][2 * j]);
                acc[h + k][2 * j + 1] = fma2(make_float2(w[k], w[k]), make_float2(v[j].z, v[j].w), acc[h + k][2 * j + 1]);
              }
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
      // The part of this (sequence, head set) is done: its outputs, or its sums.
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
      for (int j = 0; j < HL; ++j) {
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) l[j] += __shfl_xor_sync(0xffffffffu, l[j], o);
        if (t == 0) s_ml[warp * HC + r * HL + j] = make_float2(m[j], l[j]);
      }
      if (DM == 64) {  // the two halves of the warp took every other token
#pragma unroll
        for (int h = 0; h < HC; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            acc[h][i].x += __shfl_xor_sync(0xffffffffu, acc[h][i].x, 16);
            acc[h][i].y += __shfl_xor_sync(0xffffffffu, acc[h][i].y, 16);
          }
      }
#pragma unroll
      for (int n = 0; n < HC; n += 4) {  // four heads at a time
        if (TP == 1 || lane < 16)
#pragma unroll
          for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int j = 0; j < PL; ++j)
              *reinterpret_cast<float4*>(s_sum + (warp * 4 + h) * G::kPitch + (lane + 32 * j) * 4) =
                  make_float4(acc[n + h][2 * j].x, acc[n + h][2 * j].y, acc[n + h][2 * j + 1].x, acc[n + h][2 * j + 1].y);
        if (wt > 1) __syncthreads();
        else __syncwarp();
        // the warps of a head take its four query heads' columns in turn
        for (int i = my_tile * 32 + lane; i < 4 * DM; i += wt * 32) {
          const int h = i / DM, d = i % DM, hn = n + h;
          if (g0 + hn >= GQ) break;
          float top = -INFINITY, sum = 0.0f, v = 0.0f;
          for (int w = my_head; w < kWarps; w += wh) top = fmaxf(top, s_ml[w * HC + hn].x);
          const float mm = top == -INFINITY ? 0.0f : top;
          for (int w = my_head; w < kWarps; w += wh) {
            const float2 ml = s_ml[w * HC + hn];
            const float f = exp2_fast(ml.x - mm);
            sum += ml.y * f;
            v += s_sum[(w * 4 + h) * G::kPitch + d] * f;
          }
          const int64_t hq = static_cast<int64_t>(hk) * GQ + g0 + hn;
          if (d < a.D) {
            if (whole) static_cast<float*>(a.o)[seq * a.o_s + hq * a.o_h + d] = paged_mean<float>(v, sum);
            else part[hn * stride + d] = v;
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
      tile0 = use.tile;
      clear_sums();
    }
    copies_wait<0>();
  } else {
    paged_empty<float>(a);
  }
  if (threadIdx.x == 0) a.rec[blockIdx.x] = rec;
}

template <int DM, int HC>
cudaError_t launch(const PagedArgs& a, int sms, cudaStream_t s) {
  using G = Geo<DM, HC>;
  static SmemLimit limit;
  static_assert(G::kSmem <= (G::kCtas == 1 ? 227 : 113) * 1024, "shared memory");
  auto kern = paged_f32_kernel<DM, HC>;
  if (cudaError_t e = limit.allow(kern, G::kSmem)) return e;
  const PagedShape p = paged_shape_f32(a.Hq / a.Hk, a.Hk, a.D, a.k_head < a.k_token);
  const int ctas = p.ctas * sms;
  if (cudaError_t e = launch_early(kern, dim3(static_cast<unsigned>(ctas)), G::kThreads, G::kSmem, s, a, p.groups, log2_of(p.wh))) return e;
  return launch_paged_join<float>(a, ctas, HC, p.groups, p.wh, s);
}

}  // namespace

PagedShape paged_shape_f32(int G, int Hk, int D, bool together) {
  return paged_shape(G, Hk, G > 4 ? 8 : 4, D <= 128 ? 8 : 4, D <= 64 ? 2 : 1, together);
}

// D a multiple of 4, all rows 16-byte aligned.
cudaError_t launch_paged_f32(const PagedArgs& a, int sms, cudaStream_t s) {
  const bool wide = a.Hq / a.Hk > 4;
  if (a.D <= 64) return wide ? launch<64, 8>(a, sms, s) : launch<64, 4>(a, sms, s);
  if (a.D <= 128) return wide ? launch<128, 8>(a, sms, s) : launch<128, 4>(a, sms, s);
  return wide ? launch<256, 8>(a, sms, s) : launch<256, 4>(a, sms, s);
}

}  // namespace nf4
