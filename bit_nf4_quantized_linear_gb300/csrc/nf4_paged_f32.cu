// nf4_paged_f32.cu -- attention of one query token a sequence over the paged cache in fp32
// (nf4_paged_attention): rows of whole 16-byte pieces, up to 128 values.
//
// The arithmetic is fp32 on the ordinary cores, 4 D operations a query head and token against
// 8 D bytes a key head and token: up to a group of some eight heads HBM bounds it, if the rows
// come in time and few instructions move them about.  They stream through per-warp rings as in
// the tensor-core kernel (paged_ring.cuh), 8 tokens a warp's tile.  Scores: a lane takes one
// token and a quarter of its columns; every 16 bytes of a key meet 16 of each head's query
// (a broadcast); the quarters are added so that a quarter's lanes end with its heads.  Sums: a
// lane takes 16 bytes of columns of all tokens, the weights come back through shared memory.
// Packed fp32 pairs halve the multiply-adds.
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

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = kPagedTile / kWarps;  // tokens of a warp's tile
static_assert(kRows == 8, "a lane a token and quarter");

template <int DM, int HC>
struct Geo {
  static constexpr int kStages = 3;
  static constexpr int kCtas = DM == 64 ? 2 : 1;  // a SM
  static constexpr int kPitch = DM + 4;           // floats between heads of a warp's sums
  static constexpr int kRing = kWarps * kStages * TileCopies<float, DM, kRows>::kStage;
  static constexpr int kSums = kWarps * 4 * kPitch * 4;  // four heads at a time
  static constexpr int kQ = HC * DM * 4;
  static constexpr int kP = kWarps * kRows * HC * 4;
  static constexpr int kMl = kWarps * HC * 8;
  static constexpr int kSmem = kRing + kSums + kQ + kP + kMl + kWarps * kStages * 4;
};

template <int DM, int HC>
__global__ void __launch_bounds__(kThreads, Geo<DM, HC>::kCtas) paged_f32_kernel(PagedArgs a, int groups) {
  using G = Geo<DM, HC>;
  using Copies = TileCopies<float, DM, kRows>;
  constexpr int HL = HC / 4;          // heads of a quarter's lanes
  constexpr int PQ = DM / 16;         // 16-byte pieces of a quarter row
  constexpr int TP = 128 / DM;        // tokens that a warp's read of one piece a lane covers
  extern __shared__ __align__(128) unsigned char dyn[];
  float* s_sum = reinterpret_cast<float*>(dyn + G::kRing);          // [kWarps][4][kPitch]
  float* s_q = reinterpret_cast<float*>(dyn + G::kRing + G::kSums); // [HC][DM]
  float* s_p = s_q + HC * DM;                                       // [kWarps][kRows][HC]
  float2* s_ml = reinterpret_cast<float2*>(s_p + kWarps * kRows * HC);  // [kWarps][HC]
  uint32_t* s_valid = reinterpret_cast<uint32_t*>(s_ml + kWarps * HC);  // [kWarps][kStages]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned char* ring = dyn + warp * G::kStages * Copies::kStage;
  s_p += warp * kRows * HC;
  s_valid += warp * G::kStages;
  grid_allow();
  grid_wait();
  const int heads = a.Hk * groups, GQ = a.Hq / a.Hk;
  const PagedRun run = paged_run(a, heads, reinterpret_cast<int64_t*>(s_sum));
  PagedRec rec{0, 0, 0};

  if (run.u0 < run.u1) {
    Walk load(a, run, heads);
    Walk use = load;
    const Copies copies(a, nf4ptx::smem_addr(ring), s_valid, groups);
#pragma unroll
    for (int i = 0; i < G::kStages; ++i) {
      copies.start(a, load, load.tile * kPagedTile + warp * kRows, i);
      if (load.left > 0) load.next(a, heads);
    }
    auto fetch_queries = [&]() {
      const int hk = groups == 1 ? use.head : use.head / groups, g0 = (use.head - hk * groups) * HC;
      const float* q = static_cast<const float*>(a.q) + use.seq * a.q_s + (static_cast<int64_t>(hk) * GQ + g0) * a.q_h;
      for (int i = threadIdx.x; i < HC * DM; i += kThreads) {
        const int h = i / DM, d = i % DM;
        s_q[i] = g0 + h < GQ && d < a.D ? q[h * a.q_h + d] : 0.0f;
      }
    };
    // lane (t, r): token t = lane % 8; as quarter r = lane / 8 it keeps heads r HL .. r HL + HL - 1
    const int t = lane & 7, r = lane >> 3;
    float2 acc[HC][2];
    float m[HL], l[HL];
    auto clear_sums = [&]() {
#pragma unroll
      for (int h = 0; h < HC; ++h) acc[h][0] = acc[h][1] = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int j = 0; j < HL; ++j) {
        m[j] = -INFINITY;
        l[j] = 0.0f;
      }
    };
    const float c = a.scale * kLog2e;
    fetch_queries();
    clear_sums();
    paged_empty<float>(a);
    __syncthreads();
    int st = 0, tile0 = use.tile;  // where the part of this (sequence, head group) begins
    while (use.left > 0) {
      copies_wait<G::kStages - 1>();
      __syncwarp();
      if (use.tile * kPagedTile + warp * kRows < use.len) {
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
          s_p[t * HC + r * HL + j] = p;
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int h = 0; h < HC; ++h) {
            const float f = __shfl_sync(0xffffffffu, down[h % HL], h / HL * 8);
#pragma unroll
            for (int i = 0; i < 2; ++i) acc[h][i] = mul2(acc[h][i], make_float2(f, f));
          }
        }
        __syncwarp();
        const int piece = lane % (DM / 4), sub = lane / (DM / 4);
#pragma unroll
        for (int i = 0; i < kRows / TP; ++i) {
          const int tok = i * TP + sub;
          const float4 v = *reinterpret_cast<const float4*>(values + at_chunk<DM * 4>(tok, piece));
#pragma unroll
          for (int h = 0; h < HC; h += 4) {
            const float4 p = *reinterpret_cast<const float4*>(s_p + tok * HC + h);
            const float w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              acc[h + j][0] = fma2(make_float2(w[j], w[j]), make_float2(v.x, v.y), acc[h + j][0]);
              acc[h + j][1] = fma2(make_float2(w[j], w[j]), make_float2(v.z, v.w), acc[h + j][1]);
            }
          }
        }
      }
      __syncwarp();
      copies.start(a, load, load.tile * kPagedTile + warp * kRows, st);
      if (load.left > 0) load.next(a, heads);
      st = st + 1 == G::kStages ? 0 : st + 1;

      const bool ends = use.tile + 1 == use.tiles;
      if (!ends && use.left > 1) {
        use.next(a, heads);
        continue;
      }
      // The part of this (sequence, head group) is done: add the warps' sums, four heads at a time.
      const Walk was = use;
      use.next(a, heads);
      const int hk = groups == 1 ? was.head : was.head / groups, g0 = (was.head - hk * groups) * HC;
      const bool whole = ends && tile0 == 0;
      const int stride = paged_part_stride(a.D);
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
      for (int n = 0; n < HC; n += 4) {
        if (lane < DM / 4)
#pragma unroll
          for (int h = 0; h < 4; ++h)
            *reinterpret_cast<float4*>(s_sum + (warp * 4 + h) * G::kPitch + lane * 4) =
                make_float4(acc[n + h][0].x, acc[n + h][0].y, acc[n + h][1].x, acc[n + h][1].y);
        __syncthreads();
        if (n == 0 && use.left > 0) fetch_queries();
        const int h = threadIdx.x >> 6, hn = n + h;  // 64 threads a head
        if (g0 + hn < GQ) {
          float top = -INFINITY, sum = 0.0f, f[kWarps];
#pragma unroll
          for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w * HC + hn].x);
          const float mm = top == -INFINITY ? 0.0f : top;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 ml = s_ml[w * HC + hn];
            f[w] = exp2_fast(ml.x - mm);
            sum += ml.y * f[w];
          }
          const int64_t hq = static_cast<int64_t>(hk) * GQ + g0 + hn;
          float* o = static_cast<float*>(a.o) + was.seq * a.o_s + hq * a.o_h;
          float* part = a.part + (static_cast<int64_t>(blockIdx.x * 2 + (tile0 == 0)) * HC + hn) * stride;
          for (int d = threadIdx.x & 63; d < a.D; d += 64) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += s_sum[(w * 4 + h) * G::kPitch + d] * f[w];
            if (whole) o[d] = v / sum;
            else part[d] = v;
          }
          if ((threadIdx.x & 63) == 0) {
            if (whole) {
              if (a.lse) a.lse[was.seq * a.Hq + hq] = top * kLn2 + logf(sum);
            } else {
              part[stride - 4] = top;
              part[stride - 3] = sum;
            }
          }
        }
        __syncthreads();
      }
      if (tile0 > 0) rec.flags |= ends ? 6 : 2;
      if (tile0 == 0 && !ends) {
        rec.flags |= 1;
        rec.seq = was.seq;
        rec.head = was.head;
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
  static_assert(G::kCtas * 2 * HC <= kPagedSlots && G::kCtas <= kPagedCtas, "workspace");
  static_assert(G::kSmem <= (G::kCtas == 1 ? 227 : 113) * 1024, "shared memory");
  auto kern = paged_f32_kernel<DM, HC>;
  if (cudaError_t e = limit.allow(kern, G::kSmem)) return e;
  const int groups = (a.Hq / a.Hk + HC - 1) / HC, ctas = G::kCtas * sms;
  if (cudaError_t e = launch_early(kern, dim3(static_cast<unsigned>(ctas)), kThreads, G::kSmem, s, a, groups)) return e;
  return launch_paged_join<float>(a, ctas, HC, groups, s);
}

}  // namespace

// D a multiple of 4 up to 128, all rows 16-byte aligned.
cudaError_t launch_paged_f32(const PagedArgs& a, int sms, cudaStream_t s) {
  const bool wide = a.Hq / a.Hk > 4;
  if (a.D <= 64) return wide ? launch<64, 8>(a, sms, s) : launch<64, 4>(a, sms, s);
  return wide ? launch<128, 8>(a, sms, s) : launch<128, 4>(a, sms, s);
}

}  // namespace nf4
