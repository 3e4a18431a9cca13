// kv4_attention.cu -- affinity_kv4_attention: causal softmax attention over a paged cache held in 4 bits (kv4.cuh), for
// a batch whose sequences share a prefix.  Formulas, rows, key tiles, items and the join are those of attention.cu and
// step.cuh.
//
// What the cache holds is exact in fp16, so both products run on fp16 operands:
//   queries       q 2^-e, e for each row and head so that its largest element is in [2^13, 2^14): a bf16 number keeps
//                 its 8 bits unless it is 2^27 below that element.  The scores' factor is scale k_scale 2^e.
//   probabilities exp(s - m) 2^7, m the running maximum: 11 bits (the 16-bit cache's are rounded to bf16's 8), and
//                 nothing above 2^-31 is lost.
// fp32 queries and probabilities are the sum of two fp16 numbers each, 22 bits, and two products.
#include "affinity.h"
#include "internal.h"
#include "kv4.cuh"
#include "launch.cuh"
#include "sm103_primitives.cuh"
#include "step.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

namespace aff {
namespace {

constexpr float kRescale = 8.f;              // log2 growth of the maximum that O is rescaled for
constexpr float kShift = 7.f;                // log2 of the probabilities' factor: they stay below 2^15
constexpr float kLn2 = 0.69314718055994531f;
constexpr uint32_t kStatusInvalid = 1;

struct Kv4AttnParams {
  StepGeom g;
  Kv4Pool pool;
  const void* q;
  int64_t q_stride;
  void* out;
  float* lse;               // [T][H] or null
  float score_log2;         // scale k_scale log2(e)
  float v_scale;
};

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 halves(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit elements, two to a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ WorkItem load_item(const WorkItem* p) {
  WorkItem it;
  const int4* s = reinterpret_cast<const int4*>(p);
  int4* d = reinterpret_cast<int4*>(&it);
  d[0] = s[0];
  d[1] = s[1];
  d[2] = s[2];
  return it;
}
// The factor of a row of queries (its largest magnitude, as bits) and the inverse, both powers of two.
__device__ __forceinline__ float query_factor(uint32_t top, float* inverse) {
  int e = (int)(top >> 23);
  if (e == 255) e = 127 + 13;                 // infinite or NaN: as it is
  const int up = min(127 + 13 - e, 126);      // a row of zeros or subnormals: 2^126
  *inverse = __uint_as_float((uint32_t)(127 - up) << 23);
  return __uint_as_float((uint32_t)(127 + up) << 23);
}

// ---------------------------------------------------------------- few rows
// Items of at most 8 rows, bound by the bytes of the cache.  Eight warps share an item: 16 keys at a time are a warp's
// unit, straight from global memory to the registers of the products that read them, and nothing is exchanged before
// the item's end.  Products are transposed, keys as the long side:  S^T = K Q^T and O^T += V^T P^T.
//   K  lane (key quad, c) holds its key's elements 8 W c .. + 8 W - 1 as they lie in memory (W words of codes); the
//      contraction does not care which elements are a slice's, so the queries are dealt the same way.
//   V  lane (quad, c) holds elements 4 W quad .. of keys 4 c .. 4 c + 3; a byte of two keys' codes for the same
//      element makes the pair that V^T wants, two shifts and two selections for 16 elements.
// Rows of S^T are dealt to keys so that a lane's four probabilities' keys are those it holds the values of.
constexpr int kFewThreads = 256;
constexpr int kFewPitch = 132;               // floats of a staged row

template <int NC>
struct FewShape {
  static constexpr int W = NC >= 3 ? 4 : NC;           // words of codes a lane holds of a key
  static constexpr int VW = W == 4 ? 2 : 1;            // of a value (W == 1: half a word)
};

template <int NC>
struct FewRaw {                              // a unit as it lies in memory
  static constexpr int W = FewShape<NC>::W, VW = FewShape<NC>::VW;
  uint32_t k[2][W], ks[W == 4 ? 2 : 1], v[4][VW], vs;
};

struct FewUnit {
  int tile, sub;                             // of the walk
  int key0, keys;                            // first key within the segment, keys (at most 16); 0: past the end
  bool pre;
  int page, in_page;                         // of the four keys that this lane holds the values of; page -1: none
};

template <int NC, bool F32>
__global__ void __launch_bounds__(kFewThreads, 2) kv4_few_kernel(const __grid_constant__ Kv4AttnParams p) {
  constexpr int W = FewShape<NC>::W, VW = FewShape<NC>::VW, KS = 2 * W, MT = 2 * W;
  __shared__ __align__(16) float po[8][8][kFewPitch];
  __shared__ float2 ml[8][8];
  __shared__ int nan_key[2][8];              // the first key, not seen by every row, whose values of a block are NaN
  __shared__ int claim;
  pdl_enter();
  const StepGeom& g = p.g;
  const bool fits = plan_matches(g);
  const int n_items = fits ? g.head->n_items : 0;
  if ((!fits || n_items < 0) && threadIdx.x == 0) latch_status(&g.head->status, fits ? kStatusRange : kStatusInvalid);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane >> 2, c = lane & 3;
  const int k_off = (quad >> 1) * 4 + (quad & 1);          // this lane's keys of a unit: k_off, k_off + 2
  const bool k0_has = 8 * W * c < g.d, k1_has = W == 4 && 8 * W * c + 16 < g.d;      // blocks of this lane's key elements
  const bool v_has = 4 * W * quad < g.d;
  const int v_block = 4 * W * quad / 16;
  const int subs = (g.key_tile + 15) / 16;
  if (threadIdx.x < 8) nan_key[0][threadIdx.x] = INT32_MAX;
  int turn = 0;

  for (int i = blockIdx.x; i < n_items; i = claim) {
    const WorkItem it = load_item(g.items + i);
    const int n = it.alt == 1 ? it.n0 + it.n1 : it.alt == 2 ? it.n0 : it.n1;
    for (int r0 = 0; r0 < it.nrows; r0 += 8, turn ^= 1) {
      const int nrows = min(it.nrows - r0, 8), row0 = it.row0 + r0;
      __syncthreads();                       // what lies in shared memory has been read
      if (threadIdx.x == 0 && r0 == 0) claim = gridDim.x + (int)atomicAdd(&g.head->few_claimed, 1u);
      if (threadIdx.x < 8) nan_key[turn ^ 1][threadIdx.x] = INT32_MAX;

      // ---- queries: B operand of S^T, row quad
      uint32_t qh[KS][2], ql[F32 ? KS : 1][2];
      float inverse;
      {
        const int rr = row0 + quad, tok = g.by_R(rr);
        const int64_t at = (int64_t)tok * p.q_stride + (it.group * g.R + rr - tok * g.R) * g.d;
        float x[8 * W];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const int e0 = 8 * W * c + 8 * j;
          const bool has = quad < nrows && e0 < g.d;
          if constexpr (F32) {
            const float* src = static_cast<const float*>(p.q) + at + e0;
            const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
            const float4 a = has ? __ldg(reinterpret_cast<const float4*>(src)) : z;
            const float4 b = has ? __ldg(reinterpret_cast<const float4*>(src) + 1) : z;
            x[8 * j] = a.x; x[8 * j + 1] = a.y; x[8 * j + 2] = a.z; x[8 * j + 3] = a.w;
            x[8 * j + 4] = b.x; x[8 * j + 5] = b.y; x[8 * j + 6] = b.z; x[8 * j + 7] = b.w;
          } else {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (has) w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at + e0));
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              x[8 * j + 2 * y] = __uint_as_float(u[y] << 16);
              x[8 * j + 2 * y + 1] = __uint_as_float(u[y] & 0xffff0000u);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 8 * W; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float f = query_factor(top, &inverse);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float a = x[4 * s + 2 * h] * f, b = x[4 * s + 2 * h + 1] * f;
            qh[s][h] = f16x2(a, b);
            if constexpr (F32) {
              const float2 r = halves(qh[s][h]);
              ql[s][h] = f16x2(a - r.x, b - r.y);
            }
          }
      }
      // rows 2 c and 2 c + 1: the scores' factor, own keys in view, maximum (log2) that O and l refer to, sum
      float sc[2], m[2], l[2], o[MT][4];
      int own_vis[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 2 * c + e;
        sc[e] = __shfl_sync(0xffffffffu, inverse, r * 4) * p.score_log2;
        own_vis[e] = r >= nrows ? 0 : it.seq < 0 ? INT32_MAX : g.by_R(row0 + r) + it.own_off + 1;
        m[e] = -INFINITY;
        l[e] = 0.f;
      }
      const int all_see = it.seq < 0 ? INT32_MAX : g.by_R(row0) + it.own_off + 1;    // own keys that every row sees
#pragma unroll
      for (int t = 0; t < MT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;

      // ---- the walk over this warp's units
      const uint8_t* const kg = p.pool.k + it.group * p.pool.group_stride;
      const uint8_t* const vg = p.pool.v + it.group * p.pool.group_stride;
      const int end = it.t0 + n;
      auto locate = [&](FewUnit& u) {        // the unit at (tile, sub) or the next one that holds a key; asks for its page
        u.keys = 0;
        u.page = -1;
        while (u.tile < end) {
          u.pre = u.tile < it.np;
          int first;
          const int keys = tile_span(g, u.pre ? g.prefix_len : it.own_len, u.pre ? u.tile : u.tile - it.np, &first) - 16 * u.sub;
          u.key0 = first + 16 * u.sub;
          u.sub += 8;
          while (u.sub >= subs) {
            u.sub -= subs;
            ++u.tile;
          }
          if (keys > 0) {
            u.keys = min(keys, 16);
            break;
          }
        }
        if (4 * c < u.keys) {
          const int32_t* table = u.pre ? g.prefix_pages : g.pages + (int64_t)it.seq * g.pages_stride;
          const int pi = g.by_page(u.key0 + 4 * c);
          u.page = __ldg(table + pi);
          u.in_page = u.key0 + 4 * c - pi * g.page_size;
        }
      };
      auto load = [&](FewRaw<NC>& r, FewUnit& u) {
        if (4 * c < u.keys && (u.page < 0 || u.page >= g.n_pages)) {      // read as zeros: report it
          latch_status(&g.head->status, kStatusRange);
          u.page = -1;
        }
        const int kp = __shfl_sync(0xffffffffu, u.page, quad >> 1), ki = __shfl_sync(0xffffffffu, u.in_page, quad >> 1);
#pragma unroll
        for (int x = 0; x < W; ++x) r.k[0][x] = r.k[1][x] = 0;
#pragma unroll
        for (int x = 0; x < (W == 4 ? 2 : 1); ++x) r.ks[x] = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int y = 0; y < VW; ++y) r.v[x][y] = 0;
        r.vs = 0;
        if (kp >= 0 && k0_has) {
          const uint8_t* page = kg + kp * p.pool.page_stride;
          const uint8_t* at = page + (ki + (quad & 1)) * 16 * p.pool.n + c * 4 * W;
          const uint8_t* s = page + p.pool.scales + ((ki >> 2) * 2 * p.pool.n + (W == 4 ? 2 * c : W == 2 ? c : c >> 1)) * 4;
#pragma unroll
          for (int x = 0; x < 2; ++x, at += 32 * p.pool.n) {
            if constexpr (W == 4) {
              const uint4 w = __ldg(reinterpret_cast<const uint4*>(at));
              r.k[x][0] = w.x; r.k[x][1] = w.y; r.k[x][2] = w.z; r.k[x][3] = w.w;
            } else if constexpr (W == 2) {
              const uint2 w = __ldg(reinterpret_cast<const uint2*>(at));
              r.k[x][0] = w.x; r.k[x][1] = w.y;
            } else {
              r.k[x][0] = __ldg(reinterpret_cast<const uint32_t*>(at));
            }
          }
          if constexpr (W == 4) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(s));
            r.ks[0] = w.x;
            r.ks[1] = k1_has ? w.y : 0;
          } else {
            r.ks[0] = __ldg(reinterpret_cast<const uint32_t*>(s));
          }
        }
        if (u.page >= 0 && v_has) {
          const uint8_t* page = vg + u.page * p.pool.page_stride;
          const uint8_t* at = page + u.in_page * 16 * p.pool.n + quad * 2 * W;
#pragma unroll
          for (int x = 0; x < 4; ++x, at += 16 * p.pool.n) {
            if constexpr (W == 4) {
              const uint2 w = __ldg(reinterpret_cast<const uint2*>(at));
              r.v[x][0] = w.x; r.v[x][1] = w.y;
            } else if constexpr (W == 2) {
              r.v[x][0] = __ldg(reinterpret_cast<const uint32_t*>(at));
            } else {
              r.v[x][0] = __ldg(reinterpret_cast<const uint16_t*>(at));
            }
          }
          r.vs = __ldg(reinterpret_cast<const uint32_t*>(page + p.pool.scales + ((u.in_page >> 2) * 2 * p.pool.n + v_block) * 4));
          const int left = u.keys - 4 * c;
          if (left < 4) r.vs &= (1u << 8 * left) - 1;       // keys past the end: zero
        }
      };
      auto work = [&](const FewRaw<NC>& r, const FewUnit& u) {
        // ---- scores
        uint32_t ka[2], kb[2];               // scales of this lane's blocks, twice, of either key
        if constexpr (W == 4) {
          const uint32_t b = quad & 1;
          const uint32_t a2 = kv4_scale_pair(prmt(r.ks[0], r.ks[1], b | (4 + b) << 4));
          const uint32_t b2 = kv4_scale_pair(prmt(r.ks[0], r.ks[1], (b + 2) | (b + 6) << 4));
          ka[0] = prmt(a2, a2, 0x1010); ka[1] = prmt(a2, a2, 0x3232);
          kb[0] = prmt(b2, b2, 0x1010); kb[1] = prmt(b2, b2, 0x3232);
        } else {
          const uint32_t b = quad & 1;
          const uint32_t two = kv4_scale_pair(prmt(r.ks[0], 0, b | (b + 2) << 4));
          ka[0] = ka[1] = prmt(two, two, 0x1010);
          kb[0] = kb[1] = prmt(two, two, 0x3232);
        }
        float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < W; ++w) {
          uint32_t a[4], b[4];
          kv4_decode(r.k[0][w], a);
          kv4_decode(r.k[1][w], b);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] = mul_f16x2(a[e], ka[w >> 1]);
            b[e] = mul_f16x2(b[e], kb[w >> 1]);
          }
          mma_16x8x16(s, a[0], b[0], a[1], b[1], qh[2 * w][0], qh[2 * w][1]);
          mma_16x8x16(s2, a[2], b[2], a[3], b[3], qh[2 * w + 1][0], qh[2 * w + 1][1]);
          if constexpr (F32) {
            mma_16x8x16(s, a[0], b[0], a[1], b[1], ql[2 * w][0], ql[2 * w][1]);
            mma_16x8x16(s2, a[2], b[2], a[3], b[3], ql[2 * w + 1][0], ql[2 * w + 1][1]);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += s2[e];
        // ---- s[e]: key k_off, row 2 c + e; s[2 + e]: key k_off + 2
        if (!(u.keys == 16 && all_see > 0 && (u.pre || u.key0 + 16 <= all_see))) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int vis = own_vis[e] <= 0 ? 0 : u.pre ? u.keys : min(u.keys, own_vis[e] - u.key0);
            if (k_off >= vis) s[e] = -INFINITY;          // chosen, not added: a NaN behind the mask is gone
            if (k_off + 2 >= vis) s[2 + e] = -INFINITY;
          }
        }
        bool grow = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) grow |= fmaxf(s[e], s[2 + e]) * sc[e] - m[e] > kRescale;
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(s[e], s[2 + e]) * sc[e];
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float f = mx > m[e] ? ex2(m[e] - mx) : 1.f;
            m[e] = fmaxf(m[e], mx);
            l[e] *= f;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              o[t][e] *= f;
              o[t][2 + e] *= f;
            }
          }
        }
        float x[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float neg = m[e] == -INFINITY ? kShift : kShift - m[e];
          x[e] = ex2(fmaf(s[e], sc[e], neg));
          x[2 + e] = ex2(fmaf(s[2 + e], sc[e], neg));
          l[e] += x[e] + x[2 + e];
        }
        // keys x rows -> rows x keys, the B operand of O^T
        const uint32_t p0 = f16x2(x[0], x[1]), p1 = f16x2(x[2], x[3]);
        const uint32_t ph0 = transpose8(p0), ph1 = transpose8(p1);
        uint32_t pl0 = 0, pl1 = 0;
        if constexpr (F32) {
          const float2 r0 = halves(p0), r1 = halves(p1);
          pl0 = transpose8(f16x2(x[0] - r0.x, x[1] - r0.y));
          pl1 = transpose8(f16x2(x[2] - r1.x, x[3] - r1.y));
        }
        // ---- values
        uint32_t vs = r.vs;
        const uint32_t odd = kv4_nan_scales(vs);
        if (__any_sync(0xffffffffu, odd)) {              // rare: NaN values that some row does not see are taken out
#pragma unroll 1
          for (int x = 0; x < 4; ++x) {
            const int key = u.key0 + 4 * c + x;
            if (!u.pre && (odd >> (8 * x + 7) & 1u) && key >= all_see) {
              vs &= ~(0xffu << 8 * x);
              atomicMin(&nan_key[turn][v_block], key);
            }
          }
        }
        const uint32_t v01 = kv4_scale_pair(vs), v23 = kv4_scale_pair(vs >> 16);
#pragma unroll
        for (int j = 0; j < VW; ++j) {
          uint32_t a0[4], a1[4], a2[4], a3[4];           // elements 2 b, 2 b + 1 of keys 0, 1; of keys 2, 3
          constexpr uint32_t lo = 0x0f0f0f0fu;
          kv4_decode((r.v[0][j] & lo) | ((r.v[1][j] << 4) & ~lo), a0);
          kv4_decode(((r.v[0][j] >> 4) & lo) | (r.v[1][j] & ~lo), a1);
          kv4_decode((r.v[2][j] & lo) | ((r.v[3][j] << 4) & ~lo), a2);
          kv4_decode(((r.v[2][j] >> 4) & lo) | (r.v[3][j] & ~lo), a3);
#pragma unroll
          for (int b = 0; b < (W == 1 ? 2 : 4); ++b) {
            const int t = 4 * j + b;
            const uint32_t w0 = mul_f16x2(a0[b], v01), w1 = mul_f16x2(a1[b], v01), w2 = mul_f16x2(a2[b], v23),
                           w3 = mul_f16x2(a3[b], v23);
            if constexpr (F32) {
              // summed apart: the products' own accumulation cuts bits off, which would add up over long keys
              float z[4] = {0.f, 0.f, 0.f, 0.f};
              mma_16x8x16(z, w0, w1, w2, w3, pl0, pl1);
              mma_16x8x16(z, w0, w1, w2, w3, ph0, ph1);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[t][e] += z[e];
            } else {
              mma_16x8x16(o[t], w0, w1, w2, w3, ph0, ph1);
            }
          }
        }
      };
      FewUnit ua{it.t0, warp, 0, 0, false, -1, 0}, ub;
      while (ua.sub >= subs) {
        ua.sub -= subs;
        ++ua.tile;
      }
      FewRaw<NC> ra, rb;
      locate(ua);
      load(ra, ua);
      ub = ua;
      locate(ub);
      while (ua.keys > 0) {
        load(rb, ub);
        FewUnit next = ub;
        locate(next);
        work(ra, ua);
        ua = next;
        load(ra, ua);
        if (ub.keys > 0) {
          next = ua;
          locate(next);
          work(rb, ub);
          ub = next;
        }
      }

      // ---- the warps' parts
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], x);
        const int r = 2 * c + e;
        if (r >= nrows) continue;
        if (quad == 0) ml[warp][r] = make_float2(m[e], l[e]);
        float* dst = &po[warp][r][4 * W * quad];
#pragma unroll
        for (int t = 0; t < MT; t += 2)
          *reinterpret_cast<float4*>(dst + 2 * t) = make_float4(o[t][e], o[t][2 + e], o[t + 1][e], o[t + 1][2 + e]);
      }
      __syncthreads();
      const int r = warp, e0 = 4 * lane;
      if (r < nrows) {
        const int rr = row0 + r, tok = g.by_R(rr), h = it.group * g.R + rr - tok * g.R;
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) top = fmaxf(top, ml[w][r].x);
        const float ref = top == -INFINITY ? 0.f : top;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const float2 s = ml[w][r];
          if (s.y == 0.f) continue;                      // nothing seen by this warp
          const float f = s.x == -INFINITY ? 1.f : ex2(s.x - ref);
          sum += f * s.y;
          const float4 v = *reinterpret_cast<const float4*>(&po[w][r][min(e0, 4 * W * 8 - 4)]);
          acc.x += f * v.x;
          acc.y += f * v.y;
          acc.z += f * v.z;
          acc.w += f * v.w;
        }
        const float inv = sum == 0.f ? 0.f : p.v_scale / sum;
        acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (sum == 0.f) acc = make_float4(0.f, 0.f, 0.f, 0.f);
        const int vis = it.seq < 0 ? 0 : tok + it.own_off + 1;
        if (e0 < g.d) {
          if (nan_key[turn][e0 / 16] < vis) acc.x = acc.y = acc.z = acc.w = __int_as_float(0x7fc00000);
          if (it.part_row >= 0) {
            *reinterpret_cast<float4*>(g.part_out + (int64_t)(it.part_row + r0 + r) * g.d + e0) = acc;
          } else if constexpr (F32) {
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + ((int64_t)tok * g.H + h) * g.d + e0) = acc;
          } else {
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + ((int64_t)tok * g.H + h) * g.d + e0) =
                make_uint2(bf16x2(acc.x, acc.y), bf16x2(acc.z, acc.w));
          }
        }
        if (lane == 0) {
          const float lse = sum == 0.f ? -INFINITY : (ref - kShift) * kLn2 + logf(sum);
          if (it.part_row >= 0) g.part_lse[it.part_row + r0 + r] = lse;
          else if (p.lse) p.lse[(int64_t)tok * g.H + h] = lse;
        }
      }
    }
  }
  // every claim of this CTA has been made: the last one leaves the counters as the next call needs them
  if (fits && threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(&g.head->few_done, 1u) == gridDim.x - 1) {
      g.head->few_claimed = 0;
      g.head->few_done = 0;
    }
  }
}

template <int NC>
aff_status launch_few(const Kv4AttnParams& p, unsigned grid, cudaStream_t s) {
  if (p.g.dtype == AFF_BF16) AFF_CUDA(launch_pdl(kv4_few_kernel<NC, false>, grid, kFewThreads, 0, s, p));
  else AFF_CUDA(launch_pdl(kv4_few_kernel<NC, true>, grid, kFewThreads, 0, s, p));
  return AFF_OK;
}

}  // namespace
}  // namespace aff

using namespace aff;

extern "C" aff_status affinity_kv4_attention(const void* q, int64_t q_stride, const aff_kv4_cache* cache,
                                             const aff_step* step, float scale, void* out, float* lse, void* plan,
                                             size_t plan_bytes, aff_stream_t stream) {
  Kv4AttnParams p{};
  aff_status st = kv4_geom(step, cache, plan, &p.g);
  if (st != AFF_OK) return st;
  const StepGeom& g = p.g;
  if (!q || !out || q_stride < (int64_t)g.H * g.d) return AFF_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return AFF_ERR_INVALID_ARG;
  if (g.d > 128) return AFF_ERR_UNSUPPORTED_SHAPE;
  const int es = g.dtype == AFF_BF16 ? 2 : 4;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15u || q_stride * es % 16 ||
      reinterpret_cast<uintptr_t>(lse) & 3u)
    return AFF_ERR_ALIGNMENT;
  if ((st = check_plan(g, plan, plan_bytes)) != AFF_OK) return st;
  int sms = 0;
  if ((st = check_device(&sms)) != AFF_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  p.pool = kv4_pool(cache);
  p.q = q;
  p.q_stride = q_stride;
  p.out = out;
  p.lse = lse;
  p.score_log2 = scale * 1.4426950408889634f * cache->k_scale;
  p.v_scale = cache->v_scale;
  const unsigned few_grid = (unsigned)(g.max_items < 2 * sms ? g.max_items : 2 * sms);
  switch (p.pool.n) {
    case 1: st = launch_few<1>(p, few_grid, s); break;
    case 2: st = launch_few<2>(p, few_grid, s); break;
    case 3: st = launch_few<3>(p, few_grid, s); break;
    default: st = launch_few<4>(p, few_grid, s); break;
  }
  if (st != AFF_OK) return st;
  return g.may_split ? launch_join(g, out, lse, s) : AFF_OK;
}
