// kv_append.cu -- affinity_kv_append: a step's queries, keys and values, once
// over.  Each query and key row (one token, one head) is normalised (optional),
// rotated and written: queries to q_out, keys to their slot of the paged cache;
// value rows are copied to theirs.
//
//   z = row / sqrt(mean(row^2) + eps) * gain           (or z = row)
//   pair (a, b) of z -> (a cos - b sin, a sin + b cos)  at position prefix + own index
//
// Memory bound: T (H + 2G) d elements in and out, nothing reused but the cosine
// and sine row of a token, which its H + G rows share through L1.  65536 tokens of
// 16 + 2 x 8 heads of 128 in bf16 with norms: 188 us, 5.7 TB/s, 84 % of the measured
// copy; 22681 ragged tokens of 96-wide fp32 heads: 32 us, 5.4 TB/s; a step of eight
// tokens: 8 us, the launch.  A row is held
// by `lanes` neighbouring lanes (a power of two), each with both halves of its
// pairs, so that the rotation needs no exchange and the norm only a shuffle sum.
#include "affinity.h"
#include "internal.h"
#include "launch.cuh"
#include "sm103_primitives.cuh"
#include "step.cuh"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

namespace aff {
namespace {

constexpr int kThreads = 256;

struct AppendParams {
  StepGeom g;
  const void *q, *k, *v;
  void *q_out, *kc, *vc;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  int64_t page_stride, group_stride, token_stride;
  const float *cos, *sin;
  const void *q_gain, *k_gain;
  int64_t n_pos;
  float eps, inv_d;
  int32_t rot, interleaved, lanes, lane_bits;
};

// VW neighbouring elements as they lie in memory.  bf16 pairs stay whole 32-bit words: taken apart by a shift
// and a mask, put together by one conversion.
template <typename E, int VW>
struct alignas(sizeof(E) * VW) Vec {
  E e[VW];
  __device__ __forceinline__ void get(float (&f)[VW]) const {
#pragma unroll
    for (int i = 0; i < VW; ++i) f[i] = (float)e[i];
  }
  __device__ __forceinline__ void put(const float (&f)[VW]) {
#pragma unroll
    for (int i = 0; i < VW; ++i) e[i] = (E)f[i];
  }
};
template <int VW>
struct alignas(2 * VW) PairVec {
  uint32_t w[VW / 2];
  __device__ __forceinline__ void get(float (&f)[VW]) const {
#pragma unroll
    for (int i = 0; i < VW / 2; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void put(const float (&f)[VW]) {
#pragma unroll
    for (int i = 0; i < VW / 2; ++i)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
  }
};
template <>
struct alignas(4) Vec<__nv_bfloat16, 2> : PairVec<2> {};
template <>
struct alignas(8) Vec<__nv_bfloat16, 4> : PairVec<4> {};
template <>
struct alignas(16) Vec<__nv_bfloat16, 8> : PairVec<8> {};

// Units a lane can hold (d <= 256 in 32 lanes of 2 VW elements) and rows of a thread.
__host__ __device__ constexpr int units_of(int vw) { return vw >= 4 ? 1 : 4 / vw; }
// (65536 tokens of 32 bf16 rows: 248 us with one row a thread, 196 with two, 226 with four; 22681 x 28 fp32
// rows: 35.6, 34.2, 32.3.)
__host__ __device__ constexpr int rows_of(int vw) { return vw == 8 ? 2 : vw == 4 ? 4 : 1; }

__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float z = x * c - y * s;
  y = x * s + y * c;
  x = z;
}

// A run of a row that nothing else reads.
template <typename E, int VW>
__device__ __forceinline__ Vec<E, VW> load_once(const Vec<E, VW>* at) {
  if constexpr (sizeof(Vec<E, VW>) == 16) {
    union {
      uint4 w;
      Vec<E, VW> v;
    } x;
    x.w = __ldcs(reinterpret_cast<const uint4*>(at));
    return x.v;
  } else {
    return *at;
  }
}

// VW neighbouring floats, aligned to VW (up to 4).
template <int VW>
__device__ __forceinline__ void load_row(const float* at, float (&v)[VW]) {
  if constexpr (VW >= 4) {
#pragma unroll
    for (int e = 0; e < VW; e += 4) {
      const float4 w = __ldg(reinterpret_cast<const float4*>(at + e));
      v[e] = w.x; v[e + 1] = w.y; v[e + 2] = w.z; v[e + 3] = w.w;
    }
  } else if constexpr (VW == 2) {
    const float2 w = __ldg(reinterpret_cast<const float2*>(at));
    v[0] = w.x; v[1] = w.y;
  } else {
    v[0] = __ldg(at);
  }
}

// A block is (a part of) one token.  A row is dealt to `lanes` threads, a thread has kPer rows, `slots`
// apart: their loads are all in flight at once, and the token's cosines and sines are read once for them.
// Unit u of a row is two runs of VW elements: of the rotated part the two halves of VW pairs (or,
// interleaved, two neighbouring runs whose pairs lie side by side), past it and in value rows neighbours.
template <typename E, int VW>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kUnits = units_of(VW), kPer = rows_of(VW);
  pdl_enter();
  const StepGeom& g = p.g;
  const int t = blockIdx.x, lane = threadIdx.x & (p.lanes - 1);
  const int slots = blockDim.x >> p.lane_bits;
  const int r0 = blockIdx.y * slots * kPer + (threadIdx.x >> p.lane_bits);
  const int half = p.rot / 2, rot_units = half / VW, n_rot = g.H + g.G, rows = n_rot + g.G;
  using V = Vec<E, VW>;
  // the rows first: they do not depend on where their token stands
  V va[kPer][kUnits], vb[kPer][kUnits];
  auto first_run = [&](int u, bool turned) {
    if (!turned) return 2 * u * VW;
    return u >= rot_units ? p.rot + 2 * (u - rot_units) * VW : p.interleaved ? 2 * u * VW : u * VW;
  };
  auto second_run = [&](int u, int j, bool turned) {
    return turned && u < rot_units && !p.interleaved ? j + half : j + VW;      // VW divides rot / 2 and d - rot (host)
  };
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = r0 + k * slots;
    const E* src = r < g.H   ? static_cast<const E*>(p.q) + (int64_t)t * p.q_stride + r * g.d
                   : r < n_rot ? static_cast<const E*>(p.k) + (int64_t)t * p.k_stride + (r - g.H) * g.d
                               : static_cast<const E*>(p.v) + (int64_t)t * p.v_stride + (r - n_rot) * g.d;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int u = lane + i * p.lanes, ja = first_run(u, r < n_rot), jb = second_run(u, ja, r < n_rot);
      va[k][i] = V{};
      vb[k][i] = V{};
      if (r < rows && ja < g.d) va[k][i] = load_once(reinterpret_cast<const V*>(src + ja));
      if (r < rows && jb < g.d) vb[k][i] = load_once(reinterpret_cast<const V*>(src + jb));
    }
  }
  const TokenInfo ti = g.tok[t];
  const bool fits = plan_matches(g);
  if (!fits || g.head->n_items < 0) {            // a plan of other shapes, or of a malformed step
    if (threadIdx.x == 0) latch_status(&g.head->status, fits ? kStatusRange : 1);
    return;
  }
  if (ti.own == -2 && threadIdx.x == 0) latch_status(&g.head->status, kStatusRange);
  const int64_t pos = (int64_t)g.prefix_len + ti.own;
  bool stand = ti.own >= 0;                      // the token is no padding
  if (stand && pos >= p.n_pos) {
    stand = false;
    if (threadIdx.x == 0) latch_status(&g.head->status, kStatusRange);
  }
  float c[kUnits][VW], s[kUnits][VW];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = lane + i * p.lanes;
    if (stand && u < rot_units) {
      load_row<VW>(p.cos + pos * half + u * VW, c[i]);
      load_row<VW>(p.sin + pos * half + u * VW, s[i]);
    }
  }
  const int64_t at = (ti.slot >> 32) * p.page_stride + (ti.slot & 0xffffffff) * p.token_stride;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = r0 + k * slots;
    const bool is_q = r < g.H, turned = r < n_rot;
    float a[kUnits][VW], b[kUnits][VW], inv = 1.f;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      va[k][i].get(a[i]);
      vb[k][i].get(b[i]);
    }
    const E* gain = static_cast<const E*>(is_q ? p.q_gain : p.k_gain);
    if (p.q_gain || p.k_gain) {
      // every lane of the warp takes part in the sum
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < kUnits; ++i)
#pragma unroll
        for (int e = 0; e < VW; ++e) ss += a[i][e] * a[i][e] + b[i][e] * b[i][e];
      for (int o = p.lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      inv = rsqrtf(ss * p.inv_d + p.eps);
    }
    if (r >= rows || (!stand && !is_q)) continue;      // padding is not stored; its query row is zero
    E* dst = is_q ? static_cast<E*>(p.q_out) + (int64_t)t * p.q_out_stride + r * g.d
                  : static_cast<E*>(turned ? p.kc : p.vc) + at + (turned ? r - g.H : r - n_rot) * p.group_stride;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int u = lane + i * p.lanes, ja = first_run(u, turned), jb = second_run(u, ja, turned);
      if (ja >= g.d) continue;
      const bool hb = jb < g.d;
      V wa = va[k][i], wb = vb[k][i];
      if (!stand) {
        wa = wb = V{};
      } else if (turned) {
        if (gain) {
          const V ga = *reinterpret_cast<const V*>(gain + ja);
          V gb{};
          if (hb) gb = *reinterpret_cast<const V*>(gain + jb);
          float fa[VW], fb[VW];
          ga.get(fa);
          gb.get(fb);
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            a[i][e] *= inv * fa[e];
            b[i][e] *= inv * fb[e];
          }
        }
        if (u < rot_units) {
          if (!p.interleaved) {
#pragma unroll
            for (int e = 0; e < VW; ++e) turn(a[i][e], b[i][e], c[i][e], s[i][e]);
          } else if constexpr (VW > 1) {
            // pairs (2e, 2e + 1) of the 2 VW neighbours: the first VW / 2 in a, the others in b
#pragma unroll
            for (int e = 0; e < VW / 2; ++e) {
              turn(a[i][2 * e], a[i][2 * e + 1], c[i][e], s[i][e]);
              turn(b[i][2 * e], b[i][2 * e + 1], c[i][e + VW / 2], s[i][e + VW / 2]);
            }
          } else {
            turn(a[i][0], b[i][0], c[i][0], s[i][0]);
          }
        }
        wa.put(a[i]);
        wb.put(b[i]);
      }
      *reinterpret_cast<V*>(dst + ja) = wa;
      if (hb) *reinterpret_cast<V*>(dst + jb) = wb;
    }
  }
}

template <typename E, int VW>
aff_status launch(AppendParams& p, cudaStream_t s) {
  const int units = (p.g.d + 2 * VW - 1) / (2 * VW);   // the rotated part is whole units, the plain part may end in half a one
  p.lanes = 1;
  p.lane_bits = 0;
  while (p.lanes < units && p.lanes < 32) {
    p.lanes *= 2;
    ++p.lane_bits;
  }
  p.inv_d = 1.f / (float)p.g.d;
  const int need = (p.g.H + 2 * p.g.G + rows_of(VW) - 1) / rows_of(VW) * p.lanes;
  const int threads = need < kThreads ? (need + 31) / 32 * 32 : kThreads;
  AFF_CUDA(launch_pdl(kv_append_kernel<E, VW>, dim3((unsigned)p.g.T, (unsigned)((need + threads - 1) / threads)), threads, 0,
                      s, p));
  return AFF_OK;
}

}  // namespace
}  // namespace aff

using namespace aff;

extern "C" aff_status affinity_kv_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                         const void* v, int64_t v_stride, const aff_kv_cache* cache,
                                         const aff_step* step, const aff_rotary* rotary, void* q_out,
                                         int64_t q_out_stride, void* plan, size_t plan_bytes, aff_stream_t stream) {
  AppendParams p{};
  aff_status st = step_geom(step, cache, plan, &p.g);
  if (st != AFF_OK) return st;
  if (!q || !k || !v || !q_out || !rotary) return AFF_ERR_INVALID_ARG;
  const StepGeom& g = p.g;
  const int64_t hd = (int64_t)g.H * g.d, gd = (int64_t)g.G * g.d;
  if (q_stride < hd || k_stride < gd || v_stride < gd || q_out_stride < hd) return AFF_ERR_INVALID_ARG;
  if (rotary->rot < 0 || rotary->rot % 2 || rotary->n_pos < 0 || (rotary->rot > 0 && (!rotary->cos || !rotary->sin)) ||
      !(std::isfinite(rotary->eps) && rotary->eps >= 0.f))
    return AFF_ERR_INVALID_ARG;
  if (rotary->rot > g.d) return AFF_ERR_UNSUPPORTED_SHAPE;
  const int es = g.dtype == AFF_BF16 ? 2 : 4;
  const void* ptrs[] = {q, k, v, q_out, rotary->cos, rotary->sin, rotary->q_gain, rotary->k_gain};
  for (const void* x : ptrs)
    if (reinterpret_cast<uintptr_t>(x) & 15u) return AFF_ERR_ALIGNMENT;
  if (q_stride * es % 16 || k_stride * es % 16 || v_stride * es % 16 || q_out_stride * es % 16)
    return AFF_ERR_ALIGNMENT;
  if ((st = check_plan(g, plan, plan_bytes)) != AFF_OK) return st;
  int sms = 0;
  if ((st = check_device(&sms)) != AFF_OK) return st;
  p.q = q; p.k = k; p.v = v; p.q_out = q_out; p.kc = cache->k; p.vc = cache->v;
  p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride; p.q_out_stride = q_out_stride;
  p.page_stride = cache->page_stride; p.group_stride = cache->group_stride; p.token_stride = cache->token_stride;
  p.cos = rotary->cos; p.sin = rotary->sin;
  p.q_gain = rotary->q_gain; p.k_gain = rotary->k_gain;
  p.n_pos = rotary->rot ? rotary->n_pos : INT64_MAX;
  p.eps = rotary->eps;
  p.rot = rotary->rot;
  p.interleaved = rotary->interleaved != 0;
  // the widest run that divides half the rotated part and the plain part
  const int half = p.rot / 2, rest = g.d - p.rot;
  auto fits = [&](int w) { return half % w == 0 && rest % w == 0; };
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (g.dtype == AFF_BF16) {
    if (fits(8)) return launch<__nv_bfloat16, 8>(p, s);
    if (fits(4)) return launch<__nv_bfloat16, 4>(p, s);
    if (fits(2)) return launch<__nv_bfloat16, 2>(p, s);
    return launch<__nv_bfloat16, 1>(p, s);
  }
  if (fits(4)) return launch<float, 4>(p, s);
  if (fits(2)) return launch<float, 2>(p, s);
  return launch<float, 1>(p, s);
}
