// kv_append.cu -- affinity_kv_append: a step's queries, keys and values, once
// over.  Each query and key row (one token, one head) is normalised (optional),
// rotated and written: queries to q_out, keys to their slot of the paged cache;
// value rows are copied to theirs.
//
//   z = row / sqrt(mean(row^2) + eps) * gain           (or z = row)
//   pair (a, b) of z -> (a cos - b sin, a sin + b cos)  at position prefix + own index
//
// Memory bound: T (H + 2G) d elements in and out, nothing reused but the cosine
// and sine row of a token, which its H + G rows share through L1.  A row is held
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
  float eps;
  int32_t rot, interleaved, lanes;
};

template <typename E, int VW>
struct alignas(sizeof(E) * VW) Vec {
  E e[VW];
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

// One row.  Unit u of the row is two runs of VW elements: below rot / 2 units'
// worth they are the two halves of VW pairs (or, interleaved, two neighbouring
// runs whose pairs lie side by side); past rot they are plain neighbours.
template <typename E, int VW>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kUnits = VW >= 4 ? 1 : 4 / VW;   // units a lane can hold: d <= 256 in 32 lanes of 2 VW elements
  pdl_enter();
  const StepGeom& g = p.g;
  const int rows = g.H + 2 * g.G;
  const int64_t at = (int64_t)blockIdx.x * (kThreads / p.lanes) + threadIdx.x / p.lanes;
  const int lane = threadIdx.x & (p.lanes - 1);
  const bool live = at < (int64_t)g.T * rows && plan_matches(g);
  if (at < (int64_t)g.T * rows && !live && threadIdx.x == 0) latch_status(&g.head->status, 1);
  const int t = live ? (int)(at / rows) : 0;
  const int r = live ? (int)(at - (int64_t)t * rows) : 0;
  TokenInfo ti{-1, -1, -1};
  if (live) ti = g.tok[t];
  const bool is_q = r < g.H, is_k = !is_q && r < g.H + g.G;
  const int64_t pos = (int64_t)g.prefix_len + ti.own;
  bool stand = live && ti.own >= 0;              // the token is no padding
  if (stand && (is_q || is_k) && pos >= p.n_pos) {
    stand = false;
    if (lane == 0) latch_status(&g.head->status, kStatusRange);
  }
  const E* src;
  E* dst = nullptr;
  if (is_q) {
    src = static_cast<const E*>(p.q) + (int64_t)t * p.q_stride + (int64_t)r * g.d;
    dst = static_cast<E*>(p.q_out) + (int64_t)t * p.q_out_stride + (int64_t)r * g.d;
  } else {
    const int grp = is_k ? r - g.H : r - g.H - g.G;
    src = is_k ? static_cast<const E*>(p.k) + (int64_t)t * p.k_stride + (int64_t)grp * g.d
               : static_cast<const E*>(p.v) + (int64_t)t * p.v_stride + (int64_t)grp * g.d;
    if (stand) {
      const int64_t page = ti.slot / g.page_size, off = ti.slot - page * g.page_size;
      dst = static_cast<E*>(is_k ? p.kc : p.vc) + page * p.page_stride + grp * p.group_stride + off * p.token_stride;
    }
  }
  const int half = p.rot / 2;
  const int rot_units = (is_q || is_k) ? half / VW : 0;   // VW divides rot / 2 and d - rot (host)
  const int rot_end = (is_q || is_k) ? p.rot : 0;
  using V = Vec<E, VW>;
  float a[kUnits][VW], b[kUnits][VW];
  int ja[kUnits], jb[kUnits];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = lane + i * p.lanes;
    if (u < rot_units) {
      ja[i] = p.interleaved ? 2 * u * VW : u * VW;
      jb[i] = p.interleaved ? ja[i] + VW : ja[i] + half;
    } else {
      ja[i] = rot_end + 2 * (u - rot_units) * VW;
      jb[i] = ja[i] + VW;
    }
    const bool ha = stand && ja[i] < g.d, hb = stand && jb[i] < g.d;
    V va{}, vb{};
    if (ha) va = *reinterpret_cast<const V*>(src + ja[i]);
    if (hb) vb = *reinterpret_cast<const V*>(src + jb[i]);
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      a[i][e] = ha ? to_f(va.e[e]) : 0.f;
      b[i][e] = hb ? to_f(vb.e[e]) : 0.f;
      ss += a[i][e] * a[i][e] + b[i][e] * b[i][e];
    }
  }
  const E* gain = static_cast<const E*>(is_q ? p.q_gain : is_k ? p.k_gain : nullptr);
  // every lane of the warp takes part in the sum
  for (int o = p.lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float inv = gain ? rsqrtf(ss / (float)g.d + p.eps) : 1.f;
  if (!live) return;
  if (!stand && !is_q) return;                   // padding is not stored; its query row is zero
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = lane + i * p.lanes;
    if (ja[i] >= g.d) continue;
    const bool hb = jb[i] < g.d;
    if (gain && stand) {
      const V ga = *reinterpret_cast<const V*>(gain + ja[i]);
      V gb{};
      if (hb) gb = *reinterpret_cast<const V*>(gain + jb[i]);
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        a[i][e] *= inv * to_f(ga.e[e]);
        if (hb) b[i][e] *= inv * to_f(gb.e[e]);
      }
    }
    if (u < rot_units && stand) {
      const float* cs = p.cos + pos * half + (p.interleaved ? u * VW : ja[i]);
      const float* sn = p.sin + pos * half + (p.interleaved ? u * VW : ja[i]);
      float c[VW], s[VW];
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        c[e] = cs[e];
        s[e] = sn[e];
      }
      if (!p.interleaved) {
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          const float x = a[i][e], y = b[i][e];
          a[i][e] = x * c[e] - y * s[e];
          b[i][e] = x * s[e] + y * c[e];
        }
      } else if constexpr (VW > 1) {
        // pairs (2e, 2e + 1) of the 2 VW neighbours: the first VW / 2 in a, the others in b
#pragma unroll
        for (int e = 0; e < VW / 2; ++e) {
          float x = a[i][2 * e], y = a[i][2 * e + 1];
          a[i][2 * e] = x * c[e] - y * s[e];
          a[i][2 * e + 1] = x * s[e] + y * c[e];
          x = b[i][2 * e], y = b[i][2 * e + 1];
          b[i][2 * e] = x * c[e + VW / 2] - y * s[e + VW / 2];
          b[i][2 * e + 1] = x * s[e + VW / 2] + y * c[e + VW / 2];
        }
      } else {
        const float x = a[i][0], y = b[i][0];
        a[i][0] = x * c[0] - y * s[0];
        b[i][0] = x * s[0] + y * c[0];
      }
    }
    V va, vb;
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      from_f(a[i][e], va.e[e]);
      from_f(b[i][e], vb.e[e]);
    }
    *reinterpret_cast<V*>(dst + ja[i]) = va;
    if (hb) *reinterpret_cast<V*>(dst + jb[i]) = vb;
  }
}

template <typename E, int VW>
aff_status launch(AppendParams& p, cudaStream_t s) {
  const int units = (p.g.d + 2 * VW - 1) / (2 * VW);   // the rotated part is whole units, the plain part may end in half a one
  p.lanes = 1;
  while (p.lanes < units && p.lanes < 32) p.lanes *= 2;
  const int64_t rows = (int64_t)p.g.T * (p.g.H + 2 * p.g.G);
  const int64_t per = kThreads / p.lanes;
  AFF_CUDA(launch_pdl(kv_append_kernel<E, VW>, (unsigned)((rows + per - 1) / per), kThreads, 0, s, p));
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
