// block_norm.cu -- affinity_block_norm: what stands between two blocks of a
// layer, in one pass over the residual stream:
//
//   u = f / rms(f) * post_gain      (or u = f)
//   y = x + scale * gate * u        the new residual
//   h = y / rms(y) * pre_gain       the next block's input (optional)
//   rms(v) = sqrt(mean(v^2) + eps)
//
// Memory bound: x, f (and a gate per token) in, y and h out, each element once;
// the gains and shared gate rows stay in L1/L2.  A row's elements stay in the
// registers of its `group` of threads between the two norms, so nothing is read
// twice; h is normalised from the fp32 sum, not from the rounded y.
// 65536 rows of 1024 bf16: 87 us, 6.2 TB/s, 91 % of the measured copy (fp32: 160 us,
// 6.7 TB/s); rows of odd
// width start anywhere, so their elements are loaded one by one: 12484 rows of 893
// in 31 us, 2.9 TB/s, bound by the number of loads (pairs, 894: 24 us); eight rows:
// 8 us, the launch.
#include "affinity.h"
#include "internal.h"
#include "launch.cuh"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

namespace aff {
namespace {

struct NormParams {
  const void *x, *f, *gate, *post_gain, *pre_gain;
  void *y, *h;
  int64_t x_stride, f_stride, gate_stride, y_stride, h_stride;
  int64_t T, rows_per_gate;
  int32_t D;
  float scale, eps;
};

template <typename E, int VW>
struct alignas(sizeof(E) * VW) Vec {
  E e[VW];
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

// Sum over the row's threads: a whole number of warps each; `sh` has one float per warp of the block.
template <int kGroup, int kBlock>
__device__ __forceinline__ float row_sum(float v, float* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (kGroup > 32) {
    constexpr int kWarps = kGroup / 32;
    const int warp = threadIdx.x >> 5;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[warp] = v;
    __syncthreads();
    const int first = warp / kWarps * kWarps;
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += sh[first + i];
  }
  return v;
}

// kBlock threads hold kBlock / kGroup rows; a thread has up to kVecs runs of VW elements.
template <typename E, int VW, int kVecs, int kGroup, int kBlock>
__global__ void __launch_bounds__(kBlock) block_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sh[kBlock / 32];
  pdl_enter();
  using V = Vec<E, VW>;
  const int64_t t = (int64_t)blockIdx.x * (kBlock / kGroup) + threadIdx.x / kGroup;
  const int i0 = threadIdx.x % kGroup;
  const bool live = t < p.T;
  const E* x = static_cast<const E*>(p.x) + t * p.x_stride;
  const E* f = static_cast<const E*>(p.f) + t * p.f_stride;
  const E* gate = p.gate && live ? static_cast<const E*>(p.gate) + t / p.rows_per_gate * p.gate_stride : nullptr;
  const float inv_d = 1.f / (float)p.D;
  V vx[kVecs], vf[kVecs];
  bool has[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int j = (i0 + i * kGroup) * VW;
    has[i] = live && j < p.D;
    vx[i] = V{};
    vf[i] = V{};
    if (has[i]) {
      vf[i] = *reinterpret_cast<const V*>(f + j);
      vx[i] = *reinterpret_cast<const V*>(x + j);
    }
  }
  float inv = 1.f;
  if (p.post_gain) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        const float v = to_f(vf[i].e[e]);
        ss += v * v;
      }
    inv = rsqrtf(row_sum<kGroup, kBlock>(ss, sh) * inv_d + p.eps);
  }
  float yv[kVecs][VW];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int j = (i0 + i * kGroup) * VW;
    V pg{}, gt{};
    if (has[i] && p.post_gain) pg = *reinterpret_cast<const V*>(static_cast<const E*>(p.post_gain) + j);
    if (has[i] && gate) gt = *reinterpret_cast<const V*>(gate + j);
    V out;
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      float u = to_f(vf[i].e[e]);
      if (p.post_gain) u *= inv * to_f(pg.e[e]);
      if (gate) u *= to_f(gt.e[e]);
      yv[i][e] = to_f(vx[i].e[e]) + p.scale * u;
      ss += yv[i][e] * yv[i][e];
      from_f(yv[i][e], out.e[e]);
    }
    if (has[i]) *reinterpret_cast<V*>(static_cast<E*>(p.y) + t * p.y_stride + j) = out;
  }
  if (!p.h) return;
  const float ry = rsqrtf(row_sum<kGroup, kBlock>(ss, sh) * inv_d + p.eps);
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int j = (i0 + i * kGroup) * VW;
    if (!has[i]) continue;
    const V pg = *reinterpret_cast<const V*>(static_cast<const E*>(p.pre_gain) + j);
    V out;
#pragma unroll
    for (int e = 0; e < VW; ++e) from_f(yv[i][e] * ry * to_f(pg.e[e]), out.e[e]);
    *reinterpret_cast<V*>(static_cast<E*>(p.h) + t * p.h_stride + j) = out;
  }
}

template <typename E, int VW, int kVecs, int kGroup, int kBlock>
aff_status go(const NormParams& p, cudaStream_t s) {
  const int64_t per = kBlock / kGroup;
  const int64_t blocks = (p.T + per - 1) / per;
  if (blocks > INT32_MAX) return AFF_ERR_UNSUPPORTED_SHAPE;
  AFF_CUDA(launch_pdl(block_norm_kernel<E, VW, kVecs, kGroup, kBlock>, (unsigned)blocks, kBlock, 0, s, p));
  return AFF_OK;
}

// Few rows: a thread has one run of VW elements, for latency.  Many rows (more than kManyRows, enough to
// give every SM several): up to four runs each, so that a row takes one or a few warps and more of its
// bytes are in flight per thread.  One row to a block: 65536 rows of 1024 bf16 take 88 us with a warp to a
// row and a block, 101 with four rows to a block, 108 with 128 threads to a row.  Single elements and pairs:
// up to eight runs (12484 x 893: 31 us; 36 with up to four, 115 with one).
constexpr int64_t kManyRows = 152 * 8;

template <typename E, int VW>
aff_status pick(const NormParams& p, cudaStream_t s) {
  const int runs = (p.D + VW - 1) / VW;
  if constexpr (VW > 2) {
    if (p.T > kManyRows && runs > 32) {
      if (runs <= 64) return go<E, VW, 2, 32, 32>(p, s);
      if (runs <= 96) return go<E, VW, 3, 32, 32>(p, s);
      if (runs <= 128) return go<E, VW, 4, 32, 32>(p, s);
      if (runs <= 192) return go<E, VW, 3, 64, 64>(p, s);
      if (runs <= 256) return go<E, VW, 4, 64, 64>(p, s);
      if (runs <= 384) return go<E, VW, 3, 128, 128>(p, s);
      if (runs <= 512) return go<E, VW, 4, 128, 128>(p, s);
      if (runs <= 768) return go<E, VW, 3, 256, 256>(p, s);
      if (runs <= 1024) return go<E, VW, 4, 256, 256>(p, s);
    }
  }
  if constexpr (VW <= 2) {
    if (p.T > kManyRows && runs > 64) {
      if (runs <= 128) return go<E, VW, 4, 32, 32>(p, s);
      if (runs <= 256) return go<E, VW, 8, 32, 32>(p, s);
      if (runs <= 512) return go<E, VW, 8, 64, 64>(p, s);
      if (runs <= 1024) return go<E, VW, 8, 128, 128>(p, s);
      if (runs <= 2048) return go<E, VW, 8, 256, 256>(p, s);
    }
  }
  if (runs <= 32) return go<E, VW, 1, 32, 128>(p, s);
  if (runs <= 64) return go<E, VW, 1, 64, 64>(p, s);
  if (runs <= 128) return go<E, VW, 1, 128, 128>(p, s);
  if (runs <= 256) return go<E, VW, 1, 256, 256>(p, s);
  if (runs <= 512) return go<E, VW, 1, 512, 512>(p, s);
  if (runs <= 1024) return go<E, VW, 1, 1024, 1024>(p, s);
  if (runs <= 2048) return go<E, VW, 2, 1024, 1024>(p, s);
  if (runs <= 4096) return go<E, VW, 4, 1024, 1024>(p, s);
  if constexpr (VW <= 2) {
    if (runs <= 8192) return go<E, VW, 8, 1024, 1024>(p, s);
  }
  if constexpr (VW == 1) {
    if (runs <= 16384) return go<E, VW, 16, 1024, 1024>(p, s);
  }
  return AFF_ERR_UNSUPPORTED_SHAPE;
}

}  // namespace
}  // namespace aff

using namespace aff;

extern "C" aff_status affinity_block_norm(const aff_block_norm* a, aff_stream_t stream) {
  if (!a) return AFF_ERR_INVALID_ARG;
  if (a->dtype != AFF_BF16 && a->dtype != AFF_FP32) return AFF_ERR_UNSUPPORTED_DTYPE;
  if (!a->x || !a->f || !a->y || (a->h != nullptr) != (a->pre_gain != nullptr)) return AFF_ERR_INVALID_ARG;
  if (a->T < 1 || a->D < 1 || a->x_stride < a->D || a->f_stride < a->D || a->y_stride < a->D ||
      (a->h && a->h_stride < a->D) || (a->gate && (a->rows_per_gate < 1 || a->gate_stride < a->D)))
    return AFF_ERR_INVALID_ARG;
  if (!(std::isfinite(a->eps) && a->eps >= 0.f) || !std::isfinite(a->scale)) return AFF_ERR_INVALID_ARG;
  if (a->D > 16384) return AFF_ERR_UNSUPPORTED_SHAPE;
  const int es = a->dtype == AFF_BF16 ? 2 : 4;
  uintptr_t all = 0;
  int64_t strides = 0;
  const void* ptrs[] = {a->x, a->f, a->y, a->h, a->gate, a->post_gain, a->pre_gain};
  for (const void* q : ptrs) all |= reinterpret_cast<uintptr_t>(q);
  if (all & 15u) return AFF_ERR_ALIGNMENT;
  strides = a->x_stride | a->f_stride | a->y_stride | (a->h ? a->h_stride : 0) | (a->gate ? a->gate_stride : 0);
  int sms = 0;
  aff_status st = check_device(&sms);
  if (st != AFF_OK) return st;
  NormParams p{};
  p.x = a->x; p.f = a->f; p.gate = a->gate; p.post_gain = a->post_gain; p.pre_gain = a->pre_gain;
  p.y = a->y; p.h = a->h;
  p.x_stride = a->x_stride; p.f_stride = a->f_stride; p.gate_stride = a->gate_stride;
  p.y_stride = a->y_stride; p.h_stride = a->h_stride;
  p.T = a->T; p.rows_per_gate = a->gate ? a->rows_per_gate : 1;
  p.D = (int)a->D;
  p.scale = a->scale;
  p.eps = a->eps;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // 16-byte runs where every row starts on one, else pairs, else single elements
  const int64_t together = a->D | strides;
  const bool wide = together * es % 16 == 0, pairs = together % 2 == 0;
  if (a->dtype == AFF_BF16)
    return wide ? pick<__nv_bfloat16, 8>(p, s) : pairs ? pick<__nv_bfloat16, 2>(p, s) : pick<__nv_bfloat16, 1>(p, s);
  return wide ? pick<float, 4>(p, s) : pairs ? pick<float, 2>(p, s) : pick<float, 1>(p, s);
}
