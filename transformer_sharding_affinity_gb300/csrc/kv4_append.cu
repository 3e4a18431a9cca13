// kv4_append.cu -- affinity_kv4_append: a step's queries, keys and values, once over, into a cache in 4 bits; and
// affinity_kv4_read, a step's tokens back.  Norms and rotation as in kv_append.cu; then, for keys and values,
//
//   scale = e4m3(max_block |x| / (6 g)),   code = e2m1(x / (scale g))       (kv4.cuh, include/affinity.h)
//
// T (H + 2G) d elements in, T H d elements and 9/16 byte for each of 2 T G d out.  64 x 1024 tokens of 16 + 2 x 8 heads of
// 128, bf16, normalised and turned: 285 us, 3.1 TB/s.  Bound by issue (918 instructions of a warp for 8 rows of 128, 73 %
// of the slots): an element's bounds are quantised beside it.
// What counted: packed arithmetic and quotients by reciprocal and remainder instead of division (500 -> 356 us, with
// 64 x 1024 tokens read back), bounds for each element and only those in doubt in 64 bits (-> 347).  Two tokens to a
// thread instead of two rows of one: 428; one row to a thread 411; 80 registers instead of 64: 358, 48: 425.  Of the 347,
// 47 go to the bounds and 47 to the path in 64 bits, most of that for the last ones' latency at the kernel's end.
//
// Borders.  A code changes where x / (scale g) passes one of seven values, a scale where the maximum does, so a last
// bit of fp32 may move an element by a third of its size.  Values and plain keys are exact in the activations'
// type, and their quotients are too wherever they lie on a border: q + (x - q s) / s, with q off by an ulp or two, is the
// rounded quotient (the remainder is exact, as s has four bits), and that reaches a border only from it: fp32 decides.
// Rotated and normalised keys are off by at most kMarginNorm or kMarginTurn of the products they are the sum of.
// Where that crosses a border of codes, the element is compared with it in 64 bits; where it crosses one of scales, or more
// than one of codes, the row is computed again in 64 bits, rounded to odd before each of the two conversions, so that the
// double rounding does not show.  1 in 60000 normalised elements is in doubt; the 64-bit units have a sixty-fourth of
// the others' rate, so a narrow margin is worth its arithmetic.
#include "affinity.h"
#include "internal.h"
#include "kv4.cuh"
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
// What fp32 keys may be off by, in units of 2^-24 of the products they are the sum of.  Turned: a product and a fused
// product and sum, 2; with a norm before it: the sum of squares (a lane's chain of four, two sums, four levels of
// shuffles) 10, the mean and eps 3, together halved by the root; the root after a step of Newton's 1.5; the gain's two
// products 2.  Rounded up to 4 and 14.
constexpr float kMarginTurn = 4.f / (1 << 24), kMarginNorm = 14.f / (1 << 24);

struct AppendParams {
  StepGeom g;
  Kv4Pool pool;
  const void *q, *k, *v;
  void* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  const float *cos, *sin;
  const void *q_gain, *k_gain;
  int64_t n_pos;
  float eps, inv_d;
  float k_scale, v_scale, k_inv, v_inv;      // and their reciprocals
  int32_t rot, interleaved, lanes, lane_bits;
};

// Eight numbers, as four pairs for the packed instructions.
struct Eight {
  uint64_t p[4];
};
// Eight neighbouring elements.
template <typename E>
struct Run;
template <>
struct Run<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* at) { w = __ldcs(reinterpret_cast<const uint4*>(at)); }
  __device__ __forceinline__ void load_shared(const __nv_bfloat16* at) { w = __ldg(reinterpret_cast<const uint4*>(at)); }
  __device__ __forceinline__ void clear() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ Eight get() const {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    Eight f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.p[i] = pk_u(x[i] << 16, x[i] & 0xffff0000u);
    return f;
  }
  static __device__ __forceinline__ void put(__nv_bfloat16* at, const Eight& f) {
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpk(f.p[i]);
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(x[i]) : "f"(v.y), "f"(v.x));
    }
    *reinterpret_cast<uint4*>(at) = make_uint4(x[0], x[1], x[2], x[3]);
  }
};
template <>
struct Run<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* at) {
    a = __ldcs(reinterpret_cast<const float4*>(at));
    b = __ldcs(reinterpret_cast<const float4*>(at) + 1);
  }
  __device__ __forceinline__ void load_shared(const float* at) {
    a = __ldg(reinterpret_cast<const float4*>(at));
    b = __ldg(reinterpret_cast<const float4*>(at) + 1);
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ Eight get() const { return {{pk(a.x, a.y), pk(a.z, a.w), pk(b.x, b.y), pk(b.z, b.w)}}; }
  static __device__ __forceinline__ void put(float* at, const Eight& f) {
    const float2 x = unpk(f.p[0]), y = unpk(f.p[1]), z = unpk(f.p[2]), w = unpk(f.p[3]);
    reinterpret_cast<float4*>(at)[0] = make_float4(x.x, x.y, y.x, y.y);
    reinterpret_cast<float4*>(at)[1] = make_float4(z.x, z.y, w.x, w.y);
  }
};

// Eight numbers to eight codes.
__device__ __forceinline__ uint32_t to_codes(const Eight& x) {
  const float2 a = unpk(x.p[0]), b = unpk(x.p[1]), c = unpk(x.p[2]), d = unpk(x.p[3]);
  uint32_t w;
  asm("{.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};}"
      : "=r"(w)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
  return w;
}
// Two scales, the first in the low byte.
__device__ __forceinline__ uint32_t to_scales(float a, float b) {
  uint32_t r;
  asm("{.reg .b16 x;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\tmov.b32 %0, {x, 0};}" : "=r"(r) : "f"(a), "f"(b));
  return r;
}
// The value of a scale byte that is no NaN.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  float r;
  asm("{.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;}" : "=f"(r) : "r"(kv4_scale_pair(byte)));
  return r;
}
// x / 6 rounded to nearest (x >= 0), for x past 4096 what saturates as x / 6 does.
__device__ __forceinline__ float sixth(float x) {
  x = fminf(x, 4096.f);
  const float q = x * (1.f / 6.f);
  return fmaf(fmaf(-q, 6.f, x), 1.f / 6.f, q);
}
__device__ __forceinline__ float reciprocal(float x) {      // within an ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The larger of m and two magnitudes; NaN if one is.
__device__ __forceinline__ float largest(float m, uint64_t pair) {
  const float2 v = unpk(pair);
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float larger(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float largest(const Eight& f) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = largest(m, f.p[i]);
  return m;
}

// The scale of a block whose maximum is `top`, which may be off by `error`; *near_border is set where that could matter, or
// where an element that is off by as much could be one of three codes (their borders are half a step apart or more).
struct Scale {
  uint32_t byte;
  float step, inv;                               // scale g and its reciprocal, 0 where that is 0 or the block not finite
};
__device__ __forceinline__ Scale make_scale(float top, float g, float inv_g, float error, bool inexact, bool* near_border) {
  const bool finite = top < INFINITY;
  const uint32_t two = to_scales(sixth(top * inv_g), 0.f) & 0xff;
  const float s = finite ? scale_value(two) : 0.f, inv = s > 0.f ? reciprocal(s) * inv_g : 0.f;
  if (inexact) {
    const uint32_t both = to_scales(sixth((top + error) * inv_g), sixth(fmaxf(top - error, 0.f) * inv_g));
    if (finite && ((both & 0xff) != both >> 8 || error * inv > 0.2f)) *near_border = true;
  }
  return {finite ? two : 0x7f, s * g, inv};
}

// The codes of eight elements of a block, which may be off by e_i margin where `inexact`: lo and hi differ in the elements
// for which that could matter.
struct Quantised {
  uint32_t codes, lo, hi;
};
__device__ __forceinline__ Quantised quantise(Eight x, float top, float g, const Scale& s, const Eight& e, float margin,
                                              bool inexact) {
  if (top >= 4096.f * g) {                       // far past what saturates: the quotients might overflow
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpk(x.p[i]);
      x.p[i] = pk(fminf(fmaxf(v.x, -4096.f * g), 4096.f * g), fminf(fmaxf(v.y, -4096.f * g), 4096.f * g));
    }
  }
  const uint64_t inv2 = pk(s.inv, s.inv), less2 = pk(-s.step, -s.step);
  Eight q;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t q0 = mul2(x.p[i], inv2);
    q.p[i] = fma2(fma2(q0, less2, x.p[i]), inv2, q0);
  }
  Quantised r{0, 0, 0};
  if (s.byte == 0x7f) return r;
  if (!inexact) {
    r.codes = to_codes(q);
  } else {
    const float d = margin * s.inv;
    Eight lo, hi;                                // away from zero and towards it, or the other way round
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi.p[i] = fma2(e.p[i], pk(d, d), q.p[i]);
      lo.p[i] = fma2(e.p[i], pk(-d, -d), q.p[i]);
    }
    r.codes = to_codes(hi);                        // (of an element in doubt neither is taken)
    r.lo = to_codes(lo) & 0x77777777u;
    r.hi = r.codes & 0x77777777u;
  }
  return r;
}

// x to fp32, towards zero, its last bit set where something was cut off: a rounding of the result to fewer bits is
// that of x.
__device__ __forceinline__ float to_odd(double x) {
  const float f = __double2float_rz(x);
  return (double)f == x || isnan(x) ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// Where the other run of a block is: runs of eight are numbered along the head, 2 i and 2 i + 1 are a block.
struct Partner {
  int lane_a, lane_b;          // of the warp
  bool b_of_a, b_of_b;         // whether it is that lane's second run
};

struct ExactRow {
  const void *src, *gain;      // of the row
  const float *cos, *sin;      // of its position and this lane's pairs; null: not rotated
  int ja, jb, lanes, d;
  bool interleaved;
  float eps, inv_g;
};
struct Codes {
  uint32_t a, b, scale_a, scale_b;
};

// A key row in 64 bits, by the row's lanes.  Loops stay loops: a rare path, and small.  `a`, `b`: the lane's runs as fp32
// has them.  Where no scale is in doubt (`whole` false), the elements that are, alone: each is on one side or the other
// of the border between its two codes, which is exact (make_scale sees to it that there are no more than two).
template <typename E>
__device__ __noinline__ Codes exact_codes(const ExactRow r, const Partner p, bool split, Codes c, const Quantised a,
                                          const Quantised b, bool whole) {
  const E* src = static_cast<const E*>(r.src);
  const E* gain = static_cast<const E*>(r.gain);
  const bool has = r.ja < r.d;
  double inv = 1.0;
  if (gain) {
    double ss = 0.0;
#pragma unroll 1
    for (int e = 0; has && e < 16; ++e) {
      const double x = (double)(float)src[e < 8 ? r.ja + e : r.jb + e - 8];
      ss += x * x;
    }
    for (int o = r.lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    inv = 1.0 / sqrt(ss / r.d + (double)r.eps);
  }
  // pair e: elements (ja + e, jb + e), or two neighbours
  auto pair = [&](int e, double* x, double* y) {
    const int i = r.interleaved ? r.ja + 2 * e : r.ja + e, j = r.interleaved ? i + 1 : r.jb + e;
    *x = (double)(float)src[i] * inv;
    *y = (double)(float)src[j] * inv;
    if (gain) {
      *x *= (double)(float)gain[i];
      *y *= (double)(float)gain[j];
    }
    if (r.cos) {
      const double c = r.cos[e], s = r.sin[e], z = *x * c - *y * s;
      *y = *x * s + *y * c;
      *x = z;
    }
  };
  if (!whole) {
    const float step_a = scale_value(c.scale_a), step_b = scale_value(c.scale_b);
    uint32_t in_a = a.lo ^ a.hi, in_b = b.lo ^ b.hi;
#pragma unroll 1
    while (has && (in_a | in_b)) {
      const bool second = in_a == 0;
      const int i = (__ffs(second ? in_b : in_a) - 1) >> 2, at = (second ? 8 : 0) + i;
      double x, y;
      pair(r.interleaved ? at >> 1 : i, &x, &y);
      const double z = (r.interleaved ? at & 1 : second) ? y : x, v = fabs(z) * r.inv_g;
      const uint32_t u = (second ? b.lo : a.lo) >> (4 * i) & 7, w = (second ? b.hi : a.hi) >> (4 * i) & 7, low = min(u, w);
      const float mid = low < 4 ? 0.25f + 0.5f * low : low == 4 ? 2.5f : low == 5 ? 3.5f : 5.f;
      const double border = (double)(mid * (second ? step_b : step_a));
      const uint32_t code = v > border || (v == border && (low & 1)) ? low + 1 : low;
      uint32_t& word = second ? c.b : c.a;
      word = (word & ~(15u << 4 * i)) | (code | (z < 0.0 ? 8u : 0u)) << 4 * i;
      (second ? in_b : in_a) &= ~(15u << 4 * i);
    }
    return c;
  }
  double top_a = 0.0, top_b = 0.0;
#pragma unroll 1
  for (int e = 0; has && e < 8; ++e) {
    double x, y;
    pair(e, &x, &y);
    if (r.interleaved) {
      x = fmax(fabs(x), fabs(y));
      if (e < 4) top_a = fmax(top_a, x);
      else top_b = fmax(top_b, x);
    } else {
      top_a = fmax(top_a, fabs(x));
      top_b = fmax(top_b, fabs(y));
    }
  }
  const double aa = __shfl_sync(0xffffffffu, top_a, p.lane_a), ab = __shfl_sync(0xffffffffu, top_b, p.lane_a);
  const double ba = __shfl_sync(0xffffffffu, top_a, p.lane_b), bb = __shfl_sync(0xffffffffu, top_b, p.lane_b);
  const double other_a = split ? (p.b_of_a ? ab : aa) : top_b, other_b = split ? (p.b_of_b ? bb : ba) : top_a;
  top_a = fmax(top_a, other_a);
  top_b = fmax(top_b, other_b);
  c = Codes{0, 0, to_scales(to_odd(top_a * r.inv_g / 6.0), 0.f) & 0xff, to_scales(to_odd(top_b * r.inv_g / 6.0), 0.f) & 0xff};
  const double sa = scale_value(c.scale_a), sb = scale_value(c.scale_b);
  auto code = [&](double x, double s) {
    return to_codes(Eight{{pk(s > 0.0 ? to_odd(x * r.inv_g / s) : 0.f, 0.f), 0, 0, 0}}) & 15u;
  };
#pragma unroll 1
  for (int e = 0; has && e < 8; ++e) {
    double x, y;
    pair(e, &x, &y);
    if (r.interleaved) {
      const double s = e < 4 ? sa : sb;
      const uint32_t two = (code(x, s) | code(y, s) << 4) << (8 * (e & 3));
      if (e < 4) c.a |= two;
      else c.b |= two;
    } else {
      c.a |= code(x, sa) << (4 * e);
      c.b |= code(y, sb) << (4 * e);
    }
  }
  return c;
}

// (x, y) turned, both of each pair of pairs.
__device__ __forceinline__ void turn2(uint64_t& x, uint64_t& y, uint64_t c, uint64_t s) {
  const float2 t = unpk(s);
  const uint64_t minus = pk(-t.x, -t.y);
  const uint64_t z = fma2(y, minus, mul2(x, c));
  y = fma2(x, s, mul2(y, c));
  x = z;
}
__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float z = x * c - y * s;
  y = x * s + y * c;
  x = z;
}

// A block is (a part of) one token; a row is dealt to `lanes` neighbouring threads, each with two runs of eight
// elements: of the rotated part the two halves of eight pairs (or, interleaved, two neighbouring runs whose pairs
// lie side by side), past it and in value rows neighbours.  A thread has kPer rows, `slots` apart.
template <typename E>
__global__ void __launch_bounds__(kThreads, 4) kv4_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kPer = 2;
  pdl_enter();
  const StepGeom& g = p.g;
  const int t = blockIdx.x, lane = threadIdx.x & (p.lanes - 1);
  const int slots = blockDim.x >> p.lane_bits;
  const int r0 = blockIdx.y * slots * kPer + (threadIdx.x >> p.lane_bits);
  const int half = p.rot / 2, units = half / 8, n_rot = g.H + g.G, rows = n_rot + g.G;
  // this lane's runs in a row that is turned and in one that is not
  const bool rotates = lane < units, split = rotates && !p.interleaved;
  const int ja = rotates ? (p.interleaved ? 16 : 8) * lane : p.rot + 16 * (lane - units);
  const int jb = split ? ja + half : ja + 8;
  // the rows first: they do not depend on where their token stands
  Run<E> va[kPer], vb[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = r0 + k * slots;
    const E* src = r < g.H   ? static_cast<const E*>(p.q) + (int64_t)t * p.q_stride + r * g.d
                   : r < n_rot ? static_cast<const E*>(p.k) + (int64_t)t * p.k_stride + (r - g.H) * g.d
                               : static_cast<const E*>(p.v) + (int64_t)t * p.v_stride + (r - n_rot) * g.d;
    const int a = r < n_rot ? ja : 16 * lane, b = r < n_rot ? jb : 16 * lane + 8;
    va[k].clear();
    vb[k].clear();
    if (r < rows && a < g.d) {          // d is whole units of 16: both runs are there, or none
      va[k].load(src + a);
      vb[k].load(src + b);
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
  const float *cos = p.cos + pos * half + 8 * lane, *sin = p.sin + pos * half + 8 * lane;
  const int64_t page = (ti.slot >> 32) * p.pool.page_stride;
  const int token = (int)(ti.slot & 0xffffffff);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = r0 + k * slots;
    const bool is_q = r < g.H, turned = r < n_rot, live = r < rows && stand;
    Eight a = va[k].get(), b = vb[k].get();
    const E* gain = static_cast<const E*>(is_q ? p.q_gain : turned ? p.k_gain : nullptr);
    float inv = 1.f;
    if ((p.q_gain || p.k_gain) && !__all_sync(0xffffffffu, !turned)) {
      // every lane of the warp takes part in the sum
      uint64_t s2 = mul2(a.p[0], a.p[0]), s3 = mul2(b.p[0], b.p[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        s2 = fma2(a.p[i], a.p[i], s2);
        s3 = fma2(b.p[i], b.p[i], s3);
      }
      const float2 x = unpk(s2), y = unpk(s3);
      float ss = (x.x + x.y) + (y.x + y.y);
      for (int o = p.lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float m = ss * p.inv_d + p.eps;
      inv = rsqrtf(m);
      const float more = fmaf(0.5f * inv, fmaf(-m * inv, inv, 1.f), inv);      // a step of Newton's
      if (m > 1e-30f && m < 1e30f) inv = more;
    }
    const int at_a = turned ? ja : 16 * lane, at_b = turned ? jb : 16 * lane + 8;
    const bool has = at_a < g.d;
    Eight ea{{0, 0, 0, 0}}, eb = ea;               // what the products are at most, by magnitude, but for cos and sin
    const bool inexact = turned && !is_q && (gain || rotates);
    float margin = gain ? kMarginNorm : kMarginTurn;
    if (turned && live && has) {
      if (gain) {
        Run<E> ga, gb;
        ga.load_shared(gain + at_a);
        gb.load_shared(gain + at_b);
        const Eight fa = ga.get(), fb = gb.get();
        const uint64_t inv2 = pk(inv, inv);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a.p[i] = mul2(a.p[i], mul2(inv2, fa.p[i]));
          b.p[i] = mul2(b.p[i], mul2(inv2, fb.p[i]));
        }
      }
      if (inexact) {
        ea = a;
        eb = b;
      }
      if (rotates) {
        Eight c, s;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float4 x = __ldg(reinterpret_cast<const float4*>(cos + 2 * i)), y = __ldg(reinterpret_cast<const float4*>(sin + 2 * i));
          c.p[i] = pk(x.x, x.y);
          c.p[i + 1] = pk(x.z, x.w);
          s.p[i] = pk(y.x, y.y);
          s.p[i + 1] = pk(y.z, y.w);
        }
        if (inexact) {
          margin *= larger(largest(c), largest(s));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 x = unpk(a.p[i]), y = unpk(b.p[i]);
            if (p.interleaved) {
              const float ex = fabsf(x.x) + fabsf(x.y), ey = fabsf(y.x) + fabsf(y.y);
              ea.p[i] = pk(ex, ex);
              eb.p[i] = pk(ey, ey);
            } else {
              ea.p[i] = eb.p[i] = pk(fabsf(x.x) + fabsf(y.x), fabsf(x.y) + fabsf(y.y));
            }
          }
        }
        if (!p.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) turn2(a.p[i], b.p[i], c.p[i], s.p[i]);
        } else {
          // pairs (2e, 2e + 1) of 16 neighbours: the first four in a, the others in b
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float2 x = unpk(a.p[i]), y = unpk(b.p[i]);
            const float2 ca = unpk(c.p[i >> 1]), sa = unpk(s.p[i >> 1]), cb = unpk(c.p[2 + (i >> 1)]), sb = unpk(s.p[2 + (i >> 1)]);
            turn(x.x, x.y, i & 1 ? ca.y : ca.x, i & 1 ? sa.y : sa.x);
            turn(y.x, y.y, i & 1 ? cb.y : cb.x, i & 1 ? sb.y : sb.x);
            a.p[i] = pk(x.x, x.y);
            b.p[i] = pk(y.x, y.y);
          }
        }
      }
    }
    if (is_q) {
      if (r < rows && has) {
        if (!stand) {
#pragma unroll
          for (int i = 0; i < 4; ++i) a.p[i] = b.p[i] = 0;       // padding
        }
        E* dst = static_cast<E*>(p.q_out) + (int64_t)t * p.q_out_stride + r * g.d;
        Run<E>::put(dst + at_a, a);
        Run<E>::put(dst + at_b, b);
      }
    }
    if (__all_sync(0xffffffffu, is_q || r >= rows)) continue;
    // the blocks' maxima: of this lane's runs and of the runs beside them
    float top_a = largest(a), top_b = largest(b);
    Partner with{0, 0, false, false};
    const bool across = split && turned;
    if (__any_sync(0xffffffffu, across)) {
      const int base = (threadIdx.x & 31) & ~(p.lanes - 1), ra = lane ^ 1, rb = (units + lane) ^ 1;
      with.b_of_a = ra >= units;
      with.lane_a = split ? base + (with.b_of_a ? ra - units : ra) : base + lane;
      with.b_of_b = rb >= units;
      with.lane_b = split ? base + (with.b_of_b ? rb - units : rb) : base + lane;
      float oa, ob;
      if (units & 1) {
        const float aa = __shfl_sync(0xffffffffu, top_a, with.lane_a), ab = __shfl_sync(0xffffffffu, top_b, with.lane_a);
        const float ba = __shfl_sync(0xffffffffu, top_a, with.lane_b), bb = __shfl_sync(0xffffffffu, top_b, with.lane_b);
        oa = with.b_of_a ? ab : aa;
        ob = with.b_of_b ? bb : ba;
      } else {                                     // a run's neighbour is the same run of the next lane
        oa = __shfl_xor_sync(0xffffffffu, top_a, 1);
        ob = __shfl_xor_sync(0xffffffffu, top_b, 1);
      }
      const float ta = larger(top_a, across ? oa : top_b), tb = larger(top_b, across ? ob : top_a);
      top_a = ta;
      top_b = tb;
    } else {
      top_a = top_b = larger(top_a, top_b);
    }
    // Every lane looks with its own errors at whether a maximum is near a border: the one that has it is among them.
    const float g_scale = turned ? p.k_scale : p.v_scale, inv_g = turned ? p.k_inv : p.v_inv;
    const float error = inexact ? larger(largest(ea), largest(eb)) * margin : 0.f;
    bool scale_in_doubt = false;
    const Scale scale_a = make_scale(top_a, g_scale, inv_g, error, inexact, &scale_in_doubt);
    Scale scale_b = scale_a;
    if (__any_sync(0xffffffffu, across)) scale_b = make_scale(top_b, g_scale, inv_g, error, inexact, &scale_in_doubt);
    const Quantised qa = quantise(a, top_a, g_scale, scale_a, ea, margin, inexact);
    const Quantised qb = quantise(b, top_b, g_scale, scale_b, eb, margin, inexact);
    Codes w{qa.codes, qb.codes, scale_a.byte, scale_b.byte};
    const bool keep = live && !is_q, watch = keep && has && inexact;
    const bool whole = __any_sync(0xffffffffu, scale_in_doubt && watch);
    if (whole || __any_sync(0xffffffffu, watch && (qa.lo != qa.hi || qb.lo != qb.hi))) {
      // the key rows of the warp that are no plain copies; rows that are not stored stand in with the first of the keys
      const bool again = keep && turned;
      ExactRow x;
      x.src = static_cast<const E*>(p.k) + (int64_t)t * p.k_stride + (again ? r - g.H : 0) * g.d;
      x.gain = p.k_gain;
      x.cos = rotates && stand ? cos : nullptr;
      x.sin = sin;
      x.ja = ja;
      x.jb = jb;
      x.lanes = p.lanes;
      x.d = g.d;
      x.interleaved = rotates && p.interleaved;
      x.eps = p.eps;
      x.inv_g = p.k_inv;
      const Codes exact = exact_codes<E>(x, with, split, w, qa, qb, whole);
      if (again && inexact) {
        if (w.scale_a != 0x7f) {
          w.a = exact.a;
          w.scale_a = exact.scale_a;
        }
        if (w.scale_b != 0x7f) {
          w.b = exact.b;
          w.scale_b = exact.scale_b;
        }
      }
    }
    if (!keep || !has) continue;
    uint8_t* base = const_cast<uint8_t*>(turned ? p.pool.k : p.pool.v) + page + (turned ? r - g.H : r - n_rot) * p.pool.group_stride;
    uint8_t* codes = base + token * 16 * p.pool.n;
    if (at_b == at_a + 8) {
      *reinterpret_cast<uint2*>(codes + at_a / 2) = make_uint2(w.a, w.b);
      base[kv4_scale_at(p.pool, token, at_a / 16)] = (uint8_t)w.scale_a;
    } else {
      *reinterpret_cast<uint32_t*>(codes + at_a / 2) = w.a;
      *reinterpret_cast<uint32_t*>(codes + at_b / 2) = w.b;
      if (!(at_a & 8)) base[kv4_scale_at(p.pool, token, at_a / 16)] = (uint8_t)w.scale_a;
      if (!(at_b & 8)) base[kv4_scale_at(p.pool, token, at_b / 16)] = (uint8_t)w.scale_b;
    }
    if ((g.d & 16) && lane == 0) {                 // the last chunk's other half
      *reinterpret_cast<uint2*>(codes + g.d / 2) = make_uint2(0, 0);
      base[kv4_scale_at(p.pool, token, g.d / 16)] = 0;
    }
  }
}

template <typename E>
aff_status launch(AppendParams& p, cudaStream_t s) {
  const int units = p.g.d / 16;
  p.lanes = 1;
  p.lane_bits = 0;
  while (p.lanes < units) {
    p.lanes *= 2;
    ++p.lane_bits;
  }
  p.inv_d = 1.f / (float)p.g.d;
  const int need = (p.g.H + 2 * p.g.G + 1) / 2 * p.lanes;
  const int threads = need < kThreads ? (need + 31) / 32 * 32 : kThreads;
  AFF_CUDA(launch_pdl(kv4_append_kernel<E>, dim3((unsigned)p.g.T, (unsigned)((need + threads - 1) / threads)), threads, 0,
                      s, p));
  return AFF_OK;
}

// ---------------------------------------------------------------- reading back
struct ReadParams {
  StepGeom g;
  Kv4Pool pool;
  void *k_out, *v_out;
  float k_scale, v_scale;
};

// Eight elements to a thread, kTokens tokens of a block one after the other: 4 bytes of codes and a scale in, 16 or 32
// bytes out, neighbours beside each other on both sides.  Bound by the bytes written: 64 sequences of up to 1500 tokens, 8
// heads of 128, 37 us, 5.4 TB/s.
constexpr int kTokens = 4;
template <typename E>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const __grid_constant__ ReadParams p) {
  pdl_enter();
  const StepGeom& g = p.g;
  const bool fits = plan_matches(g);
  if (!fits || g.head->n_items < 0) {
    if (threadIdx.x == 0) latch_status(&g.head->status, fits ? kStatusRange : 1);
    return;
  }
  const int per = g.d / 8, pieces = 2 * g.G * per;
  const int i = blockIdx.y * kThreads + threadIdx.x;
  if (i >= pieces) return;
  const int value = i >= pieces / 2, rest = i - value * (pieces / 2), group = rest / per, piece = rest - group * per;
  const uint8_t* pool = (value ? p.pool.v : p.pool.k) + group * p.pool.group_stride;
  E* out = static_cast<E*>(value ? p.v_out : p.k_out) + group * g.d + piece * 8;
  const float scale = value ? p.v_scale : p.k_scale;
  const int t0 = blockIdx.x * kTokens;
  uint32_t w[kTokens], sc[kTokens];
#pragma unroll
  for (int x = 0; x < kTokens; ++x) {
    w[x] = sc[x] = 0;
    if (t0 + x >= g.T) continue;
    const TokenInfo ti = g.tok[t0 + x];
    if (ti.own < 0) {
      if (ti.own == -2 && i == 0) latch_status(&g.head->status, kStatusRange);
      continue;
    }
    const int token = (int)(ti.slot & 0xffffffff);
    const uint8_t* at = pool + (ti.slot >> 32) * p.pool.page_stride;
    w[x] = __ldg(reinterpret_cast<const uint32_t*>(at + token * 16 * p.pool.n + piece * 4));
    sc[x] = __ldg(at + kv4_scale_at(p.pool, token, piece >> 1));
  }
#pragma unroll
  for (int x = 0; x < kTokens; ++x) {
    if (t0 + x >= g.T) break;
    uint32_t h[4];
    kv4_decode(w[x], h);
    const uint32_t s2 = kv4_scale_pair(sc[x] | sc[x] << 8);
    Eight f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t v = mul_f16x2(h[e], s2);        // exact
      float x, y;
      asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;}" : "=f"(x), "=f"(y) : "r"(v));
      f.p[e] = mul2(pk(x, y), pk(scale, scale));
    }
    Run<E>::put(out + (int64_t)(t0 + x) * g.G * g.d, f);
  }
}

}  // namespace
}  // namespace aff

using namespace aff;

extern "C" aff_status affinity_kv4_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                          const void* v, int64_t v_stride, const aff_kv4_cache* cache,
                                          const aff_step* step, const aff_rotary* rotary, void* q_out,
                                          int64_t q_out_stride, void* plan, size_t plan_bytes, aff_stream_t stream) {
  AppendParams p{};
  aff_status st = kv4_geom(step, cache, plan, &p.g);
  if (st != AFF_OK) return st;
  if (!q || !k || !v || !q_out || !rotary) return AFF_ERR_INVALID_ARG;
  const StepGeom& g = p.g;
  const int64_t hd = (int64_t)g.H * g.d, gd = (int64_t)g.G * g.d;
  if (q_stride < hd || k_stride < gd || v_stride < gd || q_out_stride < hd) return AFF_ERR_INVALID_ARG;
  if (rotary->rot < 0 || rotary->rot % 2 || rotary->n_pos < 0 || (rotary->rot > 0 && (!rotary->cos || !rotary->sin)) ||
      !(std::isfinite(rotary->eps) && rotary->eps >= 0.f))
    return AFF_ERR_INVALID_ARG;
  if (rotary->rot > g.d || rotary->rot % 16) return AFF_ERR_UNSUPPORTED_SHAPE;
  const int es = g.dtype == AFF_BF16 ? 2 : 4;
  const void* ptrs[] = {q, k, v, q_out, rotary->cos, rotary->sin, rotary->q_gain, rotary->k_gain};
  for (const void* x : ptrs)
    if (reinterpret_cast<uintptr_t>(x) & 15u) return AFF_ERR_ALIGNMENT;
  if (q_stride * es % 16 || k_stride * es % 16 || v_stride * es % 16 || q_out_stride * es % 16)
    return AFF_ERR_ALIGNMENT;
  if ((st = check_plan(g, plan, plan_bytes)) != AFF_OK) return st;
  int sms = 0;
  if ((st = check_device(&sms)) != AFF_OK) return st;
  p.pool = kv4_pool(cache);
  p.q = q; p.k = k; p.v = v; p.q_out = q_out;
  p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride; p.q_out_stride = q_out_stride;
  p.cos = rotary->cos; p.sin = rotary->sin;
  p.q_gain = rotary->q_gain; p.k_gain = rotary->k_gain;
  p.n_pos = rotary->rot ? rotary->n_pos : INT64_MAX;
  p.eps = rotary->eps;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.k_inv = 1.f / cache->k_scale;
  p.v_inv = 1.f / cache->v_scale;
  p.rot = rotary->rot;
  p.interleaved = rotary->interleaved != 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return g.dtype == AFF_BF16 ? launch<__nv_bfloat16>(p, s) : launch<float>(p, s);
}

extern "C" aff_status affinity_kv4_read(const aff_kv4_cache* cache, const aff_step* step, void* k_out, void* v_out,
                                        void* plan, size_t plan_bytes, aff_stream_t stream) {
  ReadParams p{};
  aff_status st = kv4_geom(step, cache, plan, &p.g);
  if (st != AFF_OK) return st;
  if (!k_out || !v_out) return AFF_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 15u) return AFF_ERR_ALIGNMENT;
  const StepGeom& g = p.g;
  if ((st = check_plan(g, plan, plan_bytes)) != AFF_OK) return st;
  int sms = 0;
  if ((st = check_device(&sms)) != AFF_OK) return st;
  p.pool = kv4_pool(cache);
  p.k_out = k_out;
  p.v_out = v_out;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  const unsigned pieces = 2u * g.G * (g.d / 8);
  const dim3 grid((unsigned)((g.T + kTokens - 1) / kTokens), (pieces + kThreads - 1) / kThreads);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (g.dtype == AFF_BF16) AFF_CUDA(launch_pdl(kv4_read_kernel<__nv_bfloat16>, grid, kThreads, 0, s, p));
  else AFF_CUDA(launch_pdl(kv4_read_kernel<float>, grid, kThreads, 0, s, p));
  return AFF_OK;
}
