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
#include "attention_parts.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "launch.cuh"
#include "sm103_primitives.cuh"
#include "step.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

namespace aff {
namespace {

constexpr float kShift = 7.f;                // log2 of the probabilities' factor: they stay below 2^15
constexpr float kLn2 = 0.69314718055994531f;

struct Kv4AttnParams {
  StepGeom g;
  Kv4Pool pool;
  const void* q;
  int64_t q_stride;
  void* out;
  float* lse;               // [T][H] or null
  float score_log2;         // scale k_scale log2(e)
  float v_scale;
  int32_t overlap;          // the few-rows kernel follows the row tiles' and starts beside it
};

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 halves(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
__device__ __forceinline__ uint2 ld_shared8(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared4(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared2(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The factor of a row of queries (its largest magnitude, as bits) and the inverse, both powers of two.  A row with an
// infinity or a NaN has no scores.
__device__ __forceinline__ float query_factor(uint32_t top, float* inverse) {
  const int e = (int)(top >> 23);
  const int up = min(127 + 13 - e, 126);      // a row of zeros or subnormals: 2^126
  *inverse = e == 255 ? __int_as_float(0x7fc00000) : __uint_as_float((uint32_t)(127 - up) << 23);
  return __uint_as_float((uint32_t)(127 + up) << 23);
}

// ---------------------------------------------------------------- shared by both kernels
// A tile's keys or values as they lie in the cache: codes of up to 128 keys, then their scales.
__host__ __device__ constexpr int raw_bytes(int chunks) { return kKeyTile * 18 * chunks; }

__device__ __forceinline__ void copy_bulk(uint32_t to, const void* from, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(from),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void prefetch(const void* from) { asm volatile("prefetch.global.L2 [%0];" ::"l"(from)); }

// A wait that ends with the CTA's giving up: one warp alone looks at the clock.  Every role's progress frees slots, which
// that warp waits for (2 s at most) to its end; so the waits in the other roles stay a few instructions each.
template <class Bars>
__device__ __forceinline__ void await(uint64_t* bar, uint32_t parity, Bars* b) {
#pragma unroll 1
  while (!mbar_try_wait(bar, parity) && !gave_up(b)) {}
  __syncwarp();
}
template <class Bars>
__device__ __forceinline__ bool slot_ready(Bars* b, int k) {
  await(&b->slot_full[k % kSlots], (k / kSlots) & 1, b);
  return __all_sync(0xffffffffu, !gave_up(b) && b->slot[k % kSlots].row0 >= 0);
}

// A copying warp's share of a tile: a page's codes are a lane's copy, its scales another's; a page has whole groups of
// 8 tokens.
struct TileShare {
  int64_t from;             // in either pool
  uint32_t to, bytes;       // in a buffer of raw_bytes; 0 bytes: none
  uint32_t total;           // of the tile's keys, or values
};
template <int NC>
__device__ __forceinline__ TileShare tile_share(const Kv4AttnParams& p, const WorkItem& it, int tile, uint32_t* status) {
  const StepGeom& g = p.g;
  const int lane = threadIdx.x & 31, box = lane & 15;
  const bool scales = lane >= 16, pre = tile < it.np;
  const int per_page = g.tile_pages ? g.page_size : g.key_tile;
  int key0;
  const int keys = tile_keys(it, g, tile, &key0), mine = min(per_page, keys - box * per_page);
  TileShare x{0, 0, 0, (uint32_t)((keys + 7) & ~7) * 18 * NC};
  if (mine > 0) {
    const int32_t* table = pre ? g.prefix_pages : g.pages + (int64_t)it.seq * g.pages_stride;
    const int key = key0 + box * per_page, pi = g.by_page(key), token = key - pi * g.page_size;
    int page = __ldg(table + pi);
    if (page < 0 || page >= g.n_pages) {               // reported; what is copied instead does not matter
      latch_status(status, kStatusRange);
      page = 0;
    }
    x.bytes = ((mine + 7) & ~7) * (scales ? 2 * NC : 16 * NC);
    x.from = page * p.pool.page_stride + it.group * p.pool.group_stride +
             (scales ? p.pool.scales + token * 2 * NC : token * 16 * NC);
    x.to = scales ? kKeyTile * 16 * NC + box * per_page * 2 * NC : box * per_page * 16 * NC;
  }
  return x;
}

// ---------------------------------------------------------------- few rows
// Items of at most 8 rows.  Eight warps share an item: 32 keys at a time are a warp's
// unit, which it copies for itself, a unit ahead (also over an item's end), into a buffer of its own; nothing is
// exchanged before the item's end.  Two CTAs of an SM have 74 to 147 KB on their way.  Products are transposed, keys as
// the long side:  S^T = K Q^T and O^T += V^T P^T, for 16 keys at a time, their operands made in registers from the copies.
//   K  lane (key quad, c) holds its key's elements 8 W c .. + 8 W - 1 as they lie in memory (W words of codes); the
//      contraction does not care which elements are a slice's, so the queries are dealt the same way.
//   V  lane (quad, c) holds elements 4 W quad .. of keys 4 c .. 4 c + 3; a byte of two keys' codes for the same
//      element makes the pair that V^T wants, two shifts and two selections for 16 elements.
// Rows of S^T are dealt to keys so that a lane's four probabilities' keys are those it holds the values of.
// 64 tokens over 8192 keys each of 8 heads of 128: 141 us, 4.3 TB/s (a cache in bf16: 336 us).  Bound by issue, 377
// instructions of a warp for 16 keys at two thirds of the rate; steps that counted: every warp its own copies (244 -> 155 us,
// a warp that copies for all had them wait for one another), fewer instructions for copies and masks (-> 146), one barrier
// an item (-> 141; 256 tokens over up to 100 keys 37 -> 33).
// fp32 takes this path for rows of any number: 9 x 5 tokens over 1900 + 100 keys of 4 heads of 64: 11.5 us; 5 x 219 tokens,
// 16 / 8 heads of 128: 72 us.
constexpr int kFewThreads = 256;
constexpr int kFewPitch = 132;               // floats of a staged row
constexpr int kUnit = 32;                    // keys

struct alignas(16) FewShared {
  alignas(16) WorkItem slot[4];              // items k, k + 1, k + 2 in slot k % 4 ..; row0 < 0: no more
  int nan_key[4][8];                         // the first key, not seen by every row, whose values of a block are NaN
  float2 ml[8][8];                           // [warp][row]: (m, l)
};
__host__ __device__ constexpr int few_smem(int chunks, bool f32) {
  return 8 * 2 * 2 * kUnit * 18 * chunks + 8 * 8 * kFewPitch * 4 + 2 * 8 * 32 * chunks * (f32 ? 4 : 2) + (int)sizeof(FewShared);
}
static_assert(2 * (few_smem(4, false) + 1024) <= 228 * 1024, "two CTAs of an SM");

// 16 bytes from global to shared memory, past the first cache.
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
// The same, or 16 zero bytes.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// CTAs of an SM: in fp32, the widest heads take more shared memory and registers than two leave.  (Heads of 65 to 96: 30 x 32
// tokens 62 -> 47 us with two, although some registers are spilled then; one token over 3000 keys 14.4 -> 16.1.)
__host__ __device__ constexpr int few_ctas(int chunks, bool f32) { return f32 && chunks > 3 ? 1 : 2; }

template <int NC, bool F32>
__global__ void __launch_bounds__(kFewThreads, few_ctas(NC, F32)) kv4_few_kernel(const __grid_constant__ Kv4AttnParams p) {
  // W: words of codes that a lane holds of a key (of a value: half as many)
  constexpr int W = NC >= 3 ? 4 : NC, VW = W == 4 ? 2 : 1, KS = 2 * W, MT = 2 * W;
  constexpr int kRaw = kUnit * 18 * NC, kE = F32 ? 4 : 2, kQRow = 32 * NC * kE;
  extern __shared__ __align__(16) uint8_t few_raw[];       // two units of each warp: keys, values
  float* const po = reinterpret_cast<float*>(few_raw + 8 * 4 * kRaw);               // [warp][row][kFewPitch]
  uint8_t* const q_rows = reinterpret_cast<uint8_t*>(po + 8 * 8 * kFewPitch);       // two items' queries
  FewShared& sh = *reinterpret_cast<FewShared*>(q_rows + 2 * 8 * kQRow);
  const StepGeom& g = p.g;
  uint32_t* status = &g.head->status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane >> 2, c = lane & 3;
  // Beside the row tiles' kernel: that one has waited for what came before the call, and lets this one start after that; its
  // own results are waited for at the end, for the sake of what follows.  (Blocks start where that kernel's have ended.)
  if (!p.overlap) pdl_enter();
  const bool fits = plan_matches(g);
  const int n_items = fits ? g.head->n_items : 0, first = fits ? g.head->few_begin : 0;
  if ((!fits || n_items < 0) && threadIdx.x == 0) latch_status(status, fits ? kStatusRange : kStatusInvalid);

  // Items come by number for the first two rounds (beside another kernel, where blocks start one after the other: from the
  // counter) and then from a counter, two ahead; warp 0 looks after them.
  const int counted = first + (p.overlap ? 0 : 2 * gridDim.x);
  auto claim = [&](unsigned n = 1u) {
    int next = 0;
    if (lane == 0) next = counted + (int)atomicAdd(&g.head->few_claimed, n);
    return next;                             // of lane 0
  };
  auto own_item = [&](int i) {               // past the other kernel's items
    while (i < n_items && g.items[i].alt != 2) i = __shfl_sync(0xffffffffu, claim(), 0);
    return i;
  };
  auto word_of = [&](int i) {                // this lane's word of the item
    return lane < (int)(sizeof(WorkItem) / 4) && i < n_items ? reinterpret_cast<const int*>(g.items + i)[lane] : -1;
  };
  auto publish = [&](int k, int word) {
    if (lane < (int)(sizeof(WorkItem) / 4)) reinterpret_cast<int*>(&sh.slot[k & 3])[lane] = word;
    if (lane < 8) sh.nan_key[k & 3][lane] = INT32_MAX;
  };
  if (warp == 0) {
    int i0 = first + blockIdx.x, i1 = i0 + gridDim.x;
    if (p.overlap) {
      i0 = __shfl_sync(0xffffffffu, claim(2), 0);
      i1 = i0 + 1;
    }
    i0 = own_item(i0);
    i1 = own_item(i1);
    if (i0 >= n_items) {                     // the other kernel's, and none left for it: the second is the first
      i0 = i1;
      i1 = n_items;
    }
    const int w0 = word_of(i0), w1 = word_of(i1);
    publish(0, w0);
    publish(1, w1);
  }
  __syncthreads();

  const int k_off = (quad >> 1) * 4 + (quad & 1);          // this lane's keys of 16: k_off, k_off + 2
  const bool k0_has = NC == 4 || 8 * W * c < g.d, k1_has = W == 4 && 8 * W * c + 16 < g.d;      // blocks of its key elements
  const bool v_has = 4 * W * quad < g.d;
  const int v_block = 4 * W * quad / 16;
  const int subs = (g.key_tile + kUnit - 1) / kUnit;
  const uint32_t mine_at = smem_u32(few_raw) + warp * 4 * kRaw;       // this warp's two units
  // from a unit's start: this lane's share of its first 16 keys, their scales, of their values, theirs
  const uint32_t k_at = k_off * 16 * NC + c * 4 * W;
  const uint32_t ks_at = kUnit * 16 * NC + ((quad >> 1) * 2 * NC + (W == 4 ? 2 * c : W == 2 ? c : c >> 1)) * 4;
  const uint32_t v_at = kRaw + 4 * c * 16 * NC + quad * 2 * W;
  const uint32_t vs_at = kRaw + kUnit * 16 * NC + (c * 2 * NC + v_block) * 4;

  // A place in this warp's walk over an item's units, 8 apart; `tile` counts from the item's first.
  struct Walk {
    int tile, sub;
  };
  auto begin = [&]() {
    Walk w{0, warp};
    while (w.sub >= subs) {
      w.sub -= subs;
      ++w.tile;
    }
    return w;
  };
  auto step = [&](Walk& w) {
    w.sub += 8;
    while (w.sub >= subs) {
      w.sub -= subs;
      ++w.tile;
    }
  };
  struct Unit {
    int key0, left;                          // its first key within its segment, keys from it on; left 0: none
    bool pre;
  };
  const uint8_t* const k_pool = p.pool.k + lane * 16;
  const uint8_t* const v_pool = p.pool.v + lane * 16;
  // Copies the unit at w or the next one that holds a key (w moves there): 8 tokens at a time lie beside each other in a
  // page, their codes and their scales.  Lanes 0 .. 3 look the pages up.  What lies behind the last key stays as it was.
  auto copy_unit = [&](const WorkItem& it, Walk& w, int buffer) {
    Unit u{0, 0, false};
    for (; w.tile < it.n0; step(w)) {
      const int keys = tile_keys(it, g, it.t0 + w.tile, &u.key0);
      u.key0 += kUnit * w.sub;
      u.left = keys - kUnit * w.sub;
      if (u.left > 0) break;
    }
    if (w.tile >= it.n0) {
      u.left = 0;
      return u;
    }
    u.pre = it.t0 + w.tile < it.np;
    int64_t codes = 0;                       // lane x < 4: where its tokens' codes begin; their scales lie `scales` further
    int scales = 0;
    if (lane < 4 && 8 * lane < u.left) {
      const int32_t* table = u.pre ? g.prefix_pages : g.pages + (int64_t)it.seq * g.pages_stride;
      const int key = u.key0 + 8 * lane, pi = g.by_page(key), token = key - pi * g.page_size;
      int page = __ldg(table + pi);
      if (page < 0 || page >= g.n_pages) {               // reported; what is copied instead does not matter
        latch_status(status, kStatusRange);
        page = 0;
      }
      codes = page * p.pool.page_stride + it.group * p.pool.group_stride + token * 16 * NC;
      scales = p.pool.scales - token * 14 * NC;
    }
    const uint32_t to = mine_at + buffer * 2 * kRaw + lane * 16;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int q = i * 32 + lane, group = NC == 4 ? i : q / (8 * NC);
      const int64_t from = __shfl_sync(0xffffffffu, codes, group) + (NC == 4 ? 0 : (i * 32 - group * 8 * NC) * 16);
      if (8 * group < u.left) {
        copy16(to + i * 512, k_pool + from);
        copy16(to + kRaw + i * 512, v_pool + from);
      }
    }
    {
      const int q = lane % (4 * NC), value = lane / (4 * NC), group = q / NC;
      const int64_t from = __shfl_sync(0xffffffffu, codes, group);
      const int more = __shfl_sync(0xffffffffu, scales, group) + (q - group * NC - lane) * 16;
      if (value < 2 && 8 * group < u.left)
        copy16(to + value * kRaw + kUnit * 16 * NC + (q - lane) * 16, (value ? v_pool : k_pool) + from + more);
    }
    return u;
  };
  // Row `warp` of an item's queries.
  auto copy_query = [&](int k) {
    const WorkItem& it = sh.slot[k & 3];
    if (it.row0 < 0) return;
    const int rr = it.row0 + warp, tok = g.by_R(rr);
    const bool live = warp < it.nrows && lane * 16 < g.d * kE;
    const int64_t at = live ? ((int64_t)tok * p.q_stride + (it.group * g.R + rr - tok * g.R) * g.d) * kE + lane * 16 : 0;
    if (lane * 16 < kQRow)
      copy16(smem_u32(q_rows) + ((k & 1) * 8 + warp) * kQRow + lane * 16, static_cast<const uint8_t*>(p.q) + at, live);
  };
  copy_query(0);

  Walk w = begin();
  Unit carried{0, 0, false};                 // the item's first unit, where it was copied before the last one's end
  int buffer = 0;
  bool few_before = false;                   // the item before has parts in one half of their room
  asm volatile("cp.async.wait_all;" ::: "memory");         // this warp's row of queries is here
  __syncthreads();                           // everybody's
#pragma unroll 1
  for (int k = 0;; ++k) {
    const WorkItem& it = sh.slot[k & 3];
    const int nrows = it.nrows, row0 = it.row0;
    if (row0 < 0) break;
    copy_query(k + 1);
    int claimed = 0, word = 0;
    bool asked = false;
    if (warp == 0) claimed = claim();
    // ---- queries: B operand of S^T, row quad
    uint32_t qh[KS][2], ql[F32 ? KS : 1][2];
    float inverse;
    {
      const uint8_t* src = q_rows + ((k & 1) * 8 + quad) * kQRow + 8 * W * c * kE;
      const bool has = 8 * W * c < 32 * NC;
      float x[8 * W];
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        if constexpr (F32) {
          const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
          const float4 a = has ? reinterpret_cast<const float4*>(src)[2 * j] : z;
          const float4 b = has ? reinterpret_cast<const float4*>(src)[2 * j + 1] : z;
          x[8 * j] = a.x; x[8 * j + 1] = a.y; x[8 * j + 2] = a.z; x[8 * j + 3] = a.w;
          x[8 * j + 4] = b.x; x[8 * j + 5] = b.y; x[8 * j + 6] = b.z; x[8 * j + 7] = b.w;
        } else {
          const uint4 w = has ? reinterpret_cast<const uint4*>(src)[j] : make_uint4(0, 0, 0, 0);
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
      const float back = __shfl_sync(0xffffffffu, inverse, r * 4);
      own_vis[e] = r >= nrows ? 0 : it.seq < 0 ? INT32_MAX : g.by_R(row0 + r) + it.own_off + 1;
      sc[e] = own_vis[e] <= 0 ? 1.f : back * p.score_log2;
      m[e] = -INFINITY;
      l[e] = 0.f;
    }
    const int seen_by_all = all_see(it, g);
#pragma unroll
    for (int t = 0; t < MT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;


    Unit u = carried;
    if (u.left <= 0) {
      w = begin();
      u = copy_unit(it, w, buffer);
      copy_commit();
    }
    carried.left = 0;
    int units = 0;
#pragma unroll 1
    for (; u.left > 0; ++units) {
      // the next unit, of this item or else of the next
      step(w);
      const Unit next = copy_unit(it, w, buffer ^ 1);
      if (next.left <= 0 && sh.slot[(k + 1) & 3].row0 >= 0) {
        w = begin();
        carried = copy_unit(sh.slot[(k + 1) & 3], w, buffer ^ 1);
      }
      const int left = u.left, unit0 = u.key0;
      const bool pre = u.pre;
      copy_commit();
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
      const uint32_t base = mine_at + buffer * 2 * kRaw;
      float s[2][4];                         // s[h][e]: key 16 h + k_off, row 2 c + e; s[h][2 + e]: key 16 h + k_off + 2
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // (a lane without elements reads what lies beside: its scales are 0)
        uint32_t kr[2][W], ks[2] = {0, 0};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t from = base + k_at + (16 * h + 2 * x) * 16 * NC;
          if constexpr (W == 4) {
            const uint4 w = ld_shared16(from);
            kr[x][0] = w.x; kr[x][1] = w.y; kr[x][2] = w.z; kr[x][3] = w.w;
          } else if constexpr (W == 2) {
            const uint2 w = ld_shared8(from);
            kr[x][0] = w.x; kr[x][1] = w.y;
          } else {
            kr[x][0] = ld_shared4(from);
          }
        }
        if constexpr (W == 4) {
          const uint2 w = ld_shared8(base + ks_at + h * 32 * NC);
          ks[0] = k0_has ? w.x : 0;
          ks[1] = k1_has ? w.y : 0;
        } else {
          const uint32_t w = ld_shared4(base + ks_at + h * 32 * NC);
          ks[0] = k0_has ? w : 0;
        }
        uint32_t ka[2], kb[2];               // scales of this lane's blocks, twice, of either key
        if constexpr (W == 4) {
          const uint32_t b = quad & 1;
          const uint32_t a2 = kv4_scale_pair(prmt(ks[0], ks[1], b | (4 + b) << 4));
          const uint32_t b2 = kv4_scale_pair(prmt(ks[0], ks[1], (b + 2) | (b + 6) << 4));
          ka[0] = prmt(a2, a2, 0x1010); ka[1] = prmt(a2, a2, 0x3232);
          kb[0] = prmt(b2, b2, 0x1010); kb[1] = prmt(b2, b2, 0x3232);
        } else {
          const uint32_t b = quad & 1;
          const uint32_t two = kv4_scale_pair(prmt(ks[0], 0, b | (b + 2) << 4));
          ka[0] = ka[1] = prmt(two, two, 0x1010);
          kb[0] = kb[1] = prmt(two, two, 0x3232);
        }
        float s1[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < W; ++w) {
          uint32_t a[4], b[4];
          kv4_decode(kr[0][w], a);
          kv4_decode(kr[1][w], b);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] = mul_f16x2(a[e], ka[w >> 1]);
            b[e] = mul_f16x2(b[e], kb[w >> 1]);
          }
          mma_16x8x16(s1, a[0], b[0], a[1], b[1], qh[2 * w][0], qh[2 * w][1]);
          mma_16x8x16(s2, a[2], b[2], a[3], b[3], qh[2 * w + 1][0], qh[2 * w + 1][1]);
          if constexpr (F32) {
            mma_16x8x16(s1, a[0], b[0], a[1], b[1], ql[2 * w][0], ql[2 * w][1]);
            mma_16x8x16(s2, a[2], b[2], a[3], b[3], ql[2 * w + 1][0], ql[2 * w + 1][1]);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[h][e] = s1[e] + s2[e];
      }
      const bool all = left >= kUnit && seen_by_all > 0 && (pre || unit0 + kUnit <= seen_by_all);    // rows see all keys
      if (!all) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int vis = own_vis[e] <= 0 ? 0 : pre ? left : min(left, own_vis[e] - unit0);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (16 * h + k_off >= vis) s[h][e] = -INFINITY;          // chosen, not added: a NaN behind the mask is gone
            if (16 * h + k_off + 2 >= vis) s[h][2 + e] = -INFINITY;
          }
        }
      }
      float mx[2];
      bool grow = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[e] = fmaxf(fmaxf(s[0][e], s[0][2 + e]), fmaxf(s[1][e], s[1][2 + e])) * sc[e];
        grow |= mx[e] - m[e] > kRescale;
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 4));
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 8));
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 16));
          const float f = mx[e] > m[e] ? ex2(m[e] - mx[e]) : 1.f;
          m[e] = fmaxf(m[e], mx[e]);
          l[e] *= f;
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            o[t][e] *= f;
            o[t][2 + e] *= f;
          }
        }
      }
      uint32_t ph[2][2], pl[2][2];           // keys x rows -> rows x keys, the B operand of O^T
      const float neg[2] = {m[0] == -INFINITY ? kShift : kShift - m[0], m[1] == -INFINITY ? kShift : kShift - m[1]};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float a = ex2(fmaf(s[h][2 * y], sc[0], neg[0])), b = ex2(fmaf(s[h][2 * y + 1], sc[1], neg[1]));
          l[0] += a;
          l[1] += b;
          const uint32_t both = f16x2(a, b);
          ph[h][y] = transpose8(both);
          if constexpr (F32) {
            const float2 r = halves(both);
            pl[h][y] = transpose8(f16x2(a - r.x, b - r.y));
          }
        }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t vr[4][VW];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t from = base + v_at + (16 * h + x) * 16 * NC;
          if constexpr (W == 4) {
            const uint2 w = ld_shared8(from);
            vr[x][0] = w.x; vr[x][1] = w.y;
          } else if constexpr (W == 2) {
            vr[x][0] = ld_shared4(from);
          } else {
            vr[x][0] = ld_shared2(from);
          }
        }
        uint32_t vs = ld_shared4(base + vs_at + h * 32 * NC);
        if (!v_has) vs = 0;
        if (!all) {
          const int mine = left - 16 * h - 4 * c;          // keys past the end: zero
          if (mine < 4) vs &= (1u << 8 * max(mine, 0)) - 1;
          const uint32_t odd = kv4_nan_scales(vs);
          if (__any_sync(0xffffffffu, odd)) {              // rare: NaN values that some row does not see are taken out
#pragma unroll 1
            for (int x = 0; x < 4; ++x) {
              const int key = unit0 + 16 * h + 4 * c + x;
              if (!pre && (odd >> (8 * x + 7) & 1u) && key >= seen_by_all) {
                vs &= ~(0xffu << 8 * x);
                atomicMin(&sh.nan_key[k & 3][v_block], key);
              }
            }
          }
        }
        const uint32_t v01 = kv4_scale_pair(vs), v23 = kv4_scale_pair(vs >> 16);
#pragma unroll
        for (int j = 0; j < VW; ++j) {
          uint32_t a0[4], a1[4], a2[4], a3[4];           // elements 2 b, 2 b + 1 of keys 0, 1; of keys 2, 3
          constexpr uint32_t lo = 0x0f0f0f0fu;
          kv4_decode((vr[0][j] & lo) | ((vr[1][j] << 4) & ~lo), a0);
          kv4_decode(((vr[0][j] >> 4) & lo) | (vr[1][j] & ~lo), a1);
          kv4_decode((vr[2][j] & lo) | ((vr[3][j] << 4) & ~lo), a2);
          kv4_decode(((vr[2][j] >> 4) & lo) | (vr[3][j] & ~lo), a3);
#pragma unroll
          for (int b = 0; b < (W == 1 ? 2 : 4); ++b) {
            const int t = 4 * j + b;
            const uint32_t w0 = mul_f16x2(a0[b], v01), w1 = mul_f16x2(a1[b], v01), w2 = mul_f16x2(a2[b], v23),
                           w3 = mul_f16x2(a3[b], v23);
            if constexpr (F32) {
              // summed apart: the products' own accumulation cuts bits off, which would add up over long keys
              float z[4] = {0.f, 0.f, 0.f, 0.f};
              mma_16x8x16(z, w0, w1, w2, w3, pl[h][0], pl[h][1]);
              mma_16x8x16(z, w0, w1, w2, w3, ph[h][0], ph[h][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[t][e] += z[e];
            } else {
              mma_16x8x16(o[t], w0, w1, w2, w3, ph[h][0], ph[h][1]);
            }
          }
        }
      }
      __syncwarp();                          // the buffer may be filled again
      buffer ^= 1;
      if (warp == 0 && !asked) {             // once an item: the claim has come back
        word = word_of(own_item(__shfl_sync(0xffffffffu, claimed, 0)));
        asked = true;
      }
      u = next;
    }
    if (warp == 0) {
      if (!asked) word = word_of(own_item(__shfl_sync(0xffffffffu, claimed, 0)));
      publish(k + 2, word);
    }

    // ---- the warps' parts.  One barrier an item: the parts of at most 4 rows take turns in the two halves of their room, and
    // while the last warps join them, the others go on.
    if (units < 2) asm volatile("cp.async.wait_all;" ::: "memory");        // the next item's queries (the waits above: one unit late)
    if (nrows > 4 && few_before) __syncthreads();          // the item before's parts have been read
    few_before = nrows <= 4;
    const int half = nrows > 4 ? 0 : (k & 1) * 4;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], x);
      const int r = 2 * c + e;
      if (r >= nrows) continue;
      if (quad == 0) sh.ml[warp][half + r] = make_float2(m[e], l[e]);
      float* dst = po + (warp * 8 + half + r) * kFewPitch + 4 * W * quad;
#pragma unroll
      for (int t = 0; t < MT; t += 2)
        *reinterpret_cast<float4*>(dst + 2 * t) = make_float4(o[t][e], o[t][2 + e], o[t + 1][e], o[t + 1][2 + e]);
    }
    __syncthreads();
    const int r = 7 - warp, e0 = 4 * lane;
    if (r < nrows) {
      const int rr = row0 + r, tok = g.by_R(rr), h = it.group * g.R + rr - tok * g.R;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) top = fmaxf(top, sh.ml[w][half + r].x);
      const float ref = top == -INFINITY ? 0.f : top;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const float2 s = sh.ml[w][half + r];
        if (s.y == 0.f) continue;                      // nothing seen by this warp
        const float f = s.x == -INFINITY ? 1.f : ex2(s.x - ref);
        sum += f * s.y;
        const float4 v = *reinterpret_cast<const float4*>(po + (w * 8 + half + r) * kFewPitch + min(e0, 32 * W - 4));
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
        if (sh.nan_key[k & 3][e0 / 16] < vis) acc.x = acc.y = acc.z = acc.w = __int_as_float(0x7fc00000);
        if (it.part_row >= 0) {
          *reinterpret_cast<float4*>(g.part_out + (int64_t)(it.part_row + r) * g.d + e0) = acc;
        } else if constexpr (F32) {
          *reinterpret_cast<float4*>(static_cast<float*>(p.out) + ((int64_t)tok * g.H + h) * g.d + e0) = acc;
        } else {
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + ((int64_t)tok * g.H + h) * g.d + e0) =
              make_uint2(bf16x2(acc.x, acc.y), bf16x2(acc.z, acc.w));
        }
      }
      if (lane == 0) {
        const float lse = sum == 0.f ? -INFINITY : (ref - kShift) * kLn2 + logf(sum);
        if (it.part_row >= 0) g.part_lse[it.part_row + r] = lse;
        else if (p.lse) p.lse[(int64_t)tok * g.H + h] = lse;
      }
    }
    if (nrows > 4) __syncthreads();
  }
  // every claim of this CTA has been made: the last one leaves the counters as the next call needs them
  if (fits && threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(&g.head->few_done, 1u) == gridDim.x - 1) {
      g.head->few_claimed = 0;
      g.head->few_done = 0;
    }
  }
  if (p.overlap) pdl_wait();
}

// ---------------------------------------------------------------- row tiles
// Items of more rows, bf16: persistent, one CTA per SM, on the tensor cores.  A work item is up to 256 packed rows
// against a run of 128-key tiles; CTAs claim them from a counter.  Two streams of 128 rows alternate on the tensor
// core, each with two score buffers of half a tile.
//   warps 0-3, 4-7   softmax of stream 0 / 1, one thread per row
//   warp 8           claims items, and looks at the clock
//   warps 9, 10      issue the products of stream 0 / 1:  S = Q K^T (both from shared memory) and O += P V (P from
//                    tensor memory)
//   warp 11          copies tiles as they lie in the cache, keys and values into a buffer each, through the page tables
//   warps 12-15      output, while the softmax goes on to the next item
//   warps 16-19      keys, and warps 20-23 values: from that buffer to fp16 tiles in the 128-byte swizzle that the
//                    products read
//                    and the next item's queries
// Tensor memory is laid out as in attention.cu.
//
// A thread of warps 16-23 has a chunk (32 elements) of four neighbouring keys: 16 bytes of each and one word of scales
// for each of the two blocks.  The buffer is free again, and the next tile on its way, as soon as that is converted.
//
// A prompt of 8192 tokens, 32 / 8 heads of 128: 440 us, 1.25 PFLOP/s; 64 of 1024 tokens, 16 / 8 heads: 372 us (a cache in
// bf16: 350 and 277 us).  The conversion is what that costs more: it writes a tile that TMA would have written, through two
// warpgroups, whose loads and stores share an SM's issue slots and shared memory with the softmax.  No unit is full (4096
// tokens: tensor pipe 43 % of the cycles, issue slots 50 %); what is left is the tiles' chain of waits.  What counted (8192
// tokens): a warpgroup each for keys and values (967 -> 559 us); registers dealt so that tile walks spill nothing, as next
// to 220 KB of shared memory there is hardly any first cache (-> 498); tiles copied as they lie instead of loaded into
// registers a tile ahead (-> 470); shared-memory accesses that meet in no bank (-> 459); 76 KB of code instead of 113, for
// the instruction cache (-> 439; 64 x 1024 tokens 568 -> 438).  Measured slower: whole tiles of scores for half tiles
// (458 -> 515), values before queries, page look-ups a tile ahead.
constexpr int kTileThreads = 768;
// Registers of the warpgroups: 80 for each of 768 threads at the launch.
constexpr int kLaunchRegs = 80, kSoftmaxRegs = 112, kIssueRegs = 64, kOutRegs = 64, kConvertRegs = 64;
static_assert(2 * kSoftmaxRegs + kIssueRegs + kOutRegs + 2 * kConvertRegs <= 6 * kLaunchRegs, "what the launch owns");

// Ring stages that fit beside the query tiles, the copies and the staging.
__host__ __device__ constexpr int kv4_stages(int halves) { return halves == 2 ? 4 : 6; }

struct alignas(16) TileBars {
  uint64_t kv_ready[2][6], kv_empty[6];      // kv_ready: each stream's own tiles, in its own order
  uint64_t raw_full[2], raw_empty[2];        // keys, values
  uint64_t q_full[2], q_empty[2], s_full[2][2], p_full[2][2], pv_done[2][2], o_full[2], o_empty[2];   // [stream][score buffer]
  uint64_t stat_full[2], stat_empty[2], drain[2], slot_full[kSlots], slot_empty[kSlots];
  alignas(16) WorkItem slot[kSlots];         // row0 < 0: no more
  int nan_key[kSlots][8];                    // the first key, not seen by every row, whose values of a block are NaN
  uint32_t tmem;
  int abort_flag;
};
constexpr int kTileStage = 4 * 32 * 64;                // output staging: 32 rows of 64 bytes for each output warp
constexpr int kTileSmem = 1024 + 6 * 2 * kHalfBytes + 2 * raw_bytes(4) + kTileStage + 2 * kRows * 8 + kSlots * 2 * kRows * 4 +
                          (int)sizeof(TileBars);
static_assert(kTileSmem <= kSmemMax, "fits an SM");

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

template <int NC>
__global__ void __launch_bounds__(kTileThreads, 1)
kv4_tile_kernel(const __grid_constant__ Kv4AttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  constexpr int kHalves = NC > 2 ? 2 : 1, kD = 32 * NC, kSlices = 2 * NC, kStages = kv4_stages(kHalves);
  constexpr int kTileBytes = kHalves * kHalfBytes, kRaw = raw_bytes(NC);
  const StepGeom& g = p.g;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_smem = smem;                              // two row tiles
  uint8_t* kv_smem = smem + 2 * kTileBytes;
  uint8_t* raw_smem = kv_smem + kStages * kTileBytes;                  // keys, values: codes, then scales
  uint8_t* out_smem = raw_smem + 2 * kRaw;
  float2* stats = reinterpret_cast<float2*>(out_smem + kTileStage);     // [stream][row]: (m, l)
  float* q_factor = reinterpret_cast<float*>(stats + 2 * kRows);        // [slot][stream][row]: of the scores
  TileBars* bars = reinterpret_cast<TileBars*>(q_factor + kSlots * 2 * kRows);
  uint32_t* status = &g.head->status;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars->kv_ready[0][i], 4);
      mbar_init(&bars->kv_ready[1][i], 4);
      mbar_init(&bars->kv_empty[i], 2);      // the streams; the converting warps stand in for one that does not use it
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->q_full[s], 8);
      mbar_init(&bars->q_empty[s], 1);
      mbar_init(&bars->drain[s], 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bars->s_full[s][b], 1);
        mbar_init(&bars->p_full[s][b], 4);
        mbar_init(&bars->pv_done[s][b], 1);
      }
      mbar_init(&bars->o_full[s], 1);
      mbar_init(&bars->stat_full[s], 4);
      mbar_init(&bars->stat_empty[s], 4);
      mbar_init(&bars->o_empty[s], 4);
      mbar_init(&bars->raw_full[s], 1);
      mbar_init(&bars->raw_empty[s], 4);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&bars->slot_full[i], 1);
      mbar_init(&bars->slot_empty[i], 23);   // softmax warps 8, output 4, product 2, converting 8, copying 1
    }
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&bars->tmem, kTmemCols);
    tmem_relinquish();
  }
  pdl_enter();
  if (p.overlap) pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  const bool fits = plan_matches(g);
  const bool good = fits && g.head->n_items >= 0;
  // a plan of other shapes, or of a malformed step: said by every call, as the status is cleared when it is read
  if (!good && threadIdx.x == 0) latch_status(status, fits ? kStatusRange : kStatusInvalid);

  if (warp >= 8 && warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 8) {
      // ---------------------------------------------------------- items
      // Claimed one ahead: the first of a CTA is its own number, the others come from a counter.
      const int end = good ? g.head->tile_end : 0;
      auto publish = [&](int k, int item) {
        wait_on(&bars->slot_empty[k % kSlots], ((k / kSlots) & 1) ^ 1, bars);
        int* d = reinterpret_cast<int*>(&bars->slot[k % kSlots]);
        if (lane < (int)(sizeof(WorkItem) / 4))
          d[lane] = item < end ? reinterpret_cast<const int*>(g.items + item)[lane] : -1;
        if (lane < 8) bars->nan_key[k % kSlots][lane] = INT32_MAX;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->slot_full[k % kSlots]);
      };
      // An item's queries on their way to the second cache, by an item or so before they are read (64 sequences of 1024
      // tokens: 404 -> 388 us).  The first item's are read at once; asking for them twice cost 3 % of short items.
      auto fetch_queries = [&](int k) {
        const WorkItem& it = bars->slot[k % kSlots];
#pragma unroll 1
        for (int r = it.row0 + lane; r < it.row0 + it.nrows; r += 32) {
          const int tok = g.by_R(r);
          const uint16_t* const from = static_cast<const uint16_t*>(p.q) + (int64_t)tok * p.q_stride +
                                       (it.group * g.R + r - tok * g.R) * g.d;
          prefetch(from);
          if (NC > 2) prefetch(from + 64);
        }
      };
      auto pass_few = [&](int i) {           // past the other kernel's items
        while (i < end && g.items[i].alt == 2) {
          int next = 0;
          if (lane == 0) next = gridDim.x + (int)atomicAdd(&g.head->claimed, 1u);
          i = __shfl_sync(0xffffffffu, next, 0);
        }
        return i;
      };
      int i = pass_few(blockIdx.x), k = 0;
      publish(0, i);
      while (i < end && !gave_up(bars)) {
        int next = 0;
        if (lane == 0) next = gridDim.x + (int)atomicAdd(&g.head->claimed, 1u);
        if (k) fetch_queries(k);
        i = pass_few(__shfl_sync(0xffffffffu, next, 0));
        publish(++k, i);
      }
      // to the end of the last item (the others' slots were empty when theirs were filled again)
      for (int x = max(k - kSlots + 1, 0); x < k; ++x) wait_on(&bars->slot_empty[x % kSlots], (x / kSlots) & 1, bars);
    } else if (warp < 11) {
      // ---------------------------------------------------------- products
      // The whole warp walks, one lane issues; see attention.cu.
      const int s = warp - 9;
      const uint32_t id_qk = idesc_f16(kRows, kHalfKeys, 0);
      const uint32_t id_pv = idesc_f16(kRows, (uint32_t)kD, 0) | (1u << 16);   // V is N-major
      const uint64_t dq = smem_desc_k_sw128(smem_u32(q_smem + s * kTileBytes)), dk0 = smem_desc_k_sw128(smem_u32(kv_smem));
      const uint64_t dv0 = smem_desc_mn_sw128(smem_u32(kv_smem), kHalfBytes);
      constexpr uint32_t tile_step = kTileBytes >> 4;
      const uint32_t tS = tmem + s * kKeyTile, tO = tmem + kColO + s * kRows;
      uint32_t q_ph = 0, p_ph = 0, oe_ph = 0;
      Ring base, turn;      // the item's first ring stage; the stream's next turn
      for (int k = 0; slot_ready(bars, k); ++k) {
        const WorkItem it = uniform_item(bars, k);
        slot_done(bars, k);
        const int n = s ? it.n1 : it.n0, tiles = item_tiles(it);
        Ring rk = base;                                   // stage of the stream's next keys
        base.advance(2 * tiles, kStages);
        if (n == 0) continue;
        if (it.alt && s) rk.skip(2, kStages);
        Ring rv = rk, tk = turn, tv = turn;
        rv.skip(1, kStages);
        tv.skip(1, kStages);
        turn.advance(2 * n, kStages);
        const int stride = it.alt ? 4 : 2;                // ring steps from tile to tile of the stream
        const int ti_step = it.alt ? 2 : 1, limit = stream_limit(it, g, s);
        int ti = tile_of(it, s, 0), keys = 0, next_keys = stream_keys(it, g, ti, limit);
        await(&bars->q_full[s], q_ph, bars);
        q_ph ^= 1u;
        // Scores run a tile ahead of the values' products, in half tiles (step 0: scores alone); one copy of the loop's
        // body, and no unrolling, for the instruction cache's sake.
#pragma unroll 1
        for (int step = 0; step <= n; ++step) {
          const bool more = step < n;
          if (step) await(&bars->kv_ready[s][tv.s], tv.ph, bars);
          if (more) await(&bars->kv_ready[s][tk.s], tk.ph, bars);
          if (step == 1) {
            await(&bars->o_empty[s], oe_ph ^ 1u, bars);
            oe_ph ^= 1u;
          }
          tc_fence_after();
          const uint64_t dv = dv0 + rv.s * tile_step, dk = dk0 + rk.s * tile_step;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const int from = h * kHalfKeys;
            if (step) {
              await(&bars->p_full[s][h], p_ph, bars);
              tc_fence_after();
            }
            if (elect_one()) {
              if (step) {
                issue_values((keys - from + 15) >> 4, tO, tS + from, dv + (from * 128 >> 4), id_pv, h > 0 || step > 1);
                mma_commit(&bars->pv_done[s][h]);
                if (h == 1) mma_commit(&bars->kv_empty[rv.s]);
              }
              if (more) {
                if (next_keys > from) issue_scores<kSlices>(0, tS + from, dq, dk + (from * 128 >> 4), id_qk);
                mma_commit(&bars->s_full[s][h]);
                if (h == 1) mma_commit(&bars->kv_empty[rk.s]);
                if (h == 1 && step == n - 1) mma_commit(&bars->q_empty[s]);      // the item's last scores
              } else if (h == 1) {
                mma_commit(&bars->o_full[s]);
              }
            }
            __syncwarp();
          }
          if (step) {
            p_ph ^= 1u;
            rv.skip(stride, kStages);
            tv.skip(2, kStages);
          }
          rk.skip(stride, kStages);
          tk.skip(2, kStages);
          keys = next_keys;
          ti += ti_step;
          next_keys = step + 1 < n ? stream_keys(it, g, ti, limit) : 0;
        }
      }
      if (elect_one()) {
        mma_commit(&bars->drain[s]);
        const uint64_t t0 = global_timer_ns();
        while (!mbar_test_wait(&bars->drain[s], 0) && global_timer_ns() - t0 < 2000000000ull) {}
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- copies
      uint32_t ph = 0, copied = 0;
      for (int k = 0; slot_ready(bars, k); ++k) {
        const WorkItem& it = bars->slot[k % kSlots];
        const int n = item_tiles(it);
#pragma unroll 1
        for (int u = 0; u < n && !gave_up(bars); ++u) {
          const TileShare x = tile_share<NC>(p, it, it.t0 + u, status);
#pragma unroll 1
          for (int value = 0; value < 2; ++value) {
            await(&bars->raw_empty[value], ph ^ 1u, bars);
            if (lane == 0) mbar_arrive_expect_tx(&bars->raw_full[value], x.total);
            __syncwarp();
            if (x.bytes)
              copy_bulk(smem_u32(raw_smem) + value * kRaw + x.to, (value ? p.pool.v : p.pool.k) + x.from, x.bytes,
                        &bars->raw_full[value]);
            __syncwarp();
          }
          ph ^= 1u;
          copied = 1;
        }
        slot_done(bars, k);
      }
      if (copied) {                          // shared memory goes away: the last copies have to be there
        for (int value = 0; value < 2; ++value) {
          const uint64_t t0 = global_timer_ns();
          while (!mbar_test_wait(&bars->raw_full[value], ph ^ 1u) && global_timer_ns() - t0 < 2000000000ull) {}
        }
      }
      __syncwarp();
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int s = warp >> 2;                         // stream
    const int row = threadIdx.x & (kRows - 1);
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + s * kKeyTile;
    const uint32_t tO = tmem + lane_base + kColO + s * kRows;
    uint32_t s_ph = 0, st_ph = 0;
    for (int k = 0; slot_ready(bars, k); ++k) {
      const WorkItem it = load_item(&bars->slot[k % kSlots]);
      const int n = s ? it.n1 : it.n0;
      const int r_item = row + (it.alt ? 0 : s * kRows);
      const bool live = r_item < it.nrows;
      const bool warp_live = (row & ~31) + (it.alt ? 0 : s * kRows) < it.nrows;
      const int tok = g.by_R(it.row0 + r_item);
      // own keys in view of this row; padding rows see nothing at all
      const int own_vis = it.seq < 0 ? 0 : tok + it.own_off + 1;
      const bool blind = !live || (it.seq >= 0 && own_vis <= 0);
      float m = -INFINITY, l = 0.f, sc = 0.f;        // m: the maximum (log2) that O and l refer to
      const int limit = stream_limit(it, g, s);
      for (int j = 0; j < n; ++j) {
        const int ti = tile_of(it, s, j);
        int key0;
        const int keys = tile_keys(it, g, ti, &key0), used_keys = stream_keys(it, g, ti, limit);
        int vis_tile = ti < it.np ? keys : min(keys, own_vis - key0);      // keys in view of this row
        if (blind) vis_tile = 0;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const int vis = vis_tile - h * kHalfKeys;
          const bool masked = __any_sync(0xffffffffu, vis < kHalfKeys);
          const uint32_t tB = tS + h * kHalfKeys;
          await(&bars->s_full[s][h], s_ph, bars);
          if (j == 0 && h == 0) sc = blind ? 1.f : q_factor[((k % kSlots) * 2 + s) * kRows + row];    // there before the queries
          if (warp_live && h * kHalfKeys < used_keys) {
            tc_fence_after();
            uint32_t v[kHalfKeys];
            tmem_ld32(tB, v);
            tmem_ld32(tB + 32, v + 32);
            tmem_ld_wait();
            if (masked) {
#pragma unroll
              for (int c = 0; c < kHalfKeys; ++c)
                if (c >= vis) v[c] = 0xff800000u;      // -inf: chosen, not added, so a NaN behind the mask is gone
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < kHalfKeys; c += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], __uint_as_float(v[c + e]), __uint_as_float(v[c + e + 4]));
            const float m_new = fmaxf(m, max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * sc);
            if (j == 0 && h == 0) {
              m = m_new;
            } else {
              const bool grow = m_new - m > kRescale;
              if (__any_sync(0xffffffffu, grow)) {
                // O is this warp's once the latest product is done (those before it are: these scores were
                // issued after them)
                await(&bars->pv_done[s][h ^ 1], h ? s_ph : s_ph ^ 1u, bars);
                tc_fence_after();
                const float f = grow ? ex2(m - m_new) : 1.f;
                if (grow) m = m_new;
                l *= f;
#pragma unroll 1
                for (int c = 0; c < kD; c += 16) {
                  uint32_t o[16];
                  tmem_ld16(tO + c, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                  tmem_st16(tO + c, o);
                }
              }
            }
            const float neg = m == -INFINITY ? kShift : kShift - m;
            const uint64_t sc2 = pk(sc, sc), ng2 = pk(neg, neg);
            uint64_t sum0 = pk(0.f, 0.f), sum1 = sum0;
            uint32_t w[kHalfKeys / 2];
#pragma unroll
            for (int e = 0; e < kHalfKeys / 2; ++e) {
              const float2 x = unpk(fma2(pk_u(v[2 * e], v[2 * e + 1]), sc2, ng2));
              const float a = ex2(x.x), b = ex2(x.y);
              if (e & 1) sum1 = add2(sum1, pk(a, b));
              else sum0 = add2(sum0, pk(a, b));
              w[e] = f16x2(a, b);
            }
            tmem_st32(tB, w);
            const float2 z = unpk(add2(sum0, sum1));
            l += z.x + z.y;
            tmem_st_wait();
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->p_full[s][h]);
        }
        s_ph ^= 1u;
      }
      if (n > 0) {
        // (m, l) to the output warps, once they have taken the item's before
        await(&bars->stat_empty[s], st_ph ^ 1u, bars);
        st_ph ^= 1u;
        stats[s * kRows + row] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->stat_full[s]);
      }
      slot_done(bars, k);
    }
  } else if (warp < 16) {
    // ------------------------------------------------------------ output
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOutRegs));
    const int row = threadIdx.x & (kRows - 1);
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    // 16 bytes of row `row` of a warp's 32 rows of 64 bytes, in place c of 4: eight rows' stores meet in no bank
    auto staged = [&](int row, int c) { return smem_u32(out_smem) + (warp & 3) * 2048 + row * 64 + ((c ^ (row >> 1 & 3)) << 4); };
    uint32_t ph = 0;                                 // bit s: stream s
    for (int k = 0; slot_ready(bars, k); ++k) {
      const WorkItem it = load_item(&bars->slot[k % kSlots]);
      const bool merging = it.alt && it.n1 > 0;      // both streams hold parts of the same rows
#pragma unroll 1
      for (int s = 0; s < (it.alt ? 1 : 2); ++s) {
        const int n = s ? it.n1 : it.n0;
        const uint32_t tO = tmem + lane_base + kColO + s * kRows;
        const int r_item = row + s * kRows;
        const int rr = it.row0 + r_item;
        const bool live = r_item < it.nrows, warp_live = (row & ~31) + s * kRows < it.nrows;
        const int tok = g.by_R(rr);
        float m = -INFINITY, l = 0.f, f0 = 1.f, f1 = 0.f;
        auto take = [&](int x) {                     // stream x's (m, l); its O is complete then
          await(&bars->stat_full[x], (ph >> x) & 1u, bars);
          const float2 v = stats[x * kRows + row];
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->stat_empty[x]);
          await(&bars->o_full[x], (ph >> x) & 1u, bars);
          ph ^= 1u << x;
          return v;
        };
        if (n > 0) {
          const float2 v = take(s);
          m = v.x;
          l = v.y;
        }
        if (merging) {
          const float2 o = take(1);
          const float mm = fmaxf(m, o.x);
          if (mm != -INFINITY) {
            f0 = ex2(m - mm);
            f1 = ex2(o.x - mm);
          }
          l = l * f0 + o.y * f1;
          m = mm;
        }
        auto free_o = [&]() {                        // for the next item's products
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (n > 0) mbar_arrive(&bars->o_empty[s]);
            if (merging) mbar_arrive(&bars->o_empty[1]);
          }
        };
        if (!warp_live) {
          free_o();
          continue;
        }
        const float inv = l > 0.f || l != l ? p.v_scale / l : 0.f;      // a row without keys: zero
        f0 *= inv;
        f1 *= inv;
        tc_fence_after();
        const int h = it.group * g.R + rr - tok * g.R;
        const bool direct = it.part_row < 0;
        // 64 bytes of each row at a time go through shared memory, 32 bf16 columns of the output or 16 fp32 columns of a
        // partial row, so that four lanes store two whole sectors of a row; the rows' numbers come from their lanes.
        const int mine = !live ? -1 : direct ? tok * g.H + h : it.part_row + r_item;
        const bool none = l == 0.f, some_none = __any_sync(0xffffffffu, none);   // rows without keys are zero
        // values that are NaN and were taken out of the tiles: of the rows that see their keys
        const int* nan_key = bars->nan_key[k % kSlots];
        const bool some_nan = __any_sync(0xffffffffu, nan_key[lane & 7] != INT32_MAX);
        const int own_vis = it.seq < 0 ? 0 : tok + it.own_off + 1;
#pragma unroll 1
        for (int c = 0; c < kD; c += 16) {
          uint32_t v[16];
          if (n > 0) tmem_ld16(tO + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f0);
          if (merging) {
#pragma unroll
            for (int x = 0; x < 16; x += 8) {
              uint32_t w[8];
              tmem_ld8(tO + kRows + c + x, w);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 8; ++e)
                v[x + e] = __float_as_uint(__uint_as_float(v[x + e]) + __uint_as_float(w[e]) * f1);
            }
          }
          if (some_none) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = none ? 0u : v[e];
          }
          if (some_nan && nan_key[c / 16] < own_vis) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0x7fc00000u;
          }
          if (c + 16 >= kD) free_o();
          if (direct) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
              st_shared16(staged(lane, (c & 16) / 8 + q),
                          make_uint4(bf16x2(__uint_as_float(v[8 * q]), __uint_as_float(v[8 * q + 1])),
                                     bf16x2(__uint_as_float(v[8 * q + 2]), __uint_as_float(v[8 * q + 3])),
                                     bf16x2(__uint_as_float(v[8 * q + 4]), __uint_as_float(v[8 * q + 5])),
                                     bf16x2(__uint_as_float(v[8 * q + 6]), __uint_as_float(v[8 * q + 7]))));
            if (!(c & 16)) continue;
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              st_shared16(staged(lane, q), make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
          }
          __syncwarp();
          uint8_t* const to = direct ? static_cast<uint8_t*>(p.out) : reinterpret_cast<uint8_t*>(g.part_out);
          const int row_bytes = g.d * (direct ? 2 : 4), byte = (direct ? (c & ~31) * 2 : c * 4) + (lane & 3) * 16;
#pragma unroll
          for (int r0 = 0; r0 < 32; r0 += 8) {
            const int r = r0 + (lane >> 2);
            const int which = __shfl_sync(0xffffffffu, mine, r);
            if (which >= 0 && byte < row_bytes)
              *reinterpret_cast<uint4*>(to + (int64_t)which * row_bytes + byte) = ld_shared16(staged(r, lane & 3));
          }
          __syncwarp();
        }
        if (live) {
          const float lse = l == 0.f ? -INFINITY : (m - kShift) * kLn2 + logf(l);
          if (!direct) g.part_lse[mine] = lse;
          else if (p.lse) p.lse[mine] = lse;
        }
      }
      slot_done(bars, k);
    }
  } else {
    // ------------------------------------------------------------ keys and values
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvertRegs));
    const bool value = warp >= 20;
    const int ct = threadIdx.x & 127, cw = warp & 3;
    const bool busy = ct < 32 * NC;                  // a chunk c of keys 4 j .. 4 j + 3
    const int j = ct / NC, c = ct - j * NC;
    const bool second = 32 * c + 16 < g.d;           // the chunk's other block holds elements
    // A thread takes its keys in an order of its own, i ^ o for i = 0 .. 3, so that a quarter warp's 16-byte loads (two keys
    // beside each other, four chunks) and stores (a swizzled row's pieces) meet in no bank.
    const int o = NC > 2 ? (c >> 1) << 1 | (j & 1) : NC == 2 ? j & 3 : j >> 1 & 3;
    const uint32_t place = ((((c & 1) ^ (j & 1)) << 2) ^ o) << 4;
    const uint32_t pick = o | (4 + o) << 4;          // of a key's two scales
    const uint32_t to0 = smem_u32(kv_smem) + (c >> 1) * kHalfBytes + 4 * j * 128;
    const uint32_t raw = smem_u32(raw_smem) + value * kRaw;
    Ring r;                                          // keys and values take the ring's stages in turns
    r.s = value;
    int turn0 = value, turn1 = value;                // of the streams' own tiles
    const uint32_t at = raw + (4 * j * NC + c) * 16, sat = raw + kKeyTile * 16 * NC + (2 * j * NC + 2 * c) * 4;
    // An item's queries, a row tile a stream (the same one, where both hold the same rows), by these eight warps, 8 lanes (4)
    // to a row: copied as they are to where they will be, all on their way at once, and made fp16 there.
    auto queries = [&](int k, int w8, uint32_t& q_ph) {
      constexpr int kLanes = NC > 2 ? 8 : 4, kPer = 32 / kLanes, kChunks = (4 * NC + kLanes - 1) / kLanes, kTasks = kRows / kPer / 8;
      const WorkItem& it = bars->slot[k % kSlots];
      const int alt = it.alt, n0 = it.n0, n1 = it.n1;
      const int lc = lane % kLanes, first_row = w8 * kTasks * kPer + lane / kLanes;
      const bool twice = alt && n1 > 0;
      // chunk lc + y kLanes of row `row` of tile x
      auto place = [&](int row, int x, int y) {
        const uint32_t at = smem_u32(q_smem) + x * kTileBytes + row * 128 + ((lc ^ (row & 7)) << 4);
        return NC > 2 ? at + y * kHalfBytes : at ^ (uint32_t)(y << 6);
      };
#pragma unroll 1
      for (int x = 0; x < (alt ? 1 : 2); ++x) {
        if ((x ? n1 : n0) == 0) continue;
        await(&bars->q_empty[x], ((q_ph >> x) & 1u) ^ 1u, bars);
        q_ph ^= 1u << x;
        if (twice) {
          await(&bars->q_empty[1], ((q_ph >> 1) & 1u) ^ 1u, bars);
          q_ph ^= 2u;
        }
#pragma unroll 1
        for (int i = 0; i < kTasks; ++i) {
          const int row = first_row + i * kPer, rr = it.row0 + x * kRows + row, tok = g.by_R(rr);
          const bool live = x * kRows + row < it.nrows;
          const uint16_t* from = static_cast<const uint16_t*>(p.q);
          if (live) from += (int64_t)tok * p.q_stride + (it.group * g.R + rr - tok * g.R) * g.d;
#pragma unroll
          for (int y = 0; y < kChunks; ++y) {
            const int e = (lc + y * kLanes) * 8;
            if (e < kD) copy16(place(row, x, y), e < g.d ? from + e : from, live && e < g.d);
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
        for (int i = 0; i < kTasks; ++i) {
          const int row = first_row + i * kPer;
          uint4 w[kChunks];
          uint32_t top2 = 0;
#pragma unroll
          for (int y = 0; y < kChunks; ++y) {
            w[y] = make_uint4(0, 0, 0, 0);
            if ((lc + y * kLanes) * 8 < kD) w[y] = ld_shared16(place(row, x, y));
            top2 = max_u16x2(top2, max_u16x2(w[y].x & 0x7fff7fffu, w[y].y & 0x7fff7fffu));
            top2 = max_u16x2(top2, max_u16x2(w[y].z & 0x7fff7fffu, w[y].w & 0x7fff7fffu));
          }
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) top2 = max_u16x2(top2, __shfl_xor_sync(0xffffffffu, top2, o));
          // bf16 to fp16 by its bits: `less` from the exponent, so that the largest element's is 28 at most; what falls out
          // of fp16's range below (2^27 under the largest) becomes 0 or some subnormal number.  A row with an infinity or
          // a NaN has no scores.
          const uint32_t e = max(max(top2 & 0xffffu, top2 >> 16) >> 7, 28u), less2 = (e - 28) * 0x00800080u;
          const float inverse = e == 255 ? __int_as_float(0x7fc00000) : __uint_as_float((e - 13) << 23);
          auto bits = [&](uint32_t v) { return (max_u16x2(v & 0x7fff7fffu, less2) - less2) << 3 | (v & 0x80008000u); };
#pragma unroll
          for (int y = 0; y < kChunks; ++y) {
            if ((lc + y * kLanes) * 8 >= kD) continue;
            const uint4 h = make_uint4(bits(w[y].x), bits(w[y].y), bits(w[y].z), bits(w[y].w));
            st_shared16(place(row, x, y), h);
            if (twice) st_shared16(place(row, x, y) + kTileBytes, h);
          }
          if (lc == 0) {
            float* const f = q_factor + (k % kSlots) * 2 * kRows + row;
            f[x * kRows] = inverse * p.score_log2;
            if (twice) f[kRows] = inverse * p.score_log2;
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars->q_full[x]);
          if (twice) mbar_arrive(&bars->q_full[1]);
        }
      }
    };
    // An item's queries come behind its first keys and before its first values.
    uint32_t ph = 0, q_ph = 0;
    for (int k = 0; slot_ready(bars, k); ++k) {
      const WorkItem& it = bars->slot[k % kSlots];
      const int n = item_tiles(it), alt = it.alt;
#pragma unroll 1
      for (int step = 0; step < (n ? n + 1 : 0) && !gave_up(bars); ++step) {
        const int before = value ? 0 : 1;
        if (step == before) {
          queries(k, warp - 16, q_ph);
          continue;
        }
        const int u = step - (step > before);
        await(&bars->raw_full[value], ph, bars);
        ph ^= 1u;
        uint2 s = make_uint2(0, 0);
        if (busy) s = ld_shared8(sat);
        // ---- scales: none of what is past d or the last key
        const bool pre = it.t0 + u < it.np;
        int key0;
        const int left = tile_keys(it, g, it.t0 + u, &key0) - 4 * j;
        if (!second) s.y = 0;
        if (left < 4) {
          const uint32_t keep = (1u << 8 * max(left, 0)) - 1;
          s.x &= keep;
          s.y &= keep;
        }
        // values that are NaN and that some row does not see are taken out: 0 * NaN would stay
        if (value && __any_sync(0xffffffffu, !pre && (kv4_nan_scales(s.x) | kv4_nan_scales(s.y)) != 0)) {
          const int seen_by_all = all_see(load_item(&it), g);
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            const int key = key0 + 4 * j + i;
            if (key < seen_by_all) continue;
            const uint32_t byte = 0xffu << 8 * i, top = 0x80u << 8 * i;
            if (kv4_nan_scales(s.x) & top) {
              s.x &= ~byte;
              atomicMin(&bars->nan_key[k % kSlots][2 * c], key);
            }
            if (kv4_nan_scales(s.y) & top) {
              s.y &= ~byte;
              atomicMin(&bars->nan_key[k % kSlots][2 * c + 1], key);
            }
          }
        }
        // ---- to fp16
        await(&bars->kv_empty[r.s], r.ph ^ 1u, bars);
        if (busy) {
          const uint32_t to = to0 + r.s * kTileBytes;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t both = kv4_scale_pair(prmt(s.x, s.y, pick ^ (uint32_t)(i | i << 4)));
            const uint32_t s0 = prmt(both, both, 0x1010), s1 = prmt(both, both, 0x3232);
            const uint4 w = ld_shared16(at + (i ^ o) * 16 * NC);
            const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint32_t h[4];
              kv4_decode(words[y], h);
              const uint32_t sc = y < 2 ? s0 : s1;
              st_shared16(to + (i ^ o) * 128 + (place ^ (uint32_t)((y ^ i) << 4)),
                          make_uint4(mul_f16x2(h[0], sc), mul_f16x2(h[1], sc), mul_f16x2(h[2], sc), mul_f16x2(h[3], sc)));
            }
          }
        }
        fence_async_smem();
        __syncwarp();
        const bool use0 = alt ? !(u & 1) : u < it.n0, use1 = alt ? u & 1 : u < it.n1;
        if (lane == 0) {
          mbar_arrive(&bars->raw_empty[value]);
          if (use0) mbar_arrive(&bars->kv_ready[0][turn0]);
          if (use1) mbar_arrive(&bars->kv_ready[1][turn1]);
          if (cw == 0 && !(use0 && use1)) mbar_arrive(&bars->kv_empty[r.s]);
        }
        if (use0) turn0 = turn0 + 2 >= kStages ? value : turn0 + 2;
        if (use1) turn1 = turn1 + 2 >= kStages ? value : turn1 + 2;
        r.skip(2, kStages);
      }
      slot_done(bars, k);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && gave_up(bars)) latch_status(status, kStatusTimeout);
  // every claim of this CTA has been made: the last one leaves the counters as the next call needs them
  if (fits && threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(&g.head->done, 1u) == gridDim.x - 1) {
      g.head->claimed = 0;
      g.head->done = 0;
    }
  }
}

template <int NC>
aff_status launch_tile(const Kv4AttnParams& p, unsigned grid, cudaStream_t s) {
  // The register split needs the launch to own that many: a matter of the compiled kernel, asked once.  The
  // shared-memory limit belongs to the current device, so it is set for every call.
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    AFF_CUDA(cudaFuncGetAttributes(&fa, kv4_tile_kernel<NC>));
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) != kLaunchRegs) AFF_CUDA(cudaErrorInvalidConfiguration);
  AFF_CUDA(cudaFuncSetAttribute(kv4_tile_kernel<NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileSmem));
  AFF_CUDA(launch_pdl(kv4_tile_kernel<NC>, grid, kTileThreads, (size_t)kTileSmem, s, p));
  return AFF_OK;
}

template <int NC, bool F32>
aff_status launch_few(const Kv4AttnParams& p, int sms, cudaStream_t s) {
  const int ctas = few_ctas(NC, F32) * sms;
  const unsigned grid = (unsigned)(p.g.max_items < ctas ? p.g.max_items : ctas);
  AFF_CUDA(cudaFuncSetAttribute(kv4_few_kernel<NC, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, few_smem(NC, F32)));
  AFF_CUDA(launch_pdl(kv4_few_kernel<NC, F32>, grid, kFewThreads, (size_t)few_smem(NC, F32), s, p));
  return AFF_OK;
}
template <int NC>
aff_status launch_few(const Kv4AttnParams& p, int sms, cudaStream_t s) {
  return p.g.dtype == AFF_BF16 ? launch_few<NC, false>(p, sms, s) : launch_few<NC, true>(p, sms, s);
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
  p.score_log2 = scale * 1.4426950408889634f * cache->k_scale;
  if (!(scale > 0.f && std::isfinite(p.score_log2) && p.score_log2 > 0.f)) return AFF_ERR_INVALID_ARG;
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
  p.v_scale = cache->v_scale;
  // all rows of a step of at most 8 are one sequence's few-rows items; otherwise only the device knows (step.cuh)
  const bool tiles = g.dtype == AFF_BF16 && !(g.few && (int64_t)g.T * g.R <= g.few_rows);
  p.overlap = tiles && g.few;
  if (tiles) {
    const unsigned grid = (unsigned)(g.max_items < sms ? g.max_items : sms);
    switch (p.pool.n) {
      case 1: st = launch_tile<1>(p, grid, s); break;
      case 2: st = launch_tile<2>(p, grid, s); break;
      case 3: st = launch_tile<3>(p, grid, s); break;
      default: st = launch_tile<4>(p, grid, s); break;
    }
    if (st != AFF_OK) return st;
  }
  if (g.few) {
    switch (p.pool.n) {
      case 1: st = launch_few<1>(p, sms, s); break;
      case 2: st = launch_few<2>(p, sms, s); break;
      case 3: st = launch_few<3>(p, sms, s); break;
      default: st = launch_few<4>(p, sms, s); break;
    }
    if (st != AFF_OK) return st;
  }
  return g.may_split ? launch_join(g, out, lse, s) : AFF_OK;
}
