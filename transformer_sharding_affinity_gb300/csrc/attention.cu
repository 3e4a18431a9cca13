// attention.cu -- affinity_prefix_attention: causal softmax attention over a
// paged cache for a batch whose sequences share a prefix.  Where sequences have
// few tokens the prefix's keys and values are read once for a row tile of the
// whole batch (step.cuh, `separate`).
//
//   out[t, h] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q.k_j - m)
//   lse[t, h] = m + log sum_j p_j
//
// over the prefix's keys and the sequence's own keys j <= own index of t.
//
// bf16: attention_kernel, persistent, one CTA per SM, on the tensor cores.
//   A work item (step.cuh) is up to 256 packed rows against a run of 128-key
//   tiles; CTAs claim them from a counter.  Two streams of 128 rows alternate on
//   the tensor core, each with two score buffers of half a tile: while the threads
//   of one half turn its scores S into probabilities P, other products run.
//     warps 0-3, 4-7   softmax of stream 0 / 1, one thread per row
//     warp 8           claims items; TMA: query rows, key and value tiles through
//                      the page tables
//     warps 9, 10      issue the products of stream 0 / 1:  S = Q K^T (both from
//                      shared memory) and O += P V (P from tensor memory)
//     warp 11          passes tiles on; clears the rows of a value tile past its keys
//                      and takes out infinite and NaN values of keys that some row
//                      does not see: 0 * NaN would stay
//     warps 12-15      output, while the softmax goes on to the next item
//   Tensor memory: S of both streams (128 columns each, as two buffers of half a
//   tile's 64 keys; P overlays the first half of its buffer), O of both (128
//   columns each).
//   Items of at most 16 rows leave the tensor tiles aside: few_rows.
//   All roles' code together has to stay in the instruction cache (128 KB): at
//   126-234 KB it was what bounded the kernel (64 x 1024 tokens of 16 / 8 heads of
//   128: 453 us; 296 at 65 KB).  Hence the unrolling that is not done.
//   What bounds it now, on sizes of 128-wide heads:
//     one prompt of 8192 tokens, 32 heads: 350 us, 1.57 PFLOP/s, 84 % of the measured
//       rate: the tensor core, with the softmax's exponentials close behind;
//     64 prompts of 1024, 16 heads: 280 us, 0.98 PFLOP/s: items of 1 to 8 tiles, of
//       which one is half past the diagonal, and their beginnings and ends;
//     64 tokens against 8192 keys each: 336 us, 6.4 TB/s, 94 % of the measured copy;
//     256 tokens behind a prefix of 32768 with 1024 own keys: 291 us, 4.1 TB/s and
//       0.47 PFLOP/s: the prefix's items bound by the tensor core, the others by bytes;
//     64 tokens behind 8192 with 750 own keys: 69 us, 3.3 TB/s: the items' latencies
//       and the join (8 us).
//   None of these times holds the step's plan (step_plan.cu), made once for all layers.
//   Running maximum m and sum l are fp32 and thread-local.  O is rescaled only
//   when m has grown by more than 8 (in log2): until then p <= 2^8, far inside
//   fp32 and bf16.  P is rounded to bf16, the type of V (a product's operands
//   share it): one more rounding of at most 2^-8 per probability, unbiased and averaged
//   over the keys; l sums the unrounded p.
// fp32: attention_f32_kernel, CUDA cores, for small shapes: 26 prompts of 294 tokens
// behind 158, 700 us, 27 TFLOP/s of the cores' 74: shared-memory loads (2.8 cycles of
// the pipe for each) and four barriers a step, beside the products.  64 tokens x 1000
// keys of 8 heads, 156 us, 3.4 TB/s: a warp's loads wait for its page look-up.
// Rows in several parts are merged by join_kernel from fp32 partial rows.
#include "affinity.h"
#include "internal.h"
#include "launch.cuh"
#include "sm103_primitives.cuh"
#include "step.cuh"

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

namespace aff {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = 128;                   // rows of a stream
constexpr int kHalfBytes = kRows * 128;      // a tile's 64-column half: 128 rows of 128 bytes
constexpr int kMaxStages = 6;
constexpr int kHalfKeys = kKeyTile / 2;      // scores are computed and turned into probabilities by half tiles
constexpr int kSlots = 4;                    // items on their way through the CTA
constexpr int kStageOut = 4 * 32 * 128;      // output staging: 32 rows of 128 bytes for each output warp
constexpr int kSmemMax = 227 * 1024;
constexpr float kRescale = 8.f;              // log2 growth of the maximum that O is rescaled for
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;              // O of stream s at kColO + 128 s; S at 128 s
constexpr uint32_t kStatusInvalid = 1;

struct AttnParams {
  StepGeom g;
  const uint16_t* q;
  int64_t q_stride;
  void* out;
  float* lse;               // [T][H] or null
  float scale, scale_log2;
  int32_t halves;           // 64-column halves of a head row
  int32_t kd;               // head width rounded up to 16
  int32_t box;              // keys of a TMA box: a page, or a tile of a larger page
  int32_t stages;
  int32_t q_boxes;          // a row tile of queries is one TMA box per half: R divides 128 (map_q)
  int32_t out_boxes;        // a warp's 32 rows of the output are one box per half: R divides 32 (map_out)
  int32_t whole_rows;       // few-rows tiles: a box holds both halves (d_head 128; few_k, few_v)
  const float *kc, *vc;     // the pools as the fp32 kernel reads them (the bf16 kernel has tensor maps)
  int64_t page_stride, group_stride, token_stride;
};

constexpr int kFewPitch = 132;                                   // floats of a staged row: rows start in different banks
constexpr int kFewBytes = 8 * 2 * kFewPitch * 4 + 8 * kFewRows * 8;     // two rows and all (m, l) of each softmax warp

// Ring stages that fit beside the query tiles and the staging.
__host__ __device__ constexpr int ring_stages(int halves) {
  const int n = (kSmemMax - 1024 - kStageOut - 2 * kRows * 8 - kFewBytes - 1024) / (halves * kHalfBytes) - 2;
  return n < kMaxStages ? n : kMaxStages;
}

struct alignas(16) Bars {
  uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
  uint64_t kv_ready[3][kMaxStages];          // stream 0, stream 1, few rows: their own tiles, in their own order
  uint64_t q_full[2], q_empty[2], s_full[2][2], p_full[2][2], pv_done[2][2], o_full[2], o_empty[2];   // [stream][score buffer]
  uint64_t stat_full[2], stat_empty[2], few, few_read, drain[2], slot_full[kSlots], slot_empty[kSlots];
  alignas(16) WorkItem slot[kSlots];           // row0 < 0: no more
  int slot_item[kSlots];                       // their numbers
  uint32_t tmem;
  int abort_flag;
  int marked;                                  // items of this CTA are marked (add_specials)
};

// D[tmem] (+)= A[tmem] * B[smem]^T: the probabilities stay in tensor memory.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 lanes x 32 consecutive 32-bit columns (same lane mapping as tmem_ld16).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptor for an MN-major operand tile written by TMA
// with 128-byte swizzling: rows of 64 16-bit elements (128 B) along N, one row per
// K index; 8-row atoms (1024 B) follow each other along K, groups of 64 N elements
// lie `group_bytes` apart.  The k-th 16-element K slice starts 2048 k bytes further.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t addr, uint32_t group_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((group_bytes >> 4) & 0x3FFFu) << 16;   // leading byte offset: next 64 N elements
  d |= static_cast<uint64_t>(1024 >> 4) << 32;                       // stride byte offset: next 8 K rows
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;                               // swizzle mode: 128 B
  return d;
}

__device__ __forceinline__ void tma_load_5d(void* smem_dst, const CUtensorMap* m, uint64_t* bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3, int32_t c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
      "[%7];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tma_store_4d(const void* smem_src, const CUtensorMap* m, int32_t c0, int32_t c1, int32_t c2,
                                             int32_t c3) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];\n\t"
               "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(m)),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(smem_src))
               : "memory");
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ bool gave_up(const Bars* b) { return *reinterpret_cast<const volatile int*>(&b->abort_flag) != 0; }

// The whole warp waits, for 2 s at most; then the CTA gives up: every later wait ends soon, what is computed
// is thrown away with the status word, and the roles leave at their next item.  Little code, because the
// roles' code together has to stay in the instruction cache: the clock is read every 256 polls (a poll
// suspends for a while by itself), and only its low 32 bits.
__device__ __forceinline__ void wait_on(uint64_t* bar, uint32_t parity, Bars* b) {
  if (!mbar_try_wait(bar, parity)) {
    uint32_t t0 = 0;
#pragma unroll 1
    for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n) {
      if (n & 255u) continue;
      uint32_t t;
      asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
      if (n == 256) t0 = t;
      if (t - t0 > 2000000000u) b->abort_flag = 1;
      if (gave_up(b)) break;
    }
  }
  __syncwarp();
}

// Keys that tile `ti` of an item holds (1 .. 128), and the first of them within its segment.
__device__ __forceinline__ int tile_keys(const WorkItem& it, const StepGeom& g, int ti, int* key0) {
  const bool pre = ti < it.np;
  return tile_span(g, pre ? g.prefix_len : it.own_len, pre ? ti : ti - it.np, key0);
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

// The item in slot k.  The same in every lane and known to be: what follows from it stays in
// uniform registers, where the tensor instructions take their descriptors from.
__device__ __forceinline__ WorkItem uniform_item(const Bars* bars, int k) {
  WorkItem it = load_item(&bars->slot[k % kSlots]);
  int* v = reinterpret_cast<int*>(&it);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(WorkItem) / 4); ++i) v[i] = __shfl_sync(0xffffffffu, v[i], 0);
  return it;
}
// Waits for slot k; false when there is no item left, or the CTA has given up.
__device__ __forceinline__ bool slot_wait(Bars* b, int k) {
  wait_on(&b->slot_full[k % kSlots], (k / kSlots) & 1, b);
  return __all_sync(0xffffffffu, !gave_up(b) && b->slot[k % kSlots].row0 >= 0);
}
__device__ __forceinline__ void slot_done(Bars* b, int k) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&b->slot_empty[k % kSlots]);
}

__device__ __forceinline__ void st_shared16(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// Infinite and NaN values of keys that only some rows of an item see.  A product over the tile would carry
// 0 * inf = NaN to the rows that do not see them, so they are taken out of the tile (bf16 pairs whose exponent is
// all ones become 0) and the item is marked; add_specials puts them back for the rows that do.
// The mark, in the plan's copy of WorkItem::alt, is the CTA that has the item.
constexpr int kMarkShift = 8;
__device__ __forceinline__ int item_mark() { return (int)(blockIdx.x + 1) << kMarkShift; }

__device__ __forceinline__ void without_specials(uint4& w) {
  uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t top = ((x[i] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
    x[i] &= ~((top >> 15) * 0xffffu);
  }
}
// 128 bytes of shared memory; out of line, so that the code of the roles stays together
__device__ __noinline__ void clean_row(uint32_t at) {
#pragma unroll 1
  for (int q = 0; q < 8; ++q) {
    uint4 w = ld_shared16(at + q * 16);
    without_specials(w);
    st_shared16(at + q * 16, w);
  }
}
// sum + 0 x, both halves
__device__ __forceinline__ uint32_t add_zero_times(uint32_t x, uint32_t sum) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(x), "r"(0u), "r"(sum));
  return d;
}

// Own keys below this are seen by every row of the item (its first row sees the fewest).
__device__ __forceinline__ int all_see(const WorkItem& it, const StepGeom& g) {
  return it.seq < 0 ? INT32_MAX : g.by_R(it.row0) + it.own_off + 1;
}

// For the items that this CTA has marked, with all its outputs written: adds the values that are not finite to
// the rows that see their keys.  Such a value makes the sum inf or NaN whatever else is in it, and however small its
// probability: where that has underflowed to 0, the product over a whole tile gives 0 * inf = NaN.  The first eight
// warps; a rare case, and bounded by the items' masked keys.
__device__ __noinline__ void add_specials(const AttnParams& p, const uint16_t* v_pool, int n_items) {
  const StepGeom& g = p.g;
  const int warp = threadIdx.x >> 5, c = (threadIdx.x & 31) * 4;
#pragma unroll 1
  for (int i = 0; i < n_items; ++i) {
    const int marked = *reinterpret_cast<const volatile int32_t*>(&g.items[i].alt);
    if (marked >> kMarkShift != (int)blockIdx.x + 1) continue;
    const WorkItem it = load_item(g.items + i);
    const int from = all_see(it, g), alt = marked & ((1 << kMarkShift) - 1);
    const int n = alt ? it.n0 + it.n1 : it.n1 > it.n0 ? it.n1 : it.n0;
#pragma unroll 1
    for (int r = warp; r < it.nrows; r += 8) {
      const int rr = it.row0 + r, tok = g.by_R(rr), h = it.group * g.R + rr - tok * g.R;
      float add[4] = {0.f, 0.f, 0.f, 0.f};
      bool any = false;
#pragma unroll 1
      for (int u = max(it.np - it.t0, 0); u < n; ++u) {
        int key0;
        const int keys = tile_keys(it, g, it.t0 + u, &key0);
        const int end = min(key0 + keys, tok + it.own_off + 1);
#pragma unroll 1
        for (int key = max(key0, from); key < end; ++key) {
          const int pi = g.by_page(key), page = g.pages[(int64_t)it.seq * g.pages_stride + pi];
          if (page < 0 || page >= g.n_pages || c >= g.d) continue;
          const uint2 w = *reinterpret_cast<const uint2*>(v_pool + page * p.page_stride + it.group * p.group_stride +
                                                          (int64_t)(key - pi * g.page_size) * p.token_stride + c);
          const uint32_t x[4] = {w.x << 16, w.x & 0xffff0000u, w.y << 16, w.y & 0xffff0000u};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if ((x[e] & 0x7f800000u) == 0x7f800000u) {
              add[e] += __uint_as_float(x[e]);
              any = true;
            }
        }
      }
      if (!any) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (add[e] == 0.f) continue;               // not NaN, not inf
        if (it.part_row >= 0) {
          g.part_out[(int64_t)(it.part_row + r) * g.d + c + e] += add[e];
        } else {
          __nv_bfloat16* at = static_cast<__nv_bfloat16*>(p.out) + ((int64_t)tok * g.H + h) * g.d + c + e;
          *at = __float2bfloat16_rn(__bfloat162float(*at) + add[e]);
        }
      }
    }
  }
  // taken back for the next call
  asm volatile("bar.sync 1, 256;" ::: "memory");
  for (int i = threadIdx.x; i < n_items; i += 256) {
    volatile int32_t* alt = &g.items[i].alt;     // not from the first cache: warp 11 has changed it since
    if (*alt >> kMarkShift == (int)blockIdx.x + 1) *alt = *alt & ((1 << kMarkShift) - 1);
  }
}

// One lane of the (converged) warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

// An item's tiles pass through the ring in order, keys then values of tile t0, t0 + 1, ..
__device__ __forceinline__ int item_tiles(const WorkItem& it) { return it.alt ? it.n0 + it.n1 : it.n1; }   // n0 <= n1

// Box of a tile that holds key `key`: its page, or the only one (pages of several tiles).
__device__ __forceinline__ int box_of(const AttnParams& p, int key) { return p.g.tile_pages ? p.g.by_page(key) : 0; }

// Byte of key `key`'s first half in a few-rows tile, and from there to its second half.  Rows past the boxes' keys
// (a tile of whole pages may hold fewer than 128) are a box of their own at the tile's end.
__device__ __forceinline__ uint32_t few_row(const AttnParams& p, int key) {
  if (key >= p.g.key_tile) return (p.g.key_tile * (p.halves - 1) + key) * 128;
  const int box = box_of(p, key);
  return (box * p.halves * p.box + key - box * p.box) * 128;
}
__device__ __forceinline__ uint32_t few_half(const AttnParams& p, int key) {
  return (key >= p.g.key_tile ? kKeyTile - p.g.key_tile : p.box) * 128;
}

// Own keys that the last row of stream s sees, and the keys of its tile that it has any use for.
__device__ __forceinline__ int stream_limit(const WorkItem& it, const StepGeom& g, int s) {
  const int last = it.row0 + min(it.nrows, it.alt || s ? it.nrows : kRows) - 1;
  return min(it.own_len, g.by_R(last) + it.own_off + 1);
}
__device__ __forceinline__ int stream_keys(const WorkItem& it, const StepGeom& g, int ti, int limit) {
  const bool pre = ti < it.np;
  int key0;
  return tile_span(g, pre ? g.prefix_len : limit, pre ? ti : ti - it.np, &key0);
}

__device__ __forceinline__ int tile_of(const WorkItem& it, int s, int j) { return it.t0 + (it.alt ? 2 * j + s : j); }

// S = Q K^T over NK slices of 16 head elements, and O (+)= P V over NK slices of 16 keys.
// Straight-line code for the common widths (NK 0: any): one thread issues every product,
// and a branch for each would take longer than the 64 clocks of a 128 x 128 x 16 product.
template <int NK>
__device__ __forceinline__ void issue_scores(int nk, uint32_t dst, uint64_t da, uint64_t db, uint32_t id) {
  auto one = [&](int k) {
    const uint32_t o = ((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4;
    mma_f16_ss(dst, da + o, db + o, id, k > 0);
  };
  if constexpr (NK > 0) {
#pragma unroll
    for (int k = 0; k < NK; ++k) one(k);
  } else {
#pragma unroll 1
    for (int k = 0; k < nk; ++k) one(k);
  }
}
// The half tile's keys, up to 4 slices of 16 (`ks` counts on into the next half; a run's last half tile has fewer).
__device__ __forceinline__ void issue_values(int ks, uint32_t dst, uint32_t pa, uint64_t db, uint32_t id, uint32_t acc) {
  if (ks >= 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k) mma_f16_ts(dst, pa + k * 8, db + k * 128, id, k > 0 || acc);
  } else {
#pragma unroll 1
    for (int k = 0; k < ks; ++k) mma_f16_ts(dst, pa + k * 8, db + k * 128, id, k > 0 || acc);
  }
}

struct Ring {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void skip(int n, int stages) {      // n <= stages
    s += n;
    if (s >= stages) {
      s -= stages;
      ph ^= 1u;
    }
  }
  __device__ __forceinline__ void advance(int n, int stages) {   // any n
    const int rounds = n / stages;
    ph ^= rounds & 1u;
    skip(n - rounds * stages, stages);
  }
};

__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

// A warp's 32 query rows into their place of a 128-byte swizzled K-major tile (`tile` points at the
// first); lane i gives the address of row i (null: no such row).  16 (8) neighbouring lanes copy a row
// of up to 128 (64) elements, so that a request covers whole lines; pieces past d are zero.
__device__ __forceinline__ void copy_queries(const AttnParams& p, const uint16_t* src, uint8_t* tile) {
  const int lane = threadIdx.x & 31;
  if (!__any_sync(0xffffffffu, src != nullptr)) return;
  const int shift = p.halves == 2 ? 4 : 3, per = 32 >> shift;
  const int c = lane & ((1 << shift) - 1), sub = lane >> shift;
  const int bytes = c * 8 < p.g.d ? 16 : 0;
  const uint32_t dst = smem_u32(tile) + (c >> 3) * kHalfBytes;
#pragma unroll 1
  for (int r0 = 0; r0 < 32; r0 += per) {
    const int r = r0 + sub;
    const uint16_t* from =
        reinterpret_cast<const uint16_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), r));
    if (from && c * 8 < p.kd)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4)),
                   "l"(from + (bytes ? c * 8 : 0)), "r"(bytes)
                   : "memory");
  }
}

// 16 bytes to / from row `row` of a warp's 32 x 128-byte staging block, in place c of 8.
__device__ __forceinline__ uint32_t stage_at(uint32_t base, int row, int c) { return base + row * 128 + ((c ^ (row & 7)) << 4); }
__device__ __forceinline__ void ldmatrix4(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit elements, two to a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// An item of at most 8 * RN rows, by the eight softmax warps.  It is bound by the keys and values it reads
// (a tile's 64 KB take an SM 2800 clocks of its share of HBM), and a 128-row tensor tile would pass through
// scores, probabilities and products one after the other for rows that are mostly not there.  Here warp w
// takes keys 16 w .. + 15 of every tile with its own running maximum, sum and output on the warp's own
// products, transposed so that the rows are the short side:  S^T = K Q^T (16 keys x 8 rows) and
// O^T += V^T P^T (16 columns x 8 rows); nothing is exchanged before the end of the item.  The maximum is
// taken over a row's lanes only when some score has passed it by more than kRescale (log2).
// A tile's pages lie one after the other, each as its 64-column halves.
template <int NK, int RN>
__device__ __forceinline__ void few_rows(const AttnParams& p, const WorkItem& it, Bars* bars, uint32_t* status,
                                         uint8_t* kv_smem, uint8_t* few_smem, uint32_t first, Ring& turn,
                                         uint32_t& few_ph) {
  constexpr int kSlices = NK > 0 ? NK : kKeyTile / 16;
  const StepGeom& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nk = NK > 0 ? NK : p.kd / 16, tile_bytes = p.halves * kHalfBytes;
  const int nrows = it.nrows, quad = lane >> 2, col2 = (lane & 3) * 2;
  // B operand of S^T: row quad of each 8, columns col2, + 1 and + 8, + 9 of each slice
  uint32_t q[RN][kSlices][2];
#pragma unroll
  for (int t = 0; t < RN; ++t) {
    const int r = quad + 8 * t, rr = it.row0 + r, tok = g.by_R(rr);
    const uint16_t* src = p.q + (int64_t)tok * p.q_stride + (it.group * g.R + rr - tok * g.R) * g.d;
#pragma unroll
    for (int k = 0; k < kSlices; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = k * 16 + e * 8 + col2;
        q[t][k][e] = r < nrows && c < g.d ? __ldg(reinterpret_cast<const uint32_t*>(src + c)) : 0u;
      }
  }
  // rows col2 and col2 + 1 of each 8: own keys in view, maximum (that O and l refer to), sum
  int own_vis[RN][2];
  float m[RN][2], l[RN][2], o[RN][kSlices][4];
#pragma unroll
  for (int t = 0; t < RN; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * t + col2 + e;
      own_vis[t][e] = r >= nrows ? -1 : it.seq < 0 ? INT32_MAX : g.by_R(it.row0 + r) + it.own_off + 1;
      m[t][e] = -INFINITY;
      l[t][e] = 0.f;
#pragma unroll
      for (int n = 0; n < kSlices; ++n) o[t][n][e] = o[t][n][2 + e] = 0.f;
    }
  const int stages = NK > 0 ? ring_stages(NK > 4 ? 2 : 1) : p.stages;
  Ring rk, tk = turn;
  rk.s = first % stages;
  Ring rv = rk, tv = turn;
  rv.skip(1, stages);
  tv.skip(1, stages);
  turn.advance(2 * it.n0, stages);
  // ldmatrix: lane 8 i + j gives row j of matrix i.  A operand of S^T: (keys 0-7, 8-15) x (columns 0-7 | 8-15);
  // of O^T, transposed: (columns 0-7, 8-15) x (keys 0-7 | 8-15).
  const int kj = warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), kc = lane >> 4;
  const int vj = warp * 16 + (lane >> 4) * 8 + (lane & 7), vc = (lane >> 3) & 1;
  const uint32_t k_half = few_half(p, kj), v_half = few_half(p, vj);
  const uint32_t k_at = smem_u32(kv_smem) + few_row(p, kj), v_at = smem_u32(kv_smem) + few_row(p, vj);
  // S^T of the stream's next tile (garbage past the tile's keys: masked afterwards)
  float sc[RN][4];
  auto scores = [&]() {
    wait_on(&bars->kv_ready[2][tk.s], tk.ph, bars);
    tk.skip(2, stages);
    float s2[RN][4];                // two chains of products
#pragma unroll
    for (int t = 0; t < RN; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[t][e] = s2[t][e] = 0.f;
#pragma unroll
    for (int k0 = 0; k0 < kSlices; k0 += 4) {      // four loads ahead of their products
      uint32_t a[4][4];
#pragma unroll
      for (int k = k0; k < k0 + 4 && k < kSlices; ++k)
        if (k < nk)
          ldmatrix4(k_at + rk.s * tile_bytes + (k >> 2) * k_half + ((((k & 3) * 2 + kc) ^ (kj & 7)) << 4), a[k - k0]);
#pragma unroll
      for (int k = k0; k < k0 + 4 && k < kSlices; ++k)
#pragma unroll
        for (int t = 0; t < RN; ++t)
          if (k < nk) mma_16x8x16((k & 1) ? s2[t] : sc[t], a[k - k0], q[t][k][0], q[t][k][1]);
    }
#pragma unroll
    for (int t = 0; t < RN; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[t][e] += s2[t][e];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->kv_empty[rk.s]);
    rk.skip(2, stages);
  };
  if (it.n0 > 0) scores();
#pragma unroll 1
  for (int u = 0; u < it.n0; ++u) {
    const int ti = it.t0 + u;
    int key0;
    const int keys = tile_keys(it, g, ti, &key0);
    const bool mine = warp * 16 < keys;
    uint32_t pb[RN][2];
    // sc[t][e]: key quad, row col2 + e; sc[t][2 + e]: key quad + 8
    bool grow = false;
#pragma unroll
    for (int t = 0; t < RN; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        int vis = ti < it.np ? keys : min(keys, own_vis[t][e] - key0);
        if (own_vis[t][e] <= 0) vis = 0;
        if (warp * 16 + quad >= vis) sc[t][e] = -INFINITY;
        if (warp * 16 + quad + 8 >= vis) sc[t][2 + e] = -INFINITY;
        grow |= (fmaxf(sc[t][e], sc[t][2 + e]) - m[t][e]) * p.scale_log2 > kRescale;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int t = 0; t < RN; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(sc[t][e], sc[t][2 + e]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float f = mx > m[t][e] ? ex2((m[t][e] - mx) * p.scale_log2) : 1.f;
          m[t][e] = fmaxf(m[t][e], mx);
          l[t][e] *= f;
#pragma unroll
          for (int n = 0; n < kSlices; ++n) {
            o[t][n][e] *= f;
            o[t][n][2 + e] *= f;
          }
        }
    }
#pragma unroll
    for (int t = 0; t < RN; ++t) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float neg = m[t][e] == -INFINITY ? 0.f : -m[t][e] * p.scale_log2;
        x[e] = ex2(fmaf(sc[t][e], p.scale_log2, neg));
        x[2 + e] = ex2(fmaf(sc[t][2 + e], p.scale_log2, neg));
        l[t][e] += x[e] + x[2 + e];
      }
      pb[t][0] = transpose8(bf16x2(x[0], x[1]));      // keys x rows -> rows x keys, the B operand of O^T
      pb[t][1] = transpose8(bf16x2(x[2], x[3]));
    }
    // the next tile's scores beside this one's values: two independent chains of loads and products
    if (u + 1 < it.n0) scores();
    wait_on(&bars->kv_ready[2][tv.s], tv.ph, bars);
    tv.skip(2, stages);
    if (mine) {
#pragma unroll
      for (int n0 = 0; n0 < kSlices; n0 += 4) {
        uint32_t a[4][4];
#pragma unroll
        for (int n = n0; n < n0 + 4 && n < kSlices; ++n)
          if (n < nk)
            ldmatrix4_t(v_at + rv.s * tile_bytes + (n >> 2) * v_half + ((((n & 3) * 2 + vc) ^ (vj & 7)) << 4), a[n - n0]);
#pragma unroll
        for (int n = n0; n < n0 + 4 && n < kSlices; ++n)
#pragma unroll
          for (int t = 0; t < RN; ++t)
            if (n < nk) mma_16x8x16(o[t][n], a[n - n0], pb[t][0], pb[t][1]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->kv_empty[rv.s]);
    rv.skip(2, stages);
  }
  // ---- the eight warps' parts are added in shared memory, two rows at a time, by the first four warps;
  // the others go on to the next item at once and wait only where they would write over what is not read
  float* part = reinterpret_cast<float*>(few_smem);                       // [warp][2 rows][kFewPitch]
  float2* ml = reinterpret_cast<float2*>(part + 8 * 2 * kFewPitch);       // [warp][kFewRows]
#pragma unroll
  for (int t = 0; t < RN; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], x);
#pragma unroll
  for (int pass = 0; pass < 4 * RN; ++pass) {
    if (pass * 2 >= nrows) break;
    wait_on(&bars->few_read, few_ph ^ 1u, bars);
    if (pass == 0 && quad == 0) {
#pragma unroll
      for (int t = 0; t < RN; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) ml[warp * kFewRows + 8 * t + col2 + e] = make_float2(m[t][e], l[t][e]);
    }
    if (col2 >> 1 == (pass & 3)) {
      float* dst = part + warp * 2 * kFewPitch + quad;
#pragma unroll
      for (int n = 0; n < kSlices; ++n) {
        dst[n * 16] = o[pass >> 2][n][0];
        dst[n * 16 + kFewPitch] = o[pass >> 2][n][1];
        dst[n * 16 + 8] = o[pass >> 2][n][2];
        dst[n * 16 + 8 + kFewPitch] = o[pass >> 2][n][3];
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->few);
    few_ph ^= 1u;
    if (warp >= 4) continue;
    wait_on(&bars->few, few_ph ^ 1u, bars);
    const int rl = threadIdx.x >> 6, r_item = pass * 2 + rl, c = (threadIdx.x & 63) * 2;
    if (r_item < nrows && c < g.d) {
      float2 a[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) a[w] = ml[w * kFewRows + r_item];
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < 8; ++w) mm = fmaxf(mm, a[w].x);
      const float ref = mm == -INFINITY ? 0.f : mm;
      float sum = 0.f, x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const float2 v = *reinterpret_cast<const float2*>(part + (w * 2 + rl) * kFewPitch + c);
        if (a[w].y == 0.f) continue;              // nothing seen by this warp
        const float f = ex2((a[w].x - ref) * p.scale_log2);
        sum += a[w].y * f;
        x += v.x * f;
        y += v.y * f;
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const int rr = it.row0 + r_item, tok = g.by_R(rr), h = it.group * g.R + rr - tok * g.R;
      const float lse = sum == 0.f ? -INFINITY : mm * p.scale + logf(sum);
      if (it.part_row < 0) {
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + ((int64_t)tok * g.H + h) * g.d + c) =
            bf16x2(x * inv, y * inv);
        if (c == 0 && p.lse) p.lse[(int64_t)tok * g.H + h] = lse;
      } else {
        *reinterpret_cast<float2*>(g.part_out + (int64_t)(it.part_row + r_item) * g.d + c) = make_float2(x * inv, y * inv);
        if (c == 0) g.part_lse[it.part_row + r_item] = lse;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->few_read);
  }
}

// NK: 16-element slices of a head: 8 (d_head 128), 6 (96), 4 (64), 0 (any).  FEW: with the few-rows path;
// steps of whole prompts do without its registers and code (an 8192-token prompt: 535 -> 500 us).
template <int NK, bool FEW>
__global__ void __launch_bounds__(kThreads, 1)
attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_out,
                 const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const __grid_constant__ CUtensorMap few_k, const __grid_constant__ CUtensorMap few_v,
                 const __grid_constant__ AttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  // Registers of the softmax threads and of the others: two warpgroups each, 256 in all for two threads.
  constexpr int kSoftmaxRegs = FEW ? 168 : 144, kOtherRegs = 256 - kSoftmaxRegs;
  const StepGeom& g = p.g;
  const int stages = NK > 0 ? ring_stages(NK > 4 ? 2 : 1) : p.stages;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tile_bytes = p.halves * kHalfBytes;
  uint8_t* q_smem = smem;                              // two row tiles
  uint8_t* kv_smem = smem + 2 * tile_bytes;
  uint8_t* out_smem = kv_smem + stages * tile_bytes;
  float2* stats = reinterpret_cast<float2*>(out_smem + kStageOut);      // [stream][row]: (m, l)
  uint8_t* few_smem = reinterpret_cast<uint8_t*>(stats + 2 * kRows);
  Bars* bars = reinterpret_cast<Bars*>(few_smem + kFewBytes);
  uint32_t* status = &g.head->status;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&bars->kv_full[i], 1);
      mbar_init(&bars->kv_ready[0][i], 1);
      mbar_init(&bars->kv_ready[1][i], 1);
      mbar_init(&bars->kv_ready[2][i], 1);
      mbar_init(&bars->kv_empty[i], 9);      // few rows: 8 warps and the clearing warp, which stands in for whoever does not use it
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->q_full[s], p.q_boxes ? 1 : 4);
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
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&bars->slot_full[i], 1);
      mbar_init(&bars->slot_empty[i], 15);   // softmax warps 8, output warps 4, product warps 2, clearing warp 1
    }
    mbar_init(&bars->few, 8);
    mbar_init(&bars->few_read, 4);
    bars->abort_flag = 0;
    bars->marked = 0;
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    if (p.q_boxes) prefetch_tmap(&map_q);
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  if (warp == 9) {
    tmem_alloc(&bars->tmem, kTmemCols);
    tmem_relinquish();
  }
  pdl_enter();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  const bool fits = plan_matches(g);
  const int n_items = fits ? g.head->n_items : 0;
  // a plan of other shapes, or of a malformed step: said by every call, as the status is cleared when it is read
  if ((!fits || n_items < 0) && threadIdx.x == 0) latch_status(status, fits ? kStatusRange : kStatusInvalid);

  // The softmax threads hold a row of scores each: registers move to them from the other warps.
  if (warp >= 8 && warp < 12) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == 8) {
    // ------------------------------------------------------------ key and value tiles
    Ring r;
    int in_flight = 0;
    uint32_t q_ph = 0;                  // bit x: stream x
    // one lane per box: 64 columns of `box` keys
    const int bx = p.halves == 2 ? lane >> 1 : lane, hf = p.halves == 2 ? lane & 1 : 0;
    // Items are claimed one ahead: the first of a CTA is its own number, the others come from a counter,
    // so that CTAs with cheap items take more of them.
    auto publish = [&](int k, int item) {
      wait_on(&bars->slot_empty[k % kSlots], ((k / kSlots) & 1) ^ 1, bars);
      int* d = reinterpret_cast<int*>(&bars->slot[k % kSlots]);
      if (lane < (int)(sizeof(WorkItem) / 4))
        d[lane] = item < n_items ? reinterpret_cast<const int*>(g.items + item)[lane] : -1;
      if (lane == 0) bars->slot_item[k % kSlots] = item;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->slot_full[k % kSlots]);
    };
    int i = blockIdx.x;
    publish(0, i);
    for (int k = 0; i < n_items && !gave_up(bars); ++k) {
      const WorkItem it = load_item(g.items + i);
      int next = 0;
      if (lane == 0) next = gridDim.x + (int)atomicAdd(&g.head->claimed, 1u);
      const int n = item_tiles(it);
      // the streams' query rows, as soon as the item before has no scores left to compute
#pragma unroll 1
      for (int x = 0; x < 2; ++x) {
        if (!p.q_boxes || (FEW && it.alt == 2) || (x ? it.n1 : it.n0) == 0) continue;
        wait_on(&bars->q_empty[x], ((q_ph >> x) & 1u) ^ 1u, bars);
        q_ph ^= 1u << x;
        if (lane == 0) mbar_arrive_expect_tx(&bars->q_full[x], (uint32_t)tile_bytes);
        __syncwarp();
        if (lane < p.halves)
          tma_load_4d(q_smem + x * tile_bytes + lane * kHalfBytes, &map_q, &bars->q_full[x], lane * 64, 0, it.group,
                      g.by_R(it.row0 + (it.alt ? 0 : x * kRows)));
        __syncwarp();
      }
#pragma unroll 1
      for (int u = 0; u < n && !gave_up(bars); ++u) {
        const int ti = it.t0 + u;
        int key0;
        const int keys = tile_keys(it, g, ti, &key0);
        const int32_t* table = ti < it.np ? g.prefix_pages : g.pages + (int64_t)it.seq * g.pages_stride;
        const int boxes = g.tile_pages ? g.by_page(keys + p.box - 1) : 1;      // box: a page
        int page = 0, off = 0;
        if (bx < boxes) {
          const int idx = ti < it.np ? ti : ti - it.np;
          int pi = idx * g.tile_pages + bx;
          if (!g.tile_pages) {
            pi = g.by_page(key0);
            off = key0 - pi * g.page_size;
          }
          page = __ldg(table + pi);
          if (page < 0 || page >= g.n_pages) {      // the copy would read zeros: report it
            latch_status(status, kStatusRange);
            page = 0;
          }
        }
#pragma unroll 1
        for (int value = 0; value < 2; ++value) {
          wait_on(&bars->kv_empty[r.s], r.ph ^ 1u, bars);
          if (lane == 0) mbar_arrive_expect_tx(&bars->kv_full[r.s], (uint32_t)(boxes * p.halves * p.box * 128));
          __syncwarp();
          uint8_t* dst = kv_smem + r.s * tile_bytes;
          if (bx >= boxes) {
          } else if (!(FEW && it.alt == 2)) {
            tma_load_4d(dst + hf * kHalfBytes + bx * p.box * 128, value ? &map_v : &map_k, &bars->kv_full[r.s], hf * 64,
                        off, it.group, page);
          } else {
            dst += (bx * p.halves + hf) * p.box * 128;
            // both halves of a page in one copy: a copy of 2 KB takes its issue of 65 clocks, not its bytes
            if (!p.whole_rows)
              tma_load_4d(dst, value ? &map_v : &map_k, &bars->kv_full[r.s], hf * 64, off, it.group, page);
            else if (hf == 0)
              tma_load_5d(dst, value ? &few_v : &few_k, &bars->kv_full[r.s], 0, off, 0, it.group, page);
          }
          __syncwarp();
          r.skip(1, stages);
          in_flight = min(in_flight + 1, stages);
        }
      }
      publish(k + 1, __shfl_sync(0xffffffffu, next, 0));      // the claim has come back behind the copies
      i = __shfl_sync(0xffffffffu, next, 0);
    }
    if (gave_up(bars)) {      // wait for the copies that were issued before shared memory goes away
      for (int i = 0; i < in_flight; ++i) {
        const int st = (r.s + stages - 1 - i) % stages;
        const uint32_t ph = st < r.s ? r.ph : r.ph ^ 1u;
        const uint64_t t0 = global_timer_ns();
        while (!mbar_test_wait(&bars->kv_full[st], ph) && global_timer_ns() - t0 < 100000000ull) {}
      }
      for (int x = 0; x < 2 && p.q_boxes; ++x) {
        const uint64_t t0 = global_timer_ns();
        while (!mbar_test_wait(&bars->q_full[x], ((q_ph >> x) & 1u) ^ 1u) && global_timer_ns() - t0 < 100000000ull) {}
      }
    }
  } else if (warp < 11) {
    // ------------------------------------------------------------ products
    // The whole warp walks, one lane issues.  The tensor pipe holds about four products, so what
    // this warp does between two batches has to fit in 250 clocks or hide behind the other stream.
    const int s = warp - 9;
    const uint32_t id_qk = idesc_f16(kRows, kHalfKeys, 1);
    const uint32_t id_pv = idesc_f16(kRows, (uint32_t)p.kd, 1) | (1u << 16);   // V is N-major
    // descriptors: the high half is the same for every tile, the low half counts 16-byte steps
    const uint64_t dq = smem_desc_k_sw128(smem_u32(q_smem + s * tile_bytes)), dk0 = smem_desc_k_sw128(smem_u32(kv_smem));
    const uint64_t dv0 = smem_desc_mn_sw128(smem_u32(kv_smem), kHalfBytes);
    const uint32_t tile_step = tile_bytes >> 4, tS = tmem + s * kKeyTile, tO = tmem + kColO + s * kRows;
    const int nk = p.kd / 16;
    uint32_t q_ph = 0, p_ph = 0, oe_ph = 0;
    Ring base, turn;      // the item's first ring stage; the stream's next turn
    for (int k = 0; slot_wait(bars, k); ++k) {
      const WorkItem it = uniform_item(bars, k);
      slot_done(bars, k);
      const int n = s ? it.n1 : it.n0, tiles = item_tiles(it);
      Ring rk = base;                                   // stage of the stream's next keys
      base.advance(2 * tiles, stages);
      if (n == 0 || (FEW && it.alt == 2)) continue;
      if (it.alt && s) rk.skip(2, stages);
      // The stream's tiles become ready in its own order on barriers of its own, so that it sees every
      // phase of each.  tk and tv: the turns of its next keys and values.
      Ring rv = rk, tk = turn, tv = turn;
      rv.skip(1, stages);
      tv.skip(1, stages);
      turn.advance(2 * n, stages);
      const int stride = it.alt ? 4 : 2;                // ring steps from tile to tile of the stream; stages >= 4
      const int ti_step = it.alt ? 2 : 1, limit = stream_limit(it, g, s);
      int ti = tile_of(it, s, 0), keys = stream_keys(it, g, ti, limit);
      // Scores run a tile ahead of the values' products, in half tiles: while the softmax works on one
      // half, the half before it is multiplied with its values and the next tile's scores take its buffer.
      wait_on(&bars->q_full[s], q_ph, bars);
      q_ph ^= 1u;
      wait_on(&bars->kv_ready[s][tk.s], tk.ph, bars);
      tc_fence_after();
      // Every loop over halves is kept one: unrolled, the products' code alone would be 15 KB.
#pragma unroll 1
      for (int from = 0; from < kKeyTile; from += kHalfKeys) {
        if (elect_one()) {
          if (keys > from) issue_scores<NK>(nk, tS + from, dq, dk0 + rk.s * tile_step + (from * 128 >> 4), id_qk);
          mma_commit(&bars->s_full[s][from / kHalfKeys]);
          if (from) mma_commit(&bars->kv_empty[rk.s]);
          if (from && n == 1) mma_commit(&bars->q_empty[s]);
        }
        __syncwarp();
      }
      wait_on(&bars->o_empty[s], oe_ph ^ 1u, bars);
      oe_ph ^= 1u;
#pragma unroll 1
      for (int left = n; left > 0; --left) {
        const bool more = left > 1;
        ti += ti_step;
        const int next_keys = more ? stream_keys(it, g, ti, limit) : 0;
        wait_on(&bars->kv_ready[s][tv.s], tv.ph, bars);
        tv.skip(2, stages);
        rk.skip(stride, stages);
        tk.skip(2, stages);
        if (more) wait_on(&bars->kv_ready[s][tk.s], tk.ph, bars);
        const uint64_t dv = dv0 + rv.s * tile_step, dk = dk0 + rk.s * tile_step;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const int from = h * kHalfKeys;
          wait_on(&bars->p_full[s][h], p_ph, bars);
          tc_fence_after();
          if (elect_one()) {
            issue_values((keys - from + 15) >> 4, tO, tS + from, dv + (from * 128 >> 4), id_pv, h > 0 || left < n);
            mma_commit(&bars->pv_done[s][h]);
            if (h == 1) mma_commit(&bars->kv_empty[rv.s]);
            if (more) {
              if (next_keys > from) issue_scores<NK>(nk, tS + from, dq, dk + (from * 128 >> 4), id_qk);
              mma_commit(&bars->s_full[s][h]);
              if (h == 1) mma_commit(&bars->kv_empty[rk.s]);
              if (h == 1 && left == 2) mma_commit(&bars->q_empty[s]);      // the item's last scores
            } else if (h == 1) {
              mma_commit(&bars->o_full[s]);
            }
          }
          __syncwarp();
        }
        p_ph ^= 1u;
        rv.skip(stride, stages);
        keys = next_keys;
      }
    }
    if (elect_one()) {
      mma_commit(&bars->drain[s]);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_test_wait(&bars->drain[s], 0) && global_timer_ns() - t0 < 2000000000ull) {}
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ ragged value tiles
    // Every tile is waited for and passed on to the streams that use it, so that nobody trails a
    // barrier by a round; for a stream that does not use it this warp empties it.
    Ring r, turn[3];
    for (int k = 0; slot_wait(bars, k); ++k) {
      const WorkItem it = load_item(&bars->slot[k % kSlots]);
      const int number = bars->slot_item[k % kSlots];
      slot_done(bars, k);
      const bool few = FEW && it.alt == 2;
      const int n = item_tiles(it), seen_by_all = all_see(it, g);
#pragma unroll 1
      for (int u = 0; u < n; ++u) {
        int key0;
        const int keys = tile_keys(it, g, it.t0 + u, &key0), to = (keys + 15) & ~15;
        const bool use0 = !few && (it.alt ? !(u & 1) : u < it.n0), use1 = !few && (it.alt ? u & 1 : u < it.n1);
#pragma unroll 1
        for (int value = 0; value < 2; ++value) {
          wait_on(&bars->kv_full[r.s], r.ph, bars);
          if (value && it.t0 + u >= it.np && key0 + keys > seen_by_all) {
            // rows that some query row does not see: 16 rows of 128 bytes at a time, each lane's eight pieces in
            // an order of its own so that no two lanes meet in a bank.  0 * x summed over everything is NaN if
            // anything is not finite (a fused multiply-add per pair); only then are they looked for.
            const int h = lane & 1, from = max(seen_by_all - key0, 0) + (lane >> 1);
            auto row_at = [&](int key) {
              return smem_u32(kv_smem) + r.s * tile_bytes + (few ? few_row(p, key) : key * 128) +
                     h * (few ? few_half(p, key) : kHalfBytes);
            };
            uint32_t sum[4] = {0u, 0u, 0u, 0u};
            if (h < p.halves) {
#pragma unroll 2
              for (int key = from; key < keys; key += 16) {
                const uint32_t at = row_at(key);
                uint4 w[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) w[q] = ld_shared16(at + ((q ^ (lane & 7)) << 4));
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                  sum[0] = add_zero_times(w[q].x, sum[0]);
                  sum[1] = add_zero_times(w[q].y, sum[1]);
                  sum[2] = add_zero_times(w[q].z, sum[2]);
                  sum[3] = add_zero_times(w[q].w, sum[3]);
                }
              }
            }
            bool found = ((sum[0] | sum[1] | sum[2] | sum[3]) & 0x7fff7fffu) != 0;
            if (__any_sync(0xffffffffu, found)) {
#pragma unroll 1
              for (int key = from; key < keys && h < p.halves; key += 16) clean_row(row_at(key));
              fence_async_smem();
              if (lane == 0) {
                atomicOr(&g.items[number].alt, item_mark());
                bars->marked = 1;
              }
            }
          }
          if (value && keys < to) {
            // rows keys .. the next multiple of 16, one half of one row for each lane: whole 128-byte rows,
            // so the swizzle does not matter
            const int key = keys + (lane >> 1), h = lane & 1;
            if (key < to && h < p.halves) {
              uint4* at = reinterpret_cast<uint4*>(kv_smem + r.s * tile_bytes + (few ? few_row(p, key) : key * 128) +
                                                   h * (few ? few_half(p, key) : kHalfBytes));
#pragma unroll 1
              for (int q = 0; q < 8; ++q) at[q] = make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
          }
          __syncwarp();
          if (lane == 0) {
            if (use0) mbar_arrive(&bars->kv_ready[0][turn[0].s]);
            if (use1) mbar_arrive(&bars->kv_ready[1][turn[1].s]);
            if (few) mbar_arrive(&bars->kv_ready[2][turn[2].s]);
            mbar_arrive_n(&bars->kv_empty[r.s], few ? 1 : 9 - (use0 ? 1 : 0) - (use1 ? 1 : 0));
          }
          if (use0) turn[0].skip(1, stages);
          if (use1) turn[1].skip(1, stages);
          if (few) turn[2].skip(1, stages);
          r.skip(1, stages);
        }
      }
    }
  }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int s = warp >> 2;                         // stream
    const int row = threadIdx.x & (kRows - 1);
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + s * kKeyTile;
    const uint32_t tO = tmem + lane_base + kColO + s * kRows;
    uint32_t s_ph = 0, st_ph = 0, used = 0, few_ph = 0;
    Ring few_turn;
    for (int k = 0; slot_wait(bars, k); ++k) {
      const WorkItem it = load_item(&bars->slot[k % kSlots]);
      const uint32_t first_tile = used;
      used += 2 * item_tiles(it);
      if constexpr (FEW) {
        if (it.alt == 2) {
          if (it.nrows <= 8) few_rows<NK, 1>(p, it, bars, status, kv_smem, few_smem, first_tile, few_turn, few_ph);
          else few_rows<NK, 2>(p, it, bars, status, kv_smem, few_smem, first_tile, few_turn, few_ph);
          slot_done(bars, k);
          continue;
        }
      }
      const int n = s ? it.n1 : it.n0;
      const int r_item = row + (it.alt ? 0 : s * kRows);
      const int rr = it.row0 + r_item;
      const bool live = r_item < it.nrows;
      const bool warp_live = (row & ~31) + (it.alt ? 0 : s * kRows) < it.nrows;
      const int tok = g.by_R(rr);
      // own keys in view of this row; padding rows see nothing at all
      const int own_vis = it.seq < 0 ? 0 : tok + it.own_off + 1;
      const bool blind = !live || (it.seq >= 0 && own_vis <= 0);
      if (n > 0 && !p.q_boxes) {      // query rows that no box holds (R does not divide 128); the stream's last scores are done
        copy_queries(p, live ? p.q + (int64_t)tok * p.q_stride + (it.group * g.R + rr - tok * g.R) * g.d : nullptr,
                     q_smem + s * tile_bytes + (row & ~31) * 128);
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->q_full[s]);
      }
      float m = -INFINITY, l = 0.f;                  // m: the maximum that O and l refer to
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
          wait_on(&bars->s_full[s][h], s_ph, bars);
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
            float mx[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < kHalfKeys; c += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], __uint_as_float(v[c + e]), __uint_as_float(v[c + e + 4]));
            const float m_new = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
            if (j == 0 && h == 0) {
              m = m_new;
            } else {
              const bool grow = (m_new - m) * p.scale_log2 > kRescale;
              if (__any_sync(0xffffffffu, grow)) {
                // O is this warp's once the latest product is done (those before it are: these scores were
                // issued after them)
                wait_on(&bars->pv_done[s][h ^ 1], h ? s_ph : s_ph ^ 1u, bars);
                tc_fence_after();
                const float f = grow ? ex2((m - m_new) * p.scale_log2) : 1.f;
                if (grow) m = m_new;
                l *= f;
#pragma unroll 1
                for (int c = 0; c < p.kd; c += 16) {
                  uint32_t o[16];
                  tmem_ld16(tO + c, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                  tmem_st16(tO + c, o);
                }
              }
            }
            const float neg = m == -INFINITY ? 0.f : -m * p.scale_log2;
            const uint64_t sc2 = pk(p.scale_log2, p.scale_log2), ng2 = pk(neg, neg);
            uint64_t sum0 = pk(0.f, 0.f), sum1 = sum0;
            uint32_t w[kHalfKeys / 2];
#pragma unroll
            for (int e = 0; e < kHalfKeys / 2; ++e) {
              const float2 x = unpk(fma2(pk_u(v[2 * e], v[2 * e + 1]), sc2, ng2));
              const float a = ex2(x.x), b = ex2(x.y);
              if (e & 1) sum1 = add2(sum1, pk(a, b));
              else sum0 = add2(sum0, pk(a, b));
              w[e] = bf16x2(a, b);
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
        wait_on(&bars->stat_empty[s], st_ph ^ 1u, bars);
        st_ph ^= 1u;
        stats[s * kRows + row] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->stat_full[s]);
      }
      slot_done(bars, k);
    }
  } else {
    // ------------------------------------------------------------ output
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    const int row = threadIdx.x & (kRows - 1);
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t stage_out = smem_u32(out_smem) + (warp & 3) * 4096;
    uint32_t ph = 0;                                 // bit s: stream s
    for (int k = 0; slot_wait(bars, k); ++k) {
      const WorkItem it = load_item(&bars->slot[k % kSlots]);
      slot_done(bars, k);
      if (FEW && it.alt == 2) continue;
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
          wait_on(&bars->stat_full[x], (ph >> x) & 1u, bars);
          const float2 v = stats[x * kRows + row];
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->stat_empty[x]);
          wait_on(&bars->o_full[x], (ph >> x) & 1u, bars);
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
            f0 = ex2((m - mm) * p.scale_log2);
            f1 = ex2((o.x - mm) * p.scale_log2);
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
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;      // a row without keys: zero
        f0 *= inv;
        f1 *= inv;
        tc_fence_after();
        const int h = it.group * g.R + rr - tok * g.R;
        const bool direct = it.part_row < 0;
        // 128 bytes of each row at a time go through shared memory: 64 bf16 columns of the output, 32 fp32
        // columns of a partial row.  A warp whose 32 rows are all there (and whole tokens) writes output
        // as one bulk copy; otherwise stores of whole lines, with the rows' numbers from their lanes.
        const bool bulk = direct && p.out_boxes && (row & ~31) + s * kRows + 32 <= it.nrows;
        const int mine = !live ? -1 : direct ? tok * g.H + h : it.part_row + r_item;
        const bool none = l == 0.f, some_none = __any_sync(0xffffffffu, none);   // rows without keys are zero
        const int first_tok = __shfl_sync(0xffffffffu, tok, 0);
#pragma unroll 1
        for (int c = 0; c < p.kd; c += 32) {
          uint32_t v[32];
          if (n > 0) tmem_ld32(tO + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f0);
          if (merging) {
#pragma unroll
            for (int x = 0; x < 32; x += 16) {
              uint32_t w[16];
              tmem_ld16(tO + kRows + c + x, w);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e)
                v[x + e] = __float_as_uint(__uint_as_float(v[x + e]) + __uint_as_float(w[e]) * f1);
            }
          }
          if (some_none) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = none ? 0u : v[e];
          }
          if (c + 32 >= p.kd) free_o();
          // the block's bulk copy before has been read: of this item, or of one before it whose rows were output
          if (!(c & 32)) {
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
          }
          if (direct) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              st_shared16(stage_at(stage_out, lane, (c & 32) / 8 + q),
                          make_uint4(bf16x2(__uint_as_float(v[8 * q]), __uint_as_float(v[8 * q + 1])),
                                     bf16x2(__uint_as_float(v[8 * q + 2]), __uint_as_float(v[8 * q + 3])),
                                     bf16x2(__uint_as_float(v[8 * q + 4]), __uint_as_float(v[8 * q + 5])),
                                     bf16x2(__uint_as_float(v[8 * q + 6]), __uint_as_float(v[8 * q + 7]))));
            if (!(c & 32) && c + 32 < p.kd) continue;
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              st_shared16(stage_at(stage_out, lane, q), make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
          }
          if (bulk) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) tma_store_4d(out_smem + (warp & 3) * 4096, &map_out, c & 64, 0, it.group, first_tok);
            __syncwarp();
            continue;
          }
          __syncwarp();
          uint8_t* const to = direct ? static_cast<uint8_t*>(p.out) : reinterpret_cast<uint8_t*>(g.part_out);
          const int piece = lane & 7, row_bytes = g.d * (direct ? 2 : 4), byte = (direct ? (c & 64) * 2 : c * 4) + piece * 16;
#pragma unroll 4
          for (int r0 = 0; r0 < 32; r0 += 4) {
            const int r = r0 + (lane >> 3);
            const int which = __shfl_sync(0xffffffffu, mine, r);
            if (which >= 0 && byte < row_bytes)
              *reinterpret_cast<uint4*>(to + (int64_t)which * row_bytes + byte) = ld_shared16(stage_at(stage_out, r, piece));
          }
          __syncwarp();
        }
        if (live) {
          const float lse = l == 0.f ? -INFINITY : m * p.scale + logf(l);
          if (!direct) g.part_lse[mine] = lse;
          else if (p.lse) p.lse[mine] = lse;
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
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
  if (bars->marked && warp < 8) add_specials(p, reinterpret_cast<const uint16_t*>(p.vc), n_items);
}

template <int NK, bool FEW>
aff_status launch_attention(const CUtensorMap (&m)[6], const AttnParams& p, unsigned grid, int smem,
                            cudaStream_t s) {
  // The register split needs the launch to own 128 registers a thread: a matter of the compiled kernel, asked once.
  // The shared-memory limit belongs to the current device, so it is set for every call, as elsewhere.
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    AFF_CUDA(cudaFuncGetAttributes(&fa, attention_kernel<NK, FEW>));
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) != 128) AFF_CUDA(cudaErrorInvalidConfiguration);
  AFF_CUDA(cudaFuncSetAttribute(attention_kernel<NK, FEW>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax));
  AFF_CUDA(launch_pdl(attention_kernel<NK, FEW>, grid, kThreads, (size_t)smem, s, m[0], m[5], m[1], m[2], m[3], m[4], p));
  return AFF_OK;
}
template <bool FEW>
aff_status launch_attention(const CUtensorMap (&m)[6], const AttnParams& p, unsigned grid, int smem,
                            cudaStream_t s) {
  switch (p.kd / 16) {
    case 8: return launch_attention<8, FEW>(m, p, grid, smem, s);
    case 6: return launch_attention<6, FEW>(m, p, grid, smem, s);
    case 4: return launch_attention<4, FEW>(m, p, grid, smem, s);
    default: return launch_attention<0, FEW>(m, p, grid, smem, s);
  }
}

// ---------------------------------------------------------------- fp32
// On the CUDA cores: a product of two fp32 numbers keeps all its bits there.  Two CTAs per SM; items are
// claimed from the plan's counter.
constexpr int kF32Threads = 256;
constexpr int kF32Keys = 64;                 // keys of a step of the tiled path
constexpr int kF32Rows = 64;                 // its rows
// Most rows of the streaming path.  Up to 32: 5 x 256 tokens of 16-wide heads 39 us instead of 25, 4 x 6 tokens
// behind 3889 keys 163 instead of 119; 47 x 10 tokens x 307 keys 175 instead of 192.
constexpr int kF32Few = 16;

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 halves2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
// 16 bytes from global to shared memory, or 16 zero bytes.
__device__ __forceinline__ void copy16(void* dst, const float* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void copy_wait_but_one() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// Where key `key` of the prefix or of an item's sequence lies in the pools; -1 if its page is out of range.
__device__ __forceinline__ int64_t key_at(const AttnParams& p, const WorkItem& it, bool pre, int key) {
  const StepGeom& g = p.g;
  const int32_t* table = pre ? g.prefix_pages : g.pages + (int64_t)it.seq * g.pages_stride;
  const int pi = g.by_page(key);
  const int page = __ldg(table + pi);
  if (page < 0 || page >= g.n_pages) {
    latch_status(&g.head->status, kStatusRange);
    return -1;
  }
  return page * p.page_stride + it.group * p.group_stride + (int64_t)(key - pi * g.page_size) * p.token_stride;
}

__device__ __forceinline__ void f32_write(const AttnParams& p, const WorkItem& it, int r, int c, float4 v) {
  const StepGeom& g = p.g;
  const int rr = it.row0 + r, tok = g.by_R(rr), h = it.group * g.R + rr - tok * g.R;
  float* dst = it.part_row < 0 ? static_cast<float*>(p.out) + ((int64_t)tok * g.H + h) * g.d
                               : g.part_out + (int64_t)(it.part_row + r) * g.d;
  *reinterpret_cast<float4*>(dst + c) = v;
}
__device__ __forceinline__ void f32_write_lse(const AttnParams& p, const WorkItem& it, int r, float m, float l) {
  const StepGeom& g = p.g;
  const int rr = it.row0 + r, tok = g.by_R(rr), h = it.group * g.R + rr - tok * g.R;
  const float lse = l == 0.f ? -INFINITY : m * p.scale + logf(l);
  if (it.part_row >= 0) g.part_lse[it.part_row + r] = lse;
  else if (p.lse) p.lse[(int64_t)tok * g.H + h] = lse;
}

// Up to 64 rows against 64 keys a step.  Thread (ty, tx) holds rows 4 ty .. + 3: the scores of keys tx + 16 b and
// output columns 4 tx .. + 3 of each 64.  Both products take two fp32 lanes an instruction, which leaves issue
// slots for the shared-memory loads.  Probabilities pass through shared memory by key, so that a thread's four
// rows are one load.  Rows of q and k are swizzled by 16-byte chunks: no load has a bank conflict.  The next keys
// are copied in behind this step's softmax and second product, the next values behind the first product; the
// other CTA of the SM fills what remains.
__device__ void f32_tile(const AttnParams& p, const WorkItem& it, float* smem) {
  const StepGeom& g = p.g;
  constexpr int ld = 128;
  const int d = g.d;
  float* qs = smem;                       // [row][chunk ^ row % 8]
  float* ks = qs + kF32Rows * ld;         // [key][chunk ^ key % 8]
  float* vs = ks + kF32Keys * ld;         // [key]
  float* ps = vs + kF32Keys * ld;         // [key][chunk ^ key % 8] of 64 rows
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, sw = tx & 7;
  const int cr = threadIdx.x >> 3, cc = (threadIdx.x & 7) * 4;          // copies: rows cr, cr + 32; 16 bytes of each 128
  const float* q = reinterpret_cast<const float*>(p.q);
  for (int r = cr; r < kF32Rows; r += 32) {
    const int rr = it.row0 + min(r, it.nrows - 1), tok = g.by_R(rr);
    const float* src = q + (int64_t)tok * p.q_stride + (int64_t)(it.group * g.R + rr - tok * g.R) * d;
    for (int c = cc; c < d; c += 32) copy16(qs + r * ld + (c ^ ((r & 7) * 4)), src + c, r < it.nrows);
  }
  float m[4], l[4];
  uint64_t o[4][4];
  int own_vis[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int r = ty * 4 + a;
    m[a] = -INFINITY;
    l[a] = 0.f;
    own_vis[a] = r >= it.nrows ? 0 : it.seq < 0 ? 1 : g.by_R(it.row0 + r) + it.own_off + 1;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[a][e] = 0;
  }
  // the walk: half tiles of 64 keys; `keys` 0 at its end
  struct Half {
    int tile, half, key0, keys;
    bool pre;
  };
  auto span = [&](Half& s) {
    s.keys = 0;
    while (s.tile < it.t0 + it.n0) {
      s.pre = s.tile < it.np;
      const int n = tile_keys(it, g, s.tile, &s.key0);
      if (s.half * kF32Keys < n) {
        s.key0 += s.half * kF32Keys;
        s.keys = min(n - s.half * kF32Keys, kF32Keys);
        return;
      }
      s.half = 0;
      ++s.tile;
    }
  };
  int64_t at[2];                          // of the rows this thread copies
  auto locate = [&](const Half& s) {
#pragma unroll
    for (int x = 0; x < 2; ++x) at[x] = cr + 32 * x < s.keys ? key_at(p, it, s.pre, s.key0 + cr + 32 * x) : -1;
  };
  auto copy = [&](const Half& s, float* dst, const float* pool, int swizzle) {
#pragma unroll
    for (int x = 0; x < 2 && s.keys > 0; ++x) {
      const int r = cr + 32 * x;
      for (int c = cc; c < d; c += 32) copy16(dst + r * ld + (c ^ swizzle), at[x] < 0 ? pool : pool + at[x] + c, at[x] >= 0);
    }
    copy_commit();
  };
  Half cur{it.t0, 0, 0, 0, false};
  span(cur);
  locate(cur);
  copy(cur, ks, p.kc, (cr & 7) * 4);
  copy(cur, vs, p.vc, 0);
  while (cur.keys > 0) {
    Half next = cur;
    ++next.half;
    span(next);
    copy_wait_but_one();
    __syncthreads();                      // the keys are here
    float s[4][4];
    {
      uint64_t acc[4][4];
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[a][b] = 0;
#pragma unroll 4
      for (int c = 0; c < d; c += 4) {
        ulonglong2 kf[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) kf[b] = *reinterpret_cast<const ulonglong2*>(ks + (tx + 16 * b) * ld + (c ^ (sw * 4)));
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const int r = ty * 4 + a;
          const ulonglong2 qf = *reinterpret_cast<const ulonglong2*>(qs + r * ld + (c ^ ((r & 7) * 4)));
#pragma unroll
          for (int b = 0; b < 4; ++b) acc[a][b] = fma2(qf.y, kf[b].y, fma2(qf.x, kf[b].x, acc[a][b]));
        }
      }
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const float2 v = halves2(acc[a][b]);
          s[a][b] = v.x + v.y;
        }
    }
    __syncthreads();                      // the keys are read
    locate(next);
    copy(next, ks, p.kc, (cr & 7) * 4);
    int last = 0, first = kF32Keys;       // keys of this step that any, and that all of the thread's rows see
    int seen[4];                          // by each of them
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int vis = own_vis[a] <= 0 ? 0 : cur.pre ? cur.keys : min(cur.keys, own_vis[a] - cur.key0);
      seen[a] = vis;
      last = max(last, vis);
      first = min(first, vis);
      float mx = -INFINITY;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (tx + 16 * b >= vis) s[a][b] = -INFINITY;
        mx = fmaxf(mx, s[a][b]);
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float m_new = fmaxf(m[a], mx);
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      const float f = m[a] == -INFINITY ? 0.f : expf((m[a] - ref) * p.scale);
      float sum = 0.f;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        s[a][b] = expf((s[a][b] - ref) * p.scale);
        sum += s[a][b];
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l[a] = l[a] * f + sum;
      m[a] = m_new;
      const uint64_t ff = pair2(f, f);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[a][e] = fma2(o[a][e], ff, 0);
    }
#pragma unroll
    for (int b = 0; b < 4; ++b)
      *reinterpret_cast<float4*>(ps + (tx + 16 * b) * kF32Rows + ((ty ^ sw) * 4)) = make_float4(s[0][b], s[1][b], s[2][b], s[3][b]);
    copy_wait_but_one();
    __syncthreads();                      // the values are here
    first = __reduce_min_sync(0xffffffffu, first);
    last = __reduce_max_sync(0xffffffffu, last);
    auto add = [&](int k, auto masked) {
      const float4 w = *reinterpret_cast<const float4*>(ps + k * kF32Rows + ((ty ^ (k & 7)) * 4));
      const float wa[4] = {w.x, w.y, w.z, w.w};
      ulonglong2 v0 = make_ulonglong2(0, 0), v1 = v0;
      if (4 * tx < d) v0 = *reinterpret_cast<const ulonglong2*>(vs + k * ld + 4 * tx);
      if (64 + 4 * tx < d) v1 = *reinterpret_cast<const ulonglong2*>(vs + k * ld + 64 + 4 * tx);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        if (decltype(masked)::value && k >= seen[a]) continue;                // whatever lies there stays out
        const uint64_t ww = pair2(wa[a], wa[a]);
        o[a][0] = fma2(ww, v0.x, o[a][0]);
        o[a][1] = fma2(ww, v0.y, o[a][1]);
        o[a][2] = fma2(ww, v1.x, o[a][2]);
        o[a][3] = fma2(ww, v1.y, o[a][3]);
      }
    };
    int k = 0;
#pragma unroll 2
    for (; k < first; ++k) add(k, std::false_type());
#pragma unroll 1
    for (; k < last; ++k) add(k, std::true_type());
    __syncthreads();                      // the values and the probabilities are read
    copy(next, vs, p.vc, 0);
    cur = next;
  }
  copy_wait_all();                        // an item without keys leaves its queries under way
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int r = ty * 4 + a;
    if (r >= it.nrows) continue;
    const float inv = l[a] == 0.f ? 0.f : 1.f / l[a];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int c = 64 * x + 4 * tx;
      if (c >= d) continue;
      const float2 v0 = halves2(o[a][2 * x]), v1 = halves2(o[a][2 * x + 1]);
      f32_write(p, it, r, c, l[a] == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                                         : make_float4(v0.x * inv, v0.y * inv, v1.x * inv, v1.y * inv));
    }
    if (tx == 0) f32_write_lse(p, it, r, m[a], l[a]);
  }
}

// Up to 16 rows: bound by the cache's bytes.  A warp takes NR rows (1, 2, 4) and every n-th run of eight keys, straight
// from global memory to registers (a key's row is one load of the warp, 4 columns to a lane); warps with other
// rows of the same keys find them in the first cache.  The 8 NR dot products of a run are summed over the lanes
// by halving: 31 shuffles for four rows leave lane 8 r + k with the score of row r and key k (4 / NR lanes each).  A warp's running maximum and
// sum are its own; the warps' parts are joined at the end of the item.
template <int NR>
__device__ void f32_few(const AttnParams& p, const WorkItem& it, float* smem) {
  const StepGeom& g = p.g;
  const int d = g.d, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int S = NR == 1 ? 2 : NR == 2 ? 1 : 0;                      // a score lies in 2^S neighbouring lanes
  const int blocks = it.nrows <= NR ? 1 : it.nrows <= 8 ? 2 : 4;       // of NR rows; warp % blocks takes one
  const int r0 = (warp % blocks) * NR, stride = 8 / blocks;
  const int kk = (lane >> S) & 7;
  const int c = 4 * lane;
  const bool has = c < d;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 q[NR], o[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    q[r] = o[r] = zero;
    if (has && r0 + r < it.nrows) {
      const int rr = it.row0 + r0 + r, tok = g.by_R(rr);
      q[r] = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.q) + (int64_t)tok * p.q_stride +
                                              (int64_t)(it.group * g.R + rr - tok * g.R) * d + c);
    }
  }
  const int row = r0 + (lane >> (3 + S));                                   // the row whose scores this lane ends up with
  const int own_vis = row >= it.nrows ? 0 : it.seq < 0 ? 1 : g.by_R(it.row0 + row) + it.own_off + 1;
  float m = -INFINITY, l = 0.f;
  const int runs = (g.key_tile + 7) / 8, end = it.t0 + it.n0;
  struct Run {
    int tile, sub, key, keys;             // key: this lane's (kk of the run), keys: of the run
    bool pre;
  };
  auto step_to = [&](Run& s) {            // the next run that holds a key; keys 0 at the end
    s.keys = 0;
    while (s.tile < end) {
      s.pre = s.tile < it.np;
      int key0;
      const int n = tile_keys(it, g, s.tile, &key0) - 8 * s.sub;
      if (n > 0) {
        s.keys = min(n, 8);
        s.key = key0 + 8 * s.sub + kk;
      }
      s.sub += stride;
      while (s.sub >= runs) {
        s.sub -= runs;
        ++s.tile;
      }
      if (n > 0) return;
    }
  };
  auto locate = [&](const Run& s) { return kk < s.keys ? key_at(p, it, s.pre, s.key) : (int64_t)-1; };
  auto load = [&](float4 (&x)[8], const float* pool, int64_t at) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t a = __shfl_sync(0xffffffffu, at, k << S);
      x[k] = has && a >= 0 ? __ldg(reinterpret_cast<const float4*>(pool + a + c)) : zero;
    }
  };
  Run cur{it.t0 + (warp / blocks) / runs, (warp / blocks) % runs, 0, 0, false}, next;
  step_to(cur);
  next = cur;
  step_to(next);
  int64_t at = locate(cur);
  float4 kf[8], vf[8];
  load(kf, p.kc, at);
  while (cur.keys > 0) {
    load(vf, p.vc, at);
    float s[8 * NR];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int k = 0; k < 8; ++k) s[r * 8 + k] = q[r].x * kf[k].x + q[r].y * kf[k].y + q[r].z * kf[k].z + q[r].w * kf[k].w;
#pragma unroll
    for (int n = 4 * NR, w = 16; w > 0; n >>= 1, w >>= 1) {
      const bool up = lane & w;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float send = up ? s[i] : s[i + n], keep = up ? s[i + n] : s[i];
        s[i] = keep + __shfl_xor_sync(0xffffffffu, send, w);
      }
      if (n == 0) s[0] += __shfl_xor_sync(0xffffffffu, s[0], w);
    }
    at = locate(next);
    load(kf, p.kc, at);
    const bool seen = own_vis > 0 && kk < cur.keys && (cur.pre || cur.key < own_vis);
    const float sc = seen ? s[0] : -INFINITY;
    float mx = sc;
#pragma unroll
    for (int x = 4; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x << S));
    const float m_new = fmaxf(m, mx), ref = m_new == -INFINITY ? 0.f : m_new;
    const float f = m == -INFINITY ? 0.f : expf((m - ref) * p.scale);
    const float e = expf((sc - ref) * p.scale);
    l = l * f + e;                        // this lane's keys alone
    m = m_new;
    const unsigned see = __ballot_sync(0xffffffffu, seen);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float fr = __shfl_sync(0xffffffffu, f, 8 * r << S);
      o[r].x *= fr;
      o[r].y *= fr;
      o[r].z *= fr;
      o[r].w *= fr;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float w = __shfl_sync(0xffffffffu, e, (8 * r + k) << S);
        if (see != ~0u && !(see >> ((8 * r + k) << S) & 1u)) continue;   // masked: whatever lies there
        o[r].x += w * vf[k].x;
        o[r].y += w * vf[k].y;
        o[r].z += w * vf[k].z;
        o[r].w += w * vf[k].w;
      }
    }
    cur = next;
    step_to(next);
  }
#pragma unroll
  for (int x = 4; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x << S);
  // ---- join the warps' parts
  float* po = smem;                                                     // [warp][4][128]
  float2* ml = reinterpret_cast<float2*>(smem + 8 * 4 * 128);           // [warp][4]
#pragma unroll
  for (int r = 0; r < NR; ++r)
    if (has) *reinterpret_cast<float4*>(po + (warp * 4 + r) * 128 + c) = o[r];
  if ((lane & ((8 << S) - 1)) == 0) ml[warp * 4 + (lane >> (3 + S))] = make_float2(m, l);
  __syncthreads();
  for (int r = warp; r < it.nrows; r += 8) {
    const int b = r / NR;
    float top = -INFINITY, sum = 0.f;
    for (int w = b; w < 8; w += blocks) top = fmaxf(top, ml[w * 4 + r % NR].x);
    const float ref = top == -INFINITY ? 0.f : top;
    float4 acc = zero;
    for (int w = b; w < 8; w += blocks) {
      const float2 s = ml[w * 4 + r % NR];
      const float f = s.x == -INFINITY ? 0.f : expf((s.x - ref) * p.scale);
      sum += f * s.y;
      const float4 v = has ? *reinterpret_cast<const float4*>(po + (w * 4 + r % NR) * 128 + c) : zero;
      acc.x += f * v.x;
      acc.y += f * v.y;
      acc.z += f * v.z;
      acc.w += f * v.w;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (has) f32_write(p, it, r, c, sum == 0.f ? zero : make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    if (lane == 0) f32_write_lse(p, it, r, top, sum);
  }
}

constexpr int kF32Smem = ((kF32Rows + 2 * kF32Keys) * 128 + kF32Keys * kF32Rows) * 4;       // twice on an SM
static_assert((8 * 4 * 128 + 8 * 4 * 2) * 4 <= kF32Smem, "f32_few's joining fits");

__global__ void __launch_bounds__(kF32Threads, 2) attention_f32_kernel(const __grid_constant__ AttnParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ int claim;
  pdl_enter();
  const StepGeom& g = p.g;
  const bool fits = plan_matches(g);
  const int n = fits ? g.head->n_items : 0;
  if ((!fits || n < 0) && threadIdx.x == 0) latch_status(&g.head->status, fits ? kStatusRange : kStatusInvalid);
  // as in the bf16 kernel: the first item by number, the others from the counter
  for (int i = blockIdx.x; i < n; i = claim) {
    const WorkItem it = load_item(g.items + i);
    __syncthreads();                      // claim and shared memory are free again
    if (threadIdx.x == 0) claim = gridDim.x + (int)atomicAdd(&g.head->claimed, 1u);
    float* smem = reinterpret_cast<float*>(smem_raw);
    if (it.nrows > kF32Few) f32_tile(p, it, smem);
    else if (it.nrows > 2) f32_few<4>(p, it, smem);
    else if (it.nrows == 2) f32_few<2>(p, it, smem);
    else f32_few<1>(p, it, smem);
    __syncthreads();
  }
  if (fits && threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(&g.head->done, 1u) == gridDim.x - 1) {
      g.head->claimed = 0;
      g.head->done = 0;
    }
  }
}

// ---------------------------------------------------------------- join
__device__ __forceinline__ void put4(float* dst, float4 v) { *reinterpret_cast<float4*>(dst) = v; }
__device__ __forceinline__ void put4(__nv_bfloat16* dst, float4 v) {
  *reinterpret_cast<uint2*>(dst) = make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
}

// One warp per row (token, head): out = sum_p w_p out_p / sum_p w_p, w_p = exp(lse_p - max lse),
// over the row's parts in a fixed order.  Rows that an item wrote whole are skipped; padding is zero.
template <typename E>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ AttnParams p) {
  pdl_enter();
  const StepGeom& g = p.g;
  const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (at >= (int64_t)g.T * g.H || !plan_matches(g) || g.head->n_items < 0) return;
  const int t = (int)(at / g.H), h = (int)(at - (int64_t)t * g.H);
  const int group = g.by_R(h), rr = t * g.R + h - group * g.R;
  const TokenInfo ti = g.tok[t];
  const PlanHeader& hd = *g.head;
  int n_pre = 0, pre0 = 0, pre_step = 0, n_own = 0, own0 = 0, own_step = 0;
  if (ti.seq >= 0 && (ti.own >= 0 || !g.separate)) {
    const SeqInfo si = g.seq[ti.seq];
    const SeqShape s = seq_shape(g, si.q0, si.q1, si.kv);
    const int local = rr - s.q0 * g.R, k = local / s.tr;
    const int tiles = key_tiles(g, s, (k + 1) * s.tr);
    int per;
    n_own = job_parts(tiles, s.tr > 128 ? 2 : 1, hd.unit, &per);
    if (n_own == 1 && !g.separate) return;
    if (tiles == 0) n_own = 0;
    own_step = s.nt == 1 ? s.rows : s.tr;
    own0 = si.part_row + (group * s.nt + k) * si.parts * own_step + local - k * s.tr;
    if (g.separate) {
      const int kp = rr / g.prefix_rows;
      n_pre = hd.prefix_parts;
      pre_step = g.prefix_rows;
      pre0 = (group * g.prefix_tiles + kp) * n_pre * pre_step + rr - kp * pre_step;
    }
  }
  const int n = n_pre + n_own;
  auto row_of = [&](int i) { return i < n_pre ? pre0 + i * pre_step : own0 + (i - n_pre) * own_step; };
  // eight parts' rows in flight, the first of them beside their log-sum-exps; an empty part's row is zero
  float4 v[8];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int x = 0; x < 8; ++x)
      v[x] = i0 + x < n && 4 * lane < g.d ? *reinterpret_cast<const float4*>(g.part_out + (int64_t)row_of(i0 + x) * g.d + 4 * lane)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  fetch(0);
  float mx = -INFINITY;
  for (int i = lane; i < n; i += 32) mx = fmaxf(mx, g.part_lse[row_of(i)]);
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float ref = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < n; i0 += 8) {
    if (i0 > 0) fetch(i0);
    const float w_mine = lane < 8 && i0 + lane < n ? expf(g.part_lse[row_of(i0 + lane)] - ref) : 0.f;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float w = __shfl_sync(0xffffffffu, w_mine, x);      // 0 beside the others' or of no part: 0 * NaN stays NaN
      sum += w;
      acc.x += w * v[x].x;
      acc.y += w * v[x].y;
      acc.z += w * v[x].z;
      acc.w += w * v[x].w;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (4 * lane < g.d)
    put4(static_cast<E*>(p.out) + at * g.d + 4 * lane, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  if (lane == 0 && p.lse) p.lse[at] = sum == 0.f ? -INFINITY : ref + logf(sum);
}

}  // namespace
}  // namespace aff

using namespace aff;

extern "C" aff_status affinity_prefix_attention(const void* q, int64_t q_stride, const aff_kv_cache* cache,
                                                const aff_step* step, float scale, void* out, float* lse, void* plan,
                                                size_t plan_bytes, aff_stream_t stream) {
  AttnParams p{};
  aff_status st = step_geom(step, cache, plan, &p.g);
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
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride = q_stride;
  p.out = out;
  p.lse = lse;
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.kc = static_cast<const float*>(cache->k);
  p.vc = static_cast<const float*>(cache->v);
  p.page_stride = cache->page_stride;
  p.group_stride = cache->group_stride;
  p.token_stride = cache->token_stride;
  const unsigned grid = (unsigned)(g.max_items < sms ? g.max_items : sms);
  if (g.dtype == AFF_FP32) {
    AFF_CUDA(cudaFuncSetAttribute(attention_f32_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kF32Smem));
    AFF_CUDA(launch_pdl(attention_f32_kernel, grid * 2, kF32Threads, kF32Smem, s, p));
  } else {
    p.halves = g.d > 64 ? 2 : 1;
    p.kd = (g.d + 15) / 16 * 16;
    p.box = g.tile_pages ? g.page_size : g.key_tile;
    const int tile = p.halves * kHalfBytes;
    static_assert(sizeof(Bars) <= 1024, "ring_stages leaves 1024 bytes for the barriers");
    p.stages = ring_stages(p.halves);
    const int smem = 1024 + (2 + p.stages) * tile + kStageOut + 2 * kRows * (int)sizeof(float2) + kFewBytes + (int)sizeof(Bars);
    CUtensorMap m[6];          // queries, keys, values; keys and values with whole rows; output
    const uint64_t tok = (uint64_t)cache->token_stride * 2, grp = (uint64_t)cache->group_stride * 2,
                   pag = (uint64_t)cache->page_stride * 2;
    const uint64_t dims[4] = {(uint64_t)g.d, (uint64_t)g.page_size, (uint64_t)g.G, (uint64_t)g.n_pages};
    const uint64_t str[3] = {tok, grp, pag};
    if ((st = map_16bit_sw128(&m[1], cache->k, 4, dims, str, (uint32_t)p.box, 1)) != AFF_OK) return st;
    if ((st = map_16bit_sw128(&m[2], cache->v, 4, dims, str, (uint32_t)p.box, 1)) != AFF_OK) return st;
    m[3] = m[1];
    m[4] = m[2];
    p.q_boxes = kRows % g.R == 0;
    m[0] = m[1];
    if (p.q_boxes) {
      const uint64_t qd[4] = {(uint64_t)g.d, (uint64_t)g.R, (uint64_t)g.G, (uint64_t)g.T};
      const uint64_t qs[3] = {(uint64_t)g.d * 2, (uint64_t)g.R * g.d * 2, (uint64_t)q_stride * 2};
      if ((st = map_16bit_sw128(&m[0], q, 4, qd, qs, (uint32_t)g.R, 1, (uint32_t)(kRows / g.R), 3)) != AFF_OK) return st;
    }
    m[5] = m[1];
    p.out_boxes = 32 % g.R == 0;
    if (p.out_boxes) {
      const uint64_t od[4] = {(uint64_t)g.d, (uint64_t)g.R, (uint64_t)g.G, (uint64_t)g.T};
      const uint64_t os[3] = {(uint64_t)g.d * 2, (uint64_t)g.R * g.d * 2, (uint64_t)g.H * g.d * 2};
      if ((st = map_16bit_sw128(&m[5], out, 4, od, os, (uint32_t)g.R, 1, (uint32_t)(32 / g.R), 3)) != AFF_OK) return st;
    }
    p.whole_rows = g.few && g.d == 128;
    if (p.whole_rows) {       // the halves as a dimension of their own
      const uint64_t dims5[5] = {64, (uint64_t)g.page_size, 2, (uint64_t)g.G, (uint64_t)g.n_pages};
      const uint64_t str5[4] = {tok, 128, grp, pag};
      if ((st = map_16bit_sw128(&m[3], cache->k, 5, dims5, str5, (uint32_t)p.box, 1, 2, 2)) != AFF_OK) return st;
      if ((st = map_16bit_sw128(&m[4], cache->v, 5, dims5, str5, (uint32_t)p.box, 1, 2, 2)) != AFF_OK) return st;
    }
    st = g.few ? launch_attention<true>(m, p, grid, smem, s) : launch_attention<false>(m, p, grid, smem, s);
    if (st != AFF_OK) return st;
  }
  if (g.may_split) {
    const unsigned blocks = (unsigned)(((int64_t)g.T * g.H + 7) / 8);
    if (g.dtype == AFF_BF16) AFF_CUDA(launch_pdl(join_kernel<__nv_bfloat16>, blocks, 256, 0, s, p));
    else AFF_CUDA(launch_pdl(join_kernel<float>, blocks, 256, 0, s, p));
  }
  return AFF_OK;
}
