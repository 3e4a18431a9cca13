// attention_parts.cuh -- what the two tensor-core attention kernels (attention.cu, kv4_attention.cu) share: tensor
// memory and descriptor wrappers, waits, the walk over an item's key tiles, the ring of tiles and the issue of products.
// `Bars` is a kernel's own struct of barriers: abort_flag, slot_full[kSlots], slot_empty[kSlots], slot[kSlots].
#pragma once

#include "sm103_primitives.cuh"
#include "step.cuh"

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace aff {

constexpr int kRows = 128;                   // rows of a stream
constexpr int kHalfBytes = kRows * 128;      // a tile's 64-column half: 128 rows of 128 bytes
constexpr int kHalfKeys = kKeyTile / 2;      // scores are computed and turned into probabilities by half tiles
constexpr int kSlots = 4;                    // items on their way through the CTA
constexpr int kStageOut = 4 * 32 * 128;      // output staging: 32 rows of 128 bytes for each output warp
constexpr int kSmemMax = 227 * 1024;
constexpr float kRescale = 8.f;              // log2 growth of the maximum that O is rescaled for
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;              // O of stream s at kColO + 128 s; S at 128 s
constexpr uint32_t kStatusInvalid = 1;

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

template <class Bars>
__device__ __forceinline__ bool gave_up(const Bars* b) { return *reinterpret_cast<const volatile int*>(&b->abort_flag) != 0; }

// The whole warp waits, for 2 s at most; then the CTA gives up: every later wait ends soon, what is computed
// is thrown away with the status word, and the roles leave at their next item.  Little code, because the
// roles' code together has to stay in the instruction cache: the clock is read every 256 polls (a poll
// suspends for a while by itself), and only its low 32 bits.
template <class Bars>
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
template <class Bars>
__device__ __forceinline__ WorkItem uniform_item(const Bars* bars, int k) {
  WorkItem it = load_item(&bars->slot[k % kSlots]);
  int* v = reinterpret_cast<int*>(&it);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(WorkItem) / 4); ++i) v[i] = __shfl_sync(0xffffffffu, v[i], 0);
  return it;
}
// Waits for slot k; false when there is no item left, or the CTA has given up.
template <class Bars>
__device__ __forceinline__ bool slot_wait(Bars* b, int k) {
  wait_on(&b->slot_full[k % kSlots], (k / kSlots) & 1, b);
  return __all_sync(0xffffffffu, !gave_up(b) && b->slot[k % kSlots].row0 >= 0);
}
template <class Bars>
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

// Own keys below this are seen by every row of the item (its first row sees the fewest).
__device__ __forceinline__ int all_see(const WorkItem& it, const StepGeom& g) {
  return it.seq < 0 ? INT32_MAX : g.by_R(it.row0) + it.own_off + 1;
}

// One lane of the (converged) warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

// An item's tiles pass through the ring in order, keys then values of tile t0, t0 + 1, ..
__device__ __forceinline__ int item_tiles(const WorkItem& it) { return it.alt ? it.n0 + it.n1 : it.n1; }   // n0 <= n1

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

// 16 bytes to / from row `row` of a warp's 32 x 128-byte staging block, in place c of 8.
__device__ __forceinline__ uint32_t stage_at(uint32_t base, int row, int c) { return base + row * 128 + ((c ^ (row & 7)) << 4); }

// Transpose of an 8 x 8 matrix of 16-bit elements, two to a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

}  // namespace aff
