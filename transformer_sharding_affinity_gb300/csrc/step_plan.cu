// step_plan.cu -- affinity_step_plan: one launch that writes a step's plan
// (step.cuh).  Block 0 cuts the jobs; the other blocks fill the token table.
// Once a step, not once a layer, and bound by latency: block 0's passes over the
// sequences (kept in shared memory) and the items' stores.  1 sequence 13 us, 64
// sequences 18 us, 256 sequences 27 us.
#include "affinity.h"
#include "internal.h"
#include "launch.cuh"
#include "sm103_primitives.cuh"
#include "step.cuh"

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

namespace aff {
namespace {

constexpr int kThreads = 1024;
// Items that a cut of unequal jobs aims at for each SM (64 single tokens of ragged sequences behind 8192 keys:
// 74 us with 2, 70 with 4 and 8).
constexpr int kItemsPerSm = 4;
constexpr int kMinUnit = 4;       // least cost of an item then
constexpr int kMaxParts = 64;     // most parts that equal jobs are cut into

__device__ int64_t warp_sum(int64_t v) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the block; the result is in every thread.
__device__ int64_t block_sum(int64_t v, int64_t* sh) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(sh[threadIdx.x & 31]);
}

__device__ int warp_inclusive(int v) {
  const int lane = threadIdx.x & 31;
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Sum over the threads before this one; *total over the block.
__device__ int block_exclusive(int v, int* total, int* sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int incl = warp_inclusive(v);
  __syncthreads();
  if (lane == 31) sh[warp] = incl;
  __syncthreads();
  const int warps = warp_inclusive(sh[lane]);
  *total = __shfl_sync(0xffffffffu, warps, 31);
  return __shfl_sync(0xffffffffu, warps, warp) - __shfl_sync(0xffffffffu, sh[lane], warp) + incl - v;
}

// Parts (1 .. most) of each of `jobs` equal jobs of `cost`: the least of the time of the fullest slot, where an
// item takes its cost and `start` for its beginning and end, and of a part's trip through memory.  A unit of cost
// is `tile` times as long as such a trip.  Warp-wide.
__device__ int best_parts(int64_t jobs, int64_t cost, int most, int slots, int tile, int start) {
  int64_t best = INT64_MAX;
  for (int parts = 1 + (threadIdx.x & 31); parts <= kMaxParts; parts += 32) {
    if (parts > most || parts > cost) continue;
    const int64_t rounds = (jobs * parts + slots - 1) / slots;
    best = min(best, (rounds * ((cost + parts - 1) / parts * tile + start) + parts) << 8 | parts);
  }
  for (int o = 16; o > 0; o >>= 1) best = min(best, (int64_t)__shfl_xor_sync(0xffffffffu, best, o));
  return best == INT64_MAX ? 1 : (int)(best & 255);
}

// A sequence's (row tile, group) pairs, late row tiles first: they have the most keys.
struct Job {
  int k, group, tiles, parts, per, streams;
};

__device__ __forceinline__ Job job_of(const StepGeom& g, const SeqShape& s, int i, int unit) {
  Job j;
  const int q = g.by_G(i);
  j.k = s.nt - 1 - q;
  j.group = i - q * g.G;
  j.streams = s.tr > 128 ? 2 : 1;
  j.tiles = key_tiles(g, s, (j.k + 1) * s.tr);
  j.parts = job_parts(j.tiles, j.streams, unit, &j.per);
  if (j.tiles == 0 && g.separate) j.parts = 0;     // the join writes such rows
  return j;
}

// One block.  Sequences are taken kThreads at a time, one to a thread, their numbers kept in shared memory
// (reloaded only when there are more of them); their jobs are then cut by a warp each.
__device__ void plan_items(const StepGeom& g) {
  __shared__ int64_t wide_sh[32];
  __shared__ int sh[32];
  __shared__ int s_q0[kThreads], s_q1[kThreads], s_kv[kThreads], s_item[kThreads], s_row[kThreads], s_most[kThreads];
  __shared__ int s_min, s_max, s_parts[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, me = threadIdx.x;
  if (me == 0) {
    s_min = INT32_MAX;
    s_max = 0;
  }
  auto load = [&](int b) {       // sequence b as given; false if it is malformed
    s_q0[me] = s_q1[me] = s_kv[me] = 0;
    if (b >= g.B) return true;
    const int q0 = g.q_start[b], q1 = g.q_start[b + 1], kv = g.kv_len[b];
    const bool good = !(b == 0 && q0 != 0) && q1 >= q0 && q0 >= 0 && q1 <= g.T && kv >= 0 &&
                      kv <= (int64_t)g.pages_stride * g.page_size;
    if (good) {
      s_q0[me] = q0;
      s_q1[me] = q1;
      s_kv[me] = kv;
    }
    return good;
  };
  auto shape = [&](int i) { return seq_shape(g, s_q0[i], s_q1[i], s_kv[i]); };
  const bool one_load = g.B <= kThreads;

  // ---- check the batch; the cost of all own jobs of one group, in key tiles x streams, and their extremes
  int64_t cost = 0, jobs = 0, rows_all = 0, bad = 0;
  int least = INT32_MAX, most_cost = 0;
  for (int b0 = 0; b0 < g.B; b0 += kThreads) {
    if (!load(b0 + me)) bad = 1;
    if (!g.may_split) continue;
    const SeqShape s = shape(me);
    rows_all += s.nt <= 1 ? s.rows : s.nt * s.tr;
    for (int k = 0; k < s.nt; ++k) {
      const int c = key_tiles(g, s, (k + 1) * s.tr) * (s.tr > 128 ? 2 : 1);
      if (c == 0) continue;
      cost += c;
      ++jobs;
      least = min(least, c);
      most_cost = max(most_cost, c);
    }
  }
  if (block_sum(bad, wide_sh)) {
    if (me == 0) {
      g.head->n_items = -1;
      latch_status(&g.head->status, kStatusRange);
    }
    return;
  }

  // ---- how jobs are cut
  const int prefix_streams = g.prefix_rows > 128 ? 2 : 1;
  int unit = 0, prefix_parts = 0, prefix_per = 0;
  if (g.may_split) {
    cost = block_sum(cost, wide_sh);
    jobs = block_sum(jobs, wide_sh);
    rows_all = block_sum(rows_all, wide_sh);
    least = __reduce_min_sync(0xffffffffu, least);
    most_cost = __reduce_max_sync(0xffffffffu, most_cost);
    if (lane == 0) {
      atomicMin(&s_min, least);
      atomicMax(&s_max, most_cost);
    }
    __syncthreads();
    // fp32: two CTAs per SM, tiles that take some four times as long
    const bool f32 = g.dtype != AFF_BF16;
    const int slots = f32 ? 2 * kPlanSms : kPlanSms, tile = f32 ? 4 : 1;
    const int start = g.few ? 2 : 5;      // an item's beginning and end, in the cost of a bf16 tile
    if (warp < 2) {                                // warp 0: own jobs, warp 1: the prefix's
      // half of the room for cuts (a row tile for every SM and stream) each
      const int64_t row_jobs = (warp ? (int64_t)g.prefix_tiles * g.prefix_rows : rows_all) * g.G;     // rows of a part
      const int64_t most = 1 + (int64_t)kPlanSms * g.big / max(row_jobs, (int64_t)1);
      const int parts = warp ? best_parts((int64_t)g.prefix_tiles * g.G, (int64_t)g.np * prefix_streams,
                                          (int)min(most, (int64_t)kMaxParts), slots, tile, start)
                             : best_parts(jobs * g.G, s_max, (int)min(most, (int64_t)kMaxParts), slots, tile, start);
      if (lane == 0) s_parts[warp] = parts;
    }
    __syncthreads();
    if (g.separate) {
      prefix_per = (g.np + s_parts[1] - 1) / s_parts[1];
      prefix_parts = (g.np + prefix_per - 1) / prefix_per;
    }
    // equal jobs: the best number of parts; unequal ones: a few items for every SM to even out with
    const int64_t aim = slots * kItemsPerSm;
    if (s_max > 0 && s_min >= s_max - s_max / 8) unit = (s_max + s_parts[0] - 1) / s_parts[0];
    else unit = (int)min(max((int64_t)kMinUnit / tile, (cost * g.G + aim - 1) / aim), (int64_t)INT32_MAX / 4);
  }

  // ---- the smallest unit (by doubling) whose partial rows and items fit; uncut jobs always do
  while (unit > 0) {
    int64_t rows = 0, items = 0;
    for (int b0 = 0; b0 < g.B; b0 += kThreads) {
      if (!one_load) load(b0 + me);
      const SeqShape s = shape(me);
      if (s.rows == 0) continue;
      int per;
      const int most = job_parts(key_tiles(g, s, s.rows), s.tr > 128 ? 2 : 1, unit, &per);
      if (g.separate || most > 1) rows += (int64_t)most * g.G * (s.nt == 1 ? s.rows : s.nt * s.tr);
      items += (int64_t)most * s.nt * g.G;
    }
    const int64_t prefix_jobs = (int64_t)prefix_parts * g.prefix_tiles * g.G;
    rows = block_sum(rows, wide_sh) + prefix_jobs * g.prefix_rows;
    items = block_sum(items, wide_sh) + prefix_jobs;
    if (rows <= g.max_part_rows && items <= g.max_items) break;
    unit = unit > (1 << 28) ? 0 : unit * 2;
    if (unit == 0 && g.separate) {               // nothing is cut
      prefix_per = g.np;
      prefix_parts = 1;
    }
  }

  // ---- first item and first partial row of every sequence, then its items
  const int prefix_items = prefix_parts * g.prefix_tiles * g.G;
  int item_base = prefix_items;
  int row_base = prefix_parts * g.prefix_tiles * g.prefix_rows * g.G;
  for (int b0 = 0; b0 < g.B; b0 += kThreads) {
    if (!one_load) {
      __syncthreads();
      load(b0 + me);
    }
    const SeqShape s = shape(me);
    int n_items = 0, n_rows = 0, most = 0, total;
    if (s.rows > 0) {
      int per;
      most = job_parts(key_tiles(g, s, s.rows), s.tr > 128 ? 2 : 1, unit, &per);
      if (g.separate || most > 1) n_rows = most * g.G * (s.nt == 1 ? s.rows : s.nt * s.tr);
      if (most == 1 && !g.separate) n_items = s.nt * g.G;      // every job, whether it has keys or not
      else
        for (int k = 0; k < s.nt; ++k) n_items += job_of(g, s, k * g.G, unit).parts * g.G;
    }
    s_item[me] = item_base + block_exclusive(n_items, &total, sh);
    item_base += total;
    s_row[me] = row_base + block_exclusive(n_rows, &total, sh);
    row_base += total;
    s_most[me] = most;
    if (b0 + me < g.B) g.seq[b0 + me] = SeqInfo{s.q0, s.q1, s.kv, s_row[me], most, {0, 0, 0}};
    __syncthreads();
    for (int x = warp; x < min(kThreads, g.B - b0); x += kThreads / 32) {
      const SeqShape s = shape(x);
      const int n_jobs = s.nt * g.G;
      int at = s_item[x];
      for (int i0 = 0; i0 < n_jobs; i0 += 32) {
        const int i = i0 + lane;
        Job j{};
        if (i < n_jobs) j = job_of(g, s, i, unit);
        const int incl = warp_inclusive(j.parts);
        int w = at + incl - j.parts;
        at += __shfl_sync(0xffffffffu, incl, 31);
        if (i >= n_jobs) continue;
        const int r0 = j.k * s.tr;
        const int nrows = min(s.tr, s.rows - r0);
        const int slot_rows = s.nt == 1 ? s.rows : s.tr;
        const bool direct = j.parts == 1 && !g.separate;
        const int alt = g.dtype != AFF_BF16 ? 0 : g.few && nrows <= kFewRows ? 2 : nrows <= 128;
        const int first = key_tiles(g, s, r0 + 128);    // key tiles that stream 0's rows meet
        WorkItem it;
        it.row0 = s.q0 * g.R + r0;
        it.nrows = nrows;
        it.group = j.group;
        it.seq = b0 + x;
        it.own_off = s.kv - s.q1;                  // token t has own index kv - (q1 - q0) + t - q0
        it.own_len = keys_in_view(g, s, r0 + nrows);
        it.alt = alt;
        it.np = g.separate ? 0 : g.np;
        for (int p = 0; p < j.parts; ++p, ++w) {
          if (w >= g.max_items) break;
          it.t0 = p * j.per;
          const int n = min(j.per, j.tiles - it.t0);
          if (g.dtype != AFF_BF16 || alt == 2) {
            it.n0 = n;
            it.n1 = 0;
          } else if (alt) {
            it.n0 = (n + 1) / 2;
            it.n1 = n / 2;
          } else {
            it.n0 = min(max(first - it.t0, 0), n);
            it.n1 = n;
          }
          it.part_row = direct ? -1 : s_row[x] + ((j.group * s.nt + j.k) * s_most[x] + p) * slot_rows;
          g.items[w] = it;
        }
      }
    }
  }

  // ---- the prefix's items, which come first: they are the longest.  (Spread among the others, to keep
  // the tensor cores and memory busy together, they ended late: 420 us instead of 345 for 256 sequences
  // behind 32768 tokens.)  Row tiles of one key run next to each other, then groups, then runs.
  for (int i = threadIdx.x; i < prefix_items; i += kThreads) {
    if (i >= g.max_items) break;
    const int k = i % g.prefix_tiles, rest = i / g.prefix_tiles;
    const int group = rest % g.G, p = rest / g.G;
    WorkItem it;
    it.row0 = k * g.prefix_rows;
    it.nrows = min(g.prefix_rows, g.T * g.R - it.row0);
    it.group = group;
    it.seq = -1;
    it.t0 = p * prefix_per;
    const int n = min(prefix_per, g.np - it.t0);
    it.alt = g.dtype != AFF_BF16 ? 0 : g.few && it.nrows <= kFewRows ? 2 : it.nrows <= 128;
    it.n0 = it.alt == 1 ? (n + 1) / 2 : n;
    it.n1 = it.alt == 1 ? n / 2 : it.alt == 2 || g.dtype != AFF_BF16 ? 0 : n;
    it.part_row = ((group * g.prefix_tiles + k) * prefix_parts + p) * g.prefix_rows;
    it.own_off = 0;
    it.own_len = 0;
    it.np = g.np;
    g.items[i] = it;
  }

  // ---- rows of tokens that belong to no sequence: the output is zero (the join writes it when it runs)
  const int tail = g.T - min(max(g.q_start[g.B], 0), g.T);
  if (tail > 0 && !g.may_split && !g.separate) {
    const int row0 = (g.T - tail) * g.R, n = ceil_div_i(tail * g.R, g.big);
    for (int i = threadIdx.x; i < n * g.G; i += kThreads) {
      if (item_base + i >= g.max_items) break;
      const int k = i / g.G;
      WorkItem it{};
      it.row0 = row0 + k * g.big;
      it.nrows = min(g.big, g.T * g.R - it.row0);
      it.group = i % g.G;
      it.seq = -1;
      it.part_row = -1;
      g.items[item_base + i] = it;
    }
    item_base += n * g.G;
  }
  if (threadIdx.x == 0) {
    PlanHeader& h = *g.head;
    h.n_items = min(item_base, g.max_items);
    h.unit = unit;
    h.prefix_parts = prefix_parts;
    h.prefix_per = prefix_per;
  }
}

__global__ void __launch_bounds__(kThreads) step_plan_kernel(const __grid_constant__ StepGeom g) {
  pdl_enter();
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < 4; ++i) g.head->key[i] = g.key[i];
    }
    plan_items(g);
    return;
  }
  // the token table: the last sequence that starts at or before the token, if it holds it
  const int t = (blockIdx.x - 1) * kThreads + threadIdx.x;
  if (t >= g.T) return;
  TokenInfo ti{-1, -1, -1};
  int lo = 0, hi = g.B;            // q_start[lo] <= t < q_start[hi] when the starts are in order
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (g.q_start[mid] <= t) lo = mid; else hi = mid;
  }
  const int q0 = g.q_start[lo], q1 = g.q_start[lo + 1], kv = g.kv_len[lo];
  if (t >= q0 && t < q1) {
    const int64_t own = (int64_t)kv - (q1 - q0) + (t - q0);
    ti.seq = lo;
    if (own >= 0 && own < (int64_t)g.pages_stride * g.page_size) {
      const int page = g.pages[(int64_t)lo * g.pages_stride + own / g.page_size];
      if (page >= 0 && page < g.n_pages) {
        ti.own = (int)own;
        ti.slot = (int64_t)page << 32 | own % g.page_size;
      } else {
        ti.own = -2;
        latch_status(&g.head->status, kStatusRange);
      }
    }
  }
  g.tok[t] = ti;
}

}  // namespace

aff_status check_plan(const StepGeom& g, const void* plan, size_t plan_bytes) {
  if (!plan || plan_bytes < g.bytes || (reinterpret_cast<uintptr_t>(plan) & 255u)) return AFF_ERR_WORKSPACE;
  return AFF_OK;
}

aff_status step_geom(const aff_step* st, const aff_kv_cache* c, void* plan, StepGeom* out) {
  if (!st || !c) return AFF_ERR_INVALID_ARG;
  if (c->dtype != AFF_BF16 && c->dtype != AFF_FP32) return AFF_ERR_UNSUPPORTED_DTYPE;
  if (!c->k || !c->v || !st->q_start || !st->kv_len || !st->pages) return AFF_ERR_INVALID_ARG;
  if (c->G < 1 || c->page_size < 1 || c->d_head < 1 || c->n_pages < 1 || st->T < 1 || st->B < 1 || st->H < 1 ||
      st->pages_stride < 1 || st->prefix_len < 0 || (st->prefix_len > 0 && !st->prefix_pages))
    return AFF_ERR_INVALID_ARG;
  const int es = c->dtype == AFF_BF16 ? 2 : 4;
  const int64_t lim = (int64_t)1 << 30;
  if (st->H % c->G || st->H > 4096 || c->d_head > 256 || c->d_head * es % 16 || c->page_size % 8 ||
      c->page_size > (1 << 20) || c->n_pages > INT32_MAX || st->T > lim / st->H || st->B > (1 << 20) ||
      st->prefix_len > lim || st->pages_stride > lim / c->page_size)
    return AFF_ERR_UNSUPPORTED_SHAPE;
  if (c->page_stride < 0 || c->group_stride < 0 || c->token_stride < c->d_head) return AFF_ERR_INVALID_ARG;
  if (c->page_stride * es % 16 || c->group_stride * es % 16 || c->token_stride * es % 16) return AFF_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) & 15u) return AFF_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(st->q_start) | reinterpret_cast<uintptr_t>(st->kv_len) |
       reinterpret_cast<uintptr_t>(st->pages) | reinterpret_cast<uintptr_t>(st->prefix_pages)) & 3u)
    return AFF_ERR_ALIGNMENT;
  StepGeom g{};
  g.T = (int)st->T;
  g.B = st->B;
  g.H = st->H;
  g.G = c->G;
  g.R = st->H / c->G;
  g.d = c->d_head;
  g.page_size = c->page_size;
  g.dtype = c->dtype;
  g.pages_stride = (int)st->pages_stride;
  g.prefix_len = (int)st->prefix_len;
  g.n_pages = c->n_pages;
  g.q_start = st->q_start;
  g.kv_len = st->kv_len;
  g.pages = st->pages;
  g.prefix_pages = st->prefix_pages;
  if (g.page_size <= kKeyTile) {
    g.tile_pages = kKeyTile / g.page_size;
    g.key_tile = g.tile_pages * g.page_size;
  } else {
    g.page_tiles = (g.page_size + kKeyTile - 1) / kKeyTile;
    g.key_tile = (g.page_size / g.page_tiles + (g.page_size % g.page_tiles != 0) + 7) / 8 * 8;
    g.page_tiles = (g.page_size + g.key_tile - 1) / g.key_tile;
  }
  g.by_R.set((uint32_t)g.R);
  g.by_G.set((uint32_t)g.G);
  g.by_page.set((uint32_t)g.page_size);
  g.by_tile.set((uint32_t)g.key_tile);
  g.by_page_tiles.set((uint32_t)std::max(g.page_tiles, 1));
  g.np = segment_tiles(g, g.prefix_len);
  const int64_t all[10] = {g.T, g.B, g.H, g.G, g.d, g.page_size, g.pages_stride, g.prefix_len, g.dtype, g.n_pages};
  for (int i = 0; i < 4; ++i) {
    uint64_t h = 0x9e3779b97f4a7c15ull * (i + 1);
    for (int64_t v : all) {
      h = (h ^ (uint64_t)v) * 0xbf58476d1ce4e5b9ull;
      h ^= h >> 29;
    }
    g.key[i] = (uint32_t)(h >> 16);
  }
  const bool bf = c->dtype == AFF_BF16;
  g.small = bf ? 128 : 16;
  g.big = bf ? 256 : 64;
  const int64_t rows = (int64_t)g.T * g.R;
  // Jobs of its own for the prefix: worth it while sequences have less than a row tile on average, which
  // would then be mostly idle for every key of the prefix (64 single tokens behind 8192 keys: 69 us, 359
  // without; 16 x 50 tokens, 100 rows each, behind 4000: 67 and 100; 64 x 33 behind 2000: 95 and 223; fp32,
  // 17 x 30 tokens behind 2145: 328 and 369).  It goes by the whole step, whatever the prefix's length: single tokens
  // beside a long prompt each read the prefix with their own keys.
  g.separate = g.prefix_len > 0 && g.B > 1 && rows < (int64_t)g.B * (bf ? g.small : g.big);
  // The few-rows path where sequences have few rows on average (64 single tokens: 69 us, 98 without); the kernel
  // without it is faster (64 x 1024 tokens: 280 us, 338 with it; 8 x 17 tokens, 34 rows each, over 3000 keys: 48 and
  // 50).  It goes by the whole step: single tokens beside prompts take the tensor tiles.
  g.few = bf && rows <= (int64_t)g.B * 32;
  g.prefix_rows = rows <= g.small ? g.small : g.big;
  g.prefix_tiles = g.separate ? (int)((rows + g.prefix_rows - 1) / g.prefix_rows) : 0;
  // Most (row tile, group) pairs: each sequence ends in at most one part-filled tile.
  const int64_t tiles = rows / g.big + g.B + 1;
  const int64_t jobs = (tiles + g.prefix_tiles) * g.G;
  const int64_t full = rows / g.big * g.G;
  g.may_split = g.separate || full < 2 * kPlanSms;
  const int64_t items = 2 * jobs + (int64_t)kPlanSms * 2 * kItemsPerSm + 2 * g.G + 64;
  int64_t part_rows = 0;
  if (g.may_split) {
    // Uncut jobs: with the prefix apart every row has a part from the prefix and one of its own
    // (a sequence of several row tiles rounds up to whole ones); joined, they write the output.
    // On top of that, room for cuts.
    const int64_t multi = std::min<int64_t>(g.B, rows / g.small + 1);
    part_rows = (int64_t)kPlanSms * 2 * g.big;
    if (g.separate) part_rows += ((int64_t)g.prefix_tiles * g.prefix_rows + rows + multi * g.big) * g.G;
  }
  if (items > INT32_MAX / 64 || part_rows > INT32_MAX / 2) return AFF_ERR_UNSUPPORTED_SHAPE;
  g.max_items = (int)items;
  g.max_part_rows = (int)part_rows;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  uint8_t* base = static_cast<uint8_t*>(plan);
  g.head = reinterpret_cast<PlanHeader*>(base + take(256));
  g.tok = reinterpret_cast<TokenInfo*>(base + take((size_t)g.T * sizeof(TokenInfo)));
  g.seq = reinterpret_cast<SeqInfo*>(base + take((size_t)g.B * sizeof(SeqInfo)));
  g.items = reinterpret_cast<WorkItem*>(base + take((size_t)g.max_items * sizeof(WorkItem)));
  g.part_lse = reinterpret_cast<float*>(base + take((size_t)part_rows * 4));
  g.part_out = reinterpret_cast<float*>(base + take((size_t)part_rows * g.d * 4));
  g.bytes = off;
  *out = g;
  return AFF_OK;
}

}  // namespace aff

using namespace aff;

extern "C" {

aff_status affinity_step_plan_size(const aff_step* step, const aff_kv_cache* cache, size_t* bytes) {
  if (!bytes) return AFF_ERR_INVALID_ARG;
  StepGeom g;
  aff_status st = step_geom(step, cache, nullptr, &g);
  if (st != AFF_OK) return st;
  *bytes = g.bytes;
  return AFF_OK;
}

aff_status affinity_step_plan(const aff_step* step, const aff_kv_cache* cache, void* plan, size_t plan_bytes,
                              aff_stream_t stream) {
  StepGeom g;
  aff_status st = step_geom(step, cache, plan, &g);
  if (st != AFF_OK) return st;
  if ((st = check_plan(g, plan, plan_bytes)) != AFF_OK) return st;
  int sms = 0;
  if ((st = check_device(&sms)) != AFF_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  AFF_CUDA(cudaMemsetAsync(plan, 0, sizeof(PlanHeader), s));
  AFF_CUDA(launch_pdl(step_plan_kernel, 1 + (g.T + kThreads - 1) / kThreads, kThreads, 0, s, g));
  return AFF_OK;
}

}  // extern "C"
