// step.cuh -- the plan of one forward step: where each of its tokens stands,
// and the attention's work items.  Written by affinity_step_plan (step_plan.cu),
// read by affinity_kv_append (kv_append.cu) and affinity_prefix_attention
// (attention.cu) of every layer of the step, or by the same over a cache in
// 4 bits (kv4_append.cu, kv4_attention.cu).
//
// Rows.  Attention works on packed rows: row t * R + r of KV group g is query
// head g * R + r of token t, R = H / G.  The heads of a group share its keys and
// values, so a tile of rows meets each key tile once.
//
// Key tiles.  A tile is up to 128 keys of one segment (the prefix, or a sequence's
// own keys): as many whole pages as fit, or, for pages of more than 128 tokens, an
// equal cut of a page.  A page's share of a tile is one TMA box then, whatever the
// page size (a 128-key tile of 24-token pages would take boxes of 8 keys).
//
// Jobs and items.  A job is a tile of rows of one group against a run of key
// tiles.  A sequence's rows are cut into tiles of `big` rows (of
// `small` rows, one tile, when it has no more than that).  The shared prefix is
// read in one of two ways, chosen on the host from the shapes alone:
//   separate   its own jobs, whose row tiles run across sequences, so each key
//              tile of the prefix is loaded once per `big` rows of the whole
//              batch; a row then has parts from the prefix and from its own keys;
//   joined     as the first key tiles of every sequence's own jobs.
// Jobs longer than `unit` are cut into items along the keys; an item that is
// its rows' only one writes the output, the others write partial rows (fp32
// output and log-sum-exp), which the join kernel merges.
#pragma once

#include "affinity.h"

#include <cuda_runtime.h>

#include <cstdint>

namespace aff {

constexpr int kKeyTile = 128;            // most keys of a tile
constexpr int kFewRows = 16;             // most rows of an item that takes the few-rows path
constexpr int kKv4FewRows = 8;           // the same over a cache in 4 bits (kv4_attention.cu)
constexpr int kPlanSms = 152;            // SMs of a GB300: sizes the plan without a device

// Division of 0 <= x < 2^31 by a number known on the host: a multiply, an add and a shift, where the
// device's own division by a variable is some forty instructions at every place it is used.
struct FastDiv {
  uint32_t m = 1, shift = 0, d = 1;
  void set(uint32_t by) {
    d = by;
    shift = 0;
    while ((1ull << shift) < by) ++shift;
    m = (uint32_t)(((1ull << 32) * ((1ull << shift) - by)) / by + 1);
  }
#ifdef __CUDACC__
  __host__ __device__
#endif
  int operator()(int x) const {
    return (int)(((uint32_t)(((uint64_t)m * (uint32_t)x) >> 32) + (uint32_t)x) >> shift);
  }
};

struct TokenInfo {       // one per token of the step; 16 bytes
  int64_t slot;          // page << 32 | offset in it, of its own key; -1: padding
  int32_t own;           // index among its sequence's own tokens, -1: padding, -2: its page is no page of the pool
  int32_t seq;           // its sequence, -1: none
};

struct SeqInfo {         // one per sequence, for the join: what the plan was made from; 32 bytes
  int32_t q0, q1, kv;    // its tokens of the step, its own keys
  int32_t part_row;      // first partial row
  int32_t parts;         // partial rows' stride in parts: those of its last row tile, which has the most keys
  int32_t reserved[3];
};

struct WorkItem {        // 48 bytes
  int32_t row0, nrows, group, seq;   // packed rows row0 .. +nrows of `group`; seq -1: prefix alone, or padding
  int32_t t0, n0, n1, part_row;      // first key tile; tiles of stream 0 and 1; partial row of row0 (-1: the output)
  int32_t own_off, own_len, alt, np; // own index = token + own_off; own keys in view; see below; prefix tiles before own tiles
};
// alt == 0: stream s holds rows s*128 .. of the item and walks tiles t0 .. t0 + n_s - 1.
// alt == 1: at most 128 rows; both streams hold them, stream s walks tiles t0 + s, t0 + s + 2, ...
// alt == 2: few rows (StepGeom::few_rows), for which a tile is split over warps by its keys; n0 tiles.
// Its higher bits are 0 but for a call under way (attention.cu).

struct PlanHeader {      // at the start of the plan buffer; its first word is the status word
  uint32_t status;
  int32_t n_items;       // -1: the step was malformed
  int32_t unit;          // most cost (key tiles x streams) of an item; 0: jobs are not cut
  int32_t prefix_parts;  // separate: parts of each prefix job
  int32_t prefix_per;    // separate: key tiles of each part
  int32_t pad[3];
  uint32_t key[4];       // a hash of the geometry it was made for
  uint32_t claimed;      // items claimed beyond the first of every CTA, and CTAs done, in the call
  uint32_t done;         // under way; the last CTA sets both back to 0
  uint32_t few_claimed;  // the same of the kernel that takes the few-rows items of a cache in 4 bits
  uint32_t few_done;
  int32_t tile_end;      // over a cache in 4 bits: the items before it hold all that are not few-rows items,
  int32_t few_begin;     // and those from here on all that are
};

// Everything the kernels need to know of the step, by value.
struct StepGeom {
  int32_t T, B, H, G, R, d;
  int32_t page_size, dtype;
  int32_t pages_stride, prefix_len;
  int32_t key_tile;      // keys of a tile (see above)
  int32_t tile_pages;    // whole pages of a tile, 0 if a page has several tiles
  int32_t page_tiles;    // tiles of a page then, else 0
  int32_t np;            // key tiles of the prefix
  int32_t separate;      // the prefix has jobs of its own
  int32_t kv4;           // the cache is in 4 bits (kv4.cuh)
  int32_t few, few_rows; // items of at most few_rows rows take the few-rows path
  int32_t may_split;     // jobs may be cut (then the join kernel runs)
  int32_t small, big;    // row tiles
  int32_t cut_rows;      // partial rows for cuts: so many for every SM, twice
  int32_t prefix_rows;   // row tile of the prefix's jobs
  int32_t prefix_tiles;  // row tiles of the prefix's jobs
  int32_t max_items, max_part_rows;
  uint32_t key[4];       // of everything the plan depends on but the arrays' contents
  FastDiv by_R, by_G, by_page, by_tile, by_page_tiles;
  int64_t n_pages;
  const int32_t *q_start, *kv_len, *pages, *prefix_pages;
  // plan buffer
  PlanHeader* head;
  TokenInfo* tok;
  SeqInfo* seq;
  WorkItem* items;
  float* part_lse;
  float* part_out;
  size_t bytes;
};

// Validates (step, cache) and lays the plan out over `plan` (may be null).  kv4: `cache` stands for one in 4 bits.
aff_status step_geom(const aff_step* step, const aff_kv_cache* cache, void* plan, StepGeom* g, bool kv4 = false);

// The same for a cache in 4 bits.
aff_status kv4_geom(const aff_step* step, const aff_kv4_cache* cache, void* plan, StepGeom* g);

// The plan buffer of a call: present, aligned, large enough.
aff_status check_plan(const StepGeom& g, const void* plan, size_t plan_bytes);

// Merges the partial rows of an attention call into its output (attention.cu).
aff_status launch_join(const StepGeom& g, void* out, float* lse, cudaStream_t stream);

#ifdef __CUDACC__
__host__ __device__ inline int ceil_div_i(int a, int b) { return (a + b - 1) / b; }

// Key tiles of a segment of `len` keys.
__host__ __device__ __forceinline__ int segment_tiles(const StepGeom& g, int len) {
  if (g.tile_pages) return g.by_tile(len + g.key_tile - 1);
  const int pages = g.by_page(len);
  return pages * g.page_tiles + g.by_tile(len - pages * g.page_size + g.key_tile - 1);
}

// First key and number of keys of tile `idx` of a segment of `len` keys.
__device__ __forceinline__ int tile_span(const StepGeom& g, int len, int idx, int* key0) {
  if (g.tile_pages) {
    *key0 = idx * g.key_tile;
    return min(g.key_tile, len - *key0);
  }
  const int page = g.by_page_tiles(idx), in_page = (idx - page * g.page_tiles) * g.key_tile;
  *key0 = page * g.page_size + in_page;
  return min(min(g.key_tile, g.page_size - in_page), len - *key0);
}

struct SeqShape {        // what a sequence's jobs are cut from
  int32_t q0, q1, kv, rows, tr, nt;
};

__device__ __forceinline__ SeqShape seq_shape(const StepGeom& g, int q0, int q1, int kv) {
  SeqShape s;
  s.q0 = q0;
  s.q1 = q1;
  s.kv = kv;
  s.rows = (q1 - q0) * g.R;
  s.tr = s.rows <= g.small ? g.small : g.big;
  s.nt = (s.rows + s.tr - 1) / s.tr;
  return s;
}

// Own keys that the last of the first `upto` rows of a sequence sees.
__device__ __forceinline__ int keys_in_view(const StepGeom& g, const SeqShape& s, int upto) {
  const int last = s.rows > 0 ? g.by_R(min(upto, s.rows) - 1) : 0;
  return min(max(s.kv - (s.q1 - s.q0) + last + 1, 0), s.kv);
}

// Key tiles that the first `upto` rows of a sequence meet in its own jobs.
__device__ __forceinline__ int key_tiles(const StepGeom& g, const SeqShape& s, int upto) {
  const int v = keys_in_view(g, s, upto);
  return v == 0 ? 0 : segment_tiles(g, v) + (g.separate ? 0 : g.np);
}

// Parts of a job of `tiles` key tiles, `streams` row tiles at a time, and the key tiles of each.  `unit` counts in
// whole tiles, rounded up: the parts then never grow fewer as a job grows, which SeqInfo::parts rests on (a bound of
// unit / streams tiles that is no whole number gives 4 parts of 8 tiles and 3 of 9).
__device__ __forceinline__ int job_parts(int tiles, int streams, int unit, int* per) {
  *per = tiles;
  if (unit <= 0 || tiles <= 0) return 1;
  const int most = (unit + streams - 1) / streams;
  const int parts = (tiles + most - 1) / most;
  *per = (tiles + parts - 1) / parts;            // at most `most`, so these parts are needed: no fewer cover the tiles
  return parts;
}

__device__ __forceinline__ bool plan_matches(const StepGeom& g) {
  const PlanHeader& h = *g.head;
  return h.key[0] == g.key[0] && h.key[1] == g.key[1] && h.key[2] == g.key[2] && h.key[3] == g.key[3];
}
#endif

}  // namespace aff
