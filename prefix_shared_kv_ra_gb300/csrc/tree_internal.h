// tree_internal.h -- workspace, parameters and request checks shared by the kernels of ra_tree_attention.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ra.h"
#include "api_common.h"
#include "ra_ptx.cuh"
#include "small_plan.cuh"

namespace ra {

constexpr int kTreeSms = 152;        // GB300; a constant, so that the workspace does not depend on the device
constexpr int kTreeSmallLeast = 2;   // units of a small call's shortest piece
constexpr int kTreeNarrowRows = 32;  // rows (drafted tokens x GQA group) of a narrow item
constexpr int kTreeTiledRows = 128;  // rows per request up to which a small call takes several narrow items

// How a call is cut: a narrow item (at most 32 rows of a kv head, on mma.sync) streams whole slot rows of a head
// group, a wide one has up to 256 rows of one kv head on the tcgen05 kernel.  A call is narrow if its requests'
// rows fit one item, and in several items per request (its keys read once per item) if it is small.
struct TreeShape {
  bool narrow;
  int32_t q_tiles;          // items that hold a request's drafted tokens, at the host's bound
  int32_t row_blocks;       // narrow: 16-row blocks per kv head (1 or 2)
  int32_t hpc;              // narrow: kv heads per item
  int32_t per_sm;           // CTAs of the attention kernel per SM
  int32_t heads;            // items per (request, query tile, split): kv heads, or head groups when narrow
  int32_t tokens_per_item;  // drafted tokens of a query tile
  int32_t unit;             // keys per unit of the plan (a key tile, or a slab pair)
  int32_t waves;            // a batch with at least this many unsplit items per SM is only balanced
  int32_t overhead;         // an item's fixed cost in units
  int32_t split_overhead;   // that of a split item: its partials are written and read again
};

// Consumer warps of a narrow CTA: as many as their registers (accumulators of D values per row) allow.
constexpr int tree_consumers(int32_t head_dim) { return head_dim == 128 ? 8 : 16; }

// Whether requests of these bounds may be cut into several narrow items.
inline bool tree_tileable(int32_t hq, int32_t hkv, int32_t max_draft) {
  const int64_t group = hq / hkv, rows = max_draft * group;
  return rows > kTreeNarrowRows && rows <= kTreeTiledRows && group <= kTreeNarrowRows;
}

inline TreeShape tree_shape(int32_t hq, int32_t hkv, int32_t head_dim, int32_t max_draft, bool tiled) {
  TreeShape s{};
  const int32_t group = hq / hkv;
  const int64_t rows = static_cast<int64_t>(max_draft) * group;
  s.narrow = rows <= kTreeNarrowRows || tiled;
  if (s.narrow) {
    s.tokens_per_item = rows <= kTreeNarrowRows ? max_draft : kTreeNarrowRows / group;
    s.row_blocks = rows <= 16 ? 1 : 2;
    for (s.hpc = tree_consumers(head_dim) / s.row_blocks; hkv % s.hpc != 0;) --s.hpc;
    // a CTA of few consumer warps waits on its own chain of slab, scores, softmax and product: two share an SM
    s.per_sm = s.hpc * s.row_blocks <= 2 ? 2 : 1;
    s.heads = hkv / s.hpc;
    s.unit = 32;
    s.waves = 3;
    s.overhead = 1;
    s.split_overhead = 1 + s.row_blocks;  // a row's fp32 partial costs what 2 of a unit's 32 keys do
  } else {
    s.heads = hkv;
    s.per_sm = 1;
    s.tokens_per_item = 2 * (128 / group);
    s.unit = 128;
    s.waves = 2;
    s.overhead = 3;
    s.split_overhead = 3 + static_cast<int32_t>((rows < 256 ? rows : 256) / 96);
  }
  s.q_tiles = (max_draft + s.tokens_per_item - 1) / s.tokens_per_item;
  return s;
}

struct TreeWorkspace {
  int32_t* header;     // [8]: listed items, claim counter, keys per split, merges
  int32_t* items;      // [8 * cap]: request, query tile, split, partial slot (-1: unsplit); P, T, table row, q row
  int32_t* merges;     // [4 * cap_merge]: request, query tile, first partial slot, splits
  int32_t* bad;        // a drafted token's V holds a value that is not finite: [batch * hkv], or for a small
                       // call [pieces * hkv] (of the keys the piece read)
  float* part_o;
  float* part_lse;
  int64_t cap, cap_parts;
  int32_t part_rows;
  size_t total;
};

// Items: one per (request, query tile) plus the extra ones of split ranges.  A range is split only if it is
// longer than the chunk, and the chunk is at least total / (waves * kTreeSms) (all ranges times the heads):
// the split ranges' pieces number at most sum ceil(n / c) <= sum 2 n / c <= 2 * waves * kTreeSms / heads.
inline TreeWorkspace layout_tree(int32_t batch, int64_t total_q, int32_t hq, int32_t hkv, int32_t d, int32_t max_draft,
                                 const TreeShape& sh, void* base) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const int32_t group = hq / hkv;
  TreeWorkspace w{};
  w.cap_parts = 2 * sh.waves * kTreeSms / sh.heads;
  w.cap = (total_q + sh.tokens_per_item - 1) / sh.tokens_per_item + batch + w.cap_parts;
  const int64_t rows = static_cast<int64_t>(max_draft < sh.tokens_per_item ? max_draft : sh.tokens_per_item) * group;
  w.part_rows = static_cast<int32_t>(rows);
  uint8_t* b = workspace_base(base);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* at = b ? b + off : nullptr;
    off += up(bytes);
    return at;
  };
  w.header = reinterpret_cast<int32_t*>(take(32));
  w.items = reinterpret_cast<int32_t*>(take(static_cast<size_t>(w.cap) * 32));
  w.merges = reinterpret_cast<int32_t*>(take(static_cast<size_t>(w.cap_parts) * 16));
  const int64_t marks = batch > w.cap_parts ? batch : w.cap_parts;  // (a small call has at most cap_parts pieces)
  w.bad = reinterpret_cast<int32_t*>(take(static_cast<size_t>(marks) * hkv * 4));
  const size_t part = static_cast<size_t>(w.cap_parts) * hkv * w.part_rows;
  w.part_lse = reinterpret_cast<float*>(take(part * 4));
  w.part_o = reinterpret_cast<float*>(take(part * d * 4));
  w.total = off + kWorkspaceSlack;
  return w;
}

struct TreeParams {
  const __nv_bfloat16 *k_pool, *v_pool, *q;
  __nv_bfloat16* o;
  int64_t num_slots, table_stride, table_rows, total_q;
  int32_t hq, hkv, group;
  float scale_log2;
  const int32_t *table, *rpi, *prefix_lens, *draft_lens, *qo_indptr;
  const uint32_t* mask;
  int32_t mask_words, batch, max_draft, max_prefix;
  TreeShape sh;
  TreeWorkspace ws;
  uint32_t* err;
};

// Request b's lengths and first row; false (reported once) if they, its table row or its rows of q are out of
// bounds: such a request writes nothing.
__device__ __forceinline__ bool tree_request(const TreeParams& p, int32_t b, int32_t& P, int32_t& T, bool report) {
  P = __ldg(p.prefix_lens + b);
  T = __ldg(p.draft_lens + b);
  const int64_t q0 = __ldg(p.qo_indptr + b);
  const int32_t row = __ldg(p.rpi + b);
  if (P < 0 || P > p.max_prefix || T < 0 || T > p.max_draft || static_cast<int64_t>(P) + T > p.table_stride ||
      q0 < 0 || q0 + T > p.total_q) {
    if (report) flag_error(p.err, RA_DEVERR_LENGTH);
    return false;
  }
  if (row < 0 || row >= p.table_rows) {
    if (report) flag_error(p.err, RA_DEVERR_TABLE);
    return false;
  }
  return T > 0;
}

// A small narrow call's split, by this warp: its entry b * q_tiles + i is query tile i of request b.
template <int N>
struct TreeSmall {
  SmallPlan<N> plan;
  PerRequest<N> P, T, row, q0, tokens;  // of the request; the tile's first query row and tokens

  __device__ __forceinline__ TreeSmall(const TreeParams& p, int32_t ctas, bool report) {
    PerRequest<N> keys;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int32_t entry = static_cast<int32_t>(threadIdx.x & 31) + 32 * i;
      const int32_t b = entry / p.sh.q_tiles, tile = entry - b * p.sh.q_tiles;
      if (b < p.batch) {
        if (!tree_request(p, b, P.v[i], T.v[i], report && tile == 0)) P.v[i] = T.v[i] = 0;
        row.v[i] = __ldg(p.rpi + b);
        q0.v[i] = __ldg(p.qo_indptr + b) + tile * p.sh.tokens_per_item;
        tokens.v[i] = min(max(T.v[i] - tile * p.sh.tokens_per_item, 0), p.sh.tokens_per_item);
      }
      keys.v[i] = tokens.v[i] > 0 ? P.v[i] + T.v[i] : 0;
    }
    plan.make(keys, p.sh.heads, ctas, kTreeSmallLeast);
  }
};

// The narrow path's attention kernel (tree_narrow.cu): behind the plan kernel (small = 0), or a small call's (1 or
// 2 query tiles per lane).
ra_status launch_tree_narrow(const TreeParams& p, int32_t head_dim, int small, const DeviceInfo& dev,
                             cudaStream_t stream);

}  // namespace ra
