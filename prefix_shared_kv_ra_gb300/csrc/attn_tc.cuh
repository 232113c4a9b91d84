// attn_tc.cuh -- persistent tcgen05 / TMEM attention kernel over the slot pool.
//
// One CTA per SM runs a stream of work items.  An item is 256 query rows of one kv head -- two
// 128-row tiles, each a GQA block of 128 / G tokens (or decode requests) x the G q heads of the kv
// head -- against a range of keys gathered from the pool through a req_to_token row.  Every
// gathered 128-key K/V tile feeds both query tiles, i.e. 256 rows of tensor-core work.  Four users:
//
//  * extend (kExtendPass): rows are suffix tokens of one request; row (token i, head g) sees
//    keys 0 .. P + i (cached prefix + causal suffix); the bf16 output is written directly.  Items
//    come from a (request, query tile) list sorted longest first, times the kv heads.
//  * cascade prefix pass (kPrefixPass): rows are the decode queries of the members of one
//    prefix group; all rows see the same range of the shared prefix, read once for the group;
//    (output, log2-sum-exp) partials are written for the decode combine pass.
//  * draft tree (kTreePass): rows are the drafted tokens of one request; all see the cached prefix,
//    and of the drafted tokens the ones their bit mask names; an item is a (request, query tile, key
//    split); an unsplit item writes bf16, a split one partials.
//  * extend with changed scores (kExtendModPass, kExtendCapPass): a row sees a range of keys with both ends its own
//    (a window, documents, a prefix seen by all), its scores have a bias by distance and may be capped.
//
// Warp roles (512 threads):
//  warps 0-3  softmax + epilogue of query tile 0, one thread per row = TMEM lane;
//  warps 4-7  the same for query tile 1;
//  warps 8-11 gather the K rows of each 128-key tile with TMA tile::gather4 (4 rows per
//             instruction) into the 128B-swizzled K-major layout tcgen05 reads; warp 8 also
//             claims the items and publishes them through a shared ring (one mbarrier each);
//  warps 12-14 gather the V rows into the MN-major layout;
//  warp 15    one thread issues tcgen05.mma in the order S0 = Q0 K^T, S1 = Q1 K^T, then per key
//             tile O0 += P0 V, S0' = Q0 K'^T, O1 += P1 V, S1' = Q1 K'^T, so the tensor core
//             works on one query tile while the other tile's softmax runs (ping-pong); the warp
//             also loads the next item's query tiles (a 3-D TMA tile load, or a gather4 of the
//             members' rows) as soon as the current item's last QK on that tile has completed.
// The K and V gathers, and so the tensor core, run on from one item into the next; the epilogue
// of an item (O / l from TMEM) overlaps the next item's first QKs, and its first PV waits on an
// "O free" barrier the epilogue releases.  TMEM columns: S0 [0,128), S1 [128,256), O0 [256,384),
// O1 [384,512); P_i is stored by the softmax warps over the first 64 columns of S_i (bf16 pairs)
// and read from there by the TS-form MMA.
//
// Online softmax in the log2 domain with a lazy rescale: a row's reference maximum moves only
// when the running maximum exceeds it by more than 8 (a factor 256), and only then is the row's
// O accumulator rescaled in TMEM.  Tiles after an item's first are exponentiated in one pass
// against the current reference and accepted when the row sum stays <= 2^15; otherwise the
// warp redoes the tile on the exact path (row maximum first).  O / l is exact softmax.
//
// Every mbarrier wait is bounded; on a timeout the CTA flags RA_DEVERR_TIMEOUT, every role
// drains and leaves (the producers at once through the CTA's abort flag, the MMA and softmax warps at
// the deadline of their next wait), and TMEM is freed.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "ra_ptx.cuh"
#include "score_mod.cuh"

namespace ra {

struct TcParams {
  const __nv_bfloat16* k_pool;
  const __nv_bfloat16* v_pool;
  int64_t num_slots;
  int32_t hkv;
  const __nv_bfloat16* q;
  int32_t hq;
  int32_t group;
  float scale_log2;
  const int32_t* table;
  int64_t table_stride;
  int64_t table_rows;
  uint32_t* err;
  int32_t* work_counter;  // item claim counter, zero before the launch
  int32_t* done_counter;  // cascade prefix pass: each CTA adds one once all its partials are written
  // extend
  const int32_t* rpi;
  const int32_t* prefix_lens;
  const int32_t* extend_lens;
  const int32_t* qo_indptr;
  int32_t max_extend_len;
  int32_t max_prefix_len;
  int64_t total_q;  // rows of q and o: every written row index is checked against it
  __nv_bfloat16* o;
  const int32_t* work_count;  // number of (request, query tile) entries in work_items
  const int32_t* work_items;  // [2 * entries]: request, query tile; longest key range first
  // cascade prefix pass
  const int32_t* group_indptr;
  const int32_t* group_reqs;
  const int32_t* group_prefix_start;  // nullable: 0
  const int32_t* group_prefix_len;    // end of the group's range
  const int32_t* group_level;         // nullable: 0
  int32_t casc_levels;                // levels of prefix partials per member
  int32_t casc_slots;                 // casc_levels x max_csplits
  int32_t num_groups;
  int32_t grid_x;  // member tiles x prefix splits per group
  int32_t batch;   // decode batch (bound for group_reqs entries)
  int32_t max_seq_len;
  int32_t cchunk;
  int32_t max_csplits;
  float* casc_o;    // [casc_slots, batch, hq, D]
  float* casc_lse;  // [casc_slots, batch, hq]
  // draft tree (rpi, prefix_lens, qo_indptr, o and the work list as for extend; extend_lens are the draft
  // lengths; work_items are [8 * entries]: request, query tile, key split, partial slot or -1; prefix length,
  // drafted tokens, table row, first query row)
  const uint32_t* tree_mask;  // [total_q, mask_words]
  int32_t mask_words;
  const int32_t* tree_chunk;  // keys per split (a multiple of 128)
  const int32_t* tree_odd;    // [batch, hkv]: a drafted token's V holds a value that is not finite
  int32_t part_rows;          // rows of a partial slot
  float* part_o;              // [slots, hkv, part_rows, D]
  float* part_lse;            // [slots, hkv, part_rows]
  // extend with changed scores (the extend arrays; work_items are [4 * entries]: request, query tile, first key of the
  // tile's rows, end of their keys; part_* as for the tree, for the pieces of split key ranges)
  const int32_t* work_slots;  // [entries]: partial slot, or -1
  ScoreMod mod;
};

// kTreeDualPass: the tree pass for calls whose items all have one live query tile.
// kExtendModPass, kExtendCapPass: extend with changed scores, without and with a cap; kExtendFixedPass: with a cap of at
// most kCapFixed log2 units, under which no reference is needed.
enum TcPass {
  kPrefixPass = 0,
  kExtendPass = 1,
  kTreePass = 2,
  kTreeDualPass = 3,
  kExtendModPass = 4,
  kExtendCapPass = 5,
  kExtendFixedPass = 6
};

namespace tc {

constexpr int kRows = 128;     // query rows per tile (MMA M)
constexpr int kTiles = 2;      // query tiles per item
constexpr int kKeys = 128;     // keys per tile (MMA N of S, K of PV)
constexpr int kKWarps = 4;                 // TMA gather throughput grows with the number of issuing warps;
constexpr int kVWarps = 3;                 // the tensor core waits on K first, so K gets one warp more
constexpr int kGroups = kKeys / 4;          // 4-key gather groups per tile
constexpr int kItemRing = 8;                // published items (the claimer runs <= KS + 2 items ahead)
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// Changed scores: a row whose sum is outside these has its reference too far from its scores (weights that vanish or
// overflow); the sum at which a row's reference is raised, and by how much a score has to exceed it then; the cap (in
// log2 units) up to which none is needed: weights of 2^-80 .. 2^80 are as exact as others in bf16 and fp32, and the sum
// of 2^24 of them stays below 2^104.
constexpr float kSumFloor = 0x1p-90f, kSumCeiling = 0x1p110f;
constexpr float kRaiseSum = 0x1p60f, kRaiseStep = 8.f;
constexpr float kFastSumLimit = 32768.0f;  // single-pass acceptance: every p of the row <= 2^15
// Warps of a pass, and the register split: the softmax warpgroups hold a 128-key P row and two 32-column S chunks; the gather
// and MMA warpgroups (the last two) need few.  setmaxnreg moves registers between them within the block's launch allocation
// (kThreads x kLaunchRegs), which the split must add up to exactly.  Four softmax warpgroups where the two halves of a
// row need not agree on anything until its end: two per query tile leave a scheduler two warps to hide each other's
// latencies, four fill it better.
template <int PASS>
struct Roles {
  static constexpr bool kWide = PASS == kExtendFixedPass;
  static constexpr int kSoftWarps = kWide ? 16 : 8;
  static constexpr int kTileThreads = 32 * kSoftWarps / kTiles;  // softmax threads of a query tile
  static constexpr int kKWarp0 = kSoftWarps;                 // K gather warps 8..11
  static constexpr int kVWarp0 = kKWarp0 + kKWarps;          // V gather warps 12..14
  static constexpr int kMmaWarp = kVWarp0 + kVWarps;         // warp 15
  static constexpr int kThreads = 32 * (kMmaWarp + 1);       // 512
  static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;  // what __launch_bounds__(kThreads, 1) compiles to
  static constexpr int kSoftmaxRegs = kWide ? 96 : 184;
  static constexpr int kOtherRegs = kWide ? 48 : 72;
  static_assert(32 * kSoftWarps * kSoftmaxRegs + 256 * kOtherRegs == kThreads * kLaunchRegs, "register split");
};

template <int D, int KS, int VS>
struct Layout {
  static constexpr int kTileBytes = kKeys * D * 2;  // one K or V tile (also one query tile: 128 rows)
  static constexpr int kQ = 0;
  static constexpr int kK = kTiles * kTileBytes;
  static constexpr int kV = kK + KS * kTileBytes;
  static constexpr int kBytes = kV + VS * kTileBytes;
  static constexpr int kDynSmem = kBytes + 1024;  // + alignment slack
};

__device__ __forceinline__ bool aborted(volatile int* flag) { return *flag != 0; }

template <bool B>
struct BoolTag {
  static constexpr bool value = B;
};

// One work item: key range, table row and query rows.
struct Job {
  int32_t kh;
  int32_t kbeg, kend, nt;  // keys [kbeg, kend) in nt 128-key tiles
  int32_t table_row;
  int32_t n_valid;   // valid tokens / members (of 2T)
  int32_t causal0;   // extend: token t of the item sees keys < causal0 + t + 1; tree: the prefix length
  int64_t q_tok0;    // extend: first q token
  int32_t mem0;      // cascade: first member index into group_reqs; tree: the request's drafted tokens; changed
                     // scores: end of the keys that every row sees
  int32_t csplit;    // cascade: prefix split
  int32_t slot;      // cascade: partial slot of the members (level x max_csplits + split); tree: partial
                     // slot of the item, -1 for an unsplit one
  int32_t dual;      // tree (dual pass): the item's one live query tile is in both tiles, which share out its key tiles
  int32_t kt0;       // tree: key tiles of the CTA's items before this one
  int32_t odd;       // tree: drafted tokens' V of this kv head hold values that are not finite
  int32_t tiles;     // query tiles holding valid rows (1: tile 1 is empty; its MMAs and softmax are skipped,
                     // while every barrier still completes its phases as for two tiles)
};

// Item -> job; false for an empty or invalid item (reported once, when `report`).
template <int PASS>
__device__ __forceinline__ bool tc_job(const TcParams& p, int32_t item, Job& j, bool report) {
  const int T = kRows / p.group;
  j.kh = item % p.hkv;
  const int32_t rest = item / p.hkv;
  j.causal0 = 0;
  j.q_tok0 = 0;
  j.mem0 = 0;
  j.csplit = 0;
  j.slot = 0;
  j.odd = 0;
  j.kt0 = 0;
  if constexpr (PASS == kTreePass || PASS == kTreeDualPass) {
    // the list holds only non-empty items of requests whose indices and lengths were checked when it was built
    const int4 e = __ldg(reinterpret_cast<const int4*>(p.work_items) + 2 * rest);
    const int4 f = __ldg(reinterpret_cast<const int4*>(p.work_items) + 2 * rest + 1);
    const int32_t chunk = __ldg(p.tree_chunk);
    j.table_row = f.z;
    j.n_valid = min(kTiles * T, f.y - e.y * kTiles * T);
    j.causal0 = f.x;
    j.mem0 = f.y;
    j.kbeg = e.z * chunk;
    j.kend = min(f.x + f.y, j.kbeg + chunk);
    j.q_tok0 = f.w + e.y * kTiles * T;
    j.slot = e.w;
    j.odd = __ldg(p.tree_odd + static_cast<int64_t>(e.x) * p.hkv + j.kh);
  } else if constexpr (PASS == kExtendModPass || PASS == kExtendCapPass || PASS == kExtendFixedPass) {
    // (as below; the list's builder found the tile's key range)
    const int4 e = __ldg(reinterpret_cast<const int4*>(p.work_items) + rest);
    const int32_t E = min(max(__ldg(p.extend_lens + e.x), 0), p.max_extend_len);
    const int32_t P = __ldg(p.prefix_lens + e.x);
    j.table_row = __ldg(p.rpi + e.x);
    if (j.table_row < 0 || j.table_row >= p.table_rows) {
      if (report && e.y == 0 && j.kh == 0) flag_error(p.err, RA_DEVERR_TABLE);
      return false;
    }
    const int64_t q_first = __ldg(p.qo_indptr + e.x);
    if (q_first < 0 || q_first + E > p.total_q) {
      if (report && e.y == 0 && j.kh == 0) flag_error(p.err, RA_DEVERR_LENGTH);
      return false;
    }
    j.n_valid = min(kTiles * T, E - e.y * kTiles * T);
    j.causal0 = P + e.y * kTiles * T;
    j.kbeg = e.z;
    j.kend = e.w;
    j.slot = __ldg(p.work_slots + rest);
    j.mem0 = p.mod.full_lens ? min(__ldg(p.mod.full_lens + e.x), P + E) : 0;
    j.q_tok0 = q_first + e.y * kTiles * T;
  } else if constexpr (PASS == kExtendPass) {
    // entry `rest` of the work list: it holds only non-empty query tiles of requests whose lengths
    // were checked (and flagged) when it was built
    const int b = __ldg(p.work_items + 2 * rest);
    const int tile = __ldg(p.work_items + 2 * rest + 1);
    const int32_t E = min(max(__ldg(p.extend_lens + b), 0), p.max_extend_len);
    const int32_t P = __ldg(p.prefix_lens + b);
    j.table_row = __ldg(p.rpi + b);
    if (j.table_row < 0 || j.table_row >= p.table_rows) {
      if (report && tile == 0 && j.kh == 0) flag_error(p.err, RA_DEVERR_TABLE);
      return false;
    }
    // the request's rows qo_indptr[b] .. qo_indptr[b] + E - 1 must lie inside o: a request whose
    // lengths disagree with total_q writes nothing (flagged once)
    const int64_t q_first = __ldg(p.qo_indptr + b);
    if (q_first < 0 || q_first + E > p.total_q) {
      if (report && tile == 0 && j.kh == 0) flag_error(p.err, RA_DEVERR_LENGTH);
      return false;
    }
    j.n_valid = min(kTiles * T, E - tile * kTiles * T);
    j.causal0 = P + tile * kTiles * T;
    j.kbeg = 0;
    j.kend = j.causal0 + j.n_valid;
    j.q_tok0 = q_first + tile * kTiles * T;
  } else {
    const int x = rest % p.grid_x;
    const int g = rest / p.grid_x;
    const int32_t m_begin = __ldg(p.group_indptr + g);
    const int32_t n_mem = __ldg(p.group_indptr + g + 1) - m_begin;
    const int mt = x / p.max_csplits;
    j.csplit = x - mt * p.max_csplits;
    if (mt * kTiles * T >= n_mem) return false;
    // the group's range [g0, Pg) of its members' positions, split into cchunk-key pieces
    const int32_t Pg = __ldg(p.group_prefix_len + g);
    const int32_t g0 = p.group_prefix_start ? __ldg(p.group_prefix_start + g) : 0;
    const int32_t lvl = p.group_level ? __ldg(p.group_level + g) : 0;
    if (Pg < 1 || Pg > p.max_seq_len || g0 < 0 || g0 >= Pg || lvl < 0 || lvl >= p.casc_levels) {
      if (report && x == 0 && j.kh == 0) flag_error(p.err, RA_DEVERR_LENGTH);
      return false;
    }
    if (j.csplit * p.cchunk >= Pg - g0) return false;
    j.kbeg = g0 + j.csplit * p.cchunk;
    j.kend = min(Pg, j.kbeg + p.cchunk);
    j.slot = lvl * p.max_csplits + j.csplit;
    j.mem0 = m_begin + mt * kTiles * T;
    j.n_valid = min(kTiles * T, n_mem - mt * kTiles * T);
    const int32_t leader = __ldg(p.group_reqs + m_begin);
    if (leader < 0 || leader >= p.batch) {
      if (report && x == 0 && j.kh == 0) flag_error(p.err, RA_DEVERR_TABLE);
      return false;
    }
    j.table_row = __ldg(p.rpi + leader);
    if (j.table_row < 0 || j.table_row >= p.table_rows) {
      if (report && x == 0 && j.kh == 0) flag_error(p.err, RA_DEVERR_TABLE);
      return false;
    }
  }
  j.nt = (j.kend - j.kbeg + kKeys - 1) / kKeys;
  j.tiles = j.n_valid > T ? 2 : 1;
  j.dual = PASS == kTreeDualPass && j.tiles == 1 && j.nt > 1;
  return j.nt > 0;
}

// The largest bias of the keys [first, end) for a row at `pos`: the nearest one's, or (negative slopes) the farthest's.
__device__ __forceinline__ float bias_bound(int32_t first, int32_t end, int32_t pos, float slope) {
  const int32_t near = pos < first ? first - pos : pos >= end ? pos - end + 1 : 0;
  const int32_t far = max(abs(pos - first), abs(pos - end + 1));
  return -slope * static_cast<float>(slope >= 0.f ? near : far);
}

// The offset of the K and V rows of a key of the item.
template <int D>
__device__ __forceinline__ int64_t key_row(const TcParams& p, const Job& jb, int32_t key) {
  int32_t slot = __ldg(p.table + static_cast<int64_t>(jb.table_row) * p.table_stride + key);
  if (slot < 0 || slot >= p.num_slots) slot = 0;
  return (static_cast<int64_t>(slot) * p.hkv + jb.kh) * D;
}

// Whether V of a key in [from, to) of the item holds a value that is not finite (by a warp, a key per lane).
template <int D>
__device__ __forceinline__ bool odd_values(const TcParams& p, const Job& jb, int32_t from, int32_t to) {
  uint32_t top = 0;
#pragma unroll 1
  for (int32_t k0 = from; k0 < to; k0 += 32) {
    const uint4* v = reinterpret_cast<const uint4*>(
        p.v_pool + key_row<D>(p, jb, min(k0 + static_cast<int32_t>(threadIdx.x & 31), to - 1)));
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
      const uint4 x = __ldg(v + i);
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                   __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
    }
  }
  return __any_sync(0xffffffffu, (top & 0xffffu) >= 0x7f80u || (top >> 16) >= 0x7f80u);
}

// A row with changed scores whose tensor-core result cannot stand, or may not: `far` says that its sum left the range of its
// reference; otherwise its output is not finite.  That is right if only values that it sees are not finite; a value that
// it does not see gets there as well (a zero weight times it is a NaN in the product over a whole tile), and an
// overflow.  True if the row was computed again, by the warp: a key per lane for the scores, D / 32 dimensions per lane
// (l * D / 32 ..) for the values, its log2-sum-exp in lse.  Rare, and slow.
template <int D, bool CAP>
__device__ __forceinline__ bool mod_row(const TcParams& p, const Job& jb, bool far, int64_t q_row, int32_t first, int32_t end,
                                        int32_t pos, float slope, float (&acc)[D / 32], float& lse) {
  constexpr int V = D / 32;
  if (!far && !odd_values<D>(p, jb, jb.kbeg, min(first, jb.kend)) && !odd_values<D>(p, jb, max(end, jb.kbeg), jb.kend) &&
      odd_values<D>(p, jb, first, end))
    return false;
  const int lane = threadIdx.x & 31;
  const uint4* q = reinterpret_cast<const uint4*>(p.q + q_row * D);
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll 1
  for (int32_t k0 = first; k0 < end; k0 += 32) {
    const int32_t key = min(k0 + lane, end - 1);
    const int64_t row = key_row<D>(p, jb, key);
    const uint4* k = reinterpret_cast<const uint4*>(p.k_pool + row);
    float s = 0.f;
#pragma unroll 4
    for (int d = 0; d < D / 8; ++d) {
      const uint4 a = __ldg(q + d), b = __ldg(k + d);
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s = fmaf(__uint_as_float(aw[i] << 16), __uint_as_float(bw[i] << 16), s);
        s = fmaf(__uint_as_float(aw[i] & 0xffff0000u), __uint_as_float(bw[i] & 0xffff0000u), s);
      }
    }
    float x = CAP ? p.mod.cap_log2 * tanh_any(s * p.mod.cap_in) : s * p.scale_log2;
    x = k0 + lane < end ? fmaf(-slope, fabsf(static_cast<float>(pos - key)), x) : -INFINITY;
    float top = x;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float m_new = fmaxf(m, top), m_sub = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = ex2(m - m_sub), w = ex2(x - m_sub);
    m = m_new;
    l = l * alpha + w;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= alpha;
    // (lanes past the end hold the last key again, with weight 0)
#pragma unroll 8
    for (int i = 0; i < 32; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const __nv_bfloat16* vr = p.v_pool + __shfl_sync(0xffffffffu, row, i) + lane * V;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(wi, __bfloat162float(vr[v]), acc[v]);
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] *= inv;
  lse = l == 0.f ? -INFINITY : m + __log2f(l);
  return true;
}

}  // namespace tc

template <int D, int KS, int VS, int PASS>
__global__ void __launch_bounds__(tc::Roles<PASS>::kThreads, 1)
    attn_tc_kernel(const __grid_constant__ TcParams p, const __grid_constant__ CUtensorMap qmap,
                   const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using namespace tc;
  using L = Layout<D, KS, VS>;
  using R = Roles<PASS>;
  constexpr int kKWarp0 = R::kKWarp0, kVWarp0 = R::kVWarp0, kMmaWarp = R::kMmaWarp;
  constexpr int kSoftmaxRegs = R::kSoftmaxRegs, kOtherRegs = R::kOtherRegs;
  constexpr bool EXTEND = PASS != kPrefixPass;  // rows are tokens of one request, items come from a list
  constexpr bool DUAL = PASS == kTreeDualPass;
  constexpr bool TREE = PASS == kTreePass || DUAL;
  constexpr bool FIXED = PASS == kExtendFixedPass;  // the softmax below FIXED's is not this pass's
  constexpr bool CAP = PASS == kExtendCapPass;
  constexpr bool MOD = PASS == kExtendModPass || CAP;
  constexpr int HALVES = D / 64;  // 128-byte (64-element) column blocks of a row
  // K/V stage release: one barrier per key tile t (ring of KVF), committed after the last MMA reading
  // K_t and V_t (PV of query tile 1).  KVF > max(KS, VS): a producer waiting for tile t's release
  // cannot see the ring slot complete tile t + KVF first (that tile needs its own next copy).
  constexpr int KVF = (KS > VS ? KS : VS) + 1;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_q[kTiles], bar_kf[KS], bar_vf[VS], bar_kvfree[KVF], bar_s[kTiles],
      bar_p[kTiles], bar_o[kTiles], bar_ofree[kTiles], bar_item[kItemRing], bar_done;
  __shared__ int32_t s_item[kItemRing];
  __shared__ Job s_job[kItemRing];  // decoded by the claimer: no role reads the work list itself
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ __align__(8) uint64_t bar_join[2];  // tree, dual items: tile 1's sums are in s_join; its O has been read
                                                 // (fixed reference: the sums of tile i's rows are in TMEM)
  __shared__ float2 s_join[DUAL ? kRows : 1];    // (reference, sum) of tile 1's rows

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = p.group;
  const int T = kRows / G;  // tokens (or members) per query tile

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto sQ = [&](int i) { return sbase + L::kQ + i * L::kTileBytes; };
  auto sK = [&](int st) { return sbase + L::kK + st * L::kTileBytes; };
  auto sV = [&](int st) { return sbase + L::kV + st * L::kTileBytes; };

  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < KS; ++s) mbar_init(smem_u32(&bar_kf[s]), kKWarps);
    for (int s = 0; s < VS; ++s) mbar_init(smem_u32(&bar_vf[s]), kVWarps);
    for (int s = 0; s < KVF; ++s) mbar_init(smem_u32(&bar_kvfree[s]), 1);
    for (int i = 0; i < kTiles; ++i) {
      mbar_init(smem_u32(&bar_q[i]), EXTEND ? 1 : kKWarps / kTiles);
      mbar_init(smem_u32(&bar_s[i]), 1);
      mbar_init(smem_u32(&bar_p[i]), R::kTileThreads);
      mbar_init(smem_u32(&bar_o[i]), 1);
      mbar_init(smem_u32(&bar_ofree[i]), R::kTileThreads);
    }
    for (int s = 0; s < kItemRing; ++s) mbar_init(smem_u32(&bar_item[s]), 1);
    mbar_init(smem_u32(&bar_done), 1);
    mbar_init(smem_u32(&bar_join[0]), R::kTileThreads);
    mbar_init(smem_u32(&bar_join[1]), R::kTileThreads);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&s_tmem), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();  // the previous kernel (the work-list pass / the key-start scatter) has completed; the set-up
  griddep_launch();  // above overlaps it
  const uint32_t tmem = s_tmem;
  volatile int* abort_flag = &s_abort;
  auto give_up = [&]() {
    *abort_flag = 1;
    flag_error(p.err, RA_DEVERR_TIMEOUT);
  };
  // item n of this CTA: 1 = `jb` holds its job, 0 = no more work, -1 = a bounded wait ran out
  auto wait_item = [&](int32_t n, Job& jb) -> int {
    if (!mbar_wait(smem_u32(&bar_item[n % kItemRing]), (n / kItemRing) & 1)) return -1;
    if (s_item[n % kItemRing] < 0) return 0;
    jb = s_job[n % kItemRing];
    return 1;
  };

  // Steps of an item (a QK and a PV on each query tile), the key tile of query tile i's step j counted from the
  // item's first, and whether there is work in it.  Both tiles of an item work on the same key tile; of a dual
  // item, whose rows fill one query tile only, tile i takes every other one: with one tile's chain of QK, softmax
  // and PV at a time the tensor core would wait for most of it (64 requests x 8..16 drafted tokens over 512..4096
  // keys, 64/8 heads: 148 us so, 134 with dual items).  A variant of its own: in the pass for 256-row items these
  // lines cost 3%.
  auto steps_of = [](const Job& b) -> int32_t { return DUAL && b.dual ? (b.nt + 1) >> 1 : b.nt; };
  auto tile_at = [](const Job& b, int32_t j, int i) -> int32_t { return DUAL && b.dual ? 2 * j + i : j; };
  auto live_at = [](const Job& b, int32_t j, int i) -> bool {
    return DUAL && b.dual ? 2 * j + i < b.nt : i == 0 || b.tiles > 1;
  };

  if (warp >= kKWarp0 && warp < kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // ================================================================ producers (TMA)
    const bool is_v = warp >= kVWarp0;
    const int nw = is_v ? kVWarps : kKWarps;
    const int pw = warp - (is_v ? kVWarp0 : kKWarp0);  // 0 .. nw-1
    const bool claimer = !is_v && pw == 0;
    const CUtensorMap* map = is_v ? &vmap : &kmap;
    if (lane == 0) prefetch_tensormap(map);
    // the claimer hands out items in order (the extend list is longest first), skipping empty ones
    int32_t n_items = 0;
    if (claimer) {
      n_items = EXTEND ? __ldg(p.work_count) * p.hkv : p.num_groups * p.grid_x * p.hkv;
    }
    // claim the next non-empty item and publish it, decoded, as entry n of the ring (warp-collective).
    // Item blockIdx.x is this CTA's first without a claim; the counter hands out the items after the grid.
    bool own_first = true;
    int32_t claimed_tiles = 0;
    (void)claimed_tiles;
    auto claim_publish = [&](int32_t n) {
      int32_t idx;
      Job cj;
      for (;;) {
        idx = static_cast<int32_t>(blockIdx.x);
        if (!own_first) {
          if (lane == 0) idx = static_cast<int32_t>(gridDim.x) + atomicAdd(p.work_counter, 1);
          idx = __shfl_sync(0xffffffffu, idx, 0);
        }
        own_first = false;
        if (idx >= n_items) {
          idx = -1;
          break;
        }
        if (tc_job<PASS>(p, idx, cj, lane == 0)) break;
      }
      if constexpr (TREE) {
        cj.kt0 = claimed_tiles;
        claimed_tiles += cj.nt;
      }
      if (lane == 0) {
        s_item[n % kItemRing] = idx;
        if (idx >= 0) s_job[n % kItemRing] = cj;
        mbar_arrive(smem_u32(&bar_item[n % kItemRing]));
      }
    };
    if (claimer) claim_publish(0);
    // warp pw of nw gathers 4-key groups g0 .. g1-1 of each 128-key tile (keys 4*g0 ..), lane i < g1-g0
    // issuing the gather4 of group g0+i.  Slot ids: lane l holds keys 4*g0 + l and 4*g0 + 32 + l of a
    // tile; the next tile's (possibly the next item's first) are loaded while this one is issued.
    const int g0 = pw * kGroups / nw, g1 = (pw + 1) * kGroups / nw;
    const int nkeys = 4 * (g1 - g0);  // <= 44
    uint64_t* full = is_v ? bar_vf : bar_kf;
    const int ns = is_v ? VS : KS;
    auto load_row = [&](const Job& jb, int j, int k) -> int32_t {  // tensor-map row (slot * Hkv + kh)
      if (k >= nkeys) return 0;
      const int32_t key = jb.kbeg + j * kKeys + 4 * g0 + k;  // keys past the range repeat the last key
      int32_t s = __ldg(p.table + static_cast<int64_t>(jb.table_row) * p.table_stride + min(key, jb.kend - 1));
      if (s < 0 || s >= p.num_slots) {
        flag_error(p.err, RA_DEVERR_SLOT);
        s = 0;
      }
      return s * p.hkv + jb.kh;
    };
    int32_t gt = 0;  // key tiles issued by this warp (all items)
    bool ok = true;
    int32_t n = 0;
    Job jb{};
    int r = wait_item(0, jb);
    if (!__all_sync(0xffffffffu, r >= 0)) ok = false;
    int32_t ca = ok && r > 0 ? load_row(jb, 0, lane) : 0, cb = ok && r > 0 ? load_row(jb, 0, lane + 32) : 0;
    while (ok && r > 0) {
      for (int j = 0; j < jb.nt; ++j) {
        if (aborted(abort_flag)) { ok = false; break; }
        // the next tile's slot ids: this item's, or the next item's first
        int32_t na = 0, nb = 0;
        if (j + 1 < jb.nt) {
          na = load_row(jb, j + 1, lane);
          nb = load_row(jb, j + 1, lane + 32);
        }
        const int st = gt % ns;
        // stage st held tile gt - ns: wait for that tile's release
        if (gt >= ns &&
            !__all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_kvfree[(gt - ns) % KVF]), ((gt - ns) / KVF) & 1))) {
          ok = false;
          break;
        }
        const uint32_t tile = is_v ? sV(st) : sK(st);
        int32_t rr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = lane * 4 + e;  // key of this lane's group (meaningful for lane < g1-g0)
          const int32_t va = __shfl_sync(0xffffffffu, ca, k & 31);
          const int32_t vb = __shfl_sync(0xffffffffu, cb, k & 31);
          rr[e] = k < 32 ? va : vb;
        }
        if (lane == 0) mbar_arrive_expect_tx(smem_u32(&full[st]), nkeys * D * 2);
        __syncwarp();
        if (lane < g1 - g0) {
          const int row = 4 * (g0 + lane);  // first tile row of this gather
#pragma unroll
          for (int h = 0; h < HALVES; ++h)
            tma_gather4(tile + h * (kRows * 128) + row * 128, map, h * 64, rr[0], rr[1], rr[2], rr[3],
                        smem_u32(&full[st]));
        }
        ++gt;
        if constexpr (!EXTEND) {
          // The members' query rows of this item: K warps 0-1 gather query tile 0, warps 2-3 tile 1, 16
          // groups of 4 rows each (one gather4 per 64-column half).  The tile is free once the previous
          // item's last QK on it has completed, which the commit of that S signals.
          if (!is_v && j == 0) {
            const int qt = pw / 2;
            if (n > 0 && !__all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_s[qt]), (gt - 2) & 1))) {
              ok = false;
              break;
            }
            const uint32_t bq = smem_u32(&bar_q[qt]);
            if (lane == 0) mbar_arrive_expect_tx(bq, 16 * 4 * D * 2);
            __syncwarp();
            if (lane < 16) {
              const int grp = (pw & 1) * 16 + lane;  // group of the tile
              int32_t qrow[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int R = grp * 4 + e;
                const int k = qt * T + R / G;
                int32_t b = __ldg(p.group_reqs + jb.mem0 + (k < jb.n_valid ? k : 0));
                b = (b < 0 || b >= p.batch) ? 0 : b;
                qrow[e] = b * p.hq + jb.kh * G + (R % G);
              }
#pragma unroll
              for (int h = 0; h < HALVES; ++h)
                tma_gather4(sQ(qt) + h * (kRows * 128) + grp * 4 * 128, &qmap, h * 64, qrow[0], qrow[1], qrow[2],
                            qrow[3], bq);
            }
          }
        }
        // the next item is claimed once this one's first tile is on its way
        if (claimer && j == 0) claim_publish(n + 1);
        ca = na;
        cb = nb;
      }
      if (!ok) break;
      ++n;
      r = wait_item(n, jb);
      if (!__all_sync(0xffffffffu, r >= 0)) { ok = false; break; }
      if (r > 0) {
        ca = load_row(jb, 0, lane);
        cb = load_row(jb, 0, lane + 32);
      }
    }
    if (!ok) {
      give_up();
      // copies this warp issued land before the CTA can leave
      for (int32_t t = (gt > ns ? gt - ns : 0); t < gt; ++t) mbar_wait(smem_u32(&full[t % ns]), (t / ns) & 1);
    }
  } else if (warp == kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // ================================================================ MMA issuer + query loads
    if (lane == 0) prefetch_tensormap(&qmap);
    constexpr uint32_t idesc_qk = idesc_bf16_f32(kRows, kKeys, 0, 0);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(kRows, D, 0, 1);
    // Every Q, K and V tile sits at a fixed shared-memory offset: one descriptor per operand kind, a
    // tile's and a K step's offsets added to its start-address field (addresses / 16 stay below 2^14).
    const uint64_t desc_q0 = sdesc_sw128(sQ(0), 16, 1024), desc_k0 = sdesc_sw128(sK(0), 16, 1024);
    const uint64_t desc_v0 = sdesc_sw128(sV(0), kRows * 128, 1024);
    constexpr uint32_t kTile16 = L::kTileBytes >> 4;
    // query tile i of an extend job into sQ(i): one 3-D TMA tile load per 64-column half (the K warps
    // gather the prefix pass's member rows)
    auto load_q = [&](const Job& jb, int i) {
      const uint32_t bq = smem_u32(&bar_q[i]);
      if constexpr (EXTEND) {
        if (lane == 0) mbar_arrive_expect_tx(bq, kRows * D * 2);
        __syncwarp();
        if (lane == 0) {
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            asm volatile(
                "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(sQ(i) + h * (kRows * 128)),
                "l"(&qmap), "r"(h * 64), "r"(jb.kh * G),
                "r"(static_cast<int32_t>(jb.q_tok0 + (DUAL && jb.dual ? 0 : i * T))), "r"(bq)
                : "memory");
          }
        }
      }
    };
    // every lane waits (the warp is otherwise idle but for lane 0); the outcome is made warp-uniform.
    // (Parking lanes 1-31 in a shuffle while lane 0 waits measured ~20% slower on GB300.)
    auto wait_all = [&](uint64_t& bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), parity));
    };
    bool ok = true;
    int32_t n = 0, g = 0;  // items done, steps done (all items)
    int32_t kt0 = 0;       // key tiles of the items done
    Job jb{}, jn{};
    int r = wait_item(0, jb);
    if (!__all_sync(0xffffffffu, r >= 0)) ok = false;
    int next = -2;  // the item after jb: -2 not looked up yet, 0 none, 1 in jn
    auto lookup_next = [&]() -> bool {  // published when jb's first K tile was issued
      if (next != -2) return true;
      const int rn = wait_item(n + 1, jn);
      if (!__all_sync(0xffffffffu, rn >= 0)) return false;
      next = rn;
      return true;
    };
    if (ok && r > 0 && EXTEND) {
      load_q(jb, 0);
      load_q(jb, 1);
    }
    // S_i = Q_i K_kt^T; for an empty query tile (live false) only the commit, which keeps bar_s's phases.  The
    // tiles share a key tile (tile 0 waits for it) unless the item is dual.
    auto qk = [&](int i, int kt, bool live, bool dual) -> bool {
      const int st = kt % KS;
      if (i == 0 || (DUAL && dual && live)) {
        if (!wait_all(bar_kf[st], (kt / KS) & 1)) return false;
        tc_fence_after();
      }
      if (lane == 0) {
        const uint64_t qd = desc_q0 + i * kTile16, kd = desc_k0 + st * kTile16;
#pragma unroll
        for (int kk = 0; kk < D / 16 && live; ++kk) {
          const uint32_t off16 = ((kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4;
          tc_mma_ss(tmem + i * kKeys, qd + off16, kd + off16, idesc_qk, kk > 0);
        }
        tc_commit(smem_u32(&bar_s[i]));
      }
      __syncwarp();
      return true;
    };
    // O_i += P_i V of the tile's step j (step gg of all items).  After the last P of the item, query tile i is
    // free (the softmax saw S_i, so its QK has completed): the next item's tile is loaded then.
    auto pv = [&](int i, int gg, int j) -> bool {
      const int kt = kt0 + tile_at(jb, j, i);
      const int st = kt % VS;
      const bool live = live_at(jb, j, i);  // an empty query tile issues no PV (its O is never read)
      if (!wait_all(bar_p[i], gg & 1)) return false;
      tc_fence_after();
      if (j == 0 && n > 0) {
        // the previous item's epilogue has read O_i
        if (!wait_all(bar_ofree[i], (n - 1) & 1)) return false;
        tc_fence_after();
      }
      if (i == 0 || (DUAL && jb.dual && live)) {
        if (!wait_all(bar_vf[st], (kt / VS) & 1)) return false;
        tc_fence_after();
      }
      if (lane == 0) {
        const uint64_t vd = desc_v0 + st * kTile16;
#pragma unroll
        for (int kk = 0; kk < kKeys / 16 && live; ++kk) {
          // (fixed reference: each half's P is over its own half of S)
          tc_mma_ts(tmem + kColO + i * 128, tmem + i * kKeys + (FIXED ? (kk >> 2) * 64 + (kk & 3) * 8 : kk * 8), vd + kk * (2048 >> 4), idesc_pv,
                    (j > 0 || kk > 0) ? 1u : 0u);
        }
        // Each commit stalls the tensor pipe briefly, so there are three per key tile: S_0, S_1 and the
        // K/V release here.  O_i needs none until the item's last tile: S_i's commit also covers PV_i.
        if (DUAL && jb.dual ? live : i == kTiles - 1) tc_commit(smem_u32(&bar_kvfree[kt % KVF]));
        if (j == steps_of(jb) - 1) tc_commit(smem_u32(&bar_o[i]));
      }
      __syncwarp();
      return true;
    };
    // Query tile i of this item is free once its last QK (key tile gl) has completed: the commit of
    // S_i signals that (the softmax warps wait on the same phase).  The next item's tile is loaded then,
    // a whole softmax ahead of the QK that needs it.
    auto reload_q = [&](int i, int gl) -> bool {
      if (!lookup_next()) return false;
      if constexpr (EXTEND) {
        if (!wait_all(bar_s[i], gl & 1)) return false;
        if (next > 0) load_q(jn, i);
      }
      return true;
    };
    // The key tiles of consecutive items form one stream: per tile PV_0, QK_0', PV_1, QK_1', where the
    // QKs after an item's last tile are the next item's first.
    if (ok && r > 0) {
      ok = wait_all(bar_q[0], 0) && wait_all(bar_q[1], 0);
      if (ok) {
        tc_fence_after();
        ok = qk(0, 0, true, jb.dual) && qk(1, tile_at(jb, 0, 1), live_at(jb, 0, 1), jb.dual);
      }
    }
    while (ok && r > 0) {
      // (no per-tile look at the abort flag: after a failure elsewhere this warp leaves through the
      // deadline of its next wait; the check on the loop's back edge measured ~1% of the kernel)
      for (int j = 0; ok && j < steps_of(jb); ++j) {
        const int gg = g + j;
        const bool last = j + 1 == steps_of(jb);
        // The QK on tile i after this key tile's PV: this item's next key tile, or after its last the next
        // item's first, once that item's query tile has landed.  One call site per query tile: the loop
        // body exists once (a copy for an item's last tile measured 6-8% slower: the MMA warp's code
        // shares an instruction cache with the softmax warps of its sub-partition).
        auto qk_after = [&](int i) -> bool {
          bool live = live_at(jb, j + 1, i), dual = DUAL && jb.dual;
          int kt = kt0 + tile_at(jb, j + 1, i);
          if (last) {
            if (next == 0) return true;
            if (!wait_all(bar_q[i], (n + 1) & 1)) return false;
            tc_fence_after();
            live = live_at(jn, 0, i);
            dual = DUAL && jn.dual;
            kt = kt0 + jb.nt + tile_at(jn, 0, i);
          }
          return qk(i, kt, live, dual);
        };
        ok = (!last || reload_q(0, gg)) && pv(0, gg, j) && (!last || reload_q(1, gg)) && qk_after(0) &&
             pv(1, gg, j) && qk_after(1);
      }
      if (!ok) break;
      g += steps_of(jb);
      kt0 += jb.nt;
      ++n;
      r = next;
      jb = jn;
      next = -2;
    }
    if (!ok) give_up();
    if (lane == 0) tc_commit(smem_u32(&bar_done));  // all MMAs of this CTA retired before TMEM is freed
    __syncwarp();
    mbar_wait(smem_u32(&bar_done), 0);
  } else if constexpr (FIXED) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ================================================================ softmax under a fixed reference (warps 0-15)
    // Capped scores are bounded, and so are their weights: t = cap log2(e) tanh(y) - slope |pos - key| - reference, where
    // the reference is only the largest bias of the row's keys.  Nothing is looked up, moved or rescaled, so each half of a
    // row's keys has a thread of its own (warpgroups 2 i and 2 i + 1 of query tile i); they add up their sums at the end.
    // P goes over the first half of the S columns it came from, 32 keys at a time.  Here tanh(y) is 1 - 2 / (e^2y + 1) for
    // every y: where y is small it is off by 2^-22, which a cap this small makes 2e-5 of a weight, and the special function
    // units have time for the two more calls that the fp32 pipe has not for the polynomial (642 -> 602 us for 8 prompts of
    // 700..1500 tokens, 64/8 heads).
    const int ti = warp >> 3, half = (warp >> 2) & 1;
    const int r = threadIdx.x & 127;  // row of the tile = TMEM lane
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t col = tmem + lane_addr + ti * kKeys + half * 64;
    const uint32_t col_o = tmem + lane_addr + kColO + ti * 128 + half * (D / 2);
    const int tok = ti * T + r / G;
    bool ok = true;
    int32_t g = 0;
    for (int32_t n = 0;; ++n) {
      Job jb;
      const int ri = wait_item(n, jb);
      if (__any_sync(0xffffffffu, ri < 0)) { ok = false; break; }
      if (ri == 0) break;
      const bool row_valid = tok < jb.n_valid;
      const int32_t pos = jb.causal0 + tok;
      int32_t lim = jb.kend, first = jb.kbeg;  // the keys this row sees: [first, lim)
      float slope = 0.f;
      if (row_valid) {
        lim = min(max(pos + 1, jb.mem0), jb.kend);
        if (p.mod.window > 0) first = max(first, pos - p.mod.window + 1);
        if (p.mod.first_key) first = max(first, __ldg(p.mod.first_key + jb.q_tok0 + tok));
        if (p.mod.slopes) slope = __ldg(p.mod.slopes + jb.kh * G + r % G) * kLog2e;
      }
      const float m = first < lim ? bias_bound(first, lim, pos, slope) : 0.f;
      float l = 0.f;
      for (int j = 0; j < jb.nt; ++j) {
        const bool fail_here = !mbar_wait(smem_u32(&bar_s[ti]), (g + j) & 1);
        if (__any_sync(0xffffffffu, fail_here)) { ok = false; break; }
        if (ti >= jb.tiles) {  // an empty query tile: no S was computed; keep bar_p's phase
          mbar_arrive(smem_u32(&bar_p[ti]));
          continue;
        }
        tc_fence_after();
        const int32_t key0 = jb.kbeg + j * kKeys + half * 64;
        const bool edge_here = key0 + 64 > min(lim, pos + 1) || key0 < first;  // hidden keys, or keys behind the row's own
        const bool sees = first < key0 + 64 && first < lim && key0 < lim;
        if (!__any_sync(0xffffffffu, sees)) {
          const uint32_t none[32] = {};
          tmem_st32(col, none);
        } else {
          const int32_t lo = first - key0, hi = lim - key0;  // this row's columns: [lo, hi)
          uint64_t sum2[2] = {0, 0};
          auto run = [&](auto edge_tag) {
            constexpr bool edge = decltype(edge_tag)::value;
            const uint64_t in2 = f2_pack(p.mod.exp2y.x, p.mod.exp2y.y), one2 = f2_pack(1.f, 1.f);
            const uint64_t cap2 = f2_pack(-2.f * p.mod.cap_log2, -2.f * p.mod.cap_log2);
            const uint64_t step2 = f2_pack(2.f * slope, 2.f * slope);
            const float top = p.mod.cap_log2 - m;
            uint32_t ba[16], bb[16], pw[16];
            auto part = [&](const uint32_t (&sr)[16], int c, int at) {  // columns c .. c + 15, weights to pw[at ..]
              const float off = static_cast<float>(key0 + c - pos);  // minus the distance of the first column
              const int32_t l0 = lo - c, h0 = hi - c;
              uint64_t add2 = f2_pack(fmaf(slope, off, top), fmaf(slope, off + 1.f, top));
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                float e0, e1, t0, t1;
                f2_unpack(f2_mul(f2_pack(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1])), in2), e0, e1);
                f2_unpack(f2_add(f2_pack(ex2(e0), ex2(e1)), one2), e0, e1);
                if (edge) add2 = f2_pack(fmaf(-slope, fabsf(off + 2 * e), top), fmaf(-slope, fabsf(off + (2 * e + 1)), top));
                f2_unpack(f2_fma(f2_pack(rcp_approx(e0), rcp_approx(e1)), cap2, add2), t0, t1);
                if (!edge) add2 = f2_add(add2, step2);
                if (edge) {
                  if (2 * e < l0 || 2 * e >= h0) t0 = -INFINITY;
                  if (2 * e + 1 < l0 || 2 * e + 1 >= h0) t1 = -INFINITY;
                }
                const float p0 = ex2(t0), p1 = ex2(t1);
                sum2[e & 1] = f2_add(sum2[e & 1], f2_pack(p0, p1));
                pw[at + e] = pack_bf16x2(p0, p1);
              }
            };
            tmem_ld16(col, ba);
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              tc_wait_ld_regs16(ba);
              tmem_ld16(col + 32 * c + 16, bb);
              part(ba, 32 * c, 0);
              tc_wait_ld_regs16(bb);
              if (c == 0) tmem_ld16(col + 32, ba);
              part(bb, 32 * c + 16, 8);
              tmem_st16(col + 16 * c, pw);
            }
          };
          if (__any_sync(0xffffffffu, edge_here)) run(BoolTag<true>{});
          else run(BoolTag<false>{});
          float a0, a1, a2, a3;
          f2_unpack(sum2[0], a0, a1);
          f2_unpack(sum2[1], a2, a3);
          l += (a0 + a1) + (a2 + a3);
        }
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(smem_u32(&bar_p[ti]));
      }
      if (!ok) break;
      g += jb.nt;
      // ---- epilogue: O / l, this thread's half of the columns.  A row's halves hand each other their sums in the first of
      // the columns that they have read (shared memory is full); then O_i is released to the next item's first PV.
      const bool late = !mbar_wait(smem_u32(&bar_o[ti]), n & 1);
      if (__any_sync(0xffffffffu, late)) { ok = false; break; }
      tc_fence_after();
      uint32_t oa[D / 64][32];
#pragma unroll
      for (int c = 0; c < D / 64; ++c) tmem_ld32(col_o + c * 32, oa[c]);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) tc_wait_ld_regs(oa[c]);
      // whether the result is finite (bad: 0) goes to the other half with the sum
      float bad[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int e = 0; e < 32; ++e) bad[e & 3] = fmaf(__uint_as_float(oa[c][e]), 0.f, bad[e & 3]);
      bad[0] = (bad[0] + bad[1]) + (bad[2] + bad[3]);
      tmem_st1(col_o, __float_as_uint(l));
      tmem_st1(col_o + 1, __float_as_uint(bad[0]));
      tc_wait_st();
      tc_fence_before();
      mbar_arrive(smem_u32(&bar_join[ti]));
      const bool stuck = !mbar_wait(smem_u32(&bar_join[ti]), n & 1);
      if (__any_sync(0xffffffffu, stuck)) { ok = false; break; }
      tc_fence_after();
      const uint32_t col_other = half == 0 ? col_o + D / 2 : col_o - D / 2;
      uint32_t other, other_bad;
      tmem_ld1(col_other, other);
      tmem_ld1(col_other + 1, other_bad);
      l += __uint_as_float(other);
      tc_fence_before();
      mbar_arrive(smem_u32(&bar_ofree[ti]));
      const bool far = first < lim && (l < kSumFloor || l > kSumCeiling);
      // (where the sum is a NaN, from a score, so is the result)
      const bool redo = row_valid && l == l && (far || !(bad[0] == 0.f && __uint_as_float(other_bad) == 0.f));
      const float inv_l = l == 0.f ? 0.f : 1.f / l;
      const int64_t row = (jb.q_tok0 + tok) * p.hq + jb.kh * G + (r % G);
      const int64_t part_row = (static_cast<int64_t>(jb.slot) * p.hkv + jb.kh) * p.part_rows + ti * kRows + r;
      if (row_valid) {
        if (jb.slot < 0) {
          uint4* dst = reinterpret_cast<uint4*>(p.o + row * D + half * (D / 2));
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = pack_bf16x2(__uint_as_float(oa[c][8 * e + 2 * k]) * inv_l, __uint_as_float(oa[c][8 * e + 2 * k + 1]) * inv_l);
              dst[4 * c + e] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
          float* dst = p.part_o + part_row * D + half * (D / 2);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float v[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(oa[c][8 * e + k]) * inv_l;
              st_global_v8(dst + 32 * c + 8 * e, v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
            }
          if (half == 0) p.part_lse[part_row] = m + __log2f(l);
        }
      }
      // such rows of the warp one by one, behind their own threads' stores, each half's columns by its own warp
      for (uint32_t rows = __ballot_sync(0xffffffffu, redo); rows != 0; rows &= rows - 1) {
        const int src = __ffs(rows) - 1;
        const int64_t row1 = __shfl_sync(0xffffffffu, row, src), at = __shfl_sync(0xffffffffu, part_row, src);
        float y[D / 32], lse;
        if (!mod_row<D, true>(p, jb, __shfl_sync(0xffffffffu, far, src), row1, __shfl_sync(0xffffffffu, first, src),
                              __shfl_sync(0xffffffffu, lim, src), __shfl_sync(0xffffffffu, pos, src),
                              __shfl_sync(0xffffffffu, slope, src), y, lse))
          continue;
        __syncwarp();
        if (lane >> 4 == half) {
#pragma unroll
          for (int v = 0; v < D / 32; ++v) {
            if (jb.slot < 0) p.o[row1 * D + lane * (D / 32) + v] = __float2bfloat16_rn(y[v]);
            else p.part_o[at * D + lane * (D / 32) + v] = y[v];
          }
        }
        if (jb.slot >= 0 && half == 0 && lane == 0) p.part_lse[at] = lse;
      }
    }
    if (!ok) give_up();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ================================================================ softmax (warps 0-7)
    const int ti = warp >> 2;              // query tile
    const int r = threadIdx.x & 127;        // row of the tile = TMEM lane
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t col_s = ti * kKeys;
    const uint32_t col_o = kColO + ti * 128;
    const int tile_tok = ti * T + r / G;    // token / member of the item
    bool ok = true;
    int32_t n = 0, g = 0, join = 0;  // (join: dual items done)
    (void)join;
    for (;; ++n) {
      Job jb;
      const int ri = wait_item(n, jb);
      if (__any_sync(0xffffffffu, ri < 0)) { ok = false; break; }
      if (ri == 0) break;
      const int tok = DUAL && jb.dual ? r / G : tile_tok;
      const bool row_valid = tok < jb.n_valid;
      int32_t lim;  // exclusive key limit of this row (tree: of the keys every row sees)
      int32_t first = 0, pos = 0;  // changed scores: the first key this row sees and its position
      float slope = 0.f;           // and its head's bias per position, in log2 units
      (void)first, (void)pos, (void)slope;
      if constexpr (MOD) {
        pos = jb.causal0 + tok;
        lim = jb.kend;
        first = jb.kbeg;
        if (row_valid) {
          lim = min(max(pos + 1, jb.mem0), jb.kend);
          if (p.mod.window > 0) first = max(first, pos - p.mod.window + 1);
          if (p.mod.first_key) first = max(first, __ldg(p.mod.first_key + jb.q_tok0 + tok));
          if (p.mod.slopes) slope = __ldg(p.mod.slopes + jb.kh * G + r % G) * kLog2e;
        }
      } else if constexpr (TREE) lim = jb.causal0;
      else if constexpr (EXTEND) lim = row_valid ? jb.causal0 + tok + 1 : jb.kend;
      else lim = jb.kend;
      float m_used = -INFINITY, l = 0.f;
      for (int j = 0; j < steps_of(jb); ++j) {
        const int gg = g + j;
        // (as in the MMA warp, no per-tile look at the abort flag: the wait's deadline ends a failed CTA)
        const bool fail_here = !mbar_wait(smem_u32(&bar_s[ti]), gg & 1);
        if (__any_sync(0xffffffffu, fail_here)) { ok = false; break; }  // warp-uniform: tcgen05.ld/st are collective
        if (!live_at(jb, j, ti)) {  // an empty query tile: no S was computed; keep bar_p's phase
          mbar_arrive(smem_u32(&bar_p[ti]));
          continue;
        }
        tc_fence_after();
        const int32_t key0 = jb.kbeg + tile_at(jb, j, ti) * kKeys;
        // (changed scores: also where a key lies behind the row's own position, for the bias by distance)
        const bool masked = MOD ? key0 + kKeys > min(lim, pos + 1) || key0 < first : key0 + kKeys > lim;
        const bool warp_masked = __any_sync(0xffffffffu, masked);
        // tree: bit e of vis[c] = key key0 + 32 c + e is visible to this row
        uint32_t vis[4];
        if constexpr (TREE) {
          vis[0] = vis[1] = vis[2] = vis[3] = 0xffffffffu;
          if (warp_masked) {
            const uint32_t* mrow = p.tree_mask + (jb.q_tok0 + (row_valid ? tok : 0)) * p.mask_words;
            auto word = [&](int32_t i) -> uint32_t {  // drafted tokens 32 i .. of this row's mask
              const int32_t left = jb.mem0 - 32 * i;
              if (left <= 0 || !row_valid) return 0u;
              const uint32_t w = __ldg(mrow + i);
              return left >= 32 ? w : w & ((1u << left) - 1u);
            };
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int32_t off = key0 + 32 * c - lim;  // the chunk's first drafted token
              if (off >= 0) vis[c] = __funnelshift_r(word(off >> 5), word((off >> 5) + 1), off & 31);
              else if (off > -32) vis[c] = (word(0) << -off) | ((1u << -off) - 1u);
            }
            // Drafted tokens' V values that are not finite are set to 0 before the product, which would carry them,
            // times a zero probability, to rows that do not see them (the merge kernel adds them to the rows that
            // do).  Both query tiles of an item read the V tile, PV_1 behind PV_0, so tile 0's threads do it, a key row
            // each (128 bytes per 64-column half, its 16-byte chunks swizzled).
            if (s_job[n % kItemRing].odd && (ti == 0 || (DUAL && jb.dual))) {
              const int32_t kt = s_job[n % kItemRing].kt0 + tile_at(jb, j, ti);
              const bool fail_v = !mbar_wait(smem_u32(&bar_vf[kt % VS]), (kt / VS) & 1);
              if (__any_sync(0xffffffffu, fail_v)) { ok = false; break; }
              if (key0 + r >= lim) {
#pragma unroll 1
                for (int e = 0; e < D / 8; ++e)
                  zero_not_finite_bf16x8(sV(kt % VS) + e / 8 * (kRows * 128) + r * 128 + e % 8 * 16);
              }
              fence_proxy_async_smem();
            }
          }
        }
        (void)vis;
        // Every tile is exponentiated against a reference in a single pass: the current one, or on the
        // item's first tile the maximum of its first 32 columns.  The row sum bounds every probability
        // of the row (p <= sum), so a sum above kFastSumLimit, or one that is not finite, marks the
        // reference as stale: the warp then redoes the tile on the exact path -- row maximum first, lazy
        // reference update, then the exponentials.  P is held in registers until the pass is accepted,
        // since it overwrites S.
        [[maybe_unused]] uint32_t pk[2][32];
        float rowsum = 0.f, alpha = 1.f, m_ref = m_used;
        bool resc = false;
        if constexpr (MOD) {
          // The same with the scores' changes, a chunk's weights going to TMEM at once, over columns of S that are done with,
          // and the tile a short loop over 32-column chunks: holding the 64 registers of P until a tile is settled, as below,
          // left too few for the rest, and unrolled code for all cases ran at the instruction cache's pace (603 -> 435 us for
          // 8 prompts of 700..1500 tokens, 64/8 heads, uncapped).
          //   t = cap log2(e) tanh(y) - slope |pos - key| - reference, y = s sm_scale / cap; or s sm_scale log2(e) - ...
          // Up to the row's position the bias is linear in the key: it and the reference are one addend, stepped along the
          // columns.  The reference only has to keep weights and sums in range (2^60 weighs as exactly as 1 in bf16 and
          // fp32): it is the largest of the row's first scores, up to 16, with the largest bias that any of its keys has (with
          // the first keys' bias, far away, it would have to move in every tile).  It is raised by whole powers of two: between
          // tiles when the sum has grown, and within one when a chunk's sum leaves the range, which scales what the tile has
          // stored so far.  That and scores beyond the polynomial's range take a chunk through a loop of its own, from S, 8
          // columns at a time.  A row whose whole sum is too small for its reference is done again in the epilogue.
          const bool sees = first < key0 + kKeys && first < lim && key0 < lim;  // any key of this tile
          if (!__any_sync(0xffffffffu, sees)) {
            const uint32_t none[32] = {};
            tmem_st32(tmem + lane_addr + col_s, none);
            tmem_st32(tmem + lane_addr + col_s + 32, none);
          } else {
            const int32_t lo = first - key0, hi = lim - key0;  // this row's columns: [lo, hi)
            if (__any_sync(0xffffffffu, m_used == -INFINITY)) {
              // 16 columns at a time, those in which a row without a reference begins
              const bool wants = m_used == -INFINITY && sees;
              float top = -INFINITY;
              int c = __reduce_min_sync(0xffffffffu, wants ? max(lo, 0) & ~15 : kKeys);
#pragma unroll 1
              while (c < kKeys) {
                uint32_t x[16];
                tmem_ld16(tmem + lane_addr + col_s + c, x);
                tc_wait_ld_regs16(x);
#pragma unroll
                for (int e = 0; e < 16; ++e) top = fmaxf(top, c + e >= lo && c + e < hi ? __uint_as_float(x[e]) : -INFINITY);
                c = __reduce_min_sync(0xffffffffu, wants && lo >= c + 16 ? lo & ~15 : kKeys);
              }
              if (top == -INFINITY) top = 0.f;  // (so are the scores that were looked at)
              else top = CAP ? p.mod.cap_log2 * tanh_any(top * p.mod.cap_in) : top * p.scale_log2;
              if (wants) m_ref = top + bias_bound(first, lim, pos, slope);
            }
            if (__any_sync(0xffffffffu, l > kRaiseSum)) {
              const float up = l > kRaiseSum ? static_cast<float>(static_cast<int32_t>(__float_as_uint(l) >> 23) - 127) : 0.f;
              resc = up > 0.f;
              m_ref += up;
              alpha = ex2(-up);
            }
            float m_sub = m_ref == -INFINITY ? 0.f : m_ref;
            uint64_t sum2[2] = {0, 0};
            // the chunks taken: 4, or the index of the first one that needs more
            auto run = [&](auto edge_tag) -> int {
              constexpr bool edge = decltype(edge_tag)::value;  // hidden keys, or keys behind the row's position
              const uint64_t in2 = f2_pack(p.mod.in2.x, p.mod.in2.y);
              const uint64_t step2 = f2_pack(2.f * slope, 2.f * slope);
              auto chunk = [&](const uint32_t (&sr)[32], int c) -> bool {
                const float off = static_cast<float>(key0 + 32 * c - pos);  // minus the distance of the first column
                const int32_t l0 = lo - 32 * c, h0 = hi - 32 * c;
                uint64_t add2 = f2_pack(fmaf(slope, off, -m_sub), fmaf(slope, off + 1.f, -m_sub));
                uint64_t part2[2] = {0, 0};
                uint32_t pw[16];
                float y_max = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const uint64_t s2 = f2_pack(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1]));
                  if (edge)
                    add2 = f2_pack(fmaf(-slope, fabsf(off + 2 * e), -m_sub), fmaf(-slope, fabsf(off + (2 * e + 1)), -m_sub));
                  float t0, t1;
                  if constexpr (CAP) {
                    const uint64_t y2 = f2_mul(s2, in2);
                    const uint64_t z2 = f2_mul(y2, y2);
                    float y0, y1;
                    f2_unpack(y2, y0, y1);
                    y_max = fmaxf(y_max, fmaxf(fabsf(y0), fabsf(y1)));
                    auto coef = [&](int i) { return f2_pack(p.mod.cap_poly[i].x, p.mod.cap_poly[i].y); };
                    uint64_t h2 = coef(kCapTerms - 1);
#pragma unroll
                    for (int i = kCapTerms - 2; i >= 0; --i) h2 = f2_fma(h2, z2, coef(i));
                    f2_unpack(f2_fma(y2, h2, add2), t0, t1);
                  } else {
                    f2_unpack(f2_fma(s2, in2, add2), t0, t1);
                  }
                  if (!edge) add2 = f2_add(add2, step2);
                  if (edge) {
                    if (2 * e < l0 || 2 * e >= h0) t0 = -INFINITY;
                    if (2 * e + 1 < l0 || 2 * e + 1 >= h0) t1 = -INFINITY;
                  }
                  const float p0 = ex2(t0), p1 = ex2(t1);
                  part2[e & 1] = f2_add(part2[e & 1], f2_pack(p0, p1));
                  pw[e] = pack_bf16x2(p0, p1);
                }
                // a score beyond the polynomial, or a sum out of range
                float q0, q1, q2, q3;
                f2_unpack(part2[0], q0, q1);
                f2_unpack(part2[1], q2, q3);
                const bool out = !((q0 + q1) + (q2 + q3) <= kRaiseSum) || (CAP && !(y_max <= kCapPolyMax));
                if (__any_sync(0xffffffffu, out)) return false;
                tmem_st16(tmem + lane_addr + col_s + 16 * c, pw);
                sum2[0] = f2_add(sum2[0], part2[0]);
                sum2[1] = f2_add(sum2[1], part2[1]);
                return true;
              };
              uint32_t ba[32], bb[32];
              tmem_ld32(tmem + lane_addr + col_s, ba);
#pragma unroll 1
              for (int c = 0; c < 4; c += 2) {
                tc_wait_ld_regs(ba);
                tmem_ld32(tmem + lane_addr + col_s + 32 * (c + 1), bb);
                const bool first_done = chunk(ba, c);
                tc_wait_ld_regs(bb);
                if (!first_done) return c;
                if (c == 0) tmem_ld32(tmem + lane_addr + col_s + 64, ba);
                if (!chunk(bb, c + 1)) {
                  if (c == 0) tc_wait_ld_regs(ba);  // (no load in flight when its registers are given up)
                  return c + 1;
                }
              }
              return 4;
            };
            const int done = warp_masked ? run(BoolTag<true>{}) : run(BoolTag<false>{});
            // the chunks from one that was refused on: any scores, from S, 8 columns at a time
#pragma unroll 1
            for (int c = done; c < 4; ++c) {
              float top = -INFINITY, down = 1.f;
#pragma unroll 1
              for (int q = 0; q < 8; ++q) {  // the largest score (q < 4), then the weights
                uint32_t x[8], w[4];
                tmem_ld8(tmem + lane_addr + col_s + 32 * c + 8 * (q & 3), x);
                tc_wait_ld_regs8(x);
                const int32_t at = 32 * c + 8 * (q & 3);
                float t[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float s1 = __uint_as_float(x[e]);
                  t[e] = CAP ? p.mod.cap_log2 * tanh_any(s1 * p.mod.cap_in) : s1 * p.scale_log2;
                  t[e] = fmaf(-slope, fabsf(static_cast<float>(key0 + at + e - pos)), t[e]);
                  if (at + e < lo || at + e >= hi) t[e] = -INFINITY;
                }
                if (q < 4) {
#pragma unroll
                  for (int e = 0; e < 8; ++e) top = fmaxf(top, t[e]);
                  continue;
                }
                if (q == 4) {
                  // (whole powers of two: what is stored is scaled without rounding)
                  const float up = top > m_sub + kRaiseStep ? ceilf(top - m_sub) : 0.f;
                  if (__any_sync(0xffffffffu, up > 0.f)) {
                    down = ex2(-up);
                    m_sub += up;
                    if (up > 0.f) m_ref = m_sub, resc = true;
                    alpha *= down;
                    sum2[0] = f2_mul(sum2[0], f2_pack(down, down));
                    sum2[1] = f2_mul(sum2[1], f2_pack(down, down));
                    tc_wait_st();  // (what follows reads this tile's stores)
#pragma unroll 1
                    for (int k = 0; k < 2 * c; ++k) {
                      uint32_t y[8];
                      tmem_ld8(tmem + lane_addr + col_s + 8 * k, y);
                      tc_wait_ld_regs8(y);
#pragma unroll
                      for (int e = 0; e < 8; ++e)
                        y[e] = pack_bf16x2(__uint_as_float(y[e] << 16) * down, __uint_as_float(y[e] & 0xffff0000u) * down);
                      tmem_st8(tmem + lane_addr + col_s + 8 * k, y);
                    }
                  }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float p0 = ex2(t[2 * e] - m_sub), p1 = ex2(t[2 * e + 1] - m_sub);
                  sum2[0] = f2_add(sum2[0], f2_pack(p0, p1));
                  w[e] = pack_bf16x2(p0, p1);
                }
                tmem_st4(tmem + lane_addr + col_s + 16 * c + 4 * (q & 3), w);
              }
            }
            float a0, a1, a2, a3;
            f2_unpack(sum2[0], a0, a1);
            f2_unpack(sum2[1], a2, a3);
            rowsum = (a0 + a1) + (a2 + a3);
          }
        } else {
        bool exact = false;
#pragma unroll 1
        for (int attempt = 0; attempt < 2; ++attempt) {
          // row max of the raw scores (scale > 0 commutes with max), 8 independent chains
          float mx8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) mx8[e] = -INFINITY;
          auto max_chunk = [&](const uint32_t (&sr)[32], int c) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const bool hidden = TREE ? !(vis[c] >> e & 1u) : masked && key0 + c * 32 + e >= lim;
              const float x = hidden ? -INFINITY : __uint_as_float(sr[e]);
              mx8[e & 7] = fmaxf(mx8[e & 7], x);
            }
          };
          auto max_of = [&]() {
            return fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                         fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]))) * p.scale_log2;
          };
          if (exact) {
            uint32_t ba[32], bb[32];
            tmem_ld32(tmem + lane_addr + col_s, ba);
            tc_wait_ld_regs(ba);
            tmem_ld32(tmem + lane_addr + col_s + 32, bb);
            max_chunk(ba, 0);
            tc_wait_ld_regs(bb);
            tmem_ld32(tmem + lane_addr + col_s + 64, ba);
            max_chunk(bb, 1);
            tc_wait_ld_regs(ba);
            tmem_ld32(tmem + lane_addr + col_s + 96, bb);
            max_chunk(ba, 2);
            tc_wait_ld_regs(bb);
            max_chunk(bb, 3);
            const float m_new = fmaxf(m_used, max_of());
            resc = m_new > m_used + kRescaleThreshold;
            m_ref = resc ? m_new : m_used;
          } else if (j == 0) {
            // the item's first tile: the reference is the maximum of chunk 0 (it holds a key of every
            // row: the row's first key is the tile's first).  O and l are empty, nothing to rescale.
            uint32_t ba[32];
            tmem_ld32(tmem + lane_addr + col_s, ba);
            tc_wait_ld_regs(ba);
            max_chunk(ba, 0);
            m_ref = max_of();
          }
          const float m_sub = (m_ref == -INFINITY) ? 0.f : m_ref;
          alpha = resc ? ex2(m_used - m_sub) : 1.f;
          // p = 2^(s * scale_log2 - m_ref): packed FMA pairs + one MUFU per score, packed to bf16 pairs
          const uint64_t scale2 = f2_pack(p.scale_log2, p.scale_log2);
          const uint64_t neg_m2 = f2_pack(-m_sub, -m_sub);
          uint64_t sum2[4] = {0, 0, 0, 0};  // 4 independent chains of (even, odd) partial sums
          // The causal / range mask is compiled only into the variant a warp takes when one of its rows
          // ends inside this tile: the other tiles issue no compare or select per score.
          auto exp_chunk = [&](const uint32_t (&sr)[32], int c, auto mask_tag) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float s0 = __uint_as_float(sr[2 * e]), s1 = __uint_as_float(sr[2 * e + 1]);
              if constexpr (decltype(mask_tag)::value) {
                if (TREE ? !(vis[c] >> (2 * e) & 1u) : key0 + c * 32 + 2 * e >= lim) s0 = -INFINITY;
                if (TREE ? !(vis[c] >> (2 * e + 1) & 1u) : key0 + c * 32 + 2 * e + 1 >= lim) s1 = -INFINITY;
              }
              float t0, t1;
              f2_unpack(f2_fma(f2_pack(s0, s1), scale2, neg_m2), t0, t1);
              const float p0 = ex2(t0), p1 = ex2(t1);
              sum2[e & 3] = f2_add(sum2[e & 3], f2_pack(p0, p1));
              pk[c >> 1][(c & 1) * 16 + e] = pack_bf16x2(p0, p1);
            }
          };
          auto exp_tile = [&](auto mask_tag) {
            uint32_t ba[32], bb[32];
            tmem_ld32(tmem + lane_addr + col_s, ba);
            tc_wait_ld_regs(ba);
            tmem_ld32(tmem + lane_addr + col_s + 32, bb);
            exp_chunk(ba, 0, mask_tag);
            tc_wait_ld_regs(bb);
            tmem_ld32(tmem + lane_addr + col_s + 64, ba);
            exp_chunk(bb, 1, mask_tag);
            tc_wait_ld_regs(ba);
            tmem_ld32(tmem + lane_addr + col_s + 96, bb);
            exp_chunk(ba, 2, mask_tag);
            tc_wait_ld_regs(bb);
            exp_chunk(bb, 3, mask_tag);
          };
          if (warp_masked) exp_tile(BoolTag<true>{});
          else exp_tile(BoolTag<false>{});
          float sum8[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) f2_unpack(sum2[e], sum8[2 * e], sum8[2 * e + 1]);
          rowsum = ((sum8[0] + sum8[1]) + (sum8[2] + sum8[3])) + ((sum8[4] + sum8[5]) + (sum8[6] + sum8[7]));
          if (exact) break;
          // (a tree row may see no key of the first tile's chunk 0, or of any tile so far: no reference yet)
          const bool stale = !(rowsum <= kFastSumLimit) || (TREE && m_ref == -INFINITY);
          if (!__any_sync(0xffffffffu, stale)) break;
          exact = true;
        }
        }
        // P (bf16 pairs) over the first 64 columns of S, read by the PV MMA
        if constexpr (!MOD) {
          tmem_st32(tmem + lane_addr + col_s, pk[0]);
          tmem_st32(tmem + lane_addr + col_s + 32, pk[1]);
        }
        l = l * alpha + rowsum;
        if (j > 0 && __any_sync(0xffffffffu, resc)) {
          // O_i holds PV_i(j-1): the commit that signalled S_i(j) covers every earlier MMA
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld32(tmem + lane_addr + col_o + c * 32, ov);
            tc_wait_ld_regs(ov);
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st32(tmem + lane_addr + col_o + c * 32, ov);
          }
        }
        m_used = m_ref;
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(smem_u32(&bar_p[ti]));
      }
      if (!ok) break;
      g += steps_of(jb);
      // ---- epilogue: O / l, then O_i is released to the next item's first PV
      const bool late = !mbar_wait(smem_u32(&bar_o[ti]), n & 1);
      if (__any_sync(0xffffffffu, late)) { ok = false; break; }
      tc_fence_after();
      float own = 1.f, other = 0.f;  // a dual item's factors of this tile's O and of tile 1's
      (void)own, (void)other;
      if constexpr (DUAL) {
        if (jb.dual && ti == 1) {
          // tile 0's threads read this tile's sums and O of the same rows
          s_join[r] = make_float2(m_used, l);
          tc_fence_before();
          mbar_arrive(smem_u32(&bar_join[0]));
          const bool stuck = !mbar_wait(smem_u32(&bar_join[1]), join & 1);
          ++join;
          if (__any_sync(0xffffffffu, stuck)) { ok = false; break; }
          tc_fence_before();
          mbar_arrive(smem_u32(&bar_ofree[ti]));
          continue;
        }
        if (jb.dual) {
          const bool stuck = !mbar_wait(smem_u32(&bar_join[0]), join & 1) || !mbar_wait(smem_u32(&bar_o[1]), n & 1);
          ++join;
          if (__any_sync(0xffffffffu, stuck)) { ok = false; break; }
          tc_fence_after();
          const float2 b = s_join[r];
          const float top = fmaxf(m_used, b.x), ref = top == -INFINITY ? 0.f : top;
          own = ex2(m_used - ref), other = ex2(b.x - ref);
          m_used = top;
          l = l * own + b.y * other;
        }
      }
      const float inv_l = (TREE || MOD) && l == 0.f ? 0.f : 1.f / l;  // a row that sees nothing gives 0
      // O of this thread's row, all columns, as the epilogues write it (a dual item's two halves joined)
      auto load_o = [&](uint32_t (&oa)[D / 32][32]) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) tmem_ld32(tmem + lane_addr + col_o + c * 32, oa[c]);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) tc_wait_ld_regs(oa[c]);  // ties each array to the wait (one real wait)
        if constexpr (DUAL) {
          if (jb.dual) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t ob[32];
              tmem_ld32(tmem + lane_addr + col_o + 128 + c * 32, ob);
              tc_wait_ld_regs(ob);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                oa[c][e] = __float_as_uint(__uint_as_float(oa[c][e]) * own + __uint_as_float(ob[e]) * other);
            }
            tc_fence_before();
            mbar_arrive(smem_u32(&bar_join[1]));
          }
        }
      };
      // changed scores: a result that is not finite (where the sum is: a NaN there comes from a score)
      [[maybe_unused]] auto odd_row = [&](const uint32_t (&oa)[D / 32][32]) -> bool {
        float bad[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e) bad[e & 3] = fmaf(__uint_as_float(oa[c][e]), 0.f, bad[e & 3]);
        return row_valid && l == l && !((bad[0] + bad[1]) + (bad[2] + bad[3]) == 0.f);
      };
      [[maybe_unused]] bool redo = false;
      [[maybe_unused]] int64_t part_row = 0;
      if (EXTEND && (!(TREE || MOD) || jb.slot < 0)) {
        __nv_bfloat16* dst = p.o + ((jb.q_tok0 + tok) * p.hq + jb.kh * G + (r % G)) * static_cast<int64_t>(D);
        uint32_t oa[D / 32][32];
        load_o(oa);
        if constexpr (MOD) redo = odd_row(oa);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const uint32_t (&ov)[32] = oa[c];
          uint32_t pko[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            pko[e] = pack_bf16x2(__uint_as_float(ov[2 * e]) * inv_l, __uint_as_float(ov[2 * e + 1]) * inv_l);
          if (row_valid) {
            uint4* d4 = reinterpret_cast<uint4*>(dst + c * 32);
#pragma unroll
            for (int e = 0; e < 4; ++e) d4[e] = make_uint4(pko[4 * e], pko[4 * e + 1], pko[4 * e + 2], pko[4 * e + 3]);
          }
        }
      } else {
        // fp32 partial rows, one per thread, at [slot][member][q head] (the G heads of a member contiguous),
        // written in whole 32-byte sectors
        // (tree, changed scores: at [slot][kv head][row of the item])
        bool write = row_valid;
        int64_t ps;
        if constexpr (TREE || MOD) {
          ps = (static_cast<int64_t>(jb.slot) * p.hkv + jb.kh) * p.part_rows + (row_valid ? ti * kRows + r : 0);
        } else {
          const int32_t member = __ldg(p.group_reqs + jb.mem0 + (row_valid ? tok : 0));
          write = row_valid && member >= 0 && member < p.batch;
          ps = (static_cast<int64_t>(jb.slot) * p.batch + (write ? member : 0)) * p.hq + jb.kh * G + (r % G);
        }
        float* dst = (TREE || MOD ? p.part_o : p.casc_o) + ps * D;
        uint32_t oa[D / 32][32];
        load_o(oa);
        if constexpr (MOD) redo = odd_row(oa), part_row = ps;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const uint32_t (&ov)[32] = oa[c];
          if (write) {
#pragma unroll
            for (int e = 0; e < 4; ++e)  // whole 32-byte sectors
              st_global_v8(dst + c * 32 + 8 * e, __uint_as_float(ov[8 * e]) * inv_l,
                           __uint_as_float(ov[8 * e + 1]) * inv_l, __uint_as_float(ov[8 * e + 2]) * inv_l,
                           __uint_as_float(ov[8 * e + 3]) * inv_l, __uint_as_float(ov[8 * e + 4]) * inv_l,
                           __uint_as_float(ov[8 * e + 5]) * inv_l, __uint_as_float(ov[8 * e + 6]) * inv_l,
                           __uint_as_float(ov[8 * e + 7]) * inv_l);
          }
        }
        if (write) (TREE || MOD ? p.part_lse : p.casc_lse)[ps] = m_used + __log2f(l);
      }
      if constexpr (MOD) {
        const bool far = row_valid && first < lim && (l < kSumFloor || l > kSumCeiling);
        // such rows of the warp one by one, behind their own threads' stores
        for (uint32_t rows = __ballot_sync(0xffffffffu, redo || far); rows != 0; rows &= rows - 1) {
          const int src = __ffs(rows) - 1;
          const int64_t row = __shfl_sync(0xffffffffu, (jb.q_tok0 + tok) * p.hq + jb.kh * G + (r % G), src);
          float y[D / 32], lse;
          if (!mod_row<D, CAP>(p, jb, __shfl_sync(0xffffffffu, far, src), row, __shfl_sync(0xffffffffu, first, src),
                               __shfl_sync(0xffffffffu, lim, src), __shfl_sync(0xffffffffu, pos, src),
                               __shfl_sync(0xffffffffu, slope, src), y, lse))
            continue;
          __syncwarp();
          const int64_t at = __shfl_sync(0xffffffffu, part_row, src);
#pragma unroll
          for (int v = 0; v < D / 32; ++v) {
            if (jb.slot < 0) p.o[row * D + lane * (D / 32) + v] = __float2bfloat16_rn(y[v]);
            else p.part_o[at * D + lane * (D / 32) + v] = y[v];
          }
          if (jb.slot >= 0 && lane == 0) p.part_lse[at] = lse;
        }
      }
      tc_fence_before();
      mbar_arrive(smem_u32(&bar_ofree[ti]));
    }
    if (!ok) give_up();
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (!EXTEND) {
    // the prefix partials of this CTA are written (the barrier orders every warp's stores before this
    // thread's fence): the decode combine merges a request's partials once every CTA has counted itself
    if (threadIdx.x == 0) {
      __threadfence();
      atomicAdd(p.done_counter, 1);
    }
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace ra
