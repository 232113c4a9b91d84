// tree.cu -- ra_tree_attention: drafted tokens of a tree over a cached prefix.
//
// Each request has T drafted tokens whose K/V sit in the pool behind its P cached ones; drafted token i
// attends to all of the prefix and to the drafted tokens its bit mask names:
//   o_i = sum_j softmax_j(scale <q_i, k_j>) v_j   over j < P and over P + t with bit t of mask_i.
// One pass does both parts; rows are (token, head of the GQA group), and only the keys of drafted tokens look
// at the masks.  T * G rows share every key of a kv head:
//  * up to 32 rows the call is bound by HBM (2 flop per byte and row), and the items of tree_narrow.cu stream
//    whole slot rows of several heads with few large copies (small calls of up to 128 rows take several such
//    items per request: 8 x 20..40 tokens of 16/16 heads 44.6 us on the wide path, 29.0 on this);
//  * more rows go to the tcgen05 attention kernel (attn_tc.cuh, kTreePass), up to 256 rows per item, each gathered
//    128-key tile feeding all of them.  It is bound by its chain of QK, softmax and PV per key tile more than by the
//    gathers: with half of each K and V row gathered, 64 requests x 32..64 tokens over 512..4096 keys, 64/8 heads,
//    take 261 us of 298, and x 8..16 tokens 128 of 134.  The chain's time does not shrink with the rows: x 4..8 tokens
//    of 32/8 heads took it 145 us and take the narrow path 112.
// Around it:
//  * the work list (one CTA, on the device, from the real lengths; small calls: every warp for itself) splits
//    the key ranges only as far as the SMs need it, since an unsplit item writes its bf16 rows directly while
//    a split one costs fp32 partials (4 * D + 4 bytes per row and split, written and read again) and a merge;
//  * a persistent merge kernel joins the splits; with nothing split it only looks at a count.
// A value of V that is not finite must not reach rows whose mask leaves its token out, but a matrix product
// multiplies it by their zero probability (0 * inf = NaN).  The drafted tokens' V are therefore looked over (by
// the narrow kernel in its slabs, for wide calls by the list kernel's other CTAs: at most a few MB), the (request, kv
// head) pairs that hold one marked, and such values set to 0 in shared memory before the product; the merge kernel
// adds them to the rows that see them.  What that costs does not depend on the prefix: 2 requests x 64 tokens of
// 64/8 heads over 1,000 keys take 32 us, 74 with one such value, and 22 ms where the head's rows are computed again
// key by key; 64 x 32..64 over 512..4096 303 us, 1.2 ms with all of them.  Prefix keys are seen by every row: there
// the product's NaN is the answer.
#include <cmath>

#include "api_common.h"
#include "attn_tc.cuh"
#include "attn_tc_host.h"
#include "slab_ring.cuh"
#include "tree_internal.h"

namespace ra {

namespace {

constexpr int kScanThreads = 1024;  // the list kernel's block: the scan's loads in flight
constexpr int kPlanThreads = 256;   // of which this many build the list: one SM's issue slots bound it
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanCached = 1024;  // requests whose lengths the list kernel keeps in shared memory
constexpr int kBins = kPlanThreads;  // size classes of the items, longest first
constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;

// CTA 0 lists the items, longest first; CTAs 1 .. (wide calls) scan the drafted tokens' V rows, one request at a time.
__global__ void __launch_bounds__(kScanThreads) tree_plan_kernel(const __grid_constant__ TreeParams p, int32_t head_dim) {
  griddep_wait();  // the call's inputs; the workspace may still be read by the call before
  griddep_launch();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (blockIdx.x > 0) {
    for (int32_t b = blockIdx.x - 1; b < p.batch; b += gridDim.x - 1) {
      for (int32_t h = t; h < p.hkv; h += kScanThreads) p.ws.bad[b * p.hkv + h] = 0;
      __syncthreads();
      int32_t P, T;
      if (!tree_request(p, b, P, T, false)) continue;
      const int32_t* slots = p.table + static_cast<int64_t>(__ldg(p.rpi + b)) * p.table_stride + P;
      const int32_t vecs = p.hkv * head_dim / 8, per_head = head_dim / 8;
      for (int32_t j = warp; j < T; j += kScanThreads / 32) {
        int32_t slot = __ldg(slots + j);
        if (slot < 0 || slot >= p.num_slots) slot = 0;  // (as the attention kernel reads it, which flags it)
        const uint4* v = reinterpret_cast<const uint4*>(p.v_pool) + static_cast<int64_t>(slot) * vecs;
        for (int32_t c = lane; c < vecs; c += 32) {
          const uint4 x = __ldg(v + c);
          const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                      __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
          if ((m & 0xffffu) >= 0x7f80u || (m >> 16) >= 0x7f80u) p.ws.bad[b * p.hkv + c / per_head] = 1;
        }
      }
    }
    return;
  }
  if (p.sh.narrow)  // the attention kernel finds the marks itself
    for (int32_t i = t; i < p.batch * p.hkv; i += kScanThreads) p.ws.bad[i] = 0;
  if (t >= kPlanThreads) return;
  auto list_sync = []() { asm volatile("bar.sync 1, %0;" ::"n"(kPlanThreads) : "memory"); };  // (the list's threads)
  __shared__ int32_t s_bin[kBins];
  __shared__ int32_t s_warp[kPlanWarps], s_long[kPlanWarps], s_entries[kPlanWarps], s_chunk[kPlanWarps];
  __shared__ float s_cost[kPlanWarps];
  __shared__ unsigned long long s_work[kPlanWarps];
  __shared__ int32_t s_parts, s_merges;
  __shared__ int4 s_req[kPlanCached];  // P, T (0 where nothing is computed), units, query tiles
  s_bin[t] = 0;
  if (t == 0) s_parts = s_merges = 0;
  const int32_t per_item = p.sh.tokens_per_item, heads = p.sh.heads, unit = p.sh.unit;
  const int32_t slots = p.sh.waves * kTreeSms;  // items that fill the SMs `waves` times
  const int32_t ctas = p.sh.per_sm * kTreeSms;
  auto request = [&](int32_t b, bool first) -> int4 {
    if (!first && b < kPlanCached) return s_req[b];
    int4 q;
    if (!tree_request(p, b, q.x, q.y, first)) return make_int4(0, 0, 0, 0);
    q.z = (q.x + q.y + unit - 1) / unit;
    q.w = (q.y + per_item - 1) / per_item;
    return q;
  };
  unsigned long long work = 0;
  int32_t entries = 0, longest = 1;
  for (int32_t b = t; b < p.batch; b += kPlanThreads) {
    const int4 q = request(b, true);
    if (b < kPlanCached) s_req[b] = q;
    work += static_cast<unsigned long long>(q.w) * q.z;
    entries += q.w;
    longest = max(longest, q.z);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) work += __shfl_xor_sync(0xffffffffu, work, off);
  entries = __reduce_add_sync(0xffffffffu, entries);
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 0) s_work[warp] = work, s_entries[warp] = entries, s_long[warp] = longest;
  list_sync();
  work = 0, entries = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) {
    work += s_work[w];
    entries += s_entries[w];
    longest = max(longest, s_long[w]);
  }
  // Units per split.  The least is total / (waves * SMs), which bounds the partials.  With that many unsplit
  // items it also balances the SMs; with fewer, the longest range is cut into the number of pieces (at most
  // two per SM and head) whose longest-first schedule is shortest: the rounds of full pieces, and what the
  // shorter last pieces take beyond the gaps of the last round.  64 numbers of pieces are weighed, four
  // threads each; the estimate may round (only the choice depends on it).  How much of the gaps is taken and
  // what the last pieces stick out by is measured (64 x 4..8 tokens of 32/8 heads over 512..4096 keys with the wide
  // path's factors 118.6 us, with their own 110.6; 8 x 32..64 tokens of 64/8 heads with the narrow path's 75.2,
  // with their own 73.0).
  const unsigned long long all = work * heads;
  const unsigned long long per_slot =
      all >> 31 ? (all + slots - 1) / slots : (static_cast<uint32_t>(all) + slots - 1) / static_cast<uint32_t>(slots);
  const int32_t least = max(1, static_cast<int32_t>(min(per_slot, static_cast<unsigned long long>(longest))));
  int32_t chunk = least;
  if (static_cast<int64_t>(entries) * heads < slots) {
    const int32_t most = max(1, min(longest, 2 * ctas / heads));
    const int32_t cand = t >> 2;
    const int32_t k = cand < 32 ? min(cand + 1, most) : min(most, 32 + (cand - 31) * max(most - 32, 0) / 32);
    const int32_t c = max((longest + k - 1) / k, least);
    const float per = 1.f / static_cast<float>(c);
    int32_t n_full = 0, n_rem = 0, rem_units = 0;
    for (int32_t b = t & 3; b < p.batch; b += 4) {
      const int4 q = request(b, false);
      const int32_t full = static_cast<int32_t>(static_cast<float>(q.z) * per + 1e-3f), rem = max(q.z - full * c, 0);
      n_full += q.w * full;
      n_rem += rem > 0 ? q.w : 0;
      rem_units += q.w * rem;
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      n_full += __shfl_xor_sync(0xffffffffu, n_full, off);
      n_rem += __shfl_xor_sync(0xffffffffu, n_rem, off);
      rem_units += __shfl_xor_sync(0xffffffffu, rem_units, off);
    }
    const float piece = static_cast<float>(c + (c < longest ? p.sh.split_overhead : p.sh.overhead));
    const float fulls = static_cast<float>(n_full * heads);
    const float sms = static_cast<float>(ctas), rounds = fmaxf(ceilf(fulls / sms), 1.f);
    const float rest = static_cast<float>(rem_units * heads) + static_cast<float>(n_rem * heads) * p.sh.split_overhead;
    const float beyond = rest - (p.sh.narrow ? 1.f : 0.8f) * (rounds * sms - fulls) * piece;
    float cost = rounds * piece + (beyond > 0.f ? beyond / sms + (p.sh.narrow ? 0.35f : 0.5f) * static_cast<float>(c) : 0.f);
    int32_t mine = c;
#pragma unroll
    for (int off = 16; off >= 4; off >>= 1) {
      const float oc = __shfl_xor_sync(0xffffffffu, cost, off);
      const int32_t om = __shfl_xor_sync(0xffffffffu, mine, off);
      if (oc < cost || (oc == cost && om > mine)) cost = oc, mine = om;  // on a tie the longer piece
    }
    if (lane == 0) s_cost[warp] = cost, s_chunk[warp] = mine;
    list_sync();
    chunk = s_chunk[0], cost = s_cost[0];
#pragma unroll
    for (int w = 1; w < kPlanWarps; ++w)
      if (s_cost[w] < cost || (s_cost[w] == cost && s_chunk[w] > chunk)) cost = s_cost[w], chunk = s_chunk[w];
  }
  // counting sort of the items by size, longest first
  const float scale = (kBins - 1) / static_cast<float>(min(chunk, longest));
  auto bin_of = [&](int32_t units) {
    return kBins - 1 - min(kBins - 1, static_cast<int32_t>(static_cast<float>(units) * scale));
  };
  const int32_t full_bin = bin_of(chunk);
  for (int32_t b = t; b < p.batch; b += kPlanThreads) {
    const int4 q = request(b, false);
    const int32_t full = q.z / chunk, rem = q.z - full * chunk;
    if (full > 0) atomicAdd(&s_bin[full_bin], full * q.w);
    if (rem > 0) atomicAdd(&s_bin[bin_of(rem)], q.w);
  }
  list_sync();
  const int32_t mine = s_bin[t];
  int32_t incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) s_warp[warp] = incl;
  list_sync();
  int32_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  s_bin[t] = before + incl - mine;
  list_sync();
  // The items of a request are its full pieces, then its shorter last one, of each query tile.  Every lane
  // takes the places of a request of its own (requests strided over the warps), then the warp writes the
  // items of its lanes' requests together.
  int4* items = reinterpret_cast<int4*>(p.ws.items);
  for (int32_t b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
    const int32_t b = b0 + lane * kPlanWarps + warp;
    const bool in = b < p.batch;
    const int4 q = in ? request(b, false) : make_int4(0, 0, 0, 0);
    const int32_t full = q.z / chunk, rem = q.z - full * chunk, splits = full + (rem > 0 ? 1 : 0);
    int32_t at_full = 0, at_rem = 0, part0 = 0, merge0 = 0, row = 0, q0 = 0;
    if (q.y > 0) {
      row = __ldg(p.rpi + b);
      q0 = __ldg(p.qo_indptr + b);
      if (full > 0) at_full = atomicAdd(&s_bin[full_bin], full * q.w);
      if (rem > 0) at_rem = atomicAdd(&s_bin[bin_of(rem)], q.w);
      if (splits > 1) {
        part0 = atomicAdd(&s_parts, splits * q.w);
        merge0 = atomicAdd(&s_merges, q.w);
      }
    }
    for (uint32_t left = __ballot_sync(0xffffffffu, q.y > 0); left != 0; left &= left - 1) {
      const int src = __ffs(left) - 1;
      auto of = [&](int32_t x) { return __shfl_sync(0xffffffffu, x, src); };
      const int32_t n = of(splits), nf = of(full), n_tiles = of(q.w), pf = of(at_full), pr = of(at_rem), part = of(part0),
                    mg = of(merge0), bb = of(b);
      const int4 about = make_int4(of(q.x), of(q.y), of(row), of(q0));
      for (int32_t i = lane; i < n_tiles * n; i += 32) {
        const int32_t tile = i / n, s = i - tile * n;
        const int32_t pos = s < nf ? pf + tile * nf + s : pr + tile;
        if (n > 1 && s == 0)
          reinterpret_cast<int4*>(p.ws.merges)[mg + tile] = make_int4(bb, tile, part + tile * n, n);
        if (pos < p.ws.cap) {
          items[2 * pos] = make_int4(bb, tile, s, n > 1 ? part + tile * n + s : -1);
          items[2 * pos + 1] = about;
        } else {
          flag_error(p.err, RA_DEVERR_LENGTH);  // draft lengths sum above total_q
        }
      }
    }
  }
  list_sync();
  if (t == 0) {
    p.ws.header[0] = static_cast<int32_t>(total < p.ws.cap ? total : p.ws.cap);
    p.ws.header[1] = 0;
    p.ws.header[2] = chunk * unit;
    p.ws.header[3] = s_merges;
  }
}

// Add to row (token i of request b, q head h) of o the values that are not finite of the drafted tokens it sees, which
// the attention kernels took as 0: one warp, D / 32 dims per lane, 4 tokens' rows in flight.  A weight is positive, so
// such a value makes the row's dimension infinite, or NaN with an infinity of the other sign.  (The row was written
// by this warp or by the kernel before.)
template <int D>
__device__ __forceinline__ void add_odd_values(const TreeParams& p, int32_t b, int32_t i, int32_t h) {
  constexpr int V = D / 32, kAhead = 4;
  const int lane = threadIdx.x & 31;
  int32_t P, T;
  if (!tree_request(p, b, P, T, false)) return;
  const int64_t row = __ldg(p.qo_indptr + b) + i;
  const int32_t* slots = p.table + static_cast<int64_t>(__ldg(p.rpi + b)) * p.table_stride + P;
  const uint32_t* mrow = p.mask + row * p.mask_words;
  float add[V] = {};
  for (int32_t j0 = 0; j0 < T; j0 += kAhead) {
    const int32_t left = T - j0;
    uint32_t seen = __ldg(mrow + (j0 >> 5)) >> (j0 & 31) & ((1u << kAhead) - 1u);
    if (left < kAhead) seen &= (1u << left) - 1u;
    if (seen == 0) continue;
    uint32_t w[kAhead][V / 2];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
#pragma unroll
      for (int e = 0; e < V / 2; ++e) w[k][e] = 0;
      if (seen >> k & 1u) {
        int32_t slot = __ldg(slots + j0 + k);
        if (slot < 0 || slot >= p.num_slots) slot = 0;
        const uint32_t* v = reinterpret_cast<const uint32_t*>(
            p.v_pool + (static_cast<int64_t>(slot) * p.hkv + h / p.group) * D + lane * V);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) w[k][e] = __ldg(v + e);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        if ((w[k][e] & 0x7f80u) == 0x7f80u) add[2 * e] += __uint_as_float(w[k][e] << 16);
        if ((w[k][e] & 0x7f800000u) == 0x7f800000u) add[2 * e + 1] += __uint_as_float(w[k][e] & 0xffff0000u);
      }
  }
  __nv_bfloat16* dst = p.o + (row * p.hq + h) * D + lane * V;
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (add[e] != 0.f) dst[e] = __float2bfloat16_rn(__bfloat162float(dst[e]) + add[e]);  // (an infinity or NaN)
}

// The same for the rows of split query tiles that a warp of the merge kernel wrote: its units' once more.
template <int D, bool FEW>
__device__ __forceinline__ void add_to_split_rows(const TreeParams& p, int per_row) {
  constexpr int kRows = FEW ? 1 : 4;  // of a warp and unit
  const int warp = threadIdx.x >> 5;
  if (FEW && warp % per_row != 0) return;
  const int rows_per_unit = FEW ? kMergeWarps / per_row : kMergeWarps * kRows;
  const int32_t tile_rows = p.hkv * p.ws.part_rows, chunks = (tile_rows + rows_per_unit - 1) / rows_per_unit;
  const int64_t units = static_cast<int64_t>(__ldcg(p.ws.header + 3)) * chunks;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t entry = u / chunks;
    const int4 e = __ldcg(reinterpret_cast<const int4*>(p.ws.merges) + entry);
    const int32_t flat0 = static_cast<int32_t>(u - entry * chunks) * rows_per_unit + (FEW ? warp / per_row : warp * kRows);
    for (int32_t flat = flat0; flat < flat0 + kRows && flat < tile_rows; ++flat) {
      const int32_t kh = flat / p.ws.part_rows, r = flat - kh * p.ws.part_rows;
      const int32_t tok = e.y * p.sh.tokens_per_item + r / p.group;
      if (tok < __ldg(p.draft_lens + e.x) && __ldcg(p.ws.bad + static_cast<int64_t>(e.x) * p.hkv + kh) != 0)
        add_odd_values<D>(p, e.x, tok, kh * p.group + r % p.group);
    }
  }
}

// The same for query tile i (of all requests and kv heads) if it is of a marked pair and was not split (its keys fit
// the chunk), by a CTA.
template <int D>
__device__ __forceinline__ void add_to_whole_rows(const TreeParams& p, int64_t i, int64_t tiles) {
  const int64_t pair = i / p.sh.q_tiles;
  if (i >= tiles || __ldcg(p.ws.bad + pair) == 0) return;
  const int32_t b = static_cast<int32_t>(pair / p.hkv), kh = static_cast<int32_t>(pair % p.hkv);
  const int32_t t0 = static_cast<int32_t>(i % p.sh.q_tiles) * p.sh.tokens_per_item;
  int32_t P, T;
  if (!tree_request(p, b, P, T, false) || P + T > __ldcg(p.ws.header + 2)) return;
  const int32_t rows = min(T - t0, p.sh.tokens_per_item) * p.group;
  for (int32_t r = threadIdx.x >> 5; r < rows; r += kMergeWarps)
    add_odd_values<D>(p, b, t0 + r / p.group, kh * p.group + r % p.group);
}

// Join the splits (o = sum_s 2^(lse_s - M) o_s / sum_s 2^(lse_s - M)), and add the values that are not finite to the rows
// of marked (request, kv head) pairs: to a split tile's row by the warp that wrote it, to the others at the end, by
// (pair, query tile) over the grid.  Persistent: a unit is kMergeThreads / 8 rows of a split query tile (all kv heads), 8 lanes
// per row, or (FEW) kMergeWarps / `per_row` rows, `per_row` warps each taking a share of a row's partials, so
// that few rows with many splits do not wait on one warp's loads.
template <int D, bool FEW>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const __grid_constant__ TreeParams p, int per_row) {
  constexpr int LPR = FEW ? 32 : 8;
  constexpr int V = D / LPR;
  __shared__ float s_acc[FEW ? kMergeWarps : 1][32 * V], s_m[kMergeWarps], s_w[kMergeWarps];
  // The attention kernel waited for the plan before it let this one launch: the plan's lists may be read at
  // once.  The partials and the marks may be read, and o written, once the attention kernel is complete.
  griddep_launch();
  // (With the wait comes the load of a mark for the query tiles that were not split, looked at in the end: of tile
  // blockIdx.x + lookers * threadIdx.x, so that marked ones are spread over the CTAs of the first wave.)
  const int32_t lookers = min(static_cast<int32_t>(gridDim.x), kTreeSms);
  const int64_t tiles = static_cast<int64_t>(p.batch) * p.hkv * p.sh.q_tiles;
  auto pair_of = [&](int64_t i) { return i < tiles ? static_cast<int32_t>(i / p.sh.q_tiles) : -1; };
  auto mark_of = [&](int32_t pair) -> int32_t { return pair >= 0 ? __ldcg(p.ws.bad + pair) : 0; };
  const int32_t first_pair = blockIdx.x < lookers ? pair_of(blockIdx.x + static_cast<int64_t>(threadIdx.x) * lookers) : -1;
  int32_t mark = 0;
  bool waited = false;
  auto wait_partials = [&]() {
    if (!waited) {
      griddep_wait();
      mark = mark_of(first_pair);
    }
    waited = true;
  };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LPR;
  const int rows_per_unit = FEW ? kMergeWarps / per_row : kMergeThreads / LPR;
  const int share = FEW ? warp % per_row : 0;
  const int mine = FEW ? warp / per_row : static_cast<int>(threadIdx.x) / LPR;
  const int32_t tile_rows = p.hkv * p.ws.part_rows;  // rows of a query tile, all kv heads
  const int32_t chunks = (tile_rows + rows_per_unit - 1) / rows_per_unit;
  const int64_t units = static_cast<int64_t>(__ldcg(p.ws.header + 3)) * chunks;
  bool marked = false;  // one of this thread's rows is of a marked pair
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t entry = u / chunks;
    const int32_t flat = static_cast<int32_t>(u - entry * chunks) * rows_per_unit + mine;
    const bool in = flat < tile_rows;
    const int32_t kh = in ? flat / p.ws.part_rows : 0, r = in ? flat - kh * p.ws.part_rows : 0;
    const int4 e = __ldcg(reinterpret_cast<const int4*>(p.ws.merges) + entry);
    const int32_t tok = e.y * p.sh.tokens_per_item + r / p.group;
    const bool live = in && tok < __ldg(p.draft_lens + e.x);
    const int64_t slot_rows = static_cast<int64_t>(p.hkv) * p.ws.part_rows;  // rows between partial slots
    const int64_t row0 = (static_cast<int64_t>(e.z) * p.hkv + kh) * p.ws.part_rows + r;
    const int64_t row = __ldg(p.qo_indptr + e.x) + tok;
    __nv_bfloat16* dst = p.o + (row * p.hq + kh * p.group + r % p.group) * D;
    wait_partials();
    marked = marked || (live && __ldcg(p.ws.bad + static_cast<int64_t>(e.x) * p.hkv + kh) != 0);
    auto lse_at = [&](int s) { return __ldcg(p.ws.part_lse + row0 + s * slot_rows); };
    auto row_at = [&](int s, float(&x)[V]) { load_row_part<LPR, V>(p.ws.part_o + (row0 + s * slot_rows) * D, sub, x); };
    float acc[V], wsum;
    if constexpr (FEW) {
      float m;
      merge_partials<V, 8>(
          live ? e.w : 0, share, per_row, lse_at,
          [&](int s, float(&x)[V]) { load_row_cg<V>(p.ws.part_o + (row0 + s * slot_rows) * D + lane * V, x); }, acc, m,
          wsum);
      __syncthreads();  // the unit before has been read
#pragma unroll
      for (int v = 0; v < V; ++v) s_acc[warp][lane * V + v] = acc[v];
      if (lane == 0) s_m[warp] = m, s_w[warp] = wsum;
      __syncthreads();
      if (share != 0 || !live) continue;
      join_shares<V>(per_row, warp, s_acc, s_m, s_w, acc, wsum);
      const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
#pragma unroll
      for (int v = 0; v < V; v += 2)
        *reinterpret_cast<__nv_bfloat162*>(dst + lane * V + v) = __floats2bfloat162_rn(acc[v] * inv, acc[v + 1] * inv);
    } else {
      merge_rows<LPR, V, 256 / D>(live ? e.w : 0, lse_at, row_at, acc, wsum);
      if (live) store_row_part<LPR, V>(dst, sub, acc, wsum == 0.f ? 0.f : 1.f / wsum);
    }
  }
  if (__any_sync(0xffffffffu, marked)) {
    __syncwarp();
    add_to_split_rows<D, FEW>(p, per_row);
  }
  wait_partials();
  if (blockIdx.x >= lookers) return;
  for (int64_t i0 = blockIdx.x; i0 < tiles; i0 += static_cast<int64_t>(lookers) * kMergeThreads) {
    if (i0 != blockIdx.x) mark = mark_of(pair_of(i0 + static_cast<int64_t>(threadIdx.x) * lookers));
    if (__syncthreads_or(mark != 0))
      for (int32_t k = 0; k < kMergeThreads; ++k) add_to_whole_rows<D>(p, i0 + static_cast<int64_t>(k) * lookers, tiles);
  }
}

// The merge of a small narrow call: a unit is kMergeWarps / `per_row` rows (request, kv head, row), of every
// request, `per_row` warps each taking a share of a row's partials.  A row whose request is one piece was written
// directly; to a row of a marked (request, kv head) its first warp adds the values that are not finite.
template <int D, int N>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_small_kernel(const __grid_constant__ TreeParams p,
                                                                         int per_row) {
  constexpr int V = D / 32;
  __shared__ float s_acc[kMergeWarps][32 * V], s_m[kMergeWarps], s_w[kMergeWarps];
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int share = warp % per_row;
  const TreeSmall<N> small(p, kTreeSms * p.sh.per_sm, false);  // (the inputs were complete before the attention kernel
                                                            // let this one launch)
  const int32_t rows = p.hkv * p.ws.part_rows;
  const int32_t flat = static_cast<int32_t>(blockIdx.x) * (kMergeWarps / per_row) + warp / per_row;
  const bool in = flat < p.batch * p.sh.q_tiles * rows;
  const int32_t tile = in ? flat / rows : 0, kh = in ? (flat - tile * rows) / p.ws.part_rows : 0;  // of a request
  const int32_t r = in ? flat - tile * rows - kh * p.ws.part_rows : 0;
  const int32_t P = of_request(small.P, tile), q0 = of_request(small.q0, tile);
  const int32_t n = of_request(small.plan.pieces, tile), first = of_request(small.plan.first, tile);
  const int32_t tok = r / p.group;
  const bool live = in && tok < of_request(small.tokens, tile);
  const int64_t row = static_cast<int64_t>(q0) + tok;
  __nv_bfloat16* dst = p.o + (row * p.hq + kh * p.group + r % p.group) * D;
  const int64_t slot_rows = static_cast<int64_t>(p.hkv) * p.ws.part_rows;  // rows between partial slots
  const int64_t row0 = (static_cast<int64_t>(first) * p.hkv + kh) * p.ws.part_rows + r;
  griddep_wait();
  // marks of the pieces that read drafted tokens: the ones from the prefix's end on
  bool marked = false;
  for (int32_t s = max(0, P / small.plan.chunk); live && s < n; ++s)
    marked = marked || __ldcg(p.ws.bad + static_cast<int64_t>(first + s) * p.hkv + kh) != 0;
  float acc[V], m, wsum;
  merge_partials<V, 8>(
      live && n > 1 ? n : 0, share, per_row, [&](int s) { return __ldcg(p.ws.part_lse + row0 + s * slot_rows); },
      [&](int s, float(&x)[V]) { load_row_cg<V>(p.ws.part_o + (row0 + s * slot_rows) * D + lane * V, x); }, acc, m, wsum);
  if (per_row > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) s_acc[warp][lane * V + v] = acc[v];
    if (lane == 0) s_m[warp] = m, s_w[warp] = wsum;
    __syncthreads();
    if (share == 0) join_shares<V>(per_row, warp, s_acc, s_m, s_w, acc, wsum);
  }
  if (!live || share != 0) return;
  if (n > 1) {
    const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
#pragma unroll
    for (int v = 0; v < V; v += 2)
      *reinterpret_cast<__nv_bfloat162*>(dst + lane * V + v) = __floats2bfloat162_rn(acc[v] * inv, acc[v + 1] * inv);
  }
  if (marked) {
    __syncwarp();
    const int32_t b = tile / p.sh.q_tiles;
    add_odd_values<D>(p, b, (tile - b * p.sh.q_tiles) * p.sh.tokens_per_item + tok, kh * p.group + r % p.group);
  }
}

template <int D, int PASS>
ra_status launch_wide(const TreeParams& p, cudaStream_t s, const DeviceInfo& dev) {
  CUtensorMap qmap, kmap, vmap;
  if (ra_status st = query_tile_map(&qmap, p.q, p.total_q, p.hq, D, p.group)) return st;
  if (ra_status st = row_gather_map(&kmap, p.k_pool, p.num_slots * p.hkv, D)) return st;
  if (ra_status st = row_gather_map(&vmap, p.v_pool, p.num_slots * p.hkv, D)) return st;
  using L = tc::Layout<D, k_stages<D>(), v_stages<D>()>;
  auto kern = attn_tc_kernel<D, k_stages<D>(), v_stages<D>(), PASS>;
  static bool configured[64] = {};
  if (L::kDynSmem > dev.max_smem_optin)
    return fail(RA_ERR_UNSUPPORTED, "tree kernel needs %d bytes of shared memory", L::kDynSmem);
  if (ra_status st = set_smem(kern, L::kDynSmem, configured, dev.device)) return st;
  TcParams tp{};
  tp.k_pool = p.k_pool;
  tp.v_pool = p.v_pool;
  tp.num_slots = p.num_slots;
  tp.hkv = p.hkv;
  tp.q = p.q;
  tp.hq = p.hq;
  tp.group = p.group;
  tp.scale_log2 = p.scale_log2;
  tp.table = p.table;
  tp.table_stride = p.table_stride;
  tp.table_rows = p.table_rows;
  tp.err = p.err;
  tp.total_q = p.total_q;
  tp.o = p.o;
  tp.work_count = p.ws.header;
  tp.work_counter = p.ws.header + 1;
  tp.work_items = p.ws.items;
  tp.tree_chunk = p.ws.header + 2;
  tp.tree_mask = p.mask;
  tp.mask_words = p.mask_words;
  tp.tree_odd = p.ws.bad;
  tp.part_rows = p.ws.part_rows;
  tp.part_o = p.ws.part_o;
  tp.part_lse = p.ws.part_lse;
  const int64_t items = p.ws.cap * p.hkv;
  const int grid = static_cast<int>(items < dev.num_sms ? items : dev.num_sms);
  return launch_pdl("attn_tc_kernel<tree>", kern, dim3(grid), dim3(tc::kThreads), L::kDynSmem, s, tp, qmap, kmap, vmap);
}

// 0: the plan kernel's list; 1 or 2: a small call, of so many query tiles per lane.  (Requests in several narrow
// items only up to 32 of these: 16 x 50..100 tokens of 8/8 heads of 64, 64 items 28.1 us, wide 16.2.)
int tree_small(const TreeShape& sh, int32_t batch, int32_t max_prefix, int32_t max_draft) {
  const int64_t tiles = static_cast<int64_t>(batch) * sh.q_tiles;
  if (!sh.narrow || (sh.q_tiles > 1 && tiles > 32) ||
      !small_call(tiles, static_cast<int64_t>(max_prefix) + max_draft, sh.heads, sh.per_sm))
    return 0;
  return tiles <= 32 ? 1 : 2;
}

ra_status launch_tree(const TreeParams& p, int32_t head_dim, const DeviceInfo& dev, cudaStream_t s) {
  if (const int small = tree_small(p.sh, p.batch, p.max_prefix, p.max_draft)) {
    if (ra_status st = launch_tree_narrow(p, head_dim, small, dev, s)) return st;
    const int64_t rows = static_cast<int64_t>(p.batch) * p.sh.q_tiles * p.hkv * p.ws.part_rows;
    int per_row = 1;
    while (per_row < kMergeWarps && rows * per_row * 2 <= static_cast<int64_t>(dev.num_sms) * 3 * kMergeWarps) per_row *= 2;
    const int64_t ctas = (rows * per_row + kMergeWarps - 1) / kMergeWarps;
    auto kern = head_dim == 128 ? (small == 1 ? tree_merge_small_kernel<128, 1> : tree_merge_small_kernel<128, 2>)
                                : (small == 1 ? tree_merge_small_kernel<64, 1> : tree_merge_small_kernel<64, 2>);
    return launch_pdl("tree_merge_small_kernel", kern, dim3(static_cast<unsigned>(ctas)), dim3(kMergeThreads), 0, s, p, per_row);
  }
  // the list kernel: one CTA for the list, and (wide) one per request, at most the other SMs, for the scan of V
  const int scan = p.sh.narrow ? 0 : p.batch < dev.num_sms - 1 ? p.batch : dev.num_sms - 1;
  if (ra_status st = launch_pdl("tree_plan_kernel", tree_plan_kernel, dim3(1 + scan), dim3(kScanThreads), 0, s, p,
                                head_dim))
    return st;
  if (p.sh.narrow) {
    if (ra_status st = launch_tree_narrow(p, head_dim, 0, dev, s)) return st;
  } else {
    const bool one_tile = p.max_draft * p.group <= tc::kRows;  // every item's rows fit one query tile
    if (ra_status st = head_dim == 128 ? (one_tile ? launch_wide<128, kTreeDualPass>(p, s, dev) : launch_wide<128, kTreePass>(p, s, dev))
                                       : (one_tile ? launch_wide<64, kTreeDualPass>(p, s, dev) : launch_wide<64, kTreePass>(p, s, dev)))
      return st;
  }
  // Persistent.  At most cap_parts / 2 query tiles are split (each into two or more).  With many splits per tile
  // (their number is bounded, so few tiles) several warps share a row: as many as leave each unit's rows enough
  // for the SMs' CTAs.
  const int64_t tiles = std::min<int64_t>(p.ws.cap_parts / 2, static_cast<int64_t>(p.batch) *
                                          ((p.max_draft + p.sh.tokens_per_item - 1) / p.sh.tokens_per_item));
  const int64_t rows = std::max<int64_t>(1, tiles) * p.hkv * p.ws.part_rows;
  const int64_t most = static_cast<int64_t>(dev.num_sms) * 8;
  int per_row = 1;
  while (per_row < kMergeWarps && rows * per_row * 2 <= static_cast<int64_t>(dev.num_sms) * 3 * kMergeWarps) per_row *= 2;
  const int64_t per_cta = per_row > 1 ? kMergeWarps / per_row : kMergeThreads / 8;
  const int64_t want = (rows + per_cta - 1) / per_cta;
  auto kern = per_row > 1 ? (head_dim == 128 ? tree_merge_kernel<128, true> : tree_merge_kernel<64, true>)
                          : (head_dim == 128 ? tree_merge_kernel<128, false> : tree_merge_kernel<64, false>);
  return launch_pdl("tree_merge_kernel", kern, dim3(static_cast<unsigned>(want < most ? want : most)),
                    dim3(kMergeThreads), 0, s, p, per_row);
}

bool tree_args_ok(int32_t batch, int64_t total_q, int32_t hq, int32_t hkv, int32_t d, int32_t max_draft) {
  return batch >= 0 && batch <= 65535 && total_q >= 0 && total_q < (int64_t(1) << 31) && hkv > 0 && hq > 0 &&
         hq % hkv == 0 && 128 % (hq / hkv) == 0 && (d == 64 || d == 128) && max_draft >= 1 && max_draft <= 1024;
}

}  // namespace
}  // namespace ra

extern "C" size_t ra_tree_workspace_bytes(int32_t batch, int64_t total_q, int32_t num_q_heads, int32_t num_kv_heads,
                                          int32_t head_dim, int32_t max_draft_len) {
  if (!ra::tree_args_ok(batch, total_q, num_q_heads, num_kv_heads, head_dim, max_draft_len)) return 0;
  auto bytes = [&](bool tiled) {
    return ra::layout_tree(batch, total_q, num_q_heads, num_kv_heads, head_dim, max_draft_len,
                           ra::tree_shape(num_q_heads, num_kv_heads, head_dim, max_draft_len, tiled), nullptr)
        .total;
  };
  const size_t whole = bytes(false), tiled = ra::tree_tileable(num_q_heads, num_kv_heads, max_draft_len) ? bytes(true) : 0;
  return whole > tiled ? whole : tiled;  // (a call's cut depends on max_prefix_len too)
}

extern "C" ra_status ra_tree_attention(const void* k_pool, const void* v_pool, int64_t num_slots, int32_t num_kv_heads,
                                       int32_t head_dim, const void* q, void* o, int32_t num_q_heads, float sm_scale,
                                       const int32_t* req_to_token, int64_t table_stride, int64_t table_rows,
                                       const int32_t* req_pool_indices, const int32_t* prefix_lens,
                                       const int32_t* draft_lens, const int32_t* qo_indptr, const uint32_t* tree_mask,
                                       int32_t mask_words, int32_t batch, int64_t total_q, int32_t max_draft_len,
                                       int32_t max_prefix_len, void* workspace, size_t workspace_bytes,
                                       uint32_t* device_error, ra_stream_t stream) {
  using namespace ra;
  clear_error();
  RA_REQUIRE(batch >= 0 && batch <= 65535, "batch must be in [0, 65535] (got %d)", batch);
  RA_REQUIRE(total_q >= 0 && total_q < (int64_t(1) << 31), "total_q out of range");
  RA_REQUIRE(num_kv_heads > 0 && num_q_heads > 0, "head counts must be > 0");
  RA_REQUIRE(num_q_heads % num_kv_heads == 0, "num_q_heads (%d) must be a multiple of num_kv_heads (%d)",
             num_q_heads, num_kv_heads);
  RA_REQUIRE(num_slots > 0, "num_slots must be > 0");
  RA_REQUIRE(std::isfinite(sm_scale) && sm_scale > 0.f, "sm_scale must be finite and > 0");
  if (head_dim != 64 && head_dim != 128) return fail(RA_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", head_dim);
  const int32_t group = num_q_heads / num_kv_heads;
  if (128 % group != 0) return fail(RA_ERR_UNSUPPORTED, "GQA group %d must divide 128", group);
  if (batch == 0 || total_q == 0) return RA_OK;
  RA_REQUIRE(max_draft_len >= 1 && max_prefix_len >= 0, "max_draft_len must be >= 1, max_prefix_len >= 0");
  if (max_draft_len > 1024) return fail(RA_ERR_UNSUPPORTED, "max_draft_len %d (supported: up to 1024)", max_draft_len);
  RA_REQUIRE(mask_words >= (max_draft_len + 31) / 32, "mask_words (%d) hold fewer than max_draft_len (%d) bits",
             mask_words, max_draft_len);
  // each request needs prefix_lens[b] + draft_lens[b] <= table_stride (checked per request on the device)
  RA_REQUIRE(table_stride >= max_draft_len && table_stride >= max_prefix_len,
             "table_stride (%lld) narrower than max_draft_len or max_prefix_len", (long long)table_stride);
  RA_REQUIRE(max_prefix_len <= (1 << 30), "max_prefix_len too large");
  RA_REQUIRE(table_rows > 0, "table_rows must be > 0");
  RA_REQUIRE(k_pool && v_pool && q && o && req_to_token && req_pool_indices && prefix_lens && draft_lens &&
                 qo_indptr && tree_mask,
             "null pointer argument");
  RA_REQUIRE(aligned16(k_pool) && aligned16(v_pool) && aligned16(q) && aligned16(o),
             "pools, q and o must be 16-byte aligned");
  RA_REQUIRE(aligned4(req_to_token) && aligned4(req_pool_indices) && aligned4(prefix_lens) && aligned4(draft_lens) &&
                 aligned4(qo_indptr) && aligned4(tree_mask),
             "index arrays and masks must be 4-byte aligned");
  TreeParams p{};
  const size_t need = ra_tree_workspace_bytes(batch, total_q, num_q_heads, num_kv_heads, head_dim, max_draft_len);
  if (!workspace || workspace_bytes < need)
    return fail(RA_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace ? workspace_bytes : 0, need);
  p.sh = tree_shape(num_q_heads, num_kv_heads, head_dim, max_draft_len, false);
  if (tree_tileable(num_q_heads, num_kv_heads, max_draft_len)) {
    const TreeShape tiled = tree_shape(num_q_heads, num_kv_heads, head_dim, max_draft_len, true);
    if (tree_small(tiled, batch, max_prefix_len, max_draft_len)) p.sh = tiled;
  }
  p.ws = layout_tree(batch, total_q, num_q_heads, num_kv_heads, head_dim, max_draft_len, p.sh, workspace);
  RA_REQUIRE(aligned16(workspace), "workspace must be 16-byte aligned");
  RA_REQUIRE(p.ws.cap * num_kv_heads < (int64_t(1) << 31), "too many items for one grid");
  RA_REQUIRE(static_cast<int64_t>(batch) * num_kv_heads < (int64_t(1) << 31), "batch x num_kv_heads too large");
  DeviceInfo dev;
  if (ra_status st = current_device(&dev)) return st;
  p.k_pool = static_cast<const __nv_bfloat16*>(k_pool);
  p.v_pool = static_cast<const __nv_bfloat16*>(v_pool);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.num_slots = num_slots;
  p.table_stride = table_stride;
  p.table_rows = table_rows;
  p.total_q = total_q;
  p.hq = num_q_heads;
  p.hkv = num_kv_heads;
  p.group = group;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.table = req_to_token;
  p.rpi = req_pool_indices;
  p.prefix_lens = prefix_lens;
  p.draft_lens = draft_lens;
  p.qo_indptr = qo_indptr;
  p.mask = tree_mask;
  p.mask_words = mask_words;
  p.batch = batch;
  p.max_draft = max_draft_len;
  p.max_prefix = max_prefix_len;
  p.err = device_error;
  return launch_tree(p, head_dim, dev, reinterpret_cast<cudaStream_t>(stream));
}
