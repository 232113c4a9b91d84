// extend_mod.cu -- ra_extend_attention_mod: attention of new tokens over the cache with changed scores (a cap by a tanh, a
// bias by distance) and masks (a sliding window, documents, a prefix that every row sees), on the tcgen05 kernel of
// ra_extend_attention.
//
// The masks are ranges of keys per row, so they act twice: in the work list, where an item (a query tile of a request) gets
// only the keys that one of its rows sees -- a window of 1024 over a context of 3300 reads a third -- and in the kernel,
// where tiles that lie inside every row's range are exponentiated without looking at it.  8 prompts of 700..1500 tokens
// over 0..2000 cached ones, 64/8 heads (425 GFLOP, 223 us of the measured matrix rate): 435 us without a cap (the plain call
// 559: its scores, three times as sharp as a model's at the start of training, send it back to its exact path), 602 with
// one, where the softmax warps issue half of the time and their special function units are busy half of it.
#include <algorithm>

#include "api_common.h"
#include "attn_tc.cuh"
#include "attn_tc_host.h"
#include "score_mod_host.h"
#include "slab_ring.cuh"

namespace ra {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanRun = 4;      // query tiles whose first keys a warp reads at once
constexpr int kPlanLows = 4096;  // query tiles whose first key is kept
constexpr int kPlanBins = 4096;  // key-tile counts above kPlanBins - 1 share the first bin
constexpr int kModSms = 152;     // GB300; a constant, so that the workspace does not depend on the device
constexpr int kSplitItems = 2 * kModSms;  // calls of fewer items (query tiles x kv heads) may split their key ranges, into
                                          // at most so many
constexpr int kUncutTiles = 4;
constexpr int kMergeThreads = 256;

struct ModWorkspace {
  int32_t* header;  // [8]: items listed, claim counter, query tiles split
  int32_t* items;   // [4 * cap]: request, query tile, first key, end of keys
  int32_t* slots;   // [cap]: partial slot, or -1
  int32_t* merges;  // [4 * cap_parts]: request, query tile, first partial slot, pieces
  float* part_lse;  // [cap_parts, hkv, part_rows]
  float* part_o;    // [cap_parts, hkv, part_rows, D]
  int64_t cap, cap_parts;
  int32_t part_rows;
  size_t total;
};

// Entries are at most sum_b ceil(E_b / tokens_per_cta) <= total_q / tokens_per_cta + batch; at least total_q /
// tokens_per_cta of them (in a call that fills its rows), so that calls of many tokens need no partials.
ModWorkspace layout_mod_workspace(int32_t batch, int64_t total_q, int32_t tokens_per_cta, int32_t group, int32_t hkv,
                                  void* base) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  ModWorkspace w{};
  const int64_t least = total_q / tokens_per_cta;
  w.cap_parts = least * hkv < kSplitItems ? kSplitItems / hkv : 0;
  w.cap = (total_q + tokens_per_cta - 1) / tokens_per_cta + batch + w.cap_parts;
  w.part_rows = static_cast<int32_t>((total_q < tokens_per_cta ? total_q : tokens_per_cta) * group);
  uint8_t* b = workspace_base(base);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* at = b ? b + off : nullptr;
    off += up(bytes);
    return at;
  };
  w.header = reinterpret_cast<int32_t*>(take(32));
  w.items = reinterpret_cast<int32_t*>(take(static_cast<size_t>(w.cap) * 16));
  w.slots = reinterpret_cast<int32_t*>(take(static_cast<size_t>(w.cap) * 4));
  w.merges = reinterpret_cast<int32_t*>(take(static_cast<size_t>(w.cap_parts) * 16));
  const size_t rows = static_cast<size_t>(w.cap_parts) * hkv * w.part_rows;
  w.part_lse = reinterpret_cast<float*>(take(rows * 4));
  w.part_o = reinterpret_cast<float*>(take(rows * 128 * 4));
  w.total = off + kWorkspaceSlack;
  return w;
}

struct PlanArgs {
  const int32_t *extend_lens, *prefix_lens, *qo_indptr;
  int32_t batch, max_extend_len, max_prefix_len;
  int64_t table_stride, total_q;
  int32_t tokens_per_cta;
  const int32_t *first_key, *full_lens;
  int32_t window;
  int32_t hkv;
  ModWorkspace ws;
  uint32_t* err;
};

// One CTA lists the (request, query tile) pairs with their key ranges, most key tiles first (a counting sort), in two
// passes: the lengths of the ranges, then the list.  Without first_key a warp takes a request and its lanes the query tiles.
// With it (DOCS) a lane takes a query tile, too, its warp reads the tiles' tokens together, four tiles in flight, and the
// second pass finds the first pass's answers in shared memory.  (A warp per request there too, tile after tile, was 70 us of
// an 81 us call of 7 requests of up to 1,749 tokens in documents of 129, 8/1 heads: now 13 of 31; 4 prompts of 2,000..4,095
// tokens in documents of 611, 16/16 heads of 64, 96 -> 74.)  Two kernels: one for both cost the calls without first_key 1 to
// 2 us of instruction fetches.
template <bool DOCS>
__global__ void __launch_bounds__(kPlanThreads) extend_mod_plan_kernel(const PlanArgs a) {
  __shared__ int32_t s_bin[kPlanBins];
  __shared__ int32_t s_low[DOCS ? kPlanLows : 1];  // the first keys of query tiles
  __shared__ int32_t s_warp[kPlanWarps], s_cost[kPlanWarps], s_chunk[kPlanWarps], s_nt[kSplitItems];
  __shared__ int32_t s_entries, s_longest, s_parts, s_merges;
  griddep_launch();  // the attention kernel may start its launch; it waits for this grid before reading the list
  // (this grid waits for the previous one before its first write, so its completion implies that one's; the call's inputs
  // that it reads before, it reads through L2: kernels that write lengths let this one launch behind their fenced writes)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kPlanBins; i += kPlanThreads) s_bin[i] = 0;
  if (threadIdx.x == 0) s_entries = s_longest = s_parts = s_merges = 0;
  __syncthreads();
  // the lengths of request b; false: nothing of it can be listed
  auto lengths = [&](int32_t b, bool report, int32_t& E, int32_t& P, int32_t& full) -> bool {
    E = __ldcg(a.extend_lens + b);
    P = __ldcg(a.prefix_lens + b);
    full = a.full_lens ? __ldcg(a.full_lens + b) : 0;
    bool bad = E < 0 || E > a.max_extend_len, skip = P < 0 || P > a.max_prefix_len;
    E = min(max(E, 0), a.max_extend_len);  // the rows within the bound are still computed
    if (!skip && static_cast<int64_t>(P) + E > a.table_stride) skip = true;
    if ((bad || skip) && report) flag_error(a.err, RA_DEVERR_LENGTH);
    full = min(full, P + E);
    return !skip;
  };
  // f(b, tile, first key, end of keys) for every query tile of this warp, called by one lane; at least one key, also where no
  // row sees any: their rows are written
  auto for_tiles = [&](bool list, auto f) {
    if constexpr (!DOCS) {
      for (int32_t b = warp; b < a.batch; b += kPlanWarps) {
        int32_t E, P, full;
        if (!lengths(b, !list && lane == 0, E, P, full)) continue;
        const int32_t tiles = (E + a.tokens_per_cta - 1) / a.tokens_per_cta;
        for (int32_t t = lane; t < tiles; t += 32) {
          const int32_t tok0 = t * a.tokens_per_cta, end = max(P + min(E, tok0 + a.tokens_per_cta), full);
          const int32_t first = a.window > 0 ? max(P + tok0 - a.window + 1, 0) : 0;
          f(b, t, min(first, end - 1), end);
        }
      }
    } else {
      // 32 requests at a time, a lane reading each one's lengths, their query tiles numbered by a scan.  The groups of
      // requests have equal shares of the warps and of s_low.
      const int32_t groups = (a.batch + 31) / 32, share = max(1, kPlanWarps / groups), lows = kPlanLows / groups;
      for (int32_t gr = warp / share; gr < groups; gr += kPlanWarps / share) {
        const int32_t b0 = gr * 32;
        int32_t E = 0, P = 0, full = 0, tiles = 0;
        int64_t q0 = -1;
        if (b0 + lane < a.batch) {
          q0 = __ldcg(a.qo_indptr + b0 + lane);
          const bool listed = lengths(b0 + lane, !list && warp % share == 0, E, P, full);
          // (a request of more rows than o has is refused when its items are claimed)
          E = listed ? static_cast<int32_t>(min(static_cast<int64_t>(E), a.total_q)) : 0;
          tiles = (E + a.tokens_per_cta - 1) / a.tokens_per_cta;
        }
        int32_t incl = tiles;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int32_t y = __shfl_up_sync(0xffffffffu, incl, off);
          if (lane >= off) incl += y;
        }
        const int32_t count = __shfl_sync(0xffffffffu, incl, 31);
        for (int32_t v = warp % share; v < count; v += share * 32) {
          const int32_t u = v + lane * share;  // this lane's query tile
          int32_t at = 0;  // its request's lane: those before it end at or before u
#pragma unroll
          for (int step = 16; step > 0; step >>= 1)
            if (__shfl_sync(0xffffffffu, incl, at + step - 1) <= u) at += step;
          const int32_t Eb = __shfl_sync(0xffffffffu, E, at), Pb = __shfl_sync(0xffffffffu, P, at);
          const int64_t qb = __shfl_sync(0xffffffffu, q0, at);
          const int32_t end_all = __shfl_sync(0xffffffffu, full, at);
          const int32_t t = u - __shfl_sync(0xffffffffu, incl - tiles, at);
          const bool live = u < count;
          const int32_t tok0 = live ? t * a.tokens_per_cta : 0, tok1 = live ? min(Eb, tok0 + a.tokens_per_cta) : 0;
          const bool known = list && u < lows;
          int32_t low = live && known ? s_low[gr * lows + u] : 0;
          if (__any_sync(0xffffffffu, live && !known)) {  // (for the whole warp: its lanes work together)
            // (rows not inside o: the request is refused when its items are claimed, its keys are not looked up)
            const int32_t n = live && !known && qb >= 0 && qb + Eb <= a.total_q ? tok1 - tok0 : 0;
            // the tile's tokens, a lane each, their first keys of kPlanRun tiles in flight at once
            for (int32_t i0 = 0; i0 < 32 && v + i0 * share < count; i0 += kPlanRun) {
              int32_t first[kPlanRun];
#pragma unroll
              for (int e = 0; e < kPlanRun; ++e) first[e] = INT32_MAX;
              const int32_t most = __reduce_max_sync(0xffffffffu, lane >= i0 && lane < i0 + kPlanRun ? n : 0);
              for (int32_t i = lane; i < most + lane; i += 32) {
                int32_t x[kPlanRun];
#pragma unroll
                for (int e = 0; e < kPlanRun; ++e) {
                  const int32_t ne = __shfl_sync(0xffffffffu, n, i0 + e);
                  const int64_t row = __shfl_sync(0xffffffffu, qb + tok0, i0 + e);
                  x[e] = i < ne ? __ldcg(a.first_key + row + i) : INT32_MAX;
                }
#pragma unroll
                for (int e = 0; e < kPlanRun; ++e) {
                  const int32_t p0 = __shfl_sync(0xffffffffu, Pb + tok0, i0 + e);
                  if (a.window > 0 && x[e] < INT32_MAX) x[e] = max(x[e], p0 + i - a.window + 1);
                  first[e] = min(first[e], x[e]);
                }
              }
#pragma unroll
              for (int e = 0; e < kPlanRun; ++e) {
                const int32_t y = __reduce_min_sync(0xffffffffu, first[e]);
                if (lane == i0 + e && n > 0) low = y;
              }
            }
            low = max(low, 0);
            if (live && !known && u < lows) s_low[gr * lows + u] = low;
          }
          const int32_t end = max(Pb + tok1, end_all);
          if (live) f(b0 + at, t, min(low, end - 1), end);
        }
      }
    }
  };
  auto tiles_of = [](int32_t first, int32_t end) { return (end - first + tc::kKeys - 1) / tc::kKeys; };
  auto bin_of = [](int32_t tiles) { return kPlanBins - 1 - min(tiles, kPlanBins - 1); };  // bin 0 = longest
  for_tiles(false, [&](int32_t, int32_t, int32_t first, int32_t end) {
    const int32_t nt = tiles_of(first, end), at = atomicAdd(&s_entries, 1);
    if (at < kSplitItems) s_nt[at] = nt;
    atomicMax(&s_longest, nt);
    atomicAdd(&s_bin[bin_of(nt)], 1);
  });
  __syncthreads();
  // Few items leave SMs idle (an item's tiles are one chain of products and softmax, 3 us each, and no second item hides
  // it): their key ranges are cut into pieces of `chunk` tiles, the partial results joined by a kernel of their own.  Each
  // warp weighs one number of pieces of the longest range: rounds of pieces over the SMs, a piece costing its tiles and
  // about 3 more, and the join about 1 (over 80 calls of 1..8 requests the geometric mean is 35.4 us with 1, 35.6 with 3,
  // 37.0 with 5).
  const int32_t entries = s_entries, longest = s_longest;
  int32_t chunk = longest;
  if (a.ws.cap_parts > 0 && static_cast<int64_t>(entries) * a.hkv < kSplitItems) {
    const int32_t c = max(1, (longest + warp) / (warp + 1));
    int32_t pieces = 0;
    for (int32_t i = lane; i < entries; i += 32) pieces += (s_nt[i] + c - 1) / c;
    pieces = __reduce_add_sync(0xffffffffu, pieces);
    const int32_t rounds = (pieces * a.hkv + kModSms - 1) / kModSms;
    if (lane == 0) {
      s_cost[warp] = c >= longest ? rounds * (longest + 3) : pieces > a.ws.cap_parts ? INT32_MAX : rounds * (c + 3) + 1;
      s_chunk[warp] = c;
    }
    __syncthreads();
    int32_t best = INT32_MAX;
    for (int w = 0; w < kPlanWarps; ++w)
      if (s_cost[w] < best) best = s_cost[w], chunk = s_chunk[w];  // (on a tie the longer piece)
    if (chunk < longest) {  // the pieces' bins (few entries: all in s_nt)
      for (int i = threadIdx.x; i < kPlanBins; i += kPlanThreads) s_bin[i] = 0;
      __syncthreads();
      for (int32_t i = threadIdx.x; i < entries; i += kPlanThreads) {
        const int32_t full = s_nt[i] / chunk, rest = s_nt[i] - full * chunk;
        if (full > 0) atomicAdd(&s_bin[bin_of(chunk)], full);
        if (rest > 0) atomicAdd(&s_bin[bin_of(rest)], 1);
      }
      __syncthreads();
    }
  }
  // exclusive scan of the bins: thread i owns bins [4i, 4i + 4)
  constexpr int kPer = kPlanBins / kPlanThreads;
  int32_t v[kPer], run = 0;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    v[e] = run;
    run += s_bin[threadIdx.x * kPer + e];
  }
  int32_t incl = run;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int32_t w = s_warp[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += y;
    }
    s_warp[lane] = w;  // inclusive over warps
  }
  __syncthreads();
  const int32_t base = (warp > 0 ? s_warp[warp - 1] : 0) + incl - run;
  const int32_t total = s_warp[kPlanWarps - 1];
#pragma unroll
  for (int e = 0; e < kPer; ++e) s_bin[threadIdx.x * kPer + e] = base + v[e];
  __syncthreads();
  griddep_wait();  // the previous kernel may be the previous call's, still claiming from this list and counter
  for_tiles(true, [&](int32_t b, int32_t t, int32_t first, int32_t end) {
    const int32_t nt = tiles_of(first, end), pieces = (nt + chunk - 1) / chunk;
    int32_t slot = -1;
    if (pieces > 1) {
      slot = atomicAdd(&s_parts, pieces);
      reinterpret_cast<int4*>(a.ws.merges)[atomicAdd(&s_merges, 1)] = make_int4(b, t, slot, pieces);
    }
    for (int32_t s = 0; s < pieces; ++s) {
      const int32_t n = min(chunk, nt - s * chunk), pos = atomicAdd(&s_bin[bin_of(n)], 1);
      if (pos < a.ws.cap) {
        const int32_t k0 = first + s * chunk * tc::kKeys;
        reinterpret_cast<int4*>(a.ws.items)[pos] = make_int4(b, t, k0, s + 1 < pieces ? k0 + chunk * tc::kKeys : end);
        a.ws.slots[pos] = slot < 0 ? -1 : slot + s;
      } else {
        flag_error(a.err, RA_DEVERR_LENGTH);  // extend_lens sum above total_q
      }
    }
  });
  __syncthreads();
  if (threadIdx.x == 0) {
    a.ws.header[0] = static_cast<int32_t>(static_cast<int64_t>(total) < a.ws.cap ? total : a.ws.cap);
    a.ws.header[1] = 0;
    a.ws.header[2] = s_merges;
  }
}

// Join the pieces of split query tiles: o = sum_s 2^(lse_s - M) o_s / sum_s 2^(lse_s - M), 8 lanes per row.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) extend_mod_merge_kernel(const __grid_constant__ TcParams p,
                                                                         const ModWorkspace ws) {
  constexpr int LPR = 8, V = D / LPR;
  griddep_launch();
  // (the list was complete before the attention kernel let this one launch; the partials are once that is)
  const int sub = threadIdx.x % LPR, T = 2 * (tc::kRows / p.group);
  const int32_t tile_rows = p.hkv * ws.part_rows, per_cta = kMergeThreads / LPR;
  const int32_t chunks = (tile_rows + per_cta - 1) / per_cta;
  const int64_t units = static_cast<int64_t>(__ldcg(ws.header + 2)) * chunks;
  griddep_wait();
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int4 e = __ldcg(reinterpret_cast<const int4*>(ws.merges) + u / chunks);
    const int32_t flat = static_cast<int32_t>(u % chunks) * per_cta + static_cast<int32_t>(threadIdx.x) / LPR;
    const int32_t kh = flat / ws.part_rows, r = flat - kh * ws.part_rows;
    const int32_t tok = e.y * T + r / p.group;
    const int32_t E = min(max(__ldg(p.extend_lens + e.x), 0), p.max_extend_len);
    const int64_t first = __ldg(p.qo_indptr + e.x);
    const int32_t table_row = __ldg(p.rpi + e.x);
    // (a request whose rows or table row are out of range wrote no partials)
    const bool live = flat < tile_rows && tok < E && first >= 0 && first + E <= p.total_q && table_row >= 0 &&
                      table_row < p.table_rows;
    const int64_t step = static_cast<int64_t>(p.hkv) * ws.part_rows;  // rows between slots
    const int64_t row0 = (static_cast<int64_t>(e.z) * p.hkv + kh) * ws.part_rows + r;
    float acc[V], sum;
    merge_rows<LPR, V, 256 / D>(
        live ? e.w : 0, [&](int s) { return __ldcg(ws.part_lse + row0 + s * step); },
        [&](int s, float(&x)[V]) { load_row_part<LPR, V>(ws.part_o + (row0 + s * step) * D, sub, x); }, acc, sum);
    if (live)
      store_row_part<LPR, V>(p.o + ((first + tok) * p.hq + kh * p.group + r % p.group) * D, sub, acc,
                             sum == 0.f ? 0.f : 1.f / sum);
  }
}

template <int D, int PASS>
ra_status launch_mod(const TcParams& p, const ModWorkspace& ws, const CUtensorMap& qmap, int64_t entries, cudaStream_t s) {
  CUtensorMap kmap, vmap;
  if (ra_status st = row_gather_map(&kmap, p.k_pool, p.num_slots * p.hkv, D)) return st;
  if (ra_status st = row_gather_map(&vmap, p.v_pool, p.num_slots * p.hkv, D)) return st;
  using L = tc::Layout<D, k_stages<D>(), v_stages<D>()>;
  auto kern = attn_tc_kernel<D, k_stages<D>(), v_stages<D>(), PASS>;
  static bool configured[64] = {};
  DeviceInfo dev;
  if (ra_status st = current_device(&dev)) return st;
  if (L::kDynSmem > dev.max_smem_optin)
    return fail(RA_ERR_UNSUPPORTED, "extend kernel needs %d bytes of shared memory", L::kDynSmem);
  if (ra_status st = set_smem<PASS>(kern, L::kDynSmem, configured, dev.device)) return st;
  const int64_t items = (entries + ws.cap_parts) * p.hkv;
  dim3 grid(static_cast<unsigned>(items < dev.num_sms ? items : dev.num_sms));
  if (ra_status st = launch_pdl("attn_tc_kernel<extend, changed scores>", kern, grid, dim3(tc::Roles<PASS>::kThreads), L::kDynSmem, s,
                                p, qmap, kmap, vmap))
    return st;
  if (ws.cap_parts == 0) return RA_OK;
  // (at most cap_parts / 2 query tiles are split, each into two pieces or more)
  const int64_t rows = std::max<int64_t>(1, std::min(entries, ws.cap_parts / 2)) * p.hkv * ws.part_rows;
  const int64_t want = (rows + kMergeThreads / 8 - 1) / (kMergeThreads / 8), most = static_cast<int64_t>(dev.num_sms) * 8;
  return launch_pdl("extend_mod_merge_kernel", extend_mod_merge_kernel<D>,
                    dim3(static_cast<unsigned>(want < most ? want : most)), dim3(kMergeThreads), 0, s, p, ws);
}

}  // namespace
}  // namespace ra

extern "C" ra_status ra_extend_attention_mod(
    const void* k_pool, const void* v_pool, int64_t num_slots, int32_t num_kv_heads, int32_t head_dim, const void* q, void* o,
    int32_t num_q_heads, float sm_scale, float score_cap, int32_t window, const float* slopes, const int32_t* first_key,
    const int32_t* full_lens, const int32_t* req_to_token, int64_t table_stride, int64_t table_rows,
    const int32_t* req_pool_indices, const int32_t* prefix_lens, const int32_t* extend_lens, const int32_t* qo_indptr,
    int32_t batch, int64_t total_q, int32_t max_extend_len, int32_t max_prefix_len, void* workspace, size_t workspace_bytes,
    uint32_t* device_error, ra_stream_t stream) {
  using namespace ra;
  clear_error();
  RA_REQUIRE(batch >= 0 && batch <= 65535, "batch must be in [0, 65535] (got %d)", batch);
  RA_REQUIRE(total_q >= 0 && total_q < (int64_t(1) << 31), "total_q out of range");
  RA_REQUIRE(num_kv_heads > 0 && num_q_heads > 0, "head counts must be > 0");
  RA_REQUIRE(num_q_heads % num_kv_heads == 0, "num_q_heads (%d) must be a multiple of num_kv_heads (%d)", num_q_heads,
             num_kv_heads);
  RA_REQUIRE(num_slots > 0, "num_slots must be > 0");
  ScoreMod mod{};
  if (ra_status st = score_mod(&mod, sm_scale, score_cap, window, slopes, first_key, full_lens)) return st;
  if (head_dim != 64 && head_dim != 128) return fail(RA_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", head_dim);
  const int32_t group = num_q_heads / num_kv_heads;
  if (128 % group != 0) return fail(RA_ERR_UNSUPPORTED, "GQA group %d must divide 128", group);
  if (batch == 0 || total_q == 0) return RA_OK;
  RA_REQUIRE(max_extend_len >= 1 && max_prefix_len >= 0, "max_extend_len must be >= 1, max_prefix_len >= 0");
  RA_REQUIRE(table_stride >= max_extend_len && table_stride > max_prefix_len,
             "table_stride (%lld) narrower than max_extend_len or max_prefix_len + 1", (long long)table_stride);
  RA_REQUIRE(table_rows > 0, "table_rows must be > 0");
  RA_REQUIRE(k_pool && v_pool && q && o && req_to_token && req_pool_indices && prefix_lens && extend_lens && qo_indptr,
             "null pointer argument");
  RA_REQUIRE(aligned16(k_pool) && aligned16(v_pool) && aligned16(q) && aligned16(o),
             "pools, q and o must be 16-byte aligned");
  RA_REQUIRE(aligned4(req_to_token) && aligned4(req_pool_indices) && aligned4(prefix_lens) && aligned4(extend_lens) &&
                 aligned4(qo_indptr),
             "index arrays must be 4-byte aligned");
  const int tokens_per_cta = tc::kTiles * (128 / group);
  ModWorkspace ws = layout_mod_workspace(batch, total_q, tokens_per_cta, group, num_kv_heads, workspace);
  if (!workspace || workspace_bytes < ws.total)
    return fail(RA_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace ? workspace_bytes : 0, ws.total);
  RA_REQUIRE(aligned16(workspace), "workspace must be 16-byte aligned");
  RA_REQUIRE(ws.cap * num_kv_heads < (int64_t(1) << 31), "too many extend tiles for one grid");

  CUtensorMap qmap;
  if (ra_status st = query_tile_map(&qmap, q, total_q, num_q_heads, head_dim, group)) return st;

  TcParams p{};
  p.k_pool = static_cast<const __nv_bfloat16*>(k_pool);
  p.v_pool = static_cast<const __nv_bfloat16*>(v_pool);
  p.num_slots = num_slots;
  p.hkv = num_kv_heads;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.hq = num_q_heads;
  p.group = group;
  p.scale_log2 = sm_scale * kLog2e;
  p.table = req_to_token;
  p.table_stride = table_stride;
  p.table_rows = table_rows;
  p.err = device_error;
  p.rpi = req_pool_indices;
  p.prefix_lens = prefix_lens;
  p.extend_lens = extend_lens;
  p.qo_indptr = qo_indptr;
  p.max_extend_len = max_extend_len;
  p.max_prefix_len = max_prefix_len;
  p.total_q = total_q;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.work_count = ws.header;
  p.work_counter = ws.header + 1;
  p.work_items = ws.items;
  p.work_slots = ws.slots;
  p.part_rows = ws.part_rows;
  p.part_o = ws.part_o;
  p.part_lse = ws.part_lse;
  p.mod = mod;
  // at most sum_b ceil(E_b / tokens_per_cta) entries; CTAs past the listed count return at once
  const int64_t entries = std::min<int64_t>(
      ws.cap - ws.cap_parts, static_cast<int64_t>(batch) * ((max_extend_len + tokens_per_cta - 1) / tokens_per_cta));
  // Ranges that the bounds hold to four key tiles are not worth cutting, and the join's launch is saved: 4 requests of 30..60
  // tokens over 100 keys, 16/16 heads of 64, 12.7 -> 10.4 us; 8 of 150..300 over 200, 32/8 heads, 38.8 -> 34.5.
  int64_t range = static_cast<int64_t>(max_prefix_len) + max_extend_len;
  if (window > 0 && !full_lens) range = std::min<int64_t>(range, static_cast<int64_t>(window) + tokens_per_cta - 1);
  if (range <= kUncutTiles * tc::kKeys) ws.cap_parts = 0;
  const PlanArgs a{extend_lens, prefix_lens, qo_indptr, batch,  max_extend_len, max_prefix_len, table_stride, total_q,
                   tokens_per_cta, first_key, full_lens, window, num_kv_heads,   ws,             device_error};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (ra_status st = launch_pdl("extend_mod_plan_kernel",
                                first_key ? extend_mod_plan_kernel<true> : extend_mod_plan_kernel<false>, dim3(1),
                                dim3(kPlanThreads), 0, s, a))
    return st;
  if (mod.cap_in > 0.f && mod.cap_log2 <= kCapFixed)
    return head_dim == 128 ? launch_mod<128, kExtendFixedPass>(p, ws, qmap, entries, s)
                           : launch_mod<64, kExtendFixedPass>(p, ws, qmap, entries, s);
  if (mod.cap_in > 0.f)
    return head_dim == 128 ? launch_mod<128, kExtendCapPass>(p, ws, qmap, entries, s)
                           : launch_mod<64, kExtendCapPass>(p, ws, qmap, entries, s);
  return head_dim == 128 ? launch_mod<128, kExtendModPass>(p, ws, qmap, entries, s)
                         : launch_mod<64, kExtendModPass>(p, ws, qmap, entries, s);
}

extern "C" size_t ra_extend_mod_workspace_bytes(int32_t batch, int64_t total_q, int32_t num_q_heads,
                                                int32_t num_kv_heads) {
  if (batch < 0 || total_q < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads) return 0;
  const int32_t group = num_q_heads / num_kv_heads;
  if (128 % group != 0) return 0;
  return ra::layout_mod_workspace(batch, total_q, ra::tc::kTiles * (128 / group), group, num_kv_heads, nullptr).total;
}
