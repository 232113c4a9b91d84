// extend_mod.cu -- ra_extend_attention_mod: attention of new tokens over the cache with changed scores (a cap by a tanh, a
// bias by distance) and masks (a sliding window, documents, a prefix that every row sees), on the tcgen05 kernel of
// ra_extend_attention.
//
// The masks are ranges of keys per row, so they act twice: in the work list, where an item (a query tile of a request) gets
// only the keys that one of its rows sees -- a window of 1024 over a context of 3300 reads a third -- and in the kernel,
// where tiles that lie inside every row's range are exponentiated without looking at it.  The cap itself is nine packed
// instructions per pair of scores (score_mod.cuh) where the softmax warps wait on latencies most of the time: 612 us with
// it, 603 without, 558 for the plain call (8 prompts of 700..1500 tokens over 0..2000 cached, 64/8 heads).
#include <algorithm>

#include "api_common.h"
#include "attn_tc.cuh"
#include "attn_tc_host.h"
#include "score_mod_host.h"

namespace ra {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanBins = 4096;  // key-tile counts above kPlanBins - 1 share the first bin

struct ModWorkspace {
  int32_t* count;
  int32_t* counter;
  int32_t* items;  // [4 * cap]
  int64_t cap;
  size_t total;
};

// Entries are at most sum_b ceil(E_b / tokens_per_cta) <= total_q / tokens_per_cta + batch.
ModWorkspace layout_mod_workspace(int32_t batch, int64_t total_q, int32_t tokens_per_cta, void* base) {
  ModWorkspace w{};
  w.cap = (total_q + tokens_per_cta - 1) / tokens_per_cta + batch;
  w.total = 16 + static_cast<size_t>(w.cap) * 16;
  uint8_t* b = static_cast<uint8_t*>(base);
  w.count = reinterpret_cast<int32_t*>(b);
  w.counter = reinterpret_cast<int32_t*>(b ? b + 4 : nullptr);
  w.items = reinterpret_cast<int32_t*>(b ? b + 16 : nullptr);
  return w;
}

struct PlanArgs {
  const int32_t *extend_lens, *prefix_lens, *qo_indptr;
  int32_t batch, max_extend_len, max_prefix_len;
  int64_t table_stride, total_q;
  int32_t tokens_per_cta;
  const int32_t *first_key, *full_lens;
  int32_t window;
  int32_t *count, *counter, *items;
  int64_t cap;
  uint32_t* err;
};

// One CTA lists the (request, query tile) pairs with their key ranges, most key tiles first (a counting sort).  A warp per
// request: without first_key a lane per query tile, with it the lanes share a tile's tokens.
__global__ void __launch_bounds__(kPlanThreads) extend_mod_plan_kernel(const PlanArgs a) {
  __shared__ int32_t s_bin[kPlanBins];
  __shared__ int32_t s_warp[kPlanThreads / 32];
  griddep_launch();  // the attention kernel may start its launch; it waits for this grid before reading the list
  // (this grid waits for the previous one before its first write, so its completion implies that one's)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kPlanBins; i += kPlanThreads) s_bin[i] = 0;
  __syncthreads();
  // f(b, tile, first key, end of keys) for every query tile of this warp's requests, called by one lane
  auto for_tiles = [&](bool report, auto f) {
    for (int b = warp; b < a.batch; b += kPlanThreads / 32) {
      int32_t E = __ldg(a.extend_lens + b);
      const int32_t P = __ldg(a.prefix_lens + b);
      if (E < 0 || E > a.max_extend_len || P < 0 || P > a.max_prefix_len) {
        if (report && lane == 0) flag_error(a.err, RA_DEVERR_LENGTH);
        E = min(max(E, 0), a.max_extend_len);  // the rows within the bound are still computed
        if (P < 0 || P > a.max_prefix_len) continue;
      }
      if (static_cast<int64_t>(P) + E > a.table_stride) {
        if (report && lane == 0) flag_error(a.err, RA_DEVERR_LENGTH);
        continue;
      }
      const int32_t tiles = (E + a.tokens_per_cta - 1) / a.tokens_per_cta;
      const int32_t full = a.full_lens ? min(__ldg(a.full_lens + b), P + E) : 0;
      const int64_t q0 = __ldg(a.qo_indptr + b);
      // (a request whose rows are not inside o is refused when its items are claimed; its keys are not looked up here)
      const bool look = a.first_key != nullptr && q0 >= 0 && q0 + E <= a.total_q;
      for (int32_t t0 = 0; t0 < tiles; t0 += look ? 1 : 32) {
        const int32_t t = look ? t0 : t0 + lane;
        const int32_t tok0 = t * a.tokens_per_cta, tok1 = min(E, tok0 + a.tokens_per_cta);
        int32_t first = a.window > 0 ? max(P + tok0 - a.window + 1, 0) : 0;
        if (look) {
          int32_t low = INT32_MAX;
          for (int32_t i = tok0 + lane; i < tok1; i += 32) {
            const int32_t w = a.window > 0 ? P + i - a.window + 1 : 0;
            low = min(low, max(w, __ldg(a.first_key + q0 + i)));
          }
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) low = min(low, __shfl_xor_sync(0xffffffffu, low, off));
          first = max(low, 0);
        }
        const int32_t end = max(P + tok1, full);
        // (at least one key, also where no row sees any: their rows are written)
        if (t < tiles && (!look || lane == 0)) f(b, t, min(first, end - 1), end);
      }
    }
  };
  auto bin_of = [](int32_t first, int32_t end) {
    return kPlanBins - 1 - min((end - first + tc::kKeys - 1) / tc::kKeys, kPlanBins - 1);  // bin 0 = longest
  };
  for_tiles(true, [&](int32_t, int32_t, int32_t first, int32_t end) { atomicAdd(&s_bin[bin_of(first, end)], 1); });
  __syncthreads();
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
  const int32_t total = s_warp[kPlanThreads / 32 - 1];
#pragma unroll
  for (int e = 0; e < kPer; ++e) s_bin[threadIdx.x * kPer + e] = base + v[e];
  __syncthreads();
  griddep_wait();  // the previous kernel may be the previous call's, still claiming from this list and counter
  for_tiles(false, [&](int32_t b, int32_t t, int32_t first, int32_t end) {
    const int32_t pos = atomicAdd(&s_bin[bin_of(first, end)], 1);
    if (pos < a.cap) reinterpret_cast<int4*>(a.items)[pos] = make_int4(b, t, first, end);
    else flag_error(a.err, RA_DEVERR_LENGTH);  // extend_lens sum above total_q
  });
  if (threadIdx.x == 0) {
    *a.count = static_cast<int32_t>(static_cast<int64_t>(total) < a.cap ? total : a.cap);
    *a.counter = 0;
  }
}

template <int D, int PASS>
ra_status launch_mod(const TcParams& p, const CUtensorMap& qmap, int64_t entries, cudaStream_t s) {
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
  if (ra_status st = set_smem(kern, L::kDynSmem, configured, dev.device)) return st;
  const int64_t items = entries * p.hkv;
  dim3 grid(static_cast<unsigned>(items < dev.num_sms ? items : dev.num_sms));
  return launch_pdl("attn_tc_kernel<extend, changed scores>", kern, grid, dim3(tc::kThreads), L::kDynSmem, s, p, qmap,
                    kmap, vmap);
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
  const ModWorkspace ws = layout_mod_workspace(batch, total_q, tokens_per_cta, workspace);
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
  p.work_count = ws.count;
  p.work_counter = ws.counter;
  p.work_items = ws.items;
  p.mod = mod;
  const PlanArgs a{extend_lens, prefix_lens, qo_indptr, batch,  max_extend_len, max_prefix_len, table_stride, total_q,
                   tokens_per_cta, first_key, full_lens, window, ws.count,       ws.counter,     ws.items,     ws.cap,
                   device_error};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (ra_status st = launch_pdl("extend_mod_plan_kernel", extend_mod_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a))
    return st;
  // at most sum_b ceil(E_b / tokens_per_cta) entries; CTAs past the listed count return at once
  const int64_t entries = std::min<int64_t>(
      ws.cap, static_cast<int64_t>(batch) * ((max_extend_len + tokens_per_cta - 1) / tokens_per_cta));
  if (mod.cap_in > 0.f)
    return head_dim == 128 ? launch_mod<128, kExtendCapPass>(p, qmap, entries, s)
                           : launch_mod<64, kExtendCapPass>(p, qmap, entries, s);
  return head_dim == 128 ? launch_mod<128, kExtendModPass>(p, qmap, entries, s)
                         : launch_mod<64, kExtendModPass>(p, qmap, entries, s);
}

extern "C" size_t ra_extend_mod_workspace_bytes(int32_t batch, int64_t total_q, int32_t num_q_heads,
                                                int32_t num_kv_heads) {
  if (batch < 0 || total_q < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads) return 0;
  const int32_t group = num_q_heads / num_kv_heads;
  if (128 % group != 0) return 0;
  return ra::layout_mod_workspace(batch, total_q, ra::tc::kTiles * (128 / group), nullptr).total;
}
