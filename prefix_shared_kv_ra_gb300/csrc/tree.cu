// tree.cu -- ra_tree_attention: drafted tokens of a tree over a cached prefix.
//
// Each request has T drafted tokens whose K/V sit in the pool behind its P cached ones; drafted token i
// attends to all of the prefix and to the drafted tokens its bit mask names:
//   o_i = sum_j softmax_j(scale <q_i, k_j>) v_j   over j < P and over P + t with bit t of mask_i.
// One pass of the tcgen05 attention kernel (attn_tc.cuh, kTreePass) does both parts: rows are (token, head
// of the GQA group), up to 256 per item, each gathered 128-key tile feeding all of them, and only the tiles
// that hold drafted tokens look at the masks.  T * G rows share every key, so wide trees are bound by the
// tensor cores and the softmax's issue slots like extend, small ones by latency and the gathers:
//  * the work list (one CTA, on the device, from the real lengths) splits the key ranges only as far as the
//    SMs need it, since an unsplit item writes its bf16 rows directly while a split one costs fp32 partials
//    (4 * D + 4 bytes per row and split, written and read again) and a merge;
//  * a persistent merge kernel joins the splits; with nothing split it only looks at a count.
// A value of V that is not finite must not reach rows whose mask leaves its token out, but a matrix product
// multiplies it by their zero probability (0 * inf = NaN).  The list kernel's other CTAs therefore scan the
// drafted tokens' V (at most a few MB) and mark the (request, kv head) pairs that hold one; the merge kernel
// recomputes those rows key by key, skipping what is masked.  Prefix keys are seen by every row: there the
// product's NaN is the answer.
#include <cmath>

#include "api_common.h"
#include "attn_tc.cuh"
#include "attn_tc_host.h"
#include "decode_internal.h"

namespace ra {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBins = 1024;        // key tiles of an item, longest first; longer ones share the first bin
constexpr int kPlanSms = 152;      // GB300; a constant, so that the workspace does not depend on the device
constexpr int kWaves = 2;          // a batch with at least this many unsplit items per SM is only balanced
constexpr int kMergeThreads = 256;
constexpr int kMergeRows = kMergeThreads / 32;  // rows per merge unit, one warp each

struct TreeWorkspace {
  int32_t* header;     // [8]: listed items, claim counter, keys per split, merges
  int32_t* items;      // [4 * cap]
  int32_t* merges;     // [4 * cap_merge]: request, query tile, first partial slot, splits
  int32_t* bad;        // [batch * hkv]: a drafted token's V holds a value that is not finite
  float* part_o;
  float* part_lse;
  int64_t cap, cap_parts;
  int32_t part_rows;
  size_t total;
};

// Items: one per (request, query tile) plus the extra ones of split ranges.  A range is split only if it is
// longer than the chunk, and the chunk is at least total / (kWaves * kPlanSms) (all ranges times the kv heads):
// the split ranges' pieces number at most sum ceil(n / c) <= sum 2 n / c <= 2 * kWaves * kPlanSms / hkv.
TreeWorkspace layout_tree(int32_t batch, int64_t total_q, int32_t hq, int32_t hkv, int32_t d, int32_t max_draft,
                          void* base) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const int32_t group = hq / hkv;
  const int32_t tokens = tc::kTiles * (128 / group);
  TreeWorkspace w{};
  w.cap_parts = 2 * kWaves * kPlanSms / hkv;
  w.cap = (total_q + tokens - 1) / tokens + batch + w.cap_parts;
  const int64_t rows = static_cast<int64_t>(max_draft) * group;
  w.part_rows = static_cast<int32_t>(rows < 256 ? rows : 256);
  uint8_t* b = static_cast<uint8_t*>(base);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* at = b ? b + off : nullptr;
    off += up(bytes);
    return at;
  };
  w.header = reinterpret_cast<int32_t*>(take(32));
  w.items = reinterpret_cast<int32_t*>(take(static_cast<size_t>(w.cap) * 16));
  w.merges = reinterpret_cast<int32_t*>(take(static_cast<size_t>(w.cap_parts) * 16));
  w.bad = reinterpret_cast<int32_t*>(take(static_cast<size_t>(batch) * hkv * 4));
  const size_t part = static_cast<size_t>(w.cap_parts) * hkv * w.part_rows;
  w.part_lse = reinterpret_cast<float*>(take(part * 4));
  w.part_o = reinterpret_cast<float*>(take(part * d * 4));
  w.total = off;
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
  int32_t tokens_per_item;
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

__device__ __forceinline__ int32_t tiles_of(int32_t keys) { return (keys + tc::kKeys - 1) / tc::kKeys; }
__device__ __forceinline__ int32_t bin_of(int32_t tiles) { return kBins - 1 - min(tiles, kBins - 1); }

// CTA 0 lists the items, longest first; CTAs 1.. scan the drafted tokens' V rows, one request at a time.
__global__ void __launch_bounds__(kPlanThreads) tree_plan_kernel(const __grid_constant__ TreeParams p, int32_t head_dim) {
  griddep_wait();  // the call's inputs; the workspace may still be read by the call before
  griddep_launch();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (blockIdx.x > 0) {
    for (int32_t b = blockIdx.x - 1; b < p.batch; b += gridDim.x - 1) {
      for (int32_t h = t; h < p.hkv; h += kPlanThreads) p.ws.bad[b * p.hkv + h] = 0;
      __syncthreads();
      int32_t P, T;
      if (!tree_request(p, b, P, T, false)) continue;
      const int32_t* slots = p.table + static_cast<int64_t>(__ldg(p.rpi + b)) * p.table_stride + P;
      const int32_t vecs = p.hkv * head_dim / 8, per_head = head_dim / 8;
      for (int32_t j = warp; j < T; j += kPlanThreads / 32) {
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
  __shared__ int32_t s_bin[kBins];
  __shared__ int32_t s_warp[kPlanThreads / 32];
  __shared__ unsigned long long s_work, s_entries, s_best;
  __shared__ int32_t s_longest, s_parts, s_merges;
  s_bin[t] = 0;
  if (t == 0) {
    s_work = s_entries = 0;
    s_best = ~0ull;
    s_longest = 1;
    s_parts = s_merges = 0;
  }
  __syncthreads();
  const int32_t per_item = p.tokens_per_item;
  unsigned long long work = 0, entries = 0;
  int32_t longest = 0;
  for (int32_t b = t; b < p.batch; b += kPlanThreads) {
    int32_t P, T;
    if (!tree_request(p, b, P, T, true)) continue;
    const int32_t q_tiles = (T + per_item - 1) / per_item, nt = tiles_of(P + T);
    work += static_cast<unsigned long long>(q_tiles) * nt;
    entries += q_tiles;
    longest = max(longest, nt);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    work += __shfl_xor_sync(0xffffffffu, work, off);
    entries += __shfl_xor_sync(0xffffffffu, entries, off);
    longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, off));
  }
  if (lane == 0) {
    atomicAdd(&s_work, work);
    atomicAdd(&s_entries, entries);
    atomicMax(&s_longest, longest);
  }
  __syncthreads();
  // Key tiles per split.  The least is total / (kWaves * kPlanSms), which bounds the partials.  With that
  // many unsplit items it also balances the SMs; with fewer, the split of the longest range into 1 .. 1024
  // pieces that gives the shortest schedule, waves * (tiles + 3) (a CTA fills and drains in ~3 tiles' time).
  const unsigned long long all = s_work * p.hkv;
  const unsigned long long per_sm = (all + kWaves * kPlanSms - 1) / (kWaves * kPlanSms);
  const int32_t least = static_cast<int32_t>(min(per_sm, static_cast<unsigned long long>(s_longest)));
  int32_t chunk = max(least, 1);
  if (s_entries * p.hkv < kWaves * kPlanSms) {
    const int32_t c = max((s_longest + t) / (t + 1), chunk);
    unsigned long long items = 0;
    for (int32_t b = 0; b < p.batch; ++b) {
      int32_t P, T;
      if (!tree_request(p, b, P, T, false)) continue;
      items += static_cast<unsigned long long>((T + per_item - 1) / per_item) * ((tiles_of(P + T) + c - 1) / c);
    }
    const unsigned long long waves = (items * p.hkv + kPlanSms - 1) / kPlanSms;
    atomicMin(&s_best, (waves * (c + 3)) << 32 | static_cast<unsigned long long>(c));
    __syncthreads();
    chunk = static_cast<int32_t>(s_best & 0xffffffffull);
  }
  // counting sort of the items by key tiles, longest first
  for (int32_t b = t; b < p.batch; b += kPlanThreads) {
    int32_t P, T;
    if (!tree_request(p, b, P, T, false)) continue;
    const int32_t q_tiles = (T + per_item - 1) / per_item, nt = tiles_of(P + T);
    const int32_t full = nt / chunk, rem = nt % chunk;
    if (full > 0) atomicAdd(&s_bin[bin_of(chunk)], full * q_tiles);
    if (rem > 0) atomicAdd(&s_bin[bin_of(rem)], q_tiles);
  }
  __syncthreads();
  const int32_t mine = s_bin[t];
  int32_t incl = mine;
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
    s_warp[lane] = w;
  }
  __syncthreads();
  s_bin[t] = (warp > 0 ? s_warp[warp - 1] : 0) + incl - mine;
  const int32_t total = s_warp[kPlanThreads / 32 - 1];
  __syncthreads();
  int4* items = reinterpret_cast<int4*>(p.ws.items);
  for (int32_t b = t; b < p.batch; b += kPlanThreads) {
    int32_t P, T;
    if (!tree_request(p, b, P, T, false)) continue;
    const int32_t q_tiles = (T + per_item - 1) / per_item, nt = tiles_of(P + T);
    const int32_t splits = (nt + chunk - 1) / chunk;
    for (int32_t i = 0; i < q_tiles; ++i) {
      int32_t part = -1;
      if (splits > 1) {
        part = atomicAdd(&s_parts, splits);
        reinterpret_cast<int4*>(p.ws.merges)[atomicAdd(&s_merges, 1)] = make_int4(b, i, part, splits);
      }
      for (int32_t s = 0; s < splits; ++s) {
        const int32_t pos = atomicAdd(&s_bin[bin_of(min(chunk, nt - s * chunk))], 1);
        if (pos < p.ws.cap) items[pos] = make_int4(b, i, s, part < 0 ? -1 : part + s);
        else flag_error(p.err, RA_DEVERR_LENGTH);  // draft lengths sum above total_q
      }
    }
  }
  __syncthreads();
  if (t == 0) {
    p.ws.header[0] = static_cast<int32_t>(total < p.ws.cap ? total : p.ws.cap);
    p.ws.header[1] = 0;
    p.ws.header[2] = chunk * tc::kKeys;
    p.ws.header[3] = s_merges;
  }
}

// Row (token i of request b, q head h) key by key, one warp: D / 32 dims per lane, online softmax.
template <int D>
__device__ void recompute_row(const TreeParams& p, int32_t b, int32_t P, int32_t T, int32_t i, int32_t h) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = __ldg(p.qo_indptr + b) + i;
  const int32_t* slots = p.table + static_cast<int64_t>(__ldg(p.rpi + b)) * p.table_stride;
  const uint32_t* mrow = p.mask + row * p.mask_words;
  float q[V], acc[V], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    q[e] = __bfloat162float(p.q[(row * p.hq + h) * D + lane * V + e]);
    acc[e] = 0.f;
  }
  for (int32_t j = 0; j < P + T; ++j) {
    if (j >= P && !(__ldg(mrow + ((j - P) >> 5)) >> ((j - P) & 31) & 1u)) continue;
    int32_t slot = __ldg(slots + j);
    if (slot < 0 || slot >= p.num_slots) slot = 0;
    const int64_t at = (static_cast<int64_t>(slot) * p.hkv + h / p.group) * D + lane * V;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) s = fmaf(q[e], __bfloat162float(p.k_pool[at + e]), s);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= p.scale_log2;
    const float m_new = fmaxf(m, s);
    const float alpha = m_new == m ? 1.f : ex2(m - m_new), w = s == -INFINITY ? 0.f : ex2(s - m_new);
    m = m_new;
    l = l * alpha + w;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = acc[e] * alpha + w * __bfloat162float(p.v_pool[at + e]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < V; ++e) p.o[(row * p.hq + h) * D + lane * V + e] = __float2bfloat16_rn(acc[e] * inv);
}

// Join the splits (o = sum_s 2^(lse_s - M) o_s / sum_s 2^(lse_s - M), a warp per row), and recompute the marked
// (request, kv head) pairs' rows.  Persistent: units of kMergeRows rows of a split query tile and kv head.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const __grid_constant__ TreeParams p) {
  constexpr int V = D / 32;
  constexpr int kAhead = 8;  // partial rows in flight per warp
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t chunks = (p.ws.part_rows + kMergeRows - 1) / kMergeRows;
  const int64_t units = static_cast<int64_t>(p.ws.header[3]) * p.hkv * chunks;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int32_t r = static_cast<int32_t>(u % chunks) * kMergeRows + warp;
    const int64_t rest = u / chunks;
    const int32_t kh = static_cast<int32_t>(rest % p.hkv);
    const int4 e = reinterpret_cast<const int4*>(p.ws.merges)[rest / p.hkv];
    const int32_t tok = e.y * p.tokens_per_item + r / p.group;
    if (r >= p.ws.part_rows || tok >= __ldg(p.draft_lens + e.x) || p.ws.bad[e.x * p.hkv + kh]) continue;
    const int64_t slot_rows = static_cast<int64_t>(p.hkv) * p.ws.part_rows;  // rows between partial slots
    const int64_t row0 = (static_cast<int64_t>(e.z) * p.hkv + kh) * p.ws.part_rows + r;
    float acc[V], mrun = -INFINITY, wsum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    for (int base = 0; base < e.w; base += 32) {
      const int cnt = min(32, e.w - base);
      const float ls = lane < cnt ? __ldcg(p.ws.part_lse + row0 + (base + lane) * slot_rows) : -INFINITY;
      float mc = ls;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, off));
      const float mnew = fmaxf(mrun, mc), mref = mnew == -INFINITY ? 0.f : mnew;
      const float sc = ex2(mrun - mref);
      wsum *= sc;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] *= sc;
      mrun = mnew;
      const float wl = ex2(ls - mref);  // 0 for a split in which the row sees nothing
      wsum += wl;
      for (int k0 = 0; k0 < cnt; k0 += kAhead) {
        float x[kAhead][V];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (k0 + k < cnt) {
            const float* src = p.ws.part_o + (row0 + (base + k0 + k) * slot_rows) * D + lane * V;
            if constexpr (V == 4) {
              const float4 y = __ldcg(reinterpret_cast<const float4*>(src));
              x[k][0] = y.x, x[k][1] = y.y, x[k][2] = y.z, x[k][3] = y.w;
            } else {
              const float2 y = __ldcg(reinterpret_cast<const float2*>(src));
              x[k][0] = y.x, x[k][1] = y.y;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const float w = __shfl_sync(0xffffffffu, wl, (k0 + k) & 31);
          if (k0 + k < cnt) {
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = fmaf(w, x[k][v], acc[v]);
          }
        }
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, off);
    const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
    const int64_t row = __ldg(p.qo_indptr + e.x) + tok;
    __nv_bfloat16* dst = p.o + (row * p.hq + kh * p.group + r % p.group) * D + lane * V;
#pragma unroll
    for (int v = 0; v < V; v += 2)
      *reinterpret_cast<__nv_bfloat162*>(dst + v) = __floats2bfloat162_rn(acc[v] * inv, acc[v + 1] * inv);
  }
  const int64_t pairs = static_cast<int64_t>(p.batch) * p.hkv;
  const int64_t threads = static_cast<int64_t>(gridDim.x) * kMergeThreads;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kMergeThreads; i0 < pairs; i0 += threads) {
    const int64_t mine = i0 + threadIdx.x;
    const bool marked = mine < pairs && p.ws.bad[mine] != 0;
    if (!__syncthreads_or(marked)) continue;
    for (int64_t pair = i0; pair < i0 + kMergeThreads && pair < pairs; ++pair) {
      const int32_t b = static_cast<int32_t>(pair / p.hkv), kh = static_cast<int32_t>(pair % p.hkv);
      int32_t P, T;
      if (!p.ws.bad[pair] || !tree_request(p, b, P, T, false)) continue;
      for (int32_t r = warp; r < T * p.group; r += kMergeThreads / 32)
        recompute_row<D>(p, b, P, T, r / p.group, kh * p.group + r % p.group);
    }
  }
}

template <int D>
ra_status launch_tree(const TcParams& tp, const TreeParams& p, const CUtensorMap& qmap, const DeviceInfo& dev,
                      cudaStream_t s) {
  CUtensorMap kmap, vmap;
  if (ra_status st = row_gather_map(&kmap, p.k_pool, p.num_slots * p.hkv, D)) return st;
  if (ra_status st = row_gather_map(&vmap, p.v_pool, p.num_slots * p.hkv, D)) return st;
  using L = tc::Layout<D, k_stages<D>(), v_stages<D>()>;
  auto kern = attn_tc_kernel<D, k_stages<D>(), v_stages<D>(), kTreePass>;
  static bool configured[64] = {};
  if (L::kDynSmem > dev.max_smem_optin)
    return fail(RA_ERR_UNSUPPORTED, "tree kernel needs %d bytes of shared memory", L::kDynSmem);
  if (ra_status st = set_smem(kern, L::kDynSmem, configured, dev.device)) return st;
  // the list kernel: one CTA for the list, one per request (at most the other SMs) for the scan of V
  const int scan = p.batch < dev.num_sms - 1 ? p.batch : dev.num_sms - 1;
  if (ra_status st = launch_pdl("tree_plan_kernel", tree_plan_kernel, dim3(1 + scan), dim3(kPlanThreads), 0, s, p, D))
    return st;
  const int64_t items = p.ws.cap * p.hkv;
  const int grid = static_cast<int>(items < dev.num_sms ? items : dev.num_sms);
  if (ra_status st = launch_pdl("attn_tc_kernel<tree>", kern, dim3(grid), dim3(tc::kThreads), L::kDynSmem, s, tp, qmap,
                                kmap, vmap))
    return st;
  // Persistent.  At most cap_parts / 2 query tiles are split (each into two or more).
  const int64_t chunks = (p.ws.part_rows + kMergeRows - 1) / kMergeRows;
  const int64_t want = std::max<int64_t>(1, p.ws.cap_parts / 2 * p.hkv * chunks), most = dev.num_sms * 4;
  return launch_pdl("tree_merge_kernel", tree_merge_kernel<D>, dim3(static_cast<unsigned>(want < most ? want : most)),
                    dim3(kMergeThreads), 0, s, p);
}

bool tree_shape_ok(int32_t batch, int64_t total_q, int32_t hq, int32_t hkv, int32_t d, int32_t max_draft) {
  return batch >= 0 && batch <= 65535 && total_q >= 0 && total_q < (int64_t(1) << 31) && hkv > 0 && hq > 0 &&
         hq % hkv == 0 && 128 % (hq / hkv) == 0 && (d == 64 || d == 128) && max_draft >= 1 && max_draft <= 1024;
}

}  // namespace
}  // namespace ra

extern "C" size_t ra_tree_workspace_bytes(int32_t batch, int64_t total_q, int32_t num_q_heads, int32_t num_kv_heads,
                                          int32_t head_dim, int32_t max_draft_len) {
  if (!ra::tree_shape_ok(batch, total_q, num_q_heads, num_kv_heads, head_dim, max_draft_len)) return 0;
  return ra::layout_tree(batch, total_q, num_q_heads, num_kv_heads, head_dim, max_draft_len, nullptr).total;
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
  p.ws = layout_tree(batch, total_q, num_q_heads, num_kv_heads, head_dim, max_draft_len, workspace);
  if (!workspace || workspace_bytes < p.ws.total)
    return fail(RA_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace ? workspace_bytes : 0, p.ws.total);
  RA_REQUIRE(aligned16(workspace), "workspace must be 16-byte aligned");
  RA_REQUIRE(p.ws.cap * num_kv_heads < (int64_t(1) << 31), "too many items for one grid");
  RA_REQUIRE(static_cast<int64_t>(batch) * num_kv_heads < (int64_t(1) << 31), "batch x num_kv_heads too large");
  DeviceInfo dev;
  if (ra_status st = current_device(&dev)) return st;
  CUtensorMap qmap;
  if (ra_status st = query_tile_map(&qmap, q, total_q, num_q_heads, head_dim, group)) return st;

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
  p.tokens_per_item = tc::kTiles * (128 / group);
  p.err = device_error;
  TcParams tp{};
  tp.k_pool = p.k_pool;
  tp.v_pool = p.v_pool;
  tp.num_slots = num_slots;
  tp.hkv = num_kv_heads;
  tp.q = p.q;
  tp.hq = num_q_heads;
  tp.group = group;
  tp.scale_log2 = p.scale_log2;
  tp.table = req_to_token;
  tp.table_stride = table_stride;
  tp.table_rows = table_rows;
  tp.err = device_error;
  tp.rpi = req_pool_indices;
  tp.prefix_lens = prefix_lens;
  tp.extend_lens = draft_lens;
  tp.qo_indptr = qo_indptr;
  tp.total_q = total_q;
  tp.o = p.o;
  tp.work_count = p.ws.header;
  tp.work_counter = p.ws.header + 1;
  tp.work_items = p.ws.items;
  tp.tree_chunk = p.ws.header + 2;
  tp.tree_mask = tree_mask;
  tp.mask_words = mask_words;
  tp.part_rows = p.ws.part_rows;
  tp.part_o = p.ws.part_o;
  tp.part_lse = p.ws.part_lse;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return head_dim == 128 ? launch_tree<128>(tp, p, qmap, dev, s) : launch_tree<64>(tp, p, qmap, dev, s);
}
