// decode_mod.cu -- ra_decode_attention_mod: split-KV decode over the bf16 pool with changed scores (a cap by a tanh, a bias by
// distance) and a first key per request (a window, a document).
//
// Like the plain decode it is bound by HBM: 4 D bytes and 4 D flop per key, q head and kv head, each byte read once for the
// whole GQA group.  Built on the slab ring: producers copy the K and V rows of a slab's keys for a group of kv heads
// (hpc * D * 2 contiguous bytes each), consumer warp w takes kv head hg * hpc + w with the keys on the M side and the
// GQA group on N (S^T = K Q^T, O^T += V^T P^T on mma.sync: a tcgen05 tile would be mostly padding), references are lazy,
// and partials are merged by a kernel that waits per request.  Keys before a request's first one are in no item, so a
// window costs what its keys do.  The changed scores cost a warp about 60 instructions per 16-key slab and 8 heads,
// beside some 100 for the products: hidden behind the copies.  224 requests of 65..13,700 keys, 64/8 heads, capped and
// biased: 340 us, 2,353 MB at the measured copy rate 347 (some of the short contexts' rows stay in L2).  Small calls plan
// in their own warps: one request of 1,500 keys 7.8 us (16.7 with a planning kernel), 64 of 1,024 keys of a window 49.
#include <cmath>

#include "api_common.h"
#include "decode_internal.h"
#include "decode_item.cuh"
#include "ra_ptx.cuh"
#include "score_mod_host.h"
#include "slab_ring.cuh"
#include "small_plan.cuh"

namespace ra {

namespace {

constexpr float kRescale = 8.0f;    // log2 units: a reference moves when a score exceeds it by more
constexpr int kSmallLeast = 1;      // units of a small call's shortest piece
constexpr int ctas_per_sm(int head_dim, int hpc) { return hpc <= (head_dim == 64 ? 3 : 2) ? 2 : 1; }

struct ModDecodeParams {
  DecodeParams d;
  int32_t row_bytes;  // hpc * D * 2
  int32_t ctas;       // small call: the grid
};

// The items of a call: the plan kernel's list, or (SMALL = 1 or 2 requests per lane) this warp's own plan.
template <int SMALL>
struct ModItems {
  const DecodeParams& p;
  SmallPlan<SMALL ? SMALL : 1> plan;
  PerRequest<SMALL ? SMALL : 1> keys, first, row, valid;

  __device__ __forceinline__ ModItems(const DecodeParams& q, int32_t ctas, bool report) : p(q) {
    if constexpr (SMALL) {
#pragma unroll
      for (int i = 0; i < SMALL; ++i) {
        const int32_t b = static_cast<int32_t>(threadIdx.x & 31) + 32 * i;
        if (b >= p.batch) continue;
        const int32_t r = __ldg(p.rpi + b);
        int32_t L = __ldg(p.seq_lens + b);
        const bool bad_row = r < 0 || r >= p.table_rows, bad_len = L < 1 || L > p.max_seq_len;
        if (report && bad_row) flag_error(p.err, RA_DEVERR_TABLE);
        else if (report && bad_len) flag_error(p.err, RA_DEVERR_LENGTH);
        if (bad_row || L < 1) continue;
        L = min(L, p.max_seq_len);
        row.v[i] = r;
        first.v[i] = mod_start(p, b, L);
        keys.v[i] = L - first.v[i];
        valid.v[i] = 1;
      }
      plan.make(keys, p.n_hgroups, ctas, kSmallLeast);
    }
  }
  __device__ __forceinline__ int32_t count() const { return (SMALL ? plan.n : p.plan[0]) * p.n_hgroups; }
  // (SMALL: warp-collective)
  __device__ __forceinline__ void item(int32_t idx, Item& it) const {
    if constexpr (SMALL) {
      it.hg = idx % p.n_hgroups;
      it.d = idx / p.n_hgroups;
      it.b = plan.request(it.d);
      it.split = it.d - of_request(plan.first, it.b);
      it.n_splits = of_request(plan.pieces, it.b);
      it.row = of_request(row, it.b);
      it.start = of_request(first, it.b);
      it.k0 = it.start + it.split * plan.chunk;
      it.k1 = min(it.start + of_request(keys, it.b), it.k0 + plan.chunk);
    } else {
      decode_item<true>(p, idx, it);
    }
  }
  // The position of request b's query.
  __device__ __forceinline__ int32_t position(int32_t b) const {
    if constexpr (SMALL) return of_request(first, b) + of_request(keys, b) - 1;
    else return min(__ldg(p.seq_lens + b), p.max_seq_len) - 1;
  }
};

// The producers' view: K row and V row of a key for the item's head group.
template <int SLAB, int SMALL>
struct ModSource {
  const ModDecodeParams& pp;
  const ModItems<SMALL>& items;
  int32_t* counter;
  int64_t num_slots;
  uint32_t* err;
  __device__ __forceinline__ ModSource(const ModDecodeParams& q, const ModItems<SMALL>& it)
      : pp(q), items(it), counter(q.d.counter), num_slots(q.d.num_slots), err(q.d.err) {}
  __device__ __forceinline__ int32_t claims() const { return items.count(); }
  __device__ __forceinline__ void item(int32_t idx, SlabKeys& k) const {
    Item it;
    items.item(idx, it);
    k = SlabKeys{pp.d.table + static_cast<int64_t>(it.row) * pp.d.table_stride, it.k0, it.k1, it.hg};
  }
  __device__ __forceinline__ uint32_t key_bytes() const { return 2 * pp.row_bytes; }
  __device__ __forceinline__ void copy(uint32_t stage, int key, int32_t slot, int32_t group, uint32_t bar) const {
    const int64_t at = (static_cast<int64_t>(slot) * pp.d.n_hgroups + group) * pp.row_bytes;
    bulk_g2s(stage + key * pp.d.row_stride, reinterpret_cast<const uint8_t*>(pp.d.k_pool) + at, pp.row_bytes, bar);
    bulk_g2s(stage + (SLAB + key) * pp.d.row_stride, reinterpret_cast<const uint8_t*>(pp.d.v_pool) + at, pp.row_bytes, bar);
  }
};

template <int D, int SLAB, int SMALL>
__global__ void __launch_bounds__(32 * (kMaxHeadsPerCta + kRingProducers + 1), 1)
    decode_mod_kernel(const __grid_constant__ ModDecodeParams pp) {
  constexpr int KT = D / 16, NB = SLAB / 16;
  const DecodeParams& p = pp.d;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int nc = p.hpc;
  const int RS = p.row_stride;
  const SlabRing rg(smem, p.nstage, p.stage_bytes);
  if (threadIdx.x == 0) rg.init(nc, 1);
  __syncthreads();
  griddep_wait();    // the plan, its reset counters and everything before them are complete
  griddep_launch();  // the combine may launch: it waits per request for the partials it merges

  if (warp > nc + kRingProducers) return;
  const ModItems<SMALL> items(p, pp.ctas, blockIdx.x == 0 && warp == 0);
  if (warp >= nc && warp < nc + kRingProducers) {
    slab_producer<SLAB>(rg, ModSource<SLAB, SMALL>(pp, items), warp - nc);
    return;
  }
  if (warp == nc + kRingProducers) {
    if constexpr (!SMALL) {  // (a small call has one item per CTA, and its merge waits for the grid)
      // ================================================================ signaller
      for (int32_t n = 0;; ++n) {
        const int e = n % kRingEntries;
        const int32_t idx = rg.entry(n);
        int32_t* count = nullptr;  // the request's count, if its partials are merged by the combine
        if (idx >= 0 && lane == 0) {
          Item it;
          decode_item<true>(p, idx, it);
          if (it.n_splits > 1) count = p.req_done + it.b;
        }
        if (idx < -1 || !mbar_wait(rg.done0 + 8 * e, (n / kRingEntries) & 1)) {
          if (lane == 0) rg.give_up(p.err);
          break;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(rg.free0 + 8 * e);
        if (idx < 0) break;
        if (count) {
          __threadfence();  // the consumers' partials (ordered before this by the done barrier) first
          atomicAdd(count, 1);
        }
        __syncwarp();
      }
    }
    return;
  }
  // ================================================================ consumers
  const int g = lane >> 2;  // key of an 8-key block (M), and for q the head of the group (N)
  const int tq = lane & 3;
  const uint32_t a_off = (lane & 15) * RS + (lane >> 4) * 16 + warp * D * 2;
  const uint32_t v_off = SLAB * RS + ((lane & 7) + ((lane >> 4) << 3)) * RS + ((lane >> 3) & 1) * 16 + warp * D * 2;
  int32_t n = 0, c = 0;
  bool clean = false;  // left through the end marker
  for (;; ++n) {
    const int32_t idx = rg.entry(n);
    if (idx < 0) {
      clean = idx == -1;
      __syncwarp();
      if (clean && lane == 0) mbar_arrive(rg.done0 + 8 * (n % kRingEntries));  // the signal warp reads the end marker
      break;
    }
    Item it;
    items.item(idx, it);
    const int32_t pos = items.position(it.b);
    const int kh = it.hg * p.hpc + warp;
    const bool h0 = 2 * tq < p.group, h1 = 2 * tq + 1 < p.group;  // q heads 2 tq and 2 tq + 1 of the group exist
    float slope0 = 0.f, slope1 = 0.f;                             // their bias per position, in log2 units
    if (p.mod.slopes) {
      const float* sl = p.mod.slopes + kh * p.group + 2 * tq;
      if (h0) slope0 = __ldg(sl) * kLog2e;
      if (h1) slope1 = __ldg(sl + 1) * kLog2e;
    }
    // Q^T fragments (B operand): column g is q head kh*G + g
    uint32_t qf[KT][2];
    {
      const bool live = g < p.group;
      const __nv_bfloat16* qrow = p.q + (static_cast<int64_t>(it.b) * p.hq + kh * p.group + (live ? g : 0)) * D;
#pragma unroll
      for (int kk = 0; kk < KT; ++kk) {
        qf[kk][0] = live ? __ldg(reinterpret_cast<const uint32_t*>(qrow + kk * 16 + 2 * tq)) : 0u;
        qf[kk][1] = live ? __ldg(reinterpret_cast<const uint32_t*>(qrow + kk * 16 + 8 + 2 * tq)) : 0u;
      }
    }
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float ref0 = 0.f, ref1 = 0.f;  // what is subtracted: m0 and m1, or 0 while every score is minus infinity
    float acc[KT][4];
#pragma unroll
    for (int mt = 0; mt < KT; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
    const int32_t n_slabs = (it.k1 - it.k0 + SLAB - 1) / SLAB;
    bool ok = true;
    for (int32_t s = 0; s < n_slabs; ++s, ++c) {
      const int st = c % rg.nstage;
      if (!mbar_wait(rg.full0 + 8 * st, (c / rg.nstage) & 1)) { ok = false; break; }
      const uint32_t stage = rg.stage0 + st * rg.stage_bytes;
      const int32_t kbase = it.k0 + s * SLAB + g;  // this lane's first key
      float x[NB][4];  // (key, head): (g, 2 tq), (g, 2 tq + 1), (g + 8, 2 tq), (g + 8, 2 tq + 1)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        // S^T[16 keys x 8 heads] = K Q^T, two independent MMA chains
        float s1[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < KT; kk += 2) {
          uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
          ldsm_x4(stage + b * 16 * RS + a_off + kk * 32, a0, a1, a2, a3);
          ldsm_x4(stage + b * 16 * RS + a_off + (kk + 1) * 32, b0, b1, b2, b3);
          mma_bf16_16816(s1, a0, a1, a2, a3, qf[kk][0], qf[kk][1]);
          mma_bf16_16816(s2, b0, b1, b2, b3, qf[kk + 1][0], qf[kk + 1][1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[b][e] = s1[e] + s2[e];
      }
      if (p.mod.cap_in > 0.f) {
        float far = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[b][e] *= p.mod.cap_in;
            far = fmaxf(far, fabsf(x[b][e]));
          }
        // (a vote: the general form costs two special functions a score)
        if (__any_sync(0xffffffffu, !(far <= kCapPolyMax))) {
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[b][e] = tanh_any(x[b][e]) * p.mod.cap_log2;
        } else {
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[b][e] = tanh_small(x[b][e]) * p.mod.cap_log2;
        }
      } else {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[b][e] *= p.scale_log2;
      }
      bool above = false;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int32_t key = kbase + 16 * b;
        const float lo = static_cast<float>(pos - key), hi = lo - 8.f;  // distances
        const bool v_lo = key < it.k1, v_hi = key + 8 < it.k1;
        x[b][0] = v_lo ? fmaf(-slope0, lo, x[b][0]) : -INFINITY;
        x[b][1] = v_lo ? fmaf(-slope1, lo, x[b][1]) : -INFINITY;
        x[b][2] = v_hi ? fmaf(-slope0, hi, x[b][2]) : -INFINITY;
        x[b][3] = v_hi ? fmaf(-slope1, hi, x[b][3]) : -INFINITY;
        above = above || x[b][0] > m0 + kRescale || x[b][2] > m0 + kRescale || x[b][1] > m1 + kRescale ||
                x[b][3] > m1 + kRescale;
      }
      // Lazy reference: it moves, and O and l are rescaled, only when a score of the slab exceeds it by more than kRescale;
      // an item's first slab moves it (its first key is in range) unless every score there is minus infinity.
      if (__any_sync(0xffffffffu, above)) {
        float mx0 = m0, mx1 = m1;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          mx0 = fmaxf(mx0, fmaxf(x[b][0], x[b][2]));
          mx1 = fmaxf(mx1, fmaxf(x[b][1], x[b][3]));
        }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
        }
        ref0 = mx0 == -INFINITY ? 0.f : mx0;
        ref1 = mx1 == -INFINITY ? 0.f : mx1;
        const float al0 = ex2(m0 - ref0), al1 = ex2(m1 - ref1);
        m0 = mx0;
        m1 = mx1;
        l0 *= al0;
        l1 *= al1;
#pragma unroll
        for (int mt = 0; mt < KT; ++mt) {
          acc[mt][0] *= al0;
          acc[mt][1] *= al1;
          acc[mt][2] *= al0;
          acc[mt][3] *= al1;
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float p0 = ex2(x[b][0] - ref0), p1 = ex2(x[b][1] - ref1), p2 = ex2(x[b][2] - ref0), p3 = ex2(x[b][3] - ref1);
        l0 += p0 + p2;
        l1 += p1 + p3;
        // P^T as the B operand: transpose the two 8x8 key blocks
        const uint32_t pb0 = movmatrix_trans(pack_bf16x2(p0, p1)), pb1 = movmatrix_trans(pack_bf16x2(p2, p3));
        // O^T[D x 8] += V^T P^T
#pragma unroll
        for (int mt = 0; mt < KT; ++mt) {
          uint32_t a0, a1, a2, a3;
          ldsm_x4_trans(stage + b * 16 * RS + v_off + mt * 32, a0, a1, a2, a3);
          mma_bf16_16816(acc[mt], a0, a1, a2, a3, pb0, pb1);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(rg.empty0 + 8 * st);
    }
    if (!ok) break;
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    // outputs: thread holds (d = mt*16 + g [+8], q head 2*tq [+1]) of this kv head
    const float inv0 = l0 == 0.f ? 0.f : 1.f / l0, inv1 = l1 == 0.f ? 0.f : 1.f / l1;
    const bool direct = it.n_splits == 1;
    const int64_t r0 = (direct ? static_cast<int64_t>(it.b) : static_cast<int64_t>(it.d)) * p.hq + kh * p.group + 2 * tq;
#pragma unroll
    for (int mt = 0; mt < KT; ++mt) {
      const int64_t at = r0 * D + mt * 16 + g;
      if (direct) {
        if (h0) p.o[at] = __float2bfloat16_rn(acc[mt][0] * inv0), p.o[at + 8] = __float2bfloat16_rn(acc[mt][2] * inv0);
        if (h1) p.o[at + D] = __float2bfloat16_rn(acc[mt][1] * inv1), p.o[at + D + 8] = __float2bfloat16_rn(acc[mt][3] * inv1);
      } else {
        if (h0) p.part_o[at] = acc[mt][0] * inv0, p.part_o[at + 8] = acc[mt][2] * inv0;
        if (h1) p.part_o[at + D] = acc[mt][1] * inv1, p.part_o[at + D + 8] = acc[mt][3] * inv1;
      }
    }
    if (!direct && g == 0) {
      if (h0) p.part_lse[r0] = m0 + __log2f(l0);
      if (h1) p.part_lse[r0 + 1] = m1 + __log2f(l1);
    }
    // this warp's part of the entry is written (__syncwarp orders the lanes' stores before lane 0's release)
    __syncwarp();
    if (lane == 0) mbar_arrive(rg.done0 + 8 * (n % kRingEntries));
  }
  if (!clean && lane == 0) rg.give_up(p.err);  // a bounded wait ran out: stop the producers as well
}

// Merge the partials of every split request, and write the zeros of those that see no key.  Launched while the decode
// kernel runs: a row (request, q head) waits only for its own request's count of finished partials; a small call's, for
// the grid.  Many rows: 8 lanes per row; few: `per_row` warps share one, each a part of its partials.
constexpr int kCombineWarps = 8;
constexpr int kRowLanes = 8;

// The request's partials, once they are written (a warp's lanes may ask for different requests): their first index and
// number; 0 if its rows were written directly or it is invalid, -1 if it sees no key.
__device__ __forceinline__ int32_t wait_partials(const DecodeParams& p, int32_t b, bool in, int32_t& i0) {
  // the plan completed before the decode kernel let this one launch
  const int32_t L = __ldg(p.seq_lens + b), row = __ldg(p.rpi + b);
  i0 = __ldcg(p.req_item0 + b);
  int32_t n = __ldcg(p.req_item0 + b + 1) - i0;
  if (!in || n == 1 || L < 1 || row < 0 || row >= p.table_rows) n = 0;
  else if (n == 0) n = -1;
  // every lane reads the count itself: with the fence its loads of the partials follow an acquire
  if (n > 0 && !wait_count(p.req_done + b, n * p.n_hgroups)) {
    flag_error(p.err, RA_DEVERR_TIMEOUT);
    n = 0;
  }
  fence_acq_rel_gpu();
  return n;
}

template <int D>
__global__ void __launch_bounds__(32 * kCombineWarps) decode_mod_combine_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int V = D / kRowLanes;
  griddep_launch();
  const int sub = (threadIdx.x & 31) % kRowLanes;
  const int32_t bh = static_cast<int32_t>(blockIdx.x * (32 * kCombineWarps / kRowLanes) + threadIdx.x / kRowLanes);
  const bool in = bh < p.batch * p.hq;
  const int32_t b = in ? bh / p.hq : 0, h = in ? bh - b * p.hq : 0;
  int32_t i0;
  const int32_t n = wait_partials(p, b, in, i0);
  __syncwarp();
  float acc[V], wsum;
  merge_rows<kRowLanes, V, 256 / D>(
      max(n, 0), [&](int s) { return __ldcg(p.part_lse + static_cast<int64_t>(i0 + s) * p.hq + h); },
      [&](int s, float(&x)[V]) {
        load_row_part<kRowLanes, V>(p.part_o + (static_cast<int64_t>(i0 + s) * p.hq + h) * D, sub, x);
      },
      acc, wsum);
  // (no weight: no key, or none with a score above minus infinity)
  if (n != 0) store_row_part<kRowLanes, V>(p.o + static_cast<int64_t>(bh) * D, sub, acc, wsum == 0.f ? 0.f : 1.f / wsum);
  griddep_wait();  // this grid's completion implies the decode kernel's
}

template <int D, int SMALL>
__global__ void __launch_bounds__(32 * kCombineWarps)
    decode_mod_combine_few_kernel(const __grid_constant__ DecodeParams p, int per_row, int32_t ctas) {
  constexpr int V = D / 32;
  __shared__ float s_acc[kCombineWarps][32 * V], s_m[kCombineWarps], s_w[kCombineWarps];
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int share = warp % per_row;
  const int32_t bh = static_cast<int32_t>(blockIdx.x) * (kCombineWarps / per_row) + warp / per_row;
  const bool in = bh < p.batch * p.hq;
  const int32_t b = in ? bh / p.hq : 0, h = in ? bh - b * p.hq : 0;
  int32_t i0, n;
  if constexpr (SMALL) {
    // (the lengths were complete before the decode kernel let this one launch)
    const ModItems<SMALL> items(p, ctas, false);
    i0 = of_request(items.plan.first, b);
    n = of_request(items.plan.pieces, b);
    if (!in || n == 1 || !of_request(items.valid, b)) n = 0;  // written directly, or invalid
    else if (n == 0) n = -1;
    griddep_wait();
  } else {
    n = wait_partials(p, b, in, i0);
    __syncwarp();
  }
  float acc[V], m, wsum;
  merge_partials<V, 8>(
      max(n, 0), share, per_row, [&](int s) { return __ldcg(p.part_lse + static_cast<int64_t>(i0 + s) * p.hq + h); },
      [&](int s, float(&x)[V]) {
        load_row_cg<V>(p.part_o + (static_cast<int64_t>(i0 + s) * p.hq + h) * D + lane * V, x);
      },
      acc, m, wsum);
#pragma unroll
  for (int v = 0; v < V; ++v) s_acc[warp][lane * V + v] = acc[v];
  if (lane == 0) s_m[warp] = m, s_w[warp] = wsum;
  __syncthreads();
  if (n != 0 && share == 0) {
    join_shares<V>(per_row, warp, s_acc, s_m, s_w, acc, wsum);
    const float inv = wsum == 0.f ? 0.f : 1.f / wsum;  // (no key, or none with a score above minus infinity)
    __nv_bfloat16* dst = p.o + static_cast<int64_t>(bh) * D + lane * V;
#pragma unroll
    for (int v = 0; v < V; v += 2)
      *reinterpret_cast<__nv_bfloat162*>(dst + v) = __floats2bfloat162_rn(acc[v] * inv, acc[v + 1] * inv);
  }
  griddep_wait();  // this grid's completion implies the decode kernel's
}

template <int D, int SLAB, int SMALL>
ra_status launch_decode(const ModDecodeParams& pp, int grid, int smem, const DeviceInfo& dev, cudaStream_t stream) {
  auto kern = decode_mod_kernel<D, SLAB, SMALL>;
  static bool configured[64] = {};
  if (!configured[dev.device]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmemLimit);
    if (e != cudaSuccess) return fail(RA_ERR_CUDA, "cudaFuncSetAttribute(decode): %s", cudaGetErrorString(e));
    configured[dev.device] = true;
  }
  return launch_pdl("decode_mod_kernel", kern, dim3(grid), dim3(32 * (pp.d.hpc + kRingProducers + 1)), smem, stream, pp);
}

template <int D, int SLAB>
ra_status launch(ModDecodeParams& pp, int32_t per_sm, int smem, const DeviceInfo& dev, cudaStream_t s) {
  DecodeParams& p = pp.d;
  const int64_t rows = static_cast<int64_t>(p.batch) * p.hq, warps = static_cast<int64_t>(dev.num_sms) * 3 * kCombineWarps;
  const int32_t most = p.mod.window > 0 && p.mod.window < p.max_seq_len ? p.mod.window : p.max_seq_len;  // keys of a request
  const bool small = small_call(p.batch, most, p.n_hgroups, per_sm), many = p.batch > 32;
  if (small) {
    pp.ctas = kSmallSms * per_sm;
    if (ra_status st = many ? launch_decode<D, SLAB, 2>(pp, pp.ctas, smem, dev, s)
                            : launch_decode<D, SLAB, 1>(pp, pp.ctas, smem, dev, s))
      return st;
  } else {
    if (ra_status st = launch_decode_plan_mod(p, s)) return st;
    const int64_t n_items = static_cast<int64_t>(p.max_items) * p.n_hgroups;  // bound of the claims
    const int64_t ctas = static_cast<int64_t>(dev.num_sms) * per_sm;
    if (ra_status st = launch_decode<D, SLAB, 0>(pp, static_cast<int>(n_items < ctas ? n_items : ctas), smem, dev, s))
      return st;
  }
  // few rows: as many warps per row as three CTAs per SM hold, or one up to 32 rows per SM (as the quantised decode)
  int per_row = 1;
  while (per_row < kCombineWarps && rows * per_row * 2 <= warps) per_row *= 2;
  if (per_row > 1 || small || rows <= static_cast<int64_t>(dev.num_sms) * 32) {
    const int64_t ctas = (rows * per_row + kCombineWarps - 1) / kCombineWarps;
    auto kern = !small ? decode_mod_combine_few_kernel<D, 0>
                       : many ? decode_mod_combine_few_kernel<D, 2> : decode_mod_combine_few_kernel<D, 1>;
    return launch_pdl("decode_mod_combine_few_kernel", kern, dim3(static_cast<unsigned>(ctas)), dim3(32 * kCombineWarps), 0,
                      s, p, per_row, pp.ctas);
  }
  const int64_t per_cta = kCombineWarps * 32 / kRowLanes;
  return launch_pdl("decode_mod_combine_kernel", decode_mod_combine_kernel<D>,
                    dim3(static_cast<unsigned>((rows + per_cta - 1) / per_cta)), dim3(32 * kCombineWarps), 0, s, p);
}

}  // namespace
}  // namespace ra

extern "C" ra_status ra_decode_attention_mod(const void* k_pool, const void* v_pool, int64_t num_slots,
                                             int32_t num_kv_heads, int32_t head_dim, const void* q, void* o,
                                             int32_t num_q_heads, float sm_scale, float score_cap, int32_t window,
                                             const float* slopes, const int32_t* first_key, const int32_t* req_to_token,
                                             int64_t table_stride, int64_t table_rows, const int32_t* req_pool_indices,
                                             const int32_t* seq_lens, int32_t batch, int32_t max_seq_len, void* workspace,
                                             size_t workspace_bytes, uint32_t* device_error, ra_stream_t stream) {
  using namespace ra;
  clear_error();
  RA_REQUIRE(batch >= 0 && batch <= 65535, "batch must be in [0, 65535] (got %d)", batch);
  RA_REQUIRE(num_kv_heads > 0 && num_q_heads > 0, "head counts must be > 0");
  RA_REQUIRE(num_q_heads % num_kv_heads == 0, "num_q_heads (%d) must be a multiple of num_kv_heads (%d)", num_q_heads,
             num_kv_heads);
  RA_REQUIRE(num_slots > 0, "num_slots must be > 0");
  ModDecodeParams pp{};
  DecodeParams& p = pp.d;
  if (ra_status st = score_mod(&p.mod, sm_scale, score_cap, window, slopes, first_key, nullptr)) return st;
  if (head_dim != 64 && head_dim != 128) return fail(RA_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", head_dim);
  const int32_t group = num_q_heads / num_kv_heads;
  if (group > 8) return fail(RA_ERR_UNSUPPORTED, "GQA group %d (decode supports up to 8)", group);
  if (batch == 0) return RA_OK;
  RA_REQUIRE(max_seq_len >= 1, "max_seq_len must be >= 1");
  RA_REQUIRE(table_stride >= max_seq_len, "table_stride (%lld) < max_seq_len (%d)", (long long)table_stride, max_seq_len);
  RA_REQUIRE(table_rows > 0, "table_rows must be > 0");
  RA_REQUIRE(k_pool && v_pool && q && o && req_to_token && req_pool_indices && seq_lens, "null pointer argument");
  RA_REQUIRE(aligned16(k_pool) && aligned16(v_pool) && aligned16(q) && aligned16(o),
             "pools, q and o must be 16-byte aligned");
  RA_REQUIRE(aligned4(req_to_token) && aligned4(req_pool_indices) && aligned4(seq_lens),
             "index arrays must be 4-byte aligned");
  // the device plan's item length must fit in 31 bits (it is at most batch x max_seq_len / plan_items)
  RA_REQUIRE(static_cast<int64_t>(batch) * max_seq_len <= static_cast<int64_t>(kSmallSms) << 30,
             "batch x max_seq_len too large");
  RA_REQUIRE(static_cast<int64_t>(batch) * num_q_heads < (int64_t(1) << 30), "batch x num_q_heads too large");
  const DecodePlan pl = plan_decode(batch, num_q_heads, num_kv_heads, head_dim, max_seq_len, 0, 0, 0);
  const DecodeWorkspace wl = layout_decode_workspace(batch, num_q_heads, num_kv_heads, head_dim, pl, 0);
  if (workspace_bytes < wl.total)
    return fail(RA_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace_bytes, wl.total);
  RA_REQUIRE(workspace && aligned16(workspace), "workspace must be non-null and 16-byte aligned");
  DeviceInfo dev;
  if (ra_status st = current_device(&dev)) return st;
  p.k_pool = static_cast<const __nv_bfloat16*>(k_pool);
  p.v_pool = static_cast<const __nv_bfloat16*>(v_pool);
  p.num_slots = num_slots;
  p.hkv = num_kv_heads;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.hq = num_q_heads;
  p.group = group;
  p.scale_log2 = sm_scale * kLog2e;
  p.table = req_to_token;
  p.table_stride = table_stride;
  p.table_rows = table_rows;
  p.rpi = req_pool_indices;
  p.seq_lens = seq_lens;
  p.batch = batch;
  p.max_seq_len = max_seq_len;
  p.err = device_error;
  bind_decode_workspace(p, wl, pl, workspace);
  // kv heads per item: the largest divisor of Hkv that is <= 8 (one consumer warp each)
  for (p.hpc = kMaxHeadsPerCta; num_kv_heads % p.hpc != 0;) --p.hpc;
  p.n_hgroups = num_kv_heads / p.hpc;
  pp.row_bytes = p.hpc * head_dim * 2;
  p.row_stride = pp.row_bytes + 16;
  // A CTA of few heads waits on its own chain of slab, scores, softmax and product: two share an SM.
  const int per_sm = ctas_per_sm(head_dim, p.hpc);
  static_assert(2 * kSmallSms <= kDecodePlanItems, "the workspace holds the plan's items");
  p.plan_items = kSmallSms * per_sm;
  p.min_chunk = 64;
  const int ring = kRingSmemLimit / per_sm - 1024 - kRingHdrBytes;  // (1 KB per CTA is the system's)
  // 32-key slabs where three of them fit the ring, else 16-key ones
  const int slab = 3 * 2 * 32 * p.row_stride <= ring ? 32 : 16;
  p.chunk_align = slab;
  p.stage_bytes = 2 * slab * p.row_stride;
  p.nstage = ring / p.stage_bytes;
  if (p.nstage > kRingMaxStages) p.nstage = kRingMaxStages;
  const int smem = kRingHdrBytes + p.nstage * p.stage_bytes;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (head_dim == 64) return slab == 32 ? launch<64, 32>(pp, per_sm, smem, dev, s) : launch<64, 16>(pp, per_sm, smem, dev, s);
  return slab == 32 ? launch<128, 32>(pp, per_sm, smem, dev, s) : launch<128, 16>(pp, per_sm, smem, dev, s);
}
