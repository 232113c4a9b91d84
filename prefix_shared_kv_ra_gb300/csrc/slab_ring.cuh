// slab_ring.cuh -- the producer side of the persistent split-KV kernels: items claimed from a counter, their
// keys streamed slab by slab into a ring of shared-memory stages by bulk copies.
//
// One CTA per SM, or two for narrow head groups.  kRingProducers warps copy the records (or K and V rows) of a slab's keys, one lane per key,
// each warp a part of the slab; the first of them also claims the items and publishes them through a ring of
// entries with one mbarrier each, so that every producer looks one slab ahead across items for its slot ids.
// Consumers take the items from the same entries (before the item's first slab has landed, so that they fetch
// its queries meanwhile), wait on a stage's full barrier and arrive on its empty barrier after use; an entry's
// free barrier takes the arrivals of its last readers (the consumers, or a warp that waits for them on its done
// barrier).  Every wait is bounded: a wait that
// runs out raises the CTA's abort flag and RA_DEVERR_TIMEOUT, and every role leaves.
#pragma once

#include <stdint.h>

#include "ra_ptx.cuh"

namespace ra {

constexpr int kRingMaxStages = 8;
constexpr int kRingEntries = 16;    // published items; the claimer runs at most nstage + 1 items ahead
constexpr int kRingProducers = 4;   // copy issue rate grows with the issuing warps
constexpr int kRingHdrBytes = 640;  // barriers, entries, abort flag
constexpr int kRingSmemLimit = 227 * 1024;

struct SlabRing {
  uint32_t full0, empty0;       // nstage mbarriers each
  uint32_t item0, done0, free0;  // kRingEntries mbarriers each: entry published, used by every consumer, free
  volatile int32_t* items;
  volatile int32_t* abort;
  uint32_t stage0;
  int nstage;
  uint32_t stage_bytes;

  __device__ __forceinline__ SlabRing(uint8_t* smem, int stages, uint32_t bytes) {
    const uint32_t base = smem_u32(smem);
    full0 = base;
    empty0 = base + 64;
    items = reinterpret_cast<volatile int32_t*>(smem + 128);
    abort = reinterpret_cast<volatile int32_t*>(smem + 192);
    item0 = base + 256;
    done0 = base + 384;
    free0 = base + 512;
    stage0 = base + kRingHdrBytes;
    nstage = stages;
    stage_bytes = bytes;
  }
  // One thread, before a __syncthreads(): `consumers` warps use each stage, `readers` arrivals free an entry.
  __device__ __forceinline__ void init(int consumers, int readers) const {
    for (int s = 0; s < nstage; ++s) {
      mbar_init(full0 + 8 * s, kRingProducers);
      mbar_init(empty0 + 8 * s, consumers);
    }
    for (int s = 0; s < kRingEntries; ++s) {
      mbar_init(item0 + 8 * s, 1);
      mbar_init(done0 + 8 * s, consumers);
      mbar_init(free0 + 8 * s, readers);
    }
    *abort = 0;
    fence_mbar_init();
  }
  // Item n's index (-1: no more work), or -2 if the wait ran out.
  __device__ __forceinline__ int32_t entry(int32_t n) const {
    if (!mbar_wait(item0 + 8 * (n % kRingEntries), (n / kRingEntries) & 1) || *abort) return -2;
    return items[n % kRingEntries];
  }
  __device__ __forceinline__ void give_up(uint32_t* err) const {
    *abort = 1;
    flag_error(err, RA_DEVERR_TIMEOUT);
  }
};

// What the producers need of an item: its keys [k0, k1) of the request whose slots are listed at `slots`, and
// the head group to copy.
struct SlabKeys {
  const int32_t* slots;
  int32_t k0, k1, group;
};

// Producer warp pw of kRingProducers (all lanes).  Src: claims() = items of the launch; item(idx, SlabKeys&);
// copy(stage, key, slot, group, bar) issues one key's copies into row `key` of a stage; key_bytes() their bytes;
// counter, num_slots, err.  A slab's keys past the item's range repeat its last key (consumers mask them).
template <int SLAB, class Src>
__device__ __forceinline__ void slab_producer(const SlabRing& rg, const Src& src, int pw) {
  constexpr int kKeys = SLAB / kRingProducers;  // keys per producer and slab
  const int lane = threadIdx.x & 31;
  const bool leader = pw == 0;
  const int key_in_slab = pw * kKeys + lane;  // this lane's key (lane < kKeys)
  const int ns = rg.nstage;
  const int32_t n_claims = src.claims();
  // a CTA's first item is its block index; the counter hands out the items after the grid (if there are any)
  auto claim = [&](bool first) -> int32_t {  // warp-collective
    int32_t idx = static_cast<int32_t>(blockIdx.x);
    if (!first) {
      if (n_claims <= static_cast<int32_t>(gridDim.x)) return -1;
      if (lane == 0) idx = static_cast<int32_t>(gridDim.x) + atomicAdd(src.counter, 1);
      idx = __shfl_sync(0xffffffffu, idx, 0);
    }
    return idx < n_claims ? idx : -1;
  };
  // entry n reuses the ring slot of entry n - kRingEntries: its last reader must be done with it
  auto publish = [&](int32_t n, int32_t idx) -> bool {
    if (n >= kRingEntries && !mbar_wait(rg.free0 + 8 * (n % kRingEntries), ((n / kRingEntries) - 1) & 1)) return false;
    if (lane == 0) {
      rg.items[n % kRingEntries] = idx;
      mbar_arrive(rg.item0 + 8 * (n % kRingEntries));
    }
    return true;
  };
  // 1: item n in `it`; 0: end of work; -1: a bounded wait ran out
  auto next_item = [&](int32_t n, SlabKeys& it) -> int {
    const int32_t idx = rg.entry(n);
    if (idx < 0) return idx + 1;
    src.item(idx, it);
    return 1;
  };
  auto load_slot = [&](const SlabKeys& it, int32_t s) -> int32_t {
    if (lane >= kKeys) return 0;
    return __ldg(it.slots + min(it.k0 + s * SLAB + key_in_slab, it.k1 - 1));
  };
  bool ok = true;
  if (leader) ok = __all_sync(0xffffffffu, publish(0, claim(true)));
  int32_t n = 0, c = 0, s = 0;
  SlabKeys it{};
  int r = ok ? next_item(0, it) : -1;
  ok = r >= 0;
  int32_t slot = r > 0 ? load_slot(it, 0) : 0;
  while (ok && r > 0) {
    const int32_t n_slabs = (it.k1 - it.k0 + SLAB - 1) / SLAB;
    // the leader claims the next item when this one has ns slabs left to issue (the claim overlaps them)
    if (leader && s == (n_slabs > ns ? n_slabs - ns : 0) && !__all_sync(0xffffffffu, publish(n + 1, claim(false)))) {
      ok = false;
      break;
    }
    // one slab ahead: the next (item, slab) and its slot id
    SlabKeys it2 = it;
    int32_t s2 = s + 1, n2 = n;
    int r2 = 1;
    if (s2 == n_slabs) {
      n2 = n + 1;
      s2 = 0;
      r2 = next_item(n2, it2);
      if (r2 < 0) { ok = false; break; }
    }
    const int32_t slot2 = r2 > 0 ? load_slot(it2, s2) : 0;
    // slab s of item n into stage c % ns
    const int st = c % ns;
    if (c >= ns && !mbar_wait(rg.empty0 + 8 * st, ((c / ns) + 1) & 1)) { ok = false; break; }
    if (*rg.abort) { ok = false; break; }
    if (lane == 0) mbar_arrive_expect_tx(rg.full0 + 8 * st, kKeys * src.key_bytes());
    __syncwarp();
    if (lane < kKeys) {
      int32_t sl = slot;
      if (sl < 0 || sl >= src.num_slots) {
        flag_error(src.err, RA_DEVERR_SLOT);
        sl = 0;
      }
      src.copy(rg.stage0 + st * rg.stage_bytes, key_in_slab, sl, it.group, rg.full0 + 8 * st);
    }
    ++c;
    it = it2;
    s = s2;
    n = n2;
    r = r2;
    slot = slot2;
  }
  if (!ok) {
    if (lane == 0) rg.give_up(src.err);
    // copies this warp issued must land before the CTA leaves
    for (int32_t j = (c > ns ? c - ns : 0); j < c; ++j) mbar_wait(rg.full0 + 8 * (j % ns), (j / ns) & 1);
  }
}

// Merge n partial rows of D floats (lane's V = D / 32 of them) with log2-sum-exps, by the `warps` warps of a row
// (w = 0 .. warps - 1 takes partials w, w + warps, ...): returns this warp's unnormalised sum relative to
// `mrun`, and its weight sum.  lse_at(s) and row_at(s) give partial s.  Partials that hold -inf weigh 0.
template <int V, int AHEAD, class Lse, class Row>
__device__ __forceinline__ void merge_partials(int n, int w, int warps, Lse lse_at, Row row_at, float (&acc)[V],
                                               float& mrun, float& wsum) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  mrun = -INFINITY;
  wsum = 0.f;
  const int mine = n > w ? (n - w + warps - 1) / warps : 0;
  for (int base = 0; base < mine; base += 32) {
    const int cnt = min(32, mine - base);
    const float ls = lane < cnt ? lse_at(w + (base + lane) * warps) : -INFINITY;
    float x[AHEAD][V];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (k < cnt) row_at(w + (base + k) * warps, x[k]);
    float mc = ls;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, off));
    const float mnew = fmaxf(mrun, mc), mref = mnew == -INFINITY ? 0.f : mnew;
    const float sc = ex2(mrun - mref);
    wsum *= sc;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= sc;
    mrun = mnew;
    const float wl = ex2(ls - mref);
    wsum += wl;
    for (int k0 = 0; k0 < cnt; k0 += AHEAD) {
      if (k0 > 0) {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
          if (k0 + k < cnt) row_at(w + (base + k0 + k) * warps, x[k]);
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const float wk = __shfl_sync(0xffffffffu, wl, (k0 + k) & 31);
        if (k0 + k < cnt) {
#pragma unroll
          for (int v = 0; v < V; ++v) acc[v] = fmaf(wk, x[k][v], acc[v]);
        }
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, off);
}

// Join the shares of the `per_row` warps from `warp` on (their sums, references and weights in shared memory).
template <int V>
__device__ __forceinline__ void join_shares(int per_row, int warp, const float (*s_acc)[32 * V], const float* s_m,
                                            const float* s_w, float (&acc)[V], float& wsum) {
  const int lane = threadIdx.x & 31;
  float top = -INFINITY;
  for (int k = 0; k < per_row; ++k) top = fmaxf(top, s_m[warp + k]);
  const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  wsum = 0.f;
  for (int k = 0; k < per_row; ++k) {
    const float f = ex2(s_m[warp + k] - ref);
    wsum = fmaf(f, s_w[warp + k], wsum);
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = fmaf(f, s_acc[warp + k][lane * V + v], acc[v]);
  }
}

// The same for several rows per warp: LPR lanes per row, lane l of a row holding its floats 4 l .. + 4 of every
// 4 * LPR (V = D / LPR of them).  n and the accessors may differ between a warp's rows; `n` 0 for none.  One
// row per warp leaves a warp waiting for one row's loads at a time (~1.7 us a row at the end of a call, when
// nothing else runs); four rows share that wait.
template <int LPR, int V, int AHEAD, class Lse, class Row>
__device__ __forceinline__ void merge_rows(int n, Lse lse_at, Row row_at, float (&acc)[V], float& wsum) {
  const int sub = (threadIdx.x & 31) % LPR;
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  float mrun = -INFINITY;
  wsum = 0.f;
  const int most = __reduce_max_sync(0xffffffffu, n);
  for (int base = 0; base < most; base += LPR) {
    const int cnt = min(LPR, n - base);  // (<= 0 for a row that is done)
    const float ls = sub < cnt ? lse_at(base + sub) : -INFINITY;
    float x[AHEAD][V];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (k < cnt) row_at(base + k, x[k]);
    float mc = ls;
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, off));
    const float mnew = fmaxf(mrun, mc), mref = mnew == -INFINITY ? 0.f : mnew;
    const float sc = ex2(mrun - mref);
    wsum *= sc;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= sc;
    mrun = mnew;
    const float wl = ex2(ls - mref);
    wsum += wl;
    const int round = min(LPR, most - base);
    for (int k0 = 0; k0 < round; k0 += AHEAD) {
      if (k0 > 0) {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
          if (k0 + k < cnt) row_at(base + k0 + k, x[k]);
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const float wk = __shfl_sync(0xffffffffu, wl, (k0 + k) % LPR, LPR);
        if (k0 + k < cnt) {
#pragma unroll
          for (int v = 0; v < V; ++v) acc[v] = fmaf(wk, x[k][v], acc[v]);
        }
      }
    }
  }
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, off);
}

// Lane `sub`'s floats of a row (through L2), and its bf16 stores, in merge_rows' layout.
template <int LPR, int V>
__device__ __forceinline__ void load_row_part(const float* row, int sub, float (&x)[V]) {
#pragma unroll
  for (int v = 0; v < V; v += 4) {
    const float4 t = __ldcg(reinterpret_cast<const float4*>(row + v * LPR) + sub);
    x[v] = t.x, x[v + 1] = t.y, x[v + 2] = t.z, x[v + 3] = t.w;
  }
}
template <int LPR, int V>
__device__ __forceinline__ void store_row_part(__nv_bfloat16* row, int sub, const float (&x)[V], float f) {
#pragma unroll
  for (int v = 0; v < V; v += 4)
    *(reinterpret_cast<uint2*>(row + v * LPR) + sub) =
        make_uint2(pack_bf16x2(x[v] * f, x[v + 1] * f), pack_bf16x2(x[v + 2] * f, x[v + 3] * f));
}

template <int V>
__device__ __forceinline__ void load_row_cg(const float* src, float (&x)[V]) {  // through L2
  if constexpr (V == 4) {
    const float4 t = __ldcg(reinterpret_cast<const float4*>(src));
    x[0] = t.x, x[1] = t.y, x[2] = t.z, x[3] = t.w;
  } else {
    const float2 t = __ldcg(reinterpret_cast<const float2*>(src));
    x[0] = t.x, x[1] = t.y;
  }
}

}  // namespace ra
