// tree_narrow.cu -- the attention pass of ra_tree_attention on items of at most 32 rows per kv head.
//
// Rows are (drafted token, head of the GQA group); an item is a key range and a query tile of one request for a
// group of hpc kv heads.  With R rows a key costs 4 * D bytes and 4 * D * R flop per kv head: up to 32 rows
// that is far under the ~290 flop per byte at which GB300's tensor cores would bound it, and HBM is the bound.  So
// the kernel is built like the decode one: copies of whole slot rows of a head group (hpc * D * 2 bytes, one
// bulk copy for K and one for V of a key) into a ring, and consumer warps on mma.sync, which take 16 rows of one
// head each: row_blocks warps share a head's keys in shared memory (D = 128: up to 8 warps, 8 heads of 16 rows or
// 4 of 32; D = 64: up to 16).  A tcgen05 tile would have 128 rows, and its swizzled operand layout would force 128-byte copies.
//
// Per warp: S = Q K^T with Q in registers (A) and K read by ldmatrix (B, keys as columns), online softmax with a
// lazy reference per row (reduced over the 4 lanes of a row), P packed from the score fragments into A
// fragments, O += P V with V read by transposing ldmatrix.  Ring rows are 16 bytes past a multiple of 128, so
// ldmatrix is free of bank conflicts.
#include <type_traits>

#include "api_common.h"
#include "slab_ring.cuh"
#include "tree_internal.h"

namespace ra {

namespace {

constexpr float kRescale = 8.0f;  // log2 units: a row's reference moves when a score exceeds it by more

struct NarrowParams {
  TreeParams t;
  int32_t row_bytes;    // hpc * D * 2
  int32_t row_stride;   // + 16
  int32_t nstage;
  int32_t stage_bytes;  // 2 * SLAB * row_stride
};

struct NarrowItem {
  int32_t k0, k1, slot, P, T, row, hg;
  int32_t q0, tokens;  // the tile's first query row and tokens
  int32_t mark;  // index of the item's marks / hkv: its request, or a small call's piece
};

// The items of a call: the plan kernel's list, or (SMALL = 1 or 2 query tiles per lane) this warp's own plan.
struct ListedItems {
  const TreeParams& p;
  __device__ __forceinline__ ListedItems(const TreeParams& q, bool) : p(q) {}
  __device__ __forceinline__ int32_t count() const { return __ldg(p.ws.header) * p.sh.heads; }
  __device__ __forceinline__ void item(int32_t idx, NarrowItem& it) const {
    const int32_t rest = idx / p.sh.heads;
    it.hg = idx - rest * p.sh.heads;
    const int4 e = __ldg(reinterpret_cast<const int4*>(p.ws.items) + 2 * rest);
    const int4 f = __ldg(reinterpret_cast<const int4*>(p.ws.items) + 2 * rest + 1);
    const int32_t chunk = __ldg(p.ws.header + 2);
    const int32_t t0 = e.y * p.sh.tokens_per_item;
    it.P = f.x, it.T = f.y, it.row = f.z, it.q0 = f.w + t0;
    it.tokens = min(p.sh.tokens_per_item, f.y - t0);
    it.slot = e.w;
    it.mark = e.x;
    it.k0 = e.z * chunk;
    it.k1 = min(f.x + f.y, it.k0 + chunk);
  }
};
template <int N>
struct SmallItems {
  const TreeParams& p;
  TreeSmall<N> small;
  __device__ __forceinline__ SmallItems(const TreeParams& q, bool report)
      : p(q), small(q, kTreeSms * q.sh.per_sm, report) {}
  __device__ __forceinline__ int32_t count() const { return small.plan.n * p.sh.heads; }
  __device__ __forceinline__ void item(int32_t idx, NarrowItem& it) const {  // warp-collective
    const int32_t d = idx / p.sh.heads;
    it.hg = idx - d * p.sh.heads;
    const int32_t b = small.plan.request(d), split = d - of_request(small.plan.first, b);  // (b: a request's tile)
    it.P = of_request(small.P, b), it.T = of_request(small.T, b), it.row = of_request(small.row, b);
    it.q0 = of_request(small.q0, b), it.tokens = of_request(small.tokens, b);
    it.slot = of_request(small.plan.pieces, b) > 1 ? d : -1;
    it.mark = d;
    it.k0 = split * small.plan.chunk;
    it.k1 = min(it.P + it.T, it.k0 + small.plan.chunk);
  }
};

// The producers' view: K row and V row of a key for the item's head group.
template <int SLAB, class Items>
struct NarrowSource {
  const NarrowParams& n;
  const Items& items;
  int32_t* counter;
  int64_t num_slots;
  uint32_t* err;
  __device__ __forceinline__ NarrowSource(const NarrowParams& q, const Items& i)
      : n(q), items(i), counter(q.t.ws.header + 1), num_slots(q.t.num_slots), err(q.t.err) {}
  __device__ __forceinline__ int32_t claims() const { return items.count(); }
  __device__ __forceinline__ void item(int32_t idx, SlabKeys& k) const {
    NarrowItem it;
    items.item(idx, it);
    k = SlabKeys{n.t.table + static_cast<int64_t>(it.row) * n.t.table_stride, it.k0, it.k1, it.hg};
  }
  __device__ __forceinline__ uint32_t key_bytes() const { return 2 * n.row_bytes; }
  __device__ __forceinline__ void copy(uint32_t stage, int key, int32_t slot, int32_t group, uint32_t bar) const {
    // a slot's row holds heads * row_bytes bytes
    const int64_t at = (static_cast<int64_t>(slot) * n.t.sh.heads + group) * n.row_bytes;
    bulk_g2s(stage + key * n.row_stride, reinterpret_cast<const uint8_t*>(n.t.k_pool) + at, n.row_bytes, bar);
    bulk_g2s(stage + (SLAB + key) * n.row_stride, reinterpret_cast<const uint8_t*>(n.t.v_pool) + at, n.row_bytes, bar);
  }
};

template <int D, int SLAB, int SMALL>
__global__ void __launch_bounds__(32 * (tree_consumers(D) + kRingProducers), 1)
    tree_narrow_kernel(const __grid_constant__ NarrowParams n) {
  const TreeParams& p = n.t;
  constexpr int KT = D / 16;     // k steps of the scores
  constexpr int NB = SLAB / 8;   // 8-key blocks of a slab
  constexpr int OB = D / 8;      // 8-value blocks of the output
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int nc = p.sh.hpc * p.sh.row_blocks;  // consumer warps at work
  const int RS = n.row_stride;
  const SlabRing rg(smem, n.nstage, n.stage_bytes);
  if (threadIdx.x == 0) rg.init(nc, nc);
  __syncthreads();
  griddep_wait();  // the plan and everything before it
  griddep_launch();
  using Items = std::conditional_t<SMALL != 0, SmallItems<SMALL ? SMALL : 1>, ListedItems>;
  const Items items(p, blockIdx.x == 0 && warp == 0);
  if (warp >= nc) {
    if (warp < nc + kRingProducers) slab_producer<SLAB>(rg, NarrowSource<SLAB, Items>(n, items), warp - nc);
    return;
  }
  // ================================================================ consumers
  const int g = lane >> 2, tq = lane & 3;
  const int hl = warp / p.sh.row_blocks, rb = warp - hl * p.sh.row_blocks;
  const int r0 = rb * 16 + g, r1 = r0 + 8;  // this lane's rows of the head
  // ldmatrix lane addresses within a 16-key block: K (keys x d, plain), V (keys x d, transposing)
  const uint32_t k_off = ((lane & 7) + ((lane >> 4) << 3)) * RS + ((lane >> 3) & 1) * 16 + hl * D * 2;
  const uint32_t v_off = (SLAB + (lane & 15)) * RS + (lane >> 4) * 16 + hl * D * 2;
  int32_t i = 0, c = 0;
  bool clean = false;
  for (;; ++i) {
    const int32_t idx = rg.entry(i);
    if (idx < 0) {
      clean = idx == -1;
      break;
    }
    NarrowItem it;
    items.item(idx, it);
    __syncwarp();
    if (lane == 0) mbar_arrive(rg.free0 + 8 * (i % kRingEntries));  // this warp has read the entry
    const int kh = it.hg * p.sh.hpc + hl;
    const int32_t rows = it.tokens * p.group;
    const bool live0 = r0 < rows, live1 = r1 < rows;
    const bool busy = rb * 16 < rows;  // a block past the request's rows only keeps the barriers' counts
    const int32_t t0 = r0 / p.group, t1 = r1 / p.group;
    // this lane's rows of q and o: (q0 + t) * hq + kh * G + head of the group
    const int64_t row0 = (it.q0 + static_cast<int64_t>(live0 ? t0 : 0)) * p.hq + kh * p.group + (live0 ? r0 - t0 * p.group : 0);
    const int64_t row1 = (it.q0 + static_cast<int64_t>(live1 ? t1 : 0)) * p.hq + kh * p.group + (live1 ? r1 - t1 * p.group : 0);
    uint32_t qf[KT][4];
    if (busy) {
      const uint32_t* q0p = reinterpret_cast<const uint32_t*>(p.q + row0 * D) + tq;
      const uint32_t* q1p = reinterpret_cast<const uint32_t*>(p.q + row1 * D) + tq;
#pragma unroll
      for (int kk = 0; kk < KT; ++kk) {
        qf[kk][0] = live0 ? __ldg(q0p + 8 * kk) : 0u;
        qf[kk][1] = live1 ? __ldg(q1p + 8 * kk) : 0u;
        qf[kk][2] = live0 ? __ldg(q0p + 8 * kk + 4) : 0u;
        qf[kk][3] = live1 ? __ldg(q1p + 8 * kk + 4) : 0u;
      }
    }
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float acc[OB][4];
#pragma unroll
    for (int j = 0; j < OB; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    const int32_t n_slabs = (it.k1 - it.k0 + SLAB - 1) / SLAB;
    bool ok = true;
    bool odd = false;  // this warp cleared a drafted token's V value that was not finite
    for (int32_t s = 0; s < n_slabs; ++s, ++c) {
      const int st = c % rg.nstage;
      if (!mbar_wait(rg.full0 + 8 * st, (c / rg.nstage) & 1)) { ok = false; break; }
      if (busy) {
        const uint32_t stage = rg.stage0 + st * rg.stage_bytes;
        const int32_t key0 = it.k0 + s * SLAB;
        if (key0 + SLAB > it.P) {
          // Drafted tokens' V values that are not finite would reach rows that do not see them through their zero
          // probability: they are set to 0 here, and the merge kernel adds them to the rows that see them.  (Prefix
          // tokens of the slab stay as they are.)  Both warps of a head do this, each before its own product: a
          // value that one of them finds already cleared is cleared for both, and whichever found it marks it.
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < SLAB / 16 * (D / 16); ++e) {
            uint32_t w[4];
            ldsm_x4(stage + v_off + (e / (D / 16)) * 16 * RS + (e % (D / 16)) * 32, w[0], w[1], w[2], w[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) top = __vmaxu2(top, w[k] & 0x7fff7fffu);
          }
          if (__any_sync(0xffffffffu, (top & 0xffffu) >= 0x7f80u || (top >> 16) >= 0x7f80u)) {
            const uint32_t v0 = stage + SLAB * RS + hl * D * 2;
            bool cleared = false;
#pragma unroll 1
            for (int e = lane; e < SLAB * (D / 8); e += 32)
              if (key0 + e / (D / 8) >= it.P)
                cleared = zero_not_finite_bf16x8(v0 + e / (D / 8) * RS + e % (D / 8) * 16) || cleared;
            fence_proxy_async_smem();  // the stage's next copies come through the async proxy
            __syncwarp();
            odd = __any_sync(0xffffffffu, cleared) || odd;
          }
        }
        float x[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b) x[b][0] = x[b][1] = x[b][2] = x[b][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) {
#pragma unroll
          for (int b = 0; b < NB; b += 2) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4(stage + k_off + b * 8 * RS + kk * 32, b0, b1, b2, b3);
            mma_bf16_16816(x[b], qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3], b0, b1);
            mma_bf16_16816(x[b + 1], qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3], b2, b3);
          }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[b][e] *= p.scale_log2;
        if (key0 + SLAB > it.P) {
          // a slab with drafted tokens (or past them): bit k of vis = key key0 + k is visible to the row
          auto visible = [&](int32_t tok, bool live) -> uint32_t {
            const uint32_t* mrow = p.mask + (it.q0 + static_cast<int64_t>(live ? tok : 0)) * p.mask_words;
            auto word = [&](int32_t w) -> uint32_t {
              const int32_t left = it.T - 32 * w;
              if (left <= 0 || !live) return 0u;
              const uint32_t bits = __ldg(mrow + w);
              return left >= 32 ? bits : bits & ((1u << left) - 1u);
            };
            const int32_t off = key0 - it.P;
            if (off >= 0) return __funnelshift_r(word(off >> 5), word((off >> 5) + 1), off & 31);
            return off <= -32 ? 0xffffffffu : (word(0) << -off) | ((1u << -off) - 1u);
          };
          const uint32_t vis0 = visible(t0, live0), vis1 = visible(t1, live1);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint32_t w0 = vis0 >> (8 * b + 2 * tq), w1 = vis1 >> (8 * b + 2 * tq);
            if (!(w0 & 1u)) x[b][0] = -INFINITY;
            if (!(w0 & 2u)) x[b][1] = -INFINITY;
            if (!(w1 & 1u)) x[b][2] = -INFINITY;
            if (!(w1 & 2u)) x[b][3] = -INFINITY;
          }
        }
        float mx0 = fmaxf(x[0][0], x[0][1]), mx1 = fmaxf(x[0][2], x[0][3]);
#pragma unroll
        for (int b = 1; b < NB; ++b) {
          mx0 = fmaxf(mx0, fmaxf(x[b][0], x[b][1]));
          mx1 = fmaxf(mx1, fmaxf(x[b][2], x[b][3]));
        }
        // lazy reference: it moves only when a score of the slab exceeds it by more than kRescale
        if (__any_sync(0xffffffffu, mx0 > m0 + kRescale || mx1 > m1 + kRescale)) {
#pragma unroll
          for (int off = 1; off < 4; off <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
          }
          mx0 = fmaxf(m0, mx0);
          mx1 = fmaxf(m1, mx1);
          // (a row that has seen nothing yet keeps -inf: l and O are 0 then)
          const float al0 = mx0 == -INFINITY ? 1.f : ex2(m0 - mx0), al1 = mx1 == -INFINITY ? 1.f : ex2(m1 - mx1);
          m0 = mx0, m1 = mx1;
          l0 *= al0;
          l1 *= al1;
#pragma unroll
          for (int j = 0; j < OB; ++j) {
            acc[j][0] *= al0;
            acc[j][1] *= al0;
            acc[j][2] *= al1;
            acc[j][3] *= al1;
          }
        }
        const float s0 = m0 == -INFINITY ? 0.f : m0, s1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          x[b][0] = ex2(x[b][0] - s0);
          x[b][1] = ex2(x[b][1] - s0);
          x[b][2] = ex2(x[b][2] - s1);
          x[b][3] = ex2(x[b][3] - s1);
          l0 += x[b][0] + x[b][1];
          l1 += x[b][2] + x[b][3];
        }
#pragma unroll
        for (int b = 0; b < NB; b += 2) {
          const uint32_t a0 = pack_bf16x2(x[b][0], x[b][1]), a1 = pack_bf16x2(x[b][2], x[b][3]);
          const uint32_t a2 = pack_bf16x2(x[b + 1][0], x[b + 1][1]), a3 = pack_bf16x2(x[b + 1][2], x[b + 1][3]);
#pragma unroll
          for (int j = 0; j < OB; j += 2) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4_trans(stage + v_off + b * 8 * RS + j * 16, b0, b1, b2, b3);
            mma_bf16_16816(acc[j], a0, a1, a2, a3, b0, b1);
            mma_bf16_16816(acc[j + 1], a0, a1, a2, a3, b2, b3);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(rg.empty0 + 8 * st);
    }
    if (!ok) break;
    // listed items add to marks the plan kernel cleared; a small call's piece writes its own, each of a head's two warps
    // a half of it
    if (lane == 0 && (SMALL || odd)) {
      int32_t* mark = p.ws.bad + static_cast<int64_t>(it.mark) * p.hkv + kh;
      if (SMALL && p.sh.row_blocks == 2) reinterpret_cast<uint16_t*>(mark)[rb] = odd;
      else *mark = odd;
    }
    if (!busy) continue;
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    // a row that sees nothing gives 0 (as a partial: weight 2^-inf)
    const float i0 = l0 == 0.f ? 0.f : 1.f / l0, i1 = l1 == 0.f ? 0.f : 1.f / l1;
    if (it.slot < 0) {
#pragma unroll
      for (int j = 0; j < OB; ++j) {
        const int d = 8 * j + 2 * tq;
        if (live0) *reinterpret_cast<uint32_t*>(p.o + row0 * D + d) = pack_bf16x2(acc[j][0] * i0, acc[j][1] * i0);
        if (live1) *reinterpret_cast<uint32_t*>(p.o + row1 * D + d) = pack_bf16x2(acc[j][2] * i1, acc[j][3] * i1);
      }
    } else {
      const int64_t ps = (static_cast<int64_t>(it.slot) * p.hkv + kh) * p.ws.part_rows;
#pragma unroll
      for (int j = 0; j < OB; ++j) {
        const int d = 8 * j + 2 * tq;
        if (live0) *reinterpret_cast<float2*>(p.ws.part_o + (ps + r0) * D + d) = make_float2(acc[j][0] * i0, acc[j][1] * i0);
        if (live1) *reinterpret_cast<float2*>(p.ws.part_o + (ps + r1) * D + d) = make_float2(acc[j][2] * i1, acc[j][3] * i1);
      }
      if (tq == 0) {
        if (live0) p.ws.part_lse[ps + r0] = m0 + __log2f(l0);
        if (live1) p.ws.part_lse[ps + r1] = m1 + __log2f(l1);
      }
    }
  }
  if (!clean && lane == 0) rg.give_up(p.err);  // a bounded wait ran out: stop the producers as well
}

int32_t stage_bytes(int32_t hpc, int32_t head_dim, int32_t slab) { return 2 * slab * (hpc * head_dim * 2 + 16); }
int32_t ring_bytes(int32_t per_sm) { return kRingSmemLimit / per_sm - 1024 - kRingHdrBytes; }  // (1 KB per CTA is the system's)

template <int D, int SLAB, int SMALL>
ra_status launch(const TreeParams& p, const DeviceInfo& dev, cudaStream_t s) {
  NarrowParams n{};
  n.t = p;
  n.row_bytes = p.sh.hpc * D * 2;
  n.row_stride = n.row_bytes + 16;
  n.stage_bytes = stage_bytes(p.sh.hpc, D, SLAB);
  n.nstage = ring_bytes(p.sh.per_sm) / n.stage_bytes;
  if (n.nstage > kRingMaxStages) n.nstage = kRingMaxStages;
  const int smem = kRingHdrBytes + n.nstage * n.stage_bytes;
  auto kern = tree_narrow_kernel<D, SLAB, SMALL>;
  static bool configured[64] = {};
  if (!configured[dev.device]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmemLimit);
    if (e != cudaSuccess) return fail(RA_ERR_CUDA, "cudaFuncSetAttribute(tree): %s", cudaGetErrorString(e));
    configured[dev.device] = true;
  }
  const int64_t items = p.ws.cap * p.sh.heads;
  const int64_t ctas = static_cast<int64_t>(SMALL ? kTreeSms : dev.num_sms) * p.sh.per_sm;
  const int grid = static_cast<int>(SMALL || items >= ctas ? ctas : items);
  return launch_pdl("tree_narrow_kernel", kern, dim3(grid),
                    dim3(32 * (p.sh.hpc * p.sh.row_blocks + kRingProducers)), smem, s, n);
}

template <int D, int SLAB>
ra_status launch_items(const TreeParams& p, int small, const DeviceInfo& dev, cudaStream_t s) {
  return small == 0 ? launch<D, SLAB, 0>(p, dev, s) : small == 1 ? launch<D, SLAB, 1>(p, dev, s) : launch<D, SLAB, 2>(p, dev, s);
}

}  // namespace

// 32-key slabs where two of them fit the ring, else 16-key ones (64 x 8 tokens over 512..4096 keys, 32- and 16-key
// slabs: 16/16 heads of 64, where one fits, 118.3 and 106.5 us; 12/12, where two do, 84.6 and 87.3; 5/5 heads of
// 128, two, 77.2 and 81.8).
ra_status launch_tree_narrow(const TreeParams& p, int32_t head_dim, int small, const DeviceInfo& dev, cudaStream_t s) {
  const bool wide = 2 * stage_bytes(p.sh.hpc, head_dim, 32) <= ring_bytes(p.sh.per_sm);
  if (head_dim == 64) return wide ? launch_items<64, 32>(p, small, dev, s) : launch_items<64, 16>(p, small, dev, s);
  return wide ? launch_items<128, 32>(p, small, dev, s) : launch_items<128, 16>(p, small, dev, s);
}

}  // namespace ra
