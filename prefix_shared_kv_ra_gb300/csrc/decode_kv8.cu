// decode_kv8.cu -- ra_kv8_decode_attention: split-KV GQA decode over a quantised pool.
//
// The same call as ra_decode_attention (plan kernel, persistent split-KV kernel, log-sum-exp combine), on
// records of e4m3 codes: a key costs about 2 * Hkv * D bytes instead of 4 * Hkv * D, and that HBM stream is
// the bound (4 flop per byte and q head of the group).  The codes go to the tensor cores as f16, which holds
// them exactly, and the products are accumulated in fp32:
//
//   x_j = sm_scale * log2(e) * 2^ek_j * <q, ck_j>             (scores, log2 domain)
//   l   = sum_j 2^(x_j - m),   O = sum_j 2^(x_j + ev_j - w) cv_j,   o = O * 2^(w - m) / l
//
// with ek_j, ev_j the exponents of key j's K and V rows and m, w two lazy references (of x_j and of
// x_j + ev_j): the V scale joins the softmax's exponent, so the weights that are rounded to f16 for the PV
// product lie within 2^8 of 1 whatever the scales are (f16: 2^-12 relative above 2^-14, 2^-25 absolute
// below, both far under the bf16 output's 2^-9).  q is multiplied by a power of two that puts its largest
// value at 2^14 and rounded to f16: exact for values down to 2^-28 of the largest.
//
// Fragments need no ldmatrix and no transpose: both contractions may take their index in any order, so
// each lane loads contiguous bytes of a row (32 of K, 16 of V at D = 128) and converts them where they are:
//  * S^T[16 keys x 8 heads] = K Q^T: lane (g, t) takes d = t * D/4 .. of keys g and g + 8; the k index of
//    the MMA is d permuted, and q's fragment is loaded in the same order;
//  * O^T[16 d x 8 heads] += V^T P^T: lane (g, t) takes d = g * D/8 .. of keys 2t, 2t+1, 2t+8, 2t+9; byte
//    permutes pair the two keys of one d, and MMA m covers d = g * D/8 + 2m (row g) and + 1 (row g + 8).
// A lane thus ends with D/8 consecutive d of two heads, stored as vectors.  A ring stage's rows are
// hpc * 2 * D + 16 bytes apart (the record's block): every fragment load is free of bank conflicts at
// D = 128.
#include <math.h>

#include "api_common.h"
#include "decode_internal.h"
#include "decode_item.cuh"
#include "kv8.cuh"
#include "ra_ptx.cuh"
#include "slab_ring.cuh"
#include "small_plan.cuh"

namespace ra {

namespace {

// Keys per ring stage.  A consumer warp's chain of loads, scores, softmax and product takes about as long for a
// slab of either size, so heads of 64 and groups of few heads get the longer one (150 requests of 1000..9000 keys:
// 8/8 heads of 64 170 us with 32, 136 with 64; 16/4 heads of 128 166 and 136).  Heads of 128 need 160 registers
// for it, so larger groups keep the short one, and so do the ones of which two CTAs share an SM.
constexpr int kFewHeads = 4;
constexpr int ctas_per_sm(int head_dim, int hpc) { return hpc <= (head_dim == 64 ? 3 : 2) ? 2 : 1; }
constexpr int slab_of(int head_dim, int hpc) {
  return head_dim == 64 || (hpc <= kFewHeads && ctas_per_sm(head_dim, hpc) == 1) ? 64 : 32;
}
constexpr float kRescale = 8.0f;   // log2 units: a reference moves when a score exceeds it by more
constexpr int kQExp = 14;          // q's largest value in f16

struct Kv8DecodeParams {
  DecodeParams d;
  const uint8_t* pool;
  int64_t slot_bytes;
  int32_t block_bytes;
  int32_t ctas;  // small call: the grid
};
constexpr int kSmallLeast = 2;  // units of a small call's shortest piece

// The items of a call: the plan kernel's list, or (SMALL = 1 or 2 requests per lane) this warp's own plan.
template <int SMALL>
struct Kv8Items {
  const DecodeParams& p;
  SmallPlan<SMALL ? SMALL : 1> plan;
  PerRequest<SMALL ? SMALL : 1> len, row;

  __device__ __forceinline__ Kv8Items(const DecodeParams& q, int32_t ctas, bool report) : p(q) {
    if constexpr (SMALL) {
      auto request = [&](int32_t b, int32_t& l, int32_t& r) {
        if (b >= p.batch) return;
        r = __ldg(p.rpi + b);
        l = __ldg(p.seq_lens + b);
        const bool bad_row = r < 0 || r >= p.table_rows, bad_len = l < 1 || l > p.max_seq_len;
        if (report && bad_row) flag_error(p.err, RA_DEVERR_TABLE);
        else if (report && bad_len) flag_error(p.err, RA_DEVERR_LENGTH);
        l = bad_row || l < 1 ? 0 : min(l, p.max_seq_len);
      };
#pragma unroll
      for (int i = 0; i < SMALL; ++i) request(static_cast<int32_t>(threadIdx.x & 31) + 32 * i, len.v[i], row.v[i]);
      plan.make(len, p.n_hgroups, ctas, kSmallLeast);
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
      it.start = 0;
      it.k0 = it.split * plan.chunk;
      it.k1 = min(of_request(len, it.b), it.k0 + plan.chunk);
    } else {
      decode_item(p, idx, it);
    }
  }
};

// The producers' view: one bulk copy per key, the head group's block of the slot's record.
template <int SMALL>
struct Kv8Source {
  const Kv8DecodeParams& pp;
  const Kv8Items<SMALL>& items;
  int32_t* counter;
  int64_t num_slots;
  uint32_t* err;
  __device__ __forceinline__ Kv8Source(const Kv8DecodeParams& q, const Kv8Items<SMALL>& it)
      : pp(q), items(it), counter(q.d.counter), num_slots(q.d.num_slots), err(q.d.err) {}
  __device__ __forceinline__ int32_t claims() const { return items.count(); }
  __device__ __forceinline__ void item(int32_t idx, SlabKeys& k) const {
    Item it;
    items.item(idx, it);
    k = SlabKeys{pp.d.table + static_cast<int64_t>(it.row) * pp.d.table_stride, it.k0, it.k1, it.hg};
  }
  __device__ __forceinline__ uint32_t key_bytes() const { return pp.block_bytes; }
  __device__ __forceinline__ void copy(uint32_t stage, int key, int32_t slot, int32_t group, uint32_t bar) const {
    bulk_g2s(stage + key * pp.block_bytes,
             pp.pool + static_cast<int64_t>(slot) * pp.slot_bytes + static_cast<int64_t>(group) * pp.block_bytes,
             pp.block_bytes, bar);
  }
};

// D[16x8] += A[16x16] (row) * B[16x8] (col), f16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// N 32-bit words from shared memory, 4 N bytes aligned to min(16, 4 N).
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 2) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                   : "r"(addr + 4 * i)
                   : "memory");
  }
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}

// Warp roles: hpc consumer warps (one kv head each), the ring's copy warps, and a signal warp that counts each
// request's finished partials for the combine and frees the item entries.
template <int D, int kSlab, int SMALL>
__global__ void __launch_bounds__(32 * ((D == 128 && kSlab == 64 ? kFewHeads : kMaxHeadsPerCta) + kRingProducers + 1), 1)
    kv8_decode_kernel(const __grid_constant__ Kv8DecodeParams pp) {
  const DecodeParams& p = pp.d;
  constexpr int KW = D / 16;  // words of a K row per lane = MMA k steps of the scores
  constexpr int VW = D / 32;  // words of a V row per lane
  constexpr int MT = D / 16;  // MMA m tiles of O^T
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int nc = p.hpc;
  const int RS = p.row_stride;
  const SlabRing rg(smem, p.nstage, p.stage_bytes);
  if (threadIdx.x == 0) rg.init(nc, 1);
  __syncthreads();
  griddep_wait();  // the plan, its reset counters and everything before them are complete
  griddep_launch();  // the combine may launch: it waits per request for the partials it merges

  if (warp > nc + kRingProducers) return;
  const Kv8Items<SMALL> items(p, pp.ctas, blockIdx.x == 0 && warp == 0);
  if (warp >= nc && warp < nc + kRingProducers) {
    slab_producer<kSlab>(rg, Kv8Source<SMALL>(pp, items), warp - nc);
    return;
  }
  if (warp == nc + kRingProducers) {
    if constexpr (!SMALL) {  // (a small call has one item per CTA, and its merge waits for the grid)
      // ================================================================ signaller
      // (the item's request is looked up while the item is at work: the signal that follows its last store is on
      // the way of the merge)
      for (int32_t n = 0;; ++n) {
        const int e = n % kRingEntries;
        const int32_t idx = rg.entry(n);
        int32_t* count = nullptr;  // the request's count, if its partials are merged by the combine
        if (idx >= 0 && lane == 0) {
          Item it;
          decode_item(p, idx, it);
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
  const int g = lane >> 2;
  const int tq = lane & 3;
  const uint32_t k_off = g * RS + warp * 2 * D + tq * (D / 4);
  const uint32_t v_off = 2 * tq * RS + warp * 2 * D + D + g * (D / 8);
  const uint32_t s_off = g * RS + nc * 2 * D + 2 * warp;  // exponent bytes of key g, this head
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
    const int kh = it.hg * p.hpc + warp;
    // Q^T fragments (B operand): column g is q head kh*G + g, scaled to f16
    uint32_t qf[KW][2];
    float c0, c1;  // score factors of heads 2 tq and 2 tq + 1
    {
      const bool live = g < p.group;
      const uint4* qrow = reinterpret_cast<const uint4*>(
          p.q + (static_cast<int64_t>(it.b) * p.hq + kh * p.group + (live ? g : 0)) * D + tq * (D / 4));
      uint32_t raw[D / 8];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint4 v = __ldg(qrow + i);
        if (!live) v = make_uint4(0, 0, 0, 0);
        raw[4 * i] = v.x, raw[4 * i + 1] = v.y, raw[4 * i + 2] = v.z, raw[4 * i + 3] = v.w;
      }
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(raw[i])), fabsf(bf16_hi(raw[i]))));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int32_t e = max(static_cast<int32_t>(__float_as_uint(mx) >> 23) - 127, -100);
      const float up = pow2f(kQExp - e);
#pragma unroll
      for (int j = 0; j < KW; ++j) {
        qf[j][0] = pack_f16x2(bf16_lo(raw[2 * j]) * up, bf16_hi(raw[2 * j]) * up);
        qf[j][1] = pack_f16x2(bf16_lo(raw[2 * j + 1]) * up, bf16_hi(raw[2 * j + 1]) * up);
      }
      c0 = p.scale_log2 * pow2f(__shfl_sync(0xffffffffu, e, 8 * tq) - kQExp);
      c1 = p.scale_log2 * pow2f(__shfl_sync(0xffffffffu, e, 8 * tq + 4) - kQExp);
    }
    float m0 = -INFINITY, m1 = -INFINITY, w0 = -INFINITY, w1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float acc[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
    const int32_t n_slabs = (it.k1 - it.k0 + kSlab - 1) / kSlab;
    bool ok = true;
    for (int32_t s = 0; s < n_slabs; ++s, ++c) {
      const int st = c % rg.nstage;
      if (!mbar_wait(rg.full0 + 8 * st, (c / rg.nstage) & 1)) { ok = false; break; }
      const uint32_t stage = rg.stage0 + st * rg.stage_bytes;
      // S^T[16 keys x 8 heads] = K Q^T for the slab's halves
      float x[kSlab / 16][4], y[kSlab / 16][4];
#pragma unroll
      for (int hf = 0; hf < kSlab / 16; ++hf) {
        const uint32_t base = stage + hf * 16 * RS;
        uint32_t a[KW], b[KW];
        lds_words<KW>(base + k_off, a);
        lds_words<KW>(base + k_off + 8 * RS, b);
        const uint32_t e_lo = lds_u16(base + s_off), e_hi = lds_u16(base + s_off + 8 * RS);
        float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < KW; ++j)
          mma_f16_16816(sc, e4m3x2_to_f16x2(a[j]), e4m3x2_to_f16x2(b[j]), e4m3x2_hi_to_f16x2(a[j]),
                        e4m3x2_hi_to_f16x2(b[j]), qf[j][0], qf[j][1]);
        const int32_t key = it.k0 + s * kSlab + hf * 16 + g;
        const bool v_lo = key < it.k1, v_hi = key + 8 < it.k1;
        const float k_lo = __uint_as_float((e_lo & 255u) << 23), k_hi = __uint_as_float((e_hi & 255u) << 23);
        const float f_lo = static_cast<float>(static_cast<int32_t>(e_lo >> 8) - 127);
        const float f_hi = static_cast<float>(static_cast<int32_t>(e_hi >> 8) - 127);
        x[hf][0] = v_lo ? sc[0] * c0 * k_lo : -INFINITY;
        x[hf][1] = v_lo ? sc[1] * c1 * k_lo : -INFINITY;
        x[hf][2] = v_hi ? sc[2] * c0 * k_hi : -INFINITY;
        x[hf][3] = v_hi ? sc[3] * c1 * k_hi : -INFINITY;
        y[hf][0] = x[hf][0] + f_lo;
        y[hf][1] = x[hf][1] + f_lo;
        y[hf][2] = x[hf][2] + f_hi;
        y[hf][3] = x[hf][3] + f_hi;
      }
      // Lazy references, as in the bf16 kernel: both move, and O and l are rescaled, only when a value of the
      // slab exceeds its reference by more than kRescale; an item's first slab always moves them (its first
      // key is in range, so the maxima are finite).
      bool above = false;
#pragma unroll
      for (int hf = 0; hf < kSlab / 16; ++hf)
        above = above || x[hf][0] > m0 + kRescale || x[hf][2] > m0 + kRescale || x[hf][1] > m1 + kRescale ||
                x[hf][3] > m1 + kRescale || y[hf][0] > w0 + kRescale || y[hf][2] > w0 + kRescale ||
                y[hf][1] > w1 + kRescale || y[hf][3] > w1 + kRescale;
      if (__any_sync(0xffffffffu, above)) {
        float mx0 = m0, mx1 = m1, wx0 = w0, wx1 = w1;
#pragma unroll
        for (int hf = 0; hf < kSlab / 16; ++hf) {
          mx0 = fmaxf(mx0, fmaxf(x[hf][0], x[hf][2]));
          mx1 = fmaxf(mx1, fmaxf(x[hf][1], x[hf][3]));
          wx0 = fmaxf(wx0, fmaxf(y[hf][0], y[hf][2]));
          wx1 = fmaxf(wx1, fmaxf(y[hf][1], y[hf][3]));
        }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
          wx0 = fmaxf(wx0, __shfl_xor_sync(0xffffffffu, wx0, off));
          wx1 = fmaxf(wx1, __shfl_xor_sync(0xffffffffu, wx1, off));
        }
        l0 *= ex2(m0 - mx0);
        l1 *= ex2(m1 - mx1);
        const float al0 = ex2(w0 - wx0), al1 = ex2(w1 - wx1);
        m0 = mx0, m1 = mx1, w0 = wx0, w1 = wx1;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          acc[mt][0] *= al0;
          acc[mt][1] *= al1;
          acc[mt][2] *= al0;
          acc[mt][3] *= al1;
        }
      }
#pragma unroll
      for (int hf = 0; hf < kSlab / 16; ++hf) {
        l0 += ex2(x[hf][0] - m0) + ex2(x[hf][2] - m0);
        l1 += ex2(x[hf][1] - m1) + ex2(x[hf][3] - m1);
        // P^T as the B operand: transpose the two 8x8 key blocks
        const uint32_t pb0 = movmatrix_trans(pack_f16x2(ex2(y[hf][0] - w0), ex2(y[hf][1] - w1)));
        const uint32_t pb1 = movmatrix_trans(pack_f16x2(ex2(y[hf][2] - w0), ex2(y[hf][3] - w1)));
        const uint32_t base = stage + hf * 16 * RS + v_off;
        uint32_t v0[VW], v1[VW], v8[VW], v9[VW];
        lds_words<VW>(base, v0);
        lds_words<VW>(base + RS, v1);
        lds_words<VW>(base + 8 * RS, v8);
        lds_words<VW>(base + 9 * RS, v9);
#pragma unroll
        for (int j = 0; j < VW; ++j) {
          const uint32_t lo = __byte_perm(v0[j], v1[j], 0x5140), lo8 = __byte_perm(v8[j], v9[j], 0x5140);
          const uint32_t hi = __byte_perm(v0[j], v1[j], 0x7362), hi8 = __byte_perm(v8[j], v9[j], 0x7362);
          mma_f16_16816(acc[2 * j], e4m3x2_to_f16x2(lo), e4m3x2_hi_to_f16x2(lo), e4m3x2_to_f16x2(lo8),
                        e4m3x2_hi_to_f16x2(lo8), pb0, pb1);
          mma_f16_16816(acc[2 * j + 1], e4m3x2_to_f16x2(hi), e4m3x2_hi_to_f16x2(hi), e4m3x2_to_f16x2(hi8),
                        e4m3x2_hi_to_f16x2(hi8), pb0, pb1);
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
    // the lane's D/8 consecutive d of heads 2 tq and 2 tq + 1; 2^(w - m) in two halves, either of which is finite
    const float h0 = ex2(0.5f * (w0 - m0)), h1 = ex2(0.5f * (w1 - m1));
    const float i0 = h0 / l0, i1 = h1 / l1;
    float o0[D / 8], o1[D / 8];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      o0[2 * mt] = acc[mt][0] * i0 * h0;
      o0[2 * mt + 1] = acc[mt][2] * i0 * h0;
      o1[2 * mt] = acc[mt][1] * i1 * h1;
      o1[2 * mt + 1] = acc[mt][3] * i1 * h1;
    }
    const bool direct = it.n_splits == 1;
    const int64_t row = direct ? static_cast<int64_t>(it.b) : static_cast<int64_t>(it.d);
    const int64_t head0 = row * p.hq + kh * p.group + 2 * tq;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      if (2 * tq + hh >= p.group) continue;
      const float(&o)[D / 8] = hh ? o1 : o0;
      const int64_t at = (head0 + hh) * D + g * (D / 8);
      if (direct) {
        uint4* dst = reinterpret_cast<uint4*>(p.o + at);
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          dst[i] = make_uint4(pack_bf16x2(o[8 * i], o[8 * i + 1]), pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
                              pack_bf16x2(o[8 * i + 4], o[8 * i + 5]), pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
      } else {
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          st_global_v8(p.part_o + at + 8 * i, o[8 * i], o[8 * i + 1], o[8 * i + 2], o[8 * i + 3], o[8 * i + 4],
                       o[8 * i + 5], o[8 * i + 6], o[8 * i + 7]);
        if (g == 0) p.part_lse[head0 + hh] = (hh ? m1 : m0) + __log2f(hh ? l1 : l0);
      }
    }
    // this warp's part of the entry is written (__syncwarp orders the lanes' stores before lane 0's release)
    __syncwarp();
    if (lane == 0) mbar_arrive(rg.done0 + 8 * (n % kRingEntries));
  }
  if (!clean && lane == 0) rg.give_up(p.err);  // a bounded wait ran out: stop the producers as well
}

// Merge the partials of every split request.  Launched while the decode kernel runs: a row (request, q head)
// waits only for its own request's count of finished (item, head group) partials.  Two forms:
//  * many rows: 8 lanes per row, a warp's four rows at once (224 requests of 64 heads: the call ends 12 us after
//    its last item with a row per warp, one after the other);
//  * few rows: `per_row` warps share one, each a part of its partials (32 rows of 108 partials: 18 us with
//    one warp each, 5 us with eight; 73 requests of 64 heads, up to 43 partials a row: 41.5 us with 8 lanes per
//    row, 36.9 with a warp).
constexpr int kCombineWarps = 8;
constexpr int kRowLanes = 8;
constexpr int kRowsPerWarp = 32 / kRowLanes;

// The request's partials, once they are written (a warp's lanes may ask for different requests): their first
// index and number, 0 if its rows were written directly or it is invalid.
__device__ __forceinline__ int32_t wait_partials(const DecodeParams& p, int32_t b, bool in, int32_t& i0) {
  // the plan completed before the decode kernel let this one launch
  const int32_t L = __ldg(p.seq_lens + b), row = __ldg(p.rpi + b);
  i0 = __ldcg(p.req_item0 + b);
  int32_t n = __ldcg(p.req_item0 + b + 1) - i0;
  if (!in || n <= 1 || L < 1 || row < 0 || row >= p.table_rows) n = 0;
  // every lane reads the count itself: with the fence its loads of the partials follow an acquire
  if (n > 0 && !wait_count(p.req_done + b, n * p.n_hgroups)) {
    flag_error(p.err, RA_DEVERR_TIMEOUT);
    n = 0;
  }
  fence_acq_rel_gpu();
  return n;
}

template <int D>
__global__ void __launch_bounds__(32 * kCombineWarps) kv8_combine_kernel(const __grid_constant__ DecodeParams p) {
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
      n, [&](int s) { return __ldcg(p.part_lse + static_cast<int64_t>(i0 + s) * p.hq + h); },
      [&](int s, float(&x)[V]) {
        load_row_part<kRowLanes, V>(p.part_o + (static_cast<int64_t>(i0 + s) * p.hq + h) * D, sub, x);
      },
      acc, wsum);
  if (n > 0) store_row_part<kRowLanes, V>(p.o + static_cast<int64_t>(bh) * D, sub, acc, 1.f / wsum);
  griddep_wait();  // this grid's completion implies the decode kernel's
}

template <int D, int SMALL>
__global__ void __launch_bounds__(32 * kCombineWarps) kv8_combine_few_kernel(const __grid_constant__ DecodeParams p,
                                                                             int per_row, int32_t ctas) {
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
    const Kv8Items<SMALL> items(p, ctas, false);
    i0 = of_request(items.plan.first, b);
    n = of_request(items.plan.pieces, b);
    if (!in || n <= 1) n = 0;  // written directly, or invalid
    griddep_wait();
  } else {
    n = wait_partials(p, b, in, i0);
    __syncwarp();
  }
  float acc[V], m, wsum;
  merge_partials<V, 8>(
      n, share, per_row, [&](int s) { return __ldcg(p.part_lse + static_cast<int64_t>(i0 + s) * p.hq + h); },
      [&](int s, float(&x)[V]) {
        load_row_cg<V>(p.part_o + (static_cast<int64_t>(i0 + s) * p.hq + h) * D + lane * V, x);
      },
      acc, m, wsum);
#pragma unroll
  for (int v = 0; v < V; ++v) s_acc[warp][lane * V + v] = acc[v];
  if (lane == 0) s_m[warp] = m, s_w[warp] = wsum;
  __syncthreads();
  if (n > 0 && share == 0) {
    join_shares<V>(per_row, warp, s_acc, s_m, s_w, acc, wsum);
    const float inv = 1.f / wsum;
    __nv_bfloat16* dst = p.o + static_cast<int64_t>(bh) * D + lane * V;
#pragma unroll
    for (int v = 0; v < V; v += 2)
      *reinterpret_cast<__nv_bfloat162*>(dst + v) = __floats2bfloat162_rn(acc[v] * inv, acc[v + 1] * inv);
  }
  griddep_wait();  // this grid's completion implies the decode kernel's
}

template <int D, int SLAB, int SMALL>
ra_status launch_decode(const Kv8DecodeParams& pp, int grid, int smem, const DeviceInfo& dev, cudaStream_t stream) {
  auto kern = kv8_decode_kernel<D, SLAB, SMALL>;
  static bool configured[64] = {};
  if (!configured[dev.device]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmemLimit);
    if (e != cudaSuccess) return fail(RA_ERR_CUDA, "cudaFuncSetAttribute(kv8 decode): %s", cudaGetErrorString(e));
    configured[dev.device] = true;
  }
  return launch_pdl("kv8_decode_kernel", kern, dim3(grid), dim3(32 * (pp.d.hpc + kRingProducers + 1)), smem, stream, pp);
}

template <int D, int SLAB>
ra_status launch(Kv8DecodeParams& pp, int32_t per_sm, int smem, const DeviceInfo& dev, cudaStream_t s) {
  DecodeParams& p = pp.d;
  const int64_t rows = static_cast<int64_t>(p.batch) * p.hq, warps = static_cast<int64_t>(dev.num_sms) * 3 * kCombineWarps;
  const bool small = small_call(p.batch, p.max_seq_len, p.n_hgroups, per_sm), many = p.batch > 32;
  if (small) {
    pp.ctas = kSmallSms * per_sm;
    if (ra_status st = many ? launch_decode<D, SLAB, 2>(pp, pp.ctas, smem, dev, s)
                            : launch_decode<D, SLAB, 1>(pp, pp.ctas, smem, dev, s))
      return st;
  } else {
    if (ra_status st = launch_decode_plan(p, 0, s)) return st;
    const int64_t n_items = static_cast<int64_t>(p.max_items) * p.n_hgroups;  // bound of the claims
    const int64_t ctas = static_cast<int64_t>(dev.num_sms) * per_sm;
    if (ra_status st = launch_decode<D, SLAB, 0>(pp, static_cast<int>(n_items < ctas ? n_items : ctas), smem, dev, s))
      return st;
  }
  // few rows: as many warps per row as three CTAs per SM hold, or one up to 32 rows per SM (101
  // requests of 64 heads: 20.4 us with 8 lanes per row, 23.3 with a warp)
  int per_row = 1;
  while (per_row < kCombineWarps && rows * per_row * 2 <= warps) per_row *= 2;
  if (per_row > 1 || small || rows <= static_cast<int64_t>(dev.num_sms) * 32) {
    const int64_t ctas = (rows * per_row + kCombineWarps - 1) / kCombineWarps;
    auto kern = !small ? kv8_combine_few_kernel<D, 0> : many ? kv8_combine_few_kernel<D, 2> : kv8_combine_few_kernel<D, 1>;
    return launch_pdl("kv8_combine_few_kernel", kern,
                      dim3(static_cast<unsigned>(ctas)), dim3(32 * kCombineWarps), 0, s, p, per_row, pp.ctas);
  }
  const int64_t per_cta = kCombineWarps * kRowsPerWarp;
  return launch_pdl("kv8_combine_kernel", kv8_combine_kernel<D>, dim3(static_cast<unsigned>((rows + per_cta - 1) / per_cta)),
                    dim3(32 * kCombineWarps), 0, s, p);
}

}  // namespace
}  // namespace ra

extern "C" ra_status ra_kv8_decode_attention(const void* kv8_pool, int64_t num_slots, int32_t num_kv_heads,
                                             int32_t head_dim, const void* q, void* o, int32_t num_q_heads,
                                             float sm_scale, const int32_t* req_to_token, int64_t table_stride,
                                             int64_t table_rows, const int32_t* req_pool_indices,
                                             const int32_t* seq_lens, int32_t batch, int32_t max_seq_len,
                                             void* workspace, size_t workspace_bytes, uint32_t* device_error,
                                             ra_stream_t stream) {
  using namespace ra;
  clear_error();
  RA_REQUIRE(batch >= 0 && batch <= 65535, "batch must be in [0, 65535] (got %d)", batch);
  RA_REQUIRE(num_kv_heads > 0 && num_q_heads > 0, "head counts must be > 0");
  RA_REQUIRE(num_q_heads % num_kv_heads == 0, "num_q_heads (%d) must be a multiple of num_kv_heads (%d)",
             num_q_heads, num_kv_heads);
  RA_REQUIRE(num_slots > 0, "num_slots must be > 0");
  RA_REQUIRE(std::isfinite(sm_scale) && sm_scale > 0.f, "sm_scale must be finite and > 0");
  if (head_dim != 64 && head_dim != 128) return fail(RA_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", head_dim);
  const int32_t group = num_q_heads / num_kv_heads;
  if (group > 8) return fail(RA_ERR_UNSUPPORTED, "GQA group %d (decode supports up to 8)", group);
  if (num_kv_heads > 1024) return fail(RA_ERR_UNSUPPORTED, "num_kv_heads %d (supported: up to 1024)", num_kv_heads);
  if (batch == 0) return RA_OK;
  RA_REQUIRE(max_seq_len >= 1, "max_seq_len must be >= 1");
  RA_REQUIRE(table_stride >= max_seq_len, "table_stride (%lld) < max_seq_len (%d)", (long long)table_stride,
             max_seq_len);
  RA_REQUIRE(table_rows > 0, "table_rows must be > 0");
  RA_REQUIRE(kv8_pool && q && o && req_to_token && req_pool_indices && seq_lens, "null pointer argument");
  RA_REQUIRE(aligned16(kv8_pool) && aligned16(q) && aligned16(o), "the pool, q and o must be 16-byte aligned");
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

  const Kv8Shape sh = kv8_shape(num_kv_heads, head_dim);
  Kv8DecodeParams pp{};
  pp.pool = static_cast<const uint8_t*>(kv8_pool);
  pp.slot_bytes = sh.slot_bytes;
  pp.block_bytes = sh.block_bytes;
  DecodeParams& p = pp.d;
  p.num_slots = num_slots;
  p.hkv = num_kv_heads;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.hq = num_q_heads;
  p.group = group;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.table = req_to_token;
  p.table_stride = table_stride;
  p.table_rows = table_rows;
  p.rpi = req_pool_indices;
  p.seq_lens = seq_lens;
  p.batch = batch;
  p.max_seq_len = max_seq_len;
  p.min_chunk = 64;
  const int slab = slab_of(head_dim, sh.hpc);
  p.chunk_align = slab;
  p.err = device_error;
  bind_decode_workspace(p, wl, pl, workspace);
  p.hpc = sh.hpc;
  p.n_hgroups = sh.blocks;
  p.row_stride = sh.block_bytes;
  p.stage_bytes = slab * p.row_stride;
  // A CTA of few heads waits on its own chain of slab, scores, softmax and product: two share an SM where their
  // registers fit (8 warps of 128 registers each; 3 heads of 128 gain more from 64-key slabs: 150 requests of
  // 1000..9000 keys, 12/3 heads 125 us as two CTAs, 116 as one; 1 head: 64 requests 47.8 and 53.6).
  const int per_sm = ctas_per_sm(head_dim, sh.hpc);
  // One full item per resident CTA, and the requests' shorter last ones, largest first, to even them out: 64 requests
  // of 512..4096 keys, 32/8 heads 57.5 us, 59.5 with three per CTA (more partials), 104 of 267..8966, 64/8 heads
  // 93.6 and 101, 200 of 1000..9000, 8/1 heads 103 and 127; the 224 of 65..13700, 64/8 heads, 190.1 with one and 189.4
  // with two.
  static_assert(2 * kSmallSms <= kDecodePlanItems, "the workspace holds the plan's items");
  p.plan_items = kSmallSms * per_sm;
  p.nstage = (kRingSmemLimit / per_sm - 1024 - kRingHdrBytes) / p.stage_bytes;  // (1 KB per CTA is the system's)
  if (p.nstage > kRingMaxStages) p.nstage = kRingMaxStages;
  const int smem = kRingHdrBytes + p.nstage * p.stage_bytes;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (head_dim == 64) return launch<64, 64>(pp, per_sm, smem, dev, s);
  return slab == 64 ? launch<128, 64>(pp, per_sm, smem, dev, s) : launch<128, 32>(pp, per_sm, smem, dev, s);
}
