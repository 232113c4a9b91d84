// kv8_store.cu -- ra_kv8_store and ra_kv8_load: rows into and out of a quantised pool.
//
// Both move each byte once and are HBM-bound (8 x 128 heads: 4096 bytes of bf16 and a 2080-byte record per
// token).  A warp takes a unit of up to 16 rows (K and V of up to 8 heads of a block) in steps of 32 lanes,
// D / 16 lanes per row, a lane holding 8 values of the row's first half and the 8 that lie D / 2 further (16-byte
// accesses of neighbouring lanes are contiguous on the bf16 side, 8-byte ones on the record's side).  A lane issues
// all its steps' loads before the first use: 4 KB in flight per warp of a full block.  The bf16 side is read and
// written with streaming hints (each byte is touched once).  65,521 tokens are stored and read back in 124 us
// (6.5 TB/s, 96% of a copy's rate), 239,251 read back in 223 us (98%).
// The store finds a row's largest magnitude with D / 16-lane shuffles; a block's 16 exponent bytes, zero past its
// rows, and the record's padding are written with it, so that only whole sectors reach DRAM.
#include "api_common.h"
#include "kv8.cuh"

namespace ra {

namespace {

constexpr int kThreads = 256;

template <int D>
struct Rows {
  static constexpr int kLanes = D / 16;          // lanes per row
  static constexpr int kPerStep = 32 / kLanes;   // rows per step (a block has at most 16)
};

// What a warp's unit is: a block, all of its steps at once (STEPS of 2 or 4 hold them); or one step (STEPS = 1), of
// `spb` > 1 units per block, or of `bps` >= 1 whole blocks.
struct Units {
  int64_t n, blocks;  // units; blocks of all tokens
  int32_t spb, bps;
};

// A lane's part of unit u: its block of its token and, in step 0, its row (n_rows and more: none).
struct Place {
  int64_t tok;
  int32_t blk, row;
};
template <int STEPS, int LANES>
__device__ __forceinline__ Place place_of(int64_t u, int32_t row0, const Units& un, const Kv8Shape& sh) {
  Place w;
  w.row = row0;
  int64_t g = u;
  if constexpr (STEPS == 1) {
    if (un.spb > 1) {
      g = u / un.spb;
      w.row += static_cast<int32_t>(u - g * un.spb) * (32 / LANES);
    } else {
      const int32_t i = w.row / (2 * sh.hpc);
      w.row -= i * 2 * sh.hpc;
      g = u * un.bps + i;
      if (i >= un.bps || g >= un.blocks) g = u * un.bps, w.row = 2 * sh.hpc;
    }
  }
  w.tok = g / sh.blocks;
  w.blk = static_cast<int32_t>(g - w.tok * sh.blocks);
  return w;
}

__device__ __forceinline__ uint2 quantise8(const uint4& v, float inv) {
  return make_uint2(f32x4_to_e4m3x4(bf16_lo(v.x) * inv, bf16_hi(v.x) * inv, bf16_lo(v.y) * inv, bf16_hi(v.y) * inv),
                    f32x4_to_e4m3x4(bf16_lo(v.z) * inv, bf16_hi(v.z) * inv, bf16_lo(v.w) * inv, bf16_hi(v.w) * inv));
}

template <int D, int STEPS>
__global__ void __launch_bounds__(kThreads, STEPS == 1 ? 8 : STEPS == 2 ? 5 : 4) kv8_store_kernel(uint8_t* __restrict__ pool, int64_t num_slots, int32_t hkv,
                                                             Kv8Shape sh, const uint4* __restrict__ k_new,
                                                             const uint4* __restrict__ v_new,
                                                             const int32_t* __restrict__ loc, Units un,
                                                             uint32_t* __restrict__ err) {
  using R = Rows<D>;
  griddep_wait();  // earlier kernels may still read the records this store overwrites
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const int sub = lane % R::kLanes, row0 = lane / R::kLanes;
  const int n_rows = 2 * sh.hpc;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); u < un.n; u += warps) {
    const Place at = place_of<STEPS, R::kLanes>(u, row0, un, sh);
    const int32_t slot = __ldg(loc + at.tok);
    uint4 a[STEPS], b[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int r = s * R::kPerStep + at.row;
      if (r < n_rows) {
        const uint4* src = ((r & 1) ? v_new : k_new) + (at.tok * hkv + at.blk * sh.hpc + (r >> 1)) * (D / 8) + sub;
        a[s] = __ldcs(src);
        b[s] = __ldcs(src + D / 16);
      } else {
        a[s] = b[s] = make_uint4(0, 0, 0, 0);
      }
    }
    const bool stored = slot >= 0 && slot < num_slots;
    if (!stored && at.row == 0 && sub == 0 && at.blk == 0) flag_error(err, RA_DEVERR_SLOT);
    if (STEPS > 1 && !stored) continue;  // (warp-uniform)
    uint8_t* rec = pool + (stored ? static_cast<int64_t>(slot) * sh.slot_bytes + at.blk * sh.block_bytes : 0);
    uint32_t eb[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      uint32_t m = max(amax_bf16x8(a[s]), amax_bf16x8(b[s]));
#pragma unroll
      for (int off = 1; off < R::kLanes; off <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
      const int32_t e = kv8_exponent(m);
      eb[s] = static_cast<uint32_t>(e + 127);
      const int r = s * R::kPerStep + at.row;
      if (stored && r < n_rows) {
        const float inv = pow2f(-e);
        uint2* dst = reinterpret_cast<uint2*>(rec + r * D) + sub;
        dst[0] = quantise8(a[s], inv);
        dst[D / 16] = quantise8(b[s], inv);
      }
    }
    // the block's 16 bytes of scales, zero past its rows, and behind the last block the record's padding
    uint8_t* tail = rec + n_rows * D;
    bool last;
    if (STEPS == 1 && un.spb > 1) {  // each row's lanes write its byte, the last row's the rest
      last = stored && at.row == n_rows - 1;
      if (stored && sub == 0 && at.row < n_rows) tail[at.row] = static_cast<uint8_t>(eb[0]);
      if (last)
        for (int i = n_rows + sub; i < 16; i += R::kLanes) tail[i] = 0;
    } else {
      const int base = STEPS == 1 ? row0 - at.row : 0;  // first row (of the warp's step) of the block
      const uint4 scales = gather_scale_bytes<STEPS, R::kPerStep, R::kLanes>(eb, n_rows, base);
      last = stored && at.row == 0;
      if (last && sub == 0) *reinterpret_cast<uint4*>(tail) = scales;
    }
    if (last && sub == 1 && at.blk == sh.blocks - 1 && sh.blocks * sh.block_bytes < sh.slot_bytes)
      reinterpret_cast<uint4*>(tail)[1] = make_uint4(0, 0, 0, 0);
  }
}

__device__ __forceinline__ uint4 restore8(const uint2& c, float s) {
  const float2 p0 = f16x2_to_f32x2(e4m3x2_to_f16x2(c.x)), p1 = f16x2_to_f32x2(e4m3x2_hi_to_f16x2(c.x));
  const float2 p2 = f16x2_to_f32x2(e4m3x2_to_f16x2(c.y)), p3 = f16x2_to_f32x2(e4m3x2_hi_to_f16x2(c.y));
  return make_uint4(pack_bf16x2(p0.x * s, p0.y * s), pack_bf16x2(p1.x * s, p1.y * s),
                    pack_bf16x2(p2.x * s, p2.y * s), pack_bf16x2(p3.x * s, p3.y * s));
}

template <int D, int STEPS>
__global__ void __launch_bounds__(kThreads, STEPS <= 2 ? 8 : 5) kv8_load_kernel(const uint8_t* __restrict__ pool, int64_t num_slots,
                                                            int32_t hkv, Kv8Shape sh, const int32_t* __restrict__ slots,
                                                            uint4* __restrict__ k_out, uint4* __restrict__ v_out,
                                                            Units un, uint32_t* __restrict__ err) {
  using R = Rows<D>;
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const int sub = lane % R::kLanes, row0 = lane / R::kLanes;
  const int n_rows = 2 * sh.hpc;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); u < un.n; u += warps) {
    const Place at = place_of<STEPS, R::kLanes>(u, row0, un, sh);
    int32_t slot = __ldg(slots + at.tok);
    if (slot < 0 || slot >= num_slots) {
      if (at.row == 0 && sub == 0 && at.blk == 0) flag_error(err, RA_DEVERR_SLOT);
      slot = 0;
    }
    const uint8_t* rec = pool + static_cast<int64_t>(slot) * sh.slot_bytes + at.blk * sh.block_bytes;
    uint2 a[STEPS], b[STEPS];
    uint32_t eb[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int r = s * R::kPerStep + at.row;
      if (r < n_rows) {
        const uint2* src = reinterpret_cast<const uint2*>(rec + r * D) + sub;
        a[s] = __ldg(src);
        b[s] = __ldg(src + D / 16);
        eb[s] = __ldg(rec + n_rows * D + r);
      }
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int r = s * R::kPerStep + at.row;
      if (r < n_rows) {
        const float scale = __uint_as_float(eb[s] << 23);
        uint4* dst = ((r & 1) ? v_out : k_out) + (at.tok * hkv + at.blk * sh.hpc + (r >> 1)) * (D / 8) + sub;
        __stcs(dst, restore8(a[s], scale));
        __stcs(dst + D / 16, restore8(b[s], scale));
      }
    }
  }
}

ra_status check_kv8(const void* pool, int64_t num_slots, int32_t num_kv_heads, int32_t head_dim, const void* k,
                    const void* v, const int32_t* slots, int64_t n) {
  RA_REQUIRE(n >= 0, "num_tokens must be >= 0 (got %lld)", (long long)n);
  RA_REQUIRE(num_slots > 0, "num_slots must be > 0");
  RA_REQUIRE(num_kv_heads > 0, "num_kv_heads must be > 0");
  if (head_dim != 64 && head_dim != 128) return fail(RA_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", head_dim);
  if (num_kv_heads > 1024) return fail(RA_ERR_UNSUPPORTED, "num_kv_heads %d (supported: up to 1024)", num_kv_heads);
  if (n == 0) return RA_OK;
  RA_REQUIRE(pool && k && v && slots, "null pointer argument");
  RA_REQUIRE(aligned16(pool) && aligned16(k) && aligned16(v), "the pool and the rows must be 16-byte aligned");
  RA_REQUIRE(aligned4(slots), "slot indices must be 4-byte aligned");
  return RA_OK;
}

// A block at once where it takes several steps and there are enough of them for the SMs' warps, else units of one
// step: as many warps as possible for few tokens (224 tokens of 8 x 128 stored and read back: 4.4 us in blocks, 3.6
// in steps), and lanes without idle rows for few heads (65,521 tokens of 2 x 64: 37.2 us, 22.3 packed).
Units units_of(const Kv8Shape& sh, int32_t head_dim, int64_t num_tokens, const DeviceInfo& dev, int32_t& steps) {
  const int32_t per_step = 32 / (head_dim / 16), n_rows = 2 * sh.hpc;
  Units un{0, num_tokens * sh.blocks, 1, 1};
  const int32_t needs = (n_rows + per_step - 1) / per_step;
  steps = un.blocks * needs < static_cast<int64_t>(dev.num_sms) * 16 ? 1 : needs <= 2 ? needs : 4;
  un.n = un.blocks;
  if (needs == 1) {
    un.bps = per_step / n_rows;
    un.n = (un.blocks + un.bps - 1) / un.bps;
  } else if (steps == 1) {
    un.spb = needs;
    un.n = un.blocks * un.spb;
  }
  return un;
}

// A unit per warp: a CTA's place is taken by the next as soon as its warps are through, which a persistent grid's
// loop leaves empty while its slowest warp works (65,521 tokens of 8 x 128 read back: 68 us in eight CTAs per SM,
// 62.8 in a CTA per eight units).
int grid_for(int64_t units) {
  const int64_t want = (units + kThreads / 32 - 1) / (kThreads / 32), most = (int64_t(1) << 31) - 1;
  return static_cast<int>(want < most ? want : most);
}

template <class K>
K by_steps(int32_t steps, K one, K two, K four) {
  return steps == 1 ? one : steps == 2 ? two : four;
}

}  // namespace
}  // namespace ra

extern "C" size_t ra_kv8_slot_bytes(int32_t num_kv_heads, int32_t head_dim) {
  if (num_kv_heads <= 0 || num_kv_heads > 1024 || (head_dim != 64 && head_dim != 128)) return 0;
  return ra::kv8_shape(num_kv_heads, head_dim).slot_bytes;
}

extern "C" ra_status ra_kv8_store(void* kv8_pool, int64_t num_slots, int32_t num_kv_heads, int32_t head_dim,
                                  const void* k_new, const void* v_new, const int32_t* out_cache_loc,
                                  int64_t num_tokens, uint32_t* device_error, ra_stream_t stream) {
  using namespace ra;
  clear_error();
  if (ra_status st = check_kv8(kv8_pool, num_slots, num_kv_heads, head_dim, k_new, v_new, out_cache_loc, num_tokens))
    return st;
  if (num_tokens == 0) return RA_OK;
  DeviceInfo dev;
  if (ra_status st = current_device(&dev)) return st;
  const Kv8Shape sh = kv8_shape(num_kv_heads, head_dim);
  int32_t steps;
  const Units un = units_of(sh, head_dim, num_tokens, dev, steps);
  auto kern = head_dim == 128
                  ? by_steps(steps, kv8_store_kernel<128, 1>, kv8_store_kernel<128, 2>, kv8_store_kernel<128, 4>)
                  : by_steps(steps, kv8_store_kernel<64, 1>, kv8_store_kernel<64, 2>, kv8_store_kernel<64, 2>);
  return launch_pdl("kv8_store_kernel", kern, dim3(grid_for(un.n)), dim3(kThreads), 0,
                    reinterpret_cast<cudaStream_t>(stream), static_cast<uint8_t*>(kv8_pool), num_slots, num_kv_heads,
                    sh, static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), out_cache_loc, un,
                    device_error);
}

extern "C" ra_status ra_kv8_load(const void* kv8_pool, int64_t num_slots, int32_t num_kv_heads, int32_t head_dim,
                                 const int32_t* slots, void* k_out, void* v_out, int64_t num_tokens,
                                 uint32_t* device_error, ra_stream_t stream) {
  using namespace ra;
  clear_error();
  if (ra_status st = check_kv8(kv8_pool, num_slots, num_kv_heads, head_dim, k_out, v_out, slots, num_tokens)) return st;
  if (num_tokens == 0) return RA_OK;
  DeviceInfo dev;
  if (ra_status st = current_device(&dev)) return st;
  const Kv8Shape sh = kv8_shape(num_kv_heads, head_dim);
  int32_t steps;
  const Units un = units_of(sh, head_dim, num_tokens, dev, steps);
  auto kern = head_dim == 128
                  ? by_steps(steps, kv8_load_kernel<128, 1>, kv8_load_kernel<128, 2>, kv8_load_kernel<128, 4>)
                  : by_steps(steps, kv8_load_kernel<64, 1>, kv8_load_kernel<64, 2>, kv8_load_kernel<64, 2>);
  return launch_pdl("kv8_load_kernel", kern, dim3(grid_for(un.n)), dim3(kThreads), 0,
                    reinterpret_cast<cudaStream_t>(stream), static_cast<const uint8_t*>(kv8_pool), num_slots,
                    num_kv_heads, sh, slots, static_cast<uint4*>(k_out), static_cast<uint4*>(v_out), un,
                    device_error);
}
