// kv8.cuh -- the quantised (e4m3) cache record and its conversions.
//
// A quantised pool is bytes [num_slots, slot_bytes]; a slot's record holds one token's K and V for every
// kv head.  It is made of blocks of hpc kv heads (the largest divisor of Hkv that is at most 8, the heads
// one decode CTA reads).  A block is, per head, D codes of K then D codes of V, followed by 16 bytes of
// exponents: byte 2h is head h's K exponent, byte 2h + 1 its V exponent, both biased by 127, the rest zero.
// A record is padded to a multiple of 32 bytes (whole L2 sectors).  So a key's K, V and scales for a head
// group are one contiguous copy, and a decode ring stage's row stride (a block) is 16 bytes past a multiple
// of 128: the eight rows of a fragment load fall into different banks.
//
// A row x[0..D) is stored as codes c = rn_e4m3(x * 2^-e), value c * 2^e, with the smallest e that keeps
// max|x| <= 448 * 2^e.  e4m3 is a float format, so a power of two costs it no precision against a real
// scale (at most one binade of its 18), and it makes the scaling exact: codes do not depend on how a
// division rounds, and a value read back is exact in bf16 (4 significant bits).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "ra_ptx.cuh"

namespace ra {

constexpr int kKv8MinExp = -118;  // 2^-e stays a normal float; rows below 2^-109 lose low bits
constexpr int kKv8MaxExp = 119;   // 448 * 2^119 is finite in bf16 (256 * 2^120 is not); larger values saturate
constexpr int kKv8ScaleBytes = 16;

struct Kv8Shape {
  int32_t hpc;          // kv heads per block
  int32_t blocks;       // blocks per record
  int32_t block_bytes;  // hpc * 2 * D + 16
  int32_t slot_bytes;   // record size
};

inline Kv8Shape kv8_shape(int32_t num_kv_heads, int32_t head_dim) {
  Kv8Shape s{};
  for (s.hpc = 8; num_kv_heads % s.hpc != 0;) --s.hpc;
  s.blocks = num_kv_heads / s.hpc;
  s.block_bytes = s.hpc * 2 * head_dim + kKv8ScaleBytes;
  s.slot_bytes = (s.blocks * s.block_bytes + 31) / 32 * 32;
  return s;
}

// Two e4m3 codes (the low 16 bits of x) -> f16 pair, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x) {
  uint32_t y;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(y) : "r"(x));
  return y;
}
// The same of the high 16 bits.
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t x) {
  uint32_t y;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(y) : "r"(x));
  return y;
}
// Round to e4m3 (nearest even, saturating; NaN -> 0x7f).
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d) {
  uint32_t y;
  asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
      : "=r"(y)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return y;
}
__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t x) {
  float2 r;
  asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(x));
  return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Exponent of a row whose largest finite magnitude has these float bits (448 = 1.75 * 2^8).
__device__ __forceinline__ int32_t kv8_exponent(uint32_t amax_bits) {
  const int32_t e = static_cast<int32_t>(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kKv8MinExp), kKv8MaxExp);
}
__device__ __forceinline__ float pow2f(int32_t e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Largest finite magnitude (float bits) of 8 bf16; infinities and NaN do not count.
__device__ __forceinline__ uint32_t amax_bf16x8(const uint4& v) {
  const uint32_t m2 = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                               __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
  uint32_t m = max(m2 & 0xffffu, m2 >> 16);
  if (m >= 0x7f80u) {  // an infinity or NaN: take the others one by one
    m = 0;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
      if (lo < 0x7f80u) m = max(m, lo);
      if (hi < 0x7f80u) m = max(m, hi);
    }
  }
  return m << 16;
}

// A warp's up-to-16 exponent bytes: row r (K and V of the block's heads interleaved, as in the record) was
// handled in step r / kRowsPerStep by the lanes from (base + r % kRowsPerStep) * kLanesPerRow (base: the block's
// first row of the step, where several blocks share one).  Every lane calls; rows past n_rows give 0.
template <int kSteps, int kRowsPerStep, int kLanesPerRow>
__device__ __forceinline__ uint4 gather_scale_bytes(const uint32_t (&eb)[kSteps], int n_rows,
                                                    int base = 0) {
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    if (r / kRowsPerStep < kSteps) {
      const uint32_t b = __shfl_sync(0xffffffffu, eb[r / kRowsPerStep], ((base + r % kRowsPerStep) * kLanesPerRow) & 31);
      if (r < n_rows) w[r >> 2] |= b << (8 * (r & 3));
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace ra
