// qk_norm_rope.cu -- ra_qk_norm_rope_store: what a layer does between its qkv projection and attention.
//
// For each token, every q and k head row x[0..D):
//   y = x * rsqrt(mean(x^2) + eps) * w          (skipped without weights)
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)   for the rot / 2 pairs of the first rot values,
// pairs (i, i + rot/2) or, interleaved, (2i, 2i + 1), with row positions[t] of a table of cosines and
// sines; q goes to q_out, k and v to the token's pool slot (bf16, or quantised to a record).  Everything
// is computed in fp32 and rounded once: to bf16, or for a quantised K to e4m3 from the fp32 value (through
// bf16 a value could be rounded to a tie of the coarser format first).
//
// Bound by HBM: each row is read and written once ((Hq + 2 Hkv) * D * 2 bytes each way per token; the
// angles add rot * 4).  A row is D / 16 lanes wide, a lane holding 8 values of its first half and the 8 that
// lie D / 2 further: with rot = D and half-split pairs both members of a pair are in one lane and the
// rotation needs no exchange; other forms fetch the partner with shuffles.  A warp takes a unit of one
// token: one or more steps of 512 / D q rows, or the 2 * hpc rows of one K/V block (hpc <= 8 heads), at once or
// (single-step units) in a step each; all
// loads of a unit are issued before the first use, and the angles and weights are loaded once per unit.  Where
// the heads of a token would leave such units part empty, units are flat: the next 512 / D q rows of all
// tokens, or as many K/V blocks as fit a step, each row's lanes with their own token.
#include <algorithm>
#include <cmath>

#include "api_common.h"
#include "kv8.cuh"

namespace ra {

namespace {

constexpr int kThreads = 256;

struct NormRopeParams {
  const __nv_bfloat16 *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const __nv_bfloat16 *q_weight, *k_weight;  // [D] or both null
  float eps;
  const int32_t* positions;
  const float* cos_sin;  // [max_position, rot]: rot / 2 cosines, rot / 2 sines
  int64_t max_position;
  int32_t rot;
  __nv_bfloat16* q_out;
  int64_t q_out_stride;
  __nv_bfloat16 *k_pool, *v_pool;  // bf16 pool
  uint8_t* kv8_pool;               // quantised pool
  int64_t num_slots;
  const int32_t* loc;
  int32_t hq, hkv;
  Kv8Shape sh;
  int32_t q_units, units_per_token;  // wide units: of a token
  int64_t tokens, flat_q;            // flat units: the q units come first
  int32_t bps;                       // flat units: K/V blocks per unit
  int32_t spb;                       // single-step units: units per K/V block
  int64_t units;
  uint32_t* err;
};

// Half-split pairs with rot = D, rot <= D / 2 (a lane's second chunk is not turned, and both members of a pair lie in
// first chunks: 8 exchanges a row where the general form makes 32; 2886 tokens, 12/3 heads, 64 of 128 values, e4m3:
// 16.5 us -> 14.0) and between; adjacent pairs.
enum Rope { kHalfFull, kHalfLow, kHalfPart, kAdjacent };

// cosines and sines of a lane's two chunks of 8 values (first-half chunk, second-half chunk)
template <int ROPE>
struct Angles {
  static constexpr int kChunks = ROPE == kHalfFull || ROPE == kHalfLow ? 1 : 2;
  float c[kChunks][8], s[kChunks][8];
};

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

template <int D, int ROPE>
__device__ __forceinline__ void load_angles(const float* row, int32_t rot, int sub, Angles<ROPE>& an) {
  const int half = rot >> 1;
  if constexpr (ROPE == kHalfFull) {
    load8(row + 8 * sub, an.c[0]);
    load8(row + half + 8 * sub, an.s[0]);
  } else {
#pragma unroll
    for (int ch = 0; ch < Angles<ROPE>::kChunks; ++ch) {
      const int e0 = ch * (D / 2) + 8 * sub;  // first value of the chunk
      if (e0 >= rot) {
#pragma unroll
        for (int j = 0; j < 8; ++j) an.c[ch][j] = 1.f, an.s[ch][j] = 0.f;
      } else if constexpr (ROPE != kAdjacent) {
        const int f = e0 < half ? e0 : e0 - half;
        load8(row + f, an.c[ch]);
        load8(row + half + f, an.s[ch]);
        if (e0 < half) {  // first members of their pairs: a cos - b sin
#pragma unroll
          for (int j = 0; j < 8; ++j) an.s[ch][j] = -an.s[ch][j];
        }
      } else {
        const float4 c4 = __ldg(reinterpret_cast<const float4*>(row + e0 / 2));
        const float4 s4 = __ldg(reinterpret_cast<const float4*>(row + half + e0 / 2));
        const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) an.c[ch][j] = cc[j >> 1], an.s[ch][j] = (j & 1) ? ss[j >> 1] : -ss[j >> 1];
      }
    }
  }
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z), x[5] = bf16_hi(v.z), x[6] = bf16_lo(v.w), x[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// Norm and rotation of one row, spread over D / 16 lanes (every lane of the warp calls).
template <int D, int ROPE>
__device__ __forceinline__ void norm_rope_row(float (&x)[2][8], bool norm, const uint4 (&w)[2], float eps, int32_t rot,
                                              int sub, const Angles<ROPE>& an) {
  constexpr int kLanes = D / 16;
  if (norm) {
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x[0][j], x[0][j], fmaf(x[1][j], x[1][j], ss));
#pragma unroll
    for (int off = 1; off < kLanes; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float r = rsqrtf(ss * (1.f / D) + eps);
#pragma unroll
    for (int ch = 0; ch < 2; ++ch) {
      float wf[8];
      unpack8(w[ch], wf);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[ch][j] = x[ch][j] * r * wf[j];
    }
  }
  if constexpr (ROPE == kHalfFull) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = x[0][j], b = x[1][j];
      x[0][j] = a * an.c[0][j] - b * an.s[0][j];
      x[1][j] = b * an.c[0][j] + a * an.s[0][j];
    }
  } else if constexpr (ROPE == kHalfLow) {
    const int hc = rot >> 4;  // chunks in half of the rotated part
    const int partner = (threadIdx.x & 31) + (sub < hc ? hc : sub < 2 * hc ? -hc : 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float y = __shfl_sync(0xffffffffu, x[0][j], partner);
      if (sub < 2 * hc) x[0][j] = x[0][j] * an.c[0][j] + y * an.s[0][j];
    }
  } else if constexpr (ROPE == kHalfPart) {
    // the partner chunk of 8 lies rot / 2 values away, in the same or the other half, on some lane of the row
    const int hc = rot >> 4;  // chunks in half of the rotated part
    const int first = (threadIdx.x & 31) - sub;
    float y[2][8];
#pragma unroll
    for (int ch = 0; ch < 2; ++ch) {
      const int c = ch * kLanes + sub;
      const int pc = c < hc ? c + hc : (c < 2 * hc ? c - hc : c);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float p0 = __shfl_sync(0xffffffffu, x[0][j], first + pc % kLanes);
        const float p1 = __shfl_sync(0xffffffffu, x[1][j], first + pc % kLanes);
        y[ch][j] = x[ch][j] * an.c[ch][j] + (pc < kLanes ? p0 : p1) * an.s[ch][j];
      }
    }
#pragma unroll
    for (int ch = 0; ch < 2; ++ch) {
      const bool turned = ch * kLanes + sub < 2 * hc;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[ch][j] = turned ? y[ch][j] : x[ch][j];
    }
  } else {
#pragma unroll
    for (int ch = 0; ch < 2; ++ch) {
      if (ch * (D / 2) + 8 * sub < rot) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float a = x[ch][j], b = x[ch][j + 1];
          x[ch][j] = a * an.c[ch][j] + b * an.s[ch][j];
          x[ch][j + 1] = b * an.c[ch][j] + a * an.s[ch][j + 1];
        }
      }
    }
  }
}

// QSTEPS: 512 / D q rows each in a unit; 0: flat units of one step
template <int D, int ROPE, bool KV8, int QSTEPS, int KVSTEPS>
__global__ void __launch_bounds__(kThreads, QSTEPS <= 1 && KVSTEPS == 1 ? 3 : 2)
    qk_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int kLanes = D / 16, kPerStep = 32 / kLanes, kKvSteps = KVSTEPS;
  constexpr bool kFlat = QSTEPS == 0;
  constexpr bool kSingle = QSTEPS == 1;  // one step per unit
  constexpr int kQSteps = kFlat ? 1 : QSTEPS;
  static_assert(!kSingle || KVSTEPS == 1, "single-step units");
  griddep_wait();  // q, k and v come from the kernel before; earlier kernels may still read the slots
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const int sub = lane % kLanes, row0 = lane / kLanes;
  const bool norm = p.q_weight != nullptr;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  const int n_rows = 2 * p.sh.hpc;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); u < p.units; u += warps) {
    // this lane's token, and its q head (the unit's first) or its block of heads and row of the block
    int64_t tok;
    int32_t h0 = 0, blk = 0, skip = 0;  // skip: what a lane's row of the block is less than its row of the warp
    bool in = true, is_q;
    if constexpr (kFlat) {
      is_q = u < p.flat_q;
      if (is_q) {
        const uint32_t g = static_cast<uint32_t>(u) * kPerStep + row0, t = g / static_cast<uint32_t>(p.hq);
        in = t < p.tokens;
        tok = in ? t : 0;
        h0 = in ? static_cast<int32_t>(g - t * p.hq) : p.hq;
      } else {
        const uint32_t i = kKvSteps == 1 ? row0 / n_rows : 0;
        const uint32_t g = static_cast<uint32_t>(u - p.flat_q) * p.bps + i, t = g / static_cast<uint32_t>(p.sh.blocks);
        in = i < static_cast<uint32_t>(p.bps) && t < p.tokens;
        tok = in ? t : 0;
        blk = in ? static_cast<int32_t>(g - t * p.sh.blocks) : 0;
        skip = i * n_rows;
      }
    } else {
      tok = u / p.units_per_token;
      const int32_t part = static_cast<int32_t>(u - tok * p.units_per_token);
      is_q = part < p.q_units;
      h0 = part * kQSteps * kPerStep + row0;
      blk = part - p.q_units;
    }
    if constexpr (kSingle) {
      if (p.spb > 1 && !is_q) {
        const int32_t step = blk % p.spb;
        blk /= p.spb;
        skip = -step * kPerStep;
      }
    }
    int64_t pos = __ldg(p.positions + tok);
    if (pos < 0 || pos >= p.max_position) {
      if (is_q && h0 == 0 && sub == 0) flag_error(p.err, RA_DEVERR_POSITION);  // (once per token)
      pos = 0;
    }
    const float* ang = p.cos_sin + pos * p.rot;
    if (is_q) {
      const __nv_bfloat16* src = p.q + tok * p.q_stride + 8 * sub;
      __nv_bfloat16* dst = p.q_out + tok * p.q_out_stride + 8 * sub;
      uint4 a[kQSteps], b[kQSteps];
#pragma unroll
      for (int s = 0; s < kQSteps; ++s) {
        const int32_t h = h0 + s * kPerStep;
        a[s] = b[s] = make_uint4(0, 0, 0, 0);
        if (h < p.hq) {
          a[s] = *reinterpret_cast<const uint4*>(src + h * D);
          b[s] = *reinterpret_cast<const uint4*>(src + h * D + D / 2);
        }
      }
      uint4 w[2] = {};
      if (norm) {
        w[0] = __ldg(reinterpret_cast<const uint4*>(p.q_weight) + sub);
        w[1] = __ldg(reinterpret_cast<const uint4*>(p.q_weight) + sub + kLanes);
      }
      Angles<ROPE> an;
      load_angles<D, ROPE>(ang, p.rot, sub, an);
#pragma unroll
      for (int s = 0; s < kQSteps; ++s) {
        const int32_t h = h0 + s * kPerStep;
        float x[2][8];
        unpack8(a[s], x[0]);
        unpack8(b[s], x[1]);
        norm_rope_row<D, ROPE>(x, norm, w, p.eps, p.rot, sub, an);
        if (h < p.hq) {
          *reinterpret_cast<uint4*>(dst + h * D) = pack8(x[0]);
          *reinterpret_cast<uint4*>(dst + h * D + D / 2) = pack8(x[1]);
        }
      }
      continue;
    }
    // K and V rows of one block of heads, interleaved (row 2h: K of head h, 2h + 1: its V)
    uint4 a[kKvSteps], b[kKvSteps];
#pragma unroll
    for (int s = 0; s < kKvSteps; ++s) {
      const int r = s * kPerStep + row0 - skip;
      a[s] = b[s] = make_uint4(0, 0, 0, 0);
      if (in && r < n_rows) {
        const __nv_bfloat16* src =
            ((r & 1) ? p.v + tok * p.v_stride : p.k + tok * p.k_stride) + (blk * p.sh.hpc + (r >> 1)) * D + 8 * sub;
        a[s] = __ldg(reinterpret_cast<const uint4*>(src));
        b[s] = __ldg(reinterpret_cast<const uint4*>(src + D / 2));
      }
    }
    const int32_t slot = __ldg(p.loc + tok);
    uint4 w[2] = {};
    if (norm) {
      w[0] = __ldg(reinterpret_cast<const uint4*>(p.k_weight) + sub);
      w[1] = __ldg(reinterpret_cast<const uint4*>(p.k_weight) + sub + kLanes);
    }
    Angles<ROPE> an;
    load_angles<D, ROPE>(ang, p.rot, sub, an);
    const bool stored = in && slot >= 0 && slot < p.num_slots;
    if (in && !stored && sub == 0 && row0 == skip && blk == 0) flag_error(p.err, RA_DEVERR_SLOT);
    if (kFlat ? !__any_sync(0xffffffffu, stored) : !stored) continue;  // (warp-uniform)
    const bool is_v = row0 & 1;  // the same in every step: kPerStep is even
    uint8_t* rec = nullptr;
    if constexpr (KV8) {
      if (stored) rec = p.kv8_pool + static_cast<int64_t>(slot) * p.sh.slot_bytes + blk * p.sh.block_bytes;
    }
    uint32_t eb[kKvSteps];
#pragma unroll
    for (int s = 0; s < kKvSteps; ++s) {
      const int r = s * kPerStep + row0 - skip;
      float x[2][8], y[2][8];
      unpack8(a[s], x[0]);
      unpack8(b[s], x[1]);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[0][j] = x[0][j], y[1][j] = x[1][j];
      norm_rope_row<D, ROPE>(y, norm, w, p.eps, p.rot, sub, an);  // (V's lanes compute it too and drop it)
      if constexpr (!KV8) {
        if (stored && r < n_rows) {
          __nv_bfloat16* dst = (is_v ? p.v_pool : p.k_pool) +
                               (static_cast<int64_t>(slot) * p.hkv + blk * p.sh.hpc + (r >> 1)) * D + 8 * sub;
          *reinterpret_cast<uint4*>(dst) = is_v ? a[s] : pack8(y[0]);
          *reinterpret_cast<uint4*>(dst + D / 2) = is_v ? b[s] : pack8(y[1]);
        }
      } else {
        uint32_t m = 0;
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[ch][j] = is_v ? x[ch][j] : y[ch][j];
            const uint32_t t = __float_as_uint(x[ch][j]) & 0x7fffffffu;
            m = max(m, t < 0x7f800000u ? t : 0u);  // infinities and NaN do not count
          }
#pragma unroll
        for (int off = 1; off < kLanes; off <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
        const int32_t e = kv8_exponent(m);
        eb[s] = static_cast<uint32_t>(e + 127);
        if (stored && r < n_rows) {
          const float inv = pow2f(-e);
          uint2* dst = reinterpret_cast<uint2*>(rec + r * D) + sub;
#pragma unroll
          for (int ch = 0; ch < 2; ++ch)
            dst[ch * (D / 16)] =
                make_uint2(f32x4_to_e4m3x4(x[ch][0] * inv, x[ch][1] * inv, x[ch][2] * inv, x[ch][3] * inv),
                           f32x4_to_e4m3x4(x[ch][4] * inv, x[ch][5] * inv, x[ch][6] * inv, x[ch][7] * inv));
        }
      }
    }
    if constexpr (KV8) {
      // the block's 16 bytes of scales, zero past its rows, and behind the last block the record's padding
      uint8_t* tail = rec + n_rows * D;
      bool last;
      if (kSingle && p.spb > 1) {  // the block's rows are in several units: each row's lanes write its byte, the
        const int r = row0 - skip;  // last row's the rest
        last = stored && r == n_rows - 1;
        if (stored && sub == 0 && r < n_rows) tail[r] = static_cast<uint8_t>(eb[0]);
        if (last)
          for (int i = n_rows + sub; i < 16; i += kLanes) tail[i] = 0;
      } else {
        const uint4 scales = gather_scale_bytes<kKvSteps, kPerStep, kLanes>(eb, n_rows, skip);
        last = stored && row0 == skip;
        if (last && sub == 0) *reinterpret_cast<uint4*>(tail) = scales;
      }
      if (last && sub == 1 && blk == p.sh.blocks - 1 && p.sh.blocks * p.sh.block_bytes < p.sh.slot_bytes)
        reinterpret_cast<uint4*>(tail)[1] = make_uint4(0, 0, 0, 0);
    }
  }
}

template <int D, bool KV8, int QSTEPS, int KVSTEPS>
ra_status launch(const NormRopeParams& p, bool interleaved, int grid, cudaStream_t s) {
  auto kern = interleaved      ? qk_norm_rope_kernel<D, kAdjacent, KV8, QSTEPS, KVSTEPS>
              : p.rot == D     ? qk_norm_rope_kernel<D, kHalfFull, KV8, QSTEPS, KVSTEPS>
              : 2 * p.rot <= D ? qk_norm_rope_kernel<D, kHalfLow, KV8, QSTEPS, KVSTEPS>
                             : qk_norm_rope_kernel<D, kHalfPart, KV8, QSTEPS, KVSTEPS>;
  return launch_pdl("qk_norm_rope_kernel", kern, dim3(grid), dim3(kThreads), 0, s, p);
}

enum Units { kWide, kOneStep, kFlatUnits };

template <int D, bool KV8>
ra_status launch_steps(const NormRopeParams& p, bool interleaved, Units units, bool deep, int grid, ra_stream_t stream) {
  constexpr int kMost = 16 / (32 / (D / 16));  // steps of 16 rows
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (units == kWide)
    return deep ? launch<D, KV8, kMost, kMost>(p, interleaved, grid, s) : launch<D, KV8, kMost, 1>(p, interleaved, grid, s);
  if (units == kOneStep) return launch<D, KV8, 1, 1>(p, interleaved, grid, s);
  return deep ? launch<D, KV8, 0, kMost>(p, interleaved, grid, s) : launch<D, KV8, 0, 1>(p, interleaved, grid, s);
}

ra_status norm_rope_call(NormRopeParams p, bool kv8, int32_t head_dim, int64_t num_tokens, int32_t interleaved,
                         ra_stream_t stream) {
  RA_REQUIRE(num_tokens >= 0, "num_tokens must be >= 0 (got %lld)", (long long)num_tokens);
  RA_REQUIRE(p.hq > 0 && p.hkv > 0, "head counts must be > 0");
  RA_REQUIRE(p.num_slots > 0, "num_slots must be > 0");
  RA_REQUIRE(p.max_position > 0, "max_position must be > 0");
  RA_REQUIRE(std::isfinite(p.eps) && p.eps >= 0.f, "eps must be finite and >= 0");
  if (head_dim != 64 && head_dim != 128) return fail(RA_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", head_dim);
  if (p.hq > 1024 || p.hkv > 1024) return fail(RA_ERR_UNSUPPORTED, "more than 1024 heads");
  RA_REQUIRE(p.rot >= 0 && p.rot <= head_dim, "rotary_dim must be in [0, head_dim] (got %d)", p.rot);
  if (p.rot % 16 != 0 || p.rot == 0)
    return fail(RA_ERR_UNSUPPORTED, "rotary_dim %d (supported: multiples of 16, from 16)", p.rot);
  RA_REQUIRE((p.q_weight == nullptr) == (p.k_weight == nullptr), "q_weight and k_weight go together");
  RA_REQUIRE(interleaved == 0 || interleaved == 1, "interleaved must be 0 or 1");
  if (num_tokens == 0) return RA_OK;
  RA_REQUIRE(p.q && p.k && p.v && p.positions && p.cos_sin && p.q_out && p.loc, "null pointer argument");
  RA_REQUIRE(kv8 ? p.kv8_pool != nullptr : p.k_pool && p.v_pool, "null pool pointer");
  const int64_t qw = static_cast<int64_t>(p.hq) * head_dim, kw = static_cast<int64_t>(p.hkv) * head_dim;
  RA_REQUIRE(p.q_stride >= qw && p.q_out_stride >= qw && p.k_stride >= kw && p.v_stride >= kw,
             "a token stride is smaller than the token's heads");
  RA_REQUIRE(p.q_stride % 8 == 0 && p.q_out_stride % 8 == 0 && p.k_stride % 8 == 0 && p.v_stride % 8 == 0,
             "token strides must be multiples of 8 elements (16 bytes)");
  RA_REQUIRE(aligned16(p.q) && aligned16(p.k) && aligned16(p.v) && aligned16(p.q_out) && aligned16(p.cos_sin) &&
                 aligned16(p.k_pool) && aligned16(p.v_pool) && aligned16(p.kv8_pool) && aligned16(p.q_weight) &&
                 aligned16(p.k_weight),
             "q, k, v, weights, cos_sin, q_out and pools must be 16-byte aligned");
  RA_REQUIRE(aligned4(p.positions) && aligned4(p.loc), "index arrays must be 4-byte aligned");
  DeviceInfo dev;
  if (ra_status st = current_device(&dev)) return st;
  p.sh = kv8_shape(p.hkv, head_dim);
  // Wide units of 16 q rows (4 KB of loads in flight per warp); where more than a quarter of the rows of a
  // token's last one were missing, flat units; and one step of one token for few tokens, where wide ones fill the
  // SMs' warps badly (a decode step of 64 has 1.6 warps per SM sub-partition with one step) and latency counts
  // (64 tokens, 32/8 heads of 128: 2.0 us, 2.9 with flat units; 300 tokens 2.7 us, 4.3 with a K/V block's four
  // steps in one unit; 806 tokens, above the limit, 3.8 us, 5.7 in single steps).  Measured with 9437 tokens: 12/3
  // heads of 128 21.8 us wide, 27.8 flat; 8/1 heads 13.4 us flat, 16.4 in single steps.
  const int32_t per_step = 32 / (head_dim / 16), n_rows = 2 * p.sh.hpc;
  const int64_t wide_units = num_tokens * ((p.hq + 15) / 16 + p.sh.blocks);
  const bool few = wide_units < static_cast<int64_t>(dev.num_sms) * 8;
  const bool filled = 4 * p.hq >= 48 * ((p.hq + 15) / 16);
  // (flat units count rows in 32 bits)
  const bool countable = num_tokens * std::max(p.hq, p.sh.blocks) < int64_t(1) << 31;
  const Units units = few ? kOneStep : filled || !countable ? kWide : kFlatUnits;
  const bool deep = n_rows > per_step;  // a K/V block takes more than one step (of a unit, or a unit each)
  p.tokens = num_tokens;
  p.spb = units == kOneStep ? (n_rows + per_step - 1) / per_step : 1;
  if (units == kFlatUnits) {
    p.bps = deep ? 1 : per_step / n_rows;
    p.flat_q = (num_tokens * p.hq + per_step - 1) / per_step;
    p.units = p.flat_q + (num_tokens * p.sh.blocks + p.bps - 1) / p.bps;
  } else {
    const int32_t q_rows = units == kWide ? 16 : per_step;
    p.q_units = (p.hq + q_rows - 1) / q_rows;
    p.units_per_token = p.q_units + p.sh.blocks * p.spb;
    p.units = num_tokens * p.units_per_token;
  }
  // Loops of as many CTAs as are resident (9437 tokens, 64/8 heads: 61.5 us, 62.9 with a second, partial wave,
  // 71.5 with a unit per warp); single steps run in waves of CTAs (300 tokens, 32/8 heads: 2.75 us, 3.7 with loops).
  const int64_t want = (p.units + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t cap = static_cast<int64_t>(dev.num_sms) * (units == kOneStep ? 8 : units == kFlatUnits && !deep ? 3 : 2);
  const int grid = static_cast<int>(want < cap ? want : cap);
  return head_dim == 128 ? (kv8 ? launch_steps<128, true>(p, interleaved, units, deep, grid, stream)
                                : launch_steps<128, false>(p, interleaved, units, deep, grid, stream))
                         : (kv8 ? launch_steps<64, true>(p, interleaved, units, deep, grid, stream)
                                : launch_steps<64, false>(p, interleaved, units, deep, grid, stream));
}

NormRopeParams common_params(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                             int64_t v_stride, int32_t hq, int32_t hkv, const void* q_weight, const void* k_weight,
                             float eps, const int32_t* positions, const float* cos_sin, int64_t max_position,
                             int32_t rotary_dim, void* q_out, int64_t q_out_stride, int64_t num_slots,
                             const int32_t* out_cache_loc, uint32_t* device_error) {
  NormRopeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_weight = static_cast<const __nv_bfloat16*>(q_weight);
  p.k_weight = static_cast<const __nv_bfloat16*>(k_weight);
  p.eps = eps;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.max_position = max_position;
  p.rot = rotary_dim;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.q_out_stride = q_out_stride;
  p.num_slots = num_slots;
  p.loc = out_cache_loc;
  p.hq = hq;
  p.hkv = hkv;
  p.err = device_error;
  return p;
}

}  // namespace
}  // namespace ra

extern "C" ra_status ra_qk_norm_rope_store(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                           const void* v, int64_t v_stride, int32_t num_q_heads, int32_t num_kv_heads,
                                           int32_t head_dim, const void* q_weight, const void* k_weight, float eps,
                                           const int32_t* positions, const float* cos_sin, int64_t max_position,
                                           int32_t rotary_dim, int32_t interleaved, void* q_out, int64_t q_out_stride,
                                           void* k_pool, void* v_pool, int64_t num_slots, const int32_t* out_cache_loc,
                                           int64_t num_tokens, uint32_t* device_error, ra_stream_t stream) {
  using namespace ra;
  clear_error();
  NormRopeParams p = common_params(q, q_stride, k, k_stride, v, v_stride, num_q_heads, num_kv_heads, q_weight, k_weight,
                                   eps, positions, cos_sin, max_position, rotary_dim, q_out, q_out_stride, num_slots,
                                   out_cache_loc, device_error);
  p.k_pool = static_cast<__nv_bfloat16*>(k_pool);
  p.v_pool = static_cast<__nv_bfloat16*>(v_pool);
  return norm_rope_call(p, false, head_dim, num_tokens, interleaved, stream);
}

extern "C" ra_status ra_qk_norm_rope_kv8_store(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                               const void* v, int64_t v_stride, int32_t num_q_heads,
                                               int32_t num_kv_heads, int32_t head_dim, const void* q_weight,
                                               const void* k_weight, float eps, const int32_t* positions,
                                               const float* cos_sin, int64_t max_position, int32_t rotary_dim,
                                               int32_t interleaved, void* q_out, int64_t q_out_stride, void* kv8_pool,
                                               int64_t num_slots, const int32_t* out_cache_loc, int64_t num_tokens,
                                               uint32_t* device_error, ra_stream_t stream) {
  using namespace ra;
  clear_error();
  NormRopeParams p = common_params(q, q_stride, k, k_stride, v, v_stride, num_q_heads, num_kv_heads, q_weight, k_weight,
                                   eps, positions, cos_sin, max_position, rotary_dim, q_out, q_out_stride, num_slots,
                                   out_cache_loc, device_error);
  p.kv8_pool = static_cast<uint8_t*>(kv8_pool);
  return norm_rope_call(p, true, head_dim, num_tokens, interleaved, stream);
}
