// score_mod.cuh -- scores capped by a tanh and their masks, shared by the attention kernels with changed scores.
//
// A capped score is cap tanh(s / cap), wanted as t = cap log2(e) tanh(y) with y = s sm_scale / cap for the base-2
// exponential.  The hardware's tanh is good to about 2^-11 only: at a score of 20 that is 1% of the weight, more than
// the rounding of the weights to bf16.  Two forms of it are used:
//  * 1 - 2 / (e^2y + 1), off by about 2^-22 everywhere: at a cap of 55 that is 2e-5 of a weight (the extend pass with a fixed
//    reference, whose caps are that small);
//  * for larger caps, and in decode, a polynomial of degree 6 in y^2 times y where |y| <= 1.25 (a minimax fit of the
//    relative error, 7e-7 in fp32 arithmetic: at a score of 50, 4e-5 of the weight), and the first form beyond, where it
//    no longer cancels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ra_ptx.cuh"

namespace ra {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kCapPolyMax = 1.25f;
constexpr int kCapTerms = 7;
constexpr float kCapFixed = 80.f;
__host__ __device__ __forceinline__ constexpr float cap_coef(int i) {
  constexpr float c[kCapTerms] = {0.9999994039535522f,    -0.3332934081554413f, 0.1329064816236496f, -0.052205443382263184f,
                                  0.018229123204946518f, -0.004626905079931021f, 0.0005844939732924104f};
  return c[i];
}

struct ScoreMod {
  const float* slopes;       // [hq] bias per position of distance (subtracted), or nullptr
  const int32_t* first_key;  // first position that a row sees ([total_q], decode: [batch]), or nullptr
  const int32_t* full_lens;  // extend: [batch], positions below it are seen by every row; or nullptr
  int32_t window;            // keys a row sees up to its own, 0: all
  float cap_in;              // sm_scale / cap (0: no cap)
  float cap_log2;            // cap log2(e)
  float2 in2;                  // pairs of equal values: cap_in, or sm_scale log2(e) without a cap;
  float2 exp2y;                // 2 cap_in log2(e): 2^(s exp2y) = e^(2 y)
  float2 cap_poly[kCapTerms];  // cap log2(e) times the coefficients
};

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(y), |y| <= kCapPolyMax.
__device__ __forceinline__ float tanh_small(float y) {
  const float z = y * y;
  float p = cap_coef(kCapTerms - 1);
#pragma unroll
  for (int i = kCapTerms - 2; i >= 0; --i) p = fmaf(p, z, cap_coef(i));
  return y * p;
}

// tanh(y) of any y; NaN stays.
__device__ __forceinline__ float tanh_any(float y) {
  const float a = fabsf(y);
  const float far = 1.f - 2.f * rcp_approx(ex2(a * (2.f * kLog2e)) + 1.f);
  return a <= kCapPolyMax ? tanh_small(y) : copysignf(far, y);
}

}  // namespace ra
