// score_mod_host.h -- checks of the score arguments of the attention calls with changed scores.
#pragma once

#include <cmath>

#include "api_common.h"
#include "score_mod.cuh"

namespace ra {

inline ra_status score_mod(ScoreMod* mod, float sm_scale, float score_cap, int32_t window, const float* slopes,
                           const int32_t* first_key, const int32_t* full_lens) {
  RA_REQUIRE(std::isfinite(sm_scale) && sm_scale > 0.f, "sm_scale must be finite and > 0");
  RA_REQUIRE(std::isfinite(score_cap) && score_cap >= 0.f, "score_cap must be finite and > 0, or 0 for none");
  RA_REQUIRE(window >= 0, "window must be > 0, or 0 for none (got %d)", window);
  RA_REQUIRE(aligned4(slopes) && aligned4(first_key) && aligned4(full_lens),
             "slopes, first_key and full_lens must be 4-byte aligned");
  mod->slopes = slopes;
  mod->first_key = first_key;
  mod->full_lens = full_lens;
  mod->window = window;
  mod->in2 = make_float2(sm_scale * kLog2e, sm_scale * kLog2e);
  if (score_cap > 0.f) {
    // beyond these the cap's products leave fp32 (and no score of one is anything but 0 or uncapped)
    RA_REQUIRE(score_cap >= 1e-6f && score_cap <= 1e12f, "score_cap must be in [1e-6, 1e12]");
    mod->cap_in = sm_scale / score_cap;
    RA_REQUIRE(mod->cap_in < 1e30f && mod->cap_in > 1e-30f, "sm_scale / score_cap out of range");
    mod->in2 = make_float2(mod->cap_in, mod->cap_in);
    mod->exp2y = make_float2(2.f * mod->cap_in * kLog2e, 2.f * mod->cap_in * kLog2e);
    mod->cap_log2 = score_cap * kLog2e;
    for (int i = 0; i < kCapTerms; ++i) mod->cap_poly[i] = make_float2(mod->cap_log2 * cap_coef(i), mod->cap_log2 * cap_coef(i));
  }
  return RA_OK;
}

}  // namespace ra
