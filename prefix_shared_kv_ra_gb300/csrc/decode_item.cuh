// decode_item.cuh -- the work items of a decode call's plan, as the decode kernels read them.
#pragma once

#include "decode_internal.h"

namespace ra {

// One work item: keys [k0, k1) of request b for the kv heads of head group hg; d is its dense index
// (request-major: the item's partial results live at d).
struct Item {
  int32_t b, split, hg, k0, k1, start, n_splits, row, d;
};

// Claim `idx` = (position in the plan's longest-first order) * n_hgroups + hg.  The plan (written by
// decode_plan_kernel) lists only non-empty items of valid requests.  Plan arrays are read with plain
// loads: they are written on the device by the kernel before this one.
template <bool MOD = false>
__device__ __forceinline__ void decode_item(const DecodeParams& p, int32_t idx, Item& it) {
  it.hg = idx % p.n_hgroups;
  it.d = p.order[idx / p.n_hgroups];
  it.b = p.item_req[it.d];
  const int32_t i0 = p.req_item0[it.b];
  it.split = it.d - i0;
  it.n_splits = p.req_item0[it.b + 1] - i0;
  it.row = __ldg(p.rpi + it.b);
  const int32_t L = min(__ldg(p.seq_lens + it.b), p.max_seq_len);
  if constexpr (MOD) {
    it.start = mod_start(p, it.b, L);
  } else {
    const int32_t start = p.key_start ? __ldg(p.key_start + it.b) : 0;
    it.start = start < 0 ? 0 : (start > L ? L : start);
  }
  const int32_t chunk = p.plan[1];
  it.k0 = it.start + it.split * chunk;
  it.k1 = min(L, it.k0 + chunk);
}

}  // namespace ra
