// small_plan.cuh -- the split of a small batch's key ranges, made by every warp for itself.
//
// A call of few requests and keys is over in a few microseconds, of which a planning kernel took three.  With at
// most 32 requests a warp holds one per lane: it reads their lengths, finds the piece length for which all pieces
// of all head groups fit the grid at once (one per CTA: no claims, no counters), and looks items up by shuffles.
// Every warp of the attention and merge kernels repeats this on the same inputs and gets the same split.
#pragma once

#include <stdint.h>

namespace ra {

constexpr int kSmallBatch = 32;
constexpr int kSmallUnit = 32;    // keys per unit
constexpr int kSmallRounds = 48;  // mean units per CTA, at the host's bounds, up to which a call is small
constexpr int kSmallSms = 152;    // GB300; a constant, so that host and device agree

// Whether a call is small, from the host's bounds.  Its pieces have to fit: sum ceil(u / c) <= U / c + batch.  The
// bound on the mean keeps the loss of the coarser schedule (up to a third: one piece per CTA, all as long as
// the longest) below what the planning kernel costs.  Measured, planning kernel and small call, at their mean
// units: quantised decode of 16 requests of 512..4096 keys (13) 25.9 and 20.6 us, of 1000..13700 (45) 50.9 and
// 46.4, of 30 of 13000..13700 (85) 137.4 and 137.1; 16 x 4..8 drafted tokens over 512..4096 keys (27) 40.9 and
// 36.5, 30 x 4..8 (51) 62.9 and 65.5.
inline bool small_call(int64_t batch, int64_t max_keys, int64_t heads, int64_t per_sm) {
  const int64_t ctas = kSmallSms * per_sm;
  return batch <= kSmallBatch && 2 * batch * heads <= ctas &&
         batch * ((max_keys + kSmallUnit - 1) / kSmallUnit) * heads <= kSmallRounds * ctas;
}

struct SmallPlan {
  int32_t pieces;  // of this lane's request
  int32_t first;   // its first piece
  int32_t chunk;   // keys per piece
  int32_t n;       // pieces of all requests

  // keys: of this lane's request (0: none).  Warp-collective, as all members.
  __device__ __forceinline__ void make(int32_t keys, int32_t heads, int32_t ctas, int32_t least) {
    const int lane = threadIdx.x & 31;
    const int32_t units = (keys + kSmallUnit - 1) / kSmallUnit;
    const int32_t all = __reduce_add_sync(0xffffffffu, units) * heads;
    int32_t c = max(least, (all + ctas - 1) / ctas);
    for (;;) {
      pieces = (units + c - 1) / c;
      n = __reduce_add_sync(0xffffffffu, pieces);
      if (n * heads <= ctas) break;  // (at the latest with one piece per request)
      c += max(1, c >> 4);
    }
    chunk = c * kSmallUnit;
    first = pieces;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, first, off);
      if (lane >= off) first += y;
    }
    first -= pieces;
  }
  // The request of piece d < n.
  __device__ __forceinline__ int32_t request(int32_t d) const {
    return 31 - __clz(__ballot_sync(0xffffffffu, pieces > 0 && first <= d));
  }
};

__device__ __forceinline__ int32_t of_lane(int32_t x, int32_t lane) { return __shfl_sync(0xffffffffu, x, lane); }

}  // namespace ra
