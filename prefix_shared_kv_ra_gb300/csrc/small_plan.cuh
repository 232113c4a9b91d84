// small_plan.cuh -- the split of a small batch's key ranges, made by every warp for itself.
//
// A call of few requests and keys is over in a few microseconds, of which a planning kernel took three.  With at
// most 64 requests a warp holds one or two per lane: it reads their lengths, finds the piece length for which all pieces
// of all head groups fit the grid at once (one per CTA: no claims, no counters), and looks items up by shuffles.
// Every warp of the attention and merge kernels repeats this on the same inputs and gets the same split.
#pragma once

#include <stdint.h>

namespace ra {

constexpr int kSmallBatch = 64;
constexpr int kSmallUnit = 32;    // keys per unit
constexpr int kSmallRounds = 48;  // mean units per CTA, at the host's bounds, up to which a call is small
constexpr int kSmallRoundsMany = 16;  // the same for more than 32 requests
constexpr int kSmallSms = 152;    // GB300; a constant, so that host and device agree

// Whether a call is small, from the host's bounds.  Its pieces have to fit: sum ceil(u / c) <= U / c + batch.  The
// bound on the mean keeps the loss of the coarser schedule (up to a third: one piece per CTA, all as long as
// the longest) below what the planning kernel costs.  Measured, planning kernel and small call, at their mean
// units: quantised decode of 16 requests of 512..4096 keys (13) 22.8 and 20.4 us, of 24 of 5000..8000 (39) 60.4 and
// 59.2; 16 x 4..8 drafted tokens over 512..4096 keys (27) 40.9 and 36.5, 30 x 4..8 (51) 62.9 and 65.5.  With more
// than 32 requests the pieces are coarser and the bound is lower: quantised decode of 64 requests of 200..1000 keys
// (13) 24.1 and 22.2, of 500..1500 (20) 30.9 and 31.8; 64 x 4..7 drafted tokens over 100..1000 keys (13) 27.5 and
// 22.9, over 1000..2000 (27) 43.4 and 44.2.
inline bool small_call(int64_t batch, int64_t max_keys, int64_t heads, int64_t per_sm) {
  const int64_t ctas = kSmallSms * per_sm;
  return batch <= kSmallBatch && 2 * batch * heads <= ctas &&
         batch * ((max_keys + kSmallUnit - 1) / kSmallUnit) * heads <=
             (batch <= 32 ? kSmallRounds : kSmallRoundsMany) * ctas;
}

// A lane's values of request `lane` (N = 1), or of `lane` and `lane` + 32 (N = 2: for 33 requests or more).
template <int N>
struct PerRequest {
  int32_t v[N] = {};
};
// The value of request r (the same for the whole warp).
template <int N>
__device__ __forceinline__ int32_t of_request(const PerRequest<N>& x, int32_t r) {
  return __shfl_sync(0xffffffffu, N == 1 || r < 32 ? x.v[0] : x.v[N - 1], r & 31);
}

template <int N>
struct SmallPlan {
  PerRequest<N> pieces;
  PerRequest<N> first;  // the request's first piece
  int32_t chunk;     // keys per piece
  int32_t n;         // pieces of all requests

  // keys: of the requests (0: none).  Warp-collective, as all members.
  __device__ __forceinline__ void make(const PerRequest<N>& keys, int32_t heads, int32_t ctas, int32_t least) {
    PerRequest<N> units;
    int32_t all = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      units.v[i] = (keys.v[i] + kSmallUnit - 1) / kSmallUnit;
      all += units.v[i];
    }
    all = __reduce_add_sync(0xffffffffu, all) * heads;
    int32_t c = max(least, (all + ctas - 1) / ctas);
    for (;;) {
      n = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) n += pieces.v[i] = (units.v[i] + c - 1) / c;
      n = __reduce_add_sync(0xffffffffu, n);
      if (n * heads <= ctas) break;  // (at the latest with one piece per request)
      c += max(1, c >> 4);
    }
    chunk = c * kSmallUnit;
    first.v[0] = before(pieces.v[0]);
    if constexpr (N == 2)
      first.v[1] = before(pieces.v[1]) + __shfl_sync(0xffffffffu, first.v[0] + pieces.v[0], 31);
  }
  // The request of piece d < n.
  __device__ __forceinline__ int32_t request(int32_t d) const {
    const uint32_t lo = __ballot_sync(0xffffffffu, pieces.v[0] > 0 && first.v[0] <= d);
    if constexpr (N == 2) {
      const uint32_t hi = __ballot_sync(0xffffffffu, pieces.v[1] > 0 && first.v[1] <= d);
      if (hi) return 63 - __clz(hi);
    }
    return 31 - __clz(lo);
  }

 private:
  // Sum of x over the lanes below.
  static __device__ __forceinline__ int32_t before(int32_t x) {
    const int lane = threadIdx.x & 31;
    int32_t sum = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += y;
    }
    return sum - x;
  }
};

}  // namespace ra
