// tree_verify.cu -- verification of drafted trees: ra_tree_verify (against the target's probabilities, from given random
// numbers) and ra_tree_verify_greedy (against the largest logit).
//
// One cluster of CTAs per request.  Warp 0 of each CTA walks the tree, every CTA the same way, with the tree in shared
// memory; the CTAs meet only where a whole row of the vocabulary is needed, each taking a slice of it.
//
// Sampling.  With p the target's row of a node and q the drafts', the residual after j refusals of tokens drawn from q is
// r_j ~ max(r_{j-1} - q, 0) (r normalised), which unrolls to r_j = max(p - t_j q, 0) with t_j = t_{j-1} + S_{j-1},
// S_j = sum_v max(p_v - t_j q_v, 0), t_0 = 0, S_0 = 1: a refusal costs one pass over the two rows and keeps nothing per
// token.  An acceptance costs none: child x is accepted when u q(x) S < max(p(x) - t q(x), 0), and p(x), q(x), u of all
// nodes are gathered before the walk in one round trip.  Drafts taken as given need no pass at all for the walk (the
// residual is p without the refused tokens).  The next token needs one: the sums of the last residual over each warp's
// slice, then the slice that holds u S, then its place there.
//
// Precision: the drawn token is a whole number that depends on where u S falls between neighbouring prefix sums, as little
// as 1e-9 apart at a vocabulary of 100,000; fp32 sums would move one draw in hundreds.  p - t q, the sums and what they are
// compared with are held as pairs of floats (unevaluated sums, about 2^-45 of a whole row's) in the fp32 pipe: this GPU's 64-bit
// rate is two values a clock and SM, and even the few scans and comparisons of a draw took 5 us of a call in it.
//
// Bound: the rows read, once each (a pass over 64 pairs of rows of 128,000 is 66 MB, 10 us of HBM), and for few requests
// the chain of gather, pass and search, about 1.5 us each.  64 trees of 8..16 drafts drawn from q over 128,000 tokens: 28 to
// 38 us by the draw, the time of the requests with the most refusals; 64 greedy trees of 32..64: 40 to 46 (logits in fp32
// 50), that of the longest accepted paths (11 rows one after another, 3.4 us each); 4 trees of given drafts: 7.
#include <cuda_bf16.h>

#include "api_common.h"
#include "ra_ptx.cuh"

namespace ra {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxTree = 1024;  // drafted tokens of a request

// Let the next kernel launch, every write of this CTA visible to it (the planning kernels of the attention calls read
// lengths before they wait for the kernel before them).
__device__ __forceinline__ void launch_behind_writes() {
  __threadfence();
  __syncthreads();
  griddep_launch();
}

// ---- unevaluated sums of two floats, |lo| at most half a last place of hi where they are results (error-free
// transformations: of a sum, Knuth; of a product, one fma)
struct Pair {
  float hi, lo;
};
// The rounding error of s = a + b.
__device__ __forceinline__ float sum_error(float a, float b, float s) {
  const float bb = __fsub_rn(s, a);
  return __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
}
__device__ __forceinline__ Pair pair_of(float hi, float lo) {  // |lo| well below |hi|
  const float s = __fadd_rn(hi, lo);
  return {s, __fsub_rn(lo, __fsub_rn(s, hi))};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  const float s = __fadd_rn(a.hi, b.hi);
  return pair_of(s, __fadd_rn(sum_error(a.hi, b.hi, s), __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ Pair operator-(Pair a, Pair b) { return a + Pair{-b.hi, -b.lo}; }
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  const float m = __fmul_rn(a.hi, b.hi);
  return pair_of(m, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, __fmaf_rn(a.hi, b.hi, -m))));
}
__device__ __forceinline__ bool operator<(Pair a, Pair b) { return (a - b).hi < 0.f; }
// Running sums: two floats' worth without the normalisation of every step.
__device__ __forceinline__ void pair_add(Pair& acc, float x) {
  const float s = __fadd_rn(acc.hi, x);
  acc.lo = __fadd_rn(acc.lo, sum_error(acc.hi, x, s));
  acc.hi = s;
}
__device__ __forceinline__ Pair pair_shfl(Pair a, int lane) {
  return {__shfl_sync(0xffffffffu, a.hi, lane), __shfl_sync(0xffffffffu, a.lo, lane)};
}
__device__ __forceinline__ Pair pair_reduce(Pair a) {  // over the warp; lane 0's result counts
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    a = a + Pair{__shfl_xor_sync(0xffffffffu, a.hi, off), __shfl_xor_sync(0xffffffffu, a.lo, off)};
  return a;
}
__device__ __forceinline__ Pair pair_scan(Pair a) {  // inclusive, over the warp
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Pair b{__shfl_up_sync(0xffffffffu, a.hi, off), __shfl_up_sync(0xffffffffu, a.lo, off)};
    if (lane >= off) a = a + b;
  }
  return a;
}

// max(p - t q, 0); 0 also for a NaN.
__device__ __forceinline__ Pair residual(float p, float q, Pair t) {
  const float m = __fmul_rn(t.hi, q), d = __fsub_rn(p, m);
  const Pair r = pair_of(d, __fmaf_rn(-t.lo, q, __fsub_rn(sum_error(p, -m, d), __fmaf_rn(t.hi, q, -m))));
  return r.hi > 0.f ? r : Pair{0.f, 0.f};
}

// The first lane whose prefix sum exceeds the goal (`base`, then the lanes' values in turn), and the sum before it; where
// there is none, the last lane with any weight.  Warp-collective.
__device__ __forceinline__ int place(Pair mine, Pair base, Pair goal, Pair* before) {
  const Pair incl = base + pair_scan(mine);
  const uint32_t over = __ballot_sync(0xffffffffu, goal < incl && mine.hi > 0.f);
  const uint32_t some = __ballot_sync(0xffffffffu, mine.hi > 0.f);
  const int at = over ? __ffs(over) - 1 : some ? 31 - __clz(some) : 0;
  *before = at > 0 ? pair_shfl(incl, (at + 31) & 31) : base;
  return at;
}

struct VerifyParams {
  const float* target;  // [total_q, vocab] rows at target_stride
  int64_t target_stride;
  const float* draft;  // likewise, or nullptr: drafts taken as given
  int64_t draft_stride;
  int32_t vocab;
  const int32_t *tokens, *parents, *draft_lens, *qo_indptr;
  const float *u_accept, *u_final;
  int64_t total_q;
  int32_t max_draft;
  int32_t *path, *accept_lens, *next_tokens;
  uint32_t* err;
};

// What the walk of a request holds in shared memory.
struct Tree {
  int32_t token[kMaxTree];
  int32_t parent[kMaxTree];
};

// The request's length and first row; 0 drafted tokens where there is nothing to verify (flagged if wrong).
__device__ __forceinline__ int32_t request_rows(const int32_t* draft_lens, const int32_t* qo_indptr, int32_t b,
                                                int32_t max_draft, int64_t total_q, int64_t* first, uint32_t* err,
                                                bool report) {
  const int32_t T = __ldg(draft_lens + b);
  *first = __ldg(qo_indptr + b);
  if (T >= 0 && T <= max_draft && *first >= 0 && *first + T <= total_q) return T;
  if (report) flag_error(err, RA_DEVERR_LENGTH);
  return 0;
}

// First child of `node` behind node `after`, or T (warp-collective, the same in every lane).
__device__ __forceinline__ int32_t next_child(const Tree& tree, int32_t node, int32_t after, int32_t T) {
  const int lane = threadIdx.x & 31;
  for (int32_t i = after + 1; i < T; i += 32) {
    const uint32_t hit = __ballot_sync(0xffffffffu, i + lane < T && tree.parent[i + lane] == node);
    if (hit) return i + __ffs(hit) - 1;
  }
  return T;
}

// Whether a child of `node` before `child` has its token (warp-collective).
__device__ __forceinline__ bool refused_before(const Tree& tree, int32_t node, int32_t child) {
  const int lane = threadIdx.x & 31;
  for (int32_t i = node + 1; i < child; i += 32) {
    const bool same = i + lane < child && tree.parent[i + lane] == node && tree.token[i + lane] == tree.token[child];
    if (__any_sync(0xffffffffu, same)) return true;
  }
  return false;
}

// A request of a padded batch, or one whose lengths are wrong.
__device__ __forceinline__ void nothing_verified(int32_t* path, int32_t* accept_lens, int32_t* next_tokens, int32_t b,
                                                 int32_t max_draft) {
  for (int32_t i = threadIdx.x; i < max_draft; i += kThreads) path[static_cast<int64_t>(b) * max_draft + i] = -1;
  if (threadIdx.x == 0) accept_lens[b] = next_tokens[b] = 0;
}

enum Command { kSum = 0, kDraw = 1 };

template <bool DRAWN>
__global__ void __launch_bounds__(kThreads, 2) tree_verify_kernel(const VerifyParams p, int32_t ctas) {
  __shared__ Tree s_tree;
  __shared__ float s_p[kMaxTree], s_q[kMaxTree], s_u[kMaxTree];
  __shared__ int32_t s_path[kMaxTree];
  __shared__ Pair s_warp[kWarps];                      // this CTA's slices' sums
  __shared__ __align__(8) Pair s_rank[2][kMaxCluster];  // every CTA's sum, by the pass's parity
  __shared__ int32_t s_command, s_node, s_more, s_owner, s_who;
  __shared__ Pair s_part[kWarps];
  __shared__ Pair s_t, s_total, s_before, s_goal;
  cluster_arrive();  // (waited for before the first store into another CTA's shared memory: it has to have started)
  griddep_wait();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int32_t b = blockIdx.x / ctas;
  const uint32_t rank = cluster_rank();
  int64_t first;
  const int32_t T = request_rows(p.draft_lens, p.qo_indptr, b, p.max_draft, p.total_q, &first, p.err, rank == 0 && t == 0);
  if (T == 0) {  // (the whole cluster)
    if (rank == 0) nothing_verified(p.path, p.accept_lens, p.next_tokens, b, p.max_draft);
    cluster_wait();
    launch_behind_writes();
    return;
  }
  for (int32_t i = t; i < T; i += kThreads) {
    const int32_t x = __ldg(p.tokens + first + i), parent = __ldg(p.parents + first + i);
    const bool known = x >= 0 && x < p.vocab, child = i > 0 && parent >= 0 && parent < i;
    s_tree.token[i] = x;
    s_tree.parent[i] = child ? parent : -1;
    if (child && !known && rank == 0) flag_error(p.err, RA_DEVERR_VALUE);
    const int64_t row = first + parent;
    s_p[i] = child && known ? fmaxf(__ldg(p.target + row * p.target_stride + x), 0.f) : 0.f;
    if (DRAWN) s_q[i] = child && known ? fmaxf(__ldg(p.draft + row * p.draft_stride + x), 0.f) : 0.f;
    s_u[i] = __ldg(p.u_accept + first + i);
  }
  const float u_final = __ldg(p.u_final + b);
  // this warp's slice of a row
  const int32_t slice = (p.vocab + ctas * kWarps - 1) / (ctas * kWarps);
  const int64_t begin = static_cast<int64_t>(slice) * (rank * kWarps + warp);
  const int32_t v0 = static_cast<int32_t>(begin < p.vocab ? begin : p.vocab);
  const int32_t v1 = static_cast<int32_t>(begin + slice < p.vocab ? begin + slice : p.vocab);
  __syncthreads();
  cluster_wait();

  const Pair kNone{0.f, 0.f}, kOne{1.f, 0.f};
  // The walk's state, in every lane of warp 0.
  int32_t node = 0, child = 0, count = 1;
  Pair tq = kNone, total = kOne;
  if (t == 0) s_path[0] = 0;
  for (int32_t pass = 0;; ++pass) {
    if (warp == 0) {
      // on from the last refused child until a row is needed
      int32_t command = kDraw;
      for (;;) {
        child = next_child(s_tree, node, child, T);
        if (child == T) break;
        const Pair u{s_u[child], 0.f};
        const float px = s_p[child], qx = DRAWN ? s_q[child] : 1.f;
        Pair r{px, 0.f};
        if (DRAWN) {
          r = residual(px, qx, tq);
        } else if (refused_before(s_tree, node, child)) {
          r = kNone;  // a token refused at this node already has no weight left
        }
        if (u * Pair{qx, 0.f} * total < r) {
          if (lane == 0) s_path[count] = child;
          ++count;
          node = child;  // (its children are behind it)
          tq = kNone;
          total = kOne;
          continue;
        }
        if (DRAWN) {
          tq = tq + total;
          command = kSum;
          break;
        }
        total = total - r;
      }
      if (lane == 0) {
        s_command = command;
        s_node = node;
        s_t = tq;
      }
    }
    __syncthreads();
    const bool draw = s_command == kDraw;
    const int32_t at = s_node;
    Pair tt = s_t;
    const float* prow = p.target + (first + at) * p.target_stride;
    const float* qrow = DRAWN ? p.draft + (first + at) * p.draft_stride : nullptr;
    bool plain = DRAWN && tt.hi == 0.f;  // the residual is p itself
    // given drafts: the children of the node (all were refused) with tokens in [from, to), each distinct token once
    // (warp-collective): f(child)
    auto for_refused = [&](int32_t from, int32_t to, auto f) {
      for (int32_t i = at; (i = next_child(s_tree, at, i, T)) < T;)
        if (s_tree.token[i] >= from && s_tree.token[i] < to && !refused_before(s_tree, at, i)) f(i);
    };
    bool holes = false;  // the tokens looked at include refused ones
    auto weight = [&](int32_t v) -> Pair {
      const float x = fmaxf(__ldg(prow + v), 0.f);
      if (DRAWN && !plain) return residual(x, fmaxf(__ldg(qrow + v), 0.f), tt);
      if (!DRAWN && holes) {
        for (int32_t i = at + 1; i < T; ++i)
          if (s_tree.parent[i] == at && s_tree.token[i] == v) return kNone;
      }
      return {x, 0.f};
    };
    // the sum of the residual over the row: each warp its slice, then the CTA, then the cluster
    auto row_sum = [&](int parity) -> Pair {
      // sum max(p - t q, 0) = (sum of p - t sum of q) over the tokens with p > t q: the sums of p and q of those are held as
      // pairs, a third fewer instructions than a pair per residual, and as good while the sum is not far below 1
      Pair acc = kNone, qacc = kNone;
      const bool both = DRAWN && !plain;
      int32_t v = v0 + lane;
      if (both) {
        constexpr int kU = 8;  // loads in flight per lane and row
        for (; v < v1; v += 32 * kU) {
          float x[kU], y[kU];
#pragma unroll
          for (int k = 0; k < kU; ++k) {
            const bool in = v + 32 * k < v1;
            x[k] = in ? __ldg(prow + v + 32 * k) : 0.f;
            y[k] = in ? __ldg(qrow + v + 32 * k) : 0.f;
          }
#pragma unroll
          for (int k = 0; k < kU; ++k) {
            y[k] = fmaxf(y[k], 0.f);
            // (the first fma has the sign of the exact difference)
            const bool keep = __fmaf_rn(-tt.lo, y[k], __fmaf_rn(-tt.hi, y[k], x[k])) > 0.f;
            pair_add(acc, keep ? x[k] : 0.f);
            pair_add(qacc, keep ? y[k] : 0.f);
          }
        }
      } else {
        constexpr int kU = 16;
        for (; v < v1; v += 32 * kU) {
          float x[kU];
#pragma unroll
          for (int k = 0; k < kU; ++k) x[k] = v + 32 * k < v1 ? __ldg(prow + v + 32 * k) : 0.f;
#pragma unroll
          for (int k = 0; k < kU; ++k) pair_add(acc, fmaxf(x[k], 0.f));
        }
      }
      acc = pair_reduce(pair_of(acc.hi, acc.lo));
      if (both) {
        acc = acc - tt * pair_reduce(pair_of(qacc.hi, qacc.lo));
      } else if (!DRAWN && !plain) {
        for_refused(v0, v1, [&](int32_t i) { acc = acc - Pair{s_p[i], 0.f}; });
      }
      if (!(acc.hi > 0.f) && acc.hi == acc.hi) acc = kNone;  // (rounding; a NaN stays)
      if (lane == 0) s_warp[warp] = acc;
      __syncthreads();
      if (warp == 0) {
        const Pair sum = pair_reduce(lane < kWarps ? s_warp[lane] : kNone);
        const uint64_t bits = static_cast<uint64_t>(__float_as_uint(sum.lo)) << 32 | __float_as_uint(sum.hi);
        const uint64_t first_bits = __shfl_sync(0xffffffffu, bits, 0);
        if (lane < ctas) st_cluster_b64(smem_u32(&s_rank[parity][rank]), lane, first_bits);
      }
      cluster_sync_all();
      if (warp == 0) {
        const Pair sum = pair_reduce(lane < ctas ? s_rank[parity][lane] : kNone);
        if (lane == 0) s_total = sum;
      }
      __syncthreads();
      return s_total;
    };
    Pair sum = row_sum(pass & 1);
    if (!draw) {
      total = sum;
      // the last refused child may have been the node's last: then this sum is the draw's
      if (warp == 0) {
        const int32_t more = next_child(s_tree, node, child, T);
        if (lane == 0) s_more = more < T;
      }
      __syncthreads();
      if (s_more) continue;
    }
    int parity = pass & 1;
    if (!(sum.hi > 0.f) && !plain) {
      // nothing left of the residual (rounding, or refused tokens that held all of p): p itself
      __syncthreads();
      plain = true;
      sum = row_sum(parity ^= 1);
    }
    if (!(sum.hi > 0.f && sum.hi < INFINITY)) {  // (also a NaN)
      if (rank == 0) {
        if (t == 0) flag_error(p.err, RA_DEVERR_VALUE), p.next_tokens[b] = 0;
      }
    } else {
      // The CTA, then the warp's slice where the prefix sums first exceed u S, by warp 0 of every CTA; then the owner's
      // whole CTA over that slice.  Where rounding leaves no place, the last with any weight.
      if (warp == 0) {
        const Pair goal = Pair{u_final, 0.f} * sum;
        Pair before;
        const int owner = place(lane < ctas ? s_rank[parity][lane] : kNone, kNone, goal, &before);
        if (lane == 0) s_owner = owner;
        if (owner == static_cast<int>(rank)) {
          const int who = place(lane < kWarps ? s_warp[lane] : kNone, before, goal, &before);
          if (lane == 0) s_who = who, s_before = before, s_goal = goal;
        }
      }
      __syncthreads();
      if (s_owner == static_cast<int>(rank)) {
        const int64_t slice0 = static_cast<int64_t>(slice) * (rank * kWarps + s_who);
        const int32_t e0 = static_cast<int32_t>(slice0 < p.vocab ? slice0 : p.vocab);
        const int32_t e1 = static_cast<int32_t>(slice0 + slice < p.vocab ? slice0 + slice : p.vocab);
        const int32_t part = (e1 - e0 + kWarps - 1) / kWarps;
        const int32_t c0 = min(e0 + warp * part, e1), c1 = min(c0 + part, e1);
        if (!DRAWN && !plain) for_refused(c0, c1, [&](int32_t) { holes = true; });
        const Pair goal = s_goal;
        Pair before = s_before, acc = kNone;
        for (int32_t v = c0 + lane; v < c1; v += 32) acc = acc + weight(v);
        acc = pair_reduce(acc);
        if (lane == 0) s_part[warp] = acc;
        __syncthreads();
        const int who = place(lane < kWarps ? s_part[lane] : kNone, before, goal, &before);
        if (who == warp) {
          // the groups of 32 tokens in turn
          int32_t found = -1, tail = c0;
          for (int32_t v = c0; v < c1 && found < 0; v += 32) {
            const Pair w = v + lane < c1 ? weight(v + lane) : kNone;
            const Pair incl = before + pair_scan(w);
            const uint32_t over = __ballot_sync(0xffffffffu, goal < incl && w.hi > 0.f);
            const uint32_t any = __ballot_sync(0xffffffffu, w.hi > 0.f);
            if (over) found = v + __ffs(over) - 1;
            if (any) tail = v + 31 - __clz(any);
            before = pair_shfl(incl, 31);
          }
          if (lane == 0) p.next_tokens[b] = found >= 0 ? found : tail;
        }
      }
    }
    __syncthreads();
    if (rank == 0) {
      // (warp 0's count, through the path's end)
      if (t == 0) p.accept_lens[b] = count, s_node = count;
      __syncthreads();
      for (int32_t i = t; i < p.max_draft; i += kThreads)
        p.path[static_cast<int64_t>(b) * p.max_draft + i] = i < s_node ? s_path[i] : -1;
    }
    launch_behind_writes();
    return;
  }
}

// ------------------------------------------------------------------ the largest logit
struct GreedyParams {
  const void* logits;  // [total_q, vocab] rows at stride
  int64_t stride;
  int32_t vocab;
  const int32_t *tokens, *parents, *draft_lens, *qo_indptr;
  int64_t total_q;
  int32_t max_draft;
  int32_t *path, *accept_lens, *next_tokens;
  uint32_t* err;
};

// A value and its token as one ordered key: larger values first, then lower tokens.  0 for a NaN; -0 counts as 0.
__device__ __forceinline__ uint64_t key_of(float x, int32_t v) {
  if (!(x == x)) return 0;
  const uint32_t u = __float_as_uint(x + 0.f);
  const uint32_t ordered = u & 0x80000000u ? ~u : u | 0x80000000u;
  return static_cast<uint64_t>(ordered) << 32 | (0xffffffffu - static_cast<uint32_t>(v));
}
__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }
// The warp's largest, in two 32-bit reductions (five shuffle steps of 64 bits took longer than the row's loads).
__device__ __forceinline__ uint64_t warp_max64(uint64_t x) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(x >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(x >> 32) == hi ? static_cast<uint32_t>(x) : 0u);
  return static_cast<uint64_t>(hi) << 32 | lo;
}

template <typename E>
__device__ __forceinline__ float value_of(E x);
template <>
__device__ __forceinline__ float value_of<float>(float x) { return x; }
template <>
__device__ __forceinline__ float value_of<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

// The largest key of this thread's share of a row: 16-byte vectors of the aligned middle, the ends value by value.
template <typename E>
__device__ __forceinline__ uint64_t row_largest(const E* row, int32_t vocab, int64_t worker, int64_t workers) {
  constexpr int kPer = 16 / sizeof(E);
  const int32_t skew = static_cast<int32_t>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(E));
  int32_t head = skew ? kPer - skew : 0;
  if (head > vocab) head = vocab;
  const int32_t vecs = (vocab - head) / kPer;
  uint64_t best = 0;
  if (worker < head) best = key_of(value_of(row[worker]), static_cast<int32_t>(worker));
  const int32_t tail = head + vecs * kPer;
  if (worker < vocab - tail) best = max64(best, key_of(value_of(row[tail + worker]), tail + static_cast<int32_t>(worker)));
  const uint4* mid = reinterpret_cast<const uint4*>(row + head);
  float top = -INFINITY;
  int32_t top_v = -1;
  constexpr int kU = 4;
  for (int64_t i0 = worker; i0 < vecs; i0 += kU * workers) {
    uint4 x[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int64_t i = i0 + k * workers;
      x[k] = i < vecs ? __ldg(mid + i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int64_t i = i0 + k * workers;
      if (i >= vecs) break;
      const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
      float f[kPer];
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if constexpr (sizeof(E) == 4) f[e] = __uint_as_float(w[e]);
        else f[e] = __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
      }
      // the vector's largest first (fmaxf passes over a NaN): its place only where it is the thread's
      float m = f[0];
#pragma unroll
      for (int e = 1; e < kPer; ++e) m = fmaxf(m, f[e]);
      if (m > top || (top_v < 0 && m == m)) {
        top = m;
        const int32_t v = head + static_cast<int32_t>(i) * kPer;
#pragma unroll
        for (int e = kPer - 1; e >= 0; --e)
          if (f[e] == m) top_v = v + e;
      }
    }
  }
  return top_v < 0 ? best : max64(best, key_of(top, top_v));
}

template <typename E>
__global__ void __launch_bounds__(kThreads, 2) tree_verify_greedy_kernel(const GreedyParams p, int32_t ctas) {
  __shared__ Tree s_tree;
  __shared__ int32_t s_path[kMaxTree];
  __shared__ uint64_t s_warp[kWarps];
  __shared__ uint64_t s_rank[2][kMaxCluster];
  __shared__ int32_t s_next, s_token;
  cluster_arrive();  // (waited for before the first store into another CTA's shared memory: it has to have started)
  griddep_wait();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int32_t b = blockIdx.x / ctas;
  const uint32_t rank = cluster_rank();
  int64_t first;
  const int32_t T = request_rows(p.draft_lens, p.qo_indptr, b, p.max_draft, p.total_q, &first, p.err, rank == 0 && t == 0);
  if (T == 0) {  // (the whole cluster)
    if (rank == 0) nothing_verified(p.path, p.accept_lens, p.next_tokens, b, p.max_draft);
    cluster_wait();
    launch_behind_writes();
    return;
  }
  for (int32_t i = t; i < T; i += kThreads) {
    const int32_t x = __ldg(p.tokens + first + i), parent = __ldg(p.parents + first + i);
    const bool child = i > 0 && parent >= 0 && parent < i;
    s_tree.token[i] = x;
    s_tree.parent[i] = child ? parent : -1;
    if (child && (x < 0 || x >= p.vocab) && rank == 0) flag_error(p.err, RA_DEVERR_VALUE);
  }
  cluster_wait();
  int32_t node = 0, count = 0;
  for (int32_t pass = 0;; ++pass) {
    if (t == 0) s_path[count] = node;
    ++count;
    uint64_t best = row_largest(static_cast<const E*>(p.logits) + (first + node) * p.stride, p.vocab,
                                static_cast<int64_t>(rank) * kThreads + t, static_cast<int64_t>(ctas) * kThreads);
    best = warp_max64(best);
    if (lane == 0) s_warp[warp] = best;
    __syncthreads();
    if (warp == 0) {
      best = warp_max64(lane < kWarps ? s_warp[lane] : 0);
      if (lane < ctas) st_cluster_b64(smem_u32(&s_rank[pass & 1][rank]), lane, best);
    }
    cluster_sync_all();
    if (warp == 0) {
      best = warp_max64(lane < ctas ? s_rank[pass & 1][lane] : 0);
      // (0: a row of NaN; no child's token then)
      const int32_t token = best ? static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(best)) : -1;
      int32_t next = -1;
      for (int32_t i = node + 1; i < T && next < 0; i += 32) {
        const uint32_t hit = __ballot_sync(0xffffffffu, token >= 0 && i + lane < T && s_tree.parent[i + lane] == node &&
                                                            s_tree.token[i + lane] == token);
        if (hit) next = i + __ffs(hit) - 1;
      }
      if (lane == 0) s_next = next, s_token = token;
    }
    __syncthreads();
    if (s_next < 0) break;
    node = s_next;
  }
  if (rank == 0) {
    for (int32_t i = t; i < p.max_draft; i += kThreads)
      p.path[static_cast<int64_t>(b) * p.max_draft + i] = i < count ? s_path[i] : -1;
    if (t == 0) {
      if (s_token < 0) flag_error(p.err, RA_DEVERR_VALUE);
      p.accept_lens[b] = count;
      p.next_tokens[b] = max(s_token, 0);
    }
  }
  launch_behind_writes();
}

// CTAs per request: 8 (the most that any GPU of the architecture runs as one cluster) unless a slice would be less than four
// values per thread (64 trees of 16 drafts over 8,000 tokens, drawn / given / greedy: 12.3 / 8.6 / 14.7 us with 2 CTAs, 13.4 /
// 9.5 / 15.0 with 4), or the requests then no longer run all at once, two CTAs an SM (64 trees of 16 drafts, drawn /
// given / greedy, over 32,000 tokens: 12.5 / 9.9 / 17.7 us with 4 CTAs, 18.5 / 16.0 / 24.4 with 8 in two waves; over
// 128,000: 34.2 / 14.1 / 25.4 and 31.7 / 19.5 / 25.9).
int cluster_ctas(int32_t vocab, int32_t batch, int sms) {
  int c = kMaxCluster;
  while (c > 1 && static_cast<int64_t>(vocab) < static_cast<int64_t>(c) * kThreads * 4) c /= 2;
  while (c > 1 && static_cast<int64_t>(batch) * c > 2 * sms) c /= 2;
  return c;
}

template <typename Params>
ra_status launch_requests(const char* what, void (*kern)(Params, int32_t), int32_t batch, int ctas, cudaStream_t stream,
                          const Params& p) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(batch) * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p, static_cast<int32_t>(ctas));
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "%s launch failed: %s", what, cudaGetErrorString(e));
  return RA_OK;
}

ra_status check_sizes(int32_t batch, int64_t total_q, int32_t vocab, int32_t max_draft) {
  RA_REQUIRE(batch >= 0 && batch <= 65535, "batch must be in [0, 65535] (got %d)", batch);
  RA_REQUIRE(total_q >= 0 && total_q <= INT32_MAX, "total_q out of range");
  RA_REQUIRE(vocab >= 1 && vocab <= (1 << 28), "vocab must be in [1, 2^28] (got %d)", vocab);
  RA_REQUIRE(max_draft >= 1, "max_draft_len must be >= 1");
  if (max_draft > kMaxTree) return fail(RA_ERR_UNSUPPORTED, "max_draft_len %d (up to %d)", max_draft, kMaxTree);
  return RA_OK;
}

}  // namespace
}  // namespace ra

extern "C" ra_status ra_tree_verify(const float* target_probs, int64_t target_stride, const float* draft_probs,
                                    int64_t draft_stride, int32_t vocab, const int32_t* draft_tokens,
                                    const int32_t* parents, const int32_t* draft_lens, const int32_t* qo_indptr,
                                    const float* accept_uniforms, const float* final_uniforms, int32_t batch,
                                    int64_t total_q, int32_t max_draft_len, int32_t* path, int32_t* accept_lens,
                                    int32_t* next_tokens, uint32_t* device_error, ra_stream_t stream) {
  using namespace ra;
  clear_error();
  if (ra_status st = check_sizes(batch, total_q, vocab, max_draft_len)) return st;
  RA_REQUIRE(target_stride >= vocab && (!draft_probs || draft_stride >= vocab), "row strides must be >= vocab");
  if (batch == 0) return RA_OK;
  RA_REQUIRE(draft_lens && qo_indptr && final_uniforms && path && accept_lens && next_tokens, "null pointer argument");
  RA_REQUIRE(total_q == 0 || (target_probs && draft_tokens && parents && accept_uniforms), "null pointer argument");
  RA_REQUIRE(aligned4(target_probs) && aligned4(draft_probs) && aligned4(draft_tokens) && aligned4(parents) &&
                 aligned4(draft_lens) && aligned4(qo_indptr) && aligned4(accept_uniforms) && aligned4(final_uniforms) &&
                 aligned4(path) && aligned4(accept_lens) && aligned4(next_tokens),
             "arrays must be 4-byte aligned");
  const VerifyParams p{target_probs, target_stride, draft_probs, draft_stride, vocab,       draft_tokens,
                       parents,      draft_lens,    qo_indptr,   accept_uniforms, final_uniforms, total_q,
                       max_draft_len, path,         accept_lens, next_tokens,  device_error};
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DeviceInfo dev;
  if (ra_status st = current_device(&dev)) return st;
  const int ctas = cluster_ctas(vocab, batch, dev.num_sms);
  return draft_probs ? launch_requests("tree_verify_kernel", tree_verify_kernel<true>, batch, ctas, s, p)
                     : launch_requests("tree_verify_kernel", tree_verify_kernel<false>, batch, ctas, s, p);
}

extern "C" ra_status ra_tree_verify_greedy(const void* target_logits, int32_t logits_fp32, int64_t logits_stride,
                                           int32_t vocab, const int32_t* draft_tokens, const int32_t* parents,
                                           const int32_t* draft_lens, const int32_t* qo_indptr, int32_t batch,
                                           int64_t total_q, int32_t max_draft_len, int32_t* path, int32_t* accept_lens,
                                           int32_t* next_tokens, uint32_t* device_error, ra_stream_t stream) {
  using namespace ra;
  clear_error();
  if (ra_status st = check_sizes(batch, total_q, vocab, max_draft_len)) return st;
  RA_REQUIRE(logits_stride >= vocab, "row strides must be >= vocab");
  RA_REQUIRE(logits_fp32 == 0 || logits_fp32 == 1, "logits_fp32 must be 0 (bf16) or 1 (fp32)");
  if (batch == 0) return RA_OK;
  RA_REQUIRE(draft_lens && qo_indptr && path && accept_lens && next_tokens, "null pointer argument");
  RA_REQUIRE(total_q == 0 || (target_logits && draft_tokens && parents), "null pointer argument");
  RA_REQUIRE(aligned4(draft_tokens) && aligned4(parents) && aligned4(draft_lens) && aligned4(qo_indptr) && aligned4(path) &&
                 aligned4(accept_lens) && aligned4(next_tokens),
             "index arrays must be 4-byte aligned");
  RA_REQUIRE(reinterpret_cast<uintptr_t>(target_logits) % (logits_fp32 ? 4 : 2) == 0, "logits must be aligned to their type");
  const GreedyParams p{target_logits, logits_stride, vocab,         draft_tokens, parents,     draft_lens,  qo_indptr,
                       total_q,       max_draft_len, path,          accept_lens,  next_tokens, device_error};
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DeviceInfo dev;
  if (ra_status st = current_device(&dev)) return st;
  const int ctas = cluster_ctas(vocab, batch, dev.num_sms);
  return logits_fp32
             ? launch_requests("tree_verify_greedy_kernel", tree_verify_greedy_kernel<float>, batch, ctas, s, p)
             : launch_requests("tree_verify_greedy_kernel", tree_verify_greedy_kernel<__nv_bfloat16>, batch, ctas, s, p);
}
