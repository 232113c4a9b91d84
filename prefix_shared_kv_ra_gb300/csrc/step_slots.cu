// step_slots.cu -- a step's bookkeeping on the GPU: ra_step_slots (slots, table entries, positions and row starts of the
// new tokens from the requests' lengths and a free list of pages) and ra_tree_commit (the accepted path of each draft
// tree written to the table, the refused slots returned to the free list).
//
// Both are exclusive sums over the requests followed by one store per token and array: 12 bytes a token, some hundred
// kilobytes at most, so launches and latencies bound them, not HBM.  One launch each: a cluster of CTAs in which every
// CTA scans all requests by itself (512 at a time; a request is four words) and then takes its share of the tokens,
// finding a token's request by a binary search in the scanned starts.  The cluster barrier keeps the outputs that may be the
// inputs' own buffers (the lengths, the free list's count) from being written before every CTA has read them, for which a
// grid of independent CTAs would need a second launch; and the commit's CTAs share out the check of the paths and
// slots.  Slots of 65,000 new tokens of 32 requests in pages of 16: 9.9 us (0.8 MB, 0.1 us of HBM); 224 trees of
// 32..64 tokens committed: 7.2, of which 1 is the check.
#include "api_common.h"
#include "ra_ptx.cuh"

namespace ra {

namespace {

constexpr int kThreads = 512;  // also the requests of one round of the scan
constexpr int kMaxCluster = 8;
constexpr int kRun = 4;        // consecutive tokens of a thread

// Let the next kernel launch, every write of this CTA visible to it: the attention calls' planning kernels read lengths,
// which these kernels write, before they wait for the kernel before them.
__device__ __forceinline__ void launch_behind_writes() {
  __threadfence();
  __syncthreads();
  griddep_launch();
}

// Inclusive sums of (a, b) over the CTA's threads; the totals in ta, tb.
__device__ __forceinline__ void scan2(int64_t& a, int64_t& b, int64_t& ta, int64_t& tb) {
  __shared__ int64_t s_a[kThreads / 32], s_b[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, a, off), y = __shfl_up_sync(0xffffffffu, b, off);
    if (lane >= off) a += x, b += y;
  }
  if (lane == 31) s_a[warp] = a, s_b[warp] = b;
  __syncthreads();
  int64_t x = lane < kThreads / 32 ? s_a[lane] : 0, y = lane < kThreads / 32 ? s_b[lane] : 0;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, x, off), v = __shfl_up_sync(0xffffffffu, y, off);
    if (lane >= off) x += u, y += v;
  }
  const int64_t pa = __shfl_sync(0xffffffffu, x, (warp + 31) & 31), pb = __shfl_sync(0xffffffffu, y, (warp + 31) & 31);
  ta = __shfl_sync(0xffffffffu, x, kThreads / 32 - 1), tb = __shfl_sync(0xffffffffu, y, kThreads / 32 - 1);
  if (warp > 0) a += pa, b += pb;
}

// Largest r < n with start[r] <= t (start[0] <= t; starts ascend).
__device__ __forceinline__ int request_of(const int32_t* start, int n, int32_t t) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

struct StepParams {
  int32_t* table;
  int64_t table_stride, table_rows;
  const int32_t *rpi, *seq_lens, *new_lens;
  int32_t batch;
  const int32_t* free_pages;
  int64_t free_capacity;
  const int32_t* free_count;
  int32_t* free_count_out;
  int32_t page;
  uint32_t page_mul;   // n / page = n * page_mul >> page_shift for 0 <= n < 2^31
  int32_t page_shift;
  int32_t last_page;   // the last whose slots fit 32 bits
  int32_t *loc, *positions;
  bool vectors;        // both are 16-byte aligned
  int64_t num_tokens;
  int32_t *qo_indptr, *seq_out;
  uint32_t* err;
  __device__ __forceinline__ int32_t page_div(int32_t n) const {
    return static_cast<int32_t>(static_cast<uint64_t>(static_cast<uint32_t>(n)) * page_mul >> page_shift);
  }
};

__global__ void __launch_bounds__(kThreads) step_slots_kernel(const StepParams p) {
  __shared__ int32_t s_start[kThreads], s_cur[kThreads], s_row[kThreads], s_prev[kThreads], s_fresh[kThreads],
      s_base[kThreads];
  __shared__ int64_t s_used[kThreads / 32];
  griddep_wait();  // the lengths and the free list may come from the kernels before
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const bool first_cta = cluster_rank() == 0;
  const int64_t worker = static_cast<int64_t>(blockIdx.x) * kThreads + t, workers = static_cast<int64_t>(gridDim.x) * kThreads;
  int64_t count = __ldg(p.free_count);
  if (count < 0 || count > p.free_capacity) {
    if (first_cta && t == 0) flag_error(p.err, RA_DEVERR_LENGTH);
    count = count < 0 ? 0 : p.free_capacity;
  }
  int64_t tokens = 0, pages = 0;   // of the requests before this round's
  int64_t taken = 0;               // pages taken so far
  for (int32_t r0 = 0; r0 < p.batch; r0 += kThreads) {
    const int32_t b = r0 + t;
    const int n = min(kThreads, p.batch - r0);
    int32_t cur = 0, len = 0, row = -1, have = 0;
    int64_t add = 0, need = 0;
    uint32_t bad = 0;
    if (b < p.batch) {
      cur = p.seq_lens[b];
      len = __ldg(p.new_lens + b);
      row = __ldg(p.rpi + b);
      if (len < 0 || cur < 0) {
        bad = RA_DEVERR_LENGTH;
        len = max(len, 0);
        cur = max(cur, 0);
      }
      if (static_cast<int64_t>(cur) + len > p.table_stride) bad = RA_DEVERR_LENGTH;
      if (row < 0 || row >= p.table_rows) bad |= RA_DEVERR_TABLE;
      have = cur > 0 ? p.page_div(cur - 1) + 1 : 0;
      add = len;
      if (!bad && len > 0) need = p.page_div(cur + len - 1) + 1 - have;  // (cur + len is within the table)
    }
    int64_t end = add, page_end = need, all_tokens, all_pages;
    scan2(end, page_end, all_tokens, all_pages);
    end += tokens;
    page_end += pages;
    // a request that the arrays or the free list do not hold takes no pages; nor does any after it that needs some
    if (!bad && need > 0 && page_end > count) bad = RA_DEVERR_FULL;
    if (end > p.num_tokens) bad |= RA_DEVERR_LENGTH;
    const int64_t used = !bad && need > 0 ? page_end : 0;
    const bool ok = b < p.batch && bad == 0;
    if (b < p.batch) {
      s_start[t] = static_cast<int32_t>(end - add < p.num_tokens ? end - add : p.num_tokens);
      s_cur[t] = cur;
      s_row[t] = ok && len > 0 ? row : -1;
      s_fresh[t] = have;
      s_base[t] = static_cast<int32_t>(page_end - need);
      // tokens that fall into the request's last page follow its last slot
      int32_t prev = 0;
      if (ok && len > 0 && have * static_cast<int64_t>(p.page) != cur) {
        prev = p.table[static_cast<int64_t>(row) * p.table_stride + cur - 1];
        if (prev < 0 || prev > INT32_MAX - p.page) {
          prev = INT32_MIN;
          bad = RA_DEVERR_SLOT;
        }
      }
      s_prev[t] = prev;
      if (bad && first_cta) flag_error(p.err, bad);
    }
    // the largest end of a request that took pages (they take them in order)
    const uint32_t takers = __ballot_sync(0xffffffffu, used > 0);
    if (takers && lane == 31 - __clz(takers)) s_used[warp] = used;
    if (!takers && lane == 0) s_used[warp] = 0;
    cluster_sync_all();  // every CTA has read this round's lengths and last slots (and wrote its shared arrays)
    for (int w = 0; w < kThreads / 32; ++w) taken = s_used[w] > taken ? s_used[w] : taken;
    if (first_cta && b < p.batch) {
      p.qo_indptr[b + 1] = static_cast<int32_t>(end < p.num_tokens ? end : p.num_tokens);
      p.seq_out[b] = ok ? cur + len : cur;
    }
    const int64_t stop = tokens + all_tokens < p.num_tokens ? tokens + all_tokens : p.num_tokens;
    // Runs of kRun tokens per thread: one search and one division each where the run lies in one request, its page ids
    // on the way at once.  (Token by token, with two runtime divisions, the 65,000 tokens of a prefill took 10 us of a
    // cluster's issue slots.)
    for (int64_t i0 = tokens + worker * kRun; i0 < stop; i0 += workers * kRun) {
      int r = request_of(s_start, n, static_cast<int32_t>(i0));
      int32_t pos[kRun], slot[kRun], id[kRun], in_page[kRun];
      int32_t* row[kRun];
      int32_t next = r + 1 < n ? s_start[r + 1] : INT32_MAX;
      bool fresh = true;  // look the request up
      int32_t pg = 0, off = 0, p0 = 0;
      const int32_t* ids = nullptr;
      int32_t* out = nullptr;
      int32_t prev = 0;
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        slot[k] = 0;
        id[k] = INT32_MIN;
        row[k] = nullptr;
        if (i0 + k >= stop) continue;  // (in 64 bits: the last run may end behind 2^31)
        const int32_t i = static_cast<int32_t>(i0 + k);
        while (i >= next) {  // (over requests without new tokens)
          ++r;
          next = r + 1 < n ? s_start[r + 1] : INT32_MAX;
          fresh = true;
        }
        if (fresh) {
          fresh = false;
          const int32_t cur = s_cur[r];
          p0 = cur + (i - s_start[r]) - i;  // position of token i: p0 + i
          pg = p.page_div(p0 + i);
          off = p0 + i - pg * p.page;
          pg -= s_fresh[r];
          ids = p.free_pages + (count - 1 - s_base[r]);
          out = s_row[r] >= 0 ? p.table + static_cast<int64_t>(s_row[r]) * p.table_stride : nullptr;
          prev = s_prev[r] >= 0 ? s_prev[r] + 1 - cur : INT32_MIN;
        }
        pos[k] = p0 + i;
        in_page[k] = off;
        if (out) {
          row[k] = out + pos[k];
          if (pg >= 0) {  // in a page taken by this call
            id[k] = __ldg(ids - pg);
            slot[k] = -1;
          } else if (prev != INT32_MIN) {
            slot[k] = prev + pos[k];
          }
        }
        if (++off == p.page) off = 0, ++pg;
      }
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        if (slot[k] < 0) {
          slot[k] = 0;
          if (id[k] >= 0 && id[k] <= p.last_page) slot[k] = id[k] * p.page + in_page[k];
          else flag_error(p.err, RA_DEVERR_SLOT);
        }
        if (row[k]) *row[k] = slot[k];
      }
      if (p.vectors && i0 % kRun == 0 && i0 + kRun <= stop) {
        *reinterpret_cast<int4*>(p.loc + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        *reinterpret_cast<int4*>(p.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      } else {
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
          if (i0 + k >= stop) break;
          p.loc[i0 + k] = slot[k];
          p.positions[i0 + k] = pos[k];
        }
      }
    }
    tokens += all_tokens;
    pages += all_pages;
    __syncthreads();  // the shared arrays are free
  }
  // entries behind the last token: the dummy slot
  for (int64_t i = tokens + worker; i < p.num_tokens; i += workers) {
    p.loc[i] = 0;
    p.positions[i] = 0;
  }
  if (first_cta && t == 0) {
    p.qo_indptr[0] = 0;
    *p.free_count_out = static_cast<int32_t>(count - taken);
  }
  launch_behind_writes();
}

struct CommitParams {
  int32_t* table;
  int64_t table_stride, table_rows;
  const int32_t *rpi, *prefix_lens, *draft_lens, *qo_indptr;
  int32_t batch;
  const int32_t* loc;
  int64_t total_q;
  const int32_t* path;
  int32_t path_stride;
  const int32_t* accept_lens;
  int32_t* seq_out;
  int32_t* free_list;
  int64_t free_capacity;
  const int32_t* free_count;
  int32_t* free_count_out;
  uint32_t* err;
};

__global__ void __launch_bounds__(kThreads) tree_commit_kernel(const CommitParams p) {
  __shared__ int32_t s_start[kThreads], s_prefix[kThreads], s_row[kThreads], s_kept[kThreads], s_len[kThreads],
      s_first[kThreads];
  __shared__ int64_t s_free[kThreads];
  __shared__ uint32_t s_wrong[2][kThreads];  // flags of the requests whose paths or slots are wrong, by the round's parity
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const uint32_t rank = cluster_rank(), ctas = gridDim.x;
  const bool first_cta = rank == 0;
  s_wrong[0][t] = s_wrong[1][t] = 0;
  cluster_arrive();  // (before the CTAs store into each other's shared memory)
  griddep_wait();
  const int64_t worker = static_cast<int64_t>(blockIdx.x) * kThreads + t, workers = static_cast<int64_t>(gridDim.x) * kThreads;
  int64_t count = __ldg(p.free_count);
  if (count < 0 || count > p.free_capacity) {
    if (first_cta && t == 0) flag_error(p.err, RA_DEVERR_LENGTH);
    count = count < 0 ? 0 : p.free_capacity;
  }
  cluster_wait();
  int64_t freed = 0;  // slots freed by the rounds before
  for (int32_t r0 = 0; r0 < p.batch; r0 += kThreads) {
    const int32_t b = r0 + t;
    const int n = min(kThreads, p.batch - r0);
    uint32_t* wrong = s_wrong[r0 / kThreads & 1];
    int32_t P = 0, T = 0, kept = 0, row = 0, first = 0;
    uint32_t bad = 0;
    if (b < p.batch) {
      P = p.prefix_lens[b];
      T = __ldg(p.draft_lens + b);
      kept = __ldg(p.accept_lens + b);
      row = __ldg(p.rpi + b);
      first = __ldg(p.qo_indptr + b);
      if (row < 0 || row >= p.table_rows) bad = RA_DEVERR_TABLE;
      if (P < 0 || T < 0 || kept < 0 || kept > T || T > p.path_stride || static_cast<int64_t>(P) + T > p.table_stride ||
          first < 0 || static_cast<int64_t>(first) + T > p.total_q)
        bad |= RA_DEVERR_LENGTH;
      if (bad) T = kept = 0;
    }
    s_kept[t] = kept;
    s_len[t] = T;
    s_first[t] = first;
    __syncthreads();
    // The paths, which what follows takes to ascend within the tree, and the slots: ra_step_slots gives a request that it has no
    // pages for, and a token whose page id is wrong, the dummy slot, which must not reach the free list.  Each request's by a
    // warp of one CTA, for all of them.
    for (int r = static_cast<int>(rank + ctas * warp); r < n; r += static_cast<int>(ctas) * (kThreads / 32)) {
      const int32_t *path = p.path + static_cast<int64_t>(r0 + r) * p.path_stride, *loc = p.loc + s_first[r];
      bool ascends = true, placed = true;
      const int32_t len = s_len[r], kept = s_kept[r];
#pragma unroll 2
      for (int k = lane; k < len; k += 32) {
        const int32_t slot = __ldg(loc + k);
        const int32_t node = k < kept ? __ldg(path + k) : k, before = k < kept && k > 0 ? __ldg(path + k - 1) : -1;
        placed &= slot > 0;
        ascends &= before < node && node < len;
      }
      const uint32_t flags = (__all_sync(0xffffffffu, ascends) ? 0u : RA_DEVERR_LENGTH) |
                             (__all_sync(0xffffffffu, placed) ? 0u : RA_DEVERR_SLOT);
      if (flags && lane < ctas) st_cluster_b32(smem_u32(wrong + r), lane, flags);
    }
    cluster_sync_all();  // every CTA has read this round's lengths, and has the answers
    bad |= wrong[t];
    wrong[t] = 0;  // (for the round after the next)
    if (bad) {
      if (first_cta) flag_error(p.err, bad);
      T = kept = 0;
    }
    int64_t end = T, gone = T - kept, all, all_gone;
    scan2(end, gone, all, all_gone);
    s_start[t] = static_cast<int32_t>(end - T);
    s_prefix[t] = P;
    s_row[t] = row;
    s_kept[t] = kept;
    s_free[t] = count + freed + gone - (T - kept);
    __syncthreads();
    if (first_cta && b < p.batch) p.seq_out[b] = P + kept;
    for (int64_t i = worker; i < all; i += workers) {
      const int r = request_of(s_start, n, static_cast<int32_t>(i));
      const int32_t node = static_cast<int32_t>(i) - s_start[r];
      // accepted nodes before this one
      const int32_t* path = p.path + static_cast<int64_t>(r0 + r) * p.path_stride;
      int lo = 0, hi = s_kept[r];
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(path + mid) < node) lo = mid + 1; else hi = mid;
      }
      const int32_t slot = __ldg(p.loc + s_first[r] + node);
      int32_t* out = p.table + static_cast<int64_t>(s_row[r]) * p.table_stride + s_prefix[r];
      if (lo < s_kept[r] && __ldg(path + lo) == node) {
        out[lo] = slot;
      } else {
        const int32_t nth = node - lo;  // of the refused ones
        out[s_kept[r] + nth] = -1;
        const int64_t at = s_free[r] + nth;
        if (at < p.free_capacity) p.free_list[at] = slot;
        else flag_error(p.err, RA_DEVERR_FULL);
      }
    }
    freed += all_gone;
    __syncthreads();  // the shared arrays are free
  }
  if (first_cta && t == 0) {
    const int64_t now = count + freed;
    *p.free_count_out = static_cast<int32_t>(now < p.free_capacity ? now : p.free_capacity);
  }
  launch_behind_writes();
}

// CTAs of the cluster: one while it gives a thread a few tokens (no barrier between SMs, and the whole call is the scan's
// latency), then as many as keep that, up to the 8 that every GPU of the architecture runs as one cluster.
unsigned cluster_ctas(int64_t tokens) {
  unsigned c = 1;
  while (c < kMaxCluster && tokens > static_cast<int64_t>(c) * kThreads * 2) c *= 2;
  return c;
}

template <typename Params>
ra_status launch_cluster(const char* what, void (*kern)(Params), unsigned ctas, cudaStream_t stream, const Params& p) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "%s launch failed: %s", what, cudaGetErrorString(e));
  return RA_OK;
}

}  // namespace
}  // namespace ra

extern "C" ra_status ra_step_slots(int32_t* req_to_token, int64_t table_stride, int64_t table_rows,
                                   const int32_t* req_pool_indices, const int32_t* seq_lens, const int32_t* new_lens,
                                   int32_t batch, const int32_t* free_pages, int64_t free_capacity,
                                   const int32_t* free_count, int32_t* free_count_out, int32_t page_size,
                                   int32_t* out_cache_loc, int32_t* positions, int64_t num_tokens, int32_t* qo_indptr,
                                   int32_t* seq_lens_out, uint32_t* device_error, ra_stream_t stream) {
  using namespace ra;
  clear_error();
  RA_REQUIRE(batch >= 0 && batch <= 65535, "batch must be in [0, 65535] (got %d)", batch);
  RA_REQUIRE(num_tokens >= 0 && num_tokens <= INT32_MAX, "num_tokens out of range");
  RA_REQUIRE(page_size >= 1 && page_size <= (1 << 20), "page_size must be in [1, 2^20] (got %d)", page_size);
  RA_REQUIRE(free_capacity >= 0 && free_capacity <= INT32_MAX, "free_capacity out of range");
  RA_REQUIRE(table_rows > 0 && table_stride > 0 && table_stride <= INT32_MAX, "table sizes must be > 0");
  RA_REQUIRE(req_to_token && free_count && free_count_out && qo_indptr, "null pointer argument");
  RA_REQUIRE(batch == 0 || (req_pool_indices && seq_lens && new_lens && seq_lens_out), "null pointer argument");
  RA_REQUIRE(num_tokens == 0 || (out_cache_loc && positions), "null pointer argument");
  RA_REQUIRE(free_capacity == 0 || free_pages, "null pointer argument");
  RA_REQUIRE(aligned4(req_to_token) && aligned4(req_pool_indices) && aligned4(seq_lens) && aligned4(new_lens) &&
                 aligned4(free_pages) && aligned4(free_count) && aligned4(free_count_out) && aligned4(out_cache_loc) &&
                 aligned4(positions) && aligned4(qo_indptr) && aligned4(seq_lens_out),
             "index arrays must be 4-byte aligned");
  // n / d for n < 2^31 by a product: with l = ceil(log2 d), m = floor(2^(31 + l) / d) + 1 fits 32 bits and exceeds
  // 2^(31 + l) / d by at most 1, so that n m / 2^(31 + l) is less than 1 / d above n / d
  int32_t shift = 31;
  while ((int64_t(1) << (shift - 31)) < page_size) ++shift;
  const uint32_t mul = static_cast<uint32_t>((int64_t(1) << shift) / page_size + 1);
  StepParams p{};
  p.table = req_to_token;
  p.table_stride = table_stride;
  p.table_rows = table_rows;
  p.rpi = req_pool_indices;
  p.seq_lens = seq_lens;
  p.new_lens = new_lens;
  p.batch = batch;
  p.free_pages = free_pages;
  p.free_capacity = free_capacity;
  p.free_count = free_count;
  p.free_count_out = free_count_out;
  p.page = page_size;
  p.page_mul = mul;
  p.page_shift = shift;
  p.last_page = (INT32_MAX - page_size) / page_size;
  p.loc = out_cache_loc;
  p.positions = positions;
  p.vectors = aligned16(out_cache_loc) && aligned16(positions);
  p.num_tokens = num_tokens;
  p.qo_indptr = qo_indptr;
  p.seq_out = seq_lens_out;
  p.err = device_error;
  return launch_cluster("step_slots_kernel", step_slots_kernel, batch == 0 ? 1 : cluster_ctas(num_tokens),
                        reinterpret_cast<cudaStream_t>(stream), p);
}

extern "C" ra_status ra_tree_commit(int32_t* req_to_token, int64_t table_stride, int64_t table_rows,
                                    const int32_t* req_pool_indices, const int32_t* prefix_lens,
                                    const int32_t* draft_lens, const int32_t* qo_indptr, int32_t batch,
                                    const int32_t* out_cache_loc, int64_t total_q, const int32_t* path,
                                    int32_t path_stride, const int32_t* accept_lens, int32_t* seq_lens_out,
                                    int32_t* free_list, int64_t free_capacity, const int32_t* free_count,
                                    int32_t* free_count_out, uint32_t* device_error, ra_stream_t stream) {
  using namespace ra;
  clear_error();
  RA_REQUIRE(batch >= 0 && batch <= 65535, "batch must be in [0, 65535] (got %d)", batch);
  RA_REQUIRE(total_q >= 0 && total_q <= INT32_MAX, "total_q out of range");
  RA_REQUIRE(free_capacity >= 0 && free_capacity <= INT32_MAX, "free_capacity out of range");
  RA_REQUIRE(table_rows > 0 && table_stride > 0 && table_stride <= INT32_MAX, "table sizes must be > 0");
  RA_REQUIRE(path_stride >= 1, "path_stride must be >= 1");
  if (path_stride > 1024) return fail(RA_ERR_UNSUPPORTED, "path_stride %d (trees of up to 1024 tokens)", path_stride);
  RA_REQUIRE(req_to_token && free_count && free_count_out, "null pointer argument");
  RA_REQUIRE(batch == 0 || (req_pool_indices && prefix_lens && draft_lens && qo_indptr && path && accept_lens && seq_lens_out),
             "null pointer argument");
  RA_REQUIRE(total_q == 0 || out_cache_loc, "null pointer argument");
  RA_REQUIRE(free_capacity == 0 || free_list, "null pointer argument");
  RA_REQUIRE(aligned4(req_to_token) && aligned4(req_pool_indices) && aligned4(prefix_lens) && aligned4(draft_lens) &&
                 aligned4(qo_indptr) && aligned4(out_cache_loc) && aligned4(path) && aligned4(accept_lens) &&
                 aligned4(seq_lens_out) && aligned4(free_list) && aligned4(free_count) && aligned4(free_count_out),
             "index arrays must be 4-byte aligned");
  const CommitParams p{req_to_token, table_stride, table_rows,  req_pool_indices, prefix_lens,   draft_lens,
                       qo_indptr,    batch,        out_cache_loc, total_q,        path,          path_stride,
                       accept_lens,  seq_lens_out, free_list,   free_capacity,    free_count,    free_count_out,
                       device_error};
  return launch_cluster("tree_commit_kernel", tree_commit_kernel, batch == 0 ? 1 : cluster_ctas(total_q),
                        reinterpret_cast<cudaStream_t>(stream), p);
}
