// step_slots.cu -- a step's bookkeeping on the GPU: ra_step_slots (slots, table entries, positions and row starts of the
// new tokens from the requests' lengths and a free list of pages) and ra_tree_commit (the accepted path of each draft
// tree written to the table, the refused slots returned to the free list).
//
// Both are exclusive sums over the requests followed by one store per token and array: 12 bytes a token, some hundred
// kilobytes at most, so launches and latencies bound them, not HBM.  One launch each: a cluster of CTAs in which every
// CTA scans all requests by itself (512 at a time; a request is four words) and then takes its share of the tokens,
// finding a token's request by a binary search in the scanned starts.  Nothing is exchanged between the CTAs; the cluster
// barrier only keeps the outputs that may be the inputs' own buffers (the lengths, the free list's count) from being
// written before every CTA has read them, which a grid of independent CTAs could not do without a second launch.
#include "api_common.h"
#include "ra_ptx.cuh"

namespace ra {

namespace {

constexpr int kThreads = 512;  // also the requests of one round of the scan
constexpr int kMaxCluster = 8;

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

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
  int32_t *loc, *positions;
  int64_t num_tokens;
  int32_t *qo_indptr, *seq_out;
  uint32_t* err;
};

__global__ void __launch_bounds__(kThreads) step_slots_kernel(const StepParams p) {
  __shared__ int32_t s_start[kThreads], s_cur[kThreads], s_row[kThreads], s_prev[kThreads], s_fresh[kThreads],
      s_base[kThreads];
  griddep_wait();  // the lengths and the free list may come from the kernels before
  const int t = threadIdx.x;
  const bool first_cta = cluster_rank() == 0;
  const int64_t worker = static_cast<int64_t>(blockIdx.x) * kThreads + t, workers = static_cast<int64_t>(gridDim.x) * kThreads;
  int64_t count = __ldg(p.free_count);
  if (count < 0 || count > p.free_capacity) {
    if (first_cta && t == 0) flag_error(p.err, RA_DEVERR_LENGTH);
    count = count < 0 ? 0 : p.free_capacity;
  }
  int64_t tokens = 0, pages = 0;   // of the requests before this round's
  int64_t used = 0;                // pages that this thread's requests end at
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
      have = static_cast<int32_t>((static_cast<int64_t>(cur) + p.page - 1) / p.page);
      add = len;
      if (!bad) need = (static_cast<int64_t>(cur) + len + p.page - 1) / p.page - have;
    }
    int64_t end = add, page_end = need, all_tokens, all_pages;
    scan2(end, page_end, all_tokens, all_pages);
    end += tokens;
    page_end += pages;
    // a request that the arrays or the free list do not hold takes no pages; nor does any after it that needs some
    if (!bad && need > 0 && page_end > count) bad = RA_DEVERR_FULL;
    if (end > p.num_tokens) bad |= RA_DEVERR_LENGTH;
    if (!bad && need > 0 && page_end > used) used = page_end;
    const bool ok = b < p.batch && bad == 0;
    if (b < p.batch) {
      s_start[t] = static_cast<int32_t>(end - add < p.num_tokens ? end - add : p.num_tokens);
      s_cur[t] = cur;
      s_row[t] = ok && len > 0 ? row : -1;
      s_fresh[t] = have;
      s_base[t] = static_cast<int32_t>(page_end - need);
      // tokens that fall into the request's last page follow its last slot
      int32_t prev = 0;
      if (ok && len > 0 && cur % p.page != 0) {
        prev = p.table[static_cast<int64_t>(row) * p.table_stride + cur - 1];
        if (prev < 0 || prev > INT32_MAX - p.page) {
          prev = INT32_MIN;
          bad = RA_DEVERR_SLOT;
        }
      }
      s_prev[t] = prev;
      if (bad && first_cta) flag_error(p.err, bad);
    }
    cluster_sync_all();  // every CTA has read this round's lengths and last slots (and wrote its shared arrays)
    if (first_cta && b < p.batch) {
      p.qo_indptr[b + 1] = static_cast<int32_t>(end < p.num_tokens ? end : p.num_tokens);
      p.seq_out[b] = ok ? cur + len : cur;
    }
    const int64_t stop = tokens + all_tokens < p.num_tokens ? tokens + all_tokens : p.num_tokens;
    for (int64_t i = tokens + worker; i < stop; i += workers) {
      const int r = request_of(s_start, n, static_cast<int32_t>(i));
      const int32_t pos = s_cur[r] + static_cast<int32_t>(i - s_start[r]);
      int32_t slot = 0;
      if (s_row[r] >= 0) {
        const int32_t pg = pos / p.page - s_fresh[r];  // >= 0: in a page taken by this call
        if (pg >= 0) {
          const int32_t id = __ldg(p.free_pages + (count - 1 - s_base[r] - pg));
          if (id >= 0 && id <= (INT32_MAX - p.page) / p.page) slot = id * p.page + pos % p.page;
          else flag_error(p.err, RA_DEVERR_SLOT);
        } else if (s_prev[r] >= 0) {
          slot = s_prev[r] + 1 + (pos - s_cur[r]);
        }
        p.table[static_cast<int64_t>(s_row[r]) * p.table_stride + pos] = slot;
      }
      p.loc[i] = slot;
      p.positions[i] = pos;
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
  if (first_cta) {
    __shared__ unsigned long long s_used;
    if (t == 0) s_used = 0;
    __syncthreads();
    if (used > 0) atomicMax(&s_used, static_cast<unsigned long long>(used));
    __syncthreads();
    if (t == 0) {
      p.qo_indptr[0] = 0;
      *p.free_count_out = static_cast<int32_t>(count - static_cast<int64_t>(s_used));
    }
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
  griddep_wait();
  const int t = threadIdx.x;
  const bool first_cta = cluster_rank() == 0;
  const int64_t worker = static_cast<int64_t>(blockIdx.x) * kThreads + t, workers = static_cast<int64_t>(gridDim.x) * kThreads;
  int64_t count = __ldg(p.free_count);
  if (count < 0 || count > p.free_capacity) {
    if (first_cta && t == 0) flag_error(p.err, RA_DEVERR_LENGTH);
    count = count < 0 ? 0 : p.free_capacity;
  }
  int64_t freed = 0;  // slots freed by the rounds before
  for (int32_t r0 = 0; r0 < p.batch; r0 += kThreads) {
    const int32_t b = r0 + t;
    const int n = min(kThreads, p.batch - r0);
    int32_t P = 0, T = 0, kept = 0, row = 0, first = 0;
    if (b < p.batch) {
      P = p.prefix_lens[b];
      T = __ldg(p.draft_lens + b);
      kept = __ldg(p.accept_lens + b);
      row = __ldg(p.rpi + b);
      first = __ldg(p.qo_indptr + b);
      uint32_t bad = 0;
      if (row < 0 || row >= p.table_rows) bad = RA_DEVERR_TABLE;
      if (P < 0 || T < 0 || kept < 0 || kept > T || T > p.path_stride || static_cast<int64_t>(P) + T > p.table_stride ||
          first < 0 || static_cast<int64_t>(first) + T > p.total_q)
        bad |= RA_DEVERR_LENGTH;
      if (bad) {
        if (first_cta) flag_error(p.err, bad);
        T = kept = 0;
      }
    }
    int64_t end = T, gone = T - kept, all, all_gone;
    scan2(end, gone, all, all_gone);
    s_start[t] = static_cast<int32_t>(end - T);
    s_prefix[t] = P;
    s_row[t] = row;
    s_kept[t] = kept;
    s_len[t] = T;
    s_first[t] = first;
    s_free[t] = count + freed + gone - (T - kept);
    cluster_sync_all();  // every CTA has read this round's lengths (and wrote its shared arrays)
    if (first_cta && b < p.batch) p.seq_out[b] = P + kept;
    for (int64_t i = worker; i < all; i += workers) {
      const int r = request_of(s_start, n, static_cast<int32_t>(i));
      const int32_t node = static_cast<int32_t>(i) - s_start[r];
      // accepted nodes before this one: the path ascends, as a node's parent is before it
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
        const int32_t nth = node - lo;
        if (nth >= s_len[r] - s_kept[r]) {  // a path that does not ascend or leaves the tree
          flag_error(p.err, RA_DEVERR_LENGTH);
          continue;
        }
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
  const StepParams p{req_to_token, table_stride,  table_rows,     req_pool_indices, seq_lens,      new_lens,
                     batch,        free_pages,    free_capacity,  free_count,       free_count_out, page_size,
                     out_cache_loc, positions,    num_tokens,     qo_indptr,        seq_lens_out,  device_error};
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
