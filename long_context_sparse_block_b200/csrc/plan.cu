// Bookkeeping of one serving step on the device: block tables, slot maps,
// positions and lengths of a packed batch, from the request lengths alone, and
// the return of a finished request's pages.
//
// With new tokens q_b and earlier tokens c_b of request b, pages of P rows:
//   cu_0 = 0, cu_{b+1} = cu_b + q_b                  (rows of the packed batch)
//   have_b = ceil(c_b / P), want_b = ceil((c_b + q_b) / P), need_b = want_b - have_b
//   off_b = sum of need over the requests before b
//   table[b, have_b + i] = free[count - 1 - off_b - i],  i < need_b
//   pos_t = c_b + t - cu_b,  slot_t = table[b, pos_t / P] * P + pos_t % P
//
// What bounds it: at the sizes of a step (a few requests to a few thousand, up
// to some 100 000 tokens, 12 bytes a token) it is a launch and a handful of
// dependent loads, not bandwidth.  So it is one launch: every CTA scans all
// requests itself (64-bit sums, a contiguous run per thread, two block scans)
// and then fills its share of the tokens and pages, found by a binary search
// in the prefix sums kept in shared memory.  More than one CTA runs as a single
// cluster: a cluster barrier between the last read of the inputs and the first
// write of the outputs lets the lengths and the free count be updated in place
// (seq_lens may be ctx_lens), which a captured decode loop needs.
#include <cooperative_groups.h>

#include "internal.h"

namespace misa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;
constexpr int kPlanMaxSeq = 8192;  // 3 words of shared memory each

struct PlanParams {
  const int32_t* q_lens;
  const int32_t* ctx_lens;
  int32_t* table;  // [n_seq, max_blocks]
  const int32_t* free_pages;
  const int32_t* free_count;
  int32_t* cu_q;
  int32_t* seq_lens;
  int32_t* positions;
  int32_t* slots;
  int32_t* seq_of;
  int32_t* granted;
  int32_t* free_count_out;
  int64_t n_pages;
  int64_t free_cap;
  int n_seq;
  int n_tok;
  int max_blocks;
  int page_shift;
  DevCtl ctl;
};

// Exclusive prefix of v over the block's threads (in thread order); total gets
// the sum.  `part` holds one word per warp.
__device__ __forceinline__ int64_t block_exclusive(int64_t v, int64_t* part, int64_t& total) {
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane_id() >= o) x += y;
  }
  __syncthreads();  // the words of an earlier scan have been read
  if (lane_id() == 31) part[warp_id()] = x;
  __syncthreads();
  int64_t before = 0;
  total = 0;
  const int nw = blockDim.x >> 5;
  for (int w = 0; w < nw; ++w) {
    if (w == warp_id()) before = total;
    total += part[w];
  }
  return before + x - v;
}

// Largest b with start[b] <= x, for x >= start[0] = 0 (start ascending).
__device__ __forceinline__ int find_run(const int* start, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(const PlanParams p) {
  extern __shared__ int smem_plan[];
  __shared__ int64_t part[kPlanThreads / 32];
  int* cu = smem_plan;                // rows before request b, at most n_tok
  int* first = smem_plan + p.n_seq;   // pages handed out before request b
  int* ctx_s = first + p.n_seq;       // earlier tokens, or -1: not granted
  const int P = 1 << p.page_shift;
  const int tid = threadIdx.x;
  const int per = (p.n_seq + kPlanThreads - 1) / kPlanThreads;  // requests per thread
  const int b0 = min(p.n_seq, tid * per), b1 = min(p.n_seq, b0 + per);

  int64_t count = 0;
  if (p.free_pages) {
    count = __ldg(p.free_count);
    if (count < 0 || count > p.free_cap) {
      if (tid == 0) report(p.ctl, DEV_BAD_INPUT);
      count = count < 0 ? 0 : p.free_cap;
    }
  }

  // rows of the packed batch
  int64_t sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int q = p.q_lens[b];
    if (q < 0) report(p.ctl, DEV_BAD_INPUT);
    sum += q > 0 ? q : 0;
  }
  int64_t rows;
  int64_t at = block_exclusive(sum, part, rows);
  if (rows > p.n_tok && tid == 0) report(p.ctl, DEV_BAD_INPUT);

  // pages wanted; a request that does not fit its table row or the token
  // buffers wants none and is not granted
  int64_t need_sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int64_t q = max(p.q_lens[b], 0), c = p.ctx_lens[b];
    bool ok = c >= 0 && c + q <= 0x7fffffffLL && at + q <= p.n_tok;
    const int64_t have = (c + P - 1) >> p.page_shift, want = (c + q + P - 1) >> p.page_shift;
    ok = ok && want <= p.max_blocks;
    if (!ok) report(p.ctl, DEV_BAD_INPUT);
    cu[b] = static_cast<int>(min(at, static_cast<int64_t>(p.n_tok)));
    ctx_s[b] = ok ? static_cast<int>(c) : -1;
    at += q;
    if (ok && p.free_pages) need_sum += want - have;
  }
  int64_t all_need;
  int64_t off = block_exclusive(need_sum, part, all_need);
  int64_t taken = 0;
  for (int b = b0; b < b1; ++b) {
    const int c = ctx_s[b];
    int64_t need = 0;
    if (c >= 0 && p.free_pages) {
      const int64_t q = max(p.q_lens[b], 0);
      need = ((c + q + P - 1) >> p.page_shift) - ((c + P - 1) >> p.page_shift);
    }
    first[b] = static_cast<int>(min(off, static_cast<int64_t>(0x7fffffff)));
    off += need;
    if (need > 0) {
      if (off <= count)
        taken += need;
      else
        ctx_s[b] = -1;  // the pool has run out
    }
  }
  int64_t all_taken;
  block_exclusive(taken, part, all_taken);  // (its barriers also publish the arrays)
  __syncthreads();
  if (all_need > count && p.free_pages && tid == 0) report(p.ctl, DEV_BAD_INPUT);

  // lengths of this thread's requests, read before anything is written
  const int rank = blockIdx.x, ranks = gridDim.x;
  int len_new[kPlanMaxSeq / kPlanThreads];
#pragma unroll
  for (int i = 0; i < kPlanMaxSeq / kPlanThreads; ++i) {
    const int b = b0 + i;
    len_new[i] = b < b1 && ctx_s[b] >= 0 ? ctx_s[b] + max(p.q_lens[b], 0) : 0;
  }
  if (ranks > 1) cooperative_groups::this_cluster().sync();

  if (rank == 0) {
#pragma unroll
    for (int i = 0; i < kPlanMaxSeq / kPlanThreads; ++i) {
      const int b = b0 + i;
      if (b < b1) {
        p.seq_lens[b] = len_new[i];
        p.granted[b] = ctx_s[b] >= 0 ? 1 : 0;
        p.cu_q[b] = cu[b];
      }
    }
    if (tid == 0) {
      p.cu_q[p.n_seq] = static_cast<int>(min(rows, static_cast<int64_t>(p.n_tok)));
      if (p.free_pages) p.free_count_out[0] = static_cast<int>(count - all_taken);
    }
  }

  const int stride = ranks * kPlanThreads, g = rank * kPlanThreads + tid;
  // pages handed out: flat page i of the granted requests (which are a prefix
  // of those that want any) is free[count - 1 - i]
  for (int64_t i = g; i < all_taken; i += stride) {
    const int b = find_run(first, p.n_seq, static_cast<int>(i));  // the last start <= i holds page i
    const int have = (ctx_s[b] + P - 1) >> p.page_shift;
    const int blk = have + static_cast<int>(i - first[b]);
    if (ctx_s[b] >= 0 && blk < p.max_blocks) {
      const int pg = __ldg(p.free_pages + count - 1 - i);
      if (pg < 0 || pg >= p.n_pages) report(p.ctl, DEV_BAD_INPUT);
      p.table[static_cast<int64_t>(b) * p.max_blocks + blk] = pg;
    }
  }
  // positions, slots and sequences of the rows
  for (int t = g; t < p.n_tok; t += stride) {
    int pos = -1, slot = -1, seq = -1;
    if (t < rows) {
      const int b = find_run(cu, p.n_seq, t);  // the last of equal starts: the one with rows
      const int c = ctx_s[b];
      if (c >= 0) {
        seq = b;
        pos = c + t - cu[b];
        const int blk = pos >> p.page_shift, have = (c + P - 1) >> p.page_shift;
        int64_t pg;
        if (p.free_pages && blk >= have)  // a page of this step: from its source
          pg = __ldg(p.free_pages + count - 1 - first[b] - (blk - have));
        else
          pg = p.table[static_cast<int64_t>(b) * p.max_blocks + blk];
        if (pg < 0 || pg >= p.n_pages)
          report(p.ctl, DEV_BAD_INPUT);
        else
          slot = static_cast<int>((pg << p.page_shift) | (pos & (P - 1)));
      }
    }
    p.positions[t] = pos;
    p.slots[t] = slot;
    p.seq_of[t] = seq;
  }
}

// Pushes the pages of every flagged request onto the free stack, in request
// order, and sets its length to zero.  One CTA: the pages of a request are
// spread over the threads.
__global__ void __launch_bounds__(kPlanThreads, 1)
release_kernel(const int32_t* release, int32_t* seq_lens, const int32_t* table, int n_seq,
               int max_blocks, int page_shift, int64_t n_pages, int32_t* free_pages,
               int64_t free_cap, int32_t* free_count, const DevCtl ctl) {
  extern __shared__ int smem_plan[];
  __shared__ int64_t part[kPlanThreads / 32];
  int* first = smem_plan;
  const int P = 1 << page_shift, tid = threadIdx.x;
  const int per = (n_seq + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(n_seq, tid * per), b1 = min(n_seq, b0 + per);
  int64_t count = *free_count;
  if (count < 0 || count > free_cap) {
    if (tid == 0) report(ctl, DEV_BAD_INPUT);
    count = count < 0 ? 0 : free_cap;
  }
  int64_t sum = 0;
  auto blocks = [&](int b) -> int64_t {
    if (!release[b]) return 0;
    int64_t nb = (static_cast<int64_t>(max(seq_lens[b], 0)) + P - 1) >> page_shift;
    if (nb > max_blocks) {
      report(ctl, DEV_BAD_INPUT);
      nb = max_blocks;
    }
    return nb;
  };
  for (int b = b0; b < b1; ++b) sum += blocks(b);
  int64_t total;
  int64_t off = block_exclusive(sum, part, total);
  for (int b = b0; b < b1; ++b) {
    first[b] = static_cast<int>(min(off, static_cast<int64_t>(0x7fffffff)));
    off += blocks(b);
  }
  __syncthreads();
  if (count + total > free_cap) {  // more pages than the stack holds: drop the rest
    if (tid == 0) report(ctl, DEV_BAD_INPUT);
    total = free_cap - count;
  }
  for (int64_t i = tid; i < total; i += kPlanThreads) {
    const int b = find_run(first, n_seq, static_cast<int>(i));  // the last start <= i holds page i
    int pg = table[static_cast<int64_t>(b) * max_blocks + (i - first[b])];
    if (pg < 0 || pg >= n_pages) report(ctl, DEV_BAD_INPUT);
    free_pages[count + i] = pg;
  }
  __syncthreads();
  for (int b = b0; b < b1; ++b)
    if (release[b]) seq_lens[b] = 0;
  if (tid == 0) *free_count = static_cast<int>(count + total);
}

}  // namespace

int plan_max_seq() { return kPlanMaxSeq; }

cudaError_t launch_plan(const int32_t* q_lens, const int32_t* ctx_lens, int n_seq, int32_t* table,
                        int max_blocks, int page_shift, int64_t n_pages, int n_tok,
                        const int32_t* free_pages, int64_t free_cap, const int32_t* free_count,
                        int32_t* cu_q, int32_t* seq_lens, int32_t* positions, int32_t* slots,
                        int32_t* seq_of, int32_t* granted, int32_t* free_count_out,
                        const DevCtl& ctl, cudaStream_t s) {
  const PlanParams p{q_lens,    ctx_lens,  table,  free_pages, free_count, cu_q,
                     seq_lens,  positions, slots,  seq_of,     granted,    free_count_out,
                     n_pages,   free_cap,  n_seq,  n_tok,      max_blocks, page_shift,
                     ctl};
  const int smem = 3 * n_seq * static_cast<int>(sizeof(int));
  if (smem > 32 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             3 * kPlanMaxSeq * static_cast<int>(sizeof(int)));
    if (e != cudaSuccess) return e;
  }
  // one CTA up to 4 rows a thread; above that a cluster of 8 shares the rows
  const bool one = n_tok <= 4 * kPlanThreads;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(one ? 1 : kPlanCluster);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = one ? 1 : kPlanCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = one ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, plan_kernel, p);
}

cudaError_t launch_release(const int32_t* release, int32_t* seq_lens, const int32_t* table,
                           int n_seq, int max_blocks, int page_shift, int64_t n_pages,
                           int32_t* free_pages, int64_t free_cap, int32_t* free_count,
                           const DevCtl& ctl, cudaStream_t s) {
  release_kernel<<<1, kPlanThreads, n_seq * sizeof(int), s>>>(release, seq_lens, table, n_seq,
                                                              max_blocks, page_shift, n_pages,
                                                              free_pages, free_cap, free_count, ctl);
  return cudaGetLastError();
}

}  // namespace misa
