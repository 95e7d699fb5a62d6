// Planning one serving step of a paged key/value cache on the GPU: from the
// requests' lengths to block-table entries, slots of the new tokens and pages
// that go back to the pool.
//
// With c = cached_lens[b], n = new_lens[b] (negative: the request has ended)
// and P = page_size:
//   held = ceil(c / P), need = ceil((c + n) / P) - held
//   cu_seqlens = exclusive prefix sum of max(n, 0), of refused requests too: the
//   caller packed their rows, and those behind them lie where that puts them
//   the k-th new page of request b is free_pages[(head + sum_{a<b} need_a + k) mod N]
//   slot of the token at position p = page(p / P) * P + p mod P
//   released: all of an ended request's pages; with a window, the pages that
//   lie wholly before the first key the step's queries can see, c - window + 1.
// The pool is a ring: pages are taken at its head and put back at its tail, so
// a step's takes and puts touch different entries and need no order between
// them.
//
// A step moves a few KB to a few hundred KB, so the call is bound by latency:
// one launch of one thread-block cluster.  Every block of the cluster computes
// the three prefix sums over the requests by itself (a second or third block
// repeating a scan of a few hundred numbers costs nothing, exchanging it would
// cost a cluster barrier), then the blocks share the tokens.  A token finds
// its request by binary search in shared memory.  The one barrier of the
// cluster separates the reads of the lengths from the writes of their
// successors, which may be the same arrays.
#pragma once
#include "paged_base.cuh"

namespace sa {

constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxBatch = 4096;
constexpr int kPlanItems = kPlanMaxBatch / kPlanThreads;  // requests per thread, at most

struct PlanParams {
  int batch, max_tokens, max_pages, page_size, num_pages;
  int page_log2;
  int window;
  const int* cached;     // [batch]
  const int* fresh;      // [batch] new tokens, negative: ended
  int* table;            // [batch][max_pages]
  int* ring;             // [num_pages]
  const int* pool;       // {head, count}
  const int* first;      // [batch] or nullptr
  int* cu;               // [batch + 1]
  int* kv;               // [batch]
  int* slots;            // [max_tokens]
  int* pool_out;         // {head, count}
  int* first_out;        // [batch] or nullptr
};

// Shared memory: per request the exclusive sums of new tokens and released
// pages (batch + 1 each), the cached length, and the first new page's index in
// the ring order (-1: the request got no room this step).
constexpr size_t plan_smem_bytes(int batch) { return (4 * static_cast<size_t>(batch) + 2) * sizeof(int); }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Sum of two counts of tokens, at most 2^31 - 1 (so it can be taken in any order):
// what a caller asks for may be more than 32 bits count, and a slot map ends far before.
__device__ __forceinline__ int plan_add(int a, int b) {
  return static_cast<int>(min(static_cast<uint32_t>(a) + static_cast<uint32_t>(b), 0x7fffffffu));
}

// Largest i in [0, n) with v[i] <= x, for non-decreasing v with v[0] <= x.
__device__ __forceinline__ int plan_find(const int* v, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (v[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) sink_attn_paged_plan_kernel(const PlanParams p) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ int plan_smem[];
  int* s_cu = plan_smem;                  // [batch + 1]
  int* s_rel = s_cu + p.batch + 1;        // [batch + 1]
  int* s_len = s_rel + p.batch + 1;       // [batch]
  int* s_page = s_len + p.batch;          // [batch]
  __shared__ int s_sum[3][32];
  __shared__ int s_taken;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t most = static_cast<int64_t>(p.max_pages) << p.page_log2;  // tokens a table row covers
  const int num = p.num_pages;
  int head = *(p.pool) % num;
  if (head < 0) head += num;
  const int count = min(max(*(p.pool + 1), 0), num);

  // Each thread owns `items` neighbouring requests.
  const int items = (p.batch + kPlanThreads - 1) / kPlanThreads;
  int n_[kPlanItems], need_[kPlanItems], rel_[kPlanItems], kv_[kPlanItems], drop_[kPlanItems];
  bool bad_ = false;
  int sum_n = 0, sum_need = 0, sum_rel = 0;
#pragma unroll
  for (int i = 0; i < kPlanItems; ++i) {
    n_[i] = need_[i] = rel_[i] = kv_[i] = drop_[i] = 0;
    const int b = tid * items + i;
    if (i >= items || b >= p.batch) continue;
    int c = p.cached[b];
    const int n = p.fresh[b];
    const int low_in = p.first ? p.first[b] : 0;
    const bool ended = n < 0;
    const bool known = c >= 0 && c <= most;  // the row can hold the tokens that it says it has
    const bool fine = known && (ended || static_cast<int64_t>(c) + n <= most);
    bad_ |= !fine;
    kv_[i] = ended ? 0 : c;
    n_[i] = ended ? 0 : n;
    c = static_cast<int>(min(static_cast<int64_t>(max(c, 0)), most));
    const int held = static_cast<int>((static_cast<int64_t>(c) + p.page_size - 1) >> p.page_log2);
    const int low = min(max(low_in, 0), held);
    if (ended) {
      rel_[i] = held - low;
    } else {
      int drop = low;
      // By the tokens it has, whether or not the new ones fit: a request at the end
      // of its row would otherwise hold pages that nobody sees until it ends.
      if (p.window > 0 && known) drop = max(low, max(0, c - p.window + 1) >> p.page_log2);
      rel_[i] = drop - low;
      drop_[i] = drop;
      if (fine) need_[i] = static_cast<int>((static_cast<int64_t>(c) + n + p.page_size - 1) >> p.page_log2) - held;
    }
    s_len[b] = c;
    s_page[b] = fine && !ended ? 0 : -1;
    sum_n = plan_add(sum_n, n_[i]);
    sum_need += need_[i];
    sum_rel += rel_[i];
  }

  // Exclusive sums over the block of the three per-thread sums.
  int in_n = sum_n, in_need = sum_need, in_rel = sum_rel;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, in_n, o), b = __shfl_up_sync(0xffffffffu, in_need, o),
              c = __shfl_up_sync(0xffffffffu, in_rel, o);
    if (lane >= o) in_n = plan_add(in_n, a), in_need += b, in_rel += c;
  }
  int before_n = __shfl_up_sync(0xffffffffu, in_n, 1);  // (a cut sum has no difference)
  if (lane == 0) before_n = 0;
  if (lane == 31) s_sum[0][warp] = in_n, s_sum[1][warp] = in_need, s_sum[2][warp] = in_rel;
  if (tid == 0) s_taken = 0;
  __syncthreads();
  if (warp < 3) {
    int v = s_sum[warp][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = plan_add(v, a);
    }
    s_sum[warp][lane] = v;
  }
  __syncthreads();
  const int total = s_sum[0][31], released = s_sum[2][31];
  int at_n = plan_add(before_n, warp ? s_sum[0][warp - 1] : 0);
  int at_need = in_need - sum_need + (warp ? s_sum[1][warp - 1] : 0);
  int at_rel = in_rel - sum_rel + (warp ? s_sum[2][warp - 1] : 0);
  bool dry = false;
  int taken = 0;
#pragma unroll
  for (int i = 0; i < kPlanItems; ++i) {
    const int b = tid * items + i;
    if (i >= items || b >= p.batch) continue;
    s_cu[b] = at_n;
    s_rel[b] = at_rel;
    if (s_page[b] == 0) {
      // Pages go to the requests in order while they last; the sum that is
      // compared grows with b, so no request behind one that got none does.
      if (need_[i] == 0 || at_need + need_[i] <= count) {
        s_page[b] = at_need;
        kv_[i] += n_[i];
        if (need_[i] > 0) taken = at_need + need_[i];
      } else {
        s_page[b] = -1;
        dry = true;
      }
    }
    at_n = plan_add(at_n, n_[i]);
    at_need += need_[i];
    at_rel += rel_[i];
  }
  if (taken > 0) atomicMax(&s_taken, taken);
  if (tid == 0) s_cu[p.batch] = total, s_rel[p.batch] = released;
  if (blockIdx.x == 0) {
    if (bad_ || (tid == 0 && total > p.max_tokens)) report_input(kDevErrPlanLengths);
    if (dry) report_input(kDevErrPoolExhausted);
  }
  __syncthreads();

  // The i-th new page of the step, i < count.
  auto new_page = [&](int i) {
    const int at = head + i;  // below 2 num <= 2^28
    return p.ring[at < num ? at : at - num];
  };
  // Tokens: slot_map and, at a page's first token, the table entry.
  const int step = static_cast<int>(gridDim.x) * kPlanThreads;
  const int self = static_cast<int>(blockIdx.x) * kPlanThreads + tid;
  for (int t = self; t < p.max_tokens; t += step) {
    int slot = -1;
    if (t < total) {
      const int b = plan_find(s_cu, p.batch, t);
      if (s_page[b] >= 0) {
        const int c = s_len[b];
        const int held = (c + p.page_size - 1) >> p.page_log2;
        const int pos = c + t - s_cu[b];
        const int j = pos >> p.page_log2;
        int* entry = p.table + static_cast<int64_t>(b) * p.max_pages + j;
        int page;
        if (j >= held) {
          page = new_page(s_page[b] + j - held);
          if ((pos & (p.page_size - 1)) == 0) *entry = page;
        } else {
          page = *entry;
        }
        if (page >= 0 && page < num) slot = (page << p.page_log2) + (pos & (p.page_size - 1));
        else report_input(kDevErrBadPage);
      }
    }
    p.slots[t] = slot;
  }
  // Tokens that the slot map has no room for (reported above) take their pages all the same.
  if (total > p.max_tokens) {
    for (int b = self; b < p.batch; b += step) {
      if (s_page[b] < 0) continue;
      const int held = (s_len[b] + p.page_size - 1) >> p.page_log2;
      const int end = (s_len[b] + p.fresh[b] + p.page_size - 1) >> p.page_log2;
      for (int j = held; j < end; ++j)
        p.table[static_cast<int64_t>(b) * p.max_pages + j] = new_page(s_page[b] + j - held);
    }
  }
  // Released pages, in the order of the requests and of their pages.
  for (int r = self; r < released; r += step) {
    const int b = plan_find(s_rel, p.batch, r);
    const int held = (s_len[b] + p.page_size - 1) >> p.page_log2;
    const int low = p.first ? min(max(p.first[b], 0), held) : 0;
    p.ring[(static_cast<int64_t>(head) + count + r) % num] =
        p.table[static_cast<int64_t>(b) * p.max_pages + low + r - s_rel[b]];
  }

  cluster_arrive();
  cluster_wait();
  if (blockIdx.x != 0) return;
#pragma unroll
  for (int i = 0; i < kPlanItems; ++i) {
    const int b = tid * items + i;
    if (i >= items || b >= p.batch) continue;
    p.kv[b] = kv_[i];
    p.cu[b] = s_cu[b];
    if (p.first_out) p.first_out[b] = drop_[i];
  }
  if (tid == 0) {
    p.cu[p.batch] = total;
    p.pool_out[0] = static_cast<int>((static_cast<int64_t>(head) + s_taken) % num);
    p.pool_out[1] = min(count - s_taken + released, num);
  }
}

}  // namespace sa
