// What the paged attention kernels share: a call's parameters and the rows and
// keys of one request.
#pragma once
#include "decode_kernel.cuh"
#include "paged_base.cuh"

namespace sa {

constexpr int kPagedMaxBatch = 4096;  // a call's request table is kept in shared memory

struct PagedParams {
  int batch, T, Hq, Hkv, G;
  int max_new;
  int page_log2, num_pages, max_pages;
  int box_log2;      // tokens of one TMA box of the few-rows kernel
  int few;           // a request of at most this many new tokens goes to the few-rows kernel
  int window;        // 0: full causal
  float scale_log2;  // scale * log2(e)
  long long q_stride;
  const __nv_bfloat16* q;
  const float* k_scale;
  const float* v_scale;
  const int* table;
  const int* cu;
  const int* kv_lens;
  const float* sinks;
  __nv_bfloat16* out;
  float* lse;
  // The few-rows kernel: chunks of key/value heads, heads of a chunk and warps
  // that share a head's rows; and its workspace, per worker two partial results
  // for each of its warps (unnormalised O, reference max, sum), the cut request
  // (and chunk) that its piece completes, and whether a request that it does
  // not complete begins in its piece.
  int chunks, per_chunk, row_parts;
  float* part_o;     // [workers][2][warps of a worker][kR][64]
  float2* part_ml;   // [workers][2][warps of a worker][kR] (m in log2 units, l)
  int4* part_unit;   // [workers] (b or -1, chunk, begins, 0)
};

// Loads of a call's inputs.  The kernels may start while the ones before them
// still write (see pdl_wait), which rules out the read-only path.  kL2: through
// L2, where those writes are once they are done; the few-rows kernel beside a
// chunk kernel never executes that wait before it reads, so nothing promises it
// that the L1 of its SM holds no older copy.  (Everywhere, that cost short
// decode steps 2 or 3%.)
template <bool kL2 = false, typename T>
__device__ __forceinline__ T paged_load(const T* at) {
  return kL2 ? __ldcg(at) : *at;
}

// One request's rows and keys.  Lengths that do not fit the call's sizes are
// cut to them (and reported by paged_check), so that no index leaves a tensor.
struct PagedRequest {
  int t0, n;   // first row of q and new tokens
  int len;     // tokens after the step
  int lo;      // first key that any of its rows sees; the last one is len - 1
};

template <bool kL2 = false>
__device__ __forceinline__ PagedRequest paged_request(const PagedParams& p, int b) {
  PagedRequest r;
  r.t0 = min(max(paged_load<kL2>(p.cu + b), 0), p.T);
  r.n = min(max(paged_load<kL2>(p.cu + b + 1), r.t0), p.T) - r.t0;
  r.len = min(max(paged_load<kL2>(p.kv_lens + b), 0), p.max_pages << p.page_log2);
  r.lo = p.window > 0 ? max(0, r.len - r.n - p.window + 1) : 0;
  return r;
}

// Reports a request whose lengths do not fit.
template <bool kL2 = false>
__device__ __forceinline__ void paged_check(const PagedParams& p, int b) {
  const int c0 = paged_load<kL2>(p.cu + b), c1 = paged_load<kL2>(p.cu + b + 1), len = paged_load<kL2>(p.kv_lens + b);
  if (c0 < 0 || c1 < c0 || c1 > p.T || c1 - c0 > p.max_new || len < 0 || len > (p.max_pages << p.page_log2))
    report_input(kDevErrPagedRows);
}

// The table's entry for the page that holds key j of request b.
template <bool kL2 = false>
__device__ __forceinline__ int paged_entry(const PagedParams& p, int b, int j) {
  return paged_load<kL2>(p.table + static_cast<long long>(b) * p.max_pages + (j >> p.page_log2));
}

// A table entry as a page: num_pages, which a TMA load reads as zeros, when it
// lies outside the pool.
__device__ __forceinline__ int paged_page(const PagedParams& p, int entry) {
  if (entry >= 0 && entry < p.num_pages) return entry;
  report_input(kDevErrBadPage);
  return p.num_pages;
}

// 4-D tiled load global -> shared (see tma_load_3d).
__device__ __forceinline__ void tma_load_4d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

}  // namespace sa
