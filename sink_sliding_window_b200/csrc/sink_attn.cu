// Host side of libsinkattn.so: argument validation, TMA descriptors and
// launches for the C ABI declared in include/sink_attn.h.  Everything here is
// plain host logic; all attention arithmetic runs in the kernels.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "sink_attn.h"

#include "common.cuh"
#include "tma_host.cuh"
#include "fwd_kernel.cuh"
#include "fwd_pair_kernel.cuh"
#include "bwd_kernels.cuh"
#include "decode_kernel.cuh"
#include "paged_plan.cuh"
#include "paged_append.cuh"
#include "paged_attn.cuh"
#include "paged_join.cuh"

namespace sa {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int ilog2_exact(int x) {
  if (x <= 0 || (x & (x - 1)) != 0) return -1;
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

// Validates the sizes and fills the geometry.  T == 0 is valid (no work).
sink_attn_status check_dims(const sink_attn_dims* d, const int* cu_seqlens, bool packed, int window, float scale,
                            Geometry* geo) {
  if (!d) return SINK_ATTN_ERR_NULL;
  if (d->batch < 0 || d->max_seqlen < 0 || d->total_tokens < 0 || d->num_q_heads <= 0 || d->num_kv_heads <= 0 ||
      d->head_dim <= 0)
    return SINK_ATTN_ERR_SHAPE;
  if (d->num_q_heads % d->num_kv_heads != 0) return SINK_ATTN_ERR_SHAPE;
  if (!packed && static_cast<int64_t>(d->batch) * d->max_seqlen != d->total_tokens)
    return SINK_ATTN_ERR_SHAPE;
  if (d->total_tokens > 0 && d->batch == 0) return SINK_ATTN_ERR_SHAPE;
  if (d->head_dim != kHeadDim) return SINK_ATTN_ERR_UNSUPPORTED;
  const int G = d->num_q_heads / d->num_kv_heads;
  const int gl = ilog2_exact(G);
  if (gl < 0 || G > kBlockM) return SINK_ATTN_ERR_UNSUPPORTED;
  if (!(scale > 0.f) || !std::isfinite(scale)) return SINK_ATTN_ERR_UNSUPPORTED;
  // Token and element indices are formed in 32-bit ints in places.
  if (static_cast<int64_t>(d->total_tokens) * d->num_q_heads * kHeadDim >= (int64_t(1) << 40) ||
      d->total_tokens > (1 << 30))
    return SINK_ATTN_ERR_UNSUPPORTED;
  geo->T = d->total_tokens;
  geo->Hq = d->num_q_heads;
  geo->Hkv = d->num_kv_heads;
  geo->G_log2 = gl;
  geo->P_log2 = 7 - gl;
  geo->num_qblocks = (d->total_tokens + (1 << geo->P_log2) - 1) >> geo->P_log2;
  geo->batch = d->batch;
  geo->seqlen = d->max_seqlen;
  geo->cu_seqlens = cu_seqlens;
  geo->window = window > 0 ? window : 0;
  if (!packed && d->total_tokens > 0 && d->max_seqlen <= 0) return SINK_ATTN_ERR_SHAPE;
  return SINK_ATTN_OK;
}

// Checks of a forward call (both forward entry points): sizes, then (for
// T > 0) pointers and alignment.  Fills the geometry.
sink_attn_status check_fwd_args(const sink_attn_dims* d, const void* q, const void* k, const void* v,
                                const float* sinks, const int* cu_seqlens, int window, float scale, const void* out,
                                const float* lse, Geometry* geo) {
  sink_attn_status st = check_dims(d, cu_seqlens, cu_seqlens != nullptr, window, scale, geo);
  if (st != SINK_ATTN_OK || geo->T == 0) return st;
  if (!q || !k || !v || !sinks || !out || !lse) return SINK_ATTN_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u) || (reinterpret_cast<uintptr_t>(sinks) & 3u) ||
      (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u))
    return SINK_ATTN_ERR_ALIGN;
  return SINK_ATTN_OK;
}

// The forward kernel sink_attn_fwd runs: two query tiles per CTA for every
// size.  Timed against one tile per CTA on B200 (interleaved CUDA-event
// runs): 21% faster on sliding-window-128 layers, where a one-tile CTA does
// only a few 64-key steps between its set-up and its epilogue, and 1-4%
// faster on full-causal layers (4k, 60k, packed documents), where both are
// bound by each warpgroup's S round trip and the exp2 unit.
int fwd_auto_kernel(const Geometry&) { return SINK_ATTN_FWD_TWO_TILES; }

// 3-D bf16 view [outer][mid][inner] with a box {box_inner, 1, box_outer}
// under the given swizzle: the pair forward's half-steps of K (32 keys x 64
// dims, 128-byte rows) and V (64 keys x 32 dims, 64-byte rows).
bool make_map_3d_box(CUtensorMap* map, const void* base, int inner, int mid, int outer, int box_inner,
                     int box_outer, CUtensorMapSwizzle swizzle) {
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(mid),
                        static_cast<cuuint64_t>(outer)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(inner) * 2, static_cast<cuuint64_t>(inner) * mid * 2};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(box_inner), 1, static_cast<cuuint32_t>(box_outer)};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Events registered by sink_attn_profile_events: [which][begin/end].
cudaEvent_t g_profile_events[2][2] = {{nullptr, nullptr}, {nullptr, nullptr}};


// Decode: sizes, split count and workspace layout of one call.
struct DecPlan {
  DecParams p;
  size_t o_off, m_off, l_off, total;  // workspace layout (bytes)
};

// CTAs that run at once (two per SM of a 148-SM B200), and a cap on the
// splits of one (sequence, key/value head).
constexpr int kDecTargetCtas = 296;
constexpr int kDecMaxSplit = 64;

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

sink_attn_status plan_decode(const sink_attn_decode_dims* d, int window, float scale, DecPlan* plan) {
  if (!d) return SINK_ATTN_ERR_NULL;
  if (d->batch < 0 || d->new_tokens <= 0 || d->cache_capacity <= 0 || d->max_seqlen < d->new_tokens ||
      d->num_q_heads <= 0 || d->num_kv_heads <= 0 || d->head_dim <= 0)
    return SINK_ATTN_ERR_SHAPE;
  if (d->num_q_heads % d->num_kv_heads != 0) return SINK_ATTN_ERR_SHAPE;
  if (d->head_dim != kHeadDim) return SINK_ATTN_ERR_UNSUPPORTED;
  const int G = d->num_q_heads / d->num_kv_heads;
  const int gl = ilog2_exact(G);
  if (gl < 0 || static_cast<int64_t>(G) * d->new_tokens > kDecRows) return SINK_ATTN_ERR_UNSUPPORTED;
  if (!(scale > 0.f) || !std::isfinite(scale)) return SINK_ATTN_ERR_UNSUPPORTED;
  // Slot and element indices are formed in 32-bit ints in places.
  if (static_cast<int64_t>(d->batch) * d->cache_capacity > (int64_t(1) << 30) ||
      static_cast<int64_t>(d->max_seqlen) + kDecTile > (int64_t(1) << 30) ||
      static_cast<int64_t>(d->batch) * d->new_tokens * d->num_q_heads > (int64_t(1) << 30))
    return SINK_ATTN_ERR_UNSUPPORTED;
  DecParams& p = plan->p;
  p.batch = d->batch;
  p.Lq = d->new_tokens;
  p.C = d->cache_capacity;
  p.Hq = d->num_q_heads;
  p.Hkv = d->num_kv_heads;
  p.G = G;
  p.G_log2 = gl;
  p.R = G * d->new_tokens;
  p.window = window > 0 ? window : 0;
  p.scale_log2 = scale * kLog2e;
  p.seqlens = nullptr;
  p.sinks = nullptr;
  p.k_scale = p.v_scale = nullptr;
  p.o_part = p.m_part = p.l_part = nullptr;
  p.out = nullptr;
  p.lse_out = nullptr;
  // Upper bound on the 128-slot tiles one sequence scans.
  int64_t slots = std::min<int64_t>(d->cache_capacity, d->max_seqlen);
  if (p.window > 0) slots = std::min<int64_t>(slots, static_cast<int64_t>(p.window) + d->new_tokens - 1 + kDecTile);
  const int tiles = static_cast<int>((slots + kDecTile - 1) / kDecTile) + 1;
  const int64_t pairs = static_cast<int64_t>(d->batch) * d->num_kv_heads;
  // Split count: the CTAs run in waves of kDecTargetCtas, each CTA over
  // ceil(tiles / split) tiles plus about one tile's worth of fixed cost
  // (set-up, Q load, partial results); pick the split with the fewest
  // tile-times, preferring fewer splits on ties.
  int split = 1;
  if (pairs > 0) {
    int64_t best = -1;
    for (int k = 1; k <= std::min(tiles, kDecMaxSplit); ++k) {
      const int64_t waves = (pairs * k + kDecTargetCtas - 1) / kDecTargetCtas;
      const int64_t cost = waves * ((tiles + k - 1) / k + 1);
      if (best < 0 || cost < best) {
        best = cost;
        split = k;
      }
    }
  }
  p.n_split = split;
  const size_t parts = static_cast<size_t>(pairs) * split * kDecRows;
  plan->o_off = 0;
  plan->m_off = round256(parts * kHeadDim * sizeof(float));
  plan->l_off = plan->m_off + round256(parts * sizeof(float));
  plan->total = plan->l_off + round256(parts * sizeof(float));
  return SINK_ATTN_OK;
}

}  // namespace

// Self-test of the bounded waits every kernel uses, on an mbarrier that
// nothing ever completes.  Thread 0 gives up after limit_ns and raises the
// CTA's abort flag; thread 32 (another warp) waits with ten times that limit
// and must leave through the flag.  out[0], out[2]: 1 if the wait returned
// true (neither should); out[1], out[3]: microseconds each waited.
__global__ void __launch_bounds__(64) sink_attn_selftest_wait_kernel(unsigned long long limit_ns, int* out) {
  __shared__ uint64_t bar[2];
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(&bar[0], 1);
    mbar_init(&bar[1], 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  volatile int* abort = &abort_flag;
  if (threadIdx.x == 0 || threadIdx.x == 32) {
    const bool first = threadIdx.x == 0;
    const uint64_t t0 = global_timer_ns();
    const bool ok = first ? mbar_wait_for(&bar[0], 0, abort, &g_device_error, kDevErrTimeoutSelfTest, limit_ns)
                          : mbar_wait_for(&bar[1], 0, abort, &g_device_error, kDevErrTimeoutSelfTestAbort,
                                          10ull * limit_ns);
    const uint64_t us = (global_timer_ns() - t0) / 1000ull;
    out[first ? 0 : 2] = ok ? 1 : 0;
    out[first ? 1 : 3] = static_cast<int>(us < 0x7fffffffull ? us : 0x7fffffffull);
  }
}

}  // namespace sa

using namespace sa;

extern "C" {

const char* sink_attn_status_string(sink_attn_status s) {
  switch (s) {
    case SINK_ATTN_OK: return "ok";
    case SINK_ATTN_ERR_NULL: return "a required pointer is NULL";
    case SINK_ATTN_ERR_SHAPE: return "inconsistent sizes";
    case SINK_ATTN_ERR_ALIGN: return "a tensor is not 16-byte aligned";
    case SINK_ATTN_ERR_UNSUPPORTED: return "unsupported configuration (D must be 64, Hq/Hkv a power of two <= 128, scale > 0)";
    case SINK_ATTN_ERR_CUDA: return "CUDA call failed";
    case SINK_ATTN_ERR_DEVICE_TIMEOUT: return "a kernel wait timed out";
    case SINK_ATTN_ERR_WORKSPACE: return "workspace missing or too small";
  }
  return "unknown status";
}

sink_attn_status sink_attn_profile_events(int which, void* ev_begin, void* ev_end) {
  if (which < 0 || which > 1) return SINK_ATTN_ERR_SHAPE;
  g_profile_events[which][0] = static_cast<cudaEvent_t>(ev_begin);
  g_profile_events[which][1] = static_cast<cudaEvent_t>(ev_end);
  return SINK_ATTN_OK;
}

sink_attn_status sink_attn_selftest_wait(unsigned long long limit_ns, int* out, void* stream) {
  if (out == nullptr || (reinterpret_cast<uintptr_t>(out) & 3u) != 0) return SINK_ATTN_ERR_ALIGN;
  if (limit_ns == 0 || limit_ns > kWaitLimitNs) return SINK_ATTN_ERR_SHAPE;
  sink_attn_selftest_wait_kernel<<<1, 64, 0, static_cast<cudaStream_t>(stream)>>>(limit_ns, out);
  return cudaGetLastError() == cudaSuccess ? SINK_ATTN_OK : SINK_ATTN_ERR_CUDA;
}

int sink_attn_last_device_error(void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(st) != cudaSuccess) return -1;
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int)) != cudaSuccess) return -1;
  if (v != 0) return cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int)) == cudaSuccess ? v : -1;
  if (cudaMemcpyFromSymbol(&v, g_input_error, sizeof(int)) != cudaSuccess) return -1;
  if (v != 0 && cudaMemcpyToSymbol(g_input_error, &zero, sizeof(int)) != cudaSuccess) return -1;
  return v;
}

int sink_attn_device_error(void* stream) { return sink_attn_last_device_error(stream); }

int sink_attn_fwd_launches(const sink_attn_dims* d) {
  Geometry geo;
  if (check_dims(d, nullptr, true, 0, 1.f, &geo) != SINK_ATTN_OK) return 0;
  return d->total_tokens > 0 ? 1 : 0;
}

sink_attn_status sink_attn_fwd(const sink_attn_dims* d, const void* q, const void* k, const void* v,
                               const float* sinks, const int* cu_seqlens, int window, float scale, void* out,
                               float* lse, void* stream) {
  return sink_attn_fwd_with(d, q, k, v, sinks, cu_seqlens, window, scale, out, lse, SINK_ATTN_FWD_AUTO, stream);
}

sink_attn_status sink_attn_fwd_pair(const sink_attn_dims* d, const void* q, const void* k, const void* v,
                                    const float* sinks, const int* cu_seqlens, int window, float scale, void* out,
                                    float* lse, void* stream) {
  return sink_attn_fwd_with(d, q, k, v, sinks, cu_seqlens, window, scale, out, lse, SINK_ATTN_FWD_CTA_PAIR,
                            stream);
}

int sink_attn_fwd_kernel_for(const sink_attn_dims* d, int window) {
  Geometry geo;
  if (check_dims(d, nullptr, true, window, 1.f, &geo) != SINK_ATTN_OK) return -1;
  return fwd_auto_kernel(geo);
}

sink_attn_status sink_attn_fwd_with(const sink_attn_dims* d, const void* q, const void* k, const void* v,
                                    const float* sinks, const int* cu_seqlens, int window, float scale, void* out,
                                    float* lse, int kernel, void* stream) {
  if (kernel < SINK_ATTN_FWD_AUTO || kernel > SINK_ATTN_FWD_CTA_PAIR) return SINK_ATTN_ERR_UNSUPPORTED;
  Geometry geo;
  sink_attn_status st = check_fwd_args(d, q, k, v, sinks, cu_seqlens, window, scale, out, lse, &geo);
  if (st != SINK_ATTN_OK || geo.T == 0) return st;
  if (kernel == SINK_ATTN_FWD_AUTO) kernel = fwd_auto_kernel(geo);

  const int G = 1 << geo.G_log2;
  const bool pair = kernel == SINK_ATTN_FWD_CTA_PAIR;
  CUtensorMap tq, tk, tv;
  if (!make_map_3d(&tq, q, kHeadDim, geo.Hq, geo.T, G, 1 << geo.P_log2)) return SINK_ATTN_ERR_CUDA;
  if (pair) {
    // Each CTA of a pair loads 32 keys x 64 dims of K and 64 keys x 32 dims
    // of V per 64-key step.
    if (!make_map_3d_box(&tk, k, kHeadDim, geo.Hkv, geo.T, kHeadDim, kHalfN / 2, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_3d_box(&tv, v, kHeadDim, geo.Hkv, geo.T, kHeadDim / 2, kHalfN, CU_TENSOR_MAP_SWIZZLE_64B))
      return SINK_ATTN_ERR_CUDA;
  } else if (!make_map_3d(&tk, k, kHeadDim, geo.Hkv, geo.T, 1, kBlockN) ||
             !make_map_3d(&tv, v, kHeadDim, geo.Hkv, geo.T, 1, kBlockN)) {
    return SINK_ATTN_ERR_CUDA;
  }

  FwdParams p;
  p.geo = geo;
  p.scale_log2 = scale * kLog2e;
  p.sinks = sinks;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  // One tile: a CTA per (query tile, head g); two tiles and pairs: a CTA per
  // two query tiles, or a pair of CTAs per two query tiles.
  const int64_t units = kernel == SINK_ATTN_FWD_ONE_TILE ? geo.num_qblocks : (geo.num_qblocks + 1) / 2;
  const int64_t grid = units * geo.Hkv * (pair ? 2 : 1);
  if (grid > 0x7fffffff) return SINK_ATTN_ERR_UNSUPPORTED;
  cudaStream_t st_ = static_cast<cudaStream_t>(stream);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kFwdThreads, 1, 1);
  cfg.stream = st_;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaError_t e;
  if (g_profile_events[0][0]) cudaEventRecord(g_profile_events[0][0], st_);
  if (kernel == SINK_ATTN_FWD_ONE_TILE) {
    static SmemAttrOnce smem_set;
    cfg.dynamicSmemBytes = fwd_smem_bytes<1>();
    e = smem_set.ensure(sink_attn_fwd_kernel<1>, cfg.dynamicSmemBytes)
            ? cudaLaunchKernelEx(&cfg, sink_attn_fwd_kernel<1>, tq, tk, tv, p)
            : cudaErrorInvalidValue;
  } else if (kernel == SINK_ATTN_FWD_TWO_TILES) {
    static SmemAttrOnce smem_set;
    cfg.dynamicSmemBytes = fwd_smem_bytes<2>();
    e = smem_set.ensure(sink_attn_fwd_kernel<2>, cfg.dynamicSmemBytes)
            ? cudaLaunchKernelEx(&cfg, sink_attn_fwd_kernel<2>, tq, tk, tv, p)
            : cudaErrorInvalidValue;
  } else {
    static SmemAttrOnce smem_set;
    cfg.dynamicSmemBytes = kF2SmemBytes;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = smem_set.ensure(sink_attn_fwd_pair_kernel, cfg.dynamicSmemBytes)
            ? cudaLaunchKernelEx(&cfg, sink_attn_fwd_pair_kernel, tq, tk, tv, p)
            : cudaErrorInvalidValue;
  }
  if (g_profile_events[0][1]) cudaEventRecord(g_profile_events[0][1], st_);
  return e == cudaSuccess ? SINK_ATTN_OK : SINK_ATTN_ERR_CUDA;
}

size_t sink_attn_bwd_workspace_size(const sink_attn_dims* d) {
  Geometry geo;
  if (check_dims(d, nullptr, true, 0, 1.f, &geo) != SINK_ATTN_OK) return 0;
  return bwd_workspace_layout(geo).total;
}

int sink_attn_bwd_launches(const sink_attn_dims* d) {
  Geometry geo;
  if (check_dims(d, nullptr, true, 0, 1.f, &geo) != SINK_ATTN_OK) return 0;
  return d->total_tokens > 0 ? kBwdLaunches : 0;
}

sink_attn_status sink_attn_bwd(const sink_attn_dims* d, const void* q, const void* k, const void* v,
                               const float* sinks, const int* cu_seqlens, int window, float scale, const void* out,
                               const float* lse, const void* dout, void* dq, void* dk, void* dv, float* dsinks,
                               void* workspace, size_t workspace_bytes, void* stream) {
  Geometry geo;
  sink_attn_status st = check_dims(d, cu_seqlens, cu_seqlens != nullptr, window, scale, &geo);
  if (st != SINK_ATTN_OK) return st;
  if (!dsinks) return SINK_ATTN_ERR_NULL;
  if (geo.T == 0) {
    // No rows: every sink gradient is an empty sum.
    return cudaMemsetAsync(dsinks, 0, sizeof(float) * geo.Hq, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SINK_ATTN_OK
               : SINK_ATTN_ERR_CUDA;
  }
  if (!q || !k || !v || !sinks || !out || !lse || !dout || !dq || !dk || !dv) return SINK_ATTN_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(dout) || !aligned16(dq) ||
      !aligned16(dk) || !aligned16(dv) || (reinterpret_cast<uintptr_t>(lse) & 3u) ||
      (reinterpret_cast<uintptr_t>(sinks) & 3u) || (reinterpret_cast<uintptr_t>(dsinks) & 3u) ||
      (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u))
    return SINK_ATTN_ERR_ALIGN;
  const BwdWorkspace ws = bwd_workspace_layout(geo);
  if (!workspace || workspace_bytes < ws.total) return SINK_ATTN_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return SINK_ATTN_ERR_ALIGN;
  return bwd_launch(geo, scale, q, k, v, sinks, out, lse, dout, dq, dk, dv, dsinks,
                    static_cast<uint8_t*>(workspace), ws, static_cast<cudaStream_t>(stream), g_profile_events[1][0],
                    g_profile_events[1][1]);
}

}  // extern "C"

// ----------------------------------------------------------------------------
// Backward without caller-provided workspace, for callers that cannot
// allocate device memory (see sink_attn_bwd_noalloc in sink_attn.h).  The
// scratch is this fixed array; host code must not use its name as a device
// address (it is a host-side stand-in), so its address is looked up once per
// device with cudaGetSymbolAddress and cached.
namespace {

static __device__ __align__(256) uint8_t g_noalloc_scratch[SINK_ATTN_NOALLOC_SCRATCH_BYTES];

std::mutex g_noalloc_mutex;
void* g_noalloc_ptr[kMaxDevices] = {};

// Device address of g_noalloc_scratch on the current device, or nullptr.
void* noalloc_scratch_for_current_device() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(g_noalloc_mutex);
  if (g_noalloc_ptr[dev] == nullptr) {
    void* ptr = nullptr;
    if (cudaGetSymbolAddress(&ptr, g_noalloc_scratch) != cudaSuccess || ptr == nullptr) return nullptr;
    g_noalloc_ptr[dev] = ptr;
  }
  return g_noalloc_ptr[dev];
}

}  // namespace

extern "C" sink_attn_status sink_attn_bwd_noalloc(const sink_attn_dims* d, const void* q, const void* k,
                                                  const void* v, const float* sinks, const int* cu_seqlens,
                                                  int window, float scale, const void* out, const float* lse,
                                                  const void* dout, void* dq, void* dk, void* dv, float* dsinks,
                                                  void* stream) {
  Geometry geo;
  sink_attn_status st = check_dims(d, cu_seqlens, cu_seqlens != nullptr, window, scale, &geo);
  if (st != SINK_ATTN_OK) return st;
  const size_t need = bwd_workspace_layout(geo).total;
  if (need > SINK_ATTN_NOALLOC_SCRATCH_BYTES) return SINK_ATTN_ERR_WORKSPACE;
  void* scratch = noalloc_scratch_for_current_device();
  if (scratch == nullptr) return SINK_ATTN_ERR_CUDA;
  return sink_attn_bwd(d, q, k, v, sinks, cu_seqlens, window, scale, out, lse, dout, dq, dk, dv, dsinks, scratch,
                       SINK_ATTN_NOALLOC_SCRATCH_BYTES, stream);
}

extern "C" {

size_t sink_attn_decode_workspace_size(const sink_attn_decode_dims* d, int window) {
  DecPlan plan;
  if (plan_decode(d, window, 1.f, &plan) != SINK_ATTN_OK) return 0;
  return plan.total;
}

int sink_attn_decode_launches(const sink_attn_decode_dims* d, int window) {
  DecPlan plan;
  if (plan_decode(d, window, 1.f, &plan) != SINK_ATTN_OK) return 0;
  return d->batch > 0 ? (plan.p.n_split > 1 ? 3 : 2) : 0;
}

}  // extern "C"

namespace {

// mode: 0 bf16 cache; 1 e4m3 cache, fp16 MMAs; 2 e4m3 cache, FP8 PV.
sink_attn_status decode_impl(const sink_attn_decode_dims* d, const void* q, const void* k_new, const void* v_new,
                             void* k_cache, void* v_cache, const int* cache_seqlens, const float* k_scale,
                             const float* v_scale, int mode, const float* sinks, int window, float scale, void* out,
                             float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const bool e4m3 = mode != 0;
  DecPlan plan;
  sink_attn_status st = plan_decode(d, window, scale, &plan);
  if (st != SINK_ATTN_OK) return st;
  if (d->batch == 0) return SINK_ATTN_OK;
  if (!q || !k_new || !v_new || !k_cache || !v_cache || !cache_seqlens || !sinks || !out || !lse ||
      (e4m3 && (!k_scale || !v_scale)))
    return SINK_ATTN_ERR_NULL;
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(out) || (reinterpret_cast<uintptr_t>(lse) & 3u) || (reinterpret_cast<uintptr_t>(sinks) & 3u) ||
      (reinterpret_cast<uintptr_t>(cache_seqlens) & 3u) || (reinterpret_cast<uintptr_t>(k_scale) & 3u) ||
      (reinterpret_cast<uintptr_t>(v_scale) & 3u))
    return SINK_ATTN_ERR_ALIGN;
  if (!workspace || workspace_bytes < plan.total || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return SINK_ATTN_ERR_WORKSPACE;
  DecParams p = plan.p;
  p.seqlens = cache_seqlens;
  p.sinks = sinks;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.o_part = reinterpret_cast<float*>(ws + plan.o_off);
  p.m_part = reinterpret_cast<float*>(ws + plan.m_off);
  p.l_part = reinterpret_cast<float*>(ws + plan.l_off);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse_out = lse;

  CUtensorMap tq, tk, tv;
  if (!make_map_3d(&tq, q, kHeadDim, p.Hq, p.batch * p.Lq, p.G, p.Lq)) return SINK_ATTN_ERR_CUDA;
  if (e4m3) {
    if (!make_map_3d_u8(&tk, k_cache, kHeadDim, p.Hkv, p.batch * p.C, 1, kDecTile) ||
        !make_map_3d_u8(&tv, v_cache, kHeadDim, p.Hkv, p.batch * p.C, 1, kDecTile))
      return SINK_ATTN_ERR_CUDA;
  } else if (!make_map_3d(&tk, k_cache, kHeadDim, p.Hkv, p.batch * p.C, 1, kDecTile) ||
             !make_map_3d(&tv, v_cache, kHeadDim, p.Hkv, p.batch * p.C, 1, kDecTile)) {
    return SINK_ATTN_ERR_CUDA;
  }
  // Register arrays sized for the real query rows.
  using Kern = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, DecParams);
  static const Kern kerns[3][4] = {
      {sink_attn_decode_kernel<8, 0>, sink_attn_decode_kernel<16, 0>, sink_attn_decode_kernel<32, 0>,
       sink_attn_decode_kernel<64, 0>},
      {sink_attn_decode_kernel<8, 1>, sink_attn_decode_kernel<16, 1>, sink_attn_decode_kernel<32, 1>,
       sink_attn_decode_kernel<64, 1>},
      {sink_attn_decode_kernel<8, 2>, sink_attn_decode_kernel<16, 2>, sink_attn_decode_kernel<32, 2>,
       sink_attn_decode_kernel<64, 2>}};
  static SmemAttrOnce smem_set[3][4];
  const int vi = p.R <= 8 ? 0 : (p.R <= 16 ? 1 : (p.R <= 32 ? 2 : 3));
  const Kern kern = kerns[mode][vi];
  const size_t smem = mode == 2 ? kDecSmemBytesPv8 : (mode == 1 ? kDecSmemBytes8 : kDecSmemBytes);
  if (!smem_set[mode][vi].ensure(kern, smem)) return SINK_ATTN_ERR_CUDA;
  const long long ctas = static_cast<long long>(p.batch) * p.Hkv * p.n_split;
  if (ctas > 0x7fffffff) return SINK_ATTN_ERR_UNSUPPORTED;

  cudaStream_t st_ = static_cast<cudaStream_t>(stream);
  if (e4m3) {
    const long long chunks = 2LL * p.batch * p.Lq * p.Hkv * (kHeadDim / 16);
    sink_attn_cache_append_e4m3_kernel<<<static_cast<unsigned>((chunks + 255) / 256), 256, 0, st_>>>(
        p, static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), static_cast<uint4*>(k_cache),
        static_cast<uint4*>(v_cache));
  } else {
    const long long chunks = 2LL * p.batch * p.Lq * p.Hkv * (kHeadDim * 2 / 16);
    sink_attn_cache_append_kernel<<<static_cast<unsigned>((chunks + 255) / 256), 256, 0, st_>>>(
        p, static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), static_cast<uint4*>(k_cache),
        static_cast<uint4*>(v_cache));
  }
  kern<<<static_cast<unsigned>(ctas), e4m3 ? kDecThreads8 : kDecThreads, smem, st_>>>(tq, tk, tv, p);
  if (p.n_split > 1) {
    const long long rows = static_cast<long long>(p.batch) * p.Lq * p.Hq;
    sink_attn_decode_combine_kernel<<<static_cast<unsigned>((rows + 3) / 4), 128, 0, st_>>>(
        p, static_cast<__nv_bfloat16*>(out), lse);
  }
  return cudaPeekAtLastError() == cudaSuccess ? SINK_ATTN_OK : SINK_ATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

sink_attn_status sink_attn_decode(const sink_attn_decode_dims* d, const void* q, const void* k_new,
                                  const void* v_new, void* k_cache, void* v_cache, const int* cache_seqlens,
                                  const float* sinks, int window, float scale, void* out, float* lse,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  return decode_impl(d, q, k_new, v_new, k_cache, v_cache, cache_seqlens, nullptr, nullptr, 0, sinks, window,
                     scale, out, lse, workspace, workspace_bytes, stream);
}

sink_attn_status sink_attn_decode_e4m3(const sink_attn_decode_dims* d, const void* q, const void* k_new,
                                       const void* v_new, void* k_cache, void* v_cache, const int* cache_seqlens,
                                       const float* k_scale, const float* v_scale, const float* sinks, int window,
                                       float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  return decode_impl(d, q, k_new, v_new, k_cache, v_cache, cache_seqlens, k_scale, v_scale, 1, sinks, window,
                     scale, out, lse, workspace, workspace_bytes, stream);
}

sink_attn_status sink_attn_decode_e4m3_f8pv(const sink_attn_decode_dims* d, const void* q, const void* k_new,
                                            const void* v_new, void* k_cache, void* v_cache,
                                            const int* cache_seqlens, const float* k_scale, const float* v_scale,
                                            const float* sinks, int window, float scale, void* out, float* lse,
                                            void* workspace, size_t workspace_bytes, void* stream) {
  return decode_impl(d, q, k_new, v_new, k_cache, v_cache, cache_seqlens, k_scale, v_scale, 2, sinks, window,
                     scale, out, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"

// ----------------------------------------------------------------------------
// Paged cache.
namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Launches a kernel that may start before the one before it on the stream has
// ended, and waits for that by itself before it touches memory (pdl_wait): the
// kernels of a serving step follow one another within a few microseconds, and
// this hides the start of each.
template <typename... A>
bool launch_early(void (*kernel)(A...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

// Sizes and strides shared by the paged append and attention.  `codes`: the
// cache holds one byte per element, so a row's 16-byte alignment needs strides
// that are multiples of 16 elements, not 8.
sink_attn_status check_paged(const sink_attn_paged_dims* d, bool codes) {
  if (!d) return SINK_ATTN_ERR_NULL;
  if (d->total_tokens < 0 || d->num_kv_heads <= 0 || d->head_dim <= 0 || d->page_size <= 0 || d->num_pages <= 0 ||
      d->page_stride < 0 || d->token_stride < 0 || d->head_stride < 0)
    return SINK_ATTN_ERR_SHAPE;
  if (d->head_dim != kHeadDim) return SINK_ATTN_ERR_UNSUPPORTED;
  if (ilog2_exact(d->page_size) < 4 || d->page_size > 1024) return SINK_ATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(d->num_pages) * d->page_size >= (int64_t(1) << 31) ||
      d->total_tokens > (1 << 30) || d->num_kv_heads > (1 << 16))
    return SINK_ATTN_ERR_UNSUPPORTED;
  // Rows of a cache do not overlap (a dimension of one element may have any
  // stride), and TMA takes strides below 2^40 bytes.
  const long long strides[3] = {d->page_stride, d->token_stride, d->head_stride};
  const int sizes[3] = {d->num_pages, d->page_size, d->num_kv_heads};
  for (int i = 0; i < 3; ++i) {
    if (sizes[i] > 1 && strides[i] < kHeadDim) return SINK_ATTN_ERR_SHAPE;
    if (strides[i] >= (1ll << 38)) return SINK_ATTN_ERR_UNSUPPORTED;
  }
  const long long unit = codes ? 16 : 8;
  if (d->page_stride % unit || d->token_stride % unit || d->head_stride % unit) return SINK_ATTN_ERR_ALIGN;
  return SINK_ATTN_OK;
}

sink_attn_status paged_append_impl(const sink_attn_paged_dims* d, const void* k_new, const void* v_new,
                                   long long k_stride, long long v_stride, const int* slot_map, void* k_cache,
                                   void* v_cache, const float* k_scale, const float* v_scale, bool codes,
                                   void* stream) {
  sink_attn_status st = check_paged(d, codes);
  if (st != SINK_ATTN_OK) return st;
  if (k_stride < 0 || v_stride < 0) return SINK_ATTN_ERR_SHAPE;
  if (d->total_tokens == 0) return SINK_ATTN_OK;
  if (!k_new || !v_new || !slot_map || !k_cache || !v_cache || (codes && (!k_scale || !v_scale)))
    return SINK_ATTN_ERR_NULL;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) || k_stride % 8 ||
      v_stride % 8 || !aligned4(slot_map) || !aligned4(k_scale) || !aligned4(v_scale))
    return SINK_ATTN_ERR_ALIGN;
  AppendParams p;
  p.tokens = d->total_tokens;
  p.Hkv = d->num_kv_heads;
  p.page_log2 = ilog2_exact(d->page_size);
  p.slots_end = static_cast<long long>(d->num_pages) * d->page_size;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.page_stride = d->page_stride;
  p.token_stride = d->token_stride;
  p.head_stride = d->head_stride;
  p.slots = slot_map;
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  const long long work = static_cast<long long>(p.tokens) * p.Hkv * (kHeadDim / 16);
  const long long blocks = (work + 255) / 256;
  if (blocks > 0x7fffffff) return SINK_ATTN_ERR_UNSUPPORTED;
  cudaStream_t st_ = static_cast<cudaStream_t>(stream);
  return launch_early(codes ? sink_attn_paged_append_kernel<true> : sink_attn_paged_append_kernel<false>,
                      dim3(static_cast<unsigned>(blocks)), 256, 0, st_, p)
             ? SINK_ATTN_OK
             : SINK_ATTN_ERR_CUDA;
}

sink_attn_status check_paged_attn(const sink_attn_paged_dims* d, bool codes) {
  sink_attn_status st = check_paged(d, codes);
  if (st != SINK_ATTN_OK) return st;
  if (d->batch < 0 || d->max_new <= 0 || d->max_pages <= 0 || d->num_q_heads <= 0 || d->q_stride < 0)
    return SINK_ATTN_ERR_SHAPE;
  if (d->num_q_heads % d->num_kv_heads != 0) return SINK_ATTN_ERR_SHAPE;
  if (d->num_q_heads / d->num_kv_heads > kBlockM || d->batch > kPagedMaxBatch) return SINK_ATTN_ERR_UNSUPPORTED;
  // Positions are 32-bit, with room for a tile behind the last one; so are the
  // blocks of keys of all requests, and a worker's share of them.
  const int64_t tokens = static_cast<int64_t>(d->max_pages) * d->page_size;
  const int64_t chunks = d->num_kv_heads;  // of heads, at most
  if (tokens > (int64_t(1) << 30) || tokens * std::max(d->batch, 1) > (int64_t(1) << 35) / chunks)
    return SINK_ATTN_ERR_UNSUPPORTED;
  if (d->total_tokens > 1 && d->q_stride < static_cast<long long>(d->num_q_heads) * kHeadDim) return SINK_ATTN_ERR_SHAPE;
  if (d->q_stride >= (1ll << 38)) return SINK_ATTN_ERR_UNSUPPORTED;
  // Units of the chunk kernel, of at least one 128-row tile each (or the end of a request).
  const int tile = kBlockM / (d->num_q_heads / d->num_kv_heads);
  if ((d->total_tokens / tile + std::min(d->batch, d->total_tokens)) * static_cast<int64_t>(d->num_kv_heads) >= kChunkMaxUnits)
    return SINK_ATTN_ERR_UNSUPPORTED;
  if (d->q_stride % 8) return SINK_ATTN_ERR_ALIGN;
  return SINK_ATTN_OK;
}

// Which kernels a call's requests go to.  A request of at most `few` new
// tokens is the few-rows kernel's, with tiles of kR rows (8 or 16) and as many
// warps a head as hold all of the call's requests, or if none do (the call has
// chunks) one token of a group.
struct PagedSplit {
  int kR, row_parts, few;
  bool rows, chunks;
};

PagedSplit split_paged(const sink_attn_paged_dims* d) {
  PagedSplit s;
  const int G = d->num_q_heads / d->num_kv_heads;
  const int64_t need = static_cast<int64_t>(std::min(d->max_new, d->total_tokens)) * G;
  const int64_t fit = need <= kRowsMaxRows ? need : G;
  s.kR = fit <= 8 ? 8 : 16;
  s.row_parts = fit <= 16 ? 1 : fit <= 32 ? 2 : 4;
  s.few = std::min(kRowsMaxRows, s.kR * s.row_parts) / G;
  s.rows = s.few > 0;
  s.chunks = need > static_cast<int64_t>(s.few) * G;
  return s;
}

// Chunks of key/value heads of the few-rows kernel, and heads of a chunk.
int rows_chunks(const sink_attn_paged_dims* d, const PagedSplit& s) {
  const int heads = kRowsWarps / s.row_parts;
  return (d->num_kv_heads + heads - 1) / heads;
}

constexpr int kPagedCtas = 148;  // one CTA per SM of a B200
constexpr int kPagedWarps = kPagedCtas * kRowsWarps;

// Upper bound of the chunk kernel's units, and of the parts its last units are
// cut into (0: their keys are too few to be cut).  The lengths are not known here.
struct ChunkBound {
  int64_t units, parts;
};

template <bool kF8>
ChunkBound chunk_bound(const sink_attn_paged_dims* d, const PagedSplit& s, int window) {
  ChunkBound c;
  const int tokens = kChunkTiles<kF8> * (kBlockM / (d->num_q_heads / d->num_kv_heads));  // of a unit
  const int64_t requests = std::min<int64_t>(d->batch, d->total_tokens / (s.few + 1));
  c.units = d->num_kv_heads * (d->total_tokens / tokens + requests);
  const int64_t keys = std::min<int64_t>(int64_t(d->max_pages) * d->page_size,
                                         window > 0 ? int64_t(window) + tokens : INT64_MAX);
  const int64_t most = std::min<int64_t>((keys / kHalfN + 1) / kChunkLeast, kChunkMostParts);  // parts of a unit
  const int64_t wave = kChunkPerSm<kF8> * kChunkSms;
  c.parts = most < 2 ? 0 : std::min(kChunkMaxWaves * wave, std::min(c.units, wave) * most);
  return c;
}

// Workspace of a call (bytes): the pieces of cut units of both kernels.
struct PagedWorkspace {
  size_t unit, ml, o;
  size_t chunk_units, chunk_unit, chunk_ml, chunk_o;
  size_t total;
};

PagedWorkspace paged_workspace(const sink_attn_paged_dims* d, const PagedSplit& s) {
  PagedWorkspace w = {};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round256(bytes);
    return here;
  };
  if (s.rows) {
    const size_t rows = static_cast<size_t>(kPagedWarps) * 2 * s.kR;
    w.unit = take(kPagedWarps * sizeof(int4));
    w.ml = take(rows * sizeof(float2));
    w.o = take(rows * kHeadDim * sizeof(float));
  }
  if (s.chunks) {
    // (Rows of parts: for either type of cache.)
    const size_t rows = static_cast<size_t>(std::max(chunk_bound<false>(d, s, 0).parts * kChunkTiles<false>,
                                                     chunk_bound<true>(d, s, 0).parts * kChunkTiles<true>)) * kBlockM;
    w.chunk_units = take(sizeof(int2));
    w.chunk_unit = take(kChunkPerSm<false> * kChunkSms * sizeof(int4));
    w.chunk_ml = take(rows * sizeof(float2));
    w.chunk_o = take(rows * kHeadDim * sizeof(float));
  }
  w.total = std::max<size_t>(at, 256);
  return w;
}

// 4-D view [page][head][token][64] of a paged cache with a box of `tokens`
// tokens of `heads` heads: 128-byte rows (bf16) under the 128-byte swizzle, or
// 64-byte rows (codes) under the 64-byte swizzle.
bool make_map_paged(CUtensorMap* map, const void* base, const sink_attn_paged_dims* d, bool codes, int tokens,
                    int heads) {
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return false;
  const cuuint64_t size = codes ? 1 : 2;
  cuuint64_t dims[4] = {kHeadDim, static_cast<cuuint64_t>(d->page_size), static_cast<cuuint64_t>(d->num_kv_heads),
                        static_cast<cuuint64_t>(d->num_pages)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(d->token_stride) * size,
                           static_cast<cuuint64_t>(d->head_stride) * size,
                           static_cast<cuuint64_t>(d->page_stride) * size};
  // The stride of a dimension of one element is never used, and may be anything.
  for (int i = 0; i < 3; ++i)
    if (dims[i + 1] == 1) strides[i] = kHeadDim * size;
  cuuint32_t box[4] = {kHeadDim, static_cast<cuuint32_t>(tokens), static_cast<cuuint32_t>(heads), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             codes ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The longest unit of a call, in blocks, is short enough that no cut is left
// inside one (see RowsAxis::cut): nothing to join.
template <bool kF8>
bool rows_never_cut(const PagedParams& p) {
  const int64_t keys = std::min(int64_t(p.max_pages) << p.page_log2,
                                p.window > 0 ? static_cast<int64_t>(p.window) + p.few - 1 : INT64_MAX);
  const int64_t lead = p.window > 0 ? (1 << p.box_log2) - 1 : 0;
  return (keys + lead + kRowsKeys<kF8> - 1) / kRowsKeys<kF8> <= 2 * kRowsSnap<kF8> + 1;
}

// kBeside: the chunk kernel runs before it on the stream.  The two share
// nothing but the SMs, which take the pieces of this kernel as they run out of
// chunks, so it does not wait for the other to end.
template <bool kF8, int kR, bool kBeside>
bool launch_rows(PagedParams& p, const sink_attn_paged_dims* d, const void* k_cache, const void* v_cache, dim3* join,
                 cudaStream_t st) {
  const int box = std::min(d->page_size, kRowsKeys<kF8>);
  p.box_log2 = ilog2_exact(box);
  CUtensorMap tm_k, tm_v;
  if (!make_map_paged(&tm_k, k_cache, d, kF8, box, p.per_chunk) ||
      !make_map_paged(&tm_v, v_cache, d, kF8, box, p.per_chunk)) return false;
  static SmemAttrOnce smem_set;
  if (!smem_set.ensure(sink_attn_paged_rows_kernel<kF8, kR, kBeside>, rows_smem_bytes(kPagedMaxBatch))) return false;
  const bool cut = !rows_never_cut<kF8>(p);
  if (!cut) p.part_unit = nullptr;
  // No more CTAs than the most blocks there can be give work to.
  const int64_t keys = p.window > 0 ? static_cast<int64_t>(p.window) + p.few - 1 + box : INT64_MAX;
  const int64_t most = (std::min(keys, int64_t(p.max_pages) << p.page_log2) + kRowsKeys<kF8> - 1) / kRowsKeys<kF8> + 1;
  const int64_t workers = std::max((most * p.batch * p.chunks + kRowsMinBlocks - 1) / kRowsMinBlocks,
                                   int64_t(p.batch) * p.chunks);
  const int per_group = p.per_chunk * p.row_parts, groups = kRowsWarps / per_group;
  const int ctas = static_cast<int>(std::min<int64_t>(kPagedCtas, workers));
  if (cut) *join = dim3(ctas * groups, per_group);
  return launch_early(sink_attn_paged_rows_kernel<kF8, kR, kBeside>, dim3(ctas), kRowsThreads, rows_smem_bytes(p.batch), st, tm_k,
                      tm_v, p);
}

template <bool kF8, int kR>
bool launch_rows(PagedParams& p, const sink_attn_paged_dims* d, const void* k_cache, const void* v_cache, bool beside,
                 dim3* join, cudaStream_t st) {
  return beside ? launch_rows<kF8, kR, true>(p, d, k_cache, v_cache, join, st)
                : launch_rows<kF8, kR, false>(p, d, k_cache, v_cache, join, st);
}

template <bool kF8>
bool launch_rows(int kR, PagedParams& p, const sink_attn_paged_dims* d, const void* k_cache, const void* v_cache,
                 bool beside, dim3* join, cudaStream_t st) {
  return kR == 8 ? launch_rows<kF8, 8>(p, d, k_cache, v_cache, beside, join, st)
                 : launch_rows<kF8, 16>(p, d, k_cache, v_cache, beside, join, st);
}

// The query tile of the chunk kernel, `tokens` tokens of one group of heads.
bool make_map_paged_q(CUtensorMap* map, const sink_attn_paged_dims* d, const void* q, int G, int tokens) {
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return false;
  cuuint64_t dims[3] = {kHeadDim, static_cast<cuuint64_t>(d->num_q_heads), static_cast<cuuint64_t>(d->total_tokens)};
  cuuint64_t strides[2] = {kHeadDim * 2, static_cast<cuuint64_t>(d->q_stride) * 2};
  if (dims[2] == 1) strides[1] = dims[1] * strides[0];
  cuuint32_t box[3] = {kHeadDim, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(tokens)};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kF8>
bool launch_chunks(ChunkParams& p, const sink_attn_paged_dims* d, const void* k_cache, const void* v_cache,
                   const PagedSplit& split, unsigned* join, cudaStream_t st) {
  const ChunkBound bound = chunk_bound<kF8>(d, split, p.a.window);
  p.wave = kChunkPerSm<kF8> * kChunkSms;
  p.tiles = kChunkTiles<kF8>;
  CUtensorMap tm_q, tm_k, tm_v;
  const int box = std::min(d->page_size, kHalfN);
  p.a.box_log2 = ilog2_exact(box);
  if (!make_map_paged_q(&tm_q, d, p.a.q, p.a.G, p.tokens) || !make_map_paged(&tm_k, k_cache, d, kF8, box, 1) ||
      !make_map_paged(&tm_v, v_cache, d, kF8, box, 1))
    return false;
  static SmemAttrOnce smem_set;
  if (!smem_set.ensure(sink_attn_paged_chunk_kernel<kF8>, chunk_smem_bytes<kF8>())) return false;
  if (bound.parts == 0) p.part_o = nullptr;
  p.max_units = static_cast<int>(bound.units);
  p.max_cut = static_cast<int>(std::min<int64_t>(bound.units, p.wave - 1));
  p.max_parts = static_cast<int>(bound.parts);
  // Units too short to be cut (a window): one wave of CTAs, each taking its
  // turns, which saves every unit the start of a CTA.  Longer ones: a CTA for
  // each, which the SMs even out among themselves (as many as whole units come
  // from the rows, four waves at least: most of the bound for requests' ends is
  // CTAs that find no work); but one wave again when most requests must be
  // single tokens, since the few-rows kernel can take its place beside this one
  // only when all CTAs of this one have started.  (Window-128 chunks: 61 us in
  // turns, 84 with a CTA each; 2048 tokens of 32768: 1445 in turns, 1383; five
  // chunks and 28 tokens: 76 in turns, 85.  A call that leaves max_new at T and
  // has three requests or more counts as single tokens: four prompts of 4096 take
  // 826 to 837 us then, 754 to 768 with max_new given.)
  const bool turns = bound.parts == 0 || d->total_tokens < static_cast<int64_t>(d->batch) * d->max_new / 2;
  const int64_t places = bound.units + bound.parts;
  // (With one CTA a SM, e4m3, four waves are enough: nobody computes while the
  // next CTA starts.  Nine prompts of 200 to 3000 tokens: 430 us, 445 with all.
  // Four of 4096 over bf16: 744 with all, 797 with four waves.)
  const int64_t whole =
      kChunkPerSm<kF8> > 1 ? static_cast<int64_t>(p.a.T / (p.tiles * p.tokens)) * p.a.Hkv : 0;  // units, but for requests' ends
  const unsigned ctas = static_cast<unsigned>(
      std::min(places, turns ? p.wave : std::max<int64_t>((kChunkMaxWaves + 1) * p.wave, whole)));
  if (bound.parts) *join = static_cast<unsigned>(p.max_cut * (p.tiles * kBlockM / 32));
  return launch_early(sink_attn_paged_chunk_kernel<kF8>, dim3(ctas), kChunkThreads<kF8>, chunk_smem_bytes<kF8>(), st, tm_q,
                      tm_k, tm_v, p);
}

sink_attn_status paged_attn_impl(const sink_attn_paged_dims* d, const void* q, const void* k_cache,
                                 const void* v_cache, const int* block_table, const int* cu_seqlens,
                                 const int* kv_lens, const float* k_scale, const float* v_scale, bool codes,
                                 const float* sinks, int window, float scale, void* out, float* lse,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  sink_attn_status st = check_paged_attn(d, codes);
  if (st != SINK_ATTN_OK) return st;
  if (!(scale > 0.f) || !std::isfinite(scale)) return SINK_ATTN_ERR_UNSUPPORTED;
  if (d->total_tokens == 0 || d->batch == 0) return SINK_ATTN_OK;
  if (!q || !k_cache || !v_cache || !block_table || !cu_seqlens || !kv_lens || !sinks || !out || !lse ||
      (codes && (!k_scale || !v_scale)))
    return SINK_ATTN_ERR_NULL;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned4(block_table) ||
      !aligned4(cu_seqlens) || !aligned4(kv_lens) || !aligned4(sinks) || !aligned4(lse) || !aligned4(k_scale) ||
      !aligned4(v_scale))
    return SINK_ATTN_ERR_ALIGN;
  const PagedSplit split = split_paged(d);
  const PagedWorkspace ws = paged_workspace(d, split);
  if (workspace_bytes < ws.total || !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return SINK_ATTN_ERR_WORKSPACE;
  PagedParams p;
  p.batch = d->batch;
  p.T = d->total_tokens;
  p.Hq = d->num_q_heads;
  p.Hkv = d->num_kv_heads;
  p.G = p.Hq / p.Hkv;
  p.max_new = d->max_new;
  p.page_log2 = ilog2_exact(d->page_size);
  p.num_pages = d->num_pages;
  p.max_pages = d->max_pages;
  p.box_log2 = 0;
  p.few = split.few;
  p.row_parts = split.row_parts;
  p.chunks = rows_chunks(d, split);
  p.per_chunk = (p.Hkv + p.chunks - 1) / p.chunks;
  // (A window beyond all positions is none, and keeps their differences in 32 bits.)
  p.window = window > 0 && window < (1 << 30) ? window : 0;
  p.scale_log2 = scale * kLog2e;
  p.q_stride = d->q_stride;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.table = block_table;
  p.cu = cu_seqlens;
  p.kv_lens = kv_lens;
  p.sinks = sinks;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  p.part_unit = reinterpret_cast<int4*>(base + ws.unit);
  p.part_ml = reinterpret_cast<float2*>(base + ws.ml);
  p.part_o = reinterpret_cast<float*>(base + ws.o);
  cudaStream_t st_ = static_cast<cudaStream_t>(stream);
  ChunkParams c = {};
  unsigned chunk_join = 0;  // CTAs of the join
  dim3 rows_join(0, 0, 1);
  if (split.chunks) {
    c.a = p;
    c.tokens = kBlockM / p.G;
    c.part_units = reinterpret_cast<int2*>(base + ws.chunk_units);
    c.part_unit = reinterpret_cast<int4*>(base + ws.chunk_unit);
    c.part_ml = reinterpret_cast<float2*>(base + ws.chunk_ml);
    c.part_o = reinterpret_cast<float*>(base + ws.chunk_o);
    if (!(codes ? launch_chunks<true>(c, d, k_cache, v_cache, split, &chunk_join, st_)
                : launch_chunks<false>(c, d, k_cache, v_cache, split, &chunk_join, st_)))
      return SINK_ATTN_ERR_CUDA;
  }
  if (split.rows && !(codes ? launch_rows<true>(split.kR, p, d, k_cache, v_cache, split.chunks, &rows_join, st_)
                            : launch_rows<false>(split.kR, p, d, k_cache, v_cache, split.chunks, &rows_join, st_)))
    return SINK_ATTN_ERR_CUDA;
  if (chunk_join) {
    c.a = p;
    const int workers = static_cast<int>(rows_join.x);
    if (!launch_early(split.kR == 8 ? sink_attn_paged_join_both_kernel<8> : sink_attn_paged_join_both_kernel<16>,
                      dim3(chunk_join + rows_join.x * rows_join.y), 256, 0, st_, c, static_cast<int>(chunk_join), workers))
      return SINK_ATTN_ERR_CUDA;
  } else if (rows_join.x &&
             !launch_early(split.kR == 8 ? sink_attn_paged_join_kernel<8> : sink_attn_paged_join_kernel<16>, rows_join, 256,
                           0, st_, p)) {
    return SINK_ATTN_ERR_CUDA;
  }
  return SINK_ATTN_OK;
}

}  // namespace

extern "C" {

sink_attn_status sink_attn_paged_plan(const sink_attn_plan_dims* d, const int* cached_lens, const int* new_lens,
                                      int* block_table, int* free_pages, const int* pool, const int* first_page,
                                      int window, int* cu_seqlens, int* kv_lens, int* slot_map, int* pool_out,
                                      int* first_page_out, void* stream) {
  if (!d) return SINK_ATTN_ERR_NULL;
  if (d->batch < 0 || d->max_tokens < 0 || d->max_pages <= 0 || d->page_size <= 0 || d->num_pages <= 0)
    return SINK_ATTN_ERR_SHAPE;
  if (ilog2_exact(d->page_size) < 4 || d->page_size > 1024 || d->batch > kPlanMaxBatch)
    return SINK_ATTN_ERR_UNSUPPORTED;
  // Slots, positions and their sums over the requests are 32-bit.
  if (static_cast<int64_t>(d->num_pages) * d->page_size >= (int64_t(1) << 31) ||
      static_cast<int64_t>(std::max(d->batch, 1)) * d->max_pages * d->page_size > (int64_t(1) << 30) ||
      d->max_tokens > (1 << 30))
    return SINK_ATTN_ERR_UNSUPPORTED;
  // Giving pages back needs the record of those already given back.
  if (window > 0 && !first_page) return SINK_ATTN_ERR_NULL;
  if ((first_page == nullptr) != (first_page_out == nullptr)) return SINK_ATTN_ERR_NULL;
  if (d->batch == 0) return SINK_ATTN_OK;
  if (!cached_lens || !new_lens || !block_table || !free_pages || !pool || !cu_seqlens || !kv_lens || !pool_out ||
      (d->max_tokens > 0 && !slot_map))
    return SINK_ATTN_ERR_NULL;
  if (!aligned4(cached_lens) || !aligned4(new_lens) || !aligned4(block_table) || !aligned4(free_pages) ||
      !aligned4(pool) || !aligned4(first_page) || !aligned4(cu_seqlens) || !aligned4(kv_lens) ||
      !aligned4(slot_map) || !aligned4(pool_out) || !aligned4(first_page_out))
    return SINK_ATTN_ERR_ALIGN;
  PlanParams p;
  p.batch = d->batch;
  p.max_tokens = d->max_tokens;
  p.max_pages = d->max_pages;
  p.page_size = d->page_size;
  p.num_pages = d->num_pages;
  p.page_log2 = ilog2_exact(d->page_size);
  p.window = window > 0 ? window : 0;
  p.cached = cached_lens;
  p.fresh = new_lens;
  p.table = block_table;
  p.ring = free_pages;
  p.pool = pool;
  p.first = first_page;
  p.cu = cu_seqlens;
  p.kv = kv_lens;
  p.slots = slot_map;
  p.pool_out = pool_out;
  p.first_out = first_page_out;
  const size_t smem = plan_smem_bytes(p.batch);
  static SmemAttrOnce smem_set;
  if (!smem_set.ensure(sink_attn_paged_plan_kernel, plan_smem_bytes(kPlanMaxBatch))) return SINK_ATTN_ERR_CUDA;
  const unsigned blocks = p.max_tokens > kPlanThreads ? 8 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(kPlanThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see launch_early
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sink_attn_paged_plan_kernel, p) == cudaSuccess ? SINK_ATTN_OK : SINK_ATTN_ERR_CUDA;
}

sink_attn_status sink_attn_paged_append(const sink_attn_paged_dims* d, const void* k_new, const void* v_new,
                                        long long k_stride, long long v_stride, const int* slot_map, void* k_cache,
                                        void* v_cache, void* stream) {
  return paged_append_impl(d, k_new, v_new, k_stride, v_stride, slot_map, k_cache, v_cache, nullptr, nullptr, false,
                           stream);
}

sink_attn_status sink_attn_paged_append_e4m3(const sink_attn_paged_dims* d, const void* k_new, const void* v_new,
                                             long long k_stride, long long v_stride, const int* slot_map,
                                             void* k_cache, void* v_cache, const float* k_scale, const float* v_scale,
                                             void* stream) {
  return paged_append_impl(d, k_new, v_new, k_stride, v_stride, slot_map, k_cache, v_cache, k_scale, v_scale, true,
                           stream);
}

size_t sink_attn_paged_workspace_size(const sink_attn_paged_dims* d) {
  return check_paged_attn(d, false) == SINK_ATTN_OK ? paged_workspace(d, split_paged(d)).total : 0;
}

sink_attn_status sink_attn_paged_attn(const sink_attn_paged_dims* d, const void* q, const void* k_cache,
                                      const void* v_cache, const int* block_table, const int* cu_seqlens,
                                      const int* kv_lens, const float* sinks, int window, float scale, void* out,
                                      float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return paged_attn_impl(d, q, k_cache, v_cache, block_table, cu_seqlens, kv_lens, nullptr, nullptr, false, sinks,
                         window, scale, out, lse, workspace, workspace_bytes, stream);
}

sink_attn_status sink_attn_paged_attn_e4m3(const sink_attn_paged_dims* d, const void* q, const void* k_cache,
                                           const void* v_cache, const int* block_table, const int* cu_seqlens,
                                           const int* kv_lens, const float* k_scale, const float* v_scale,
                                           const float* sinks, int window, float scale, void* out, float* lse,
                                           void* workspace, size_t workspace_bytes, void* stream) {
  return paged_attn_impl(d, q, k_cache, v_cache, block_table, cu_seqlens, kv_lens, k_scale, v_scale, true, sinks,
                         window, scale, out, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
