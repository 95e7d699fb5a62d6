// Paged attention of longer requests, plainly: one thread per (token, query
// head) row, which walks its visible keys with a running maximum and sum.
#pragma once
#include "paged_attn.cuh"

namespace sa {

template <bool kF8>
__device__ __forceinline__ void paged_row(const void* cache, long long at, float* x) {
  if constexpr (kF8) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(cache) + at);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 v = __ldg(s + c);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint32_t h2 = e4m3x2_to_f16x2(w[u / 2] >> (16 * (u & 1)));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
        x[16 * c + 2 * u] = f.x;
        x[16 * c + 2 * u + 1] = f.y;
      }
    }
  } else {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(cache) + at);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint4 v = __ldg(s + c);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        x[8 * c + 2 * u] = __uint_as_float(w[u] << 16);
        x[8 * c + 2 * u + 1] = __uint_as_float(w[u] & 0xFFFF0000u);
      }
    }
  }
}

template <bool kF8>
__global__ void __launch_bounds__(128) sink_attn_paged_kernel(const __grid_constant__ PagedParams p, const void* k_cache, const void* v_cache, long long page_stride, long long token_stride, long long head_stride) {
  const long long r = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int g = blockIdx.y;
  const int t = static_cast<int>(r / p.G);
  if (r == 0 && __ldg(p.cu + p.batch) > p.T) atomicCAS(&g_device_error, 0, static_cast<int>(kDevErrPagedRows));
  if (t >= p.T || t >= __ldg(p.cu + p.batch)) return;
  const int h = g * p.G + static_cast<int>(r % p.G);
  int lo = 0, hi = p.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(p.cu + mid) <= t) lo = mid; else hi = mid - 1;
  }
  const int b = lo;
  if (__ldg(p.cu + b + 1) - __ldg(p.cu + b) <= p.few) return;
  if (__ldg(p.cu + b + 1) - __ldg(p.cu + b) > p.max_new) atomicCAS(&g_device_error, 0, static_cast<int>(kDevErrPagedRows));
  const int len = min(max(__ldg(p.kv_lens + b), 0), p.max_pages << p.page_log2);
  const int i = len - (__ldg(p.cu + b + 1) - t);
  float q[kHeadDim], o[kHeadDim];
  paged_row<false>(p.q, t * p.q_stride + h * kHeadDim, q);
#pragma unroll
  for (int d = 0; d < kHeadDim; ++d) o[d] = 0.f;
  const float sl2 = kF8 ? p.scale_log2 * __ldg(p.k_scale + g) : p.scale_log2;
  float m = __ldg(p.sinks + h) * kLog2e;
  // The sum is kept in two levels, 64 keys and all of them: thousands of small
  // weights added one by one to a sum near 1 would lose their low bits.
  float l = m == -INFINITY ? 0.f : 1.f, l64 = 0.f;
  for (int j = p.window > 0 ? max(0, i - p.window + 1) : 0; j <= i; ++j) {
    const int page = __ldg(p.table + static_cast<long long>(b) * p.max_pages + (j >> p.page_log2));
    if (page < 0 || page >= p.num_pages) {
      atomicCAS(&g_device_error, 0, static_cast<int>(kDevErrBadPage));
      continue;
    }
    const long long at = page * page_stride + (j & ((1 << p.page_log2) - 1)) * token_stride + g * head_stride;
    float x[kHeadDim];
    paged_row<kF8>(k_cache, at, x);
    float s = 0.f;
#pragma unroll
    for (int d = 0; d < kHeadDim; ++d) s = fmaf(q[d], x[d], s);
    s *= sl2;
    if (s > m) {
      const float f = exp2f(m - s);
      l *= f;
      l64 *= f;
#pragma unroll
      for (int d = 0; d < kHeadDim; ++d) o[d] *= f;
      m = s;
    }
    const float w = m == -INFINITY ? 0.f : exp2f(s - m);
    l64 += w;
    if ((j & 63) == 63) l += l64, l64 = 0.f;
    paged_row<kF8>(v_cache, at, x);
#pragma unroll
    for (int d = 0; d < kHeadDim; ++d) o[d] = fmaf(w, x[d], o[d]);
  }
  l += l64;
  const float f = l > 0.f ? (kF8 ? __ldg(p.v_scale + g) : 1.f) / l : 0.f;
  __nv_bfloat16* dst = p.out + (static_cast<long long>(t) * p.Hq + h) * kHeadDim;
#pragma unroll
  for (int d = 0; d < kHeadDim; ++d) dst[d] = __float2bfloat16_rn(o[d] * f);
  p.lse[static_cast<long long>(h) * p.T + t] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace sa
