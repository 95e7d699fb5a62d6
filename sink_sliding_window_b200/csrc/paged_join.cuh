// Joins what the few-rows kernel and the chunk kernel cut along the keys: one
// launch for both, since a step of chunks and single tokens needs both and a
// launch costs as much as the work.
#pragma once
#include "paged_chunk.cuh"
#include "paged_cut.cuh"
#include "paged_rows.cuh"

namespace sa {

struct RowsJoinSmem {
  float o[8][8][kHeadDim];
  float m[8][8], l[8][8];
};

// The pieces of a cut request of the few-rows kernel, and the sink: with
// M = max(s, max_k m_k),
//   l = e^{s-M} + sum_k l_k e^{m_k-M},  out = sum_k O_k e^{m_k-M} / l,  lse = M + ln l.
// The work of one CTA is the request that worker `last` completed (mostly
// none), for one warp of that worker.  Its warps take the pieces in turn, eight
// rows at a time (a lane holds four rows' four dims), then join their own
// eight results in shared memory in the same way.
template <int kR>
__device__ __forceinline__ void rows_join(const PagedParams& p, RowsJoinSmem& sm, int last, int in_group) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The first piece is that of the nearest worker before this one whose last
  // piece begins a request: one load per lane tells for 31 of them.
  const int per_group = p.per_chunk * p.row_parts;
  const int hw = in_group / p.row_parts, row0 = 16 * (in_group - hw * p.row_parts);
  const int4 near = __ldcg(p.part_unit + max(last - lane, 0));
  const int b = __shfl_sync(0xffffffffu, near.x, 0), g = __shfl_sync(0xffffffffu, near.y, 0) * p.per_chunk + hw;
  if (b < 0 || g >= p.Hkv) return;
  const PagedRequest rq = paged_request(p, b);
  uint32_t begins = __ballot_sync(0xffffffffu, lane > 0 && lane <= last && near.z != 0);
  int start = begins ? last - (__ffs(begins) - 1) : max(0, last - 31);
  while (begins == 0 && start > 0) {
    const int w = start - 1 - lane;
    begins = __ballot_sync(0xffffffffu, w >= 0 && __ldcg(&p.part_unit[max(w, 0)].z) != 0);
    start = begins ? start - __ffs(begins) : max(0, start - 32);
  }
  const int pieces = last - start + 1;
  auto slot = [&](int k) { return (k + 1 == pieces ? 2 * last : 2 * (start + k) + 1) * per_group + in_group; };
  // (The first loads wait for neither the request's lengths nor the sinks; a
  // unit has a row at least.)
  int r0 = 0;
  do {
    const int row = row0 + r0 + warp, t = row / p.G;  // this warp's row in the end
    const int head = g * p.G + row - t * p.G;
    const float s2 = *(p.sinks + min(head, p.Hq - 1)) * kLog2e;
    // This lane's rows r0 + (lane >> 4) + 2 u, u < 4, and dims 4 (lane & 15) ..; a
    // piece's rows behind the last one are in the workspace, and never used.
    float m[4], l[4];
    float4 y[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) m[u] = -INFINITY, l[u] = 0.f, y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAtOnce = 2;
    for (int k0 = warp; k0 < pieces; k0 += 8 * kAtOnce) {
      float4 v[kAtOnce][4];
      float2 ml[kAtOnce][4];
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) {
        const int k = k0 + 8 * a;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          ml[a][u] = make_float2(-INFINITY, 0.f);
          if (k < pieces) {
            const long long at = static_cast<long long>(slot(k)) * kR + r0 + (lane >> 4) + 2 * u;
            ml[a][u] = __ldcg(p.part_ml + at);
            v[a][u] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * kHeadDim) + (lane & 15));
          } else {
            v[a][u] = make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float now = m[u];
#pragma unroll
        for (int a = 0; a < kAtOnce; ++a) now = fmaxf(now, ml[a][u].x);
        const float ref = now == -INFINITY ? 0.f : now;
        const float f0 = ex2_approx(m[u] - ref);
        m[u] = now;
        l[u] *= f0;
        y[u] = make_float4(y[u].x * f0, y[u].y * f0, y[u].z * f0, y[u].w * f0);
#pragma unroll
        for (int a = 0; a < kAtOnce; ++a) {
          const float f = ex2_approx(ml[a][u].x - ref);
          l[u] = fmaf(ml[a][u].y, f, l[u]);
          y[u].x = fmaf(v[a][u].x, f, y[u].x);
          y[u].y = fmaf(v[a][u].y, f, y[u].y);
          y[u].z = fmaf(v[a][u].z, f, y[u].z);
          y[u].w = fmaf(v[a][u].w, f, y[u].w);
        }
      }
    }
    __syncthreads();  // the last rows have been read
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = (lane >> 4) + 2 * u;
      *reinterpret_cast<float4*>(&sm.o[warp][r][4 * (lane & 15)]) = y[u];
      if ((lane & 15) == 0) sm.m[warp][r] = m[u], sm.l[warp][r] = l[u];
    }
    __syncthreads();
    // One warp per row, two dims per lane.
    if (t < rq.n) {
      float top = s2;
#pragma unroll
      for (int w = 0; w < 8; ++w) top = fmaxf(top, sm.m[w][warp]);
      const float ref = top == -INFINITY ? 0.f : top;
      float all = s2 == ref ? 1.f : ex2_approx(s2 - ref);
      float2 z = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const float f = ex2_approx(sm.m[w][warp] - ref);
        const float2 v = *reinterpret_cast<const float2*>(&sm.o[w][warp][2 * lane]);
        all = fmaf(sm.l[w][warp], f, all);
        z.x = fmaf(v.x, f, z.x);
        z.y = fmaf(v.y, f, z.y);
      }
      const float f = all > 0.f ? 1.f / all : 0.f;
      reinterpret_cast<uint32_t*>(p.out + (static_cast<long long>(rq.t0 + t) * p.Hq + head) * kHeadDim)[lane] =
          pack_bf16x2(z.x * f, z.y * f);
      if (lane == 0)
        p.lse[static_cast<long long>(head) * p.T + rq.t0 + t] = all > 0.f ? (ref + __log2f(all)) * kLn2 : -INFINITY;
    }
    r0 += 8;
  } while (r0 < min(kR, rq.n * p.G - row0));
}

// The parts of the chunk kernel's i-th cut unit, and the sink, for 32 of its
// rows: half a warp per row, four dims per lane.
__device__ __forceinline__ void chunk_join(const ChunkParams& p, int i, int rows32) {
  const int2 cut = __ldcg(p.part_units);
  if (i >= cut.x) return;
  const int4 u = __ldcg(p.part_unit + i);
  PagedRequest rq;
  if (!cut_unit_fits(u.x, u.y, u.z, u.w, p.a.batch, p.a.Hkv, cut.y, p.tiles * p.tokens, [&](int b) {
        rq = paged_request(p.a, b);
        return rq.n > p.a.few ? rq.n : 0;
      }))
    return;
  const int d = threadIdx.x & 15;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int row = rows32 * 32 + x * 16 + (threadIdx.x >> 4);
    const int r = row & (kBlockM - 1), row_t = r / p.a.G;
    const int it = (p.tiles * u.y + (row >> 7)) * p.tokens + row_t;
    if (row_t >= p.tokens || it >= rq.n) continue;
    const int h = u.z * p.a.G + r - row_t * p.a.G;
    const float s2 = *(p.a.sinks + h) * kLog2e;
    float m = -INFINITY, l = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAtOnce = 6;  // parts whose loads are in flight together
    for (int k0 = 0; k0 < u.w; k0 += kAtOnce) {
      float2 ml[kAtOnce];
      float4 v[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        if (k0 + k < u.w) {
          const long long at = (static_cast<long long>(i) * u.w + k0 + k) * p.tiles * kBlockM + row;
          ml[k] = __ldcg(p.part_ml + at);
          v[k] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * kHeadDim) + d);
        }
      }
      float now = m;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) now = fmaxf(now, ml[k].x);
      if (now == -INFINITY) continue;
      const float f0 = ex2_approx(m - now);
      m = now;
      l *= f0;
      y = make_float4(y.x * f0, y.y * f0, y.z * f0, y.w * f0);
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        // (A part of no keys has written no O.)
        if (ml[k].x == -INFINITY) continue;
        const float f = ex2_approx(ml[k].x - now);
        l = fmaf(ml[k].y, f, l);
        y.x = fmaf(v[k].x, f, y.x);
        y.y = fmaf(v[k].y, f, y.y);
        y.z = fmaf(v[k].z, f, y.z);
        y.w = fmaf(v[k].w, f, y.w);
      }
    }
    const float top = fmaxf(m, s2);
    float f = 0.f, all = 0.f;
    if (top != -INFINITY) {
      f = ex2_approx(m - top);
      all = fmaf(l, f, s2 == top ? 1.f : ex2_approx(s2 - top));
    }
    f = all > 0.f ? f / all : 0.f;
    const int t = rq.t0 + it;
    *reinterpret_cast<uint2*>(p.a.out + (static_cast<long long>(t) * p.a.Hq + h) * kHeadDim + 4 * d) =
        make_uint2(pack_bf16x2(y.x * f, y.y * f), pack_bf16x2(y.z * f, y.w * f));
    if (d == 0) p.a.lse[static_cast<long long>(h) * p.a.T + t] = all > 0.f ? (top + __log2f(all)) * kLn2 : -INFINITY;
  }
}

// A CTA per worker (x) and warp of a worker (y) of the few-rows kernel.
template <int kR>
__global__ void __launch_bounds__(256, kR == 8 ? 3 : 2) sink_attn_paged_join_kernel(const __grid_constant__ PagedParams p) {
  __shared__ RowsJoinSmem sm;
  pdl_launch_dependents();
  pdl_wait();
  rows_join<kR>(p, sm, blockIdx.x, blockIdx.y);
}

// CTAs 0 .. chunk_ctas - 1 for the chunk kernel's cut units, 32 rows each, and
// behind them the others' as above, `workers` of them (0: none).
template <int kR>
__global__ void __launch_bounds__(256, 2)
    sink_attn_paged_join_both_kernel(const __grid_constant__ ChunkParams p, int chunk_ctas, int workers) {
  __shared__ RowsJoinSmem sm;
  pdl_launch_dependents();
  pdl_wait();
  const int x = static_cast<int>(blockIdx.x) - chunk_ctas;
  if (x < 0) {
    const int blocks = p.tiles * kBlockM / 32;
    chunk_join(p, blockIdx.x / blocks, blockIdx.x % blocks);
  } else {
    rows_join<kR>(p.a, sm, x % workers, x / workers);
  }
}

}  // namespace sa
