// Paged attention of requests with few query rows (single tokens above all):
// the keys and values of a request cross HBM once, and that is what bounds it.
//
// A request's visible keys are cut into blocks of kKeys keys.  The blocks of
// all requests, in order, are one axis, of which every worker takes an equal
// piece: no share depends on how ragged the lengths are, and the host needs to
// know none of them.  A worker is a group of warps, one for each of up to
// eight key/value heads: the heads of a token lie side by side in most caches,
// so that warps which read the same tokens at about the same time read whole
// DRAM pages (with the heads one after another on the axis instead, the same
// tokens crossed HBM 1.3 times, and 64 x 6-8k took 219 us for 142 us of
// bytes).  The warps of a worker share nothing else: each fetches its blocks
// with TMA into a ring of its own in shared memory, kStages blocks ahead, and
// keeps running maximum, sum and O of its n * G query rows (n new tokens, G
// heads; one or two 16-row MMA tiles) in registers.  The tiles come to the tensor cores through
// mma.sync: with 8 or 16 rows the S and P of a block are a few registers, and
// the trip through tensor memory that the 128-row instructions need costs more
// than the multiplication (the decode kernel over linear caches makes that
// trip once per 128 keys and waits on it).
//   S = Q K^T          16 rows x 8 keys per instruction, keys by ldmatrix
//   P = 2^(S sl2 - m)  m: running maximum of the row
//   O = O 2^(m' - m) + P V
// The accumulators of S hold what the first operand of PV wants, so P never
// leaves the registers.  A request that lies within one worker's piece is
// written out by it; the pieces of a cut one go to the workspace and are joined by
// the combine kernel, which adds the sink once.  The running maximum starts at
// -inf, not at the sink: a sink far above the logits would push every weight
// below the range of fp16.
//
// e4m3: K and V are widened to fp16 (exactly) in registers, between ldmatrix
// and mma.  A 16-bit ldmatrix element is two codes, so a thread gets four
// neighbouring dims of a key where the instruction wants two and two: the dims
// of Q are permuted the same way, which a sum over dims does not see.  For V
// the transposing ldmatrix leaves two dims of two keys in a register; a byte
// permutation pairs the keys, and the dims come out as an even and an odd tile.
// Q and P are rounded to fp16 (Q is exact between 2^-14 and 65504; P <= 1 has
// 11 bits down to 2^-14 and an absolute error of 2^-25 below).
#pragma once
#include "paged_attn.cuh"

namespace sa {

constexpr int kRowsWarps = 8;
constexpr int kRowsThreads = 32 * kRowsWarps;
constexpr int kRowsStages = 3;
constexpr int kRowsTile = 4096;  // bytes of a K or a V block: 32 bf16 keys or 64 e4m3 keys
constexpr int kRowsRing = kRowsStages * 2 * kRowsTile;
constexpr int kRowsMaxRows = 32;
// A cut closer than this many blocks to a request's end moves there: joining a
// piece costs more than reading so few keys.
template <bool kF8>
constexpr int kRowsSnap = kF8 ? 1 : 2;
template <bool kF8>
constexpr int kRowsKeys = kF8 ? 64 : 32;

struct RowsCtl {
  uint64_t full[kRowsWarps][kRowsStages];
  int abort;
  int sums[kRowsWarps];
};

constexpr size_t rows_smem_bytes(int batch) {
  return 1024 + kRowsWarps * kRowsRing + sizeof(RowsCtl) + (static_cast<size_t>(batch) + 1) * sizeof(int);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool kF16>
__device__ __forceinline__ void mma_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (kF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// First key (a multiple of the TMA box) and number of blocks of a request's units.
template <bool kF8>
__device__ __forceinline__ int rows_first(const PagedParams& p, const PagedRequest& r) {
  return r.lo >> p.box_log2 << p.box_log2;
}
template <bool kF8>
__device__ __forceinline__ int rows_blocks(const PagedParams& p, const PagedRequest& r) {
  if (r.n == 0 || r.n > p.few) return 0;
  return max(1, (r.len - rows_first<kF8>(p, r) + kRowsKeys<kF8> - 1) / kRowsKeys<kF8>);
}

// The axis of all blocks: request by request, and within it chunk by chunk of
// its key/value heads (one chunk when there are at most kRowsWarps heads).
struct RowsAxis {
  const int* pre;  // blocks before request b (of one chunk), [batch + 1]
  int batch, chunks;
  long long total;
  int workers;

  __device__ __forceinline__ int find(long long x) const {  // the request of block x < total
    const int q = static_cast<int>(x / chunks);
    int lo = 0, hi = batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= q) lo = mid; else hi = mid - 1;
    }
    return lo;
  }
  // Where worker w's piece begins.
  template <int kSnap>
  __device__ __forceinline__ long long cut(int w) const {
    const long long x = w * total / workers;
    if (w >= workers || x >= total) return total;
    const int b = find(x);
    const int blocks = pre[b + 1] - pre[b];
    const int off = static_cast<int>((x - static_cast<long long>(pre[b]) * chunks) % blocks);
    if (off <= kSnap) return x - off;
    return blocks - off <= kSnap ? x + blocks - off : x;
  }
};

template <bool kF8, int kR>
__global__ void __launch_bounds__(kRowsThreads, 1)
    sink_attn_paged_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                                const __grid_constant__ PagedParams p) {
  constexpr int kKeys = kRowsKeys<kF8>;
  constexpr int kRow = kF8 ? 64 : 128;         // bytes of a key row in shared memory
  constexpr int kMT = kR == 32 ? 2 : 1;        // 16-row MMA tiles
  constexpr int kHalves = kR == 8 ? 1 : 2;     // 8-row halves of a tile that hold rows
  constexpr int kSnap = kRowsSnap<kF8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  RowsCtl* ctl = reinterpret_cast<RowsCtl*>(smem + kRowsWarps * kRowsRing);
  int* pre = reinterpret_cast<int*>(ctl + 1);
  volatile int* abort = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();  // the combine kernel waits for this one's end by itself

  if (threadIdx.x == 0) {
    for (int w = 0; w < kRowsWarps; ++w)
      for (int s = 0; s < kRowsStages; ++s) mbar_init(&ctl->full[w][s], 1);
    ctl->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // pre[]: every CTA sums the requests' blocks for itself.
  {
    const int per = (p.batch + kRowsThreads - 1) / kRowsThreads;
    const int b0 = threadIdx.x * per;
    int sum = 0;
    for (int i = 0; i < per; ++i) {
      const int b = b0 + i;
      if (b >= p.batch) break;
      if (blockIdx.x == 0) paged_check(p, b);
      const int n = rows_blocks<kF8>(p, paged_request(p, b));
      pre[b + 1] = n;
      sum += n;
    }
    int in = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += v;
    }
    if (lane == 31) ctl->sums[warp] = in;
    __syncthreads();
    int at = in - sum;
    for (int w = 0; w < warp; ++w) at += ctl->sums[w];
    for (int i = 0; i < per; ++i) {
      const int b = b0 + i;
      if (b >= p.batch) break;
      at += pre[b + 1];
      pre[b + 1] = at;
    }
    if (threadIdx.x == 0) pre[0] = 0;
    __syncthreads();
  }

  RowsAxis axis;
  axis.pre = pre;
  axis.batch = p.batch;
  axis.chunks = p.chunks;
  axis.total = static_cast<long long>(pre[p.batch]) * p.chunks;
  const int per_cta = kRowsWarps / p.per_chunk;  // workers
  axis.workers = static_cast<int>(min(static_cast<long long>(gridDim.x) * per_cta, axis.total));
  const int hw = warp % p.per_chunk;  // this warp's head within its chunk
  if (warp >= per_cta * p.per_chunk) return;
  const int worker = blockIdx.x * per_cta + warp / p.per_chunk;
  const bool reports = p.part_unit && hw == 0 && lane == 0;
  int4 unit = make_int4(-1, 0, 0, 0);  // the cut request (and chunk) that this worker completes
  const long long x0 = worker < axis.workers ? axis.cut<kSnap>(worker) : 0;
  const int count = worker < axis.workers ? static_cast<int>(axis.cut<kSnap>(worker + 1) - x0) : 0;
  if (count == 0) {
    if (reports) p.part_unit[worker] = unit;
    return;
  }

  // The request and chunk of the block that is computed next.
  int b = axis.find(x0);
  int blocks = pre[b + 1] - pre[b];
  int c = static_cast<int>((x0 - static_cast<long long>(pre[b]) * p.chunks) / blocks);
  int off = static_cast<int>((x0 - static_cast<long long>(pre[b]) * p.chunks) % blocks);
  PagedRequest rq = paged_request(p, b);
  int first = rows_first<kF8>(p, rq);

  // The same of the block that is fetched next; its pages are looked up one
  // block ahead of the copy.  (The last chunk may have fewer heads: a warp
  // without one reads the last head and writes nothing.)
  auto head_of = [&](int chunk) { return min(chunk * p.per_chunk + hw, p.Hkv - 1); };
  int fb = b, fc = c, foff = off, fblocks = blocks, flen = rq.len, ffirst = first, fetched = 0;
  uint8_t* ring = smem + warp * kRowsRing;
  uint64_t* full = ctl->full[warp];
  const int nbox = kKeys >> p.box_log2;
  const int page_mask = (1 << p.page_log2) - 1;
  int next_page = 0, next_at = 0, next_g = 0;
  bool next_want = false;
  auto lookup = [&]() {
    const int j = ffirst + foff * kKeys + (lane << p.box_log2);
    // Looked at by fetch(), so that the load is not waited for here.
    next_want = lane < nbox && j < flen;
    if (next_want) next_page = paged_entry(p, fb, j);
    next_at = j & page_mask;
    next_g = head_of(fc);
    if (++foff == fblocks) {
      foff = 0;
      if (++fc == p.chunks) {
        fc = 0;
        if (fetched + 1 < count) {
          do ++fb; while (pre[fb + 1] == pre[fb]);
          fblocks = pre[fb + 1] - pre[fb];
          const PagedRequest r = paged_request(p, fb);
          flen = r.len;
          ffirst = rows_first<kF8>(p, r);
        }
      }
    }
    ++fetched;
  };
  auto fetch = [&](int s) {  // the block looked up last, into stage s
    if (lane == 0) mbar_arrive_expect_tx(&full[s], 2 * kRowsTile);
    __syncwarp();
    if (lane < nbox) {
      uint8_t* dst = ring + s * 2 * kRowsTile + (lane << p.box_log2) * kRow;
      const int page = next_want ? paged_page(p, next_page) : p.num_pages;
      tma_load_4d(dst, &tm_k, &full[s], 0, next_g, next_at, page);
      tma_load_4d(dst + kRowsTile, &tm_v, &full[s], 0, next_g, next_at, page);
    }
    if (fetched < count) lookup();
  };
  lookup();
  for (int s = 0; s < kRowsStages && s < count; ++s) fetch(s);

  const int t4 = lane & 3, r8 = lane >> 2;
  uint32_t q[kMT][4][4];
  float o[kMT][8][4], m[kMT][2], l[kMT][2];
  int key_lo[kMT][2], key_hi[kMT][2];  // keys that this thread's rows see
  bool seg_begin = true, whole = false, real = true;
  int g = 0;
  float sl2 = 0.f;
  bool ok = true;
  int done = 0;

  for (int i = 0; i < count; ++i) {
    if (seg_begin) {
      seg_begin = false;
      whole = off == 0;
      g = head_of(c);
      real = c * p.per_chunk + hw < p.Hkv;
      sl2 = kF8 ? p.scale_log2 * __ldg(p.k_scale + g) : p.scale_log2;
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          m[mt][h] = -INFINITY;
          l[mt][h] = 0.f;
          const int row = 16 * mt + 8 * h + r8;
          const int t = row / p.G;
          key_hi[mt][h] = t < rq.n ? rq.len - rq.n + t : -1;
          key_lo[mt][h] = p.window > 0 ? key_hi[mt][h] - p.window + 1 : 0;
          const __nv_bfloat16* src =
              p.q + static_cast<long long>(rq.t0 + t) * p.q_stride + (g * p.G + row - t * p.G) * kHeadDim;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            uint32_t a = 0u, c = 0u;
            if (h < kHalves && t < rq.n) {
              if constexpr (kF8) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(src + 16 * kk + 4 * t4));
                a = bf16x2_to_f16x2_sat(v.x);
                c = bf16x2_to_f16x2_sat(v.y);
              } else {
                a = __ldg(reinterpret_cast<const uint32_t*>(src + 16 * kk + 2 * t4));
                c = __ldg(reinterpret_cast<const uint32_t*>(src + 16 * kk + 8 + 2 * t4));
              }
            }
            q[mt][kk][h] = a;
            q[mt][kk][2 + h] = c;
          }
        }
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
          for (int u = 0; u < 4; ++u) o[mt][n][u] = 0.f;
      }
    }
    const int s = i % kRowsStages;
    done = i;
    ok = warp_all(mbar_wait(&full[s], (i / kRowsStages) & 1, abort, &g_device_error, kDevErrTimeoutDecode));
    if (!ok) break;
    uint8_t* tile = ring + s * 2 * kRowsTile;
    const int base = first + off * kKeys;
    // Keys in front of the first visible one or behind the last: their slots
    // may hold any bits.  S is masked below; the values become zeros, since
    // 0 * NaN is not 0.
    const bool edge = base < rq.lo || base + kKeys > rq.len;
    if (edge) {
#pragma unroll
      for (int r = lane; r < kKeys; r += 32) {
        if (base + r < rq.lo || base + r >= rq.len) {
#pragma unroll
          for (int c = 0; c < kRow / 16; ++c)
            *reinterpret_cast<uint4*>(tile + kRowsTile + r * kRow + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();  // before the copy that reuses the stage
      __syncwarp();
    }
    // Any key of this block that some row does not see?
    const bool masked = base + kKeys - 1 > rq.len - rq.n || (p.window > 0 && base < rq.len - p.window);
    const uint32_t sk = smem_u32(tile), sv = sk + kRowsTile;

#pragma unroll
    for (int part = 0; part < kKeys / 32; ++part) {  // 32 keys at a time
      float x[kMT][4][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int u = 0; u < 4; ++u) x[mt][nt][u] = 0.f;
        const int r = 32 * part + 8 * nt + (lane & 7), ch = lane >> 3;
        if constexpr (kF8) {
          uint32_t k[4];
          ldsm4(sk + r * kRow + ((ch ^ ((r >> 1) & 3)) << 4), k);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
              mma_16816<true>(x[mt][nt], q[mt][kk], e4m3x2_to_f16x2(k[kk]), e4m3x2_to_f16x2(k[kk] >> 16));
        } else {
          uint32_t k[8];
          ldsm4(sk + r * kRow + ((ch ^ (r & 7)) << 4), k);
          ldsm4(sk + r * kRow + (((ch + 4) ^ (r & 7)) << 4), k + 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) mma_16816<false>(x[mt][nt], q[mt][kk], k[2 * kk], k[2 * kk + 1]);
        }
      }
      if (masked) {
        const int j0 = base + 32 * part + 2 * t4;
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int u = 0; u < 2 * kHalves; ++u) {
              const int j = j0 + 8 * nt + (u & 1);
              if (j < key_lo[mt][u >> 1] || j > key_hi[mt][u >> 1]) x[mt][nt][u] = -INFINITY;
            }
      }
      uint32_t pk[kMT][4][2];
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h >= kHalves) {
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) pk[mt][nt][h] = 0u;
            continue;
          }
          float top = -INFINITY;
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) top = fmax3(top, x[mt][nt][2 * h], x[mt][nt][2 * h + 1]);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2)) * sl2;
          const float old = m[mt][h];
          if (__any_sync(0xffffffffu, top > old)) {
            const float now = fmaxf(old, top);
            const float f = now == -INFINITY ? 1.f : ex2_approx(old - now);
            m[mt][h] = now;
            l[mt][h] *= f;
#pragma unroll
            for (int n = 0; n < 8; ++n) o[mt][n][2 * h] *= f, o[mt][n][2 * h + 1] *= f;
          }
          const float ref = m[mt][h] == -INFINITY ? 0.f : m[mt][h];
          float sum = 0.f;
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            const float e0 = ex2_approx(fmaf(x[mt][nt][2 * h], sl2, -ref));
            const float e1 = ex2_approx(fmaf(x[mt][nt][2 * h + 1], sl2, -ref));
            sum += e0 + e1;
            pk[mt][nt][h] = kF8 ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1);
          }
          l[mt][h] += sum;
        }
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {  // 16 keys
        const int r = 32 * part + 16 * ks + (lane & 7) + (lane & 8), ch = lane >> 4;
#pragma unroll
        for (int j = 0; j < (kF8 ? 2 : 4); ++j) {
          uint32_t v[4];
          if constexpr (kF8) {
            ldsm4_t(sv + r * kRow + (((2 * j + ch) ^ ((r >> 1) & 3)) << 4), v);
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = __byte_perm(v[u], 0u, 0x3120);
          } else {
            ldsm4_t(sv + r * kRow + (((2 * j + ch) ^ (r & 7)) << 4), v);
          }
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) {
            const uint32_t a[4] = {pk[mt][2 * ks][0], pk[mt][2 * ks][1], pk[mt][2 * ks + 1][0], pk[mt][2 * ks + 1][1]};
            if constexpr (kF8) {
#pragma unroll
              for (int u = 0; u < 2; ++u) {  // 16 dims: the even ones, the odd ones
                mma_16816<true>(o[mt][2 * (2 * j + u)], a, e4m3x2_to_f16x2(v[2 * u]), e4m3x2_to_f16x2(v[2 * u + 1]));
                mma_16816<true>(o[mt][2 * (2 * j + u) + 1], a, e4m3x2_to_f16x2(v[2 * u] >> 16),
                                e4m3x2_to_f16x2(v[2 * u + 1] >> 16));
              }
            } else {
              mma_16816<false>(o[mt][2 * j], a, v[0], v[1]);
              mma_16816<false>(o[mt][2 * j + 1], a, v[2], v[3]);
            }
          }
        }
      }
    }
    __syncwarp();  // every lane has read the stage
    if (i + kRowsStages < count) fetch(s);

    const bool unit_end = off + 1 == blocks;
    if (unit_end || i + 1 == count) {
      // ------------------------------------------- end of this piece of the request
      whole = whole && unit_end;
      const int slot = (2 * worker + (unit_end ? 0 : 1)) * p.per_chunk + hw;
      const float vs = kF8 ? __ldg(p.v_scale + g) : 1.f;
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          const int row = 16 * mt + 8 * h + r8;
          float sum = l[mt][h];
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          const int t = row / p.G;
          const bool valid = t < rq.n && real;
          const int head = valid ? g * p.G + row - t * p.G : 0;
          float f = vs;
          if (whole) {
            const float s2 = __ldg(p.sinks + head) * kLog2e;
            const float top = fmaxf(s2, m[mt][h]);
            float all = 0.f;
            f = 0.f;
            if (top != -INFINITY) {
              f = ex2_approx(m[mt][h] - top);
              all = fmaf(sum, f, s2 == top ? 1.f : ex2_approx(s2 - top));
              f = all > 0.f ? vs * f / all : 0.f;
            }
            if (valid && t4 == 0)
              p.lse[static_cast<long long>(head) * p.T + rq.t0 + t] = all > 0.f ? (top + __log2f(all)) * kLn2 : -INFINITY;
          } else if (valid && t4 == 0) {
            p.part_ml[slot * kR + row] = make_float2(m[mt][h], sum);
          }
          if (!valid) continue;
          __nv_bfloat16* dst = p.out + (static_cast<long long>(rq.t0 + t) * p.Hq + head) * kHeadDim;
          float* part = p.part_o + (static_cast<long long>(slot) * kR + row) * kHeadDim;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // 16 dims: two MMA tiles, side by side (bf16) or even and odd dims (e4m3).
            const float y0 = o[mt][2 * e][2 * h] * f, y1 = o[mt][2 * e][2 * h + 1] * f;
            const float z0 = o[mt][2 * e + 1][2 * h] * f, z1 = o[mt][2 * e + 1][2 * h + 1] * f;
            if constexpr (kF8) {
              const int d = 16 * e + 4 * t4;
              if (whole) *reinterpret_cast<uint2*>(dst + d) = make_uint2(pack_bf16x2(y0, z0), pack_bf16x2(y1, z1));
              else *reinterpret_cast<float4*>(part + d) = make_float4(y0, z0, y1, z1);
            } else {
              const int d = 16 * e + 2 * t4;
              if (whole) {
                *reinterpret_cast<uint32_t*>(dst + d) = pack_bf16x2(y0, y1);
                *reinterpret_cast<uint32_t*>(dst + d + 8) = pack_bf16x2(z0, z1);
              } else {
                *reinterpret_cast<float2*>(part + d) = make_float2(y0, y1);
                *reinterpret_cast<float2*>(part + d + 8) = make_float2(z0, z1);
              }
            }
          }
        }
      }
      if (unit_end && !whole) {
        // The last piece of a cut request: the first one belongs to the last
        // worker whose piece begins at or before the request's first block.
        const long long begin = static_cast<long long>(pre[b]) * p.chunks + static_cast<long long>(c) * blocks;
        int w0 = min(static_cast<int>(begin * axis.workers / axis.total), worker - 1);
        while (w0 > 0 && axis.cut<kSnap>(w0) > begin) --w0;
        while (axis.cut<kSnap>(w0 + 1) <= begin) ++w0;
        unit = make_int4(b, c, w0, 0);
      }
      seg_begin = true;
    }
    if (unit_end) {
      off = 0;
      if (++c == p.chunks) {
        c = 0;
        if (i + 1 < count) {
          do ++b; while (pre[b + 1] == pre[b]);
          blocks = pre[b + 1] - pre[b];
          rq = paged_request(p, b);
          first = rows_first<kF8>(p, rq);
        }
      }
    } else {
      ++off;
    }
  }
  if (!ok) {
    unit.x = -1;
    // The copies in flight still write to this CTA's shared memory.
    for (int i = done; i < min(count, done + kRowsStages); ++i) {
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(&full[i % kRowsStages], (i / kRowsStages) & 1) && global_timer_ns() - t0 < kWaitLimitNs) {
      }
    }
  }
  if (reports) p.part_unit[worker] = unit;
}

// Joins the pieces of every cut request and adds the sink: with M = max(s, max_k m_k),
//   l = e^{s-M} + sum_k l_k e^{m_k-M},  out = sum_k O_k e^{m_k-M} / l,  lse = M + ln l.
// One CTA per worker and head of a chunk, whose work is the request that the
// worker completed (mostly none); one warp per query row, half a warp per piece.
template <int kR>
__global__ void __launch_bounds__(256) sink_attn_paged_join_kernel(const __grid_constant__ PagedParams p) {
  pdl_wait();
  const int last = blockIdx.x, hw = blockIdx.y;
  const int4 unit = __ldcg(p.part_unit + last);
  const int g = unit.y * p.per_chunk + hw;
  if (unit.x < 0 || g >= p.Hkv) return;
  const int pieces = last - unit.z + 1;
  const PagedRequest rq = paged_request(p, unit.x);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto slot = [&](int k) { return (k + 1 == pieces ? 2 * last : 2 * (unit.z + k) + 1) * p.per_chunk + hw; };
  for (int row = warp; row < rq.n * p.G; row += 8) {
    const int t = row / p.G;
    const int head = g * p.G + row - t * p.G;
    const float s2 = __ldg(p.sinks + head) * kLog2e;
    float top = s2;
    for (int k = lane; k < pieces; k += 32) top = fmaxf(top, __ldcg(p.part_ml + slot(k) * kR + row).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top == -INFINITY ? 0.f : top;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    for (int k0 = 0; k0 < pieces; k0 += 32) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (k0 + lane < pieces) ml = __ldcg(p.part_ml + slot(k0 + lane) * kR + row);
      const float f = ex2_approx(ml.x - ref);
      l = fmaf(ml.y, f, l);
      // Four pieces of each half warp at a time, their loads in flight together.
      for (int k = 0; k < 32 && k0 + k < pieces; k += 8) {
        float4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int mine = k0 + k + 2 * u + (lane >> 4);
          v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (mine < pieces)
            v[u] = __ldcg(reinterpret_cast<const float4*>(p.part_o + (static_cast<long long>(slot(mine)) * kR + row) * kHeadDim) +
                          (lane & 15));
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float fk = __shfl_sync(0xffffffffu, f, k + 2 * u + (lane >> 4));
          y.x = fmaf(v[u].x, fk, y.x);
          y.y = fmaf(v[u].y, fk, y.y);
          y.z = fmaf(v[u].z, fk, y.z);
          y.w = fmaf(v[u].w, fk, y.w);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    y.x += __shfl_xor_sync(0xffffffffu, y.x, 16);
    y.y += __shfl_xor_sync(0xffffffffu, y.y, 16);
    y.z += __shfl_xor_sync(0xffffffffu, y.z, 16);
    y.w += __shfl_xor_sync(0xffffffffu, y.w, 16);
    l += s2 == ref ? 1.f : ex2_approx(s2 - ref);
    const float f = l > 0.f ? 1.f / l : 0.f;
    if (lane < 16)
      *reinterpret_cast<uint2*>(p.out + (static_cast<long long>(rq.t0 + t) * p.Hq + head) * kHeadDim + 4 * lane) =
          make_uint2(pack_bf16x2(y.x * f, y.y * f), pack_bf16x2(y.z * f, y.w * f));
    if (lane == 0)
      p.lse[static_cast<long long>(head) * p.T + rq.t0 + t] = l > 0.f ? (ref + __log2f(l)) * kLn2 : -INFINITY;
  }
}

}  // namespace sa
