// Paged attention of requests with few query rows (single tokens above all):
// the keys and values of a request cross HBM once, and that is what bounds it.
//
// A request's visible keys are cut into blocks of 32 keys
// (e4m3: 64).  The blocks of all
// requests, in order, are one axis, of which every worker takes an equal
// piece: no share depends on how ragged the lengths are, and the host needs to
// know none of them.  A worker is a group of warps, one for each of up to
// eight key/value heads.  One TMA box holds a block's tokens of all the
// worker's heads (dims ordered so that it lands head by head), which reads
// whole rows of DRAM and costs one thread two instructions a block; a warp of
// its own for the copies feeds the CTA's workers in turn, kRowsStages blocks
// ahead, with the page numbers looked up a batch ahead.  (With the heads one
// after another on the axis the same DRAM pages were opened 1.3 times and 64
// requests of 6-8k took 219 us; with every warp fetching its own head's boxes
// the issue took 570 of a block's 1650 cycles, 900 of 2700 for e4m3.)
// A warp keeps running maximum, sum and O of its head's n * G query rows (n
// new tokens, G heads; one 16-row MMA tile) in registers; with more rows two
// to four warps share a head's ring, 16 rows each, and a worker has fewer
// heads (one warp with two tiles spilled, and took 24 us for 16 requests of
// 1000 keys and four tokens; two warps take 16).  Else warps share nothing.
// The tiles come to the tensor cores through
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
// Rounding over a bf16 cache: P to bf16, since the two operands of an MMA have
// one type and V is bf16; half a step is 2^-8 of each weight.  l sums the weights
// before that, and S, m, l and O are fp32.
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

template <bool kF8>
constexpr int kRowsKeys = kF8 ? 64 : 32;  // keys of a block: 4 KB of K, 4 KB of V for each head
constexpr int kRowsStages = 3;   // of the ring when every warp has a head of its own
constexpr int kRowsMaxStages = 4 * kRowsStages;
constexpr int kRowsMaxRows = 64;  // four warps of 16 rows share a head's ring
// A cut closer than this many blocks to a request's end moves there: joining a
// piece costs more than reading so few keys.
template <bool kF8>
constexpr int kRowsSnap = kF8 ? 1 : 2;
// Fewest blocks of a worker: a piece costs its join more than these few blocks
// cost in a row (one request of 4033 keys: 16.1 us with 2, 12.9 with 4, 13.7 with 6).
constexpr int kRowsMinBlocks = 4;
constexpr int kRowsWarps = 8;  // that compute, of the one CTA of an SM
constexpr int kRowsThreads = 32 * (kRowsWarps + 1);  // the last warp copies
constexpr int kRowsTile = 4096;  // bytes of one head's K or V block

struct RowsCtl {
  uint64_t full[kRowsWarps * kRowsMaxStages];   // [worker of the CTA][stage]
  uint64_t empty[kRowsWarps * kRowsMaxStages];
  int abort;
  int sums[kRowsWarps + 1], live[kRowsWarps + 1];
  int4 cuts[kRowsWarps][2];  // where the pieces of the CTA's workers begin and end: x, b, c, off
};

constexpr size_t rows_smem_bytes(int batch) {
  return 1024 + kRowsWarps * kRowsStages * 2 * kRowsTile + sizeof(RowsCtl) +
         (static_cast<size_t>(batch) + 1) * sizeof(int);
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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// First key (a multiple of the TMA box) and number of blocks of a request's units.
__device__ __forceinline__ int rows_first(const PagedParams& p, const PagedRequest& r) {
  return r.lo >> p.box_log2 << p.box_log2;
}
template <bool kF8>
__device__ __forceinline__ int rows_blocks(const PagedParams& p, const PagedRequest& r) {
  if (r.n == 0 || r.n > p.few) return 0;
  return max(1, (r.len - rows_first(p, r) + kRowsKeys<kF8> - 1) / kRowsKeys<kF8>);
}

// A place on the axis of all blocks: block `off` of a request and a chunk of
// its key/value heads.
struct RowsAt {
  uint32_t x;
  int b, c, off;
};

// The axis: request by request, and within it chunk by chunk of its heads (one
// chunk when a CTA's warps are enough for them).  Its functions are called by whole
// warps.
template <int kSnap>
struct RowsAxis {
  const int* pre;  // blocks before request b (of one chunk), [batch + 1]
  int batch, chunks;
  uint32_t total, workers;

  // The last request whose blocks begin at or before q.
  __device__ __forceinline__ int find(int q) const {
    const int lane = lane_id();
    int lo = 0, n = batch;
    while (n > 1) {
      const int step = (n + 31) >> 5;
      const bool le = lane * step < n && pre[lo + lane * step] <= q;
      const int k = (__popc(__ballot_sync(0xffffffffu, le)) - 1) * step;
      lo += k;
      n = min(step, n - k);
    }
    return lo;
  }
  __device__ __forceinline__ int blocks(int b) const { return pre[b + 1] - pre[b]; }
  // Moves on to the next chunk, or the next request that has blocks.
  __device__ __forceinline__ void next_unit(RowsAt& a) const {
    a.off = 0;
    if (++a.c < chunks) return;
    a.c = 0;
    do ++a.b; while (a.b < batch && blocks(a.b) == 0);
  }
  // Where worker w's piece begins.
  __device__ __forceinline__ RowsAt cut(uint32_t w) const {
    RowsAt a = {total, batch, 0, 0};
    if (w >= workers) return a;
    const uint32_t share = total / workers, rest = total - share * workers;
    a.x = w * share + w * rest / workers;
    uint32_t q = a.x;
    if (chunks > 1) q /= chunks;
    a.b = find(static_cast<int>(q));
    const uint32_t n = blocks(a.b);
    const uint32_t in = a.x - static_cast<uint32_t>(pre[a.b]) * chunks;
    a.c = chunks > 1 ? in / n : 0;
    a.off = in - a.c * n;
    if (a.off <= kSnap) {
      a.x -= a.off;
      a.off = 0;
    } else if (static_cast<int>(n) - a.off <= kSnap) {
      a.x += n - a.off;
      next_unit(a);
    }
    return a;
  }
};

// kBeside: the chunk kernel of the same call runs before it on the stream.
template <bool kF8, int kR, bool kBeside>
__global__ void __launch_bounds__(kRowsThreads, 1)
    sink_attn_paged_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                                const __grid_constant__ PagedParams p) {
  constexpr int kWarps = kRowsWarps;
  constexpr int kThreads = kRowsThreads;
  constexpr int kTile = kRowsTile;
  constexpr int kKeys = kRowsKeys<kF8>;
  constexpr int kNT = kKeys / 8;  // 8-key MMA tiles of a block
  constexpr int kRow = kF8 ? 64 : 128;         // bytes of a key row in shared memory
  constexpr int kHalves = kR == 8 ? 1 : 2;     // 8-row halves of the MMA tile that hold rows
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  RowsCtl* ctl = reinterpret_cast<RowsCtl*>(smem + kWarps * kRowsStages * 2 * kTile);
  int* pre = reinterpret_cast<int*>(ctl + 1);
  volatile int* abort = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int per_group = p.per_chunk * p.row_parts;  // warps of a worker
  const int groups = kWarps / per_group;             // workers of this CTA
  const int stages = kRowsStages * p.row_parts;
  if (threadIdx.x == 0) {
    for (int w = 0; w < groups * stages; ++w) {
      mbar_init(&ctl->full[w], 1);
      mbar_init(&ctl->empty[w], per_group);
    }
    ctl->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // The call's inputs and the workspace are free to use; beside the chunk
  // kernel they are already, since that waited before it let this one start.
  // What that wait saw finished lies in L2, and there this kernel reads it
  // (paged_load, and TMA).
  if (!kBeside) pdl_wait();
  pdl_launch_dependents();
  // pre[]: every CTA sums the requests' blocks for itself.
  {
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int b0 = threadIdx.x * per;
    int sum = 0, live = 0;  // blocks, requests that have some
    for (int i = 0; i < per; ++i) {
      const int b = b0 + i;
      if (b >= p.batch) break;
      if (blockIdx.x == 0) paged_check<kBeside>(p, b);
      const int n = rows_blocks<kF8>(p, paged_request<kBeside>(p, b));
      pre[b + 1] = n;
      sum += n;
      live += n > 0;
    }
    int in = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += v;
    }
    live = __reduce_add_sync(0xffffffffu, live);
    if (lane == 31) ctl->sums[warp] = in, ctl->live[warp] = live;
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

  RowsAxis<kRowsSnap<kF8>> axis;
  axis.pre = pre;
  axis.batch = p.batch;
  axis.chunks = p.chunks;
  axis.total = static_cast<uint32_t>(pre[p.batch]) * p.chunks;
  uint32_t units = 0;
  for (int w = 0; w <= kWarps; ++w) units += ctl->live[w];
  // (A worker for each unit at least: short ones are not cut.)
  axis.workers = min(gridDim.x * groups, max(units * p.chunks, (axis.total + kRowsMinBlocks - 1) / kRowsMinBlocks));

  // Worker g of this CTA: consecutive pieces go to different SMs, so that a few
  // of them do not share one.
  auto worker_of = [&](int g) { return blockIdx.x + gridDim.x * g; };
  for (int i = warp; i < 2 * groups; i += kWarps + 1) {
    const RowsAt a = axis.cut(worker_of(i >> 1) + (i & 1));
    if (lane == 0) ctl->cuts[i >> 1][i & 1] = make_int4(static_cast<int>(a.x), a.b, a.c, a.off);
  }
  __syncthreads();
  auto cut_of = [&](int g, int end) {
    const int4 v = ctl->cuts[g][end];
    return RowsAt{static_cast<uint32_t>(v.x), v.y, v.z, v.w};
  };

  const uint32_t group_bytes = p.per_chunk * stages * 2 * kTile, stage_bytes = p.per_chunk * 2 * kTile;
  if (warp == kWarps) {
    // ------------------------------------------------------------------ copies
    if (kBeside) fence_proxy_async_global();
    // Lanes lpg * g .. of the warp keep the state of worker g and, one per
    // box, the page numbers of a batch of its next blocks; the batch after it
    // is looked up while this one is copied.
    const int nbox_log2 = (kF8 ? 6 : 5) - p.box_log2, nbox = 1 << nbox_log2, lpg = 32 / groups;
    const int mine = min(lane / lpg, groups - 1), li = lane - mine * lpg;
    RowsAt at = cut_of(mine, 0);
    const int count = static_cast<int>(cut_of(mine, 1).x - at.x);
    int left = count;
    struct Batch {
      int n, c, key, entry;  // blocks, chunk, first key, this lane's table entry
      bool want;
    };
    auto look_up = [&]() {
      Batch t = {0, 0, 0, 0, false};
      if (left == 0) return t;
      const PagedRequest r = paged_request<kBeside>(p, at.b);
      const int blocks = axis.blocks(at.b);
      t.n = min(min(lpg / nbox, blocks - at.off), left);
      t.c = at.c;
      t.key = rows_first(p, r) + at.off * kKeys;
      const int j = t.key + (li << p.box_log2);
      t.want = li < t.n * nbox && j < r.len;
      if (t.want) t.entry = paged_entry<kBeside>(p, at.b, j);
      left -= t.n;
      at.off += t.n;
      if (at.off == blocks) axis.next_unit(at);
      return t;
    };
    Batch now = look_up(), next = look_up();
    int j = 0, page = now.want ? paged_page(p, now.entry) : p.num_pages;
    const int most = __reduce_max_sync(0xffffffffu, count);
    bool ok = true;
    int s = 0, turn = 0;  // i = turn * stages + s
    for (int i = 0; ok && i < most; ++i) {
      if (j == now.n) {
        now = next;
        page = now.want ? paged_page(p, now.entry) : p.num_pages;
        next = look_up();
        j = 0;
      }
      __syncwarp();
      for (int g = 0; ok && g < groups; ++g) {
        const int src = g * lpg;
        const int jg = __shfl_sync(0xffffffffu, j, src);
        const int key = __shfl_sync(0xffffffffu, now.key, src) + jg * kKeys;
        const int head = __shfl_sync(0xffffffffu, now.c, src) * p.per_chunk;
        int pages[kKeys / 16];
#pragma unroll
        for (int x = 0; x < kKeys / 16; ++x) pages[x] = __shfl_sync(0xffffffffu, page, src + jg * nbox + min(x, nbox - 1));
        if (i >= __shfl_sync(0xffffffffu, count, src)) continue;
        if (turn > 0)
          ok = warp_all(mbar_wait(&ctl->empty[g * stages + s], (turn - 1) & 1, abort, &g_device_error,
                                  kDevErrTimeoutProducer));
        if (ok && elect_one()) {
          uint64_t* full = &ctl->full[g * stages + s];
          uint8_t* dst = smem + g * group_bytes + s * stage_bytes;
          mbar_arrive_expect_tx(full, stage_bytes);
#pragma unroll
          for (int x = 0; x < kKeys / 16; ++x) {
            if (x >= nbox) break;
            const int in_page = (key + (x << p.box_log2)) & ((1 << p.page_log2) - 1);
            uint8_t* to = dst + x * (stage_bytes / 2 >> nbox_log2);
            tma_load_4d(to, &tm_k, full, 0, in_page, head, pages[x]);
            tma_load_4d(to + stage_bytes / 2, &tm_v, full, 0, in_page, head, pages[x]);
          }
        }
        __syncwarp();
      }
      ++j;
      if (++s == stages) s = 0, ++turn;
    }
    // Beside the chunk kernel: this one has not ended before that has, so that
    // whoever waits for this one (the joins, the next call) waits for both.  One
    // CTA sees to it; the others make room.
    if (blockIdx.x == 0) pdl_wait();
    return;
  }

  // ----------------------------------------------------------------- attention
  if (warp >= groups * per_group) return;
  const int group = warp / per_group, in_group = warp - group * per_group;  // worker of the CTA, warp of the worker
  const int hw = in_group / p.row_parts, row0 = 16 * (in_group - hw * p.row_parts);  // head of the chunk, first row
  const int worker = worker_of(group);
  const bool reports = p.part_unit && in_group == 0 && lane == 0;
  int4 unit = make_int4(-1, 0, 0, 0);  // see PagedParams::part_unit
  RowsAt at = cut_of(group, 0);
  const int count = static_cast<int>(cut_of(group, 1).x - at.x);
  if (count == 0) {
    if (reports) p.part_unit[worker] = unit;
    return;
  }
  PagedRequest rq = paged_request<kBeside>(p, at.b);
  int first = rows_first(p, rq), blocks = axis.blocks(at.b);
  const uint8_t* ring = smem + group * group_bytes;
  uint64_t *full = ctl->full + group * stages, *empty = ctl->empty + group * stages;
  // Keys of this warp's head within a box, and the bytes from one box to the next.
  const int box = 1 << p.box_log2, box_bytes = p.per_chunk * box * kRow;
  const int head_bytes = hw * box * kRow;

  const int t4 = lane & 3, r8 = lane >> 2;
  uint32_t q[4][4];
  float o[8][4], m[2], l[2];
  int key_lo[2], key_hi[2];  // keys that this thread's rows see
  bool seg_begin = true, whole = false;
  // The last chunk may have fewer heads: a warp without one computes on zeros
  // and writes nothing.
  bool real = true;
  int g = 0;
  float sl2 = 0.f;
  bool ok = true;
  int done = 0, s = 0, turn = 0;

  for (int i = 0; i < count; ++i) {
    if (seg_begin) {
      seg_begin = false;
      whole = at.off == 0;
      g = min(at.c * p.per_chunk + hw, p.Hkv - 1);
      real = at.c * p.per_chunk + hw < p.Hkv;
      sl2 = kF8 ? p.scale_log2 * paged_load<kBeside>(p.k_scale + g) : p.scale_log2;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
        const int row = row0 + 8 * h + r8;
        const int t = row / p.G;
        key_hi[h] = t < rq.n ? rq.len - rq.n + t : -1;
        key_lo[h] = p.window > 0 ? key_hi[h] - p.window + 1 : 0;
        const __nv_bfloat16* src =
            p.q + static_cast<long long>(rq.t0 + t) * p.q_stride + (g * p.G + row - t * p.G) * kHeadDim;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          uint32_t a = 0u, c = 0u;
          if (h < kHalves && t < rq.n) {
            if constexpr (kF8) {
              const uint2 v = paged_load<kBeside>(reinterpret_cast<const uint2*>(src + 16 * kk + 4 * t4));
              a = bf16x2_to_f16x2_sat(v.x);
              c = bf16x2_to_f16x2_sat(v.y);
            } else {
              a = paged_load<kBeside>(reinterpret_cast<const uint32_t*>(src + 16 * kk + 2 * t4));
              c = paged_load<kBeside>(reinterpret_cast<const uint32_t*>(src + 16 * kk + 8 + 2 * t4));
            }
          }
          q[kk][h] = a;
          q[kk][2 + h] = c;
        }
      }
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int u = 0; u < 4; ++u) o[n][u] = 0.f;
    }
    done = i;
    ok = warp_all(mbar_wait(&full[s], turn & 1, abort, &g_device_error, kDevErrTimeoutDecode));
    if (!ok) break;
    const uint8_t* tile = ring + s * stage_bytes;
    const int base = first + at.off * kKeys;
    // Keys in front of the first visible one or behind the last: their slots
    // may hold any bits.  S is masked below; the values become zeros, since
    // 0 * NaN is not 0.
    const bool edge = base < rq.lo || base + kKeys > rq.len;
    if (edge) {
#pragma unroll
      for (int r = lane; r < kKeys; r += 32) {
        if (base + r < rq.lo || base + r >= rq.len) {
          uint8_t* row = const_cast<uint8_t*>(tile) + stage_bytes / 2 + (r >> p.box_log2) * box_bytes + head_bytes +
                         (r & (box - 1)) * kRow;
#pragma unroll
          for (int ch = 0; ch < kRow / 16; ++ch) *reinterpret_cast<uint4*>(row + 16 * ch) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      __syncwarp();
    }
    // Any key of this block that some row does not see?
    const bool masked = base + kKeys - 1 > rq.len - rq.n || (p.window > 0 && base < rq.len - p.window);
    const uint32_t sk = smem_u32(tile) + head_bytes, sv = sk + stage_bytes / 2;
    // Where 16 keys of this warp's K lie: in a box of their own, or in one with others.
    auto keys16 = [&](int k) -> uint32_t { return ((16 * k) >> p.box_log2) * box_bytes + ((16 * k) & (box - 1)) * kRow; };

    float x[kNT][4];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
      for (int u = 0; u < 4; ++u) x[nt][u] = 0.f;
      const int r = 8 * (nt & 1) + (lane & 7), ch = lane >> 3;
      const uint32_t sk16 = sk + keys16(nt >> 1) + r * kRow;
      if constexpr (kF8) {
        uint32_t k[4];
        ldsm4(sk16 + ((ch ^ ((r >> 1) & 3)) << 4), k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_16816<true>(x[nt], q[kk], e4m3x2_to_f16x2(k[kk]), e4m3x2_to_f16x2(k[kk] >> 16));
      } else {
        uint32_t k[8];
        ldsm4(sk16 + ((ch ^ (r & 7)) << 4), k);
        ldsm4(sk16 + (((ch + 4) ^ (r & 7)) << 4), k + 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_16816<false>(x[nt], q[kk], k[2 * kk], k[2 * kk + 1]);
      }
    }
    if (masked) {
      const int j0 = base + 2 * t4;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int u = 0; u < 2 * kHalves; ++u) {
          const int j = j0 + 8 * nt + (u & 1);
          if (j < key_lo[u >> 1] || j > key_hi[u >> 1]) x[nt][u] = -INFINITY;
        }
    }
    uint32_t pk[kNT][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h >= kHalves) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) pk[nt][h] = 0u;
        continue;
      }
      float top = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) top = fmax3(top, x[nt][2 * h], x[nt][2 * h + 1]);
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2)) * sl2;
      const float old = m[h];
      if (__any_sync(0xffffffffu, top > old)) {
        const float now = fmaxf(old, top);
        const float f = now == -INFINITY ? 1.f : ex2_approx(old - now);
        m[h] = now;
        l[h] *= f;
#pragma unroll
        for (int n = 0; n < 8; ++n) o[n][2 * h] *= f, o[n][2 * h + 1] *= f;
      }
      const float ref = m[h] == -INFINITY ? 0.f : m[h];
      float sum = 0.f;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        const float e0 = ex2_approx(fmaf(x[nt][2 * h], sl2, -ref));
        const float e1 = ex2_approx(fmaf(x[nt][2 * h + 1], sl2, -ref));
        sum += e0 + e1;
        pk[nt][h] = kF8 ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1);
      }
      l[h] += sum;
    }
#pragma unroll
    for (int ks = 0; ks < kKeys / 16; ++ks) {
      const int r = (lane & 7) + (lane & 8), ch = lane >> 4;
      const uint32_t sv16 = sv + keys16(ks) + r * kRow;
#pragma unroll
      for (int j = 0; j < (kF8 ? 2 : 4); ++j) {
        uint32_t v[4];
        if constexpr (kF8) {
          ldsm4_t(sv16 + (((2 * j + ch) ^ ((r >> 1) & 3)) << 4), v);
#pragma unroll
          for (int u = 0; u < 4; ++u) v[u] = __byte_perm(v[u], 0u, 0x3120);
        } else {
          ldsm4_t(sv16 + (((2 * j + ch) ^ (r & 7)) << 4), v);
        }
        const uint32_t a[4] = {pk[2 * ks][0], pk[2 * ks][1], pk[2 * ks + 1][0], pk[2 * ks + 1][1]};
        if constexpr (kF8) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {  // 16 dims: the even ones, the odd ones
            mma_16816<true>(o[2 * (2 * j + u)], a, e4m3x2_to_f16x2(v[2 * u]), e4m3x2_to_f16x2(v[2 * u + 1]));
            mma_16816<true>(o[2 * (2 * j + u) + 1], a, e4m3x2_to_f16x2(v[2 * u] >> 16),
                            e4m3x2_to_f16x2(v[2 * u + 1] >> 16));
          }
        } else {
          mma_16816<false>(o[2 * j], a, v[0], v[1]);
          mma_16816<false>(o[2 * j + 1], a, v[2], v[3]);
        }
      }
    }
    // This warp has read the stage, before the copy that reuses it.
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
    if (++s == stages) s = 0, ++turn;

    const bool unit_end = at.off + 1 == blocks;
    if (unit_end || i + 1 == count) {
      // ------------------------------------------- end of this piece of the request
      const bool begun = whole;
      whole = whole && unit_end;
      const int slot = (2 * worker + (unit_end ? 0 : 1)) * per_group + in_group;
      const float vs = kF8 ? paged_load<kBeside>(p.v_scale + g) : 1.f;
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const int row = row0 + 8 * h + r8;
        float sum = l[h];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const int t = row / p.G;
        const bool valid = t < rq.n && real;
        const int head = valid ? g * p.G + row - t * p.G : 0;
        float f = vs;
        if (whole) {
          const float s2 = paged_load<kBeside>(p.sinks + head) * kLog2e;
          const float top = fmaxf(s2, m[h]);
          float all = 0.f;
          f = 0.f;
          if (top != -INFINITY) {
            f = ex2_approx(m[h] - top);
            all = fmaf(sum, f, s2 == top ? 1.f : ex2_approx(s2 - top));
            f = all > 0.f ? vs * f / all : 0.f;
          }
          if (valid && t4 == 0)
            p.lse[static_cast<long long>(head) * p.T + rq.t0 + t] = all > 0.f ? (top + __log2f(all)) * kLn2 : -INFINITY;
        } else if (valid && t4 == 0) {
          p.part_ml[slot * kR + row - row0] = make_float2(m[h], sum);
        }
        if (!valid) continue;
        __nv_bfloat16* dst = p.out + (static_cast<long long>(rq.t0 + t) * p.Hq + head) * kHeadDim;
        float* part = p.part_o + (static_cast<long long>(slot) * kR + row - row0) * kHeadDim;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // 16 dims: two MMA tiles, side by side (bf16) or even and odd dims (e4m3).
          const float y0 = o[2 * e][2 * h] * f, y1 = o[2 * e][2 * h + 1] * f;
          const float z0 = o[2 * e + 1][2 * h] * f, z1 = o[2 * e + 1][2 * h + 1] * f;
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
      if (unit_end && !whole) unit.x = at.b, unit.y = at.c;
      if (!unit_end && begun) unit.z = 1;
      seg_begin = true;
    }
    if (unit_end) {
      if (i + 1 < count) {
        const int last = at.b;
        axis.next_unit(at);
        if (at.b != last) {
          blocks = axis.blocks(at.b);
          rq = paged_request<kBeside>(p, at.b);
          first = rows_first(p, rq);
        }
      }
    } else {
      ++at.off;
    }
  }
  if (!ok) {
    unit = make_int4(-1, 0, 0, 0);
    // Copies in flight still write to this CTA's shared memory.
    for (int i = done; i < min(count, done + stages); ++i) {
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(&full[i % stages], (i / stages) & 1) && global_timer_ns() - t0 < kWaitLimitNs / 4) {
      }
    }
  }
  if (reports) p.part_unit[worker] = unit;
}

}  // namespace sa
