// Paged attention of chunks: requests with more new tokens than the few-rows
// kernel takes.  Bound by the exponentials and the tensor cores, so it is the
// two-tile forward (fwd_kernel.cuh) over pages: 128 MMA rows are P = 128 / G
// tokens of one request times the G heads of a key/value head (any G: the rows
// behind P * G are idle), a CTA owns kTiles adjacent tiles, and warpgroup b
// takes the 64-key steps of tile b with S, P and O in tensor memory.
//
// Work.  A unit is (request, kTiles tiles, key/value head).  The host knows
// neither the lengths nor the number of units U; every CTA counts them for
// itself (one pass over the lengths, a scan, no list in memory) and takes one
// of every wave, the longer units of a request first.  The CTAs that run at once make a
// wave.  The units behind the last full wave are cut into k parts along their
// keys, with k such that the parts fill whole waves as well as they can
// (chunk_parts): a few rows over a long context take all SMs, and the last
// wave of 512 units (1.73 waves) is not half empty.  Parts go to the workspace
// without the sink, and a second kernel joins them.
//
// Keys come page by page: a 128-key tile is 2 to 8 TMA boxes of min(page, 64)
// tokens.  Keys that no row of the request sees (behind its last token, before
// its window) may hold any bits: their S is masked by selection and their rows
// of V are zeroed in shared memory by the softmax threads of the steps that
// hold such keys, since 0 * NaN is not 0.
//
// Rounding: P to bf16 over a bf16 cache, as the forward (both operands of an MMA
// have one type; half a step is 2^-8 of a weight), to fp16 over codes; the rest
// is fp32.
//
// e4m3: the codes come by TMA into a ring of 4 KB slots, and two warps write
// them widened to fp16 (exactly) into the same tiles that TMA fills for bf16.
// Widening costs as much for two query tiles as for four, so one CTA of four
// tiles and twenty warps takes the place of two CTAs of two tiles and ten
// warps each: with the latter, whose registers leave room for one warp to copy
// and widen, that warp took 3 us for a 64-key step.  Q is converted to fp16 in
// place (saturating at +-65504) and P rounded to fp16, whose 11 bits reach down
// to 2^-14 of the row's reference and whose absolute error is 2^-25 of it
// below.  The reference is therefore never the sink.
#pragma once
#include "fwd_kernel.cuh"
#include "paged_attn.cuh"

namespace sa {

// Query tiles of a CTA, its warps (softmax warpgroups first, then MMA, copies
// and, for e4m3, two that widen) and CTAs of a SM.
template <bool kF8>
constexpr int kChunkTiles = kF8 ? 4 : 2;
template <bool kF8>
constexpr int kChunkThreads = kF8 ? 640 : 320;
template <bool kF8>
constexpr int kChunkPerSm = kF8 ? 1 : 2;
constexpr int kChunkSms = 148;
constexpr int kChunkMaxWaves = 3;  // of parts
constexpr int kChunkFixed = 8;     // a part's set-up, ends and join, in 64-key steps
constexpr int kChunkLeast = 4;     // steps of a part
constexpr int kChunkMostParts = 32;  // of a unit
constexpr uint64_t kChunkDrainNs = 1000 * 1000;  // far longer than a copy takes
constexpr int kChunkMaxUnits = 1 << 24;  // of a call; sums of lengths that do not fit stop there
constexpr int kChunkSlots = 4;
constexpr int kChunkSlotKeys = 64;
constexpr int kChunkSlotBytes = kChunkSlotKeys * kHeadDim;  // e4m3 codes of K or V

struct ChunkParams {
  PagedParams a;
  int tokens;          // P: tokens of a query tile
  int wave;            // CTAs that run at once
  int tiles;           // kTiles
  int max_units, max_cut, max_parts;  // what the host counted on: units, cut ones, parts of them
  float* part_o;       // [part][kTiles * 128 rows][64]
  float2* part_ml;     // [part][kTiles * 128] (m in log2 units, l)
  int4* part_unit;     // [cut unit] (request, unit within its head, head, parts)
  int2* part_units;    // cut units of this call, parts of each
};

// One round's work: a unit, or a part of it.
struct ChunkUnit {
  int b;                  // request, -1: none
  PagedRequest rq;
  int g, group;           // key/value head, unit within the request's head
  int part, parts, slot;  // parts > 1: `part` of them, `slot` of the call's
  // Where the barriers' phases stand when it begins: key tiles that have been
  // through the ring, parity of q_full, q_conv and o_full, and of s_full and
  // p_full (bit w: tile w's).
  int ring;
  uint32_t q_parity, s_parity;
};

template <bool kF8>
struct ChunkCtl {
  uint64_t q_full;
  uint64_t q_conv;                 // e4m3: Q converted to fp16 in place (all softmax threads)
  uint64_t k_full[kFwdStages];     // e4m3: two arrivals, of the widening warps
  uint64_t v_full[kFwdStages];
  uint64_t kv_empty[kFwdStages];
  uint64_t codes_full[kChunkSlots];
  uint64_t codes_empty[kChunkSlots];
  uint64_t s_full[kChunkTiles<kF8>];
  uint64_t p_full[kChunkTiles<kF8>];
  uint64_t o_full;
  ChunkUnit unit[2];                   // by the round's parity
  int units[kChunkThreads<kF8> / 32];  // sums per warp
  float steps[kChunkThreads<kF8> / 32];
  int starts[kChunkThreads<kF8>];      // units before each thread's requests
  int total, full, parts;              // units, those of full waves, parts of each of the others
  uint32_t tmem_base;
  int abort;
};

template <bool kF8>
constexpr size_t chunk_smem_bytes() {
  return 1024 + kTileBytes * (kChunkTiles<kF8> + 2 * kFwdStages) + (kF8 ? kChunkSlots * kChunkSlotBytes : 0) +
         sizeof(ChunkCtl<kF8>);
}

// A request's units of one head, and about how many 64-key steps each has.
template <bool kF8>
__device__ __forceinline__ int chunk_units(const ChunkParams& p, const PagedRequest& r) {
  const int tokens = kChunkTiles<kF8> * p.tokens;
  return r.n > p.a.few ? (r.n + tokens - 1) / tokens : 0;
}
template <bool kF8>
__device__ __forceinline__ int chunk_steps(const ChunkParams& p, const PagedRequest& r) {
  const int keys = max(r.len - r.n / 2, 1);
  return (p.a.window > 0 ? min(keys, p.a.window + kChunkTiles<kF8> * p.tokens) : keys) / kHalfN + 1;
}

// A unit's (or part's) first token within the request, keys, 128-key tiles and
// 64-key steps.
struct ChunkKeys {
  int i0;
  int key0, key_hi;  // first key of the first tile, last key that any row sees
  int n_tiles, n_half;
};

template <bool kF8>
__device__ __forceinline__ ChunkKeys chunk_keys(const ChunkParams& p, const ChunkUnit& u) {
  ChunkKeys k;
  const int tokens = kChunkTiles<kF8> * p.tokens, base = u.rq.len - u.rq.n;
  k.i0 = u.group * tokens;
  k.key_hi = base + min(k.i0 + tokens, u.rq.n) - 1;
  const int lo = p.a.window > 0 ? max(0, base + k.i0 - p.a.window + 1) >> p.a.box_log2 << p.a.box_log2 : 0;
  const int halves = k.key_hi < lo ? 1 : (k.key_hi - lo) / kHalfN + 1;
  const int tiles = (halves + 1) / 2;
  int tile0 = 0;
  k.n_tiles = tiles;
  if (u.parts > 1) {
    tile0 = static_cast<int>(static_cast<int64_t>(tiles) * u.part / u.parts);
    k.n_tiles = static_cast<int>(static_cast<int64_t>(tiles) * (u.part + 1) / u.parts) - tile0;
  }
  k.n_half = min(halves - 2 * tile0, 2 * k.n_tiles);
  k.key0 = lo + tile0 * kBlockN;
  return k;
}

// Query tiles of a unit that hold tokens: the last one of a request may have fewer.
template <bool kF8>
__device__ __forceinline__ int chunk_live(const ChunkParams& p, const ChunkUnit& u, const ChunkKeys& k) {
  return min(kChunkTiles<kF8>, (u.rq.n - k.i0 + p.tokens - 1) / p.tokens);
}

// Parts of each of the `rest` units behind the last full wave, of about
// `steps` steps each: the k of k = floor(w waves / rest) with the least
// w (steps / k + fixed).
__device__ __forceinline__ int chunk_parts(int rest, int steps, int wave) {
  int best = 1;
  float least = static_cast<float>(steps + kChunkFixed);
#pragma unroll
  for (int w = 1; w <= kChunkMaxWaves; ++w) {
    int k = static_cast<int>(__fdividef(static_cast<float>(w * wave), static_cast<float>(rest)) + 0.01f);
    if (k * rest > w * wave) --k;
    k = min(min(k, steps / kChunkLeast), kChunkMostParts);
    const float cost = w * (__fdividef(static_cast<float>(steps), static_cast<float>(k)) + 2 * kChunkFixed);
    if (k >= 2 && cost < least) least = cost, best = k;
  }
  return best;
}

// Sums over a CTA's threads, in an order that all CTAs share: upto, the units
// of the threads up to this one, and the totals.
template <bool kF8>
__device__ __forceinline__ void chunk_scan(ChunkCtl<kF8>* cc, int units, float steps, int& upto, int& all_units,
                                           float& all_steps) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  upto = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
    steps += __shfl_xor_sync(0xffffffffu, steps, o);
  }
  if (lane == 31) cc->units[warp] = min(upto, kChunkMaxUnits), cc->steps[warp] = steps;
  __syncthreads();
  all_units = 0;
  all_steps = 0.f;
#pragma unroll
  for (int w = 0; w < kChunkThreads<kF8> / 32; ++w) {
    if (w < warp) upto += cc->units[w];
    all_units += cc->units[w];
    all_steps += cc->steps[w];
  }
}

// Bits lo .. hi of a word (both inclusive and possibly outside of it).
__device__ __forceinline__ uint32_t chunk_bits(int lo, int hi) {
  const uint32_t from = lo <= 0 ? 0xFFFFFFFFu : lo > 31 ? 0u : 0xFFFFFFFFu << lo;
  return hi < 0 ? 0u : hi >= 31 ? from : from & (0xFFFFFFFFu >> (31 - hi));
}

template <bool kF8>
__global__ void __launch_bounds__(kChunkThreads<kF8>, kChunkPerSm<kF8>)
    sink_attn_paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ ChunkParams p) {
  constexpr int kThreads = kChunkThreads<kF8>;
  constexpr int kTiles = kChunkTiles<kF8>;
  constexpr int kMmaWarp = 4 * kTiles, kCopyWarp = kMmaWarp + 1;
  constexpr uint32_t kTmemO = kTiles * kHalfN;  // columns: S / P of each tile, then O of each
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sQ = smem;
  uint8_t* sK = smem + kTiles * kTileBytes;
  uint8_t* sV = sK + kFwdStages * kTileBytes;
  uint8_t* sB = sV + kFwdStages * kTileBytes;
  auto* ctl = reinterpret_cast<ChunkCtl<kF8>*>(sB + (kF8 ? kChunkSlots * kChunkSlotBytes : 0));
  volatile int* abort = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // In this order: the few-rows kernel beside this one does not wait again.
  pdl_wait();
  pdl_launch_dependents();

  // -------------------------------------------------------- the units of the call
  const int per = (p.a.batch + kThreads - 1) / kThreads, b0 = threadIdx.x * per;  // this thread's requests
  {
    int units = 0;
    float steps = 0.f;
    for (int i = 0; i < per && b0 + i < p.a.batch; ++i) {
      if (blockIdx.x == 0) paged_check(p.a, b0 + i);
      const PagedRequest r = paged_request(p.a, b0 + i);
      const int n = chunk_units<kF8>(p, r) * p.a.Hkv;
      units = min(units + min(n, kChunkMaxUnits), kChunkMaxUnits);
      steps += static_cast<float>(n) * chunk_steps<kF8>(p, r);
    }
    int upto, total;
    float all_steps;
    chunk_scan<kF8>(ctl, units, steps, upto, total, all_steps);
    ctl->starts[threadIdx.x] = upto - units;
    if (threadIdx.x == 0) {
      // More units than rows can make come from cu_seqlens that do not increase
      // (paged_check has told): none is taken.
      if (total > p.max_units) total = 0;
      const int full = total / p.wave * p.wave, rest = total - full;
      int parts = p.part_o && rest ? chunk_parts(rest, static_cast<int>(all_steps / total), p.wave) : 1;
      if (rest > p.max_cut || rest * parts > p.max_parts) parts = 1;
      if (blockIdx.x == 0 && p.part_units) *p.part_units = make_int2(parts > 1 ? rest : 0, parts);
      ctl->total = total;
      ctl->full = parts > 1 ? full : total;
      ctl->parts = parts;
      ctl->abort = 0;
      mbar_init(&ctl->q_full, 1);
      mbar_init(&ctl->q_conv, kTiles * kBlockM);  // every softmax thread, with or without rows
      for (int s = 0; s < kFwdStages; ++s) {
        mbar_init(&ctl->k_full[s], kF8 ? 2 : 1);
        mbar_init(&ctl->v_full[s], kF8 ? 2 : 1);
        mbar_init(&ctl->kv_empty[s], 1);
      }
      for (int s = 0; s < kChunkSlots; ++s) {
        mbar_init(&ctl->codes_full[s], 1);
        mbar_init(&ctl->codes_empty[s], 1);
      }
      for (int w = 0; w < kTiles; ++w) {
        mbar_init(&ctl->s_full[w], 1);
        mbar_init(&ctl->p_full[w], kBlockM);
      }
      mbar_init(&ctl->o_full, 1);
      fence_mbar_init();
    }
    __syncthreads();
  }
  const int places = ctl->full + (ctl->total - ctl->full) * ctl->parts;
  if (static_cast<int>(blockIdx.x) >= places) return;

  // A CTA takes one of every gridDim.x places in the list of units and parts,
  // to and fro, since the units of a request get shorter along it.  Its rounds
  // are apart by a barrier of all threads; the mbarriers' phases run on.
  auto round_end = [&]() {
    __syncwarp();
    named_barrier(1, kThreads);
  };

  if (warp == kCopyWarp) {
    // -------------------------------------------------------------------- copies
    // This warp finds the next round's unit, looks up its first pages and copies
    // as many of its key tiles as the ring holds while the others still compute
    // (a window's unit takes 8 us; finding the next one in between took 3 more).
    // Lane x looks up the page of box x, a tile ahead of the copies.  e4m3: four
    // slots a tile, 64 keys each, two of K and two of V.
    constexpr int kAhead = kF8 ? 1 : kFwdStages;  // tiles that the ring takes before the round begins
    const int box_log2 = p.a.box_log2, nbox = kBlockN >> box_log2, page_mask = (1 << p.a.page_log2) - 1;
    const int per_slot = kChunkSlotKeys >> box_log2;
    int ring = 0;
    uint32_t q_parity = 0, s_parity = 0;
    // Round `round`'s unit, by the whole warp.
    auto find = [&](int round) {
      const int first = round * static_cast<int>(gridDim.x);
      const int place = first + static_cast<int>(round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      ChunkUnit u;
      u.b = -1;
      if (first >= places || place >= places) return u;  // nor is there one in any later round
      int unit = place;
      u.part = u.slot = 0;
      u.parts = 1;
      if (place >= ctl->full) {
        u.parts = ctl->parts;
        u.slot = place - ctl->full;
        unit = ctl->full + u.slot / u.parts;
        u.part = u.slot % u.parts;
      }
      int thread = -1;  // the last one whose requests begin at or before the unit
      for (int t = 0; t < kThreads; t += 32) thread += __popc(__ballot_sync(0xffffffffu, ctl->starts[t + lane] <= unit));
      int at = ctl->starts[thread];
      for (u.b = thread * per;; ++u.b) {
        u.rq = paged_request(p.a, u.b);
        const int n = chunk_units<kF8>(p, u.rq) * p.a.Hkv;
        if (unit < at + n) break;
        at += n;
      }
      u.g = (unit - at) % p.a.Hkv;
      u.group = chunk_units<kF8>(p, u.rq) - 1 - (unit - at) / p.a.Hkv;
      u.ring = ring;
      u.q_parity = q_parity;
      u.s_parity = s_parity;
      return u;
    };
    ChunkUnit u;
    ChunkKeys k = {};
    u.b = -1;
    int done = 0, next = 0;  // tiles of the round's unit that have been copied, table entry for the one after them
    bool ok = true;
    for (int round = -1;; ++round) {
      if (round >= 0 && u.b < 0) break;
      // First what is left of this round's tiles, then the first ones of the next.
      for (int ahead = 0; ahead < 2; ++ahead) {
        if (ahead) {
          u = find(round + 1);
          if (lane == 0) ctl->unit[(round + 1) & 1] = u;
          if (round < 0) round_end();  // the first round begins before its copies
          if (u.b < 0) break;
          k = chunk_keys<kF8>(p, u);
          ring += k.n_tiles;
          if (k.n_half > 0) q_parity ^= 1;
          if (k.n_half & 1) s_parity ^= (1u << chunk_live<kF8>(p, u, k)) - 1;
          done = 0;
        } else if (round < 0) {
          continue;
        }
        auto wanted = [&](int j) { return lane < nbox && k.key0 + j * kBlockN + (lane << box_log2) <= k.key_hi; };
        auto entry = [&](int j) { return paged_entry(p.a, u.b, k.key0 + j * kBlockN + (lane << box_log2)); };
        if (ahead && wanted(0)) next = entry(0);
        const int to = ahead ? min(k.n_tiles, kAhead) : k.n_tiles;
        for (; ok && done < to; ++done) {
          const int tile = u.ring + done;
          const int mine = wanted(done) ? paged_page(p.a, next) : p.a.num_pages;
          if (done + 1 < k.n_tiles && wanted(done + 1)) next = entry(done + 1);
          const int at = (k.key0 + done * kBlockN + (lane << box_log2)) & page_mask;
          if constexpr (!kF8) {
            const int s = tile % kFwdStages, turn = tile / kFwdStages;
            if (turn > 0)
              ok = warp_all(mbar_wait(&ctl->kv_empty[s], (turn - 1) & 1, abort, &g_device_error, kDevErrTimeoutProducer));
            if (!ok) break;
            if (elect_one()) {
              mbar_arrive_expect_tx(&ctl->k_full[s], kTileBytes);
              mbar_arrive_expect_tx(&ctl->v_full[s], kTileBytes);
            }
            __syncwarp();
            if (lane < nbox) {  // K first: S waits for it
              const int dst = s * kTileBytes + (lane << box_log2) * kHeadDim * 2;
              tma_load_4d(sK + dst, &tm_k, &ctl->k_full[s], 0, at, u.g, mine);
              tma_load_4d(sV + dst, &tm_v, &ctl->v_full[s], 0, at, u.g, mine);
            }
            __syncwarp();
          } else {
            for (int e = 0; ok && e < kChunkSlots; ++e) {
              if (tile > 0)
                ok = warp_all(mbar_wait(&ctl->codes_empty[e], (tile - 1) & 1, abort, &g_device_error,
                                        kDevErrTimeoutProducer));
              if (!ok) break;
              if (elect_one()) mbar_arrive_expect_tx(&ctl->codes_full[e], kChunkSlotBytes);
              __syncwarp();
              const int x = lane - (e & 1) * per_slot;
              if (x >= 0 && x < per_slot)
                tma_load_4d(sB + e * kChunkSlotBytes + (x << box_log2) * kHeadDim, e < 2 ? &tm_k : &tm_v,
                            &ctl->codes_full[e], 0, at, u.g, mine);
              __syncwarp();
            }
          }
        }
      }
      if (round < 0) continue;
      round_end();
      if (ctl->abort) break;
    }
    if (ctl->abort) {
      // Copies in flight still write to this CTA's shared memory.
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < kChunkDrainNs) {
      }
    }
  } else {
    if (warp == kMmaWarp) {
      tmem_alloc(&ctl->tmem_base, 2 * kTmemO);
      tmem_relinquish();
    }
    tc_fence_before();
    round_end();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;

    for (int round = 0;; ++round) {
      const ChunkUnit& u = ctl->unit[round & 1];
      const int b = u.b;
      if (b < 0) break;
      const PagedRequest rq = u.rq;
      const int g = u.g;
      const int G = p.a.G, base = rq.len - rq.n;  // position of the request's first new token
      const ChunkKeys keys = chunk_keys<kF8>(p, u);
      const int i0 = keys.i0, key0 = keys.key0, n_tiles = keys.n_tiles, n_half = keys.n_half;
      const int live = chunk_live<kF8>(p, u, keys);
      const int ring0 = u.ring;  // tile j of the unit is the ring's ring0 + j
      const uint32_t qp = u.q_parity, sp = u.s_parity;

      if (warp >= kMmaWarp) {
        if (warp == kMmaWarp) {
          // ---------------------------------------------------------- MMA issuer
          // As in the two-tile forward, the tiles in turn: S_b(h) -> P_b(h) -> O_b += P_b V(h) ->
          // S_b(h+1) into the buffer that P_b(h) just left.
          if (n_half > 0 && elect_one()) {
            mbar_arrive_expect_tx(&ctl->q_full, kTiles * p.tokens * G * kHeadDim * 2);
            for (int w = 0; w < kTiles; ++w)
              tma_load_3d(sQ + w * kTileBytes, &tm_q, &ctl->q_full, 0, g * G, rq.t0 + i0 + w * p.tokens);
            const uint32_t tS = tmem;
            const uint32_t tO = tmem + kTmemO;
            const int s0 = ring0 % kFwdStages;
            bool ok = mbar_wait(kF8 ? &ctl->q_conv : &ctl->q_full, qp, abort, &g_device_error, kDevErrTimeoutMma) &&
                      mbar_wait(&ctl->k_full[s0], (ring0 / kFwdStages) & 1, abort, &g_device_error, kDevErrTimeoutMma);
            if (ok) {
              tc_fence_after();
#pragma unroll
              for (int w = 0; w < kTiles; ++w) {
                if (w >= live) break;
                fwd_issue_qk<kF8>(tS + w * kHalfN, smem_u32(sQ + w * kTileBytes), smem_u32(sK + s0 * kTileBytes));
                tc_commit(&ctl->s_full[w]);
              }
            }
            for (int h = 0; ok && h < n_half; ++h) {
              const int j = ring0 + (h >> 1), s = j % kFwdStages;
              const int hn = h + 1, jn = ring0 + (hn >> 1), sn = jn % kFwdStages;
              ok = mbar_wait(&ctl->v_full[s], (j / kFwdStages) & 1, abort, &g_device_error, kDevErrTimeoutMma) &&
                   (hn >= n_half ||
                    mbar_wait(&ctl->k_full[sn], (jn / kFwdStages) & 1, abort, &g_device_error, kDevErrTimeoutMma));
              for (int w = 0; ok && w < live; ++w) {
                ok = mbar_wait(&ctl->p_full[w], (h ^ (sp >> w)) & 1, abort, &g_device_error, kDevErrTimeoutMma);
                if (!ok) break;
                tc_fence_after();
                fwd_issue_pv<kF8>(tO + w * kHeadDim, tS + w * kHalfN, smem_u32(sV + s * kTileBytes) + (h & 1) * kHalfBytes,
                                  h > 0);
                if (hn < n_half) {
                  fwd_issue_qk<kF8>(tS + w * kHalfN, smem_u32(sQ + w * kTileBytes),
                                    smem_u32(sK + sn * kTileBytes) + (hn & 1) * kHalfBytes);
                  tc_commit(&ctl->s_full[w]);
                }
              }
              if (ok && ((h & 1) == 1 || h == n_half - 1)) tc_commit(&ctl->kv_empty[s]);
            }
            if (ok) tc_commit(&ctl->o_full);
          }
        } else if (kF8) {
          // ------------------------------------------------------------ e4m3: widen
          // This warp takes every other slot.  Rows that no row of the request sees
          // become zeros.
          bool ok = true;
          for (int q = warp - kCopyWarp - 1; q < 4 * n_tiles; q += 2) {
            const int j = q >> 2, e = q & 3, at_slot = q % kChunkSlots;
            const int s = (ring0 + j) % kFwdStages, turn = (ring0 + j) / kFwdStages;
            if (e < 2 && turn > 0)
              ok = warp_all(mbar_wait(&ctl->kv_empty[s], (turn - 1) & 1, abort, &g_device_error, kDevErrTimeoutProducer));
            ok = ok && warp_all(mbar_wait(&ctl->codes_full[at_slot], (ring0 + j) & 1, abort, &g_device_error,
                                          kDevErrTimeoutProducer));
            if (!ok) break;
            uint4 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {  // 16 codes: row lane / 4 + 8 u, 16-byte piece lane % 4
              const int row = (lane >> 2) + 8 * u;
              v[u] = *reinterpret_cast<const uint4*>(sB + at_slot * kChunkSlotBytes + row * kHeadDim +
                                                     (((lane & 3) ^ ((row >> 1) & 3)) << 4));
            }
            uint8_t* tile = (e < 2 ? sK : sV) + s * kTileBytes + (e & 1) * kChunkSlotKeys * 128;
            const int key = key0 + j * kBlockN + (e & 1) * kChunkSlotKeys + (lane >> 2);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const int row = (lane >> 2) + 8 * u;
              if (key + 8 * u < rq.lo || key + 8 * u >= rq.len) v[u] = make_uint4(0u, 0u, 0u, 0u);
              const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
              for (int c = 0; c < 2; ++c)
                *reinterpret_cast<uint4*>(tile + row * 128 + (((2 * (lane & 3) + c) ^ (row & 7)) << 4)) =
                    make_uint4(e4m3x2_to_f16x2(w[2 * c]), e4m3x2_to_f16x2(w[2 * c] >> 16), e4m3x2_to_f16x2(w[2 * c + 1]),
                               e4m3x2_to_f16x2(w[2 * c + 1] >> 16));
            }
            fence_proxy_async_smem();  // the tile for the MMA; the slot's reads before its next copy
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&ctl->codes_empty[at_slot]);
              mbar_arrive(e < 2 ? &ctl->k_full[s] : &ctl->v_full[s]);
            }
          }
        }
      } else {
        // --------------------------------------------- softmax (1 row per thread)
        // (What the steps' loop does not need often is read from `u` again: it has
        // no register to spare.)
        const int wg = warp >> 2;
        const int r = threadIdx.x & (kBlockM - 1);
        const int row_t = r / G;
        const int it = i0 + wg * p.tokens + row_t;  // token within the request
        const bool valid = row_t < p.tokens && it < rq.n;
        const int h = g * G + r - row_t * G;
        // Allowed keys [lo_r, hi_r] of this row; empty for idle rows.
        const int hi_r = valid ? base + it : -1;
        const int lo_r = valid && p.a.window > 0 ? max(0, hi_r - p.a.window + 1) : 0;
        // Keys that every row of this warpgroup's tile sees: [all_lo, all_hi].
        const int w0 = i0 + wg * p.tokens, w1 = min(w0 + p.tokens, rq.n) - 1;
        const int all_hi = w0 <= w1 ? base + w0 : -1;
        const int all_lo = p.a.window > 0 ? max(0, base + w1 - p.a.window + 1) : 0;
        float m_ref = -INFINITY, l = 0.f;
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_base + wg * kHalfN;
        const uint32_t tO = tmem + lane_base + kTmemO + wg * kHeadDim;
        const float sl2 = kF8 ? p.a.scale_log2 * *(p.a.k_scale + g) : p.a.scale_log2;
        // A part of a unit with fewer key tiles than parts may have none.
        bool ok = n_half > 0 && wg < live;
        const float s2 = valid ? *(p.a.sinks + h) * kLog2e : 0.f;
        if constexpr (kF8) {
          if (n_half > 0 && wg >= live) mbar_arrive(&ctl->q_conv);
          ok = ok && warp_all(mbar_wait(&ctl->q_full, qp, abort, &g_device_error, kDevErrTimeoutSoftmax));
          if (ok) {
            // Rows of 128 bytes, so elementwise in place whatever the swizzle.
            uint32_t* row = reinterpret_cast<uint32_t*>(sQ + wg * kTileBytes + r * 128);
#pragma unroll 8
            for (int c = 0; c < 32; ++c) {
              const int at = (c + r) & 31;  // 32 lanes, 32 banks
              row[at] = bf16x2_to_f16x2_sat(row[at]);
            }
            fence_proxy_async_smem();
            mbar_arrive(&ctl->q_conv);
          }
        }

        for (int hs = 0; ok && hs < n_half; ++hs) {
          ok = warp_all(mbar_wait(&ctl->s_full[wg], (hs ^ (u.s_parity >> wg)) & 1, abort, &g_device_error, kDevErrTimeoutSoftmax));
          if (!ok) break;
          tc_fence_after();
          uint32_t sr[kHalfN];
          tmem_ld64(tS, sr);
          const int ks = key0 + hs * kHalfN;
          if (ks + kHalfN - 1 > all_hi || ks < all_lo) {
            // One bit per key: a test and a selection each, where two compares of
            // the key's place made a window layer's steps half as long again.
            const uint32_t seen[2] = {chunk_bits(lo_r - ks, hi_r - ks), chunk_bits(lo_r - ks - 32, hi_r - ks - 32)};
#pragma unroll
            for (int c = 0; c < kHalfN; ++c) sr[c] = seen[c >> 5] >> (c & 31) & 1u ? sr[c] : 0xFF800000u;
          }
          const FwdRowStep st = fwd_row_step<false, kF8>(sr, 0, 0, sl2, m_ref);
          l = l * st.alpha + st.sum;
          __syncwarp();
          tmem_st32(tS, sr);
          if (hs > 0 && __any_sync(0xffffffffu, st.need)) {
            uint32_t o[kHeadDim];
            tmem_ld64(tO, o);
#pragma unroll
            for (int c = 0; c < kHeadDim; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * st.alpha);
            tmem_st32(tO, o);
            tmem_st32(tO + 32, o + 32);
          }
          m_ref = st.m_new;
          if constexpr (!kF8) {
            // Keys of the step that no row of the request sees: zero rows of V.
            // Both warpgroups write them, each before its own PV.
            if (ks < u.rq.lo || ks + kHalfN > u.rq.len) {
              const int j = u.ring + (hs >> 1), s = j % kFwdStages;
              ok = warp_all(mbar_wait(&ctl->v_full[s], (j / kFwdStages) & 1, abort, &g_device_error, kDevErrTimeoutSoftmax));
              if (!ok) break;
              const int key = ks + (r >> 1);
              if (key < u.rq.lo || key >= u.rq.len) {
                uint4* row = reinterpret_cast<uint4*>(sV + s * kTileBytes + ((hs & 1) * kHalfN + (r >> 1)) * 128 + (r & 1) * 64);
#pragma unroll
                for (int c = 0; c < 4; ++c) row[c] = make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();
            }
          }
          tc_fence_before();
          mbar_arrive(&ctl->p_full[wg]);
        }

        // ---------------------------------------------------------------- epilogue
        if (n_half == 0) {
          p.part_ml[static_cast<long long>(u.slot) * kTiles * kBlockM + wg * kBlockM + r] = make_float2(-INFINITY, 0.f);
          if (u.part == 0 && threadIdx.x == 0) p.part_unit[u.slot / u.parts] = make_int4(u.b, u.group, u.g, u.parts);
        }
        if (ok) ok = mbar_wait(&ctl->o_full, u.q_parity, abort, &g_device_error, kDevErrTimeoutEpilogue);
        ok = warp_all(ok);
        if (ok) {
          tc_fence_after();
          uint32_t o[kHeadDim];
          __syncwarp();
          tmem_ld64(tO, o);
          const float vs = kF8 ? *(p.a.v_scale + u.g) : 1.f;
          const int row_e = r / G, it_e = (u.group * kTiles + wg) * p.tokens + row_e, h_e = u.g * G + r - row_e * G;
          const bool valid_e = row_e < p.tokens && it_e < u.rq.n;
          if (u.parts > 1) {
            const long long at = static_cast<long long>(u.slot) * kTiles * kBlockM + wg * kBlockM + r;
            p.part_ml[at] = make_float2(m_ref, l);
            if (u.part == 0 && threadIdx.x == 0) p.part_unit[u.slot / u.parts] = make_int4(u.b, u.group, u.g, u.parts);
            float4* dst = reinterpret_cast<float4*>(p.part_o + at * kHeadDim);
            if (valid_e) {
#pragma unroll
              for (int c = 0; c < kHeadDim / 4; ++c)
                dst[c] = make_float4(__uint_as_float(o[4 * c]) * vs, __uint_as_float(o[4 * c + 1]) * vs,
                                     __uint_as_float(o[4 * c + 2]) * vs, __uint_as_float(o[4 * c + 3]) * vs);
            }
          } else {
            const float top = fmaxf(s2, m_ref);
            float f = 0.f, all = 0.f;
            if (top != -INFINITY) {
              f = ex2_approx(m_ref - top);
              all = fmaf(l, f, s2 == top ? 1.f : ex2_approx(s2 - top));
            }
            f = all > 0.f ? vs * f / all : 0.f;
            const int t = u.rq.t0 + it_e;
            if (valid_e) p.a.lse[static_cast<long long>(h_e) * p.a.T + t] = all > 0.f ? (top + __log2f(all)) * kLn2 : -INFINITY;
            // The warp's 32 rows through its part of the Q tile, which no MMA reads
            // any more, so that eight lanes write a row's 128 bytes (rows written
            // each by its own thread took 1.9 us).
            uint8_t* rows = sQ + wg * kTileBytes + (r & ~31) * 128;
#pragma unroll
            for (int c = 0; c < kHeadDim / 8; ++c) {
              uint4 v;
              v.x = pack_bf16x2(__uint_as_float(o[8 * c + 0]) * f, __uint_as_float(o[8 * c + 1]) * f);
              v.y = pack_bf16x2(__uint_as_float(o[8 * c + 2]) * f, __uint_as_float(o[8 * c + 3]) * f);
              v.z = pack_bf16x2(__uint_as_float(o[8 * c + 4]) * f, __uint_as_float(o[8 * c + 5]) * f);
              v.w = pack_bf16x2(__uint_as_float(o[8 * c + 6]) * f, __uint_as_float(o[8 * c + 7]) * f);
              *reinterpret_cast<uint4*>(rows + lane * 128 + ((c ^ (lane & 7)) << 4)) = v;
            }
            const long long mine = valid_e ? (static_cast<long long>(t) * p.a.Hq + h_e) * kHeadDim : -1;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int row = 4 * i + (lane >> 3), c = lane & 7;
              const uint4 v = *reinterpret_cast<const uint4*>(rows + row * 128 + ((c ^ (row & 7)) << 4));
              const long long to = __shfl_sync(0xffffffffu, mine, row);
              if (to >= 0) *reinterpret_cast<uint4*>(p.a.out + to + 8 * c) = v;
            }
            fence_proxy_async_smem();  // before the next round's Q
          }
        }
      }
      tc_fence_before();
      round_end();
      tc_fence_after();
      if (ctl->abort) break;
    }
  }

  round_end();
  if (warp == kMmaWarp) tmem_dealloc(ctl->tmem_base, 2 * kTmemO);
}

}  // namespace sa
