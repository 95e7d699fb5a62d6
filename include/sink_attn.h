/*
 * sink_attn.h - C ABI of libsinkattn.so: causal grouped-query attention with
 * a learned per-head attention sink, an optional sliding window and optional
 * packed documents (varlen), forward and backward, for NVIDIA B200 (sm_100a).
 *
 * The operation.  Attention sinks are named in "gpt-oss implementation"
 * (Megatron-LM issue 1739), section "Attention Mechanisms / Attention Sinks"
 * (after StreamingLLM), in "Tricks from OpenAI gpt-oss you can use with
 * transformers" ("Flash Attention 3 with support for attention sinks") and
 * in tpu-inference PR 861 (a kernel argument `attention_sink`).  The pages
 * name the sink without writing it out; the reading implemented here is the
 * gpt-oss one: one extra logit s_h per query head joins each row's softmax
 * denominator and carries no value:
 *
 *   l_ij  = scale * q_i . k_j                      (j allowed for row i)
 *   m_i   = max(s_h, max_j l_ij)
 *   out_i = sum_j e^{l_ij - m_i} v_j / (e^{s_h - m_i} + sum_j e^{l_ij - m_i})
 *   lse_i = m_i + ln(e^{s_h - m_i} + sum_j e^{l_ij - m_i})   (sink included)
 *
 * s_h is used as given (it is not multiplied by `scale`); s_h = -INFINITY
 * turns the sink off.  Query head h reads key/value head h / (Hq / Hkv).
 *
 * Allowed keys.  Positions are local to a document.  For doc-local query
 * position i, key j is allowed iff j <= i and, when window > 0, i - j < window
 * (a window of `window` keys including the query itself).  window <= 0 is
 * full causal.  The alternating sliding-window / full-causal layer pattern of
 * "gpt-oss implementation" ("Alternating Sliding-Window Attention Pattern")
 * is the caller choosing `window` per layer.  Documents follow the
 * intra-document masking request in the same issue: no attention crosses a
 * cu_seqlens boundary.
 *
 * Backward (derivative of the above; dout given):
 *   P_ij = e^{l_ij - lse_i}, P_sink,i = e^{s_h - lse_i}, D_i = dout_i . out_i
 *   dS_ij = P_ij (dout_i . v_j - D_i)
 *   dq_i = scale sum_j dS_ij k_j, dk_j = scale sum_{i, h in group} dS_ij q_i,
 *   dv_j = sum_{i, h in group} P_ij dout_i, dsinks_h = -sum_i P_sink,i D_i.
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller; the
 *     library never allocates, frees or synchronises, and every call is
 *     asynchronous on `stream` (a cudaStream_t passed as void*, NULL = the
 *     legacy default stream).
 *   - Arguments are validated on the host before any launch; a failed check
 *     returns an error status and launches nothing.
 *   - Layouts are dense and row-major: q/out/dout/dq [T][Hq][D],
 *     k/v/dk/dv [T][Hkv][D] (bf16), lse [Hq][T] (fp32), sinks/dsinks [Hq]
 *     (fp32), cu_seqlens [batch+1] (int32, device, cu_seqlens[0] = 0,
 *     cu_seqlens[batch] = T, non-decreasing).
 *   - Supported: D = 64; Hq % Hkv == 0 with G = Hq / Hkv a power of two
 *     <= 128 (any whole number <= 128 over a paged cache); scale finite and
 *     > 0; bf16 tensors 16-byte aligned.
 *   - A device-side wait that exceeds its time limit (about one second; it
 *     never happens in a correct build) makes the kernel record an error
 *     code and return instead of hanging; sink_attn_last_device_error()
 *     reads it.
 */
#ifndef SINK_ATTN_H_
#define SINK_ATTN_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SINK_ATTN_OK = 0,
    SINK_ATTN_ERR_NULL = 1,          /* a required pointer is NULL */
    SINK_ATTN_ERR_SHAPE = 2,         /* inconsistent or negative sizes */
    SINK_ATTN_ERR_ALIGN = 3,         /* a tensor is not 16-byte aligned */
    SINK_ATTN_ERR_UNSUPPORTED = 4,   /* valid, but outside what this library implements */
    SINK_ATTN_ERR_CUDA = 5,          /* a CUDA runtime/driver call failed */
    SINK_ATTN_ERR_DEVICE_TIMEOUT = 6,/* a kernel gave up on a wait (see sink_attn_last_device_error) */
    SINK_ATTN_ERR_WORKSPACE = 7      /* workspace missing or smaller than sink_attn_bwd_workspace_size() */
} sink_attn_status;

typedef struct {
    int batch;        /* B: number of documents (cu_seqlens has batch+1 entries) */
    int max_seqlen;   /* >= every document length; with cu_seqlens == NULL the
                         common length S of every document (T = B * S) */
    int total_tokens; /* T */
    int num_q_heads;  /* Hq */
    int num_kv_heads; /* Hkv */
    int head_dim;     /* D (64) */
} sink_attn_dims;

/* Forward.  q [T][Hq][D] bf16, k, v [T][Hkv][D] bf16, sinks [Hq] fp32 (may
 * hold -INFINITY), cu_seqlens int32 [batch+1] on the device or NULL (then
 * every document has length max_seqlen).  Writes out [T][Hq][D] bf16 and
 * lse [Hq][T] fp32 (natural log, sink included).  T = 0 is a no-op.  Runs
 * the kernel sink_attn_fwd_kernel_for() names (two query tiles per CTA). */
sink_attn_status sink_attn_fwd(const sink_attn_dims* dims,
                               const void* q, const void* k, const void* v,
                               const float* sinks, const int* cu_seqlens,
                               int window, float scale,
                               void* out, float* lse, void* stream);

/* Forward on CTA pairs: the same operation, arguments, layouts, ownership
 * and errors as sink_attn_fwd() (the online softmax with the sink logit as
 * the first reference max, "Tricks from OpenAI gpt-oss you can use with
 * transformers", kernels section; the window and document masks of "gpt-oss
 * implementation", alternating sliding-window pattern), computed by a kernel
 * launched as clusters of two CTAs whose tensor-core MMAs run on the CTA
 * pair (M = 256 rows: two adjacent query tiles of one key/value head).  Each
 * CTA loads half of every key and value step, and one thread issues the
 * pair's MMAs.  The two tiles of a pair walk the union of their key ranges,
 * so a row's keys may be split into 64-key steps at other boundaries than
 * in sink_attn_fwd(): the results agree with it to rounding, not bit for
 * bit.  Returns SINK_ATTN_ERR_CUDA if the device cannot run clusters of two
 * CTAs of this kernel. */
sink_attn_status sink_attn_fwd_pair(const sink_attn_dims* dims,
                                    const void* q, const void* k, const void* v,
                                    const float* sinks, const int* cu_seqlens,
                                    int window, float scale,
                                    void* out, float* lse, void* stream);

/* The forward kernels of this library.  All compute the same operation with
 * the same arguments; they differ in how query tiles (128 rows: 128/G tokens
 * x the G query heads of one key/value head) map to CTAs, and their results
 * agree to rounding, not bit for bit, because a row's keys may be split into
 * 64-key steps at other boundaries. */
typedef enum {
    SINK_ATTN_FWD_AUTO = 0,      /* the kernel sink_attn_fwd() picks for the sizes */
    SINK_ATTN_FWD_ONE_TILE = 1,  /* one query tile per CTA; its two softmax warpgroups take alternate
                                    64-key steps and merge at the end */
    SINK_ATTN_FWD_TWO_TILES = 2, /* two adjacent query tiles per CTA, one per softmax warpgroup, sharing
                                    one key/value stream (short key ranges: sliding-window layers) */
    SINK_ATTN_FWD_CTA_PAIR = 3   /* two adjacent query tiles on a pair of CTAs (cluster of two) with
                                    M = 256 tensor-core MMAs, as sink_attn_fwd_pair() */
} sink_attn_fwd_kernel_id;

/* The forward with an explicit kernel (a sink_attn_fwd_kernel_id); arguments,
 * layouts and errors as sink_attn_fwd().  An unknown id returns
 * SINK_ATTN_ERR_UNSUPPORTED before any launch. */
sink_attn_status sink_attn_fwd_with(const sink_attn_dims* dims,
                                    const void* q, const void* k, const void* v,
                                    const float* sinks, const int* cu_seqlens,
                                    int window, float scale,
                                    void* out, float* lse, int kernel, void* stream);

/* The sink_attn_fwd_kernel_id sink_attn_fwd() runs for these sizes and
 * window (never SINK_ATTN_FWD_AUTO), or -1 when the sizes are invalid. */
int sink_attn_fwd_kernel_for(const sink_attn_dims* dims, int window);

/* Bytes of device workspace sink_attn_bwd() needs for these sizes
 * (fp32 dq accumulator, per-row D_i, per-block sink partials, padding).
 * Returns 0 when the sizes are invalid. */
size_t sink_attn_bwd_workspace_size(const sink_attn_dims* dims);

/* Backward.  Inputs as for the forward plus the forward's saved out and lse
 * and the upstream gradient dout [T][Hq][D] bf16.  Writes (overwrites, does
 * not accumulate) dq [T][Hq][D], dk, dv [T][Hkv][D] (bf16) and dsinks [Hq]
 * (fp32).  dsinks is reduced in a fixed order and is bitwise reproducible
 * run to run; dq is summed over key tiles in an fp32 accumulator by TMA
 * bulk reduce-adds (performed in L2 in whatever order the tiles finish), so
 * it may differ in the last bits between runs.  `workspace` is caller-owned
 * device memory of at least sink_attn_bwd_workspace_size(dims) bytes,
 * 256-byte aligned; its contents on entry do not matter. */
sink_attn_status sink_attn_bwd(const sink_attn_dims* dims,
                               const void* q, const void* k, const void* v,
                               const float* sinks, const int* cu_seqlens,
                               int window, float scale,
                               const void* out, const float* lse, const void* dout,
                               void* dq, void* dk, void* dv, float* dsinks,
                               void* workspace, size_t workspace_bytes,
                               void* stream);

/* Size of the library's built-in backward scratch buffer used by
 * sink_attn_bwd_noalloc(): 32 MiB. */
#define SINK_ATTN_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)

/* Backward for callers that cannot allocate device memory.  This entry point
 * is an addition of this library; the pages describe nothing like it.
 *
 * Some callers cannot call cudaMalloc or hand over a workspace: code running
 * inside a memory pool or allocator callback that must not re-enter the
 * allocator, host code that is not allowed to grow device memory after
 * start-up, or a binding whose only way to pass memory is the tensors it
 * already owns.  This entry point computes exactly what sink_attn_bwd()
 * computes, with the same arguments minus the workspace: its scratch (fp32 dq
 * accumulator, D_i, sink partials) lives in a fixed array of
 * SINK_ATTN_NOALLOC_SCRATCH_BYTES inside the library, which every GPU that
 * loads the library holds until the process exits.  It calls no cudaMalloc,
 * cudaFree or other allocating routine.
 *
 *  - Sizes whose sink_attn_bwd_workspace_size() exceeds the array are refused
 *    with SINK_ATTN_ERR_WORKSPACE before any launch (at 64 query heads and
 *    head dim 64 that is about 2000 tokens; at 8 query heads about 16000).
 *  - The first call on each device looks up the array's device address
 *    (cudaGetSymbolAddress, with that device current); make that first call
 *    before capturing a stream into a CUDA graph.
 *  - Every call on a device shares the one array and leaves its contents
 *    behind; the kernels re-initialise everything they read (the dq
 *    accumulator is zeroed each call).  Calls whose execution overlaps on the
 *    GPU (different streams, or different host threads) race on the array and
 *    give wrong results: serialise them. */
sink_attn_status sink_attn_bwd_noalloc(const sink_attn_dims* dims,
                                       const void* q, const void* k, const void* v,
                                       const float* sinks, const int* cu_seqlens,
                                       int window, float scale,
                                       const void* out, const float* lse, const void* dout,
                                       void* dq, void* dk, void* dv, float* dsinks,
                                       void* stream);

/* ------------------------------------------------------------------ decode
 * Decode forward over a key/value cache: a few new tokens per sequence are
 * appended to the cache and their queries attend to everything the cache
 * holds for that sequence, with the same sink, window and causal rules as
 * sink_attn_fwd().  This is the incremental form of the forward the pages use
 * for generation with the alternating sliding-window / full layers
 * ("Tricks from OpenAI gpt-oss you can use with transformers", list item
 * "Dynamic Sliding Window Layer & Cache"); the pages do not describe the
 * cache itself, so its layout is this library's own:
 *
 *   - Sequence b owns cache_capacity (C) slots of k_cache / v_cache, each
 *     slot [Hkv][D] bf16: k_cache, v_cache are [batch][C][Hkv][D].  The token
 *     at position p lives in slot p mod C.  With C >= every sequence length
 *     this is a plain linear cache; a sliding-window layer may keep a ring of
 *     C >= window + new_tokens - 1 slots, which holds every key a new query
 *     can see.  A ring smaller than that loses keys: the kernel then records
 *     device error 0x201 (see sink_attn_device_error) and its output is not
 *     defined.
 *   - cache_seqlens [batch] (int32, device) = L0_b, the tokens of sequence b
 *     in the cache before this call.  The call writes the new tokens at
 *     positions L0_b .. L0_b + new_tokens - 1 (slots mod C) and does not
 *     modify cache_seqlens; the caller advances it by new_tokens.
 *   - New query t of sequence b has position i = L0_b + t and sees key
 *     position j iff j <= i and (window <= 0 or i - j < window).
 */
typedef struct {
    int batch;          /* sequences */
    int new_tokens;     /* Lq >= 1: new tokens per sequence (1 for one-token decode) */
    int cache_capacity; /* C: slots per sequence */
    int max_seqlen;     /* upper bound on L0_b + new_tokens over b (sizes the split grid) */
    int num_q_heads;    /* Hq */
    int num_kv_heads;   /* Hkv */
    int head_dim;       /* D (64) */
} sink_attn_decode_dims;

/* Bytes of device workspace sink_attn_decode() needs (per-split partial
 * results); 0 when the sizes are invalid.  Depends on `window`. */
size_t sink_attn_decode_workspace_size(const sink_attn_decode_dims* dims, int window);

/* Decode.  q [batch][new_tokens][Hq][D] bf16, k_new / v_new
 * [batch][new_tokens][Hkv][D] bf16 (appended to the cache by this call),
 * k_cache / v_cache as above (read and written), cache_seqlens as above,
 * sinks [Hq] fp32.  Writes out [batch][new_tokens][Hq][D] bf16 and
 * lse [Hq][batch * new_tokens] fp32 (natural log, sink included).
 * Supported: D = 64, G = Hq / Hkv a power of two with G * new_tokens <= 64.
 * `workspace`: caller-owned device memory of at least
 * sink_attn_decode_workspace_size(dims, window) bytes, 256-byte aligned.
 * batch = 0 is a no-op.  Launches two or three kernels on `stream` (see
 * sink_attn_decode_launches). */
sink_attn_status sink_attn_decode(const sink_attn_decode_dims* dims,
                                  const void* q, const void* k_new, const void* v_new,
                                  void* k_cache, void* v_cache, const int* cache_seqlens,
                                  const float* sinks, int window, float scale,
                                  void* out, float* lse,
                                  void* workspace, size_t workspace_bytes,
                                  void* stream);

/* Decode over an FP8 (e4m3) cache.  As sink_attn_decode(), except that
 * k_cache / v_cache hold e4m3 codes, one byte per element,
 * [batch][C][Hkv][D], with one dequantisation scale per key/value head:
 * key = code * k_scale[g], value = code * v_scale[g] (k_scale, v_scale:
 * fp32 [Hkv], device, > 0).  The pages list FP8 training recipes (Megatron-LM
 * issue 1739 and its example scripts); this is the place on this path where
 * FP8 pays on B200 at head dim 64: decode is HBM-bound, and e4m3 storage
 * halves the bytes the cache moves.  The kernel widens the codes to fp16
 * (every e4m3 value is exact in fp16) and runs fp16 MMAs, so the queries are
 * converted from bf16 to fp16 for them: a query element beyond the fp16
 * range saturates to +-65504, the one input-range limit of this variant
 * (sink_attn_decode has none).  The call quantises the new tokens' k_new / v_new
 * (bf16) as code = e4m3(x * (1 / scale)), rounded to nearest even and
 * saturated to +-448, into their slots.  The workspace size is that of
 * sink_attn_decode_workspace_size(). */
sink_attn_status sink_attn_decode_e4m3(const sink_attn_decode_dims* dims,
                                       const void* q, const void* k_new, const void* v_new,
                                       void* k_cache, void* v_cache, const int* cache_seqlens,
                                       const float* k_scale, const float* v_scale,
                                       const float* sinks, int window, float scale,
                                       void* out, float* lse,
                                       void* workspace, size_t workspace_bytes,
                                       void* stream);

/* Decode over an FP8 (e4m3) cache with the PV product on the FP8 tensor-core
 * path (tcgen05 kind::f8f6f4).  Arguments, cache layout, quantisation of the
 * new tokens and workspace as for sink_attn_decode_e4m3().  The value codes
 * are read as stored (not widened to fp16), and the unnormalised weights
 * p_j = 2^(x_j - m) of each row (m the kernel's running reference of the
 * row, p_j <= 2^8) are rounded to e4m3 (nearest even, saturating) before
 * the MMA; the row sums use the same rounded weights, so every output row is
 * still a convex combination of its cached values.  The rounding moves each
 * weight by at most 2^-4 of itself (e4m3's 3 mantissa bits; below e4m3's
 * normal range, 2^-6, by at most 2^-10), which bounds the extra error of a
 * row with normalised weights pi_j by
 *   |out - exact| <= 2^-4 sum_j pi_j |v_j - out| + 2^-10 max_j pi_j sum_j |v_j - out|
 *   |lse - exact| <= 2^-4 + 2^-10 max_j pi_j * (keys seen)
 * on top of sink_attn_decode_e4m3's own rounding.  The logits keep the fp16
 * path of sink_attn_decode_e4m3 (keys widened to fp16, queries converted to
 * fp16): e4m3 queries would move every logit by up to 2^-4 of its terms. */
sink_attn_status sink_attn_decode_e4m3_f8pv(const sink_attn_decode_dims* dims,
                                            const void* q, const void* k_new, const void* v_new,
                                            void* k_cache, void* v_cache, const int* cache_seqlens,
                                            const float* k_scale, const float* v_scale,
                                            const float* sinks, int window, float scale,
                                            void* out, float* lse,
                                            void* workspace, size_t workspace_bytes,
                                            void* stream);

/* Number of kernels one sink_attn_decode / sink_attn_decode_e4m3 call
 * launches for these sizes and window (0 when batch = 0): append, attend and
 * combine, or only the first two when one CTA per (sequence, key/value head)
 * covers the cache (the attend kernel then finishes the rows itself). */
int sink_attn_decode_launches(const sink_attn_decode_dims* dims, int window);

/* ------------------------------------------------------------- paged cache
 * Serving over a paged key/value cache: the keys and values of all requests
 * live in a pool of num_pages pages of page_size tokens each, and a request
 * owns the pages its row of block_table names.  A serving step is
 *
 *   sink_attn_paged_plan    lengths -> block-table entries, slots, cu_seqlens
 *   sink_attn_paged_append  the new keys and values into their slots (per layer)
 *   sink_attn_paged_attn    the new tokens' attention over the pages (per layer)
 *
 * It is the paged counterpart of the "Dynamic Sliding Window Layer & Cache" of
 * "Tricks from OpenAI gpt-oss you can use with transformers": the pages do not
 * describe a paged cache, so its layout is this library's own.
 *
 *   - k_cache / v_cache hold [num_pages][page_size][Hkv][D] elements, bf16 or
 *     e4m3 codes, at any strides (in elements, the same for both): the D
 *     elements of a row are contiguous, rows are 16-byte aligned.  Token-major
 *     pages, head-major pages and the two halves of one fused tensor are all
 *     given by their strides.
 *   - The token at position p of request b lies in page
 *     block_table[b][p / page_size] at offset p mod page_size; its slot is
 *     page * page_size + offset (int32; num_pages * page_size < 2^31).
 *     Entries of pages that no query of a call can see are not read and may
 *     hold anything, -1 for example; slots that hold no token which some new
 *     token of the request sees may hold any bits, NaN included.  The others
 *     hold finite numbers: an infinity or a NaN in one may reach the rows of the
 *     same request that do not see it.
 *   - The new tokens of a step are packed: request b's are rows
 *     cu_seqlens[b] .. cu_seqlens[b+1] - 1 of q.  kv_lens[b] counts its tokens
 *     after the step, so its new token t has position
 *     kv_lens[b] - (cu_seqlens[b+1] - cu_seqlens[b]) + t.
 *   - page_size is a power of two from 16 to 1024.  A cache's rows do not
 *     overlap: the stride of a dimension of several elements is at least D.
 *   - What only the device can see (a page outside the pool, lengths that do
 *     not fit) never leads to an access out of range: it is recorded as a
 *     device error (0x202 the pool ran dry, 0x203 a page outside the pool,
 *     0x204 lengths that do not fit the table or the slot map, 0x205 rows
 *     that do not fit total_tokens or max_new), see sink_attn_device_error().
 */

/* Planning a step.  One launch; nothing is read back to the host, so a step
 * can be captured into a CUDA graph and replayed with new lengths.
 *
 * In: cached_lens [batch] (tokens in the cache before the step), new_lens
 * [batch] (new tokens; 0: idle; negative: the request has ended), pool = {head,
 * count}: the free pages are free_pages[(head + i) mod num_pages], i < count,
 * first_page [batch] or NULL (leading pages of the request that it gave back
 * earlier).  In and out: block_table [batch][max_pages], free_pages
 * [num_pages].  Out: cu_seqlens [batch + 1], kv_lens [batch], slot_map
 * [max_tokens], pool_out (2 ints), first_page_out [batch] (NULL with
 * first_page).  All int32, 4-byte aligned.
 *
 *   - Request b needs ceil((c + n) / P) - ceil(c / P) new pages; they are taken
 *     from the head of the ring in the order of the requests and written to its
 *     table row.  A request that needs pages when those left do not suffice
 *     gets none, nor does any request behind it that needs some: its slots are
 *     -1, its kv_lens stays cached_lens, and device error 0x202 is recorded.
 *     So it is with a request whose tokens do not fit its table row (0x204).
 *     Its rows keep their places in cu_seqlens (whose sums end at 2^31 - 1),
 *     and what attention writes into them means nothing.
 *   - An ended request gives back its pages (from first_page on); its kv_lens
 *     and first_page_out become 0.
 *   - With window > 0 (needs first_page) a request gives back the pages wholly
 *     before position cached_lens - window + 1, which no query of this step or
 *     a later one sees, also when its new tokens get no room.  Pages given back
 *     go to the tail of the ring, in the order of requests and pages; this step
 *     takes none of them.
 *   - slot_map[t] is the slot of packed token t, and -1 from the last token on
 *     up to max_tokens.
 *   - kv_lens may be cached_lens, pool_out may be pool and first_page_out may
 *     be first_page; other overlaps are not allowed.  Where they are distinct,
 *     the call can be repeated and gives the same again.
 *
 * batch is at most 4096, batch * max_pages * page_size at most 2^30.  batch = 0
 * is a no-op. */
typedef struct {
    int batch;      /* requests */
    int max_tokens; /* entries of slot_map */
    int max_pages;  /* entries of a block-table row */
    int page_size;
    int num_pages;  /* pages of the pool, entries of free_pages */
} sink_attn_plan_dims;

sink_attn_status sink_attn_paged_plan(const sink_attn_plan_dims* dims,
                                      const int* cached_lens, const int* new_lens,
                                      int* block_table, int* free_pages, const int* pool,
                                      const int* first_page, int window,
                                      int* cu_seqlens, int* kv_lens, int* slot_map,
                                      int* pool_out, int* first_page_out, void* stream);

typedef struct {
    int batch;        /* requests (attention only) */
    int total_tokens; /* T: rows of q / out, or of k_new / v_new and slot_map */
    int max_new;      /* attention only: >= the new tokens of every request */
    int num_q_heads;  /* Hq (attention only) */
    int num_kv_heads; /* Hkv */
    int head_dim;     /* D (64) */
    int page_size;
    int num_pages;
    int max_pages;         /* entries of a block-table row (attention only) */
    long long page_stride; /* strides of k_cache and v_cache, in elements */
    long long token_stride;
    long long head_stride;
    long long q_stride;    /* elements between tokens of q (attention only) */
} sink_attn_paged_dims;

/* Appends new keys and values: row t of k_new / v_new ([T][Hkv][D] bf16, k_stride
 * and v_stride elements between tokens) goes to slot slot_map[t]; a negative
 * slot is skipped.  If a slot occurs twice, which of its tokens it holds
 * afterwards is not defined.  T = 0 is a no-op. */
sink_attn_status sink_attn_paged_append(const sink_attn_paged_dims* dims,
                                        const void* k_new, const void* v_new,
                                        long long k_stride, long long v_stride, const int* slot_map,
                                        void* k_cache, void* v_cache, void* stream);

/* The same into an e4m3 cache: code = e4m3(x * (1 / scale)), rounded to nearest
 * even and saturated to +-448, with one scale per key/value head (fp32 [Hkv],
 * device, > 0). */
sink_attn_status sink_attn_paged_append_e4m3(const sink_attn_paged_dims* dims,
                                             const void* k_new, const void* v_new,
                                             long long k_stride, long long v_stride, const int* slot_map,
                                             void* k_cache, void* v_cache,
                                             const float* k_scale, const float* v_scale, void* stream);

/* Bytes of device workspace sink_attn_paged_attn() and its e4m3 form need (0
 * when the sizes are invalid). */
size_t sink_attn_paged_workspace_size(const sink_attn_paged_dims* dims);

/* Attention of a step's new tokens, one or many per request, over the paged
 * cache: the forward's operation (sink, window, causal order by position).
 * q [T][Hq][D] bf16 (q_stride elements between tokens), block_table
 * [batch][max_pages], cu_seqlens [batch + 1] and kv_lens [batch] (int32,
 * device), sinks [Hq] fp32.  Writes out [T][Hq][D] bf16 (dense) and lse
 * [Hq][T] fp32 of the rows before cu_seqlens[batch]; rows behind them are left
 * as they were.  A row that sees no key gets out = 0 and lse = its sink.
 * G = Hq / Hkv is any whole number up to 128; batch is at most 4096, and batch *
 * max_pages * page_size * Hkv at most 2^35.  q_stride >= Hq * D where T > 1.
 * Requests of few tokens and of many go to different kernels, which run side by
 * side.  Few are up to max_new tokens where max_new * G <= 64, and in calls with
 * longer requests up to 8 / G, one at least (none for G > 64).  So max_new tells
 * which kernels a call needs, and with batch and T whether its chunks come among
 * mostly single tokens, which are shared out in another way: a decode step should
 * say 1, and a step of prompts its longest one (three or more of them with
 * max_new = T take up to a tenth longer).  Nothing is read back to the host: the
 * lengths may change between replays of a captured call.  `workspace`:
 * caller-owned, 256-byte aligned, of sink_attn_paged_workspace_size(dims) bytes
 * and any content; calls whose execution may overlap need one each.  T = 0 or
 * batch = 0 is a no-op. */
sink_attn_status sink_attn_paged_attn(const sink_attn_paged_dims* dims,
                                      const void* q, const void* k_cache, const void* v_cache,
                                      const int* block_table, const int* cu_seqlens, const int* kv_lens,
                                      const float* sinks, int window, float scale,
                                      void* out, float* lse,
                                      void* workspace, size_t workspace_bytes, void* stream);

/* The same over e4m3 codes: key = code * k_scale[g], value = code * v_scale[g]
 * (fp32 [Hkv], device, > 0).  Codes are widened to fp16, exactly; q is rounded to
 * fp16 (exact from 2^-14 up to 65504, where it saturates), and so are the
 * softmax weights. */
sink_attn_status sink_attn_paged_attn_e4m3(const sink_attn_paged_dims* dims,
                                           const void* q, const void* k_cache, const void* v_cache,
                                           const int* block_table, const int* cu_seqlens, const int* kv_lens,
                                           const float* k_scale, const float* v_scale,
                                           const float* sinks, int window, float scale,
                                           void* out, float* lse,
                                           void* workspace, size_t workspace_bytes, void* stream);

/* Human-readable name of a status code (static string, never NULL). */
const char* sink_attn_status_string(sink_attn_status s);

/* Synchronises `stream` (a cudaStream_t passed as void*), then returns and
 * clears a device error code recorded on the current device: 0 = none, -1 = the
 * synchronisation or the read failed.  There are two records, of the first wait
 * that timed out (0x1..) and of the first input that a kernel found wrong
 * (0x2..: a decode ring too small for its window, a pool that ran dry and so
 * on); a time-out is returned first, and the other by the call after that.
 * These are the only entry points that synchronise.  sink_attn_device_error is
 * the same function under a shorter name. */
int sink_attn_last_device_error(void* stream);
int sink_attn_device_error(void* stream);

/* Self-test of the bounded device waits (failure detection without a fault):
 * one block waits on mbarriers that nothing completes.  One thread gives up
 * after limit_ns (0 < limit_ns <= 1 s), records error code 0x107 and raises
 * the block's abort flag; a thread of another warp, waiting with ten times
 * that limit, must leave through the flag without recording its own code
 * (0x108).  `out`: device pointer to 4 ints (4-byte aligned), written as
 * {first wait returned true, its microseconds, second wait returned true,
 * its microseconds}.  Asynchronous on `stream`; read the recorded code with
 * sink_attn_device_error().  Returns SINK_ATTN_ERR_ALIGN for a NULL or
 * misaligned `out`, SINK_ATTN_ERR_SHAPE for a limit outside the range. */
sink_attn_status sink_attn_selftest_wait(unsigned long long limit_ns, int* out, void* stream);

/* Profiling aid.  Registers two CUDA events (cudaEvent_t passed as void*)
 * that later calls record on their stream immediately before and after one
 * kernel launch: which = 0 -> the forward kernel of sink_attn_fwd,
 * which = 1 -> the main (tensor-core) kernel of sink_attn_bwd.  Passing NULL
 * events clears the slot.  Process-wide and not thread-safe; the events stay
 * owned by the caller.  Returns SINK_ATTN_ERR_SHAPE for an unknown `which`. */
sink_attn_status sink_attn_profile_events(int which, void* ev_begin, void* ev_end);

/* Number of kernels one sink_attn_fwd / sink_attn_bwd call launches for
 * these sizes (0 when T = 0). */
int sink_attn_fwd_launches(const sink_attn_dims* dims);
int sink_attn_bwd_launches(const sink_attn_dims* dims);

#ifdef __cplusplus
}
#endif

#endif /* SINK_ATTN_H_ */
