/*
 * vericache.h -- C ABI of the VeriCache draft/verify hot path for NVIDIA B200 (sm_100a).
 *
 * The operations follow two web summaries:
 *   [VC]  "Riepilogo Tecnico: VeriCache" (gist.science/it/paper/2605.17613; Arabic
 *         translation gist.science/ar/paper/2605.17613): draft over the compressed
 *         cache, verify all drafts in one pass over the full cache, greedy acceptance
 *         with a bonus token, and streaming of the full cache from CPU memory over
 *         PCIe overlapped with other requests' drafting.
 *   [CKV] "Riassunto Tecnico: CentroidKV" (gist.science/it/paper/2506.11418): per-slot
 *         degree n_t that enters the softmax as a logarithmic term.
 *
 * Conventions for every call:
 *   - All tensor pointers are DEVICE pointers owned by the caller, except the host
 *     source of vc_stage_full_kv.  The library allocates nothing; scratch space is a
 *     caller-provided workspace whose size the matching *_workspace_size call gives.
 *   - bf16 tensors are IEEE bfloat16 (2 bytes), fp16 tensors IEEE half.  Shapes are
 *     row-major and contiguous unless a capacity (…_cap) gives the row stride.
 *   - Calls only enqueue work on the given stream and return at once.  The return
 *     code covers argument validation and launch errors; errors found on the device
 *     (out-of-range slot indices, NaN logits) are written to caller-provided flags
 *     that the caller reads after synchronising.
 *   - Every pointer passed to a kernel must be 16-byte aligned.
 *   - There is no fallback path: an unsupported shape returns VC_ERR_UNSUPPORTED.
 */
#ifndef VERICACHE_H
#define VERICACHE_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define VC_ABI_VERSION 1

typedef enum {
  VC_OK = 0,
  VC_ERR_INVALID = 1,      /* bad argument: NULL, negative size, misaligned, … */
  VC_ERR_UNSUPPORTED = 2,  /* valid but not implemented (e.g. head dim 96) */
  VC_ERR_CUDA = 3,         /* a CUDA runtime call or launch failed */
  VC_ERR_TIMEOUT = 4       /* a bounded host wait ran out */
} vc_status;

typedef enum {
  VC_CACHE_INDEXED = 0,    /* bf16 rows picked by a slot index list, with degrees */
  VC_CACHE_INT4 = 1        /* 4-bit group-quantised rows (see the layout below) */
} vc_cache_kind;

/* Human-readable name of a status code (static string). */
const char* vc_status_string(int status);
/* Detail of the last failing call in this thread (static thread-local buffer). */
const char* vc_last_error(void);
/* VC_ABI_VERSION of the loaded library. */
int vc_abi_version(void);

/* ------------------------------------------------------------------------------
 * Compressed cache KV_comp of one attention layer ([VC] "Algoritmo Principale",
 * step 1; [VC] "Supporto Architetturale": one interface for eviction and
 * quantisation compressors).
 *
 * Common:  B batch, Hq query heads, Hkv kv heads (Hq % Hkv == 0, g = Hq/Hkv <= 8),
 *          D head dim in {64, 128}.  Query head h reads kv head h / g.
 * Tail:    k_tail, v_tail bf16 [B, Hkv, R_cap, D]; the first n_tail rows are live
 *          (tokens appended while drafting), each of degree 1.  May be NULL when
 *          n_tail == 0.
 *
 * VC_CACHE_INDEXED (token eviction, optionally merged centroids):
 *   k, v      bf16 [B, Hkv, T_cap, D]  base rows (a full cache viewed through idx,
 *                                      or compact slot rows when idx == NULL)
 *   idx       int32 [B, Hkv, S_cap]    base row of slot s, 0 <= idx < T_cap; NULL
 *                                      means slot s is row s (needs S <= T_cap)
 *   deg       int32 [B, Hkv, S_cap]    degree n_s >= 1 of slot s ([CKV] item 4:
 *                                      score += ln n_s); NULL means all 1
 *   S         live slots per (batch, kv head), same for all
 *   err_flag  int32 [1] or NULL: set to 1 when an idx entry is out of range (the
 *             entry is clamped and the result is then meaningless) or a degree < 1
 *
 * VC_CACHE_INT4 (asymmetric 4-bit groups; x_hat = q * scale + zero):
 *   Per (batch, kv head) the S quantised tokens (S % 32 == 0, capacity T_cap tokens,
 *   T_cap % 32 == 0) form blocks of 32.  Words are little-endian uint32 of 8 nibbles
 *   (nibble p at bits 4p..4p+3); pair j (0..3) of a word keeps its first element in
 *   nibble j and its second in nibble j + 4.
 *   kq        uint32 [B, Hkv, T_cap/32, 32, 4, D/32]: pair j of word (token t, c, w)
 *             holds channels e, e+1 of token t, e = 2c + 32w + 16*(j/2) + 8*(j%2)
 *   k_scale, k_zero  fp16 [B, Hkv, T_cap/32, D]: one group per (block, channel)
 *   vq        uint32 [B, Hkv, T_cap/32, D, 4]: pair j of word (channel d, c) holds
 *             channel d of tokens 2c + 8j and 2c + 8j + 1 of the block
 *   v_scale, v_zero  fp16 [B, Hkv, T_cap/32, D/32, 32]: one group per (token,
 *             32 consecutive channels), stored block, channel group, token
 *   All quantised tokens have degree 1.
 * ---------------------------------------------------------------------------- */
typedef struct vc_comp_cache {
  int32_t kind;                 /* vc_cache_kind */
  int32_t B, Hq, Hkv, D;
  int32_t S;                    /* live slots (indexed) or quantised tokens (int4) */
  int32_t S_cap;                /* row stride of idx / deg (indexed) */
  int64_t T_cap;                /* base rows (indexed) or token capacity (int4) */
  /* VC_CACHE_INDEXED */
  const void* k;
  const void* v;
  const int32_t* idx;
  const int32_t* deg;
  /* VC_CACHE_INT4 */
  const uint32_t* kq;
  const void* k_scale;
  const void* k_zero;
  const uint32_t* vq;
  const void* v_scale;
  const void* v_zero;
  /* tail */
  const void* k_tail;
  const void* v_tail;
  int32_t R_cap;
  int32_t n_tail;
  /* device error flag, may be NULL */
  int32_t* err_flag;
} vc_comp_cache;

/* Output precision flag shared by the attention calls: write `out` as fp32 instead of
 * bf16 (the fp32 value is the one the bf16 output is rounded from, to nearest even). */
#define VC_OUT_F32 4

/* ------------------------------------------------------------------------------
 * Draft attention: one decode step of every query head over KV_comp plus the tail
 * ([VC] "Algoritmo Principale", step 1, with the [CKV] log-degree term):
 *   s_t = (q . k_t) * scale + ln n_t ;  o = sum_t softmax(s)_t v_t
 *   q    bf16 [B, Hq, D]            out  bf16 [B, Hq, D] (fp32 with flags & VC_OUT_F32)
 *   lse  fp32 [B, Hq] or NULL: ln sum_t exp(s_t)
 *   scale <= 0 selects D^-1/2.
 * Split-K over slots: ws must hold vc_draft_workspace_size(cache) bytes (device).
 * S + n_tail must be >= 1.
 * ---------------------------------------------------------------------------- */
size_t vc_draft_workspace_size(const vc_comp_cache* cache);
vc_status vc_draft_attn(const void* q, const vc_comp_cache* cache, float scale, int flags,
                        void* out, float* lse, void* ws, size_t ws_bytes,
                        cudaStream_t stream);

/* Draft attention that allocates nothing and takes no workspace (the pages have no
 * counterpart: this serves callers that cannot hand the library scratch memory, such as
 * a plugin whose host runtime owns all device memory and offers no allocator, a process
 * whose memory pool is fully reserved up front, or a path that must not call cudaMalloc
 * because it can block and synchronise the device).  Same arguments and result as
 * vc_draft_attn, without ws / ws_bytes: the split-K partials go to a fixed 8 MiB array in
 * the library's device image, which every GPU that loads the library holds until exit.
 *   - A cache whose partials need more than 8 MiB (vc_draft_workspace_size) is rejected
 *     with VC_ERR_UNSUPPORTED before anything is launched.
 *   - The first call on each device does a one-time set-up (it looks up the array's
 *     device address with that device current); make that first call before any stream
 *     capture begins.  The address is kept per CUDA context, so the set-up runs again
 *     on the first call after a cudaDeviceReset or under another context.
 *   - All calls on a device share the one array and it keeps the last call's contents
 *     (nothing in it needs to start at zero).  Calls that overlap on the GPU -- on
 *     different streams, or from different threads -- race on it: serialise them. */
vc_status vc_draft_attn_noalloc(const void* q, const vc_comp_cache* cache, float scale,
                                int flags, void* out, float* lse, cudaStream_t stream);

/* ------------------------------------------------------------------------------
 * Verify attention ([VC] "Algoritmo Principale", step 2: one pass over KV_full checks
 * all drafted tokens in parallel).  Row i (0 <= i < n_q, n_q = k + 1: the pending
 * token and the k drafts) sits at absolute position P + i and attends every key at
 * position <= P + i: the prefix plus the block, causal inside the block.  No degree
 * term.
 *   q     bf16 [B, n_q, Hq, D]
 *   k, v  bf16 [B, Hkv, L_cap, D]: row r holds the key / value at absolute position
 *         kv_start + r, for r < kv_len (kv_len <= L_cap).  The block's own keys
 *         (positions P .. P+n_q-1) must already be written where they fall.
 *   Single pass (m == l == acc == NULL): kv_start == 0, kv_len == P + n_q; writes out
 *         bf16 [B, n_q, Hq, D] (fp32 with flags & VC_OUT_F32).
 *   Chunked (long context with KV_full streamed from host memory, [VC] "Supporto
 *         Architetturale"): m, l fp32 [B, n_q, Hq] and acc fp32 [B, n_q, Hq, D] carry
 *         the softmax state (running max of s * log2(e), sum of 2^(s*log2(e) - max),
 *         weighted values) between
 *         calls over consecutive key ranges in increasing kv_start.  VC_VERIFY_FIRST
 *         resets the state before adding this range; VC_VERIFY_LAST writes out after
 *         adding it.  Ranges must tile [0, P + n_q) exactly, in order.
 *   Results do not depend on n_q or on other rows: key tiles and split boundaries sit
 *   at fixed absolute positions, and splits are merged in a fixed order.  The split
 *   window (a multiple of 64 keys in [2048, 4096]; 4096 when B * Hkv * L_cap / 4096 is
 *   under one CTA per SM) is chosen from B * Hkv and L_cap only, so that the CTAs fill the
 *   SMs' last wave; every call on one cache uses the same one.
 *   ws: vc_verify_workspace_size(...) bytes of device memory (enough for any window).
 *   Supported: D in {64, 128}, g <= 8, n_q * g <= 1024.
 * ---------------------------------------------------------------------------- */
#define VC_VERIFY_FIRST 1
#define VC_VERIFY_LAST 2
size_t vc_verify_workspace_size(int B, int n_q, int Hq, int Hkv, int D,
                                int64_t kv_start, int64_t kv_len);
vc_status vc_verify_attn(const void* q, int B, int n_q, int Hq, int Hkv, int D,
                         const void* k, const void* v, int64_t L_cap,
                         int64_t kv_start, int64_t kv_len, int64_t P,
                         float* m, float* l, float* acc, int flags, float scale,
                         void* out, void* ws, size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------------
 * Greedy acceptance ([VC] "Algoritmo Principale", step 3).
 *   logits  fp32 [B, n_q, V]; drafts int32 [B, n_q - 1] or NULL
 *   target[b, i] = argmax_v logits[b, i, v] (ties: lowest v; a NaN counts as larger
 *                  than any number, the first NaN wins)           int32 [B, n_q]
 *   accept_len[b] = a = first i < n_q-1 with target[b,i] != drafts[b,i], else n_q-1
 *   commit[b, :] = target[b, 0..a], then -1                        int32 [B, n_q]
 *   n_commit[b] = a + 1 (a == n_q-1: every draft plus the bonus token)
 *   err_flag[b] = 1 if row b had a NaN, else 0                    int32 [B] or NULL
 * With accept_len == commit == n_commit == NULL only target (and err_flag) are written
 * (the argmax of each draft step) and drafts is not read.  Otherwise all three must be
 * set and drafts must be non-NULL unless n_q == 1 (no drafts: a = 0).
 * ---------------------------------------------------------------------------- */
vc_status vc_accept(const float* logits, const int32_t* drafts, int B, int n_q, int V,
                    int32_t* target, int32_t* accept_len, int32_t* commit,
                    int32_t* n_commit, int32_t* err_flag, cudaStream_t stream);

/* ------------------------------------------------------------------------------
 * Staging of KV_full from pinned host memory to HBM over PCIe on a side stream
 * ([VC] "Scaglionamento tra Risorse (P1)" and "Supporto Architetturale": the full
 * cache lives in CPU memory and verification loads it over PCIe while other
 * requests draft).  Copies [0, bytes) of src to dst in chunks of chunk_bytes with
 * one cudaMemcpyAsync each (copy engine, no SMs) and records chunk_done[i] after
 * chunk i, so a verify call on another stream can wait on exactly its chunk.
 *   src_host must be page-locked (cudaHostAlloc / cudaHostRegister): checked.
 *   chunk_done may be NULL (n_events == 0); otherwise n_events >= number of chunks.
 * ---------------------------------------------------------------------------- */
vc_status vc_stage_full_kv(void* dst_dev, const void* src_host, size_t bytes,
                           size_t chunk_bytes, cudaStream_t copy_stream,
                           cudaEvent_t* chunk_done, int n_events);

/* Host wait on an event with a time limit (polls cudaEventQuery).  Returns VC_OK,
 * VC_ERR_TIMEOUT after timeout_s seconds, or VC_ERR_CUDA. */
vc_status vc_event_wait(cudaEvent_t ev, double timeout_s);

/* ----------------------------------------------------------------------------
 * One round of Chunked Soft Matching: CentroidKV's one-pass clustering of a KV cache
 * ([CKV] "Riassunto Tecnico: CentroidKV", section "Metodologia", items 2-4).  For each
 * (batch, kv head) pair, rows [0, n_sinks) and [T - n_recent, T) are kept as they are;
 * the rows between are cut into consecutive chunks of `chunk` rows (the last may be
 * shorter).  In a chunk, A = rows at even offsets, B = rows at odd offsets; each A row is
 * matched to its most similar B row by cosine of the key rows (lowest B row on ties; an
 * all-zero row has cosine 0 with everything); the m = floor(r * |A|) A rows with the
 * highest similarity (lower row on ties) merge into their matches.  A B row and the A
 * rows merged into it become one centroid: K and V = degree-weighted means (fp32 sums,
 * the B row first, then its A rows in ascending order, rounded to bf16 once), degree =
 * the sum.  A one-row chunk (no B row) merges nothing.  Output order: sinks, each chunk's surviving rows in their order (a centroid in
 * its B row's place), recent rows.  The result is a compact cache (idx = NULL, deg =
 * deg_out) for vc_draft_attn.  A decreasing r over successive rounds (r_j = r_init -
 * j * delta_r) is the caller's schedule.  Similarities use bf16 products with fp32
 * accumulation; a near-tie may resolve either way.
 *
 *   k, v      bf16 [pairs, T_cap, D] (device), the cache rows [0, T) of each pair
 *   deg       int32 [pairs, T_cap] degrees >= 1, or NULL (all 1)
 *   k_out, v_out  bf16 [pairs, T_cap_out, D]; deg_out int32 [pairs, T_cap_out]
 *             (must not overlap the inputs); rows [0, vc_csm_out_len(...)) are written
 *   dest      int32 [pairs, T_cap] or NULL: output row of every input row (the
 *             centroid's row for a merged row)
 *   D in {64, 128}; 2 <= chunk <= 256; 0 <= r <= 1; n_sinks + n_recent <= T <= T_cap;
 *   T < 2^31; pairs <= 65535; pointers 16-byte aligned.
 * ---------------------------------------------------------------------------- */
int64_t vc_csm_out_len(int64_t T, int n_sinks, int n_recent, int chunk, double r);
vc_status vc_csm_compress(const void* k, const void* v, const int32_t* deg, int pairs, int D,
                          int64_t T, int64_t T_cap, int n_sinks, int n_recent, int chunk,
                          double r, void* k_out, void* v_out, int32_t* deg_out,
                          int64_t T_cap_out, int32_t* dest, cudaStream_t stream);

/* ----------------------------------------------------------------------------
 * Int4 compressor: quantise whole 32-token blocks of bf16 K/V rows into the
 * VC_CACHE_INT4 layout above ([VC] "Supporto Architetturale": quantisation plugs into
 * the uniform compression interface; [CKV] "Problematica": quantisation among the known
 * KV-cache reductions).  Groups as in the layout: keys per channel over the block's 32
 * tokens, values per token over 32 consecutive channels;
 *     z = fp16(min), s = fp16((max - min) / 15) (1 if that is 0),
 *     n = clamp(rint((x - z) / s), 0, 15), round half to even, in fp64.
 * This is how tokens leaving a bf16 window join the quantised part of the cache: call it
 * on each 32 rows that leave, with blk0 = the next free block.
 *   k, v      bf16 [pairs, src_cap, D]; rows src_t0 .. src_t0 + 32 n_blocks - 1 of every
 *             pair are read
 *   kq, k_scale, k_zero, vq, v_scale, v_zero: the int4 arrays with capacity blk_cap
 *             blocks per pair (T_cap = 32 blk_cap); blocks blk0 .. blk0 + n_blocks - 1
 *             of every pair are written, nothing else
 *   D in {64, 128}; pairs <= 65535; pointers (and row src_t0) 16-byte aligned.
 *   Groups with values beyond the fp16 range cannot be represented (result unspecified).
 * ---------------------------------------------------------------------------- */
vc_status vc_int4_quantize(const void* k, const void* v, int pairs, int D, int64_t src_cap,
                           int64_t src_t0, int n_blocks, uint32_t* kq, void* k_scale,
                           void* k_zero, uint32_t* vq, void* v_scale, void* v_zero,
                           int64_t blk_cap, int64_t blk0, cudaStream_t stream);

/* ----------------------------------------------------------------------------
 * Token eviction by attention score ([CKV] "Problematica": eviction drops the tokens
 * with the lowest attention scores; [CKV] "Metodologia" item 2 "Preservazione": sinks and
 * recent tokens are always kept; [VC] "Supporto Architetturale": eviction compressors
 * plug into the same interface).
 *
 * vc_evict_scores: for a prompt of n tokens, the attention mass each key receives from
 * the last W prompt queries over the g query heads of its kv head:
 *     score[b, j, t] = sum_{w < W, h in group j} softmax_{t' <= n-W+w}(q . k_t' * scale)[t]
 *   q      bf16 [B, W, Hq, D]: the queries of positions n-W .. n-1 (as attention sees
 *          them, i.e. after any rotary embedding)
 *   k      bf16 [B, Hkv, L_cap, D]: keys of positions 0 .. n-1 in rows 0 .. n-1
 *   score  fp32 [B, Hkv, score_cap], entries [0, n) written (each a fixed-order fp32 sum)
 *   ws     device workspace of vc_evict_workspace_size(B, W, Hq) bytes
 *   scale <= 0 selects D^-1/2.  D in {64, 128}, g <= 8, W <= 32, W <= n <= L_cap.
 *
 * vc_evict_select: per row r (e.g. (batch, kv head)) of score [rows, score_cap], the kept
 * positions in ascending order: [0, n_sinks), then the budget - n_sinks - n_recent
 * highest-scoring positions of [n_sinks, n - n_recent) (equal scores: the lower position
 * first), then [n - n_recent, n); budget >= n keeps 0 .. n-1.  Writes idx int32
 * [rows, S_cap], entries [0, min(budget, n)).  Exact: depends only on the scores' order.
 * ---------------------------------------------------------------------------- */
size_t vc_evict_workspace_size(int B, int W, int Hq);
vc_status vc_evict_scores(const void* q, int B, int W, int Hq, int Hkv, int D, const void* k,
                          int64_t L_cap, int64_t n, float scale, float* score,
                          int64_t score_cap, void* ws, size_t ws_bytes, cudaStream_t stream);
vc_status vc_evict_select(const float* score, int rows, int64_t score_cap, int64_t n,
                          int budget, int n_sinks, int n_recent, int32_t* idx, int64_t S_cap,
                          cudaStream_t stream);

/* ----------------------------------------------------------------------------
 * Paged cache: K and V rows of B sequences of different lengths in pages of a shared
 * pool, for serving (the full cache of one attention layer, or a lighter copy of it with
 * 8-bit rows; [VC] "Supporto Architetturale": caches plug into one interface).
 *
 *   type         VC_PAGE_BF16, or 8-bit rows with one fp32 scale per (token, kv head) of K
 *                and of V: VC_PAGE_E4M3 (8-bit float, 4 exponent and 3 fraction bits) or
 *                VC_PAGE_INT8; the row's value is code * scale
 *   B, Hkv, D    sequences, kv heads (65535 each at most), head dim in {64, 128}
 *   page         tokens per page: 16, 32, 64, 128 or 256
 *   n_pages      pages of the pool; max_pages: columns of page_table (n_pages * page and
 *                max_pages * page at most 2^31 - 2^16)
 *   k, v         the pools [n_pages, Hkv, page, D] by strides: element (p, h, t, d) at
 *                p * page_stride + h * head_stride + t * row_stride + d, strides counted in
 *                elements; 16-byte aligned base, each stride a positive multiple of 16 bytes
 *                (a stride whose dimension has one entry is not read)
 *   k_scale, v_scale  fp32 [n_pages, Hkv, page] contiguous, > 0 (8-bit types; else NULL).
 *                Attention may take a value scale under 2^-90 as 2^-90 (few rows do).
 *   page_table   int32 [B, max_pages]: position t of sequence b is row t % page of page
 *                page_table[b, t / page]; entries past the sequence's last page are not read
 *   kv_len       int32 [B]: tokens of each sequence, the new ones of a call included
 *   err_flag     int32 [1] or NULL; the calls OR bits into it (the caller zeroes it):
 *                VC_PAGED_BAD_PAGE    a page id outside [0, n_pages): such a page is not
 *                                     written, reads as rows of zeros
 *                VC_PAGED_BAD_LENGTH  a kv_len outside [0, max_pages * page], or cu_q not
 *                                     ascending within [0, N] (each is clamped)
 *                VC_PAGED_NOT_FINITE  (vc_paged_write, 8-bit types) a NaN or infinity in a
 *                                     written row: the scale comes from the finite values,
 *                                     an infinity takes the largest code, a NaN the NaN
 *                                     code (e4m3) or 0 (int8)
 *
 * New tokens of a call (queries, or K/V rows to write) lie one after the other: sequence b
 * has rows cu_q[b] .. cu_q[b + 1] - 1 of N (cu_q int32 [B + 1] on the device, ascending), or
 * N / B rows each when cu_q is NULL (then N % B == 0).  With n_b rows, row i of sequence b
 * is at position kv_len[b] - n_b + i.  Rows from cu_q[B] on are neither read nor written.
 * kv_len[b] < n_b is allowed: rows at negative positions see nothing and are not written to
 * the cache.  A sequence may have no rows or no tokens.
 * ---------------------------------------------------------------------------- */
typedef enum {
  VC_PAGE_BF16 = 0,
  VC_PAGE_E4M3 = 1,
  VC_PAGE_INT8 = 2
} vc_page_type;

#define VC_PAGED_BAD_PAGE 1
#define VC_PAGED_BAD_LENGTH 2
#define VC_PAGED_NOT_FINITE 4

typedef struct vc_paged_cache {
  int32_t type;                 /* vc_page_type */
  int32_t B, Hkv, D;
  int32_t page, n_pages, max_pages;
  void* k;
  void* v;
  int64_t k_page_stride, k_head_stride, k_row_stride;
  int64_t v_page_stride, v_head_stride, v_row_stride;
  float* k_scale;
  float* v_scale;
  const int32_t* page_table;
  const int32_t* kv_len;
  int32_t* err_flag;
} vc_paged_cache;

/* Write new K and V rows into their pages.  k, v bf16 [N, Hkv, D]: row i, head h at
 * i * tok_stride + h * head_stride elements (multiples of 8; 16-byte aligned base), so they
 * may be parts of a fused projection.  bf16 pages take the rows as they are.  8-bit pages:
 *     a = max |x| over the row's D values;  scale = a / top  (fp32; 1 if a == 0),
 *     code = round(x * top / a) to nearest even,  top = 448 (e4m3) or 127 (int8).
 * Two rows of a call must not fall on one slot (sequences share only pages that no call
 * writes). */
vc_status vc_paged_write(const vc_paged_cache* cache, const void* k, int64_t k_tok_stride,
                         int64_t k_head_stride, const void* v, int64_t v_tok_stride,
                         int64_t v_head_stride, int N, const int32_t* cu_q,
                         cudaStream_t stream);

/* Read rows back into a contiguous bf16 cache (the layout of vc_verify_attn and of the
 * compressors): row r of k_out, v_out bf16 [B, Hkv, T_cap, D] becomes position start + r
 * of the sequence (8-bit rows: the fp32 product code * scale, rounded to bf16), for
 * 0 <= r < T_cap and 0 <= start + r < kv_len[b]; other rows are left as they were.  start is
 * starts[b] (device int32 [B]) or start0 when starts is NULL. */
vc_status vc_paged_read(const vc_paged_cache* cache, int64_t start0, const int32_t* starts,
                        void* k_out, void* v_out, int64_t T_cap, cudaStream_t stream);

/* Attention of the new tokens over the paged cache (their own K/V written before): row i
 * of sequence b attends the keys at positions <= kv_len[b] - n_b + i,
 *     s_t = (q . k_t) * scale,  o = sum_t softmax(s)_t v_t,  lse = ln sum_t exp(s_t);
 * a row that sees no key gets o = 0, lse = -inf.
 *   q    bf16 [N, Hq, D]: token i, head h at i * q_tok_stride + h * q_head_stride elements
 *        (multiples of 8; 16-byte aligned base); Hq % Hkv == 0, any group size
 *   max_q  an upper bound on the rows of any sequence, or <= 0 when none is known (N then).
 *        A sequence with more rows is flagged (VC_PAGED_BAD_LENGTH) and may be left out.
 *   out  bf16 [N, Hq, D] (fp32 with flags & VC_OUT_F32), contiguous; lse fp32 [N, Hq] or NULL
 *   ws   device workspace of vc_paged_attn_workspace_size(cache, N, Hq, max_q) bytes (at
 *        present a function of D and of the device's SM count alone, of nothing on the
 *        device); calls that may run at the same time need workspaces of their own
 *   scale <= 0 selects D^-1/2.
 * The keys of each (sequence, kv head, row group) are dealt to the SMs in equal parts
 * computed on the device from the lengths, so the call can be captured in a CUDA graph and
 * replayed for other lengths.  Scores and softmax sums are fp32; weights enter P V in bf16
 * (fp16 for 8-bit rows of small blocks).  Results are the same for every run of the same
 * call, but the way the keys are split, and with it the last bits, depends on the batch.
 * Keys and values of live positions must be finite; those of other slots may hold
 * anything.  (A NaN in a live row, the e4m3 code for it included, reaches every row that sees
 * it; in a value also rows before it in the same call.)  A score that passes fp32's range,
 * before or after scale, makes its row NaN (+inf), and a row whose scores are all -inf counts as
 * one that sees no key.  Values are summed in fp32 at up to 2^8 times their weight before the
 * division, so |v| times the number of keys has to stay under 2^120. */
size_t vc_paged_attn_workspace_size(const vc_paged_cache* cache, int N, int Hq, int max_q);
vc_status vc_paged_attn(const vc_paged_cache* cache, const void* q, int64_t q_tok_stride,
                        int64_t q_head_stride, int N, int Hq, const int32_t* cu_q, int max_q,
                        float scale, int flags, void* out, float* lse, void* ws,
                        size_t ws_bytes, cudaStream_t stream);

/* ----------------------------------------------------------------------------
 * Acceptance by sampling: drafted tokens are checked against the target's probabilities
 * with given random numbers, so that the committed tokens are distributed as samples of
 * the target (the counterpart of vc_accept for users who sample).  With
 * p_i = softmax(logits[b, i] / T), q_i = softmax(draft_logits[b, i] / T):
 *     a = first i < n with not (u[b, i] * q_i(d_i) < p_i(d_i)), else n   (n = n_drafts[b])
 *     commit[b, :] = d_0 .. d_(a-1), x, then -1;  accept_len[b] = a;  n_commit[b] = a + 1
 *     x = the first index whose running sum of w exceeds u[b, n_q - 1] times the total of w,
 *     w = max(p_a - q_a, 0) if a < n (p_a if that is 0 everywhere), p_n if a == n.
 * draft_logits NULL: q_i is 1 at d_i (drafts of a greedy drafter).  T = 0 (or under 2^-60):
 * p_i is 1 at the first largest logit and q_i at d_i (greedy acceptance).
 *   logits  fp32, or bf16 with flags & VC_LOGITS_BF16, [B, n_q, V]; draft_logits [B, n_q - 1, V]
 *           of the same type or NULL; both with a 16-byte aligned base (a part of a batch with
 *           odd V may not have one: refused); -inf marks a token that cannot be drawn, and a
 *           logit further below its row's largest than fp32's range may count as one
 *   drafts  int32 [B, n_q - 1] (may be NULL when n_q == 1)
 *   u       fp64 [B, n_q], each in [0, 1): entries 0 .. n_q - 2 decide the drafts, the last
 *           draws x
 *   temperature  fp32 [B] or NULL (1); n_drafts int32 [B] or NULL (n_q - 1)
 *   accept_len int32 [B], commit int32 [B, n_q], n_commit int32 [B]
 *   err_flag int32 [B] or NULL: 0, or 1 if something was not valid: a draft outside [0, V)
 *           (refused), n_drafts outside [0, n_q - 1] (clamped), a temperature that is
 *           negative or not finite (taken as 0), a target row that was looked at (positions
 *           0 .. a) with a NaN, a +inf or nothing above -inf (its draft is refused and x is
 *           vc_accept's argmax of that row), a draft row with the same (q_i is 1 at d_i)
 *   ws      vc_accept_sample_workspace_size(...) bytes, 16-byte aligned; B <= 65535, n_q <= 257,
 *           V < 2^31 - 2^16
 * The same inputs give the same tokens.  The running sums that x is picked by are fp64; the sums
 * that turn logits into p_i(d_i) and q_i(d_i) are of fp32 terms, off by some 1e-7 of their value
 * (under 1e-5 for 128K tokens), so that a draft with u q_i(d_i) that near to p_i(d_i) may be
 * decided the other way.
 * ---------------------------------------------------------------------------- */
#define VC_LOGITS_BF16 8
size_t vc_accept_sample_workspace_size(int B, int n_q, int V);
vc_status vc_accept_sample(const void* logits, const void* draft_logits, const int32_t* drafts,
                           const double* u, const float* temperature, const int32_t* n_drafts,
                           int B, int n_q, int V, int flags, int32_t* accept_len,
                           int32_t* commit, int32_t* n_commit, int32_t* err_flag, void* ws,
                           size_t ws_bytes, cudaStream_t stream);

/* The library's device error word on the current device (synchronous read; clear != 0
 * resets it).  Bit 0: a bounded wait inside a verify-attention CTA expired (the call's
 * output is then invalid; the CTA released its resources and exited).  Bit 1: the same in
 * paged attention. */
vc_status vc_device_error(int32_t* value, int clear);

/* Failure detection (no counterpart in the pages).  Sets the time limit of every
 * pipeline wait inside the verify and paged attention kernels for the launches that follow
 * (a process-wide setting; default 2 s; seconds == 0 restores it; at most 60 s) and
 * returns the previous limit in *previous (may be NULL).  A wait that runs out raises its
 * bit of the device error word and the CTA exits cleanly, leaving the context usable;
 * a very short limit makes that happen on purpose, which is how the error path is tested
 * without any device fault.
 * Staging has a host-side injection point for the same purpose: with the environment
 * variable VC_FAULT_INJECT=stage_fail, vc_stage_full_kv returns VC_ERR_CUDA before
 * enqueueing anything. */
vc_status vc_set_wait_limit(double seconds, double* previous);

#ifdef __cplusplus
}
#endif
#endif /* VERICACHE_H */
