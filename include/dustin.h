/*
 * dustin.h -- C ABI of the GB300 (sm_103a) sparse-verification hot path.
 *
 * The calls follow the method described in "Technical Summary: Dustin"
 * (gist.science/paper/2606.24957):
 *   dustin_score       section 1 "Hybrid Attention Aggregation" + section 2
 *                      "Efficient Estimation via Semantic Retrieval Heads":
 *                      draft-look-ahead and target-historical attention on a few
 *                      SRH heads, summed into a global per-token importance map.
 *   dustin_select      section 1: fixed-size verification set I_verify -- a
 *                      protected sink prefix and recent window, then the top-m
 *                      tokens by the draft signal, then the rest of the budget by
 *                      the target signal.
 *   dustin_verify_attn section 3 "Verification Workflow", steps 3-4: the target
 *                      verifies the gamma+1 draft/bonus queries against the
 *                      selected rows only.
 *   dense_verify_attn  "Problem Statement": standard verification that loads
 *                      the full KV cache (the comparator).
 *   dustin_kv_append   section 3, step 5: accepted tokens are appended.
 *   dustin_verify_step score -> select -> verify in one call on one stream.
 * Beside them, not in the pages: attention through a sliding window with sinks
 * (dustin_window_attn) and behind a prefix that a batch shares
 * (dustin_prefix_attn), and caches bounded by accumulated attention weight
 * (dustin_accumulate, dustin_evict); and a cache in pages for ragged batches
 * (dustin_page_map, dustin_norm_rope, dustin_paged_attn).
 *
 * Conventions (all calls):
 *  - The caller owns every buffer.  Pointers named "device" are CUDA device
 *    pointers; "host" arrays are read during the call only.  No call allocates
 *    device memory: scratch lives in a caller-provided workspace of
 *    dustin_workspace_bytes() bytes (256-byte aligned), initialised once with
 *    dustin_workspace_init().
 *  - Arguments are validated on the host before anything is launched; on any
 *    error the call returns a negative dustin_status and launches nothing.
 *  - Work is enqueued asynchronously on the given stream.  Kernels never trap:
 *    device-side anomalies (an index outside the context, a NaN importance
 *    value, an append past the capacity, a bounded wait that gave up) set bits
 *    of a sticky error word in the workspace, read by dustin_check().
 *  - bf16 tensors are raw bf16 bit patterns; fp32 outputs are IEEE floats.
 *  - Context length per sequence is the device array seq_len[B]; positions at
 *    or beyond seq_len[b] are never read.
 *  - No call is thread-safe with respect to a shared workspace.
 */
#ifndef DUSTIN_H
#define DUSTIN_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DUSTIN_OK = 0,
  DUSTIN_EINVAL = -1,     /* bad argument: null pointer, size, stride, alignment */
  DUSTIN_ERANGE = -2,     /* a size beyond the library's limits (see DUSTIN_MAX_*) */
  DUSTIN_ECUDA = -3,      /* a CUDA runtime/driver call failed */
  DUSTIN_EDEVICE = -4,    /* dustin_check: a kernel flagged an anomaly */
  DUSTIN_EWORKSPACE = -5  /* workspace null, misaligned or smaller than required */
} dustin_status;

/* Bits of the device error word (dustin_check). */
#define DUSTIN_DEV_INDEX   1   /* an I_verify entry outside [-1, seq_len[b]) (skipped) */
#define DUSTIN_DEV_NAN     2   /* a NaN or negative importance value (ranked as 0) */
#define DUSTIN_DEV_APPEND  4   /* n_accept outside [0, gamma+1] or append past Lcap (skipped) */
#define DUSTIN_DEV_TIMEOUT 8   /* a bounded wait on an on-chip barrier gave up */
#define DUSTIN_DEV_SEQLEN 16   /* seq_len[b] outside [0, Lcap] (sequence skipped) */
#define DUSTIN_DEV_PAGES  32   /* a pool with too few free pages, or whose counts are inconsistent */

/* Limits. */
#define DUSTIN_MAX_SRH 32           /* SRH entries per call */
#define DUSTIN_MAX_PAIRS 32         /* (SRH head x query row) pairs sharing one KV head */
#define DUSTIN_MAX_LAYERS 16        /* layers per verify / append call */
#define DUSTIN_MAX_QROWS 128        /* (gamma+1) * (Hq/Hkv) verify query rows per KV head */
#define DUSTIN_MAX_BLOCK 64         /* gamma+1 draft-block rows per verify call */
#define DUSTIN_MAX_LCAP (1 << 20)   /* positions per cache */
#define DUSTIN_MAX_REQUESTS 8192    /* requests per paged-cache call */
#define DUSTIN_MAX_TOKENS (1 << 20) /* packed token rows per paged-cache call */
#define DUSTIN_MAX_HEADS 65536      /* query heads, and KV heads, per paged-cache call */

/* A bf16 KV-cache view, element (b, g, pos, j) at
 *   ptr + b*sb + g*sh + pos*sl + j          (strides in elements).
 * d must be 64 or 128; rows (j = 0..d-1) are contiguous.  ptr must be 16-byte
 * aligned and sb, sh, sl multiples of 8.  The cache holds Lcap positions. */
typedef struct {
  void* ptr;
  int32_t hkv;
  int32_t d;
  int64_t sb, sh, sl;
} dustin_kv;

/* Budget and shape parameters shared by all calls. */
typedef struct {
  int32_t B;       /* sequences in the batch, >= 1 */
  int32_t Lcap;    /* capacity (positions) of every cache, 1..DUSTIN_MAX_LCAP */
  int32_t gamma;   /* draft block length (>= 0); verification uses gamma+1 queries */
  int32_t sinks;   /* protected prefix length */
  int32_t window;  /* protected recent-window length; sinks + window <= k */
  int32_t m;       /* draft-tier size (clipped to what the budget leaves) */
  int32_t k;       /* budget |I_verify|, >= 1 */
} dustin_params;

/* One attention signal used for scoring (section 1 of the pages): the draft
 * model's look-ahead queries (channel 0, nq = gamma rows) or the target
 * model's previous-step queries (channel 1, nq = gamma+1 rows). */
typedef struct {
  int32_t n_layers;        /* entries of q[] and k[] */
  int32_t hq;              /* query heads of that model; k[l].hkv must divide it */
  int32_t nq;              /* query rows per sequence */
  const void* const* q;    /* host array [n_layers] of device pointers,
                              bf16 [B][nq][hq][d] contiguous (entries of layers
                              that hold no SRH may be NULL) */
  const dustin_kv* k;      /* host array [n_layers] of key-cache views */
} dustin_signal;

/* One Semantic Retrieval Head: channel 0 = draft look-ahead, 1 = target
 * historical; layer indexes that channel's dustin_signal; q_head < hq. */
typedef struct {
  int32_t channel;
  int32_t layer;
  int32_t q_head;
} dustin_srh;

/* One target layer for verification. */
typedef struct {
  const void* q;    /* device, bf16 [B][gamma+1][hq][d]: verify queries */
  dustin_kv k, v;   /* that layer's full caches (same hkv, d, strides) */
  const void* kb;   /* device, bf16 [B][hkv][gamma+1][d]: the draft block's keys */
  const void* vb;   /* device, bf16 [B][hkv][gamma+1][d]: the draft block's values */
  float* o;         /* device, fp32 [B][gamma+1][hq][d]: output */
} dustin_verify_layer;

/* Arguments of dustin_verify_step. */
typedef struct {
  dustin_params p;
  const dustin_signal* draft;          /* channel 0 */
  const dustin_signal* target;         /* channel 1 */
  const dustin_srh* srh;
  int32_t n_srh;
  int32_t hq;                          /* target query heads for verification */
  int32_t n_layers;                    /* verified layers, all sharing one I_verify */
  const dustin_verify_layer* layers;   /* host array [n_layers] */
  const int32_t* seq_len;              /* device [B] */
  float* importance;                   /* device fp32 [B][2][Lcap] (output) */
  int32_t* i_verify;                   /* device int32 [B][k] (output) */
  cudaEvent_t* stage_events;           /* NULL, or host array of 5 events recorded on
                                          the stream: before score, after the stream
                                          kernel of the first scoring group (before its
                                          normalise kernel), after all score kernels,
                                          after select, after verify */
} dustin_step;

/* Library version string (static storage). */
const char* dustin_version(void);

/* Bytes of workspace needed by every call made with these arguments: score
 * sizes its per-KV-head partial maps from the SRH list, verification its
 * per-unit partials from (hq, hkv, d, n_layers).  Pass n_srh = 0 (and NULL
 * pointers) when nothing is scored and n_layers = 0 when nothing is verified.
 * Returns 0 if the arguments are invalid.  Every workspace holds at least
 * 256 + 65536 bytes (the error word and a reserved area). */
size_t dustin_workspace_bytes(const dustin_params* p, const dustin_signal* draft,
                              const dustin_signal* target, const dustin_srh* srh,
                              int32_t n_srh, int32_t hq, int32_t hkv, int32_t d,
                              int32_t n_layers);

/* Clears the error word and the reserved area of a workspace
 * (asynchronously, on stream).  Call it once before first use, and again
 * after dustin_check has reported DUSTIN_DEV_TIMEOUT. */
int dustin_workspace_init(void* ws, size_t ws_bytes, cudaStream_t stream);

/* Synchronises the stream, returns the error word in *flags (if non-NULL),
 * clears it, and returns DUSTIN_EDEVICE if it was non-zero. */
int dustin_check(void* ws, cudaStream_t stream, int32_t* flags);

/* Hybrid SRH importance scoring (section 1 + 2 of the pages).
 * importance: device fp32 [B][2][Lcap]; channel 0 = draft look-ahead, 1 =
 *   target historical.  importance[b][c][i] = sum over the SRHs of channel c
 *   and their query rows t of softmax_i(q_t . k_i / sqrt(d)) over the
 *   seq_len[b] context positions; entries at or beyond seq_len[b] are 0.
 * seq_len: device int32 [B]. */
int dustin_score(const dustin_params* p, const dustin_signal* draft,
                 const dustin_signal* target, const dustin_srh* srh, int32_t n_srh,
                 const int32_t* seq_len, float* importance, void* ws, size_t ws_bytes,
                 cudaStream_t stream);

/* Budgeted tiered selection (section 1 of the pages).
 * i_verify: device int32 [B][k] = [sinks | window | draft tier | target tier],
 *   each segment ascending; the draft tier holds the top-m' unprotected
 *   positions by importance[b][0] (m' = min(m, k - |protected|)), the target
 *   tier the top remaining ones by importance[b][1]; equal values go to the
 *   lower position.  If k >= seq_len[b] the row is 0..seq_len[b]-1 followed by
 *   -1 padding. */
int dustin_select(const dustin_params* p, const float* importance, const int32_t* seq_len,
                  int32_t* i_verify, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Sparse verification attention (section 3, steps 3-4 of the pages).
 * For sequence b, verify query t (0..gamma) of head h (KV head
 * g = h / (hq/hkv)) attends to the cache rows i_verify[b][*] (entries -1
 * skipped) plus the draft-block rows u <= t, with softmax(q.k/sqrt(d)) weights
 * over values; o = fp32 [B][gamma+1][hq][d].  q, kb, vb as in
 * dustin_verify_layer. */
int dustin_verify_attn(const dustin_params* p, int32_t hq, const void* q, dustin_kv k,
                       dustin_kv v, const void* kb, const void* vb, const int32_t* i_verify,
                       const int32_t* seq_len, float* o, void* ws, size_t ws_bytes,
                       cudaStream_t stream);

/* Dense (full-cache) verification: dustin_verify_attn with every context
 * row 0..seq_len[b]-1 (the pages' "Problem Statement" comparator). */
int dense_verify_attn(const dustin_params* p, int32_t hq, const void* q, dustin_kv k,
                      dustin_kv v, const void* kb, const void* vb, const int32_t* seq_len,
                      float* o, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Append accepted draft rows (section 3, step 5 of the pages).
 * For every layer l and sequence b: rows 0..n_accept[b]-1 of kb[l]/vb[l]
 * (device bf16 [B][hkv][gamma+1][d]) are copied to positions
 * seq_len[b].. of k[l]/v[l]; then seq_len[b] += n_accept[b].  A sequence whose
 * n_accept is outside [0, gamma+1] or whose append would pass Lcap is left
 * untouched and flagged (DUSTIN_DEV_APPEND). */
int dustin_kv_append(const dustin_params* p, int32_t n_layers, const dustin_kv* k,
                     const dustin_kv* v, const void* const* kb, const void* const* vb,
                     const int32_t* n_accept, int32_t* seq_len, void* ws, size_t ws_bytes,
                     cudaStream_t stream);

/* The literal "compressed target KV cache" of section 3, step 3 of the pages,
 * for callers that verify several passes against one selection.  For every
 * layer l, sequence b, KV head g and j < k: row j of kc[l]/vc[l] (bf16
 * [B][hkv][>= k][d], same hkv and d as k[l]/v[l]) becomes row i_verify[b][j]
 * of k[l]/v[l]; entries -1 give zero rows, other indices outside
 * [0, seq_len[b]) give zero rows and set DUSTIN_DEV_INDEX.  seq_len_c[b]
 * (device, out) = the number of entries of i_verify[b] before its first -1
 * (the -1 entries must form a suffix, as dustin_select writes them).
 * dense_verify_attn over (kc, vc, seq_len_c) with Lcap = k then gives the same
 * result as dustin_verify_attn over (k, v, i_verify).  That equality holds
 * only for calls that do not set DUSTIN_DEV_INDEX: sparse verification skips
 * an invalid entry, while dense verification over the compact cache attends
 * to its zero row.  seq_len_c must not be seq_len (other CTAs still read
 * seq_len while it is written): DUSTIN_EINVAL.  dustin_verify_attn itself
 * gathers the rows in-kernel and never writes such a copy. */
int dustin_compact_kv(const dustin_params* p, int32_t n_layers, const dustin_kv* k,
                      const dustin_kv* v, const int32_t* i_verify, const int32_t* seq_len,
                      const dustin_kv* kc, const dustin_kv* vc, int32_t* seq_len_c, void* ws,
                      size_t ws_bytes, cudaStream_t stream);

/* score -> select -> sparse verify of every layer, on one stream. */
int dustin_verify_step(const dustin_step* s, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Host-only query (no device work): how many kernels one dustin_verify_step
 * call with these arguments launches, and how many sequences each scoring
 * group holds.  Scoring runs over groups of *group_size sequences so that a
 * group's logits stay resident in L2; each group takes two kernels (stream,
 * normalise), select takes one, and verification two (the stream-K kernel and
 * the merge of the units it split).  Returns DUSTIN_EINVAL / DUSTIN_ERANGE for arguments
 * dustin_verify_step would reject while planning the scoring. */
int dustin_step_launches(const dustin_step* s, int32_t* n_launches, int32_t* group_size);

/* Host-only query (no device work): the stream-K split that
 * dustin_verify_attn (dense = 0), dense_verify_attn (dense = 1) and the
 * verification of dustin_verify_step use on the current device for this
 * shape.  Units are (layer, sequence, KV head) triples, unit
 * u = (l * B + b) * hkv + g, each of *tiles_per_unit tiles of 64 keys (the
 * context tiles, then one draft-block tile); the T = units * tiles_per_unit
 * tiles are cut among *grid CTAs, CTA c taking tiles [c*T/grid,
 * (c+1)*T/grid).  The grid is two CTAs per SM when (gamma+1)*hq/hkv <= 64
 * and two CTAs' shared-memory layouts fit an SM, else one (at most T).  A
 * unit whose tiles fall to several CTAs is merged by the second verification
 * kernel.  DUSTIN_EINVAL / DUSTIN_ERANGE as the
 * verification calls would return for the shape. */
int dustin_verify_split(const dustin_params* p, int32_t hq, int32_t hkv, int32_t d,
                        int32_t n_layers, int32_t dense, int32_t* grid, int32_t* tiles_per_unit);

/* ---- cache operators ------------------------------------------------------
 * Attention whose output is bf16 (the type the next projection reads) with its
 * log-sum-exp, and the calls that keep a cache within a budget by the weight
 * its rows have been given.  The pages have no counterpart; they share the
 * types and conventions above.  A pass of a server that bounds its caches:
 * dustin_prefix_attn (o, lse) -> accept -> dustin_kv_append ->
 * dustin_accumulate -> dustin_evict. */

/* Bytes of workspace that dustin_window_attn (prefix_cap = 0),
 * dustin_prefix_attn, dustin_accumulate and dustin_evict (n_layers) need with
 * these arguments; hq = 0: no attention, n_layers = 0: no eviction.  Returns 0
 * if the arguments are invalid. */
size_t dustin_cache_workspace_bytes(const dustin_params* p, int32_t hq, int32_t hkv, int32_t d,
                                    int32_t n_layers, int32_t prefix_cap);

/* Attention of the draft block through a sliding window with sinks.  Query t of
 * sequence b has position i = seq_len[b] + t; cache row j < seq_len[b] has
 * position j, block row u position seq_len[b] + u.  A key at position j is
 * visible iff j <= i and (i - j < p->window or j < p->sinks): the window counts
 * the query's own position, and the first p->sinks positions stay visible.
 * Cache and block rows that no query of the block sees are never read (they may
 * hold anything); keys and values that some query sees must be finite.  A query row
 * that is not finite and sees a key gives NaN in its own o and lse.
 *   o    device, bf16 [B][gamma+1][hq][d]: softmax(q.k/sqrt(d)) v over the
 *        visible keys, 0 where there is none (window = 0)
 *   lse  device, fp32 [B][gamma+1][hq], or NULL: ln sum exp(q.k/sqrt(d)), -inf
 *        where no key is visible
 * o and lse share memory neither with each other nor with an input (the same
 * pointer twice: DUSTIN_EINVAL).  The softmax weights are rounded to bf16 for the
 * product with v, each by at most 2^-8 of itself, and o once more; their sum, and
 * so lse, takes them unrounded in fp32.  q, k, v, kb, vb as in
 * dustin_verify_layer; hkv * B <= 16384 (DUSTIN_ERANGE).
 * p->m and p->k are not used beyond their checks.  A sequence whose seq_len is
 * outside [0, Lcap] is flagged (DUSTIN_DEV_SEQLEN) and taken as empty. */
int dustin_window_attn(const dustin_params* p, int32_t hq, const void* q, dustin_kv k, dustin_kv v,
                       const void* kb, const void* vb, const int32_t* seq_len, void* o, float* lse,
                       void* ws, size_t ws_bytes, cudaStream_t stream);

/* Attention of the draft block of a batch whose sequences share a prefix: the
 * keys of sequence b are rows 0..*prefix_len-1 of the one prefix cache, then
 * its own rows 0..seq_len[b]-1, then the block rows u <= t.  The prefix is read
 * once for the whole batch.
 *   pk, pv      the prefix caches, [hkv][prefix_cap][d] (their sb is not used)
 *   prefix_len  device int32 scalar, 0..prefix_cap (0: plain dense attention);
 *               outside: flagged (DUSTIN_DEV_SEQLEN), taken as 0
 * The rest as in dustin_window_attn, without a window: p->sinks and p->window
 * are not used. */
int dustin_prefix_attn(const dustin_params* p, int32_t hq, const void* q, dustin_kv pk, dustin_kv pv,
                       int32_t prefix_cap, const int32_t* prefix_len, dustin_kv k, dustin_kv v,
                       const void* kb, const void* vb, const int32_t* seq_len, void* o, float* lse,
                       void* ws, size_t ws_bytes, cudaStream_t stream);

/* Adds the attention that the accepted rows of a block paid to each row of a
 * cache.  Call it after the accepted rows were appended: the last n = n_new[b]
 * of the L = seq_len[b] cache rows are theirs, and query t < n (the first n of
 * the block's gamma+1 queries) sits at row L - n + t.  For every KV head g and
 * row j < L
 *   weight[b][g][j] += sum over t < n with j <= L - n + t, over the query heads
 *                      of g, of exp(q.k_j/sqrt(d) - lse[b][t][h]),
 * with weight taken as 0 and pos[b][g][j] set to n_seen[b] - (L - j) for the new
 * rows j >= L - n.  A row whose lse is -inf adds nothing, one whose lse is NaN
 * makes the weights that it counts in NaN (which dustin_evict flags).
 *   q, lse         of the attention call that verified the block
 *   n_seen         device int32 [B]: tokens the sequence has had so far, the new
 *                  ones included (n_seen[b] >= seq_len[b]; more once rows were evicted)
 *   weight, pos    device fp32 / int32 [B][hkv][Lcap], no input's memory
 *                  (DUSTIN_EINVAL); rows at or beyond seq_len[b] are left as
 *                  they were
 * A sequence whose n is outside [0, min(gamma+1, L)], L outside [0, Lcap] or
 * n_seen below L is left untouched and flagged (DUSTIN_DEV_APPEND). */
int dustin_accumulate(const dustin_params* p, int32_t hq, const void* q, const float* lse, dustin_kv k,
                      const int32_t* n_new, const int32_t* seq_len, const int32_t* n_seen, float* weight,
                      int32_t* pos, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Evicts from the caches of n_layers layers, in place, down to p->k rows.  For
 * every layer, sequence and KV head with more than k rows the kept ones are
 * those with pos < p->sinks or pos >= n_seen[b] - p->window, then the largest
 * weights; equal weights go to the lower row, and should more than k rows be
 * protected (repeated positions) the lower ones stay.  The rows dropped below k,
 * ascending, take the kept rows at or beyond k, ascending -- K and V rows,
 * weight and pos -- so that as few rows move as can; rows at or beyond k keep
 * their old contents.  Then seq_len[b] = min(seq_len[b], k).  A NaN or negative
 * weight of a row that is not protected ranks as 0 and sets DUSTIN_DEV_NAN.  Every
 * buffer may be given once only (DUSTIN_EINVAL); a sequence whose seq_len is
 * outside [0, Lcap] is left untouched and flagged (DUSTIN_DEV_SEQLEN).
 *
 * More than DUSTIN_MAX_LAYERS layers take a call per group of layers, each with
 * the lengths from before: give every call but the last a copy of seq_len.  A
 * group that is given lengths already lowered to k moves nothing and keeps its
 * first k rows whatever their weight, and no flag tells.
 *
 * Afterwards row j of a cache is no longer position j, and not the same position
 * in every KV head; pos tells which.  What takes the order of rows for that of
 * positions, or rows of all heads together, is not for such caches:
 * dustin_window_attn, dustin_score, dustin_select and the rows it selects.  The
 * rest is: the own part of dustin_prefix_attn, dense_verify_attn,
 * dustin_kv_append, dustin_accumulate and dustin_evict again. */
int dustin_evict(const dustin_params* p, int32_t n_layers, const dustin_kv* k, const dustin_kv* v,
                 float* const* weight, int32_t* const* pos, const int32_t* n_seen, int32_t* seq_len,
                 void* ws, size_t ws_bytes, cudaStream_t stream);

/* ---- paged cache ------------------------------------------------------------
 * A cache in pages for a server whose batch mixes requests of any length, with
 * one or many new tokens each: single tokens, draft blocks, chunks of prompts.
 * The pages have no counterpart.  A pass, all of it on the GPU and without a host
 * copy of any length, so that it can be captured into one graph:
 *   dustin_page_map   pages for the new tokens, where each of them goes
 *   per layer:        dustin_norm_rope (rotates, writes K and V) -> dustin_paged_attn
 *   seq_len[b] += the tokens that stay; the next dustin_page_map takes back the
 *                     pages that rejected tokens and finished requests held.
 * The new tokens of all requests are packed: request b has rows cu[b] ..
 * cu[b+1]-1 of the N rows of every token array; rows at or beyond cu[B] belong to
 * no request (padding of a captured batch).  One table serves all layers, each
 * of which has a cache of its own. */

/* A pool of n_pages pages of `page` rows: element (id, g, r, j) at
 *   ptr + id*sp + g*sh + r*sl + j         (strides in elements).
 * d is 64 or 128, rows are contiguous, ptr is 16-byte aligned, sp, sh and sl are
 * positive multiples of 8 below 2^35, and n_pages * page < 2^31.  Row `pos` of request b is
 * row pos % page of page table[b][pos / page]. */
typedef struct {
  void* ptr;
  int32_t hkv, d;
  int32_t n_pages, page;
  int64_t sp, sh, sl;
} dustin_paged_kv;

/* Shape of a ragged batch. */
typedef struct {
  int32_t B;          /* requests, 1..DUSTIN_MAX_REQUESTS */
  int32_t N;          /* rows of the packed token arrays, 1..DUSTIN_MAX_TOKENS */
  int32_t max_new;    /* new tokens of one request at most, 1..DUSTIN_MAX_TOKENS */
  int32_t max_pages;  /* entries of a request's row of the table, >= 1;
                         max_pages * page <= DUSTIN_MAX_LCAP (DUSTIN_ERANGE) */
} dustin_batch;

/* What dustin_norm_rope does to heads. */
typedef struct {
  int32_t N;            /* token rows, 1..DUSTIN_MAX_TOKENS */
  int32_t hq;           /* query heads */
  int32_t rot;          /* rotated elements of a head, the first ones: a multiple of 16, 0..d */
  int32_t interleaved;  /* 0: pairs (j, j + rot/2), 1: pairs (2j, 2j + 1) */
  float eps;            /* >= 0, finite */
} dustin_rope;

/* Bytes of workspace that dustin_paged_attn needs with these arguments.
 * dustin_page_map and dustin_norm_rope need the same call's with hq = 0.
 * Returns 0 if the arguments are invalid. */
size_t dustin_paged_workspace_bytes(const dustin_batch* bt, int32_t hq, int32_t hkv, int32_t d);

/* Pages, block tables and slots of a batch.  Request b has seq_len[b] rows in the
 * cache and n_new[b] new tokens, together need = ceil((seq_len + n_new) / page)
 * pages, and holds held[b]: entries 0..held[b]-1 of its row of the table.  The
 * pool of free pages is the stack free_list[0..*n_free).
 *  1. A request with held > need gives back entries need..held-1 of its row: all
 *     these pages are pushed, in the order of requests and, within one, of its row.
 *  2. A request with held < need takes need - held pages, popped one by one into
 *     entries held..need-1, in the same order.  From the first request that the
 *     pool has too few pages for on, no request gets any (DUSTIN_DEV_PAGES).
 * A request that holds the pages that it needs afterwards is served.
 *   table      device int32 [B][max_pages], in and out; entries at or beyond
 *              held[b] are left as they were
 *   held       device int32 [B], in and out (not served: unchanged)
 *   free_list  device int32 [n_pages], in and out; n_free device int32, in and out.
 *              Entries at or beyond *n_free are left as the pushes wrote them.
 *   cu         device int32 [B+1], out: cu[b] = min(N, sum of n_new before b)
 *   kv_len     device int32 [B], out: seq_len + n_new, or 0 if not served
 *   slot       device int32 [N], out: for a served request's token at position
 *              p = seq_len + t, table[b][p / page] * page + p % page; else -1
 *   pos        device int32 [N], out: p, also if not served; 0 for padding rows
 * A request whose numbers are inconsistent (negative, n_new > max_new, more rows
 * than max_pages pages hold, tokens past row N, held outside [0, max_pages]) is
 * flagged (DUSTIN_DEV_SEQLEN), not served, and keeps its pages.  A pool whose
 * count is outside [0, n_pages] or would pass n_pages with the pages given back
 * is flagged (DUSTIN_DEV_PAGES) and left alone: nothing is given back or taken.
 * A table entry outside [0, n_pages) gives slot -1 and DUSTIN_DEV_INDEX.  A page
 * belongs to one request: tables that share pages are not for this call, which
 * would give such a page back twice.  `page` is any positive number, and the
 * table has fewer than 2^31 entries (DUSTIN_ERANGE).  No two of the buffers may be
 * the same (DUSTIN_EINVAL). */
int dustin_page_map(const dustin_batch* bt, int32_t page, int32_t n_pages, const int32_t* seq_len,
                    const int32_t* n_new, int32_t* table, int32_t* held, int32_t* free_list,
                    int32_t* n_free, int32_t* cu, int32_t* kv_len, int32_t* slot, int32_t* pos, void* ws,
                    size_t ws_bytes, cudaStream_t stream);

/* Norm of each head, position rotation and cache write of one layer's new tokens.
 *   y = x / sqrt(mean(x^2) + eps) * w          (w NULL: y = x)
 * for each head x of q (w = q_w) and k (w = k_w), then for each pair (a, b) of
 * the first rot elements, the j-th one turned by t = pos[i] * inv_freq[j]:
 *   (a cos t - b sin t, b cos t + a sin t).
 * q goes to q_out; k and v (v as it is) go to the caches at slot[i].
 *   q, k, v   device, bf16 rows of hq, hkv, hkv heads of d: row i at
 *             ptr + i * stride (elements, a multiple of 8, at least the row), as the
 *             slices of one projection's output are
 *   q_w, k_w  device bf16 [d], 16-byte aligned, or NULL
 *   inv_freq  device fp32 [rot/2], below 2^39 in size, or NULL with rot = 0
 *   pos, slot device int32 [N].  slot -1: the row's k and v are not written (its q
 *             is); any other value outside [0, n_pages * page) as well, with
 *             DUSTIN_DEV_INDEX.  No slot may occur twice.
 *   q_out     device bf16 rows of hq heads; may be q itself with the same stride
 *   kc, vc    caches of the same hkv, d, n_pages and page; `page` is any positive
 *             number, so that a contiguous cache [B][hkv][Lcap][d] is a pool of B
 *             pages of Lcap rows, with slot = b * Lcap + position
 * Everything is fp32 with one rounding at the end.  Angles are reduced to a turn in whole
 * numbers, to 2^-33 of it at any position where |inv_freq| < 2^39, and then rounded to
 * fp32's 24 bits of half a turn, so that far positions lose nothing.  Heads are normed however small
 * they are (with eps < 2^-100, one whose squares underflow is scaled by a power of two
 * first); elements of a normed head, and w, stay below about 2^60.  A head of zeros
 * with eps = 0 is NaN, 0 / 0. */
int dustin_norm_rope(const dustin_rope* r, const void* q, int64_t q_stride, const void* k,
                     int64_t k_stride, const void* v, int64_t v_stride, const void* q_w, const void* k_w,
                     const float* inv_freq, const int32_t* pos, const int32_t* slot, void* q_out,
                     int64_t q_out_stride, dustin_paged_kv kc, dustin_paged_kv vc, void* ws,
                     size_t ws_bytes, cudaStream_t stream);

/* Attention of a ragged batch's new tokens over a paged cache that holds their own
 * rows already.  Request b has n = cu[b+1] - cu[b] query rows; row t is at position
 * p = kv_len[b] - n + t and sees the cache rows 0..p:
 *   o    device bf16 [N][hq][d], 32-byte aligned: softmax(q.k/sqrt(d)) v, 0 where p < 0
 *   lse  device fp32 [N][hq], or NULL: ln sum exp(q.k/sqrt(d)), -inf where p < 0
 *   q    device bf16 [N][hq][d];  hq / hkv <= 128
 *   table, cu, kv_len  of dustin_page_map (or of the caller's own)
 * Rows at or beyond cu[B] are left as they were.  A request whose numbers are
 * inconsistent (cu not ascending within [0, N], n > max_new, kv_len outside
 * [0, max_pages * page]) is flagged (DUSTIN_DEV_SEQLEN) and its rows are left as
 * they were.  A table entry that is needed and outside [0, n_pages) is flagged
 * (DUSTIN_DEV_INDEX); its rows count as rows of zeros.  Cache rows at or beyond
 * kv_len[b] may hold anything; keys and values below it must be finite.  A query
 * row that is not finite and sees a key gives NaN in its own o and lse.  Softmax
 * weights are rounded to bf16 for the product with v, each by at most 2^-8 of
 * itself (2^-16 where max_new * hq / hkv <= 128), and o once more; their sum, and so
 * lse, takes them unrounded in fp32.  The order of the fp32 sums goes by the whole
 * batch: a request's bits may differ between batches, not between runs of one.
 * max_new and N shape the launch; both may be larger than what a batch brings.
 * `page` is 16, 32, 64 or a multiple of 128 (DUSTIN_EINVAL).  o and lse are no
 * input's memory (DUSTIN_EINVAL). */
int dustin_paged_attn(const dustin_batch* bt, int32_t hq, const void* q, dustin_paged_kv kc,
                      dustin_paged_kv vc, const int32_t* table, const int32_t* cu, const int32_t* kv_len,
                      void* o, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Self-test of the bounded waits (no counterpart in the pages).  Every
 * on-chip wait of the kernels above gives up after 2 s, sets
 * DUSTIN_DEV_TIMEOUT in the error word and raises a CTA-wide abort flag that
 * makes the CTA's other waits give up at once.  This call runs that wait in
 * one CTA on an mbarrier that nothing ever arrives on, with no copy or MMA in
 * flight: one thread waits limit_ns nanoseconds (1000 .. 1e9) and gives up,
 * a second waits with the kernels' own 2 s limit and stops when the first
 * raises the abort flag.  waited_ns: device int64 [2], 8-byte aligned (out):
 * how long each waited (-1 if its wait had succeeded).  Afterwards
 * dustin_check(ws) reports DUSTIN_DEV_TIMEOUT and the context stays usable.
 * ws needs only its 256-byte header. */
int dustin_wait_selftest(int64_t limit_ns, int64_t* waited_ns, void* ws, size_t ws_bytes,
                         cudaStream_t stream);

/* Bytes of the library-owned scratch array used by dustin_score_noalloc. */
#define DUSTIN_NOALLOC_SCRATCH_BYTES (16u << 20)

/* dustin_score without a caller workspace.  The pages have no counterpart to
 * this call: it exists for callers that cannot call cudaMalloc (or any other
 * allocator) at the point where they score -- for example code running inside
 * an allocator-free runtime, a host callback, or a component that must not
 * touch the process's memory pools.  Results are the same as dustin_score's.
 *
 * Scratch lives in one file-scope device array of DUSTIN_NOALLOC_SCRATCH_BYTES
 * (16 MiB) inside the library; every GPU that loads the library holds it
 * until the process exits.  The call allocates nothing: no cudaMalloc,
 * cudaFree or allocating library routine.  The first call on each device
 * looks up the array's device address (cudaGetSymbolAddress, with that device
 * current); make that first call before any stream capture.
 *
 * Limits: the scratch of at least one sequence -- its logits (SRH pairs x
 * Lcap x 4 bytes) and their statistics, plus a 256-byte header -- must fit in
 * the array; larger batches are scored in groups of sequences that fit.
 * Otherwise DUSTIN_ERANGE is returned and nothing is launched.
 *
 * The device error word (DUSTIN_DEV_* bits) lives in the array's first bytes.
 * It is sticky across calls, like a workspace's: dustin_score_noalloc_check
 * reads and clears it.
 *
 * All calls share the one array and it keeps the last call's contents: calls
 * that overlap on the GPU (different streams, or different host threads
 * without ordering) race on it and must be serialised by the caller. */
int dustin_score_noalloc(const dustin_params* p, const dustin_signal* draft,
                         const dustin_signal* target, const dustin_srh* srh, int32_t n_srh,
                         const int32_t* seq_len, float* importance, cudaStream_t stream);

/* dustin_check for the static array of dustin_score_noalloc on the current
 * device: synchronises the stream, returns the error word of every
 * dustin_score_noalloc call since the last check in *flags (if non-NULL),
 * clears it, and returns DUSTIN_EDEVICE if it was non-zero.  Allocates
 * nothing; DUSTIN_ECUDA if a CUDA call fails. */
int dustin_score_noalloc_check(cudaStream_t stream, int32_t* flags);

#ifdef __cplusplus
}
#endif

#endif /* DUSTIN_H */
