// Internal launch interface between the C-ABI layer (api.cu) and the kernels.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/dustin.h"

namespace dustin {

// Runs set() once per device (function attributes belong to the current one).
// done: one word of device bits per call site.
template <typename F>
cudaError_t once_per_device(std::atomic<uint64_t>& done, F set) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = set();
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Launches kern<<<grid, block, smem, stream>>>(args) with programmatic stream
// serialisation, so that it may begin while the previous kernel in the stream
// drains (the kernel itself waits with pdl_wait before reading its inputs).
template <typename Kern, typename Args>
cudaError_t launch_pdl(Kern kern, dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       const Args& args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args);
}

// ------------------------------------------------------------------ verify

struct VerifyLayerDev {
  const uint16_t* q;   // [B][T][hq][D]
  const uint16_t* k;   // cache base
  const uint16_t* v;
  const uint16_t* kb;  // [B][hkv][T][D]
  const uint16_t* vb;
  float* o;            // [B][T][hq][D]
  int64_t ksb, ksh, ksl, vsb, vsh, vsl;
};

// Shared-memory layout of the verification kernel (bytes from its 1024-byte
// aligned base), chosen on the host per launch.
struct VLay {
  int NP, nst;           // 64-column panels per row; K/V stages
  uint32_t q_panel, q_buf, ring_off, kv_panel, half_bytes, stage_bytes;
  uint32_t mask_off, bar_off, misc_off, total;
};

struct VerifyArgs {
  int B, Lcap, T, hq, hkv, G, NQ;
  int k;                // budget (sparse); unused for dense
  int dense;            // 1: keys are positions 0..seq_len-1
  int n_layers;
  int ctx_tiles;        // 64-key tiles of context per unit
  int tiles_u;          // ctx_tiles + 1 (the draft-block tile)
  long long total;      // units * tiles_u
  int max_seg;          // partial slots per unit
  long long slot_floats;  // floats per partial slot (multiple of 4)
  float scale_log2;     // log2(e) / sqrt(D)
  VLay lay;
  const int32_t* ivf;   // [B][k] (sparse)
  const int32_t* seq_len;
  int* err;
  float* partial;       // [units][max_seg][slot_floats]: O [NQ][D], m [NQ], l [NQ]
  VerifyLayerDev layer[DUSTIN_MAX_LAYERS];
  // per layer: the queries as 3-D (d, hq, B*T) with box (64, G, T) and the
  // 128-byte swizzle, so one load brings a unit's G x T query rows
  CUtensorMap qmap[DUSTIN_MAX_LAYERS];
  // dense mode, tma = 1: per layer the K and V caches as tensor maps with a
  // (64 columns, 64 rows) box and the 128-byte swizzle (rank 2: rows
  // B*hkv*Lcap of a packed cache; rank 4: (d, Lcap, hkv, B) of a strided one),
  // so that a context tile wholly inside the sequence comes in 2 * D / 64
  // boxes instead of row gathers
  int tma;
  int kvrank[DUSTIN_MAX_LAYERS];
  CUtensorMap kmap[DUSTIN_MAX_LAYERS];
  CUtensorMap vmap[DUSTIN_MAX_LAYERS];
};

// The segment merge that follows the stream-K kernel.
struct VerifyCombineArgs {
  int NQ, T, hq, hkv, G, units_per_layer, tiles_u, main_grid, max_seg;
  long long total, slot_floats;
  const float* partial;
  float* o[DUSTIN_MAX_LAYERS];
};

struct VerifyLaunch {
  int D, NST;
  int cps;               // CTAs per SM (1 or 2)
  VLay lay;
  int ctx_tiles, tiles_u, grid, max_seg;
  long long units, total, slot_floats;
  size_t smem;
};

// Grid sizes never exceed kVerifyGridMax, which bounds the partial slots.
constexpr int kVerifyGridMax = 1024;
VerifyLaunch verify_plan(int D, int NQ, int nkeys_cap, int B, int hkv, int n_layers, int dense,
                         int num_sms);
size_t verify_scratch_bytes(const VerifyLaunch& pl);
cudaError_t verify_launch(const VerifyArgs& a, const VerifyLaunch& pl, cudaStream_t stream);

// ------------------------------------------------------------------- score

struct ScoreSlab {
  int channel;   // 0 draft, 1 target
  int cache;     // index into ScoreArgs::map
  int g;         // KV head
  int D;         // head dim (64 or 128)
  int nq;        // query rows per sequence
  int hq;        // query heads of the model
  int npairs;    // heads.size() * nq
  int nheads;
  int heads[DUSTIN_MAX_PAIRS];
  int rows;      // positions per tile (128 for d = 128, 256 for d = 64)
  int tiles;     // tiles per sequence: ceil(Lcap / rows)
  long long logit_off;   // float offset of this slab's logits [nb][npairs][LSP]
  int row2d;     // 0: 4-D map; else 2-D map over packed rows, value = hkv of the cache
  int cost;      // relative cost of one tile (bytes plus logits written), for balancing
  const uint16_t* q;     // [B][nq][hq][D]
};

// Per-slab facts of one group launch in a compact form: the normalise kernel
// copies the table to shared memory once (kernel-parameter reads with a
// per-thread index are slow) and walks it there.
struct SlabInfo {
  long long logit_off;   // float offset of the slab's logits
  long long first_tile;  // first flattened tile of the slab
  long long cost_start;  // cost before that tile
  int npairs, tiles, cost, row0;   // row0: the slab's first logits row (channel 0 first)
  int slab, pad;         // index of the slab in ScoreArgs::slab
};

// One stream launch as the normalise kernel sees it.
struct NormGroup {
  int b0, nb;            // its sequences
  int grid;              // CTAs of its stream kernel
  int cps;               // normalise CTAs per sequence
  long long total_cost;  // its partition's total cost
  float* logits;         // its logits buffer
  float* stats;          // its statistics buffer
};


struct ScoreArgs {
  CUtensorMap map[DUSTIN_MAX_SRH];   // one per (channel, layer) cache; box 64 x 128
  ScoreSlab slab[DUSTIN_MAX_SRH];
  long long slab_start[DUSTIN_MAX_SRH + 1];   // first flattened tile of each slab
  long long cost_start[DUSTIN_MAX_SRH + 1];   // cost before the first tile of each slab
  long long total;                            // tiles of this group
  long long total_cost;                       // sum of tile costs of this group
  int B, Lcap, LSP, n_slab, np_max;
  int n_rows, n_rows0;   // logits rows (slab, pair) per sequence, channel 0 first; rows of channel 0
  int sinks, window;     // the unprotected range of the selection histograms
  int b0, nb;            // the group of sequences handled by this launch
  int grid;              // CTAs of the stream kernel
  int max_seg;           // statistics slots per (slab, sequence)
  const int32_t* seq_len;
  int* err;
  float* logits;         // scratch, stays in L2 between the two kernels
  float* stats;          // [n_slab][nb][max_seg][np_max][2]
  float* importance;     // [B][2][Lcap]
  int* hist;             // [B][2][4096] selection histograms, or nullptr
  // stream kernel: 0 -- wait for the previous launch before starting; 1 --
  // start at once (the previous launch is the other stream kernel of a pair,
  // writing other buffers) and wait for it only before exiting, so that this
  // launch completes after it
  int wait_at_end;
  // normalise kernel: the groups it covers (one or two stream launches), each
  // with its own logits and statistics buffers and partition
  int n_groups;
  NormGroup ng[2];
  SlabInfo info[2][DUSTIN_MAX_SRH];   // per group, in row order (channel 0 slabs first)
};

struct ScoreLaunch {
  int NT;
  size_t smem;
  size_t norm_smem;      // dynamic shared memory of the normalise kernel
};

constexpr int kScoreGridMax = 256;
size_t score_stream_smem();
size_t score_norm_smem(int n_rows);
int score_norm_ctas_per_sm(int n_rows);   // resident normalise CTAs per SM
int score_rows_per_tile(int D);
int score_tile_cost(int D, int npairs);
// Launches the stream kernel of the group in a (b0, nb, logits, stats, ...).
cudaError_t score_stream_launch(const ScoreArgs& a, const ScoreLaunch& pl, cudaStream_t stream);
// Launches the normalise kernel of the groups in a.ng[0 .. n_groups).
cudaError_t score_norm_launch(const ScoreArgs& a, const ScoreLaunch& pl, cudaStream_t stream);

// ------------------------------------------------------------------ select

constexpr int kMaxSelectCtas = 8;          // scan CTAs (cluster size) per sequence

struct SelectArgs {
  int B, Lcap, k, sinks, window, m;
  int vec4;              // set by select_launch: rows read as float4
  int cs;                // set by select_launch: scan CTAs per sequence (one cluster)
  int bits_words;        // bitmap words per sequence (general path)
  const float* imp;      // [B][2][Lcap]
  int* hist;             // [B][2][4096] level-1 histograms over the unprotected
                         // positions (built by the score kernels in the fused
                         // step, by select_launch otherwise)
  const int32_t* seq_len;
  int32_t* out;          // [B][k]
  int* err;
  uint32_t* bits;        // [B][bits_words]
};

// Workspace layout of the selection scratch starting at byte offset off.
struct SelectPlan {
  int bits_words;
  size_t hist_off, bits_off, end;
};
SelectPlan select_plan(int B, int Lcap, size_t off);
// build_hist: count the histograms first (standalone call).
cudaError_t select_launch(const SelectArgs& a, bool build_hist, cudaStream_t stream);

// ------------------------------------------------------------------ append

struct AppendLayerDev {
  uint16_t* k;
  uint16_t* v;
  const uint16_t* kb;
  const uint16_t* vb;
  int64_t ksb, ksh, ksl, vsb, vsh, vsl;
};

struct AppendArgs {
  int B, Lcap, T, hkv, D, n_layers;
  const int32_t* n_accept;
  int32_t* seq_len;
  int* err;
  AppendLayerDev layer[DUSTIN_MAX_LAYERS];
};
cudaError_t append_launch(const AppendArgs& a, cudaStream_t stream);

// ----------------------------------------------------------------- compact

struct CompactLayerDev {
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* kc;
  uint16_t* vc;
  int64_t ksb, ksh, ksl, vsb, vsh, vsl;
  int64_t kcsb, kcsh, kcsl, vcsb, vcsh, vcsl;
};

struct CompactArgs {
  int B, Lcap, k, hkv, D, n_layers;
  const int32_t* ivf;        // [B][k]
  const int32_t* seq_len;
  int32_t* seq_len_c;        // [B] out: compact lengths
  int* err;
  CompactLayerDev layer[DUSTIN_MAX_LAYERS];
};
cudaError_t compact_launch(const CompactArgs& a, cudaStream_t stream);

// ------------------------------------------------- windowed / prefix attention

constexpr int kAttendTile = 64;        // keys per tile
constexpr int kAttendGridMax = 512;    // CTAs of the attention kernel at most
constexpr int kPrefixTile = 128;       // keys, and query rows, per tile of the prefix kernel
constexpr int kPrefixGridMax = 256;    // CTAs of the prefix kernel at most
constexpr int kAttendFar = 1 << 22;    // a window or sink count past every position
constexpr float kLn2 = 0.69314718055994531f;

struct AttendArgs {
  int B, Lcap, T, hq, hkv;
  int sinks, window;         // 0 .. kAttendFar; shared-prefix attention: 0 and kAttendFar
  int Pcap;                  // rows of the prefix caches (0: no prefix)
  float scale_log2;          // log2(e) / sqrt(D)
  const uint16_t* q;         // [B][T][hq][D]
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* pk;        // prefix caches: element (g, pos, x) at g*sh + pos*sl + x
  const uint16_t* pv;
  const uint16_t* kb;        // [B][hkv][T][D]
  const uint16_t* vb;
  int64_t ksb, ksh, ksl, vsb, vsh, vsl, pksh, pksl, pvsh, pvsl;
  const int32_t* seq_len;
  const int32_t* prefix_len; // device scalar, or nullptr
  int* err;
  uint16_t* o;               // [B][T][hq][D] bf16
  float* lse;                // [B][T][hq], or nullptr
  int max_tiles;             // tiles of a unit at most
  int whole;                 // set by attend_launch: CTAs take whole units
  int32_t* seg_cta;          // [units][2]: first and last CTA of each unit's segments
  float* partial;            // segment slots [units + grid][slot_floats]: O [NQ][D], m [NQ], l [NQ]
  int64_t slot_floats;
  int tma;                   // the caches have tensor maps (whole tiles come as TMA boxes)
  int krank, vrank;          // 2: map over packed rows, 4: (d, Lcap, hkv, B)
  // the prefix kernel (pgrid = 0: no prefix, and a segment of the attention
  // kernel that covers its unit writes o and lse itself)
  int pgrid;
  int nt, row_tiles, pairs;  // tokens per row tile; row tiles of a KV head; pairs of them
  float* ppartial;           // slots [(hkv * pairs + pgrid)][2][128 * (D + 2)]: O, m [128], l [128]
  int32_t* pseg_cta;         // [hkv * pairs][2]: first and last CTA of each prefix unit
  int ptma;                  // the prefix caches have tensor maps
  CUtensorMap qmap, kmap, vmap, pqmap, pkmap, pvmap;
};
// The attention kernel, the prefix kernel if there is a prefix, the merge.
cudaError_t attend_launch(AttendArgs& a, int D, int num_sms, cudaStream_t stream);
cudaError_t prefix_launch(const AttendArgs& a, int D, cudaStream_t stream);

// -------------------------------------------------------------- accumulate

constexpr int kAccumulateTile = 128;   // cache rows per tile

struct AccumulateArgs {
  int B, Lcap, T, G, hkv;
  float scale_log2;          // log2(e) / sqrt(D)
  const float* lse;          // [B][T][hkv * G]
  const int32_t* n_new;
  const int32_t* seq_len;
  const int32_t* n_seen;
  float* weight;             // [B][hkv][Lcap]
  int32_t* pos;              // [B][hkv][Lcap]
  int* err;
  int krank;                 // 2: map over packed rows, 4: (d, Lcap, hkv, B)
  CUtensorMap qmap, kmap;
};
// Whether sequence lengths (rows, new rows, positions seen) are consistent; a
// sequence that fails is flagged and left as it was.
__host__ __device__ inline bool accumulate_ok(const AccumulateArgs& a, int L, int n, int seen) {
  return L >= 0 && L <= a.Lcap && n >= 0 && n <= a.T && n <= L && seen >= L;
}
cudaError_t accumulate_launch(const AccumulateArgs& a, int D, int num_sms, cudaStream_t stream);

// ------------------------------------------------------------------- evict

struct EvictLayerDev {
  uint16_t* k;
  uint16_t* v;
  float* weight;             // [B][hkv][Lcap]
  int32_t* pos;              // [B][hkv][Lcap]
  int64_t ksb, ksh, ksl, vsb, vsh, vsl;
};

struct EvictArgs {
  int B, Lcap, hkv, D, n_layers, sinks, window, k;
  const int32_t* n_seen;
  int32_t* seq_len;
  int* err;
  int32_t* moves;            // [n_layers][B][hkv]: rows to move
  int32_t* lists;            // [n_layers][B][hkv][2][list_cap]: holes, movers
  int list_cap;              // min(k, Lcap - k), the rows a unit can move
  int keys_cap;              // set by evict_launch: keys a CTA keeps in shared memory
  int vec4;                  // set by evict_launch: weights and positions read four at a time
  EvictLayerDev layer[DUSTIN_MAX_LAYERS];
};
cudaError_t evict_launch(EvictArgs& a, int num_sms, cudaStream_t stream);

// ------------------------------------------------------------- paged cache

struct PageMapArgs {
  int B, N, max_new, max_pages, page, n_pages;
  const int32_t* seq_len;
  const int32_t* n_new;
  int32_t* table;            // [B][max_pages]
  int32_t* held;             // [B]
  int32_t* free_list;        // [n_pages]
  int32_t* n_free;
  int32_t* cu;               // [B + 1]
  int32_t* kv_len;           // [B]
  int32_t* slot;             // [N]
  int32_t* pos;              // [N]
  int* err;
};
cudaError_t page_map_launch(const PageMapArgs& a, cudaStream_t stream);

struct RopeArgs {
  int N, hq, hkv, rot, interleaved;
  float eps;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t qst, kst, vst;     // rows, in elements
  const uint16_t* q_w;       // [D], or nullptr
  const uint16_t* k_w;
  const float* inv_freq;     // [rot / 2]
  const int32_t* pos;
  const int32_t* slot;
  uint16_t* q_out;
  int64_t ost;
  uint16_t* kc;
  uint16_t* vc;
  int64_t ksp, ksh, ksl, vsp, vsh, vsl;
  int n_pages, page;
  int* err;
};
cudaError_t rope_launch(const RopeArgs& a, int D, int num_sms, cudaStream_t stream);

struct PagedArgs {
  int B, N, hq, hkv, max_new, max_pages;
  int page, n_pages;
  float scale_log2;          // log2(e) / sqrt(D)
  const int32_t* table;      // [B][max_pages]
  const int32_t* cu;         // [B + 1]
  const int32_t* kv_len;     // [B]
  uint16_t* o;               // [N][hq][D] bf16
  float* lse;                // [N][hq], or nullptr
  int* err;
  int nt, qt;                // tokens of a row tile, and of a query load
  int merged;                // a load of the pools brings all columns (else 64)
  int map_panels, map_groups;   // what a KV head adds to the third and fourth coordinate of a load
  int4* split;               // [kPagedGridMax][2] of the unit that a CTA starts and does not end: first row of its
                             // request, KV head, pair, last CTA (-1: none); its rows and cache rows
  float* partial;            // slots [kPagedGridMax][2][lanes][128 * (D + 2)]: O, m [128], l [128]
  CUtensorMap qmap, kmap, vmap;
};
constexpr int kPagedTile = 128;      // keys, and query rows, per tile
constexpr int kPagedGridMax = 256;   // CTAs at most
// Whether the batch's requests have one row tile each (the shape with one lane).
inline int paged_lanes(int hq, int hkv, int max_new) { return max_new <= kPagedTile / (hq / hkv) ? 1 : 2; }
// Whether a request's numbers are consistent; one that fails is flagged and its
// rows are left as they were.
__host__ __device__ inline bool paged_ok(const PagedArgs& a, int c0, int c1, int kv) {
  return c0 >= 0 && c1 >= c0 && c1 <= a.N && c1 - c0 <= a.max_new && kv >= 0 && kv <= (long long)a.max_pages * a.page;
}
cudaError_t paged_launch(PagedArgs& a, int D, int num_sms, cudaStream_t stream);

// ------------------------------------------------------------ wait self-test
cudaError_t wait_selftest_launch(int* err, long long* waited, unsigned long long limit_ns,
                                 cudaStream_t stream);

}  // namespace dustin
