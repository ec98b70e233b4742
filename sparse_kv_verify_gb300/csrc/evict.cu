// Eviction from a cache by accumulated attention weight.
//
// A (layer, sequence, KV head) unit with n = seq_len[b] > k rows keeps k of
// them: those at positions below `sinks` or among the last `window` positions
// seen, then the largest weights (equal weights: the lower row).  The rows it
// drops below k, in order, take the rows it keeps at or beyond k, in order --
// sources and destinations never overlap, so the move is in place, needs no
// order among its rows, and moves as few as can be.
//
// Two launches:
//   select  one cluster of CTAs per unit.  Every row's 32-bit key (all ones for
//           a protected row, else the weight's bits, which order like the
//           weight) is formed once and kept in shared memory (a CTA with more than
//           kKeysMax rows forms it anew in every pass); three histogram passes of
//           12, 10 and 10 bits, summed over the cluster's CTAs, give the k-th
//           largest key and how many rows that equal it stay.  With kept(j) =
//           rows kept before row j, a hole j < k is the (j - kept(j))-th and a
//           mover j >= k the (kept(j) - kept(k))-th of its list, so both lists
//           are written from one ordered count of keys above and equal to the
//           threshold.
//   move    bound by the bytes of the rows: every warp moves four rows at a
//           time, a row's K and V by half a warp each, loads before stores.
//           It also sets the lengths, which the first launch read.
//
// Cold caches, 128 units (16 sequences x 8 KV heads), d = 128: 32 K rows to 2048:
// select 34 us, move 45 us for 252 MB (5.6 TB/s); 2054 rows to 2048: select 9.4,
// move 5.5.  The first with eight rows in flight instead of four takes 4.8 us
// more, with plain instead of streaming stores 6.7 us more.
#include <algorithm>

#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace dustin {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 4096;            // of the first histogram pass; the others use 1024
constexpr int kKeysMax = 48 * 1024;      // keys that a CTA keeps in shared memory
constexpr int kMaxCluster = 8;
constexpr int kSliceMin = 4096;          // rows per CTA below which more CTAs do not help

struct Counts {
  int gt, tie, gt_below, tie_below;      // keys above / at the threshold; of these the rows < k
};

struct Rule {                            // what a row's key depends on
  const float* weight;
  const int32_t* pos;
  int sinks, recent, last;               // last: the unit's last row
  int* err;
};
__device__ __forceinline__ uint32_t key_of(const Rule& R, int p, float w) {
  return p < R.sinks || p >= R.recent ? 0xFFFFFFFFu : importance_key(w, R.err);
}
// The keys of rows j .. j + 3; rows past the last one repeat it.
__device__ __noinline__ uint4 keys_by_row(const Rule& R, int j) {
  uint32_t key[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int y = min(j + x, R.last);
    key[x] = key_of(R, __ldcg(R.pos + y), __ldcg(R.weight + y));
  }
  return make_uint4(key[0], key[1], key[2], key[3]);
}

// (One launch runs this code once, so its loops are kept short: at n = 2054 the
// instruction fetches of unrolled passes took longer than their work.)
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const __grid_constant__ EvictArgs A) {
  extern __shared__ __align__(16) uint32_t keys[];     // [keys_cap]
  __shared__ int hist[kBins];
  __shared__ int warp_sum[kWarps];
  __shared__ Counts warp_cnt[kWarps];
  __shared__ Counts cta_cnt;
  __shared__ int s_bin, s_need;
  pdl_launch_dependents();
  pdl_wait();
  const cg::cluster_group cluster = cg::this_cluster();
  const int cs = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  auto sync_all = [&] {
    if (cs > 1) cluster.sync();
    else __syncthreads();
  };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int unit = blockIdx.x / cs, l = blockIdx.y;
  const int b = unit / A.hkv, g = unit % A.hkv, k = A.k;
  const size_t lu = size_t(l) * A.B * A.hkv + unit;
  const int n = A.seq_len[b], seen = A.n_seen[b];
  if (n < 0 || n > A.Lcap || n <= k) {   // the whole cluster leaves
    if (rank == 0 && tid == 0) {
      if ((n < 0 || n > A.Lcap) && g == 0 && l == 0) flag_error(A.err, DUSTIN_DEV_SEQLEN);
      A.moves[lu] = 0;
    }
    return;
  }
  const Rule R{A.layer[l].weight + size_t(unit) * A.Lcap, A.layer[l].pos + size_t(unit) * A.Lcap, A.sinks,
               seen - A.window, n - 1, A.err};
  // this CTA's rows [j0, j1); a warp takes 128 of them at a time, four
  // neighbours to a lane
  const int slice = ((n + cs - 1) / cs + 127) & ~127;
  const int j0 = min(rank * slice, n), j1 = min(j0 + slice, n);
  const bool cached = slice <= A.keys_cap;
  if (cached) {
    if (A.vec4) {   // (a unit's rows are a multiple of four, so none lies outside)
#pragma unroll 4
      for (int j = j0 + 4 * tid; j < j1; j += 4 * kThreads) {
        const int4 p = __ldcg(reinterpret_cast<const int4*>(R.pos + j));
        const float4 w = __ldcg(reinterpret_cast<const float4*>(R.weight + j));
        uint4 key;
        key.x = key_of(R, p.x, w.x);
        key.y = j + 1 < j1 ? key_of(R, p.y, w.y) : 0u;   // rows past the last hold anything
        key.z = j + 2 < j1 ? key_of(R, p.z, w.z) : 0u;
        key.w = j + 3 < j1 ? key_of(R, p.w, w.w) : 0u;
        *reinterpret_cast<uint4*>(keys + (j - j0)) = key;
      }
    } else {
#pragma unroll 1
      for (int j = j0 + 4 * tid; j < j1; j += 4 * kThreads) *reinterpret_cast<uint4*>(keys + (j - j0)) = keys_by_row(R, j);
    }
  }
  auto key4 = [&](int j, uint32_t* key) {
    const uint4 q = cached ? *reinterpret_cast<const uint4*>(keys + (j - j0)) : keys_by_row(R, j);
    key[0] = q.x;
    key[1] = q.y;
    key[2] = q.z;
    key[3] = q.w;
  };

  // the k-th largest key, digit by digit
  uint32_t high = 0;      // digits so far
  int need = k;           // rows still to take among the keys that share them
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = 20 - 10 * pass, bits = pass == 0 ? 12 : 10;
    constexpr int kPer = kBins / kThreads;              // bins of a thread
#pragma unroll
    for (int x = 0; x < kPer; ++x) hist[tid + x * kThreads] = 0;
    __syncthreads();
#pragma unroll 1
    for (int jb = j0 + 128 * warp; jb < j1; jb += 4 * kThreads) {
      const int j = jb + 4 * lane;
      uint32_t key[4];
      key4(j, key);
      int live = 0;                      // rows that share the digits so far
#pragma unroll
      for (int x = 0; x < 4; ++x) live |= (j + x < j1 && (pass == 0 || (key[x] >> (shift + bits)) == high)) << x;
      if (!__any_sync(0xffffffffu, live)) continue;
      // a warp whose rows share a bin (a protected run, weights that were never
      // touched) counts them at once, and the zeros of any warp go together:
      // atomics on one bin run one after another
      const uint32_t first = __shfl_sync(0xffffffffu, key[0] >> shift, 0);
      const bool same = live == 15 && (key[0] >> shift) == first && (key[1] >> shift) == first &&
                        (key[2] >> shift) == first && (key[3] >> shift) == first;
      const int mask = (1 << bits) - 1;
      if (__all_sync(0xffffffffu, same)) {
        if (lane == 0) atomicAdd(&hist[first & mask], 128);
        continue;
      }
      int zeros = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int bin = int(key[x] >> shift) & mask;
        const bool in = (live >> x) & 1;
        zeros += in && bin == 0;
        if (in && bin != 0) atomicAdd(&hist[bin], 1);
      }
      zeros = __reduce_add_sync(0xffffffffu, zeros);
      if (lane == 0 && zeros) atomicAdd(&hist[0], zeros);
    }
    sync_all();
    // from the top: thread t sums bins top - 4 t .. over the cluster
    const int top = kBins - 1 - kPer * tid;
    int h[kPer] = {};
#pragma unroll 1
    for (int r = 0; r < cs; ++r) {
      const int4 v = *reinterpret_cast<const int4*>((cs > 1 ? cluster.map_shared_rank(hist, r) : hist) + top - 3);
      h[0] += v.w;
      h[1] += v.z;
      h[2] += v.y;
      h[3] += v.x;
    }
    const int sum = (h[0] + h[1]) + (h[2] + h[3]);
    int inc = sum;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, x);
      if (lane >= x) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int begin = int(__reduce_add_sync(0xffffffffu, unsigned(lane < warp ? warp_sum[lane] : 0))) + inc - sum;
    if (begin < need && need <= begin + sum) {
      // the bin that holds the need-th row from the top
      int x = 0;
#pragma unroll
      for (int y = 0; y < kPer - 1; ++y)
        if (x == y && begin + h[y] < need) {
          begin += h[y];
          ++x;
        }
      s_bin = top - x;
      s_need = need - begin;
    }
    sync_all();   // (the other CTAs have read this histogram)
    high = (high << bits) | uint32_t(s_bin);
    need = s_need;
  }
  const uint32_t thr = high;

  // counts per warp: warp w has the rows [j0 + w * span, ...) of this CTA
  const int span = ((j1 - j0 + kWarps - 1) / kWarps + 127) & ~127;
  const int w0 = min(j0 + warp * span, j1), w1 = min(w0 + span, j1);
  Counts c{0, 0, 0, 0};
#pragma unroll 1
  for (int jb = w0; jb < w1; jb += 128) {
    const int j = jb + 4 * lane;
    uint32_t key[4];
    key4(j, key);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int gt = j + x < w1 && key[x] > thr, tie = j + x < w1 && key[x] == thr;
      c.gt += gt;
      c.tie += tie;
      c.gt_below += j + x < k ? gt : 0;
      c.tie_below += j + x < k ? tie : 0;
    }
  }
  c.gt = __reduce_add_sync(0xffffffffu, c.gt);
  c.tie = __reduce_add_sync(0xffffffffu, c.tie);
  c.gt_below = __reduce_add_sync(0xffffffffu, c.gt_below);
  c.tie_below = __reduce_add_sync(0xffffffffu, c.tie_below);
  if (lane == 0) warp_cnt[warp] = c;
  __syncthreads();
  if (warp == 0) {
    Counts t = warp_cnt[lane];
    t.gt = __reduce_add_sync(0xffffffffu, t.gt);
    t.tie = __reduce_add_sync(0xffffffffu, t.tie);
    t.gt_below = __reduce_add_sync(0xffffffffu, t.gt_below);
    t.tie_below = __reduce_add_sync(0xffffffffu, t.tie_below);
    if (lane == 0) cta_cnt = t;
  }
  sync_all();
  int gt = 0, tie = 0, gt_k = 0, tie_k = 0;   // before this warp's rows; before row k
#pragma unroll 1
  for (int r = 0; r < cs; ++r) {
    const Counts* t = cs > 1 ? cluster.map_shared_rank(&cta_cnt, r) : &cta_cnt;
    if (r < rank) {
      gt += t->gt;
      tie += t->tie;
    }
    gt_k += t->gt_below;
    tie_k += t->tie_below;
  }
  gt += int(__reduce_add_sync(0xffffffffu, unsigned(lane < warp ? warp_cnt[lane].gt : 0)));
  tie += int(__reduce_add_sync(0xffffffffu, unsigned(lane < warp ? warp_cnt[lane].tie : 0)));
  const int kept_k = gt_k + min(tie_k, need);
  int32_t* dst = A.lists + lu * 2 * A.list_cap;
  int32_t* src = dst + A.list_cap;
  if (rank == 0 && tid == 0) A.moves[lu] = k - kept_k;
  const unsigned lt = (1u << lane) - 1u;
#pragma unroll 1
  for (int jb = w0; jb < w1; jb += 128) {
    const int j = jb + 4 * lane;
    uint32_t key[4];
    key4(j, key);
    // rows above and at the threshold before this lane's, in the warp
    int above = 0, ties = 0, gt_j = gt, tie_j = tie;
    bool some = false;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const bool in = j + x < w1, eq = in && key[x] == thr;
      const unsigned m = __ballot_sync(0xffffffffu, in && key[x] > thr);
      above += __popc(m);
      gt_j += __popc(m & lt);
      some |= eq;
    }
    if (__any_sync(0xffffffffu, some)) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const unsigned m = __ballot_sync(0xffffffffu, j + x < w1 && key[x] == thr);
        ties += __popc(m);
        tie_j += __popc(m & lt);
      }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (j + x >= w1) break;
      const bool over = key[x] > thr, equal = key[x] == thr;
      const int kept = gt_j + min(tie_j, need);
      const bool keep = over || (equal && tie_j < need);
      if (j + x < k && !keep) dst[j + x - kept] = j + x;
      if (j + x >= k && keep) src[kept - kept_k] = j + x;
      gt_j += over;
      tie_j += equal;
    }
    gt += above;
    tie += ties;
  }
  if (cs > 1) cluster.sync();   // no CTA leaves while its counts are read
}

constexpr int kMoveThreads = 256;
constexpr int kRows = 4;                 // rows a warp has in flight

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs A) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int CH = D / 8;              // 16-byte chunks per row
  constexpr int RPW = 16 / CH;           // rows a half-warp covers at once
  const int unit = blockIdx.y, l = blockIdx.z;
  if (blockIdx.x == 0 && unit == 0 && l == 0)
    for (int b = threadIdx.x; b < A.B; b += kMoveThreads) {
      const int n = A.seq_len[b];
      if (n > A.k && n <= A.Lcap) A.seq_len[b] = A.k;
    }
  const size_t lu = size_t(l) * A.B * A.hkv + unit;
  const int m = A.moves[lu];
  const int32_t* dst = A.lists + lu * 2 * A.list_cap;
  const int32_t* src = dst + A.list_cap;
  const EvictLayerDev& Ly = A.layer[l];
  const int b = unit / A.hkv, g = unit % A.hkv;
  const int lane = threadIdx.x & 31, half = lane >> 4, c = lane & (CH - 1), sub = (lane & 15) / CH;
  uint16_t* base = half ? Ly.v + size_t(b) * Ly.vsb + size_t(g) * Ly.vsh : Ly.k + size_t(b) * Ly.ksb + size_t(g) * Ly.ksh;
  const int64_t sl = half ? Ly.vsl : Ly.ksl;
  uint32_t* weight = reinterpret_cast<uint32_t*>(Ly.weight + size_t(unit) * A.Lcap);
  int32_t* pos = Ly.pos + size_t(unit) * A.Lcap;
  constexpr int STEP = kRows * RPW;      // rows of a warp at once
  const int warps = gridDim.x * (kMoveThreads / 32);
  for (int r0 = (blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5)) * STEP; r0 < m; r0 += warps * STEP) {
    // lane x holds the x-th pair of rows
    int to = 0, of = 0;
    const bool mine = lane < STEP && r0 + lane < m;
    if (mine) {
      to = __ldcg(dst + r0 + lane);
      of = __ldcg(src + r0 + lane);
    }
    uint4 v[kRows];
#pragma unroll
    for (int y = 0; y < kRows; ++y) {
      const int x = y * RPW + sub;
      const int row = __shfl_sync(0xffffffffu, of, x);
      if (r0 + x < m) v[y] = __ldcs(reinterpret_cast<const uint4*>(base + size_t(row) * sl) + c);
    }
    if (mine) {
      weight[to] = weight[of];
      pos[to] = pos[of];
    }
#pragma unroll
    for (int y = 0; y < kRows; ++y) {
      const int x = y * RPW + sub;
      const int row = __shfl_sync(0xffffffffu, to, x);
      if (r0 + x < m) __stcs(reinterpret_cast<uint4*>(base + size_t(row) * sl) + c, v[y]);
    }
  }
}

}  // namespace

cudaError_t evict_launch(EvictArgs& a, int num_sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t attr = once_per_device(done, [] {
    return cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeysMax * 4);
  });
  if (attr != cudaSuccess) return attr;
  const int units = a.B * a.hkv;
  // CTAs per unit: as many as find an SM each, while a CTA keeps kSliceMin rows
  int cs = 1;
  while (cs < kMaxCluster && (long long)units * a.n_layers * cs * 2 <= num_sms && a.Lcap / (cs * 2) >= kSliceMin) cs *= 2;
  a.keys_cap = std::min(((a.Lcap + cs - 1) / cs + 127) & ~127, kKeysMax);
  a.vec4 = a.Lcap % 4 == 0;   // a unit's weights and positions start on 16 bytes
  for (int l = 0; l < a.n_layers; ++l)
    a.vec4 = a.vec4 && ((reinterpret_cast<uintptr_t>(a.layer[l].weight) | reinterpret_cast<uintptr_t>(a.layer[l].pos)) & 15u) == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(units * cs), unsigned(a.n_layers));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = size_t(a.keys_cap) * 4;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = unsigned(cs);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a);
  if (e != cudaSuccess) return e;
  // about sixteen blocks of eight warps per SM over all units, none without rows
  const int rows = std::min(a.k, a.Lcap - a.k);
  if (rows < 1) return cudaSuccess;   // a cache of at most k rows never evicts
  const long long want = std::max(1LL, 16LL * num_sms / ((long long)units * a.n_layers));
  const int per = kMoveThreads / 32 * kRows * (a.D == 64 ? 2 : 1);
  const dim3 grid(unsigned(std::min<long long>(want, (rows + per - 1) / per)), unsigned(units), unsigned(a.n_layers));
  return a.D == 128 ? launch_pdl(evict_move_kernel<128>, grid, dim3(kMoveThreads), 0, stream, a)
                    : launch_pdl(evict_move_kernel<64>, grid, dim3(kMoveThreads), 0, stream, a);
}

}  // namespace dustin
