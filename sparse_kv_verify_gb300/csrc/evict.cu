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
//           weight) is formed once and kept in shared memory; three histogram
//           passes of 11, 11 and 10 bits, summed over the cluster's CTAs, give
//           the k-th largest key and how many rows that equal it stay.  With
//           kept(j) = rows kept before row j, a hole j < k is the
//           (j - kept(j))-th and a mover j >= k the (kept(j) - kept(k))-th of
//           its list, so both lists are written from one ordered count of keys
//           above and equal to the threshold.
//   move    bound by the bytes of the rows: every warp moves eight rows at a
//           time, a row's K and V by half a warp each, loads before stores.
//           It also sets the lengths, which the first launch read.
#include <algorithm>

#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace dustin {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kKeysMax = 48 * 1024;      // keys that a CTA keeps in shared memory
constexpr int kMaxCluster = 8;
constexpr int kSliceMin = 4096;          // rows per CTA below which more CTAs do not help

struct Counts {
  int gt, tie, gt_below, tie_below;      // keys above / at the threshold; of these the rows < k
};

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
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int unit = blockIdx.x / cs, l = blockIdx.y;
  const int b = unit / A.hkv, g = unit % A.hkv, k = A.k;
  const size_t lu = size_t(l) * A.B * A.hkv + unit;
  const int n = A.seq_len[b];
  if (n < 0 || n > A.Lcap || n <= k) {   // the whole cluster leaves
    if (rank == 0 && tid == 0) {
      if ((n < 0 || n > A.Lcap) && g == 0 && l == 0) flag_error(A.err, DUSTIN_DEV_SEQLEN);
      A.moves[lu] = 0;
    }
    return;
  }
  const float* weight = A.layer[l].weight + size_t(unit) * A.Lcap;
  const int32_t* pos = A.layer[l].pos + size_t(unit) * A.Lcap;
  const int recent = A.n_seen[b] - A.window;
  // this CTA's rows [j0, j1); a warp takes 128 of them at a time, four
  // neighbours to a lane
  const int slice = ((n + cs - 1) / cs + 127) & ~127;
  const int j0 = min(rank * slice, n), j1 = min(j0 + slice, n);
  const bool cached = slice <= A.keys_cap;
  auto key_of = [&](int p, float w) -> uint32_t {
    return p < A.sinks || p >= recent ? 0xFFFFFFFFu : importance_key(w, A.err);
  };
  // keys of rows j .. j + 3 (j a multiple of 4; 0 for rows at or beyond j1)
  auto fresh4 = [&](int j) -> uint4 {
    uint4 key = make_uint4(0, 0, 0, 0);
    if (A.vec4 && j + 4 <= j1) {
      const int4 p = __ldcg(reinterpret_cast<const int4*>(pos + j));
      const float4 w = __ldcg(reinterpret_cast<const float4*>(weight + j));
      key = make_uint4(key_of(p.x, w.x), key_of(p.y, w.y), key_of(p.z, w.z), key_of(p.w, w.w));
    } else {
      if (j < j1) key.x = key_of(__ldcg(pos + j), __ldcg(weight + j));
      if (j + 1 < j1) key.y = key_of(__ldcg(pos + j + 1), __ldcg(weight + j + 1));
      if (j + 2 < j1) key.z = key_of(__ldcg(pos + j + 2), __ldcg(weight + j + 2));
      if (j + 3 < j1) key.w = key_of(__ldcg(pos + j + 3), __ldcg(weight + j + 3));
    }
    return key;
  };
  auto key4 = [&](int j) -> uint4 { return cached ? *reinterpret_cast<const uint4*>(keys + (j - j0)) : fresh4(j); };

  if (cached) {   // (a thread reads back the keys that it wrote)
#pragma unroll 4
    for (int j = j0 + 4 * tid; j < j1; j += 4 * kThreads) *reinterpret_cast<uint4*>(keys + (j - j0)) = fresh4(j);
  }

  // the k-th largest key, digit by digit
  uint32_t high = 0;      // digits so far
  int need = k;           // rows still to take among the keys that share them
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    for (int x = tid; x < kBins; x += kThreads) hist[x] = 0;
    __syncthreads();
#pragma unroll 4
    for (int jb = j0 + 128 * warp; jb < j1; jb += 4 * kThreads) {
      const int j = jb + 4 * lane;
      const uint4 q = key4(j);
      const uint32_t key[4] = {q.x, q.y, q.z, q.w};
      int bin[4];
      bool in[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        in[x] = j + x < j1 && (pass == 0 || (key[x] >> (shift + bits)) == high);
        bin[x] = int((key[x] >> shift) & ((1u << bits) - 1u));
      }
      // a warp whose rows share a bin (a protected run, weights that were never
      // touched) counts them at once
      const bool one = bin[0] == bin[1] && bin[0] == bin[2] && bin[0] == bin[3] && in[0] && in[1] && in[2] && in[3];
      const int first = __shfl_sync(0xffffffffu, bin[0], 0);   // by every lane
      if (__all_sync(0xffffffffu, one && bin[0] == first)) {
        if (lane == 0) atomicAdd(&hist[first], 128);
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (in[x]) atomicAdd(&hist[bin[x]], 1);
      }
    }
    if (cs > 1) cluster.sync();
    else __syncthreads();
    // from the top: thread t sums bins 2047 - 2 t and 2046 - 2 t over the cluster
    int h0 = 0, h1 = 0;
    for (int r = 0; r < cs; ++r) {
      const int* h = cs > 1 ? cluster.map_shared_rank(hist, r) : hist;
      h0 += h[kBins - 1 - 2 * tid];
      h1 += h[kBins - 2 - 2 * tid];
    }
    int inc = h0 + h1;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, x);
      if (lane >= x) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    const int end = before + inc, begin = end - h0 - h1;
    if (begin < need && need <= end) {
      const bool top = need <= begin + h0;
      s_bin = kBins - (top ? 1 : 2) - 2 * tid;
      s_need = need - begin - (top ? 0 : h0);
    }
    if (cs > 1) cluster.sync();   // the other CTAs have read this histogram
    else __syncthreads();
    high = (high << bits) | uint32_t(s_bin);
    need = s_need;
  }
  const uint32_t thr = high;

  // counts per warp: warp w has the rows [j0 + w * span, ...) of this CTA
  const int span = ((j1 - j0 + kWarps - 1) / kWarps + 127) & ~127;
  const int w0 = min(j0 + warp * span, j1), w1 = min(w0 + span, j1);
  Counts c{0, 0, 0, 0};
#pragma unroll 2
  for (int jb = w0; jb < w1; jb += 128) {
    const int j = jb + 4 * lane;
    const uint4 q = key4(j);
    const uint32_t key[4] = {q.x, q.y, q.z, q.w};
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
  if (cs > 1) cluster.sync();
  else __syncthreads();
  int gt = 0, tie = 0, gt_k = 0, tie_k = 0;   // before this warp's rows; before row k
  for (int r = 0; r < cs; ++r) {
    const Counts* t = cs > 1 ? cluster.map_shared_rank(&cta_cnt, r) : &cta_cnt;
    if (r < rank) {
      gt += t->gt;
      tie += t->tie;
    }
    gt_k += t->gt_below;
    tie_k += t->tie_below;
  }
  for (int w = 0; w < warp; ++w) {
    gt += warp_cnt[w].gt;
    tie += warp_cnt[w].tie;
  }
  const int kept_k = gt_k + min(tie_k, need);
  int32_t* dst = A.lists + lu * 2 * A.list_cap;
  int32_t* src = dst + A.list_cap;
  if (rank == 0 && tid == 0) A.moves[lu] = k - kept_k;
#pragma unroll 2
  for (int jb = w0; jb < w1; jb += 128) {
    const int j = jb + 4 * lane;
    const uint4 q = key4(j);
    const uint32_t key[4] = {q.x, q.y, q.z, q.w};
    int mine = 0;                       // above in the high, ties in the low half
#pragma unroll
    for (int x = 0; x < 4; ++x)
      mine += j + x < w1 ? (key[x] > thr ? 1 << 16 : key[x] == thr ? 1 : 0) : 0;
    int inc = mine;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, x);
      if (lane >= x) inc += y;
    }
    const int ahead = inc - mine, all = __shfl_sync(0xffffffffu, inc, 31);
    int gt_j = gt + (ahead >> 16), tie_j = tie + (ahead & 0xFFFF);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (j + x >= w1) break;
      const bool above = key[x] > thr, equal = key[x] == thr;
      const int kept = gt_j + min(tie_j, need);
      const bool keep = above || (equal && tie_j < need);
      if (j + x < k && !keep) dst[j + x - kept] = j + x;
      if (j + x >= k && keep) src[kept - kept_k] = j + x;
      gt_j += above;
      tie_j += equal;
    }
    gt += all >> 16;
    tie += all & 0xFFFF;
  }
  if (cs > 1) cluster.sync();   // no CTA leaves while its counts are read
}

constexpr int kMoveThreads = 256;
constexpr int kRows = 8;                 // rows a warp has in flight

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
      if (r0 + x < m) reinterpret_cast<uint4*>(base + size_t(row) * sl)[c] = v[y];
    }
  }
}

}  // namespace

cudaError_t evict_launch(EvictArgs& a, int num_sms, cudaStream_t stream) {
  static const cudaError_t attr =
      cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeysMax * 4);
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
  // about eight blocks of eight warps per SM over all units, none without rows
  const int rows = std::min(a.k, a.Lcap - a.k);
  if (rows < 1) return cudaSuccess;   // a cache of at most k rows never evicts
  const long long want = std::max(1LL, 8LL * num_sms / ((long long)units * a.n_layers));
  const int per = kMoveThreads / 32 * kRows * (a.D == 64 ? 2 : 1);
  const dim3 grid(unsigned(std::min<long long>(want, (rows + per - 1) / per)), unsigned(units), unsigned(a.n_layers));
  return a.D == 128 ? launch_pdl(evict_move_kernel<128>, grid, dim3(kMoveThreads), 0, stream, a)
                    : launch_pdl(evict_move_kernel<64>, grid, dim3(kMoveThreads), 0, stream, a);
}

}  // namespace dustin
