// Eviction from a cache by accumulated attention weight.
//
// A (layer, sequence, KV head) unit with n = seq_len[b] > k rows keeps k of
// them: those at positions below `sinks` or among the last `window` positions
// seen, then the largest weights (equal weights: the lower row).  The rows it
// drops below k, in order, take the rows it keeps at or beyond k, in order --
// sources and destinations never overlap, and as few rows move as can.
//
// One CTA per unit: a radix select over the 32-bit keys finds the threshold
// and how many rows that equal it stay, one ordered scan lists holes and
// movers, then the warps copy them.
#include "common.cuh"
#include "kernels.h"

namespace dustin {

namespace {

constexpr int kThreads = 512;
constexpr int kWarpsN = kThreads / 32;

// exclusive rank of this thread's flag within the block, and the block's count
__device__ __forceinline__ int block_rank(bool f, int* warp_sum, int* total) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned bal = __ballot_sync(0xffffffffu, f);
  __syncthreads();
  if (lane == 0) warp_sum[w] = __popc(bal);
  __syncthreads();
  int before = 0, all = 0;
  for (int x = 0; x < kWarpsN; ++x) {
    before += x < w ? warp_sum[x] : 0;
    all += warp_sum[x];
  }
  *total = all;
  return before + __popc(bal & ((1u << lane) - 1u));
}

__global__ void __launch_bounds__(kThreads) evict_kernel(const __grid_constant__ EvictArgs A) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ int hist[256];
  __shared__ int warp_sum[kWarpsN];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int unit = blockIdx.x, l = blockIdx.y;
  const int b = unit / A.hkv, g = unit % A.hkv;
  const EvictLayerDev& Ly = A.layer[l];
  const int n = A.seq_len[b], k = A.k;
  if (n < 0 || n > A.Lcap) {
    if (threadIdx.x == 0 && g == 0 && l == 0) flag_error(A.err, DUSTIN_DEV_SEQLEN);
    return;
  }
  if (n <= k) return;
  float* weight = Ly.weight + size_t(unit) * A.Lcap;
  int32_t* pos = Ly.pos + size_t(unit) * A.Lcap;
  const int recent = A.n_seen[b] - A.window;
  auto key_of = [&](int j) -> uint32_t {
    const int p = pos[j];
    return p < A.sinks || p >= recent ? 0xFFFFFFFFu : importance_key(weight[j], A.err);
  };
  uint32_t prefix = 0, mask = 0;
  int need = k;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int x = threadIdx.x; x < 256; x += kThreads) hist[x] = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kThreads) {
      const uint32_t key = key_of(j);
      if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int left = need, x = 255;
      while (x > 0 && hist[x] < left) left -= hist[x--];
      s_prefix = prefix | (uint32_t(x) << shift);
      s_need = left;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    mask |= 255u << shift;
    __syncthreads();
  }
  int32_t* dst = A.lists + (size_t(l) * A.B * A.hkv + unit) * 2 * k;
  int32_t* src = dst + k;
  int ties = 0, holes = 0, movers = 0;
  for (int j0 = 0; j0 < n; j0 += kThreads) {
    const int j = j0 + threadIdx.x;
    const uint32_t key = j < n ? key_of(j) : 0u;
    const bool tie = j < n && key == prefix;
    int all;
    const int tr = ties + block_rank(tie, warp_sum, &all);
    ties += all;
    const bool keep = j < n && (key > prefix || (tie && tr < need));
    const bool hole = j < k && !keep, move = j >= k && keep;
    const int hr = block_rank(hole, warp_sum, &all);
    if (hole) dst[holes + hr] = j;
    holes += all;
    const int mr = block_rank(move, warp_sum, &all);
    if (move) src[movers + mr] = j;
    movers += all;
  }
  __syncthreads();
  const int chunks = A.D / 8;
  uint16_t* kc = Ly.k + size_t(b) * Ly.ksb + size_t(g) * Ly.ksh;
  uint16_t* vc = Ly.v + size_t(b) * Ly.vsb + size_t(g) * Ly.vsh;
  for (int x = threadIdx.x; x < movers * chunks; x += kThreads) {
    const int r = x / chunks, c = x % chunks;
    const int to = dst[r], of = src[r];
    reinterpret_cast<uint4*>(kc + size_t(to) * Ly.ksl)[c] = reinterpret_cast<const uint4*>(kc + size_t(of) * Ly.ksl)[c];
    reinterpret_cast<uint4*>(vc + size_t(to) * Ly.vsl)[c] = reinterpret_cast<const uint4*>(vc + size_t(of) * Ly.vsl)[c];
    if (c == 0) {
      weight[to] = weight[of];
      pos[to] = pos[of];
    }
  }
}

__global__ void evict_length_kernel(const __grid_constant__ EvictArgs A) {
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= A.B) return;
  const int n = A.seq_len[b];
  if (n > A.k && n <= A.Lcap) A.seq_len[b] = A.k;
}

}  // namespace

size_t evict_scratch_bytes(int B, int hkv, int n_layers, int k) {
  return size_t(n_layers) * B * hkv * 2 * size_t(k) * 4;
}

cudaError_t evict_launch(const EvictArgs& a, cudaStream_t stream) {
  const cudaError_t e = launch_pdl(evict_kernel, dim3(a.B * a.hkv, a.n_layers), dim3(kThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(evict_length_kernel, dim3((a.B + 127) / 128), dim3(128), 0, stream, a);
}

}  // namespace dustin
