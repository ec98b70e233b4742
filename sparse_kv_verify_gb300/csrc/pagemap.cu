// Block tables and slot maps of a ragged batch on the GPU (dustin_page_map).
//
// Three prefix sums over the requests carry it: tokens (cu), pages given back and
// pages taken.  With need = ceil((L + n) / page), rel = max(0, held - need) and
// take = max(0, need - held), the i-th page given back is pushed to
// free[n_free + i], the i-th page taken is free[avail - 1 - i] with
// avail = n_free + sum rel, and a request is served iff take = 0 or the inclusive
// sum of take up to it is at most avail.  Pages and tokens are then flat lists,
// each element of which finds its request by a binary search in the sums.
//
// One launch: a cluster whose CTAs all compute the sums (a few KB of lengths) and
// share the lists out among them.  Two cluster barriers order it: every CTA has
// read the state before any writes it, and the pages given back are in the pool
// before any is taken.  A token's page that is taken in this call comes from the
// pool, not from the table, so that slots need not wait for the tables.
//
// Bound by the latency of its chain (lengths -> sums -> pages -> slots): 16 requests
// of one token 2.6 us; 256 requests with 32 K tokens, 4 K pages given back and 8 K
// taken about 10 us (one CTA without the cluster: 41), 6.7 where none is given back
// or taken (7.8 with the loops unrolled by 4: the code is fetched for one pass).
#include "common.cuh"
#include "kernels.h"

namespace dustin {

namespace {

constexpr int kClusterMax = 8;

// Per request, in shared memory: rows in the cache, first token, first page given
// back, first page taken, and pages held before (bit 31: served).
struct Sums {
  int* L;
  int* cu;
  int* rel;
  int* take;
  uint32_t* held;
};

// Exclusive sums over the CTA's threads in order; *total gets the sum of all.
// `sums` holds one value per warp and is used for one scan only.
template <int NTH>
__device__ __forceinline__ long long block_scan(long long mine, long long* sums, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](long long v) {
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, v, x);
      if (lane >= x) v += y;
    }
    return v;
  };
  const long long inc = scan(mine);
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  const long long all = scan(lane < NTH / 32 ? sums[lane] : 0);   // by every warp
  const long long before = __shfl_sync(0xffffffffu, all, warp > 0 ? warp - 1 : 0);
  *total = __shfl_sync(0xffffffffu, all, 31);
  return (warp > 0 ? before : 0) + inc - mine;
}

// The last request whose sum is at most i.
__device__ __forceinline__ int find(const int* sums, int B, int i) {
  int lo = 0, hi = B;   // sums[lo] <= i < sums[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// PER: requests of a thread at most.
template <int NTH, int PER>
__global__ void __launch_bounds__(NTH) page_map_kernel(const __grid_constant__ PageMapArgs A) {
  extern __shared__ int smem[];
  __shared__ long long sums[2][32];
  __shared__ int tops[32];
  const int B = A.B, tid = threadIdx.x, ctas = gridDim.x, rank = blockIdx.x;   // one cluster
  Sums S{smem, smem + B, smem + 2 * B + 1, smem + 3 * B + 1, reinterpret_cast<uint32_t*>(smem + 4 * B + 1)};
  pdl_launch_dependents();
  pdl_wait();

  const int per = (B + NTH - 1) / NTH, b0 = min(tid * per, B), nb = min(per, B - b0);
  int L[PER], n[PER], held[PER];
#pragma unroll
  for (int y = 0; y < PER; ++y) {
    L[y] = n[y] = held[y] = 0;
    if (y < nb) {
      n[y] = __ldcg(A.n_new + b0 + y);
      L[y] = __ldcg(A.seq_len + b0 + y);
      held[y] = __ldcg(A.held + b0 + y);
    }
  }
  const int n_free = __ldcg(A.n_free);
  long long mine = 0, all;
#pragma unroll
  for (int y = 0; y < PER; ++y) mine += max(n[y], 0);
  long long at = block_scan<NTH>(mine, sums[0], &all);
  int flags = 0;
  mine = 0;   // pages given back (upper half) and taken
#pragma unroll
  for (int y = 0; y < PER; ++y) {
    if (y < nb) {
      const int b = b0 + y;
      const long long rows = (long long)L[y] + n[y];
      const bool ok = L[y] >= 0 && n[y] >= 0 && n[y] <= A.max_new && rows <= (long long)A.max_pages * A.page &&
                      at + n[y] <= A.N && held[y] >= 0 && held[y] <= A.max_pages;
      if (!ok) flags |= DUSTIN_DEV_SEQLEN;
      const int need = ok ? int((unsigned(rows) + unsigned(A.page) - 1u) / unsigned(A.page)) : held[y];
      S.L[b] = L[y];
      S.cu[b] = int(at < A.N ? at : A.N);
      S.rel[b] = max(held[y] - need, 0);
      S.take[b] = max(need - held[y], 0);
      S.held[b] = ok ? uint32_t(held[y]) | 0x80000000u : 0u;
      mine += ((long long)S.rel[b] << 32) + S.take[b];
      at += max(n[y], 0);
    }
  }
  if (tid == 0) S.cu[B] = int(all < A.N ? all : A.N);
  const int tokens = int(all < A.N ? all : A.N);
  long long moved;
  const long long moved_at = block_scan<NTH>(mine, sums[1], &moved);
  int rel_at = int(moved_at >> 32), take_at = int(moved_at & 0xFFFFFFFF), rel_all = int(moved >> 32);
  const bool pool = n_free >= 0 && n_free <= A.n_pages && rel_all <= A.n_pages - n_free;
  if (!pool) {
    flags |= DUSTIN_DEV_PAGES;
    rel_all = 0;
  }
  const int avail = pool ? n_free + rel_all : 0;
  if (ctas > 1) {   // every CTA has read the state before any writes it
    cluster_arrive();
    cluster_wait();
  }
  int taken = 0;
#pragma unroll
  for (int y = 0; y < PER; ++y) {
    if (y < nb) {
      const int b = b0 + y, r = S.rel[b], t = S.take[b];
      S.rel[b] = rel_at;
      S.take[b] = take_at;
      if (t > 0) {
        if (take_at + t <= avail) taken = take_at + t;
        else {
          S.held[b] &= 0x7FFFFFFFu;
          flags |= DUSTIN_DEV_PAGES;
        }
      }
      const bool served = S.held[b] >> 31;
      if (rank == 0) {
        if (served && (t > 0 || (r > 0 && pool))) A.held[b] = held[y] + t - r;
        A.kv_len[b] = served ? L[y] + n[y] : 0;
        A.cu[b] = S.cu[b];
      }
      rel_at += r;
      take_at += t;
    }
  }
  if (rank == 0) {
    if (tid == 0) A.cu[B] = tokens;
    if (flags) flag_error(A.err, flags);
  }
  taken = __reduce_max_sync(0xffffffffu, taken);
  if ((tid & 31) == 0) tops[tid >> 5] = taken;
  __syncthreads();
  taken = __reduce_max_sync(0xffffffffu, (tid & 31) < NTH / 32 ? tops[tid & 31] : 0);

  // pages given back: entries past need, which is held less what is given back
  const int first = rank * NTH + tid, stride = ctas * NTH;
#pragma unroll 1
  for (int i = first; i < rel_all; i += stride) {
    const int b = find(S.rel, B, i);
    const int end = b + 1 < B ? S.rel[b + 1] : rel_all, was = int(S.held[b] & 0x7FFFFFFFu);
    A.free_list[n_free + i] = __ldcg(A.table + size_t(b) * A.max_pages + was - (end - i));
  }
  if (rel_all > 0) {   // they are in the pool before any is taken
    if (ctas > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
  }
#pragma unroll 1
  for (int i = first; i < taken; i += stride) {
    const int b = find(S.take, B, i);
    A.table[size_t(b) * A.max_pages + int(S.held[b] & 0x7FFFFFFFu) + (i - S.take[b])] = __ldcg(A.free_list + avail - 1 - i);
  }
  if (rank == 0 && tid == 0 && pool) *A.n_free = avail - taken;
#pragma unroll 1
  for (int i = first; i < A.N; i += stride) {
    int p = 0, s = -1;
    if (i < tokens) {
      const int b = find(S.cu, B + 1, i);
      p = S.L[b] + (i - S.cu[b]);
      if (S.held[b] >> 31) {
        const int was = int(S.held[b] & 0x7FFFFFFFu), j = int(unsigned(p) / unsigned(A.page));
        const int id = __ldcg(j < was ? A.table + size_t(b) * A.max_pages + j : A.free_list + avail - 1 - (S.take[b] + j - was));
        if (id >= 0 && id < A.n_pages) s = id * A.page + (p - j * A.page);
        else flag_error(A.err, DUSTIN_DEV_INDEX);
      }
    }
    A.slot[i] = s;
    A.pos[i] = p;
  }
}

template <int NTH, int PER>
cudaError_t launch_t(const PageMapArgs& a, int ctas, cudaStream_t stream) {
  auto kern = page_map_kernel<NTH, PER>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                int((5 * size_t(NTH) * PER + 1) * 4));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(NTH);
  cfg.dynamicSmemBytes = size_t(5 * a.B + 1) * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

// Few rows: a CTA of few warps, whose scans and barriers are shorter.  Many: a cluster,
// which shares the rows out.  us of a graph node by N, 16 to 256 requests that move no
// page: 256 threads against 1024, N = 16 3.4 and 4.0, 256 4.0 and 4.3, 1024 5.5 and 4.5;
// one CTA of 1024 against eight, N = 2048 5.3 and 4.8, 4096 7.2 and 4.6, 8192 10.7 and
// 4.8, 32768 31.5 and 7.6.  (Each pair is even somewhat below its limit here, at about
// 500 and 1500 rows; between them and the limits 1 to 2.5 us are left.)
cudaError_t page_map_launch(const PageMapArgs& a, cudaStream_t stream) {
  if (a.B <= 256 && a.N <= 1024) return launch_t<256, 1>(a, 1, stream);
  const int ctas = a.N <= 4096 ? 1 : kClusterMax;
  return a.B <= 1024 ? launch_t<1024, 1>(a, ctas, stream) : launch_t<1024, DUSTIN_MAX_REQUESTS / 1024>(a, ctas, stream);
}

}  // namespace dustin
