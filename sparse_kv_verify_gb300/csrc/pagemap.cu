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
// One CTA; bound by the latency of its chain (lengths -> sums -> pages -> slots).
#include "common.cuh"
#include "kernels.h"

namespace dustin {

namespace {

constexpr int NTH = 1024;

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
template <typename T>
__device__ T block_scan(T mine, T* warp_sums, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T inc = mine;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, inc, x);
    if (lane >= x) inc += y;
  }
  __syncthreads();   // (warp_sums may still be read from the scan before)
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  T before = 0, all = 0;
  for (int w = 0; w < NTH / 32; ++w) {
    const T s = warp_sums[w];
    before += w < warp ? s : T(0);
    all += s;
  }
  *total = all;
  return before + inc - mine;
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

__global__ void __launch_bounds__(NTH) page_map_kernel(const __grid_constant__ PageMapArgs A) {
  extern __shared__ int smem[];
  __shared__ long long wide[NTH / 32];
  __shared__ int narrow[NTH / 32];
  const int B = A.B, tid = threadIdx.x;
  Sums S{smem, smem + B, smem + 2 * B + 1, smem + 3 * B + 1, reinterpret_cast<uint32_t*>(smem + 4 * B + 1)};
  pdl_launch_dependents();
  pdl_wait();

  const int per = (B + NTH - 1) / NTH, b0 = min(tid * per, B), b1 = min(b0 + per, B);
  long long mine = 0, all;
  for (int b = b0; b < b1; ++b) mine += max(A.n_new[b], 0);
  long long at = block_scan(mine, wide, &all);
  const int n_free = *A.n_free;
  int rel = 0, take = 0, flags = 0;
  for (int b = b0; b < b1; ++b) {
    const int L = A.seq_len[b], n = A.n_new[b], held = A.held[b];
    const long long rows = (long long)L + n;
    const bool ok = L >= 0 && n >= 0 && n <= A.max_new && rows <= (long long)A.max_pages * A.page && at + n <= A.N &&
                    held >= 0 && held <= A.max_pages;
    if (!ok) flags |= DUSTIN_DEV_SEQLEN;
    const int need = ok ? int((rows + A.page - 1) / A.page) : held;
    S.L[b] = L;
    S.cu[b] = int(at < A.N ? at : A.N);
    S.rel[b] = max(held - need, 0);
    S.take[b] = max(need - held, 0);
    S.held[b] = ok ? uint32_t(held) | 0x80000000u : 0u;
    rel += S.rel[b];
    take += S.take[b];
    at += max(n, 0);
  }
  if (tid == 0) S.cu[B] = int(all < A.N ? all : A.N);
  int rel_all, take_all;
  int rel_at = block_scan(rel, narrow, &rel_all);
  int take_at = block_scan(take, narrow, &take_all);
  const bool pool = n_free >= 0 && n_free <= A.n_pages && rel_all <= A.n_pages - n_free;
  if (!pool) {
    flags |= DUSTIN_DEV_PAGES;
    rel_all = 0;
  }
  const int avail = pool ? n_free + rel_all : 0;
  int taken = 0;
  for (int b = b0; b < b1; ++b) {
    const int r = S.rel[b], t = S.take[b];
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
    const int held = int(S.held[b] & 0x7FFFFFFFu);
    if (served && (t > 0 || (r > 0 && pool))) A.held[b] = held + t - r;
    A.kv_len[b] = served ? S.L[b] + A.n_new[b] : 0;
    A.cu[b] = S.cu[b];
    rel_at += r;
    take_at += t;
  }
  if (tid == 0) A.cu[B] = S.cu[B];
  if (flags) flag_error(A.err, flags);
  taken = __reduce_max_sync(0xffffffffu, taken);
  __syncthreads();
  if ((tid & 31) == 0) narrow[tid >> 5] = taken;
  __syncthreads();
  for (int w = 0; w < NTH / 32; ++w) taken = max(taken, narrow[w]);

  // pages given back: entries past need, which is held less what is given back
  for (int i = tid; i < rel_all; i += NTH) {
    const int b = find(S.rel, B, i);
    const int end = b + 1 < B ? S.rel[b + 1] : rel_all, held = int(S.held[b] & 0x7FFFFFFFu);
    A.free_list[n_free + i] = A.table[size_t(b) * A.max_pages + held - (end - i)];
  }
  __syncthreads();
  for (int i = tid; i < taken; i += NTH) {
    const int b = find(S.take, B, i);
    A.table[size_t(b) * A.max_pages + int(S.held[b] & 0x7FFFFFFFu) + (i - S.take[b])] = A.free_list[avail - 1 - i];
  }
  if (tid == 0 && pool) *A.n_free = avail - taken;
  __syncthreads();
  const int tokens = S.cu[B];
  for (int i = tid; i < A.N; i += NTH) {
    int p = 0, s = -1;
    if (i < tokens) {
      const int b = find(S.cu, B + 1, i);
      p = S.L[b] + (i - S.cu[b]);
      if (S.held[b] >> 31) {
        const int id = A.table[size_t(b) * A.max_pages + p / A.page];
        if (id >= 0 && id < A.n_pages) s = id * A.page + p % A.page;
        else flag_error(A.err, DUSTIN_DEV_INDEX);
      }
    }
    A.slot[i] = s;
    A.pos[i] = p;
  }
}

}  // namespace

cudaError_t page_map_launch(const PageMapArgs& a, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t attr = once_per_device(done, [] {
    return cudaFuncSetAttribute(page_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (5 * DUSTIN_MAX_REQUESTS + 1) * 4);
  });
  if (attr != cudaSuccess) return attr;
  return launch_pdl(page_map_kernel, dim3(1), dim3(NTH), size_t(5 * a.B + 1) * 4, stream, a);
}

}  // namespace dustin
