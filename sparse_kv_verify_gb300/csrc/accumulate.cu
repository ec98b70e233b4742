// Accumulated attention weights of a cache's rows.
//
// The last n = n_new[b] of the L = seq_len[b] cache rows are the accepted rows
// of the last draft block and the first n of its T query rows are theirs: query
// t sits at row L - n + t.  For every row j,
//   weight[j] += sum over t < n with j <= L - n + t and over the G query heads
//                of the KV head, of exp(q.k_j / sqrt(d) - lse[t]),
// where the new rows start from 0 and get pos[j] = n_seen[b] - (L - j).
//
// One thread per cache row; the query rows go by in shared memory.
#include "common.cuh"
#include "kernels.h"

namespace dustin {

namespace {

constexpr int kThreads = 128;

template <int D>
__global__ void __launch_bounds__(kThreads) accumulate_kernel(const __grid_constant__ AccumulateArgs A) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float q[D];
  const int g = blockIdx.y % A.hkv, b = blockIdx.y / A.hkv;
  const int L = A.seq_len[b], n = A.n_new[b], seen = A.n_seen[b];
  if (!accumulate_ok(A, L, n, seen)) {
    if (g == 0 && blockIdx.x == 0 && threadIdx.x == 0) flag_error(A.err, DUSTIN_DEV_APPEND);
    return;
  }
  const int j = blockIdx.x * kThreads + threadIdx.x;
  if (int(blockIdx.x) * kThreads >= L) return;
  const uint16_t* kr = A.k + size_t(b) * A.ksb + size_t(g) * A.ksh + size_t(j) * A.ksl;
  float k[D];
  for (int c = 0; c < D; ++c) k[c] = j < L ? __uint_as_float(uint32_t(kr[c]) << 16) : 0.f;
  float add = 0.f;
  for (int t = 0; t < n; ++t)
    for (int h = g * A.G; h < (g + 1) * A.G; ++h) {
      const size_t row = (size_t(b) * A.T + t) * A.hkv * A.G + h;
      __syncthreads();
      for (int c = threadIdx.x; c < D; c += kThreads) q[c] = __uint_as_float(uint32_t(A.q[row * D + c]) << 16);
      __syncthreads();
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < D; ++c) s = fmaf(k[c], q[c], s);
      const float lse = A.lse[row];
      if (j <= L - n + t && lse != -INFINITY) add += exp2f(s * A.scale_log2 - lse * kLog2e);
    }
  if (j < L) {
    const size_t at = (size_t(b) * A.hkv + g) * A.Lcap + j;
    const bool fresh = j >= L - n;
    A.weight[at] = (fresh ? 0.f : A.weight[at]) + add;
    if (fresh) A.pos[at] = seen - (L - j);
  }
}

}  // namespace

cudaError_t accumulate_launch(const AccumulateArgs& a, int D, cudaStream_t stream) {
  const dim3 grid((a.Lcap + kThreads - 1) / kThreads, a.B * a.hkv);
  return D == 128 ? launch_pdl(accumulate_kernel<128>, grid, dim3(kThreads), 0, stream, a)
                  : launch_pdl(accumulate_kernel<64>, grid, dim3(kThreads), 0, stream, a);
}

}  // namespace dustin
