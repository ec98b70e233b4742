// Causal attention of a ragged batch's new tokens over a paged cache
// (dustin_paged_attn): query t of request b, at position p = kv_len - n + t, gets
// o = softmax(q.k / sqrt(d)) v and lse = ln sum exp(q.k / sqrt(d)) over the cache
// rows 0..p, row j in row j % page of page table[b][j / page].
//
// One warp per (token, query head): 32 keys at a time, a lane for each key's
// score, then a lane for D / 32 columns of the output; running maximum and sum.
#include "common.cuh"
#include "kernels.h"

namespace dustin {

namespace {

constexpr int kWarps = 4;
constexpr float kNaN = __builtin_nanf("");

template <int D>
__global__ void __launch_bounds__(32 * kWarps) paged_kernel(const __grid_constant__ PagedArgs A) {
  __shared__ float qs[kWarps][D];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y * kWarps + warp, i = blockIdx.x;
  // the request of row i: the first whose tokens end behind it
  int lo = -1, hi = A.B;   // cu[lo + 1] <= i < cu[hi + 1], as far as cu ascends
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (A.cu[mid + 1] <= i) lo = mid;
    else hi = mid;
  }
  if (i == 0 && h == 0)
    for (int b = lane; b < A.B; b += 32)
      if (!paged_ok(A, A.cu[b], A.cu[b + 1], A.kv_len[b])) flag_error(A.err, DUSTIN_DEV_SEQLEN);
  const int b = hi;
  if (h >= A.hq || b >= A.B) return;
  const int c0 = A.cu[b], c1 = A.cu[b + 1], kv = A.kv_len[b];
  if (!paged_ok(A, c0, c1, kv) || i < c0) return;
  const int p = kv - (c1 - c0) + (i - c0), g = h / (A.hq / A.hkv);
  constexpr int C = D / 32;
  for (int x = lane; x < D; x += 32)
    qs[warp][x] = __uint_as_float(uint32_t(A.q[(size_t(i) * A.hq + h) * D + x]) << 16);
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[C] = {};
  for (int j0 = 0; j0 <= p; j0 += 32) {
    const int j = j0 + lane;
    float s = -INFINITY;
    int id = -1, r = 0;
    if (j <= p) {
      id = A.table[size_t(b) * A.max_pages + j / A.page];
      r = j % A.page;
      if (id < 0 || id >= A.n_pages) {
        flag_error(A.err, DUSTIN_DEV_INDEX);
        id = -1;
      }
      s = 0.f;
      if (id >= 0) {
        const uint16_t* k = A.k + id * A.ksp + g * A.ksh + r * A.ksl;
        for (int x = 0; x < D; ++x) s = fmaf(qs[warp][x], __uint_as_float(uint32_t(k[x]) << 16), s);
      }
      s *= A.scale_log2;
    }
    float top = fmaxf(m, s);
#pragma unroll
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float base = top == -INFINITY ? 0.f : top, alpha = fast_exp2(m - base), w = fast_exp2(s - base);
    m = top;
    float sum = w;
#pragma unroll
    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    l = fmaf(l, alpha, sum);
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] *= alpha;
    for (int x = 0; x < 32 && j0 + x <= p; ++x) {
      const int idx = __shfl_sync(0xffffffffu, id, x), rx = __shfl_sync(0xffffffffu, r, x);
      const float wx = bf16_round(__shfl_sync(0xffffffffu, w, x));
      if (idx < 0) continue;
      const uint16_t* v = A.v + idx * A.vsp + g * A.vsh + rx * A.vsl;
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] = fmaf(wx, __uint_as_float(uint32_t(v[lane * C + c]) << 16), o[c]);
    }
  }
  const size_t row = size_t(i) * A.hq + h;
  const float inv = l != 0.f ? 1.f / l : p >= 0 ? kNaN : 0.f;   // (a NaN stays one)
#pragma unroll
  for (int c = 0; c < C; c += 2)
    *reinterpret_cast<uint32_t*>(A.o + row * D + lane * C + c) = pack_bf16(o[c] * inv, o[c + 1] * inv);
  if (A.lse && lane == 0) A.lse[row] = l != 0.f ? (m + log2f(l)) * kLn2 : p >= 0 ? kNaN : -INFINITY;
}

}  // namespace

cudaError_t paged_launch(PagedArgs& a, int D, int, cudaStream_t stream) {
  const dim3 grid(a.N, (a.hq + kWarps - 1) / kWarps);
  return D == 128 ? launch_pdl(paged_kernel<128>, grid, dim3(32 * kWarps), 0, stream, a)
                  : launch_pdl(paged_kernel<64>, grid, dim3(32 * kWarps), 0, stream, a);
}

}  // namespace dustin
