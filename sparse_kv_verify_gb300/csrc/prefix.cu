// Shared-prefix attention for a draft block.
//
// For query t of sequence b (position i = L + t, L = seq_len[b]) the visible
// keys are the shared prefix (if any), the cache rows j < L and the block rows
// u (position L + u) with j <= i and (i - j < window or j < sinks);
// o = softmax(q.k / sqrt(d)) v and lse = ln sum exp(q.k / sqrt(d)) over them,
// o = 0 and lse = -inf where nothing is visible.
//
// One warp per query row walks its visible keys with a running maximum and
// sum; lane x holds columns x, x + 32, ... of q and of the output.
#include "common.cuh"
#include "kernels.h"

namespace dustin {

namespace {

constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) prefix_kernel(const __grid_constant__ AttendArgs A) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int NC = D / 32;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int T = A.T, hq = A.hq, G = hq / A.hkv;
  if (row >= (long long)A.B * T * hq) return;
  const int h = int(row % hq), t = int(row / hq % T), b = int(row / hq / T), g = h / G;
  int L = A.seq_len[b];
  if (L < 0 || L > A.Lcap) {
    if (lane == 0 && h == 0 && t == 0) flag_error(A.err, DUSTIN_DEV_SEQLEN);
    L = 0;
  }
  int P = 0;
  if (A.prefix_len) {
    P = *A.prefix_len;
    if (P < 0 || P > A.Pcap) {
      if (lane == 0 && row == 0) flag_error(A.err, DUSTIN_DEV_SEQLEN);
      P = 0;
    }
  }
  float q[NC], o[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    q[c] = __uint_as_float(uint32_t(A.q[row * D + 32 * c + lane]) << 16) * A.scale_log2;
    o[c] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  auto key = [&](const uint16_t* kr, const uint16_t* vr) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) s = fmaf(q[c], __uint_as_float(uint32_t(kr[32 * c + lane]) << 16), s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s);
    const float a = exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int c = 0; c < NC; ++c)
      o[c] = o[c] * a + w * __uint_as_float(uint32_t(vr[32 * c + lane]) << 16);
  };
  for (int j = 0; j < P; ++j)
    key(A.pk + size_t(g) * A.pksh + size_t(j) * A.pksl, A.pv + size_t(g) * A.pvsh + size_t(j) * A.pvsl);
  const long long i = (long long)L + t;
  const int s_end = A.sinks < L ? A.sinks : L;
  const long long lo = i - A.window + 1;
  const uint16_t* kc = A.k + size_t(b) * A.ksb + size_t(g) * A.ksh;
  const uint16_t* vc = A.v + size_t(b) * A.vsb + size_t(g) * A.vsh;
  for (int j = 0; j < s_end; ++j) key(kc + size_t(j) * A.ksl, vc + size_t(j) * A.vsl);
  for (long long j = lo > s_end ? lo : s_end; j < L; ++j)
    key(kc + size_t(j) * A.ksl, vc + size_t(j) * A.vsl);
  const size_t blk = (size_t(b) * A.hkv + g) * T * D;
  for (int u = 0; u <= t; ++u)
    if (t - u < A.window || L + u < A.sinks) key(A.kb + blk + size_t(u) * D, A.vb + blk + size_t(u) * D);
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
    A.o[row * D + 32 * c + lane] = __bfloat16_as_ushort(__float2bfloat16_rn(o[c] * inv));
  if (A.lse && lane == 0) A.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

cudaError_t prefix_launch(const AttendArgs& a, int D, cudaStream_t stream) {
  const long long rows = (long long)a.B * a.T * a.hq;
  const dim3 grid(unsigned((rows + kWarps - 1) / kWarps));
  return D == 128 ? launch_pdl(prefix_kernel<128>, grid, dim3(32 * kWarps), 0, stream, a)
                  : launch_pdl(prefix_kernel<64>, grid, dim3(32 * kWarps), 0, stream, a);
}

}  // namespace dustin
