// Norm of each head, position rotation and cache write of new tokens
// (dustin_norm_rope): y = x rsqrt(mean x^2 + eps) w, then pairs (a, b) turned by
// t = pos * inv_freq[j]: (a cos t - b sin t, b cos t + a sin t).
//
// A head is 16 elements in each of D / 16 lanes, as the two 16-byte chunks that
// hold the pairs' two halves, so that a rotation needs no exchange between lanes
// (interleaved pairs lie inside a chunk).  The angles of a token serve all its
// heads: a CTA computes them for its tokens once, into shared memory, while its
// first heads' loads are on their way; each head's loads are issued before the
// head before it is computed.
//
// Angles: inv_freq / 2 pi as a fraction of 2^64 times the position, modulo 2^64,
// is the fraction of a turn without any rounding that grows with the position;
// its upper 32 bits are the half-turns in [-1, 1) that sincospif takes.
//
// Bound by the bytes: each row is read and written once.  16384 tokens, 64/8/128:
// 112 us for 671 MB, 6.0 TB/s (0.88 of a plain copy's rate).  One token: 2.6 us, the
// latency of one launch.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace dustin {

namespace {

constexpr int NTH = 128, kPerSm = 8;   // threads of a CTA, CTAs per SM
constexpr int kTokensMax = 32;   // tokens of a CTA at most

__device__ __forceinline__ void unpack8(const uint4& u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// CTA (x, y): tokens [x tb, (x + 1) tb), every gridDim.y-th run of heads.
template <int D>
__global__ void __launch_bounds__(NTH, kPerSm) rope_kernel(const __grid_constant__ RopeArgs A, int tb) {
  constexpr int LPH = D / 16, GROUPS = NTH / LPH;   // lanes per head, heads at a time
  extern __shared__ float2 cs[];                    // [tb][rot / 2]
  __shared__ int2 rows[kTokensMax];                 // page and row of the cache, or -1
  const int tid = threadIdx.x, i0 = blockIdx.x * tb, nt = min(tb, A.N - i0);
  const int half = A.rot / 2, heads = A.hq + 2 * A.hkv;
  const int lane = tid % LPH, turned = A.rot / 16;
  const bool turns = lane < turned;
  // chunks of 8 elements of this lane, and the angles of their pairs
  int c0 = 2 * lane, c1 = 2 * lane + 1;
  if (turns && !A.interleaved) {
    c0 = lane;
    c1 = turned + lane;
  }
  auto load = [&](int t, int h, uint4& u0, uint4& u1) {
    const int64_t i = i0 + t;
    const uint16_t* src = h < A.hq           ? A.q + i * A.qst + h * D
                          : h < A.hq + A.hkv ? A.k + i * A.kst + (h - A.hq) * D
                                             : A.v + i * A.vst + (h - A.hq - A.hkv) * D;
    u0 = *reinterpret_cast<const uint4*>(src + 8 * c0);
    u1 = *reinterpret_cast<const uint4*>(src + 8 * c1);
  };
  const int step = GROUPS * gridDim.y;
  int t = 0, h = blockIdx.y * GROUPS + tid / LPH;
  auto settle = [&](int& t, int& h) {
    while (h >= heads) {
      h -= heads;
      ++t;
    }
  };
  settle(t, h);
  pdl_launch_dependents();
  pdl_wait();
  uint4 u0 = {}, u1 = {};
  if (t < nt) load(t, h, u0, u1);
  for (int x = tid; x < nt * half; x += NTH) {
    const int tx = x / half, j = x - tx * half;
    const double all = double(A.inv_freq[j]) * 0.15915494309189533577;   // 1 / (2 pi)
    const unsigned long long one = __double2ull_rn((all - floor(all)) * 18446744073709551616.0);
    const long long turn = (long long)(one * (unsigned long long)(long long)A.pos[i0 + tx]);
    float s, c;
    sincospif(float(int(turn >> 32)) * 0x1p-31f, &s, &c);
    cs[x] = make_float2(c, s);
  }
  if (tid < nt) {
    const int s = A.slot[i0 + tid];
    const bool ok = s >= 0 && (long long)s < (long long)A.n_pages * A.page;
    if (!ok && s != -1) flag_error(A.err, DUSTIN_DEV_INDEX);
    rows[tid] = ok ? make_int2(s / A.page, s % A.page) : make_int2(-1, 0);
  }
  __syncthreads();

  const uint32_t who = ((1u << LPH) - 1u) << (tid & 31 & ~(LPH - 1));   // the lanes of a head
  while (t < nt) {
    int tn = t, hn = h + step;
    settle(tn, hn);
    uint4 n0 = {}, n1 = {};
    if (tn < nt) load(tn, hn, n0, n1);
    const bool is_q = h < A.hq, is_v = h >= A.hq + A.hkv;
    if (!is_v) {
      float a[8], b[8];
      unpack8(u0, a);
      unpack8(u1, b);
      const uint16_t* w = is_q ? A.q_w : A.k_w;
      if (w) {
        float ss = 0.f;
#pragma unroll
        for (int y = 0; y < 8; ++y) ss = fmaf(a[y], a[y], fmaf(b[y], b[y], ss));
#pragma unroll
        for (int y = 1; y < LPH; y <<= 1) ss += __shfl_xor_sync(who, ss, y);
        const float r = rsqrtf(ss / D + A.eps);
        float wa[8], wb[8];
        unpack8(*reinterpret_cast<const uint4*>(w + 8 * c0), wa);
        unpack8(*reinterpret_cast<const uint4*>(w + 8 * c1), wb);
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          a[y] *= r * wa[y];
          b[y] *= r * wb[y];
        }
      }
      if (turns) {
        const float2* at = cs + t * half;
        if (A.interleaved) {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float2 p = at[4 * c0 + y], q = at[4 * c1 + y];
            const float a0 = a[2 * y], a1 = a[2 * y + 1], b0 = b[2 * y], b1 = b[2 * y + 1];
            a[2 * y] = a0 * p.x - a1 * p.y;
            a[2 * y + 1] = a1 * p.x + a0 * p.y;
            b[2 * y] = b0 * q.x - b1 * q.y;
            b[2 * y + 1] = b1 * q.x + b0 * q.y;
          }
        } else {
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const float2 p = at[8 * lane + y];
            const float a0 = a[y], b0 = b[y];
            a[y] = a0 * p.x - b0 * p.y;
            b[y] = b0 * p.x + a0 * p.y;
          }
        }
      }
      u0 = pack8(a);
      u1 = pack8(b);
    }
    const int2 row = rows[t];
    uint16_t* dst = nullptr;
    if (is_q) dst = A.q_out + int64_t(i0 + t) * A.ost + h * D;
    else if (row.x >= 0)
      dst = is_v ? A.vc + row.x * A.vsp + (h - A.hq - A.hkv) * A.vsh + row.y * A.vsl
                 : A.kc + row.x * A.ksp + (h - A.hq) * A.ksh + row.y * A.ksl;
    if (dst) {
      *reinterpret_cast<uint4*>(dst + 8 * c0) = u0;
      *reinterpret_cast<uint4*>(dst + 8 * c1) = u1;
    }
    t = tn;
    h = hn;
    u0 = n0;
    u1 = n1;
  }
}

template <int D>
cudaError_t launch_d(const RopeArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int GROUPS = NTH * 16 / D;
  const int heads = a.hq + 2 * a.hkv;
  // Tokens and splits of the heads: as many CTAs as fill the SMs where the batch is
  // short, ten runs of heads for each where it is long.  us by tokens of a CTA,
  // 64/8/128, 16384 tokens (5 runs of heads a token): 1 116, 2 112, 4 114, 6 116 (256
  // threads: 135, 120, 116, 117); 14/2/64, 5003 tokens (1 run): 2 8.0, 4 7.7, 6 9.9.
  const long long runs = ((long long)a.N * heads + GROUPS - 1) / GROUPS, ctas = (long long)kPerSm * num_sms;
  const int tb = int(std::min<long long>({kTokensMax, std::max(1LL, (long long)a.N / ctas),
                                          std::max(1, 10 * GROUPS / heads)}));
  const int splits = runs < ctas ? (heads + GROUPS - 1) / GROUPS : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.N + tb - 1) / tb, splits);
  cfg.blockDim = dim3(NTH);
  cfg.dynamicSmemBytes = size_t(tb) * (a.rot / 2) * sizeof(float2);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_kernel<D>, a, tb);
}

}  // namespace

cudaError_t rope_launch(const RopeArgs& a, int D, int num_sms, cudaStream_t stream) {
  return D == 128 ? launch_d<128>(a, num_sms, stream) : launch_d<64>(a, num_sms, stream);
}

}  // namespace dustin
