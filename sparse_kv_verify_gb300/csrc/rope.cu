// Norm of each head, position rotation and cache write of new tokens
// (dustin_norm_rope): y = x rsqrt(mean x^2 + eps) w, then pairs (a, b) turned by
// t = pos * inv_freq[j]: (a cos t - b sin t, b cos t + a sin t).
//
// A head is 16 elements in each of D / 16 lanes, as the two 16-byte chunks that
// hold the pairs' two halves, so that a rotation needs no exchange between lanes
// (interleaved pairs lie inside a chunk).  The angles of a token serve all its
// heads: a CTA computes them for its tokens once, into shared memory.
//
// Angles: inv_freq / 2 pi as a fraction of 2^64 times the position, modulo 2^64,
// is the fraction of a turn without any rounding that grows with the position;
// its upper 32 bits are the half-turns in [-1, 1) that sincospif takes.
//
// Bound by the bytes: each row is read and written once.
#include "common.cuh"
#include "kernels.h"

namespace dustin {

namespace {

constexpr int NTH = 256;

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

// TB: tokens of a CTA.
template <int D, int TB>
__global__ void __launch_bounds__(NTH) rope_kernel(const __grid_constant__ RopeArgs A) {
  constexpr int LPH = D / 16, GROUPS = NTH / LPH;   // lanes per head, heads at a time
  __shared__ float2 cs[TB][D / 2];
  __shared__ long long rows[TB];                    // slot, or -1
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, i0 = blockIdx.x * TB, nt = min(TB, A.N - i0);
  const int half = A.rot / 2;
  for (int x = tid; x < nt * half; x += NTH) {
    const int t = x / half, j = x - t * half;
    const double turns = double(A.inv_freq[j]) * 0.15915494309189533577;   // 1 / (2 pi)
    const unsigned long long step = __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
    const long long turn = (long long)(step * (unsigned long long)(long long)A.pos[i0 + t]);
    float s, c;
    sincospif(float(int(turn >> 32)) * 0x1p-31f, &s, &c);
    cs[t][j] = make_float2(c, s);
  }
  if (tid < nt) {
    const int s = A.slot[i0 + tid];
    const bool ok = s >= 0 && (long long)s < (long long)A.n_pages * A.page;
    if (!ok && s != -1) flag_error(A.err, DUSTIN_DEV_INDEX);
    rows[tid] = ok ? s : -1;
  }
  __syncthreads();

  const int lane = tid % LPH, turned = A.rot / 16;
  const bool turns = lane < turned;
  // chunks of 8 elements of this lane, and the angles of their pairs
  int c0 = 2 * lane, c1 = 2 * lane + 1;
  if (turns && !A.interleaved) {
    c0 = lane;
    c1 = turned + lane;
  }
  const int heads = A.hq + 2 * A.hkv;
  for (int x = tid / LPH; x < nt * heads; x += GROUPS) {
    const int t = x / heads, h = x - t * heads, i = i0 + t;
    const bool is_q = h < A.hq, is_v = h >= A.hq + A.hkv;
    const int g = is_q ? h : is_v ? h - A.hq - A.hkv : h - A.hq;
    const long long row = rows[t];
    const uint16_t* src = (is_q ? A.q + i * A.qst : is_v ? A.v + i * A.vst : A.k + i * A.kst) + g * D;
    uint4 u0 = *reinterpret_cast<const uint4*>(src + 8 * c0), u1 = *reinterpret_cast<const uint4*>(src + 8 * c1);
    if (!is_v) {
      float a[8], b[8];
      unpack8(u0, a);
      unpack8(u1, b);
      const uint16_t* w = is_q ? A.q_w : A.k_w;
      if (w) {
        float ss = 0.f;
#pragma unroll
        for (int y = 0; y < 8; ++y) ss = fmaf(a[y], a[y], fmaf(b[y], b[y], ss));
        const uint32_t who = ((1u << LPH) - 1u) << (tid & 31 & ~(LPH - 1));   // the lanes of this head
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
        if (A.interleaved) {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float2 p = cs[t][4 * c0 + y], q = cs[t][4 * c1 + y];
            const float a0 = a[2 * y], a1 = a[2 * y + 1], b0 = b[2 * y], b1 = b[2 * y + 1];
            a[2 * y] = a0 * p.x - a1 * p.y;
            a[2 * y + 1] = a1 * p.x + a0 * p.y;
            b[2 * y] = b0 * q.x - b1 * q.y;
            b[2 * y + 1] = b1 * q.x + b0 * q.y;
          }
        } else {
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const float2 p = cs[t][8 * lane + y];
            const float a0 = a[y], b0 = b[y];
            a[y] = a0 * p.x - b0 * p.y;
            b[y] = b0 * p.x + a0 * p.y;
          }
        }
      }
      u0 = pack8(a);
      u1 = pack8(b);
    }
    uint16_t* dst;
    if (is_q) {
      dst = A.q_out + i * A.ost + g * D;
    } else {
      if (row < 0) continue;
      const int id = int(row / A.page), r = int(row - (long long)id * A.page);
      dst = is_v ? A.vc + id * A.vsp + g * A.vsh + r * A.vsl : A.kc + id * A.ksp + g * A.ksh + r * A.ksl;
    }
    *reinterpret_cast<uint4*>(dst + 8 * c0) = u0;
    *reinterpret_cast<uint4*>(dst + 8 * c1) = u1;
  }
}

template <int D>
cudaError_t launch_d(const RopeArgs& a, cudaStream_t stream) {
  constexpr int TB = 4;
  return launch_pdl(rope_kernel<D, TB>, dim3((a.N + TB - 1) / TB), dim3(NTH), 0, stream, a);
}

}  // namespace

cudaError_t rope_launch(const RopeArgs& a, int D, int, cudaStream_t stream) {
  return D == 128 ? launch_d<128>(a, stream) : launch_d<64>(a, stream);
}

}  // namespace dustin
