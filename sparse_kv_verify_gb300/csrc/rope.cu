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
// Angles: inv_freq / 2 pi as a fraction of 2^64 (whole numbers, turns.h) times the
// position, modulo 2^64, is the fraction of a turn, within 2^-33 at any position;
// its upper 32 bits are the half-turns in [-1, 1) that sincospif takes, in fp32's
// 24 bits.
//
// Bound by the bytes: each row is read and written once.  16384 tokens, 64/8/128:
// 104 us for 671 MB, 6.4 TB/s (a plain copy of as many bytes takes 101).  Two elements
// an instruction (f32x2) where the layout allows it: one at a time the issue of
// instructions cost 8 us more.  One token: 2.4 us, the latency of one launch.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "turns.h"

namespace dustin {

namespace {

constexpr int NTH = 128, kPerSm = 8;   // threads of a CTA, CTAs per SM
constexpr int kTokensMax = 32;   // tokens of a CTA at most

// A head whose mean of squares (with eps) is below kTiny, where squares may be
// denormal or 0, is multiplied by kUp first and eps by its square: bf16's smallest
// element, 2^-133, then has a square of 2^-114, and a head's largest one is below
// 2^60.  Only where eps allows such a mean: with the branch, taken or not, 16384 tokens
// of 64/8/128 take 107.8 instead of 104.7 us, 5003 of 14/2/64 9.7 instead of 7.3 (64
// registers instead of 56, and the loads behind it are kept back).
constexpr float kTiny = 0x1p-100f, kUp = 0x1p76f;

// Two floats for the packed instructions.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void halves(f32x2 x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ void unpack8(const uint4& u, f32x2* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack8(const f32x2* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    halves(x[i], a, b);
    w[i] = pack_bf16(a, b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// CTA (x, y): tokens [x tb, (x + 1) tb), every gridDim.y-th run of heads.
template <int D, bool TINY>
__global__ void __launch_bounds__(NTH, kPerSm) rope_kernel(const __grid_constant__ RopeArgs A, int tb) {
  constexpr int LPH = D / 16, GROUPS = NTH / LPH;   // lanes per head, heads at a time
  extern __shared__ __align__(16) float cs[];       // [tb]: cosines [rot / 2], sines [rot / 2], in an order of `place`
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
  // where a pair's angle is: a lane's eight as two runs of four, so that the lanes'
  // 16-byte loads are next to one another
  auto place = [&](int j) { return A.interleaved ? j : ((j >> 2) & 1) * (half / 2) + (j >> 3) * 4 + (j & 3); };
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
    const long long turn = (long long)(turn_of(__float_as_uint(A.inv_freq[j])) * (unsigned long long)(long long)A.pos[i0 + tx]);
    float s, c;
    sincospif(float(int(turn >> 32)) * 0x1p-31f, &s, &c);
    float* at = cs + tx * A.rot + place(j);
    at[0] = c;
    at[half] = s;
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
      f32x2 a[4], b[4];
      unpack8(u0, a);
      unpack8(u1, b);
      const uint16_t* w = is_q ? A.q_w : A.k_w;
      if (w) {
        auto squares = [&] {   // of the head, their sum
          f32x2 sa = mul2(a[0], a[0]), sb = mul2(b[0], b[0]);
#pragma unroll
          for (int y = 1; y < 4; ++y) {
            sa = fma2(a[y], a[y], sa);
            sb = fma2(b[y], b[y], sb);
          }
          float s0, s1, s2, s3;
          halves(sa, s0, s1);
          halves(sb, s2, s3);
          float ss = (s0 + s1) + (s2 + s3);
#pragma unroll
          for (int y = 1; y < LPH; y <<= 1) ss += __shfl_xor_sync(who, ss, y);
          return ss;
        };
        float mean = squares() / D + A.eps;
        if constexpr (TINY) {
          if (mean < kTiny) {   // (the same for all lanes of the head)
            const f32x2 up = pair(kUp, kUp);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              a[y] = mul2(a[y], up);
              b[y] = mul2(b[y], up);
            }
            mean = squares() / D + A.eps * kUp * kUp;
          }
        }
        const float r = rsqrtf(mean);
        const f32x2 r2 = pair(r, r);
        f32x2 wa[4], wb[4];
        unpack8(*reinterpret_cast<const uint4*>(w + 8 * c0), wa);
        unpack8(*reinterpret_cast<const uint4*>(w + 8 * c1), wb);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          a[y] = mul2(a[y], mul2(r2, wa[y]));
          b[y] = mul2(b[y], mul2(r2, wb[y]));
        }
      }
      if (turns) {
        const float* at = cs + t * A.rot;
        if (A.interleaved) {
          auto turn = [&](f32x2& x, int j) {
            const float c = at[j], s = at[half + j];
            float x0, x1;
            halves(x, x0, x1);
            x = pair(x0 * c - x1 * s, x1 * c + x0 * s);
          };
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            turn(a[y], 4 * c0 + y);
            turn(b[y], 4 * c1 + y);
          }
        } else {
          const f32x2 minus = pair(-1.f, -1.f);
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(at + z * (half / 2) + 4 * lane);
            const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(at + half + z * (half / 2) + 4 * lane);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const f32x2 a0 = a[2 * z + y], b0 = b[2 * z + y], cy = y ? c.y : c.x, sy = y ? s.y : s.x;
              a[2 * z + y] = fma2(mul2(b0, minus), sy, mul2(a0, cy));
              b[2 * z + y] = fma2(a0, sy, mul2(b0, cy));
            }
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

template <int D, bool TINY>
cudaError_t launch_d(const RopeArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int GROUPS = NTH * 16 / D;
  const int heads = a.hq + 2 * a.hkv;
  // Tokens and splits of the heads: as many CTAs as fill the SMs where the batch is
  // short, ten runs of heads for each where it is long.  us by tokens of a CTA,
  // 64/8/128, 16384 tokens (5 runs of heads a token): 1 107.6, 2 104.8, 4 106.2;
  // 14/2/64, 5003 tokens (1 run): 2 8.4, 4 7.7, 6 9.1.
  const long long runs = ((long long)a.N * heads + GROUPS - 1) / GROUPS, ctas = (long long)kPerSm * num_sms;
  const int tb = int(std::min<long long>({kTokensMax, std::max(1LL, (long long)a.N / ctas),
                                          std::max(1, 10 * GROUPS / heads)}));
  const int splits = runs < ctas ? (heads + GROUPS - 1) / GROUPS : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.N + tb - 1) / tb, splits);
  cfg.blockDim = dim3(NTH);
  cfg.dynamicSmemBytes = size_t(tb) * a.rot * sizeof(float);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_kernel<D, TINY>, a, tb);
}

}  // namespace

cudaError_t rope_launch(const RopeArgs& a, int D, int num_sms, cudaStream_t stream) {
  const bool normed = a.q_w || a.k_w;
  if (normed && a.eps < kTiny) return D == 128 ? launch_d<128, true>(a, num_sms, stream) : launch_d<64, true>(a, num_sms, stream);
  return D == 128 ? launch_d<128, false>(a, num_sms, stream) : launch_d<64, false>(a, num_sms, stream);
}

}  // namespace dustin
