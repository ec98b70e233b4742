// Accumulated attention weights of a cache's rows.
//
// The last n = n_new[b] of the L = seq_len[b] cache rows are the accepted rows
// of the last draft block and the first n of its T query rows are theirs: query
// t sits at row L - n + t.  For every row j,
//   weight[j] += sum over t < n with j <= L - n + t and over the G query heads
//                of the KV head, of exp(q.k_j / sqrt(d) - lse[t]),
// where the new rows start from 0 and get pos[j] = n_seen[b] - (L - j).
//
// K is read once and bounds the kernel (2 d bytes a row against 8 of weight).
// Tiles of 128 cache rows are the M side of the product, the n * G query rows
// the N side: S^T has a cache row per tensor-memory lane and a query row per
// column, so that a row's weight is a sum over one thread's own registers --
// no exchange, no atomics, one owner per weight.  Rows of a tile at or beyond L
// fill lanes that are never stored.
//
// The batch's tiles are shared evenly among two CTAs per SM.  Roles: warps 0-3
// sum (thread = cache row), warp 4 issues the TMA loads of K tiles into a ring
// and of each unit's query rows, warp 5 issues the MMAs into one of two S
// buffers.
//
// B = 16, L = 24 K .. 32 K, T = 6, 64/8/128: 141 us for 970 MB, 6.9 TB/s, which is
// the rate of a plain copy; one token over 4097 rows 5.3 us, latency of one launch.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "share.cuh"
#include "tc.cuh"

namespace dustin {

namespace {

constexpr int TK = kAccumulateTile;   // cache rows per tile
constexpr int NTH = 192;
constexpr int kLoadWarp = 4, kMmaWarp = 5;
constexpr int kCols = 256;            // tensor memory: two S buffers of 128 columns
constexpr uint32_t kSmemMax = 113 * 1024;   // two CTAs per SM

struct Lay {
  uint32_t q_panel, ring_off, stage, bar_off, lse_off, misc_off, total;
  int nst;
};
// the query rows [D / 64 panels][rows rounded to 32][128 B], K stages, barriers
__host__ __device__ inline Lay make_lay(int D, int NQ) {
  Lay L;
  const uint32_t rows = uint32_t(NQ + 31) & ~31u;
  L.q_panel = rows * 128;
  L.ring_off = uint32_t(D / 64) * L.q_panel;   // panels are whole 4 KB
  L.stage = uint32_t(D / 64) * TK * 128;
  L.nst = int((kSmemMax - 4096 - L.ring_off) / L.stage);
  if (L.nst > 6) L.nst = 6;
  L.bar_off = L.ring_off + uint32_t(L.nst) * L.stage;
  L.lse_off = L.bar_off + 24 * 8;
  L.misc_off = L.lse_off + 4 * 128 * 4;
  L.total = L.misc_off + 48 + 1024;
  return L;
}

// rows, accepted rows and tiles of a sequence's units (0 tiles: nothing to add,
// or inconsistent lengths)
struct Seq {
  int L, n, seen, tiles;
};
__device__ __forceinline__ Seq seq_of(const AccumulateArgs& A, int b) {
  Seq s{A.seq_len[b], A.n_new[b], A.n_seen[b], 0};
  if (accumulate_ok(A, s.L, s.n, s.seen) && s.n > 0) s.tiles = (s.L + TK - 1) / TK;
  return s;
}

// This CTA's runs: tiles [ta, ta + n) of unit (b, g).
struct Walk {
  long long left;
  int b, g, ta, n;
  Seq s;
};
__device__ __forceinline__ void walk_init(Walk& w, const AccumulateArgs& A, const Share& sh) {
  w.left = sh.count;
  w.b = sh.b;
  if (w.left > 0) {
    w.s = seq_of(A, w.b);
    w.g = int(sh.offset / w.s.tiles);
    w.ta = int(sh.offset - (long long)w.g * w.s.tiles);
    w.n = int(w.left < w.s.tiles - w.ta ? w.left : w.s.tiles - w.ta);
  }
}
__device__ __forceinline__ void walk_next(Walk& w, const AccumulateArgs& A) {
  w.left -= w.n;
  if (w.left <= 0) return;
  if (++w.g == A.hkv) {
    w.g = 0;
    do w.s = seq_of(A, ++w.b);
    while (w.s.tiles == 0 && w.b + 1 < A.B);
  }
  w.ta = 0;
  w.n = int(w.left < w.s.tiles ? w.left : w.s.tiles);
}

template <int D>
__global__ void __launch_bounds__(NTH, 2) accumulate_kernel(const __grid_constant__ AccumulateArgs A) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int NQ = A.T * A.G;
  const Lay Ly = make_lay(D, NQ);
  const int NST = Ly.nst;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Ly.bar_off);   // [8]
  uint64_t* empty = full + 8;                                        // [8]
  uint64_t* q_full = empty + 8;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;    // [2]
  uint64_t* s_empty = s_full + 2;    // [2]
  uint64_t* mma_done = s_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Ly.misc_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Ly.misc_off + 8);
  Share* share = reinterpret_cast<Share*>(smem + Ly.misc_off + 16);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&s_empty[x], 128);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "n"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_launch_dependents();
  pdl_wait();
  if (warp == kLoadWarp) {
    const Share sh = share_of(A.B, [&](int b) { return seq_of(A, b).tiles * A.hkv; });
    if (lane == 0) *share = sh;
    if (blockIdx.x == 0)
      for (int b = lane; b < A.B; b += 32)
        if (!accumulate_ok(A, A.seq_len[b], A.n_new[b], A.n_seen[b])) flag_error(A.err, DUSTIN_DEV_APPEND);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk w;
  walk_init(w, A, *share);

  if (warp == kLoadWarp) {
    if (lane == 0) {
      // ============================================================== loads
      const uint64_t pol = policy_evict_first();
      int gi = 0, units = 0;
      bool live = true;
      for (; w.left > 0 && live; walk_next(w, A), ++units) {
        if (units > 0 && !mbar_wait(q_empty, uint32_t(units - 1) & 1u, A.err, abort_flag)) break;
        mbar_arrive_expect_tx(q_full, uint32_t(NQ) * D * 2);
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          tma_load_3d(sbase + uint32_t(h) * Ly.q_panel, &A.qmap, h * 64, w.g * A.G, w.b * A.T, q_full);
        for (int i = 0; i < w.n; ++i, ++gi) {
          const int st = gi % NST;
          if (gi >= NST && !mbar_wait(&empty[st], uint32_t(gi / NST - 1) & 1u, A.err, abort_flag)) {
            live = false;
            break;
          }
          mbar_arrive_expect_tx(&full[st], Ly.stage);
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            const uint32_t dst = sbase + Ly.ring_off + uint32_t(st) * Ly.stage + uint32_t(h) * (TK * 128);
            const int row = (w.ta + i) * TK;
            if (A.krank == 2) tma_load_2d_u32(dst, &A.kmap, h * 64, (w.b * A.hkv + w.g) * A.Lcap + row, &full[st], pol);
            else tma_load_4d_u32(dst, &A.kmap, h * 64, row, w.g, w.b, &full[st], pol);
          }
        }
      }
      // every load has landed before the CTA may exit
      if (units > 0) mbar_drain(q_full, uint32_t(units - 1) & 1u, A.err);
      for (int j = gi > NST ? gi - NST : 0; j < gi; ++j) mbar_drain(&full[j % NST], uint32_t(j / NST) & 1u, A.err);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      // =============================================================== MMAs
      int gi = 0, units = 0;
      bool issued = false, live = true;
      for (; w.left > 0 && live; walk_next(w, A), ++units) {
        if (!mbar_wait(q_full, uint32_t(units) & 1u, A.err, abort_flag)) break;
        const uint32_t idesc = tc_idesc(TK, 32, 0) + (uint32_t((w.s.n * A.G + 31) / 32 - 1) << 19);   // N = 32 .. 128
        for (int i = 0; i < w.n; ++i, ++gi) {
          const int st = gi % NST;
          if ((gi >= 2 && !mbar_wait(&s_empty[gi & 1], uint32_t((gi >> 1) - 1) & 1u, A.err, abort_flag)) ||
              !mbar_wait(&full[st], uint32_t(gi / NST) & 1u, A.err, abort_flag)) {
            live = false;
            break;
          }
          issued = true;
          tc_fence_after();
          const uint32_t k = sbase + Ly.ring_off + uint32_t(st) * Ly.stage;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = uint32_t((kk & 3) * 32);
            tc_mma_ss(tmem + uint32_t((gi & 1) * 128), tc_desc(k + uint32_t(kk >> 2) * (TK * 128) + off, 16, 1024),
                      tc_desc(sbase + uint32_t(kk >> 2) * Ly.q_panel + off, 16, 1024), idesc, kk > 0);
          }
          tc_commit(&empty[st]);
          tc_commit(&s_full[gi & 1]);
        }
        if (live) tc_commit(q_empty);
      }
      if (issued) {   // every MMA has completed before tensor memory is freed
        tc_commit(mma_done);
        mbar_drain(mma_done, 0, A.err);
      }
    }
    __syncwarp();
  } else {
    // ================================================================ sums
    // this warp's copy of the unit's lse in the log2 domain (+inf adds nothing)
    float* lse2 = reinterpret_cast<float*>(smem + Ly.lse_off) + 128 * warp;
    const float scale = A.scale_log2;
    int gi = 0;
    bool live = true;
    for (; w.left > 0 && live; walk_next(w, A)) {
      const int nr = w.s.n * A.G;   // query rows that count
      __syncwarp();
      for (int r = lane; r < nr; r += 32) {
        const float x = A.lse[(size_t(w.b) * A.T + r / A.G) * (A.hkv * A.G) + size_t(w.g) * A.G + r % A.G];
        lse2[r] = x == -INFINITY ? INFINITY : x * kLog2e;
      }
      __syncwarp();
      for (int i = 0; i < w.n; ++i, ++gi) {
        const int j = (w.ta + i) * TK + tid;
        const int u = j - (w.s.L - w.s.n);            // >= 0: the u-th new row
        const size_t at = (size_t(w.b) * A.hkv + w.g) * A.Lcap + j;
        float sum = 0.f;
        if (u < 0) sum = A.weight[at];                // in flight while S is computed
        const int r0 = u > 0 ? u * A.G : 0;           // earlier queries do not see it
        if (!__all_sync(0xffffffffu, mbar_wait(&s_full[gi & 1], uint32_t(gi >> 1) & 1u, A.err, abort_flag))) {
          live = false;
          break;
        }
        tc_fence_after();
        float add[4] = {0.f, 0.f, 0.f, 0.f};
        const uint32_t s_tmem = tmem + (uint32_t(warp * 32) << 16) + uint32_t((gi & 1) * 128);
        for (int c = 0; c < nr; c += 32) {
          uint32_t s[32];
          tc_ld32(s_tmem + uint32_t(c), s);
          if (__all_sync(0xffffffffu, r0 <= c) && c + 32 <= nr) {
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
              const float4 l = *reinterpret_cast<const float4*>(lse2 + c + x);
              add[0] += fast_exp2(fmaf(__uint_as_float(s[x]), scale, -l.x));
              add[1] += fast_exp2(fmaf(__uint_as_float(s[x + 1]), scale, -l.y));
              add[2] += fast_exp2(fmaf(__uint_as_float(s[x + 2]), scale, -l.z));
              add[3] += fast_exp2(fmaf(__uint_as_float(s[x + 3]), scale, -l.w));
            }
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const bool in = c + x < nr && c + x >= r0;
              const float l = lse2[c + x < nr ? c + x : 0];
              add[x & 3] += in ? fast_exp2(fmaf(__uint_as_float(s[x]), scale, -l)) : 0.f;
            }
          }
        }
        tc_fence_before();
        mbar_arrive(&s_empty[gi & 1]);
        if (j < w.s.L) {
          A.weight[at] = sum + ((add[0] + add[1]) + (add[2] + add[3]));
          if (u >= 0) A.pos[at] = w.s.seen - (w.s.L - j);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kCols) : "memory");
}

template <int D>
cudaError_t launch_d(const AccumulateArgs& a, int num_sms, cudaStream_t stream) {
  auto kern = accumulate_kernel<D>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t attr = once_per_device(done, [&] {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmemMax));
    if (e == cudaSuccess)   // room for two CTAs' shared memory
      e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                               int(cudaSharedmemCarveoutMaxShared));
    return e;
  });
  if (attr != cudaSuccess) return attr;
  const long long most = (long long)a.B * a.hkv * ((a.Lcap + TK - 1) / TK);
  const int grid = int(std::min<long long>(2LL * num_sms, most));
  return launch_pdl(kern, dim3(grid), dim3(NTH), make_lay(D, a.T * a.G).total, stream, a);
}

}  // namespace

cudaError_t accumulate_launch(const AccumulateArgs& a, int D, int num_sms, cudaStream_t stream) {
  return D == 128 ? launch_d<128>(a, num_sms, stream) : launch_d<64>(a, num_sms, stream);
}

}  // namespace dustin
