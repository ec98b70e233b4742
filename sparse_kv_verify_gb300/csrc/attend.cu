// Windowed attention with sinks for a draft block, and the sequences' own part
// of shared-prefix attention.
//
// For query t of sequence b (position i = L + t, L = seq_len[b]) the visible
// keys are the cache rows j < L and the block rows u (position L + u) with
// j <= i and (i - j < window or j < sinks); o = softmax(q.k / sqrt(d)) v and
// lse = ln sum exp(q.k / sqrt(d)) over them, o = 0 and lse = -inf where nothing
// is visible.
//
// Tiles: a unit (sequence b, KV head g) reads the 64-row tiles of the ranges
// [0, min(sinks, L)) and [max(L - window + 1, sinks), L) -- one range [0, L)
// where they meet -- and one tile of block rows.  Only a range's last tile and
// the block tile are partial; a row's own window start and the causal rule are
// masks inside a tile.  How many tiles a unit has depends on its sequence's
// length, which only the device knows: every CTA sums the tile counts of the
// batch (one warp) and takes its equal share of the flattened tiles (stream-K),
// so that ragged lengths and any B and hkv load the SMs alike.  Where units are
// short, CTAs take whole units instead and nothing needs merging (whole_units
// below).
//
// Roles inside a CTA (warp specialised, handing over through mbarriers):
//   warps 4-7    loaders: a whole tile comes as tiled TMA loads (a K and a V
//                box of 64 rows per 64 columns) issued by one thread, a partial
//                one as 16-byte cp.async of its rows with the others
//                zero-filled (rows past a range may hold anything), both into
//                the 128-byte-swizzled layout that the MMAs read;
//   warp 8       one thread issues S = Q K^T into one of two buffers in tensor
//                memory as soon as a tile's rows have landed;
//   warp 9       one thread issues O += P V with P read from tensor memory;
//   warps 0-3    softmax in the log2 domain, the reference maximum moved only
//                when a tile passes it by more than 2^8 (O is rarely rescaled).
//                P is rounded to bf16 for the second MMA; the row sum adds the
//                unrounded fp32 values, so lse keeps fp32 accuracy.
//
// A segment that covers a whole unit writes o and lse; otherwise its row
// maxima, sums and unnormalised O go to slot unit + cta of the workspace (both
// indices only grow along the flattened tiles, so no two segments share one),
// and a second kernel merges them.
//
// Bound by the K and V rows (4 d bytes a row against 4 d T G operations).  B = 16,
// T = 6, 64/8/128, window 4096 over up to 32 K rows: 53 us for 273 MB (5.1 TB/s;
// with cold caches the kernel 47 to 52 and the merge 8).  One token through a
// window of 128: 8.0 us, latency of one launch (the call's host part is 4.3).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "share.cuh"
#include "tc.cuh"

namespace dustin {

namespace {

constexpr int TK = kAttendTile;     // keys per tile (and the largest draft block)
constexpr int kSoftmaxWarps = 4;    // one thread per tensor-memory lane
constexpr int kLoaders = 4;         // loader warps, kKpw keys of a partial tile each
constexpr int kKpw = TK / kLoaders;
constexpr int kLoaderWarp0 = kSoftmaxWarps, kMmaWarp = kSoftmaxWarps + kLoaders;
constexpr int kPvWarp = kMmaWarp + 1;
constexpr int NTH = 32 * (kPvWarp + 1);
constexpr int kSCol = 0;            // S buffers: columns [0, 64) and [64, 128)
constexpr int kPCol = 128;          // P buffers (bf16 pairs) with one CTA per SM
constexpr uint32_t kSmemPerSm = 228 * 1024;
constexpr float kNaN = __builtin_nanf("");
static_assert(TK == DUSTIN_MAX_BLOCK, "the draft block must fit one tile");

// Tensor memory, query buffers and K/V stages per head dimension and CTAs per
// SM: with two CTAs per SM (256 columns each) P is stored over the S buffer it
// came from, and the next segment's query rows wait for this one's MMAs.
template <int D, int CPS>
struct Cfg {
  static constexpr int cols = CPS == 2 ? 256 : (D == 128 ? 512 : 256);
  static constexpr int o_col = CPS == 2 ? 128 : (D == 128 ? 256 : 192);
  static constexpr int p_col = CPS == 2 ? kSCol : kPCol;
  static constexpr int p_stride = CPS == 2 ? TK : TK / 2;
  static constexpr int nqb = CPS == 2 ? 1 : 2;
  static constexpr int nst = CPS == 2 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 8);
  static constexpr uint32_t kv_panel = TK * 128;
  static constexpr uint32_t half = (D / 64) * kv_panel;
  static constexpr uint32_t stage = 2 * half;
};

struct Lay {
  uint32_t q_panel, q_buf, ring_off, bar_off, misc_off, total;
};

template <int D, int CPS>
__host__ __device__ constexpr Lay make_lay(int NQ) {
  using C = Cfg<D, CPS>;
  Lay L{};
  const int q_rows = NQ < 8 ? 8 : (NQ + 7) & ~7;
  L.q_panel = uint32_t(q_rows) * 128;
  L.q_buf = (D / 64) * L.q_panel;
  L.ring_off = (C::nqb * L.q_buf + 1023u) & ~1023u;
  L.bar_off = L.ring_off + C::nst * C::stage;
  L.misc_off = L.bar_off + uint32_t(2 * C::nst + 4 + 2 * C::nqb + 2) * 8;
  L.total = L.misc_off + 48 + 1024;
  return L;
}

// Where a row's sum of weights is 0 either it sees no key, or every score that it
// sees is -inf (a query with an infinite element), which is NaN like the 0 / 0 it
// stands for.  A query sees position 0 as a sink and itself in its window, so the
// call's parameters tell the two apart.
__device__ __forceinline__ bool sees_a_key(const AttendArgs& A) { return A.window > 0 || A.sinks > 0; }
__device__ __forceinline__ float row_scale(const AttendArgs& A, float sum) {
  return sum != 0.f ? 1.f / sum : sees_a_key(A) ? kNaN : 0.f;   // (a NaN stays one)
}
__device__ __forceinline__ float row_lse(const AttendArgs& A, float top, float sum) {
  return sum != 0.f ? (top + log2f(sum)) * kLn2 : sees_a_key(A) ? kNaN : -INFINITY;
}

// The tiles of one sequence's units.
struct Tiles {
  int L, w0;      // rows; start of the window range
  int nA, nB, n;  // tiles of the first and the window range; all, the block tile included
  int a_end;      // rows of the first range
  int nblk;       // block rows that some query sees: all, or without a window the sinks among them
};
__device__ __forceinline__ Tiles tiles_of(const AttendArgs& A, int b) {
  Tiles s;
  int L = A.seq_len[b];
  if (L < 0 || L > A.Lcap) L = 0;
  s.L = L;
  s.a_end = min(A.sinks, L);
  int w0 = A.window > 0 ? L - A.window + 1 : L;   // the first query's window
  if (A.window > 0 && w0 <= s.a_end) {            // the ranges meet: one range [0, L)
    s.a_end = L;
    w0 = L;
  }
  s.w0 = w0;
  s.nA = (s.a_end + TK - 1) / TK;
  s.nB = (L - w0 + TK - 1) / TK;
  s.n = s.nA + s.nB + 1;
  s.nblk = A.window > 0 ? A.T : min(max(A.sinks - L, 0), A.T);
  return s;
}

// Walks this CTA's segments: tiles [ta, ta + n) of unit (b, g).
struct Walk {
  long long left;     // tiles (A.whole: units) this CTA still has
  int b, g, ta, n;
  Tiles s;
};
__device__ __forceinline__ void walk_init(Walk& w, const AttendArgs& A, const Share& sh) {
  w.left = sh.count;
  w.b = sh.b;
  if (w.left > 0) {
    w.s = tiles_of(A, w.b);
    if (A.whole) {
      w.g = int(sh.offset);
      w.ta = 0;
      w.n = w.s.n;
      return;
    }
    w.g = int(sh.offset / w.s.n);
    w.ta = int(sh.offset - (long long)w.g * w.s.n);
    w.n = int(w.left < w.s.n - w.ta ? w.left : w.s.n - w.ta);
  }
}
__device__ __forceinline__ void walk_next(Walk& w, const AttendArgs& A) {
  w.left -= A.whole ? 1 : w.n;
  if (w.left <= 0) return;
  if (++w.g == A.hkv) {
    w.g = 0;
    ++w.b;
    w.s = tiles_of(A, w.b);
  }
  w.ta = 0;
  w.n = A.whole || w.left > w.s.n ? w.s.n : int(w.left);
}

// First key position and number of rows of tile tt.
__device__ __forceinline__ void tile_rows(const Walk& w, int tt, int& base, int& nv, bool& blk) {
  const Tiles& s = w.s;
  blk = tt == s.n - 1;
  if (blk) {
    base = s.L;
    nv = s.nblk;
  } else if (tt < s.nA) {
    base = tt * TK;
    nv = min(TK, s.a_end - base);
  } else {
    base = s.w0 + (tt - s.nA) * TK;
    nv = min(TK, s.L - base);
  }
}

// M: rows of the MMAs, 64 when the query rows fit (16 rows per lane quarter),
// else 128 (one row per lane).  CPS: CTAs per SM (2 only with M = 64).
template <int D, int M, int CPS>
__global__ void __launch_bounds__(NTH, CPS) attend_kernel(const __grid_constant__ AttendArgs A) {
  static_assert(M == 64 || M == 128, "MMA rows");
  static_assert(CPS == 1 || (CPS == 2 && M == 64), "two CTAs per SM only with 64-row MMAs");
  using C = Cfg<D, CPS>;
  constexpr int NST = C::nst, NQB = C::nqb;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int T = A.T, GQ = A.hq / A.hkv, NQ = T * GQ;
  const Lay Ly = make_lay<D, CPS>(NQ);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Ly.bar_off);
  uint64_t* empty = full + NST;
  uint64_t* s_full = empty + NST;
  uint64_t* p_full = s_full + 2;
  uint64_t* q_full = p_full + 2;
  uint64_t* q_empty = q_full + NQB;
  uint64_t* mma_done = q_empty + NQB;
  uint64_t* pv_done = mma_done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Ly.misc_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Ly.misc_off + 8);
  int* q_hi = reinterpret_cast<int*>(smem + Ly.misc_off + 12);   // query loads issued: [0, q_hi)
  Share* share = reinterpret_cast<Share*>(smem + Ly.misc_off + 16);

  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const int n_act = M == 64 ? (NQ + 15) >> 4 : (NQ + 31) >> 5;   // softmax warps holding query rows
  if (tid == 32) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&full[s], 32 * kLoaders + kLoaders);
      mbar_init(&empty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 32 * n_act);
    }
    for (int x = 0; x < NQB; ++x) {
      mbar_init(&q_full[x], 1);
      mbar_init(&q_empty[x], 1);
    }
    mbar_init(mma_done, 1);
    mbar_init(pv_done, 1);
    *abort_flag = 0;
    *q_hi = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "n"(C::cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  // (only now: the prefix kernel does not wait for this one before it reads its
  // inputs, so what wrote them has to be over when it starts)
  pdl_launch_dependents();
  if (warp == 0) {
    Share sh;
    if (A.whole) {   // units [c U / G, (c + 1) U / G), first one (b, offset)
      const long long units = (long long)A.B * A.hkv, u0 = blockIdx.x * units / gridDim.x;
      sh.count = (blockIdx.x + 1) * units / gridDim.x - u0;
      sh.b = int(u0 / A.hkv);
      sh.offset = u0 - (long long)sh.b * A.hkv;
    } else {
      sh = share_of(A.B, [&](int b) { return tiles_of(A, b).n * A.hkv; });
    }
    if (lane == 0) *share = sh;
    if (blockIdx.x == 0)
      for (int b = lane; b < A.B; b += 32)
        if (A.seq_len[b] < 0 || A.seq_len[b] > A.Lcap) flag_error(A.err, DUSTIN_DEV_SEQLEN);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk w;
  walk_init(w, A, *share);

  if (warp >= kLoaderWarp0 && warp < kLoaderWarp0 + kLoaders) {
    // =============================================================== loaders
    const int lw = warp - kLoaderWarp0;
    constexpr int CH = D / 8;             // 16-byte chunks per row
    constexpr int KPI = 32 / CH;          // rows per warp instruction
    constexpr int NI = kKpw / KPI;        // instructions per tensor
    const int c = lane % CH, ksub = lane / CH;
    int gi = 0, s = 0;
    bool live = true;     // false once a wait gave up
    uint32_t tmask = 0;   // bit j: tile gi - 1 - j came by TMA boxes
    const uint64_t pol = policy_evict_first();
    for (; w.left > 0 && live; walk_next(w, A), ++s) {
      // this segment's query rows -> query buffer s % NQB, once the MMAs of the
      // segment that used it last are done.  One warp does this for every segment:
      // a wait by parity is only right for a thread that has seen the phase before
      // (the last warp, so that the TMA loads of the first one run on).
      const int qb = s % NQB;
      if (lw == kLoaders - 1) {
        bool ok = true;
        if (lane == 0) {
          if (s >= NQB) ok = mbar_wait(&q_empty[qb], uint32_t(s / NQB - 1) & 1u, A.err, abort_flag);
          if (ok) {
            mbar_arrive_expect_tx(&q_full[qb], uint32_t(NQ) * D * 2);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_load_3d(sbase + qb * Ly.q_buf + h * Ly.q_panel, &A.qmap, h * 64, w.g * GQ, w.b * T, &q_full[qb]);
            atomicMax(q_hi, s + 1);
          }
        }
        if (!__shfl_sync(0xffffffffu, int(ok), 0)) break;
      }
      const uint16_t* kbase = A.k + size_t(w.b) * A.ksb + size_t(w.g) * A.ksh;
      const uint16_t* vbase = A.v + size_t(w.b) * A.vsb + size_t(w.g) * A.vsh;
      const size_t blk_off = (size_t(w.b) * A.hkv + w.g) * T * D;
      for (int i = 0; i < w.n; ++i, ++gi) {
        int base, nv;
        bool blk;
        tile_rows(w, w.ta + i, base, nv, blk);
        const int st = gi % NST;
        if (gi >= NST &&
            !__all_sync(0xffffffffu, mbar_wait(&empty[st], uint32_t(gi / NST - 1) & 1u, A.err, abort_flag))) {
          live = false;
          break;
        }
        const uint32_t stage = sbase + Ly.ring_off + uint32_t(st) * C::stage;
        const bool by_tma = A.tma && !blk && nv == TK;
        tmask = (tmask << 1) | uint32_t(by_tma);
        if (by_tma) {
          // boxes issued by one lane, the byte count armed with its arrival
          // (the other threads arrive as for gathered rows, with nothing in flight)
          if (lw == 0 && lane == 0) {
            mbar_arrive_expect_tx(&full[st], C::stage);
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
              const uint32_t dk = stage + h * C::kv_panel, dv = dk + C::half;
              const int row = (w.b * A.hkv + w.g) * A.Lcap + base;
              if (A.krank == 2) tma_load_2d_u32(dk, &A.kmap, h * 64, row, &full[st], pol);
              else tma_load_4d_u32(dk, &A.kmap, h * 64, base, w.g, w.b, &full[st], pol);
              if (A.vrank == 2) tma_load_2d_u32(dv, &A.vmap, h * 64, row, &full[st], pol);
              else tma_load_4d_u32(dv, &A.vmap, h * 64, base, w.g, w.b, &full[st], pol);
            }
          } else if (lane == 0) {
            mbar_arrive(&full[st]);
          }
          cp_async_arrive_noinc(&full[st]);
          continue;
        }
        const uint16_t* ksrc = blk ? A.kb + blk_off : kbase + size_t(base) * A.ksl;
        const uint16_t* vsrc = blk ? A.vb + blk_off : vbase + size_t(base) * A.vsl;
        const int64_t kst = blk ? D : A.ksl, vst = blk ? D : A.vsl;
#pragma unroll
        for (int m = 0; m < 2 * NI; ++m) {
          const int which = m / NI;
          const int key = kKpw * lw + (m % NI) * KPI + ksub;
          const bool ok = key < nv;
          const uint16_t* src = which ? vsrc + size_t(ok ? key : 0) * vst : ksrc + size_t(ok ? key : 0) * kst;
          cp_async16(stage + which * C::half + uint32_t(c >> 3) * C::kv_panel + swz(key, c & 7), src + c * 8,
                     ok ? 16u : 0u);
        }
        cp_async_arrive_noinc(&full[st]);
        if (lane == 0) mbar_arrive(&full[st]);
      }
    }
    cp_async_wait_all();
    // the boxes this lane issued for the last NST tiles have landed (each is
    // the latest phase of its stage) before the CTA may exit
    if (lw == 0 && lane == 0)
      for (int j = 0; j < NST && j < gi; ++j)
        if ((tmask >> j) & 1u) mbar_drain(&full[(gi - 1 - j) % NST], uint32_t((gi - 1 - j) / NST) & 1u, A.err);
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ================================================================ S MMAs
    if (lane == 0) {
      constexpr uint32_t kIdS = tc_idesc(M, TK, 0);
      int gi = 0, s = 0;
      bool issued = false, live = true;
      for (; w.left > 0 && live; walk_next(w, A), ++s) {
        const int qb = s % NQB;
        const uint32_t qbuf = sbase + qb * Ly.q_buf;
        if (!mbar_wait(&q_full[qb], uint32_t(s / NQB) & 1u, A.err, abort_flag)) break;
        for (int i = 0; i < w.n; ++i, ++gi) {
          const int st = gi % NST;
          if ((gi >= 2 && !(CPS == 2 ? mbar_wait(&empty[(gi - 2) % NST], uint32_t((gi - 2) / NST) & 1u, A.err, abort_flag)
                                     : mbar_wait(&p_full[gi & 1], uint32_t((gi >> 1) - 1) & 1u, A.err, abort_flag))) ||
              !mbar_wait(&full[st], uint32_t(gi / NST) & 1u, A.err, abort_flag)) {
            live = false;
            break;
          }
          issued = true;
          fence_proxy_async();   // partial tiles were written by cp.async (generic proxy)
          tc_fence_after();
          const uint32_t kst = sbase + Ly.ring_off + uint32_t(st) * C::stage;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t koff = uint32_t((kk & 3) * 32);
            const uint64_t a = tc_desc(qbuf + (kk >> 2) * Ly.q_panel + koff, 16, 1024);
            const uint64_t bd = tc_desc(kst + (kk >> 2) * C::kv_panel + koff, 16, 1024);
            tc_mma_ss(tmem + uint32_t(kSCol + (gi & 1) * TK), a, bd, kIdS, kk > 0);
          }
          tc_commit(&s_full[gi & 1]);
        }
        if (live) tc_commit(&q_empty[qb]);   // the segment's query rows are no longer read
      }
      if (issued) {   // every MMA this thread issued has completed before tensor memory is freed
        tc_commit(mma_done);
        mbar_drain(mma_done, 0, A.err);
      }
    }
    __syncwarp();
  } else if (warp == kPvWarp) {
    // ============================================================== P V MMAs
    if (lane == 0) {
      constexpr uint32_t kIdPV = tc_idesc(M, D, 1);
      int gi = 0;
      bool issued = false, live = true;
      for (; w.left > 0 && live; walk_next(w, A)) {
        for (int i = 0; i < w.n; ++i, ++gi) {
          if (!mbar_wait(&p_full[gi & 1], uint32_t(gi >> 1) & 1u, A.err, abort_flag)) {
            live = false;
            break;
          }
          issued = true;
          tc_fence_after();
          const int st = gi % NST;
          const uint32_t vst = sbase + Ly.ring_off + uint32_t(st) * C::stage + C::half;
          const uint32_t p_tmem = tmem + uint32_t(C::p_col + (gi & 1) * C::p_stride);
#pragma unroll
          for (int kk = 0; kk < TK / 16; ++kk)
            tc_mma_ts(tmem + C::o_col, p_tmem + uint32_t(kk * 8), tc_desc(vst + uint32_t(kk * 2048), C::kv_panel, 1024),
                      kIdPV, (i > 0 || kk > 0) ? 1 : 0);
          tc_commit(&empty[st]);   // S and P V of tile gi done: its stage is free
        }
      }
      if (issued) {
        tc_commit(pv_done);
        mbar_drain(pv_done, 0, A.err);
      }
    }
    __syncwarp();
  } else if (warp < n_act) {
    // =============================================================== softmax
    // M = 128: thread tid holds row tid.  M = 64: warp x holds rows 16 x ..
    // 16 x + 15; thread y takes rows 16 x + y / 4 and that + 8 and, of each, the
    // keys 8 c + 2 (y % 4) + {0, 1}; the four threads of a quad share maxima by
    // shuffles and add their partial sums up at the end.
    constexpr int R = M == 64 ? 2 : 1;          // rows of this thread
    constexpr int KR = M == 64 ? 16 : 64;       // scores of each row
    const int q4 = lane & 3;
    int row[R], tq[R];
    bool act[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      row[r] = M == 64 ? 16 * warp + (lane >> 2) + 8 * r : tid;
      act[r] = row[r] < NQ;
      tq[r] = act[r] ? row[r] / GQ : 0;
    }
    const float scale = A.scale_log2;
    const uint32_t lane_base = tmem + (uint32_t(warp * 32) << 16);
    const uint32_t o_lane = lane_base + uint32_t(C::o_col);
    int gi = 0;
    bool live = true;   // false once a wait gave up (warp-uniform)
    for (; w.left > 0 && live; walk_next(w, A)) {
      float mref[R], lsum[R];   // reference maxima (log2 domain), this thread's share of the row sums
#pragma unroll
      for (int r = 0; r < R; ++r) {
        mref[r] = -INFINITY;
        lsum[r] = 0.f;
      }
      for (int i = 0; i < w.n; ++i, ++gi) {
        int base, nv;
        bool blk;
        tile_rows(w, w.ta + i, base, nv, blk);
        if (!__all_sync(0xffffffffu, mbar_wait(&s_full[gi & 1], uint32_t(gi >> 1) & 1u, A.err, abort_flag))) {
          live = false;
          break;
        }
        tc_fence_after();
        float x[R][KR];
        if constexpr (M == 64) {
          uint32_t sv[32];
          tc_ld16x256_x8(lane_base + uint32_t(kSCol + (gi & 1) * TK), sv);
#pragma unroll
          for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int r = 0; r < R; ++r) {
              x[r][2 * c] = __uint_as_float(sv[4 * c + 2 * r]);
              x[r][2 * c + 1] = __uint_as_float(sv[4 * c + 2 * r + 1]);
            }
        } else {
          tc_ld32(lane_base + uint32_t(kSCol + (gi & 1) * TK), reinterpret_cast<uint32_t*>(x[0]));
          tc_ld32(lane_base + uint32_t(kSCol + (gi & 1) * TK + 32), reinterpret_cast<uint32_t*>(x[0] + 32));
        }
        // masks: rows past nv, keys outside a row's window (sinks apart), u > t
        const int lo0 = w.s.L - A.window + 1 - base;   // row 0's first key in the window
        const int sk = A.sinks - base;                 // keys before it are sinks
        if (blk || nv < TK || (lo0 + T - 1 > 0 && sk < TK)) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const int lo = lo0 + tq[r], hi = blk ? tq[r] + 1 : nv;
#pragma unroll
            for (int j = 0; j < KR; ++j) {
              const int key = M == 64 ? 8 * (j >> 1) + 2 * q4 + (j & 1) : j;
              x[r][j] = key < hi && (key >= lo || key < sk) ? x[r][j] : -INFINITY;
            }
          }
        }
        float mx[R], alpha[R], nb[R];
        bool moved = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float m4[4] = {x[r][0], x[r][1], x[r][2], x[r][3]};
#pragma unroll
          for (int j = 4; j < KR; ++j) m4[j & 3] = fmaxf(m4[j & 3], x[r][j]);
          mx[r] = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          if constexpr (M == 64) {
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
          }
          // (a row past NQ takes -inf as its max: it never rescales O, and its
          // P and O rows are never read)
          mx[r] = act[r] ? mx[r] * scale : -INFINITY;
          alpha[r] = 1.f;
          if (mx[r] > mref[r] + 8.f) {   // also the first tile with a visible key
            alpha[r] = fast_exp2(mref[r] - mx[r]);
            mref[r] = mx[r];
            lsum[r] *= alpha[r];
            moved = true;
          }
          nb[r] = mref[r] == -INFINITY ? 0.f : -mref[r];
        }
        uint32_t pk[R * KR / 2];   // M = 64: entry 2 c + r is row r's pair of chunk c
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float l2[2] = {0.f, 0.f};
#pragma unroll
          for (int j = 0; j < KR; j += 2) {
            const float p0 = fast_exp2(fmaf(x[r][j], scale, nb[r])), p1 = fast_exp2(fmaf(x[r][j + 1], scale, nb[r]));
            pk[M == 64 ? j + r : j / 2] = pack_bf16(p0, p1);
            l2[0] += p0;
            l2[1] += p1;
          }
          lsum[r] += l2[0] + l2[1];
        }
        // rescale O once P V of the previous tile is in (the first tile of a
        // segment overwrites O); tensor-memory accesses are collective
        if (i > 0 && __any_sync(0xffffffffu, moved)) {
          if (!__all_sync(0xffffffffu, mbar_wait(&empty[(gi - 1) % NST], uint32_t((gi - 1) / NST) & 1u, A.err, abort_flag))) {
            live = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            if constexpr (M == 64) {
              uint32_t o[16];
              tc_ld16x256_x4(o_lane + uint32_t(c), o);
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * alpha[(y >> 1) & 1]);
              tc_st16x256_x4(o_lane + uint32_t(c), o);
            } else {
              uint32_t o[32];
              tc_ld32(o_lane + uint32_t(c), o);
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * alpha[0]);
              tc_st32(o_lane + uint32_t(c), o);
            }
          }
        }
        // P buffer gi % 2 is free once P V of tile gi - 2 has completed (when P
        // is stored over S, S of tile gi was issued only after that)
        if (CPS == 1 && gi >= 2 &&
            !__all_sync(0xffffffffu, mbar_wait(&empty[(gi - 2) % NST], uint32_t((gi - 2) / NST) & 1u, A.err, abort_flag))) {
          live = false;
          break;
        }
        const uint32_t p_tmem = lane_base + uint32_t(C::p_col + (gi & 1) * C::p_stride);
        if constexpr (M == 64) tc_st16x128_x8(p_tmem, pk);
        else tc_st32(p_tmem, pk);
        tc_fence_before();
        mbar_arrive(&p_full[gi & 1]);
      }
      if (!live) break;
      // ----------------------------------------------------------- epilogue
      const bool whole = A.pgrid == 0 && w.n == w.s.n;
      const long long unit = (long long)w.b * A.hkv + w.g;
      if (tid == 0) {
        if (w.ta == 0) A.seg_cta[2 * unit] = int(blockIdx.x);
        if (w.ta + w.n == w.s.n) A.seg_cta[2 * unit + 1] = int(blockIdx.x);
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&empty[(gi - 1) % NST], uint32_t((gi - 1) / NST) & 1u, A.err, abort_flag))) {
        live = false;
        break;
      }
      tc_fence_after();
      float* part = A.partial + (size_t(unit) + blockIdx.x) * A.slot_floats;
      size_t orow[R];
      float osc[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if constexpr (M == 64) {
          lsum[r] += __shfl_xor_sync(0xffffffffu, lsum[r], 1);
          lsum[r] += __shfl_xor_sync(0xffffffffu, lsum[r], 2);
        }
        const int rr = act[r] ? row[r] : 0;
        orow[r] = (size_t(w.b) * T + rr / GQ) * A.hq + size_t(w.g) * GQ + rr % GQ;
        osc[r] = row_scale(A, lsum[r]);
        if (act[r] && (M == 128 || q4 == 0)) {
          if (whole) {
            if (A.lse) A.lse[orow[r]] = row_lse(A, mref[r], lsum[r]);
          } else {
            part[size_t(NQ) * D + row[r]] = mref[r];
            part[size_t(NQ) * D + NQ + row[r]] = lsum[r];
          }
        }
      }
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        if constexpr (M == 64) {
          uint32_t o[16];
          tc_ld16x256_x4(o_lane + uint32_t(c), o);   // collective: every lane loads
#pragma unroll
          for (int cc = 0; cc < 4; ++cc)
#pragma unroll
            for (int r = 0; r < R; ++r) {
              if (!act[r]) continue;
              const int col = c + 8 * cc + 2 * q4;
              const float o0 = __uint_as_float(o[4 * cc + 2 * r]), o1 = __uint_as_float(o[4 * cc + 2 * r + 1]);
              if (whole) *reinterpret_cast<uint32_t*>(A.o + orow[r] * D + col) = pack_bf16(o0 * osc[r], o1 * osc[r]);
              else *reinterpret_cast<float2*>(part + size_t(row[r]) * D + col) = make_float2(o0, o1);
            }
        } else {
          uint32_t o[32];
          tc_ld32(o_lane + uint32_t(c), o);
          if (act[0]) {
#pragma unroll
            for (int y = 0; y < 32; y += 8) {
              float f[8];
#pragma unroll
              for (int z = 0; z < 8; ++z) f[z] = __uint_as_float(o[y + z]);
              if (whole) {
                *reinterpret_cast<uint4*>(A.o + orow[0] * D + c + y) =
                    make_uint4(pack_bf16(f[0] * osc[0], f[1] * osc[0]), pack_bf16(f[2] * osc[0], f[3] * osc[0]),
                               pack_bf16(f[4] * osc[0], f[5] * osc[0]), pack_bf16(f[6] * osc[0], f[7] * osc[0]));
              } else {
                float4* dst = reinterpret_cast<float4*>(part + size_t(row[0]) * D + c + y);
                dst[0] = make_float4(f[0], f[1], f[2], f[3]);
                dst[1] = make_float4(f[4], f[5], f[6], f[7]);
              }
            }
          }
        }
      }
      tc_fence_before();
    }
  }

  // Every query load has been issued: the last NQB of them (each the latest
  // phase of its buffer) have landed before the CTA exits.
  __syncthreads();
  if (warp == kLoaderWarp0 && lane == 0) {
    const int hi = *q_hi;
    for (int x = hi - NQB < 0 ? 0 : hi - NQB; x < hi; ++x) mbar_drain(&q_full[x % NQB], uint32_t(x / NQB) & 1u, A.err);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::cols) : "memory");
}

// Log-sum-exp merge of a unit's segments: one thread per four output columns.
// A segment is (unnormalised O, log2-domain reference maximum m, sum l).
constexpr int kMergeThreads = 128;

template <int D, bool PREFIX>
__global__ void __launch_bounds__(kMergeThreads) attend_merge_kernel(const __grid_constant__ AttendArgs A) {
  pdl_launch_dependents();
  const int unit = blockIdx.y, T = A.T, GQ = A.hq / A.hkv, NQ = T * GQ;
  const int x = blockIdx.x * kMergeThreads + threadIdx.x;
  const int r = x / (D / 4), c4 = x - r * (D / 4);
  const int b = unit / A.hkv, g = unit % A.hkv;
  pdl_wait();   // before any CTA leaves: this kernel completes after the one before it
  // (within the slots whatever they hold: a kernel that gave up may not have set them)
  const int c0 = min(max(__ldcg(A.seg_cta + 2 * unit), 0), kAttendGridMax - 1);
  const int c1 = min(max(__ldcg(A.seg_cta + 2 * unit + 1), c0), kAttendGridMax - 1);
  if (!PREFIX && c0 == c1) return;   // written by its CTA
  if (x >= NQ * (D / 4)) return;
  // this thread's columns, m and l of own segment 0 and of prefix segment 0
  const int own = c1 - c0 + 1;
  const float* po = A.partial + (size_t(unit) + c0) * A.slot_floats;
  const size_t ov = size_t(r) * D + 4 * c4, om = size_t(NQ) * D + r;
  constexpr size_t kLane = size_t(kPrefixTile) * (D + 2);
  const float* pp = nullptr;
  int row = 0, all = own;
  if constexpr (PREFIX) {
    const int P = __ldcg(A.prefix_len);
    if (P > 0 && P <= A.Pcap) {
      const int tok = b * T + r / GQ, tile = tok / A.nt, pu = g * A.pairs + (tile >> 1);
      const int p0 = min(max(__ldcg(A.pseg_cta + 2 * pu), 0), kPrefixGridMax - 1);
      const int p1 = min(max(__ldcg(A.pseg_cta + 2 * pu + 1), p0), kPrefixGridMax - 1);
      row = (tok - tile * A.nt) * GQ + r % GQ;
      pp = A.ppartial + ((size_t(pu) + p0) * 2 + (tile & 1)) * kLane;
      all += p1 - p0 + 1;
    }
  }
  constexpr int kDepth = 8;   // segments whose loads are in flight
  float top = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = 0; c < all; c += kDepth) {
    float m[kDepth], l[kDepth];
    float4 o[kDepth];
#pragma unroll
    for (int y = 0; y < kDepth; ++y) {
      const int z = c + y;
      m[y] = -INFINITY;
      l[y] = 0.f;
      o[y] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (z < all) {
        const bool mine = !PREFIX || z < own;
        const float* s = mine ? po + size_t(z) * A.slot_floats : pp + size_t(z - own) * 2 * kLane;
        const float* ml = s + (mine ? om : size_t(kPrefixTile) * D + row);
        m[y] = __ldcg(ml);
        l[y] = __ldcg(ml + (mine ? NQ : kPrefixTile));
        o[y] = __ldcg(reinterpret_cast<const float4*>(s + (mine ? ov : size_t(row) * D + 4 * c4)));
      }
    }
    float ref = top;
#pragma unroll
    for (int y = 0; y < kDepth; ++y) ref = fmaxf(ref, m[y]);
    const float base = ref == -INFINITY ? 0.f : ref;
    const float w0 = fast_exp2(top - base);   // 2^-inf = 0
    top = ref;
    sum *= w0;
    acc = make_float4(acc.x * w0, acc.y * w0, acc.z * w0, acc.w * w0);
#pragma unroll
    for (int y = 0; y < kDepth; ++y) {
      const float w = fast_exp2(m[y] - base);
      sum = fmaf(l[y], w, sum);
      acc.x = fmaf(o[y].x, w, acc.x);
      acc.y = fmaf(o[y].y, w, acc.y);
      acc.z = fmaf(o[y].z, w, acc.z);
      acc.w = fmaf(o[y].w, w, acc.w);
    }
  }
  const size_t orow = (size_t(b) * T + r / GQ) * A.hq + size_t(g) * GQ + r % GQ;
  const float inv = row_scale(A, sum);
  reinterpret_cast<uint2*>(A.o + orow * D)[c4] =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (A.lse && c4 == 0) A.lse[orow] = row_lse(A, top, sum);
}

template <int D, int M, int CPS>
cudaError_t launch_attend(const AttendArgs& a, int grid, size_t smem, cudaStream_t stream) {
  auto kern = attend_kernel<D, M, CPS>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t attr = once_per_device(done, [&] {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e == cudaSuccess && CPS > 1)   // room for CPS CTAs' shared memory
      e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                               int(cudaSharedmemCarveoutMaxShared));
    return e;
  });
  if (attr != cudaSuccess) return attr;
  return launch_pdl(kern, dim3(grid), dim3(NTH), smem, stream, a);
}

// Whole units per CTA or tiles split evenly: whole units save the merge and the
// partials' traffic, worth about 4 tiles of a CTA's time for a few units and 11
// from a hundred on, and cost the tiles that the busiest CTA has beyond its
// share.  The host knows no lengths, so the rule takes every unit to be as long as
// it can be; where one sequence is long and the others short, whole units leave
// their CTAs all of its tiles, so no CTA gets more than kWholeTiles in that way.
// us whole / split, T = 1, 64/8/128, calls in a graph, by units and window (tiles),
// with every sequence longer than the window, and with one that long among
// sequences of 60 rows:
//     8 units   128 (3)  6.9 /  7.9,   448 (8) 10.0 / 8.2
//    32         448 (8) 10.3 /  9.8,  1024 (17) 15.8 / 11.9
//   128         448 (8) 11.3 / 14.1,  one long: 10.8 / 10.0
//   128        1024 (17) 17.8 / 16.9, one long: 16.4 / 12.9
//   304        1024 (17) 27.1 / 29.3, one long: 17.5 / 13.8
//   304        2048 (33) 49.5 / 51.7, one long: 27.4 / 14.6
//   304        4096 (65) 94.0 / 95.7, one long: 47.5 / 18.4
//   608         448 (8) 24.5 / 27.4,  one long: 19.4 / 17.7
//   608        1024 (17) 49.7 / 52.8, one long: 31.0 / 18.5
// (14/2/64, 304 units: 1024 15.4 / 17.2 and 14.6 / 12.1, 2048 28.7 / 30.6 and 22.9 / 12.6).
constexpr int kWholeTiles = 20;
bool whole_units(long long units, int tiles, long long ctas) {
  const long long busiest = (units + ctas - 1) / ctas * tiles;
  const long long share = std::max(1LL, units * tiles / ctas);
  return busiest <= kWholeTiles && busiest - share <= std::min(11LL, 4 + units / 16);
}

// The own parts and the prefix one after the other on all SMs, or side by side,
// the own parts with one CTA on each of x SMs?  us that an SM needs, measured at
// 64/8/128 (lengths by their capacities, as the host knows no more): an own tile
// of 64 rows 0.6 and a unit 2 alone on the SM, a tile 0.7 of all SMs' time when
// the whole GPU streams them; a prefix tile of 128 rows 1.1 with one row tile,
// 1.75 with two; one after the other costs about 5 us more.  Long calls stay one
// after the other: there the own parts' CTAs came to share SMs and held the call
// up (768 rows over 32 K 120 -> 146 us).  So do calls whose one part would get so
// few SMs that it takes more than 20 us longer on them than on all: where the
// other part is much shorter than its cache, that is what the call waits for.
// us side by side / one after the other, single tokens of 4 sequences in a graph,
// with lengths as the caches have room for, and with a prefix of 100 rows:
//   prefix cache  8 K, own  576   18.0 / 24.1, 15.4 / 17.2   side by side
//                32 K       576   36.9 / 45.5, 24.2 / 17.2   side by side
//                32 K      2048   43.5 / 47.9, 32.0 / 19.3   side by side
//                64 K       576   56.8 / 63.1, 41.4 / 17.3   one after the other
//                64 K      2048   66.9 / 66.0, 49.4 / 19.3   one after the other
// Returns x, or 0.
int beside_sms(long long units, long long own_tiles, long long prefix_tiles, bool two, int num_sms) {
  const double own = 0.6 * double(own_tiles) + 2.0 * double(units), prefix = (two ? 1.75 : 1.1) * double(prefix_tiles);
  const int x = std::min(std::max(int(num_sms * own / (own + prefix) + 0.5), 1), num_sms / 2);
  const double own_all = 0.7 * double(own_tiles) / num_sms, prefix_all = prefix / num_sms;
  const double own_few = own / x, prefix_few = prefix / (num_sms - x), after = own_all + prefix_all + 5;
  if (after > 40 || std::max(own_few, prefix_few) >= after) return 0;
  return std::max(own_few - own_all, prefix_few - prefix_all) <= 20 ? x : 0;
}

// 64-row MMAs while the query rows fit, two CTAs per SM while two fit (at d = 64
// for every count of rows, so the shape between has no kernel there).
template <int D>
constexpr bool two_fit(int NQ) {
  return NQ <= 64 && 2 * (make_lay<D, 2>(NQ).total + 1024) <= kSmemPerSm;
}
template <int D>
cudaError_t launch_own(const AttendArgs& a, int NQ, int grid, cudaStream_t stream) {
  if (two_fit<D>(NQ)) return launch_attend<D, 64, 2>(a, grid, make_lay<D, 2>(NQ).total, stream);
  if constexpr (!two_fit<D>(64))
    if (NQ <= 64) return launch_attend<D, 64, 1>(a, grid, make_lay<D, 1>(NQ).total, stream);
  return launch_attend<D, 128, 1>(a, grid, make_lay<D, 1>(NQ).total, stream);
}

template <int D>
cudaError_t launch_d(AttendArgs& a, int num_sms, cudaStream_t stream) {
  const int NQ = a.T * (a.hq / a.hkv);
  const long long units = (long long)a.B * a.hkv;
  int ctas = std::min((two_fit<D>(NQ) ? 2 : 1) * num_sms, kAttendGridMax);
  if (a.pgrid) {
    const int x = beside_sms(units, units * a.max_tiles, (a.Pcap + kPrefixTile - 1) / kPrefixTile * (long long)a.hkv * a.pairs,
                             a.row_tiles > 1, num_sms);
    if (x) {
      ctas = x;
      a.pgrid = std::min(num_sms - x, kPrefixGridMax);
    }
  }
  a.whole = whole_units(units, a.max_tiles, ctas);
  const int grid = int(std::min<long long>(ctas, units * (a.whole ? 1 : a.max_tiles)));
  cudaError_t e = launch_own<D>(a, NQ, grid, stream);
  if (e != cudaSuccess || (a.whole && !a.pgrid)) return e;
  if (a.pgrid) e = prefix_launch(a, D, stream);
  if (e != cudaSuccess) return e;
  const dim3 mgrid((NQ * (D / 4) + kMergeThreads - 1) / kMergeThreads, unsigned(a.B * a.hkv));
  return a.pgrid ? launch_pdl(attend_merge_kernel<D, true>, mgrid, dim3(kMergeThreads), 0, stream, a)
                 : launch_pdl(attend_merge_kernel<D, false>, mgrid, dim3(kMergeThreads), 0, stream, a);
}

}  // namespace

cudaError_t attend_launch(AttendArgs& a, int D, int num_sms, cudaStream_t stream) {
  return D == 128 ? launch_d<128>(a, num_sms, stream) : launch_d<64>(a, num_sms, stream);
}

}  // namespace dustin
