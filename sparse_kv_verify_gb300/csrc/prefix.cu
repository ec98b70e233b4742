// The shared prefix of a batch, read once for all of its query rows.
//
// The B * T tokens of the batch, G query heads each, are the rows of tiles of
// nt = 128 / G tokens (rows t * G + h; the last tile and, where G does not
// divide 128, every tile leave MMA rows unused).  A unit is (KV head, pair of
// row tiles); its n = ceil(P / 128) key tiles, flattened over the units, are
// shared evenly among one CTA per SM.  Each key tile's K and V rows are read
// from memory once per pair of row tiles -- 256 query rows -- so that from
// about 280 rows on the two products bound the kernel, not the bytes.
//
// Roles (handing over through mbarriers):
//   warps 0-3, 4-7  softmax of row tile 0 and 1 ("lanes"), one thread per row: a
//                   step's scores in registers, P (bf16) stored over them; the
//                   reference maximum moves only when a step passes it by more
//                   than 2^8, and then the thread rescales its row of O;
//   warp 9          K and V tiles into a ring of 128-row stages, one tiled TMA
//                   load each;
//   warp 8          the tile that ends the prefix, by cp.async with its rows past
//                   the end zero-filled (they may hold anything, and 0 * NaN is
//                   not 0);
//   warp 10         one thread issues the MMAs, per step i and lane a batch
//                   O += P(i) V(i), S(i + NB) = Q K(i + NB)^T over the S and P that
//                   the first product has read (MMAs of one thread run in the
//                   order of issue).
//
// Two shapes of the pipeline:
//   two row tiles   steps of 128 keys, one S buffer per lane (NB = 1): while one
//                   lane's softmax works the tensor core has the other lane's
//                   products.  Bound by the chain of a lane, products (2 x 512
//                   cycles) -> S -> softmax (about 1250) -> P; steps of 64 keys
//                   keep the softmax fed but pay the hand-overs twice and an S
//                   product that shared memory bounds (48 cycles for 32).
//   one row tile    (at most 128 query rows in all) the products wait for nobody
//                   else, so steps of 64 keys with two S buffers (NB = 2): S of
//                   the next step is there when the softmax comes to it.
// us of the whole call, one row tile in the one-tile / two-tile shape: 32 rows
// over P = 8192 at 64/8/128 20.1 / 21.6; 14/2/64 behind 3001 rows 13.0 / 13.4.
// Two row tiles with steps of 128 / 64 keys (runs on two machines, which differ
// by up to 5 %): 1280 rows over 64 K 301 / 339.
//
// 1280 rows over 64 K: this kernel 243 to 254 us, 1.35 to 1.42 PFLOP/s (0.71 to
// 0.75 of cuBLAS's measured rate): 1.8 us per 128 keys and two row tiles.  Over
// 16 K the tensor pipe is active 47 % of the time and DRAM 12 %.
//
// Tensor memory: S of lane 0 and 1 in columns [0, 128) and [128, 256), O in
// [256, 256 + D) and [384, 384 + D).  Every segment (unit x CTA) writes its row
// maxima, sums and unnormalised O to slot (unit + cta) * 2 + lane; the merge
// kernel adds the sequences' own part.
#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace dustin {

namespace {

constexpr int TK = kPrefixTile;      // keys per tile, and query rows per row tile
constexpr int kGatherWarp = 8, kLoadWarp = 9, kMmaWarp = 10;
constexpr int NTH = 384;             // 168 registers a thread (a softmax thread holds a row's scores)
constexpr int kSCol = 0, kOCol = 256;                // lane 1: + 128

template <int D, int LANES>
struct Cfg {
  static constexpr int nb = LANES == 2 ? 1 : 2;      // S buffers per lane, and steps per tile
  static constexpr int step = TK / nb;               // keys per step
  static constexpr int nst = LANES == 2 ? (D == 128 ? 5 : 8) : (D == 128 ? 6 : 12);   // K or V tiles in the ring
  static constexpr uint32_t panel = TK * 128;        // 64 columns of a K, V or Q tile
  static constexpr uint32_t stage = (D / 64) * panel;
  static constexpr uint32_t ring_off = LANES * stage;   // after the query tiles
  static constexpr uint32_t bar_off = ring_off + nst * stage;
  static constexpr uint32_t misc_off = bar_off + (2 * nst + 17) * 8;   // barriers
  static constexpr uint32_t total = misc_off + 16 + 1024;
};

// The 128 rows from `row` on of KV head g of a prefix cache.
__device__ __forceinline__ void tma_load_tile(uint32_t dst, const CUtensorMap* map, int row, int g, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %2, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(g), "r"(smem_u32(bar))
      : "memory");
}

// One segment of this CTA: key tiles [i0, i0 + n) of unit u.
struct Seg {
  int u, i0, n, g, pair;
  bool two;   // the pair has a second row tile
};
__device__ __forceinline__ bool next_seg(Seg& s, long long& t, long long t1, int tiles, const AttendArgs& A) {
  if (t >= t1) return false;
  s.u = int(t / tiles);
  s.i0 = int(t - (long long)s.u * tiles);
  const long long left = t1 - t;
  s.n = int(left < tiles - s.i0 ? left : tiles - s.i0);
  t += s.n;
  s.g = s.u / A.pairs;
  s.pair = s.u - s.g * A.pairs;
  s.two = 2 * s.pair + 1 < A.row_tiles;
  return true;
}

template <int D, int LANES>
__global__ void __launch_bounds__(NTH, 1) prefix_kernel(const __grid_constant__ AttendArgs A) {
  using C = Cfg<D, LANES>;
  constexpr int NST = C::nst, NB = C::nb, SK = C::step;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::bar_off);
  uint64_t* empty = full + NST;
  uint64_t* q_full = empty + NST;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;      // [lane][buffer] a batch with an S is done
  uint64_t* p_full = s_full + 4;       // [lane][buffer] P is stored over S
  uint64_t* o_full = p_full + 4;       // [lane][z] the z-th of a segment's last NB batches, without an S, is done
  uint64_t* mma_done = o_full + 4;
  uint64_t* go = mma_done + 1;         // a tile that comes by cp.async has a stage
  uint64_t* gathered = go + 1;         // its rows are in
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::misc_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::misc_off + 8);

  const int tid = threadIdx.x, warp = tid >> 5, lane_id = tid & 31;
  const int G = A.hq / A.hkv;
  const int n_act = (A.nt * G + 31) >> 5;   // softmax warps per lane that hold rows
  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int x = 0; x < 4; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 32 * n_act);
      mbar_init(&o_full[x], 1);
    }
    mbar_init(mma_done, 1);
    mbar_init(go, 1);
    mbar_init(gathered, 32);
    *abort_flag = 0;
    fence_barrier_init();
  }
  // This kernel starts on the SMs that the sequences' own part (the launch before
  // it) leaves; it shares no buffer with that launch, which let this one start
  // only after its own wait for everything before.  The wait before exit makes
  // this kernel end after it, for the merge.
  pdl_launch_dependents();
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "n"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  int P = __ldcg(A.prefix_len);
  if (P < 0 || P > A.Pcap) {
    if (blockIdx.x == 0 && tid == 0) flag_error(A.err, DUSTIN_DEV_SEQLEN);
    P = 0;
  }
  const int tiles = (P + TK - 1) / TK;
  const long long total = (long long)A.hkv * A.pairs * tiles;
  const long long ctas = total < gridDim.x ? total : gridDim.x;   // each with a tile
  long long t = 0, t1 = 0;
  if (blockIdx.x < ctas) {
    t = blockIdx.x * total / ctas;
    t1 = (blockIdx.x + 1) * total / ctas;
  }
  Seg sg;

  if (warp < 4 * LANES) {
    // =============================================================== softmax
    const int ln = warp >> 2;                       // lane (row tile of the pair)
    const int row = tid & 127;
    if ((warp & 3) < n_act) {
      const float scale = A.scale_log2;
      const uint32_t lane_base = tmem + (uint32_t((warp & 3) * 32) << 16);
      const uint32_t s_tmem = lane_base + uint32_t(kSCol + 128 * ln), o_tmem = lane_base + uint32_t(kOCol + 128 * ln);
      // S of the lane's J-th step completes phase J / NB of s_full[lane][J % NB], in
      // one batch with P V of step J - NB; P V of step n - NB + z of a segment
      // completes a phase of o_full[lane][z].  Every thread waits for every phase
      // in turn, and the one after it needs a P that the thread stores later: no
      // wait by parity can be lapped or pass early.
      auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
        return bool(__all_sync(0xffffffffu, mbar_wait(bar, parity, A.err, abort_flag)));
      };
      auto wait_s = [&](int J) { return wait_warp(&s_full[2 * ln + J % NB], uint32_t(J / NB) & 1u); };
      int j0 = 0, segs = 0;   // steps and segments of the lane before this segment
      auto wait_o = [&](int z) { return wait_warp(&o_full[2 * ln + z], uint32_t(segs) & 1u); };
      bool live = true;
      while (live && next_seg(sg, t, t1, tiles, A)) {
        if (ln == 1 && !sg.two) continue;
        const int tok = (2 * sg.pair + ln) * A.nt + row / G;
        const bool act = row < A.nt * G && tok < A.B * A.T;
        const int n = NB * sg.n;                    // steps
        float mref = -INFINITY, lsum = 0.f;
        for (int i = 0; i < n; ++i) {
          const int nv = P - (NB * sg.i0 + i) * SK;  // keys of this step, if under SK
          const uint32_t sb = s_tmem + uint32_t((j0 + i) % NB * SK);
          if (!wait_s(j0 + i)) {
            live = false;
            break;
          }
          tc_fence_after();
          float x[SK];
#pragma unroll
          for (int c = 0; c < SK; c += 64) tc_ld64(sb + uint32_t(c), reinterpret_cast<uint32_t*>(x + c));
          if (nv < SK) {
#pragma unroll
            for (int j = 0; j < SK; ++j) x[j] = j < nv ? x[j] : -INFINITY;
          }
          float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int j = 4; j + 8 <= SK; j += 8)
#pragma unroll
            for (int y = 0; y < 4; ++y) m4[y] = fmaxf(m4[y], fmaxf(x[j + y], x[j + 4 + y]));
#pragma unroll
          for (int y = 0; y < 4; ++y) m4[y] = fmaxf(m4[y], x[SK - 4 + y]);
          const float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          // (a row that is not in use never rescales O; its P and O are never read)
          const float mx = act ? top * scale : -INFINITY;
          float alpha = 1.f;
          if (mx > mref + 8.f) {
            alpha = fast_exp2(mref - mx);   // 0 while mref is -inf
            mref = mx;
            lsum *= alpha;
          }
          const float nb = mref == -INFINITY ? 0.f : -mref;
          // rescale this row of O once P V of the step before is in (NB = 1: it
          // came with S of this step; NB = 2: it comes with S of the next one, or
          // alone after the last)
          if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            if (NB > 1 && !(i + 1 < n ? wait_s(j0 + i + 1) : wait_o(0))) {
              live = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tc_ld32(o_tmem + uint32_t(c), o);
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * alpha);
              tc_st32(o_tmem + uint32_t(c), o);
            }
          }
          float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
          for (int h = 0; h < SK / 32; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              float* y = x + 32 * h + j;
              fma2(y[0], y[1], scale, nb);
              fma2(y[2], y[3], scale, nb);
              const float p0 = fast_exp2(y[0]), p1 = fast_exp2(y[1]), p2 = fast_exp2(y[2]), p3 = fast_exp2(y[3]);
              add2(l0, l1, p0, p1);
              add2(l2, l3, p2, p3);
              pk[j / 2] = pack_bf16(p0, p1);
              pk[j / 2 + 1] = pack_bf16(p2, p3);
            }
            tc_st16(sb + uint32_t(16 * h), pk);
          }
          tc_wait_st();
          lsum += (l0 + l1) + (l2 + l3);
          tc_fence_before();
          mbar_arrive(&p_full[2 * ln + (j0 + i) % NB]);
        }
        if (!live) break;
        // --------------------------------------------------------- epilogue
#pragma unroll
        for (int z = 0; z < NB; ++z) live = live && wait_o(z);
        if (!live) break;
        j0 += n;
        ++segs;
        tc_fence_after();
        if (tid == 0) {   // (lane 0 has a row tile in every unit)
          if (sg.i0 == 0) A.pseg_cta[2 * sg.u] = int(blockIdx.x);
          if (sg.i0 + sg.n == tiles) A.pseg_cta[2 * sg.u + 1] = int(blockIdx.x);
        }
        float* part = A.ppartial + ((size_t(sg.u) + blockIdx.x) * 2 + ln) * (size_t(TK) * (D + 2));
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tc_ld32(o_tmem + uint32_t(c), o);   // collective: every lane loads
          if (act) {
            float4* dst = reinterpret_cast<float4*>(part + size_t(row) * D + c);
#pragma unroll
            for (int y = 0; y < 32; y += 4)
              dst[y / 4] = make_float4(__uint_as_float(o[y]), __uint_as_float(o[y + 1]), __uint_as_float(o[y + 2]),
                                       __uint_as_float(o[y + 3]));
          }
        }
        if (act) {
          part[size_t(TK) * D + row] = mref;
          part[size_t(TK) * D + TK + row] = lsum;
        }
        tc_fence_before();
      }
    }
  } else if (warp == kLoadWarp) {
    if (lane_id == 0) {
      // ============================================================== loads
      int gi = 0, st = 0, segs = 0, gathers = 0;
      uint32_t ph = 0;                            // of stage st
      bool live = true;
      while (live && next_seg(sg, t, t1, tiles, A)) {
        // this segment's query tiles, once the last one's S MMAs have read theirs
        if (segs > 0 && !mbar_wait(q_empty, uint32_t(segs - 1) & 1u, A.err, abort_flag)) break;
        const uint32_t bytes = uint32_t(A.nt * G) * D * 2;
        mbar_arrive_expect_tx(q_full, sg.two ? 2 * bytes : bytes);
        for (int ln = 0; ln < (sg.two ? 2 : 1); ++ln)
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(sbase + uint32_t(ln) * C::stage + uint32_t(h) * C::panel, &A.pqmap, h * 64, sg.g * G,
                        (2 * sg.pair + ln) * A.nt, q_full);
        ++segs;
        for (int i = 0; i < 2 * sg.n; ++i) {      // K and V of each tile in turn
          const int base = (sg.i0 + (i >> 1)) * TK;
          if (gi >= NST && !mbar_wait(&empty[st], ph ^ 1u, A.err, abort_flag)) {
            live = false;
            break;
          }
          if (base + TK <= P && A.ptma) {
            mbar_arrive_expect_tx(&full[st], C::stage);
            tma_load_tile(sbase + C::ring_off + uint32_t(st) * C::stage, i & 1 ? &A.pvmap : &A.pkmap, base, sg.g, &full[st]);
          } else {   // rows by the gathering warps
            mbar_arrive(go);
            if (!mbar_wait(gathered, uint32_t(gathers++) & 1u, A.err, abort_flag)) {
              live = false;
              break;
            }
            mbar_arrive(&full[st]);
          }
          ++gi;
          if (++st == NST) {
            st = 0;
            ph ^= 1u;
          }
        }
      }
      // what is in flight has landed before the CTA may exit: the query tiles
      // and the latest load of each stage
      if (segs > 0) mbar_drain(q_full, uint32_t(segs - 1) & 1u, A.err);
      for (int j = gi > NST ? gi - NST : 0; j < gi; ++j) mbar_drain(&full[j % NST], uint32_t(j / NST) & 1u, A.err);
    }
    __syncwarp();
  } else if (warp == kGatherWarp) {
    // ============================================================== gathers
    // the tile that ends the prefix, row by row (or every tile, of caches that
    // no tensor map describes); the loading thread, which alone follows the
    // ring, lets these start and waits for them before it goes on
    constexpr int CH = D / 8;             // 16-byte chunks per row
    constexpr int KPI = 32 / CH;          // rows per warp instruction
    const int c = lane_id % CH, ksub = lane_id / CH;
    int gi = 0, gathers = 0;
    bool live = true;
    while (live && next_seg(sg, t, t1, tiles, A)) {
      for (int i = 0; i < 2 * sg.n; ++i, ++gi) {
        const int base = (sg.i0 + (i >> 1)) * TK;
        if (base + TK <= P && A.ptma) continue;
        if (!mbar_wait(go, uint32_t(gathers++) & 1u, A.err, abort_flag)) {
          live = false;
          break;
        }
        const bool is_v = i & 1;
        const uint32_t stage = sbase + C::ring_off + uint32_t(gi % NST) * C::stage;
        const uint16_t* src = is_v ? A.pv + size_t(sg.g) * A.pvsh : A.pk + size_t(sg.g) * A.pksh;
        const int64_t sl = is_v ? A.pvsl : A.pksl;
#pragma unroll 8
        for (int m = 0; m < TK / KPI; ++m) {
          const int key = m * KPI + ksub;
          const bool ok = base + key < P;
          cp_async16(stage + uint32_t(c >> 3) * C::panel + swz(key, c & 7), src + size_t(ok ? base + key : 0) * sl + c * 8,
                     ok ? 16u : 0u);
        }
        cp_async_wait_all();
        fence_proxy_async();
        mbar_arrive(gathered);
      }
    }
    __syncwarp();
  } else {
    if (warp == kMmaWarp) {
      // ================================================================ MMAs
      constexpr uint32_t kIdS = tc_idesc(128, SK, 0), kIdPV = tc_idesc(128, D, 1);
      const uint64_t q_desc = tc_desc(sbase, 16, 1024);
      const uint64_t k_desc = tc_desc(sbase + C::ring_off, 16, 1024), v_desc = tc_desc(sbase + C::ring_off, C::panel, 1024);
      int st = 0, segs = 0;                 // ring stage to consume next; segments
      uint32_t ph = 0, pp = 0;              // its phase; phases of the P buffers (bit 2 lane + buffer)
      bool issued = false, live = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return bool(__all_sync(0xffffffffu, mbar_wait(bar, parity, A.err, abort_flag)));
      };
      // the warp runs together and one elected lane issues; branches go by votes,
      // so that the compiler too knows the warp as converged
      auto uni = [](bool x) { return __any_sync(0xffffffffu, x) != 0; };
      auto next_stage = [&] {
        if (++st == NST) {
          st = 0;
          ph ^= 1u;
        }
      };
      while (live && uni(next_seg(sg, t, t1, tiles, A))) {
        const bool two = uni(sg.two);
        live = wait(q_full, uint32_t(segs++) & 1u);
        const int n = NB * sg.n;
        int sv = 0, sk = 0;                 // stages of V and of K
        for (int i = -NB; live && uni(i < n); ++i) {
          const bool first = NB == 1 || !(i & 1), last = NB == 1 || (i & 1);   // step of its tiles
          const bool pv = i >= 0, s = uni(i + NB < n);
          if (pv && first) {
            sv = st;
            live = wait(&full[sv], ph);
            next_stage();
          }
          if (live && s && first) {
            sk = st;
            live = wait(&full[sk], ph);
            next_stage();
          }
#pragma unroll
          for (int ln = 0; ln < LANES; ++ln) {
            if (!live || (ln == 1 && !two)) break;
            const int buf = NB == 1 ? 0 : i & 1;   // of step i and of step i + NB
            if (pv) {
              live = wait(&p_full[2 * ln + buf], (pp >> (2 * ln + buf)) & 1u);
              if (!live) break;
              pp ^= 1u << (2 * ln + buf);
            }
            issued = true;
            tc_fence_after();
            const uint32_t sp = tmem + uint32_t(kSCol + 128 * ln + buf * SK);
            if (pv) {
              const uint64_t v = v_desc + uint64_t(sv) * (C::stage >> 4) + (first ? 0u : uint32_t(SK * 8));
#pragma unroll
              for (int kk = 0; kk < SK / 16; ++kk)
                tc_mma_ts_elect(tmem + uint32_t(kOCol + 128 * ln), sp + uint32_t(kk * 8), v + uint32_t(kk * 128), kIdPV,
                          (i > 0 || kk > 0) ? 1 : 0);
            }
            if (s) {
              const uint64_t q = q_desc + uint64_t(ln) * (C::stage >> 4);
              const uint64_t k = k_desc + uint64_t(sk) * (C::stage >> 4) + (first ? 0u : uint32_t(SK * 8));
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = uint32_t(kk >> 2) * (C::panel >> 4) + uint32_t((kk & 3) * 2);
                tc_mma_ss_elect(sp, q + off, k + off, kIdS, kk > 0);
              }
            }
            tc_commit_elect(s ? &s_full[2 * ln + buf] : &o_full[2 * ln + buf]);   // (n is even where NB = 2)
          }
          if (!live) break;
          if (pv && last) tc_commit_elect(&empty[sv]);
          if (s && last) tc_commit_elect(&empty[sk]);
          if (uni(i + NB + 1 == n)) tc_commit_elect(q_empty);   // the query tiles are no longer read
        }
      }
      if (issued) {   // every MMA has completed before tensor memory is freed
        tc_commit_elect(mma_done);
        if (lane_id == 0) mbar_drain(mma_done, 0, A.err);
      }
    }
    __syncwarp();
  }

  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
}

template <int D, int LANES>
cudaError_t launch_t(const AttendArgs& a, cudaStream_t stream) {
  using C = Cfg<D, LANES>;
  static_assert(C::total <= 227 * 1024, "shared memory of a CTA");
  auto kern = prefix_kernel<D, LANES>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t attr = once_per_device(
      done, [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::total)); });
  if (attr != cudaSuccess) return attr;
  return launch_pdl(kern, dim3(a.pgrid), dim3(NTH), C::total, stream, a);
}

}  // namespace

cudaError_t prefix_launch(const AttendArgs& a, int D, cudaStream_t stream) {
  if (a.row_tiles == 1) return D == 128 ? launch_t<128, 1>(a, stream) : launch_t<64, 1>(a, stream);
  return D == 128 ? launch_t<128, 2>(a, stream) : launch_t<64, 2>(a, stream);
}

}  // namespace dustin
