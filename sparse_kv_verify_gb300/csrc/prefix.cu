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
//   warps 0-3, 4-7  softmax of row tile 0 and 1 ("lanes"), one thread per row:
//                   128 scores in registers, P (bf16) stored over them; the
//                   reference maximum moves only when a tile passes it by more
//                   than 2^8, and then the thread rescales its row of O;
//   warps 8, 9       K and V tiles into a ring of 128-row stages: one thread
//                   issues tiled TMA loads; the tile that ends the prefix comes
//                   by cp.async, its rows past the end zero-filled (they may
//                   hold anything, and 0 * NaN is not 0);
//   warp 10         one thread issues the MMAs, per key tile i and lane:
//                   O += P(i) V(i), then S(i + 1) = Q K(i + 1)^T over the S and
//                   P that the first of the two has read (MMAs of one thread
//                   run in the order of issue).  While one lane's softmax
//                   works, the tensor core has the other lane's products.
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

constexpr int TK = 128;              // keys per tile
constexpr int kLoaders = 2;
constexpr int kLoaderWarp0 = 8, kMmaWarp = 10;
constexpr int NTH = 384;             // 168 registers a thread (a softmax thread holds a row's 128 scores)
constexpr int kSCol = 0, kOCol = 256;                // lane 1: + 128

template <int D>
struct Cfg {
  static constexpr int nst = D == 128 ? 5 : 8;       // K or V tiles in the ring
  static constexpr uint32_t panel = TK * 128;        // 64 columns of a K, V or Q tile
  static constexpr uint32_t stage = (D / 64) * panel;
  static constexpr uint32_t ring_off = 2 * stage;    // after the two Q tiles
  static constexpr uint32_t bar_off = ring_off + nst * stage;
  static constexpr uint32_t misc_off = bar_off + (2 * nst + 11) * 8;   // barriers
  static constexpr uint32_t total = misc_off + 16 + 1024;
};

// 128 consecutive 32-bit columns of this thread's lane.
__device__ __forceinline__ void tc_ld128(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x128.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,"
      "%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,"
      "%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,%80,%81,%82,%83,%84,%85,%86,%87,"
      "%88,%89,%90,%91,%92,%93,%94,%95,%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,"
      "%110,%111,%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%128];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]),
        "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]),
        "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]),
        "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]),
        "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]),
        "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]),
        "=r"(r[103]), "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]), "=r"(r[109]),
        "=r"(r[110]), "=r"(r[111]), "=r"(r[112]), "=r"(r[113]), "=r"(r[114]), "=r"(r[115]), "=r"(r[116]),
        "=r"(r[117]), "=r"(r[118]), "=r"(r[119]), "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]),
        "=r"(r[124]), "=r"(r[125]), "=r"(r[126]), "=r"(r[127])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// (a, b) * (s, s) + (c, c), and (a, b) + (c, d), as one packed instruction each
__device__ __forceinline__ void fma2(float& a, float& b, float s, float c) {
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %2};\n mov.b64 z, {%3, %3};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
      : "+f"(a), "+f"(b)
      : "f"(s), "f"(c));
}
__device__ __forceinline__ void add2(float& a, float& b, float c, float d) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n"
      " add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d));
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

template <int D>
__global__ void __launch_bounds__(NTH, 1) prefix_kernel(const __grid_constant__ AttendArgs A) {
  using C = Cfg<D>;
  constexpr int NST = C::nst;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::bar_off);
  uint64_t* empty = full + NST;
  uint64_t* q_full = empty + NST;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;      // [2] S of the lane's next tile is in
  uint64_t* p_full = s_full + 2;       // [2] P is stored
  uint64_t* o_full = p_full + 2;       // [2] the segment's last P V is in
  uint64_t* mma_done = o_full + 2;
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
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 32 * n_act);
      mbar_init(&o_full[x], 1);
    }
    mbar_init(mma_done, 1);
    mbar_init(go, 1);
    mbar_init(gathered, 32 * kLoaders);
    *abort_flag = 0;
    fence_barrier_init();
  }
  pdl_launch_dependents();
  pdl_wait();
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "n"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  int P = *A.prefix_len;
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

  if (warp < 8) {
    // =============================================================== softmax
    const int ln = warp >> 2;                       // lane (row tile of the pair)
    const int row = tid & 127;
    if ((warp & 3) < n_act) {
      const float scale = A.scale_log2;
      const uint32_t lane_base = tmem + (uint32_t((warp & 3) * 32) << 16);
      const uint32_t s_tmem = lane_base + uint32_t(kSCol + 128 * ln), o_tmem = lane_base + uint32_t(kOCol + 128 * ln);
      int gi = 0, segs = 0;
      bool live = true;
      while (live && next_seg(sg, t, t1, tiles, A)) {
        if (ln == 1 && !sg.two) continue;
        const int tok = (2 * sg.pair + ln) * A.nt + row / G;
        const bool act = row < A.nt * G && tok < A.B * A.T;
        float mref = -INFINITY, lsum = 0.f;
        for (int i = 0; i < sg.n; ++i, ++gi) {
          const int nv = P - (sg.i0 + i) * TK;      // keys of this tile, if under TK
          if (!__all_sync(0xffffffffu, mbar_wait(&s_full[ln], uint32_t(gi) & 1u, A.err, abort_flag))) {
            live = false;
            break;
          }
          tc_fence_after();
          float x[TK];
          tc_ld128(s_tmem, reinterpret_cast<uint32_t*>(x));
          if (nv < TK) {
#pragma unroll
            for (int j = 0; j < TK; ++j) x[j] = j < nv ? x[j] : -INFINITY;
          }
          float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int j = 4; j < TK; j += 8)
#pragma unroll
            for (int y = 0; y < 4; ++y) m4[y] = j + 4 + y < TK ? fmaxf(m4[y], fmaxf(x[j + y], x[j + 4 + y])) : fmaxf(m4[y], x[j + y]);
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
          // rescale this row of O: S of this tile came after P V of the last one
          if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
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
          for (int h = 0; h < 4; ++h) {
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
            tc_st16(s_tmem + uint32_t(16 * h), pk);
          }
          tc_wait_st();
          lsum += (l0 + l1) + (l2 + l3);
          tc_fence_before();
          mbar_arrive(&p_full[ln]);
        }
        if (!live) break;
        // --------------------------------------------------------- epilogue
        if (!__all_sync(0xffffffffu, mbar_wait(&o_full[ln], uint32_t(segs++) & 1u, A.err, abort_flag))) break;
        tc_fence_after();
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
  } else if (warp < kLoaderWarp0 + kLoaders) {
    // =============================================================== loaders
    const int lw = warp - kLoaderWarp0;
    constexpr int CH = D / 8;             // 16-byte chunks per row
    constexpr int KPI = 32 / CH;          // rows per warp instruction
    const int c = lane_id % CH, ksub = lane_id / CH;
    const uint64_t pol = policy_evict_last();   // the other pairs of this head read it again
    const bool lead = lw == 0 && lane_id == 0;
    int gi = 0, segs = 0, q_issued = 0, gathers = 0;
    bool live = true;
    while (live && next_seg(sg, t, t1, tiles, A)) {
      if (lead) {
        // this segment's query tiles, once the last one's S MMAs have read theirs
        if (segs > 0 && !mbar_wait(q_empty, uint32_t(segs - 1) & 1u, A.err, abort_flag)) break;
        const uint32_t bytes = uint32_t(A.nt * G) * D * 2;
        mbar_arrive_expect_tx(q_full, sg.two ? 2 * bytes : bytes);
        for (int ln = 0; ln < (sg.two ? 2 : 1); ++ln)
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(sbase + uint32_t(ln) * C::stage + uint32_t(h) * C::panel, &A.pqmap, h * 64, sg.g * G,
                        (2 * sg.pair + ln) * A.nt, q_full);
        ++q_issued;
      }
      ++segs;
      for (int i = 0; i < 2 * sg.n; ++i, ++gi) {   // K and V of each tile in turn
        const int st = gi % NST;
        const int base = (sg.i0 + (i >> 1)) * TK;
        const bool is_v = i & 1, whole = base + TK <= P && A.ptma;
        if (whole && !lead) continue;
        if (lead && gi >= NST && !mbar_wait(&empty[st], uint32_t(gi / NST - 1) & 1u, A.err, abort_flag)) {
          live = false;
          break;
        }
        const uint32_t stage = sbase + C::ring_off + uint32_t(st) * C::stage;
        if (whole) {
          mbar_arrive_expect_tx(&full[st], C::stage);
          const CUtensorMap* map = is_v ? &A.pvmap : &A.pkmap;
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            const uint32_t dst = stage + uint32_t(h) * C::panel;
            if ((is_v ? A.pvrank : A.pkrank) == 2) tma_load_2d_u32(dst, map, h * 64, sg.g * A.Pcap + base, &full[st], pol);
            else tma_load_4d_u32(dst, map, h * 64, base, sg.g, 0, &full[st], pol);
          }
          continue;
        }
        // rows by every loader thread: the leading one, which alone follows the
        // ring, lets the others start and waits for them before it goes on
        if (lead) {
          mbar_arrive(go);
        } else if (!mbar_wait(go, uint32_t(gathers) & 1u, A.err, abort_flag)) {
          live = false;
          break;
        }
        const uint16_t* src = is_v ? A.pv + size_t(sg.g) * A.pvsh : A.pk + size_t(sg.g) * A.pksh;
        const int64_t sl = is_v ? A.pvsl : A.pksl;
#pragma unroll 4
        for (int m = 0; m < TK / kLoaders / KPI; ++m) {
          const int key = TK / kLoaders * lw + m * KPI + ksub;
          const bool ok = base + key < P;
          cp_async16(stage + uint32_t(c >> 3) * C::panel + swz(key, c & 7), src + size_t(ok ? base + key : 0) * sl + c * 8,
                     ok ? 16u : 0u);
        }
        cp_async_wait_all();
        fence_proxy_async();
        mbar_arrive(gathered);
        if (lead) {
          if (!mbar_wait(gathered, uint32_t(gathers) & 1u, A.err, abort_flag)) {
            live = false;
            break;
          }
          mbar_arrive(&full[st]);
        }
        ++gathers;
      }
    }
    cp_async_wait_all();
    // what is in flight has landed before the CTA may exit: the query tiles and
    // the latest load of each stage
    if (lead) {
      if (q_issued > 0) mbar_drain(q_full, uint32_t(q_issued - 1) & 1u, A.err);
      for (int j = gi > NST ? gi - NST : 0; j < gi; ++j) mbar_drain(&full[j % NST], uint32_t(j / NST) & 1u, A.err);
    }
    __syncwarp();
  } else {
    if (warp == kMmaWarp && lane_id == 0) {
      // ================================================================ MMAs
      constexpr uint32_t kIdS = tc_idesc(128, TK, 0), kIdPV = tc_idesc(128, D, 1);
      int gi = 0, segs = 0;            // ring position (K of the current tile), segments
      uint32_t np[2] = {0, 0};         // tiles of each lane so far
      bool issued = false, live = true;
      auto wait_full = [&](int x) { return mbar_wait(&full[x % NST], uint32_t(x / NST) & 1u, A.err, abort_flag); };
      auto s_mma = [&](int ln, int x) {   // S = Q K^T with K in ring position x
        const uint32_t q = sbase + uint32_t(ln) * C::stage, k = sbase + C::ring_off + uint32_t(x % NST) * C::stage;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = uint32_t(kk >> 2) * C::panel + uint32_t((kk & 3) * 32);
          tc_mma_ss(tmem + uint32_t(kSCol + 128 * ln), tc_desc(q + off, 16, 1024), tc_desc(k + off, 16, 1024), kIdS, kk > 0);
        }
        tc_commit(&s_full[ln]);
      };
      auto pv_mma = [&](int ln, int x, bool acc) {   // O (+)= P V with V in ring position x
        const uint32_t v = sbase + C::ring_off + uint32_t(x % NST) * C::stage;
#pragma unroll
        for (int kk = 0; kk < TK / 16; ++kk)
          tc_mma_ts(tmem + uint32_t(kOCol + 128 * ln), tmem + uint32_t(kSCol + 128 * ln + kk * 8),
                    tc_desc(v + uint32_t(kk * 2048), C::panel, 1024), kIdPV, (acc || kk > 0) ? 1 : 0);
      };
      while (live && next_seg(sg, t, t1, tiles, A)) {
        const int lanes = sg.two ? 2 : 1;
        if (!mbar_wait(q_full, uint32_t(segs++) & 1u, A.err, abort_flag) || !wait_full(gi)) break;
        issued = true;
        tc_fence_after();
        for (int ln = 0; ln < lanes; ++ln) s_mma(ln, gi);
        tc_commit(&empty[gi % NST]);
        if (sg.n == 1) tc_commit(q_empty);
        for (int i = 0; i < sg.n && live; ++i, gi += 2) {
          const bool more = i + 1 < sg.n;
          for (int ln = 0; ln < lanes; ++ln) {
            if (!mbar_wait(&p_full[ln], np[ln]++ & 1u, A.err, abort_flag) || (ln == 0 && !wait_full(gi + 1))) {
              live = false;
              break;
            }
            tc_fence_after();
            pv_mma(ln, gi + 1, i > 0);
            if (more) {
              if (ln == 0 && !wait_full(gi + 2)) {
                live = false;
                break;
              }
              s_mma(ln, gi + 2);
            } else {
              tc_commit(&o_full[ln]);
            }
          }
          if (!live) break;
          tc_commit(&empty[(gi + 1) % NST]);
          if (more) {
            tc_commit(&empty[(gi + 2) % NST]);
            if (i + 2 == sg.n) tc_commit(q_empty);   // the query tiles are no longer read
          }
        }
      }
      if (issued) {   // every MMA has completed before tensor memory is freed
        tc_commit(mma_done);
        mbar_drain(mma_done, 0, A.err);
      }
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
}

template <int D>
cudaError_t launch_d(const AttendArgs& a, cudaStream_t stream) {
  auto kern = prefix_kernel<D>;
  static const cudaError_t attr =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Cfg<D>::total));
  if (attr != cudaSuccess) return attr;
  return launch_pdl(kern, dim3(a.pgrid), dim3(NTH), Cfg<D>::total, stream, a);
}

static_assert(Cfg<128>::total <= 227 * 1024 && Cfg<64>::total <= 227 * 1024, "shared memory of a CTA");

}  // namespace

cudaError_t prefix_launch(const AttendArgs& a, int D, cudaStream_t stream) {
  return D == 128 ? launch_d<128>(a, stream) : launch_d<64>(a, stream);
}

}  // namespace dustin
