// Causal attention of a ragged batch's new tokens over a paged cache
// (dustin_paged_attn): query t of request b, at position p = kv_len - n + t, gets
// o = softmax(q.k / sqrt(d)) v and lse = ln sum exp(q.k / sqrt(d)) over the cache
// rows 0..p, row j in row j % page of page table[b][j / page].
//
// Row tiles: nt = 128 / G tokens of a request, G query heads each, are the rows
// t * G + h of a tile (G query heads share a KV head).  A unit is (request, KV
// head, pair of row tiles; one row tile where no request has more) and reads the
// 128-key tiles of the rows that its last token sees; masks inside a tile are the
// causal rule's.  How many units and tiles there are only the device knows: every
// CTA sums the requests' costs (one warp) and takes its equal share of the
// flattened tiles, so that single tokens behind long contexts and chunks of
// prompts load the SMs alike; a cut near the end of a unit is moved there.  K and V
// rows are read once per pair of row tiles.
//
// Roles (handing over through mbarriers and named barriers):
//   warps 0-3, 4-7  softmax of row tile 0 and 1 ("lanes"), one thread per row: a
//                   step's scores in registers, P (bf16) stored over them.  The
//                   reference maximum is the first step's; a later step is weighed
//                   against it at once, and only where a row's weights sum to more
//                   than 2^12 again against a new one, with which the thread rescales
//                   its row of O (looking for each step's maximum first took 2.48
//                   instead of 2.39 ms for 4096 tokens over 28 K).  P is rounded to
//                   bf16 for the second product; the row sum adds the unrounded fp32
//                   values, so lse keeps fp32 accuracy;
//   two warps       K and V tiles into a ring of 128-row stages, a page's rows in one
//                   tiled TMA load, the pages of a tile by as many threads, half
//                   of them by each warp (a load takes about 95 cycles, however
//                   small).  A stage holds groups of 8 rows one after another, a
//                   group as its 64-column panels of 8 swizzled rows; pools whose
//                   strides keep a load from more than 64 columns have a load and
//                   a run of groups per panel instead;
//   a warp          waits for the loads, and zeroes the rows of a V tile past the
//                   request's last one (they may hold anything, and 0 * NaN is not 0;
//                   what K holds there gives scores that the mask drops);
//   a warp          one elected thread issues the MMAs, per step i and lane a batch
//                   O += P(i) V(i), S(i + NB) = Q K(i + NB)^T over the S and P that
//                   the first product has read (MMAs of one thread run in the
//                   order of issue).  It is told of P and of loads by named
//                   barriers: an mbarrier's state is read behind its products that
//                   the tensor core has not taken yet, about 480 cycles.
// Batches whose requests may have two row tiles: steps of 128 keys, one S buffer
// per lane (NB = 1); while one lane's softmax works the tensor core has the other
// lane's products.  A unit with one row tile (single tokens beside a chunk) gives
// every other key tile to lane 1, and lane 0 adds both lanes up at its end.
// Batches of one row tile each: one lane, steps of 64 keys with two S buffers
// (NB = 2).  Bytes bound them, so the second product is taken twice there, of P and
// of what P's rounding left over: o's error is its own rounding's, 0.0016 to 0.0017 of
// o against float64 over 1 to 8 requests of 2 to 8 K rows.  The same requests in the
// other shape, with P alone, have 0.0017 to 0.0022, chunks up to 0.0023.  (243 instead of 242 us for the
// case below.)
//
// Tensor memory: S of lane 0 and 1 in columns [0, 128) and [128, 256), O in
// [256, 256 + D) and [384, 384 + D).  A segment that covers its unit writes o and
// lse.  Otherwise its row maxima, sums and unnormalised O go to a slot of its CTA
// (0: the unit began in an earlier CTA, 1: here), and a second kernel merges them (a
// unit's last CTA merging it in this kernel took 22 us longer for prompts, and 1 for
// a token).
//
// What bounds it, 64/8/128:
//   draft blocks of 16 requests over up to 32 K rows: the bytes, 241 us for 1.61 GB
//   (6.7 TB/s, the rate of a plain copy);
//   a 4096-token chunk over 28 K: 2.38 ms, 1.73 PFLOP/s (0.91 of cuBLAS's measured
//   rate) while the clock holds; run on end it meets the power limit, 2.76 ms (cuBLAS
//   then falls to 0.90 of its rate, too).  A step of both lanes takes 2900 cycles
//   for 2048 of products: the chain of a lane, products -> S -> softmax (1300 to
//   1500) -> P, is longer than the other lane's products hide;
//   short prompts: about 3 us for a unit's start and end, as much as 2 tiles; most of it
//   is the fetching of code that runs once a unit, which is why loops off the path of a
//   step are rolled (12 % of the code, 10 % of the time of 8 prompts: 200 us);
//   tokens beside a chunk (32 over up to 16 K rows, and 1000 tokens): 362 us, bytes and
//   products one after another, as a CTA has units of one kind at a time;
//   one token over 4 K: 13 us, the latency of two launches;
//   more than some hundred requests: also the search for the shares (cut_of), below.
// At d = 64 a step has half of those products and as much softmax: about 2300 cycles for 1024
// of products, 1.90 ms for the same chunk.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace dustin {

namespace {

constexpr int TK = kPagedTile;       // keys per tile, and query rows per row tile
constexpr int kSCol = 0, kOCol = 256;                // lane 1: + 128
constexpr int kPBar = 1, kLandedBar = 5;             // named barriers: P of [lane][buffer] is stored; loads are in
constexpr float kNaN = __builtin_nanf("");
constexpr float kFarPast = 0x1p12f;   // sum of a step's weights past which a row takes a new reference maximum

// The cost of a unit: `tile` for each key tile (two lanes' products; or one row
// tile's, whose time is its bytes'), and for its start and end `extra`.  Fitted to
// the CTAs' times over batches of prompts and of single tokens beside a chunk, with
// 64/8/128: two lanes 1.33 us a tile and 3.2 a unit, one row tile 0.97 and 1.6.  d = 64
// takes the same weights; they were not fitted there.
template <int LANES>
struct Cost {
  static constexpr int tile(bool two) { return LANES == 1 ? 1 : two ? 11 : 8; }
  static constexpr int extra(bool two) { return LANES == 1 ? 2 : two ? 27 : 13; }
  static constexpr int least = tile(LANES == 2);   // of a share, so that a CTA inside a unit has a tile
  static constexpr int snap = LANES == 1 ? 2 : 55; // a cut moves this far to the next end of a unit, to save a merge
};

// A cut of the flattened cost: at `at` of pair p of (request b, KV head g), all in
// all at `pos`.
struct Cut {
  long long pos;
  int b, g, p, at;
};
// This CTA's share: from `from` to `to`, of `total` in `ctas` shares.
struct Start {
  Cut from;
  long long to, total;
  int ctas, snap;
};

template <int D, int LANES>
struct Cfg {
  // warps behind the lanes' softmax warps
  static constexpr int land_warp = 4 * LANES, load_warp = land_warp + 1, mma_warp = land_warp + 2, load_warp2 = land_warp + 3;
  // 384 threads: 168 registers each at the launch.  256: they leave registers for a
  // CTA of the merge, which then need not be launched when this kernel's have ended.
  static constexpr int threads = 32 * (land_warp + 4);
  static constexpr int nb = LANES == 2 ? 1 : 2;      // S buffers per lane, and steps per tile
  static constexpr int step = TK / nb;               // keys per step
  static constexpr int nst = LANES == 2 ? (D == 128 ? 5 : 8) : (D == 128 ? 6 : 12);   // K or V tiles in the ring
  static constexpr uint32_t panel = TK * 128;        // 64 columns of a K, V or Q tile
  static constexpr uint32_t stage = (D / 64) * panel;
  static constexpr uint32_t ring_off = LANES * stage;   // after the query tiles
  static constexpr uint32_t bar_off = ring_off + nst * stage;
  static constexpr uint32_t misc_off = bar_off + (3 * nst + 13) * 8;   // barriers
  static constexpr uint32_t total = misc_off + 16 + sizeof(Start) + (LANES == 2 ? TK * 8 : 0) + 1024;
};

// A row whose sum of weights is 0 sees no key (its position is before the first),
// or every score that it sees is -inf, which is NaN like the 0 / 0 it stands for.
__device__ __forceinline__ float row_scale(float sum, int position) {
  return sum != 0.f ? 1.f / sum : position >= 0 ? kNaN : 0.f;   // (a NaN stays one)
}
__device__ __forceinline__ float row_lse(float top, float sum, int position) {
  return sum != 0.f ? (top + log2f(sum)) * kLn2 : position >= 0 ? kNaN : -INFINITY;
}

// a / b for a, b >= 0, where both mostly fit 32 bits.  Otherwise bit by bit, in a
// short loop: a 64-bit division's code, in all the places that divide, would push
// the rest out of the instruction cache.
__device__ __forceinline__ long long quot(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (long long)(uint32_t(a) / uint32_t(b));
  unsigned long long q = 0, r = 0;
#pragma unroll 1
  for (int x = 63; x >= 0; --x) {
    r = (r << 1) | ((unsigned long long)a >> x & 1u);
    q <<= 1;
    if (r >= (unsigned long long)b) {
      r -= b;
      q |= 1u;
    }
  }
  return (long long)q;
}

// A request: its packed rows [c0, c0 + n), cache rows, units of a KV head.
struct Request {
  int c0, n, kv, pairs;
};
template <int LANES>
__device__ __forceinline__ Request request_of(const PagedArgs& A, int b) {
  Request r;
  // (plain loads: the kernel before this one may write these while this one waits for it)
  const int c1 = A.cu[b + 1];
  r.c0 = A.cu[b];
  r.kv = A.kv_len[b];
  const bool ok = paged_ok(A, r.c0, c1, r.kv);
  r.n = ok ? c1 - r.c0 : 0;
  r.pairs = (r.n + LANES * A.nt - 1) / (LANES * A.nt);
  return r;
}
// Key tiles of the p-th unit: of the rows that its last token sees, one at least.
template <int LANES>
__device__ __forceinline__ int unit_tiles(const PagedArgs& A, const Request& r, int p) {
  const int seen = r.kv - r.n + min(r.n, (p + 1) * LANES * A.nt);
  return max(1, (seen + TK - 1) / TK);
}
template <int LANES>
__device__ __forceinline__ bool unit_two(const PagedArgs& A, const Request& r, int p) {
  return LANES == 2 && (2 * p + 1) * A.nt < r.n;
}
template <int LANES>
__device__ __forceinline__ int unit_cost(const PagedArgs& A, const Request& r, int p) {
  const bool two = unit_two<LANES>(A, r, p);
  return unit_tiles<LANES>(A, r, p) * Cost<LANES>::tile(two) + Cost<LANES>::extra(two);
}
// All units of a KV head, by one thread: few of them.
template <int LANES>
__device__ __forceinline__ long long head_cost(const PagedArgs& A, const Request& r) {
  if constexpr (LANES == 1) return r.pairs ? unit_cost<LANES>(A, r, 0) : 0;   // (max_new fits a row tile)
  long long all = 0;
#pragma unroll 1
  for (int p = 0; p < r.pairs; ++p) all += unit_cost<LANES>(A, r, p);
  return all;
}
constexpr int kFewPairs = 4;
constexpr int kZeroTiles = 4;   // key tiles of a segment from which on its unused query rows are zeroed (0.3 us)
// The same by a whole warp, of a request that all its threads have.
template <int LANES>
__device__ __forceinline__ long long head_cost_warp(const PagedArgs& A, const Request& r) {
  if (LANES == 1 || r.pairs <= kFewPairs) return head_cost<LANES>(A, r);
  long long all = 0;
#pragma unroll 1
  for (int p = threadIdx.x & 31; p < r.pairs; p += 32) all += unit_cost<LANES>(A, r, p);
#pragma unroll 1
  for (int x = 16; x; x >>= 1) all += __shfl_xor_sync(0xffffffffu, all, x);
  return all;
}

// Called by one whole warp: the cut before this CTA's share (next = 0) or after it
// (next = 1) where the batch's cost is cut into equal runs, moved to the end of a
// unit where one is near.  Each lane sums a run of neighbouring requests, those of
// many units together with the others; one scan over the lanes finds the one whose
// run holds the cut.  CTAs without a share get two equal cuts.
// All other warps wait for it.  One token over 4 K among idle requests, us by their
// number, in the shape with one lane: up to 32 12.8, 128 13.6, 512 15.5, 2048 26.8,
// 8192 69.9; with two lanes 16.3, 17.3, 20.3, 36.5, 97.9.
template <int LANES>
__device__ __forceinline__ Cut cut_of(const PagedArgs& A, int next, Start& out) {
  const int lane = threadIdx.x & 31;
  const int per = (A.B + 31) / 32, b0 = lane * per;
  long long mine = 0;
#pragma unroll 1
  for (int k = 0; k < per; ++k) {   // the lanes' k-th requests
    Request r{0, 0, 0, 0};
    if (b0 + k < A.B) r = request_of<LANES>(A, b0 + k);
    if (LANES == 1 || r.pairs <= kFewPairs) mine += head_cost<LANES>(A, r) * A.hkv;
    if constexpr (LANES == 2)
#pragma unroll 1
    for (uint32_t many = __ballot_sync(0xffffffffu, r.pairs > kFewPairs); many; many &= many - 1) {
      const int src = __ffs(many) - 1;
      const Request x{0, __shfl_sync(0xffffffffu, r.n, src), __shfl_sync(0xffffffffu, r.kv, src),
                      __shfl_sync(0xffffffffu, r.pairs, src)};
      const long long all = head_cost_warp<LANES>(A, x) * A.hkv;
      if (lane == src) mine += all;
    }
  }
  long long inc = mine;
#pragma unroll 1
  for (int x = 1; x < 32; x <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, x);
    if (lane >= x) inc += y;
  }
  const long long total = __shfl_sync(0xffffffffu, inc, 31);
  // each share holds `least` at least
  const long long runs = max(quot(total, Cost<LANES>::least), total > 0 ? 1LL : 0LL);
  const int ctas = int(runs < gridDim.x ? runs : gridDim.x), c = int(blockIdx.x) + next;
  out.total = total;
  out.ctas = ctas;
  out.snap = ctas ? int(min((long long)Cost<LANES>::snap, quot(total, 16 * ctas))) : 0;
  if (c >= ctas) return Cut{total, A.B, 0, 0, 0};
  Cut s{quot(c * total, ctas), 0, 0, 0, 0};
  // the lane whose requests hold the cut, then the request, the KV head and the unit
  const int src = __ffs(__ballot_sync(0xffffffffu, s.pos < inc)) - 1;
  long long at = s.pos - __shfl_sync(0xffffffffu, inc - mine, src), head = 0;
  Request r{};
#pragma unroll 1
  for (s.b = src * per;; ++s.b) {
    r = request_of<LANES>(A, s.b);
    head = head_cost_warp<LANES>(A, r);
    if (at < head * A.hkv || s.b + 1 == A.B) break;
    at -= head * A.hkv;
  }
  s.g = int(quot(at, head));
  at -= s.g * head;
  int cost = 0;
  if constexpr (LANES == 1) {
    cost = int(head);
    s.at = int(at);
  }
#pragma unroll 1
  for (; LANES == 2 && s.p < r.pairs; s.p += 32) {
    const int p = s.p + lane;
    cost = p < r.pairs ? unit_cost<LANES>(A, r, p) : 0;
    int upto = cost;
#pragma unroll 1
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, x);
      if (lane >= x) upto += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, at < upto);
    if (past) {
      const int src = __ffs(past) - 1;
      s.p += src;
      s.at = int(at - __shfl_sync(0xffffffffu, upto - cost, src));
      cost = __shfl_sync(0xffffffffu, cost, src);
      break;
    }
    at -= __shfl_sync(0xffffffffu, upto, 31);
  }
  if (s.at <= out.snap) {
    s.pos -= s.at;
    s.at = 0;
  } else if (cost - s.at <= out.snap) {   // the next unit's start
    s.pos += cost - s.at;
    s.at = 0;
    if (++s.p == r.pairs) {
      s.p = 0;
      if (++s.g == A.hkv) {
        s.g = 0;
#pragma unroll 1
        do ++s.b;
        while (s.b < A.B && request_of<LANES>(A, s.b).n == 0);
      }
    }
  }
  return s;
}

// 32 bytes to global memory in one instruction: a thread stores to a row of its own,
// so that each store is a sector, and half as many pass the load-store unit.
__device__ __forceinline__ void store32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// (a, b) * (s, s)
__device__ __forceinline__ void mul2(float& a, float& b, float s) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %2};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "+f"(a), "+f"(b)
      : "f"(s));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  asm("max.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(b), "f"(c));
  return a;
}

// mbar_wait that gives up at once where another wait of the CTA has: the softmax
// warps and the landing warp then run on without data (the call is flagged), so that
// the named barriers, which know no limit, are all met.
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, int* err, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  return !*abort && mbar_wait(bar, parity, err, abort);
}
__device__ __forceinline__ void named_arrive(int id, int threads) {
  asm volatile("barrier.cta.arrive.aligned %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Groups of 8 rows (all columns, or 64) of a page: coordinates (x, row 0 of a
// group, c2, c3, page).
template <bool ONCE>   // rows that nobody else reads: they leave L2 first
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int x, int c2, int c3, int page,
                                            uint64_t* bar, uint64_t policy) {
  if constexpr (ONCE)
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(0), "r"(c2), "r"(c3), "r"(page), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(0), "r"(c2), "r"(c3), "r"(page), "r"(smem_u32(bar))
        : "memory");
}


// Walks this CTA's segments: key tiles [i0, i0 + n) of unit (b, g, p).
template <int LANES>
struct Walk {
  long long left;   // cost from this segment's on
  int b, g, p, at, i0, n, tiles, used;
  bool two;         // the unit has a second row tile
  Request r;
  // The segment from cost `at` of the unit on.  The extra cost comes first; a
  // tile belongs to the share that its cost ends in.  A segment without a tile can
  // only be a share's last, as a share is no less than a tile.
  __device__ __forceinline__ void cut(const PagedArgs& A, int from) {
    at = from;
    two = unit_two<LANES>(A, r, p);
    tiles = unit_tiles<LANES>(A, r, p);
    const int extra = Cost<LANES>::extra(two), tile = Cost<LANES>::tile(two), all = tiles * tile + extra - at;
    used = int(left < all ? left : all);
    i0 = max(0, at - extra) / tile;
    n = max(0, at + used - extra) / tile - i0;
    if (n == 0) left = 0;
  }
  __device__ __forceinline__ void init(const PagedArgs& A, const Start& s) {
    left = s.to - s.from.pos;
    b = s.from.b;
    g = s.from.g;
    p = s.from.p;
    if (left <= 0) return;
    r = request_of<LANES>(A, b);
    cut(A, s.from.at);
  }
  __device__ __forceinline__ void next(const PagedArgs& A) {
    left -= used;
    if (left <= 0) return;
    if (++p == r.pairs) {
      p = 0;
      if (++g == A.hkv) {
        g = 0;
        do r = request_of<LANES>(A, ++b);
        while (r.n == 0 && b + 1 < A.B);
      }
    }
    cut(A, 0);
  }
  // the unit's first token within the request
  __device__ __forceinline__ int first(const PagedArgs& A) const { return p * LANES * A.nt; }
};

template <int D, int LANES>
__global__ void __launch_bounds__(Cfg<D, LANES>::threads, 1) paged_kernel(const __grid_constant__ PagedArgs A) {
  using C = Cfg<D, LANES>;
  constexpr int NST = C::nst, NB = C::nb, SK = C::step;
  constexpr bool LOW = LANES == 1;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::bar_off);
  uint64_t* empty = full + NST;
  uint64_t* q_full = empty + NST;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;      // [lane][buffer] a batch with an S is done
  uint64_t* o_full = s_full + 4;       // [lane][z] the z-th of a segment's last NB batches, without an S, is done
  uint64_t* mma_done = o_full + 4;
  uint64_t* pair_full = mma_done + 1;  // lane 1's part of a unit with one row tile is complete
  uint64_t* pair_empty = pair_full + 1;   // and has been read
  uint64_t* landed = pair_empty + 1;   // [stage] the rows of a V tile that ends past the request are in
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::misc_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::misc_off + 8);
  Start* start = reinterpret_cast<Start*>(smem + C::misc_off + 16);
  float2* pair_ml = reinterpret_cast<float2*>(smem + C::misc_off + 16 + sizeof(Start));   // lane 1's maxima and sums
  static_assert(C::misc_off % 8 == 0 && sizeof(Start) % 8 == 0, "alignment of the shared-memory tail");

  const int tid = threadIdx.x, warp = tid >> 5, lane_id = tid & 31;
  const int G = A.hq / A.hkv;
  const int n_act = (A.qt * G + 31) >> 5;   // softmax warps per lane that hold rows
  if (tid == 32) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);   // the products that read the stage, and the second loading warp
      mbar_init(&landed[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int x = 0; x < 4; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&o_full[x], 1);
    }
    mbar_init(mma_done, 1);
    mbar_init(pair_full, 32 * n_act);
    mbar_init(pair_empty, 32 * n_act);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (tid == 64) {
    prefetch_tensormap(&A.qmap);
    prefetch_tensormap(&A.kmap);
    prefetch_tensormap(&A.vmap);
  }
  // Query rows that no load writes are zeros: the tensor core takes less power for
  // them, and under the power limit that is time.
  for (int x = A.qt * G * 8 + tid; x < TK * 8; x += C::threads)
    for (int h = 0; h < LANES * (D / 64); ++h)
      *reinterpret_cast<uint4*>(smem + uint32_t(h) * C::panel + x * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
  if (warp == C::mma_warp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "n"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_launch_dependents();
  pdl_wait();
  if (warp < 2) {   // the share's start and its end
    Start s;
    const Cut cut = cut_of<LANES>(A, warp, s);
    if (lane_id == 0) {
      if (warp == 0) {
        start->from = cut;
        start->total = s.total;
        start->ctas = s.ctas;
        start->snap = s.snap;
      } else {
        start->to = cut.pos;
      }
    }
  } else if (warp == 2 && blockIdx.x == 0) {
    for (int b = lane_id; b < A.B; b += 32)
      if (!paged_ok(A, A.cu[b], A.cu[b + 1], A.kv_len[b])) flag_error(A.err, DUSTIN_DEV_SEQLEN);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk<LANES> w;
  if (warp < 4 * LANES) {
    // =============================================================== softmax
    // a softmax thread holds a row's scores: 200 x 256 + 96 x 128 of the 168 x 384
    // registers of the launch (LANES = 1 needs no more than these)
    if constexpr (LANES == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    w.init(A, *start);
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
        wait_on(bar, parity, A.err, abort_flag);
        __syncwarp();
      };
      auto wait_s = [&](int J) { wait_warp(&s_full[2 * ln + J % NB], uint32_t(J / NB) & 1u); };
      int j0 = 0, segs = 0;   // steps and segments of the lane before this segment
      auto wait_o = [&](int z) { wait_warp(&o_full[2 * ln + z], uint32_t(segs) & 1u); };
      int4 split = make_int4(0, 0, 0, -1);   // the unit that this CTA starts and does not end, and the last CTA of it
      Request whose{0, 0, 0, 0};
      uint32_t pairs = 0;     // phase of pair_full and pair_empty
      for (; w.left > 0; w.next(A)) {
        // a unit with one row tile gives its odd tiles to lane 1
        const bool halves = LANES == 2 && !w.two;
        if (halves && ln == 1 && w.n == 1) continue;
        const int tok = w.first(A) + (halves ? 0 : ln * A.nt) + row / G;   // within the request
        const bool act = row < A.qt * G && tok < w.r.n;
        const int position = w.r.kv - w.r.n + tok;
        const int n = halves ? (w.n + 1 - ln) / 2 : NB * w.n;              // steps
        const int key0 = NB * w.i0 + (halves ? ln : 0), keyd = halves ? 2 : 1;
        float mref = -INFINITY, lsum = 0.f;
        for (int i = 0; i < n; ++i) {
          const int nv = position + 1 - (key0 + i * keyd) * SK;      // keys of this step that the row sees, if under SK
          const uint32_t sb = s_tmem + uint32_t((j0 + i) % NB * SK);
          wait_s(j0 + i);
          tc_fence_after();
          float alpha = 1.f, step = 0.f;
          uint32_t pk[SK / 2], lo[LOW ? SK / 2 : 1];
          // P of this step against the reference maximum.  Rows with `mine` take the
          // step's maximum first: those that have none yet, and, the second time, those
          // whose weights came out too large for the one they have (sums and O are fp32
          // and the rounding of P is relative, so until then it needs no change).
          bool mine = act && mref == -INFINITY;
#pragma unroll 1
          for (int time = 0;; ++time) {
            float x[SK];
#pragma unroll
            for (int c = 0; c < SK; c += 64) tc_ld64(sb + uint32_t(c), reinterpret_cast<uint32_t*>(x + c));
            if (nv < SK) {
#pragma unroll
              for (int j = 0; j < SK; ++j) x[j] = j < nv ? x[j] : -INFINITY;
            }
            if (__any_sync(0xffffffffu, mine)) {
              float m4[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) m4[y] = fmaxf(x[2 * y], x[2 * y + 1]);
#pragma unroll
              for (int j = 8; j < SK; j += 8)
#pragma unroll
                for (int y = 0; y < 4; ++y) m4[y] = max3(m4[y], x[j + 2 * y], x[j + 2 * y + 1]);
              const float mx = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]) * scale;
              if (mine && mx > mref) {
                alpha = fast_exp2(mref - mx);   // 0 while mref is -inf
                mref = mx;
              }
            }
            // (the weights of a row that is not in use are 0, which costs the product less power)
            const float nb = !act ? -INFINITY : mref == -INFINITY ? 0.f : -mref;
            float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
            for (int j = 0; j < SK; j += 4) {
              float* y = x + j;
              fma2(y[0], y[1], scale, nb);
              fma2(y[2], y[3], scale, nb);
              const float p0 = fast_exp2(y[0]), p1 = fast_exp2(y[1]), p2 = fast_exp2(y[2]), p3 = fast_exp2(y[3]);
              add2(l0, l1, p0, p1);
              add2(l2, l3, p2, p3);
              pk[j / 2] = pack_bf16(p0, p1);
              pk[j / 2 + 1] = pack_bf16(p2, p3);
              if constexpr (LOW) {
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  float r0 = z ? p2 : p0, r1 = z ? p3 : p1;
                  const uint32_t h = pk[j / 2 + z];
                  add2(r0, r1, -__uint_as_float(h << 16), -__uint_as_float(h & 0xFFFF0000u));
                  lo[j / 2 + z] = pack_bf16(r0, r1);
                }
              }
            }
            step = (l0 + l1) + (l2 + l3);
            mine = act && !mine && !(step <= kFarPast);
            if (time > 0 || !__any_sync(0xffffffffu, mine)) break;
          }
          // rescale this row of O once P V of the step before is in (NB = 1: it
          // came with S of this step; NB = 2: it comes with S of the next one, or
          // alone after the last)
          if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            if (NB > 1) {
              if (i + 1 < n) wait_s(j0 + i + 1);
              else wait_o(0);
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
#pragma unroll
          for (int h = 0; h < SK / 32; ++h) {
            tc_st16(sb + uint32_t(16 * h), pk + 16 * h);
            if constexpr (LOW) tc_st16(sb + uint32_t(SK / 2 + 16 * h), lo + 16 * h);
          }
          tc_wait_st();
          lsum = fmaf(lsum, alpha, step);
          tc_fence_before();
          named_arrive(kPBar + 2 * ln + (j0 + i) % NB, 32 * n_act + 32);
        }
        // --------------------------------------------------------- epilogue
#pragma unroll
        for (int z = 0; z < NB; ++z) wait_o(z);
        j0 += n;
        ++segs;
        tc_fence_after();
        // lane 1's part of a unit with one row tile goes into lane 0's (the two
        // lanes' warps of a row reach the same tensor-memory lanes)
        const bool join = halves && w.n > 1;
        float w0 = 1.f, w1 = 0.f;
        if (join) {
          if (ln == 1) {
            pair_ml[row] = make_float2(mref, lsum);
            tc_fence_before();
            mbar_arrive(pair_full);
            wait_warp(pair_empty, pairs);
            pairs ^= 1u;
            tc_fence_after();
            continue;
          }
          wait_warp(pair_full, pairs);
          pairs ^= 1u;
          tc_fence_after();
          const float2 ml = pair_ml[row];
          const float ref = fmaxf(mref, ml.x), base = ref == -INFINITY ? 0.f : ref;
          w0 = fast_exp2(mref - base);
          w1 = fast_exp2(ml.x - base);
          lsum = fmaf(lsum, w0, ml.y * w1);
          mref = ref;
        }
        const bool whole = w.n == w.tiles;
        // (tid 0: lane 0 has a row tile in every unit)
        if (tid == 0 && !whole && w.i0 == 0) {
          // the CTA that the unit's cost ends in
          const long long end = start->to - w.used + unit_cost<LANES>(A, w.r, w.p) - w.at;
          int last = int(quot(end * start->ctas - 1, start->total));
          if (end - quot(last * start->total, start->ctas) <= start->snap) --last;   // (its share was moved past the unit)
          split = make_int4(w.r.c0, w.g, w.p, last);
          whose = w.r;
        }
        float* part = A.partial + ((size_t(blockIdx.x) * 2 + (w.i0 == 0)) * LANES + ln) * (size_t(TK) * (D + 2));
        const size_t orow = size_t(w.r.c0 + (act ? tok : 0)) * A.hq + size_t(w.g) * G + row % G;
        const float inv = row_scale(lsum, position);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tc_ld32(o_tmem + uint32_t(c), o);   // collective: every lane loads
          if (join) {
            uint32_t o1[32];
            tc_ld32(o_tmem + uint32_t(128 + c), o1);
#pragma unroll
            for (int y = 0; y < 32; ++y)
              o[y] = __float_as_uint(fmaf(__uint_as_float(o[y]), w0, __uint_as_float(o1[y]) * w1));
          }
          if (act && whole) {
#pragma unroll
            for (int y = 0; y < 16; ++y) {
              float2 p = make_float2(__uint_as_float(o[2 * y]), __uint_as_float(o[2 * y + 1]));
              mul2(p.x, p.y, inv);
              o[y] = pack_bf16(p.x, p.y);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) store32(A.o + orow * D + c + 16 * y, o + 8 * y);
          } else if (act) {
#pragma unroll
            for (int y = 0; y < 4; ++y) store32(part + size_t(row) * D + c + 8 * y, o + 8 * y);
          }
        }
        if (join) {
          tc_fence_before();
          mbar_arrive(pair_empty);
        }
        if (act) {
          if (whole) {
            if (A.lse) A.lse[orow] = row_lse(mref, lsum, position);
          } else {
            part[size_t(TK) * D + row] = mref;
            part[size_t(TK) * D + TK + row] = lsum;
          }
        }
        tc_fence_before();
      }
      if (tid == 0) {
        A.split[2 * blockIdx.x] = split;
        A.split[2 * blockIdx.x + 1] = make_int4(whose.n, whose.kv, 0, 0);
      }
    }
  } else {
    if constexpr (LANES == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    w.init(A, *start);
    if (warp == C::load_warp || warp == C::load_warp2) {
      // ================================================================ loads
      // Both warps follow every phase of `empty`; the first alone arms the stages.
      // No wait by parity can be lapped or pass early: the phase after the one
      // that a warp waits for needs that warp past the wait, the first because it arms
      // the stage's next load, the second because it arrives at `empty` itself.  (The
      // load that it may have in that stage does not do: with pages of a tile or more it
      // has none in the whole call, and else none in a tile of one page.)
      const bool lead = warp == C::load_warp;
      // rows that one unit alone reads leave L2 first (64 requests of 512 to 1024 rows 46.0 -> 43.8 us;
      // for the units of one row tile beside a chunk it was worse, 430 -> 449)
      const uint64_t policy = LANES == 1 ? policy_evict_first() : 0;
      const int box = min(A.page, TK);                  // rows of a load
      const int per_tile = TK / box, tiles = A.page / box;   // pages of a tile, and tiles of a page (one of them is 1)
      // every other page by each warp, or a panel of each page
      const bool panels = D == 128 && !A.merged;
      const int h = lead ? 0 : 1, own_x = panels ? h * 64 : 0;
      const bool own = panels || (lane_id & 1) == h;
      const uint32_t own_off = panels ? uint32_t(lane_id * box * 128 + h * int(C::panel)) : uint32_t(lane_id * box * D * 2);
      int gi = 0, st = 0, segs = 0;
      uint32_t ph = 0;                                  // of stage st
      uint32_t tails = 0, tail_ph = 0;                  // stages whose latest load is waited for by `landed`; its phases
      bool live = true;
      auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
        return bool(__all_sync(0xffffffffu, wait_on(bar, parity, A.err, abort_flag)));
      };
      for (; live && w.left > 0; w.next(A)) {
        // this thread's entry of the table for a tile, read a tile ahead of its use
        auto needs = [&](int i) { return i < w.n && lane_id < per_tile && (w.i0 + i) * TK + lane_id * box < w.r.kv; };
        const int32_t* entry = A.table + size_t(w.b) * A.max_pages + w.i0 / tiles * per_tile + lane_id;
        int row = w.i0 % tiles;                           // the tile within its page
        int ahead = needs(0) ? *entry : 0;
        // this segment's query tiles, once the last one's S MMAs have read theirs
        if (lead) {
          if (segs > 0 && !wait_warp(q_empty, uint32_t(segs - 1) & 1u)) break;
          if (lane_id == 0) {
            const bool two = w.two;
            const uint32_t bytes = uint32_t(A.qt * G) * D * 2;
            mbar_arrive_expect_tx(q_full, two ? 2 * bytes : bytes);
            for (int ln = 0; ln < (two ? 2 : 1); ++ln)
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                tma_load_3d(sbase + uint32_t(ln) * C::stage + uint32_t(h) * C::panel, &A.qmap, h * 64, w.g * G,
                            w.r.c0 + w.first(A) + ln * A.nt, q_full);
          }
          ++segs;
        }
        // K(0), then K(i), V(i - 1) for each tile, V(n - 1): the order of their use
        int id = -1, at = 0;
        for (int i = 0; live && i <= w.n; ++i) {
          const int before = id, row_before = at;
          id = -1;
          at = row;
          if (needs(i)) {
            id = ahead;
            if (id < 0 || id >= A.n_pages) {
              flag_error(A.err, DUSTIN_DEV_INDEX);
              id = A.n_pages;   // past the end: the load fills in zeros
            }
          }
          if (++row == tiles) {
            row = 0;
            entry += per_tile;
          }
          ahead = needs(i + 1) ? *entry : 0;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            if (kv ? i == 0 : i == w.n) continue;
            const int base = (w.i0 + i - kv) * TK, page = kv ? before : id;
            if (gi >= NST && !wait_warp(&empty[st], ph ^ 1u)) {
              live = false;
              break;
            }
            const int np = __popc(__ballot_sync(0xffffffffu, page >= 0));   // pages of the tile
            const int r8 = (kv ? row_before : at) * (TK / 8);   // groups of 8 rows before it
            const bool tail = kv && base + TK > w.r.kv;
            uint64_t* bar = tail ? &landed[st] : &full[st];
            if (lead && lane_id == 0) mbar_arrive_expect_tx(bar, uint32_t(np * box) * D * 2);
            __syncwarp();
            const uint32_t dst = sbase + C::ring_off + uint32_t(st) * C::stage;
            const CUtensorMap* map = kv ? &A.vmap : &A.kmap;
            const int c2 = A.merged ? w.g * A.map_panels : r8, c3 = A.merged ? w.g * A.map_groups + r8 : w.g;
            if (page >= 0 && own) tma_load_5d<LANES == 1>(dst + own_off, map, own_x, c2, c3, page, bar, policy);
            if (!lead && lane_id == 0) mbar_arrive(&empty[st]);   // (all lanes have passed the wait above)
            if (tail) tail_ph ^= 1u << st;
            tails = tail ? tails | 1u << st : tails & ~(1u << st);
            ++gi;
            if (++st == NST) {
              st = 0;
              ph ^= 1u;
            }
          }
        }
      }
      // what is in flight has landed before the CTA may exit: the query tiles
      // and the latest load of each stage
      if (lead && lane_id == 0) {
        if (segs > 0) mbar_drain(q_full, uint32_t(segs - 1) & 1u, A.err);
        for (int j = gi > NST ? gi - NST : 0; j < gi; ++j) {
          const int x = j % NST;
          if ((tails >> x) & 1u) mbar_drain(&landed[x], ((tail_ph >> x) & 1u) ^ 1u, A.err);
          else mbar_drain(&full[x], uint32_t(j / NST) & 1u, A.err);
        }
      }
      __syncwarp();
    } else if (warp == C::land_warp) {
      // ============================================================ landings
      // waits for what the products read and lets the MMA warp go on by a named barrier:
      // a wait on an mbarrier by that warp would stand behind its queued products
      int st = 0, segs = 0;
      uint32_t ph = 0, tail_ph = 0;   // phases of stage st, and of `landed`
      auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
        wait_on(bar, parity, A.err, abort_flag);
        __syncwarp();
      };
      for (; w.left > 0; w.next(A)) {
        wait_warp(q_full, uint32_t(segs++) & 1u);
        if (LANES == 2 && !w.two && w.n >= kZeroTiles) {   // rows of other requests' tokens, as above
          for (int x = (w.r.n - w.first(A)) * G * 8 + lane_id; x < TK * 8; x += 32)
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              *reinterpret_cast<uint4*>(smem + uint32_t(h) * C::panel + x * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async();
          __syncwarp();
        }
        const int nv = max(w.r.kv - (w.i0 + w.n - 1) * TK, 0);   // rows of the segment's last tile
        const bool halves = LANES == 2 && !w.two;
        // K(0), then K(i), V(i - 1) for each tile, V(n - 1)
#pragma unroll 1
        for (int t = 0; t < 2 * w.n; ++t) {
          const bool is_v = t == 2 * w.n - 1 || (t > 0 && !(t & 1));
          if (t == 2 * w.n - 1 && nv < TK) {
            wait_warp(&landed[st], (tail_ph >> st) & 1u);
            tail_ph ^= 1u << st;
            unsigned char* rows = smem + C::ring_off + uint32_t(st) * C::stage;
            const uint32_t panel = A.merged ? 1024 : C::panel, group = A.merged ? (D / 64) * 1024 : 1024;
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              for (int x = nv * 8 + lane_id; x < TK * 8; x += 32)   // 16 bytes each, 64 of them a group
                *reinterpret_cast<uint4*>(rows + h * panel + (x >> 6) * group + (x & 63) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async();
            __syncwarp();
            if (lane_id == 0) mbar_arrive(&full[st]);   // every load is a phase of `full`
          } else {
            wait_warp(&full[st], ph);
          }
          // a batch takes K(i + 1) and V(i), or, where the lanes share the tiles, V(i) and K(i + 2)
          if (t == 0 || (halves ? !is_v || t >= 2 * w.n - 2 : is_v)) named_sync(kLandedBar, 64);
          if (++st == NST) {
            st = 0;
            ph ^= 1u;
          }
        }
      }
      __syncwarp();
    } else {
      if (warp == C::mma_warp) {
        // ================================================================ MMAs
        constexpr uint32_t kIdS = tc_idesc(128, SK, 0), kIdPV = tc_idesc(128, D, 1);
        const uint64_t q_desc = tc_desc(sbase, 16, 1024);
        const uint32_t panel = A.merged ? 1024 : C::panel, group = A.merged ? (D / 64) * 1024 : 1024;
        const uint64_t k_desc = tc_desc(sbase + C::ring_off, 16, group), v_desc = tc_desc(sbase + C::ring_off, panel, group);
        const uint32_t kpanel = panel >> 4, keys16 = group >> 3;   // per panel, and per 16 keys
        int st = 0;                           // ring stage to consume next
        bool issued = false;
        // the warp runs together and one elected lane issues; branches go by votes,
        // so that the compiler too knows the warp as converged
        auto uni = [](bool x) { return __any_sync(0xffffffffu, x) != 0; };
        auto take = [&](int& stage) {
          stage = st;
          st = st + 1 == NST ? 0 : st + 1;
        };
        // One segment.  HALVES: its unit has one row tile, whose odd tiles are lane 1's.
        auto segment = [&](auto halves, bool two) {
          constexpr bool HALVES = decltype(halves)::value;
          constexpr int kUnroll = LANES == 2 ? 4 : 8;   // of S's products (8: prompts 205 instead of 199 us)
          constexpr int lead = HALVES ? 2 : NB;   // steps that S runs ahead of P V
          const int n = NB * w.n;                 // steps (of both lanes together where they share the tiles)
          int sv = 0, sk = 0;                     // stages of V and of K
          for (int i = -lead; uni(i < n); ++i) {
            const bool first = NB == 1 || !(i & 1), last = NB == 1 || (i & 1);   // step of its tiles
            const bool pv = i >= 0, s = uni(i + lead < n);
            // tiles come as K(0), K(1), V(0), K(2), V(1), ...
            if ((pv || s) && first) named_sync(kLandedBar, 64);
            if (HALVES && pv) take(sv);
            if (s && first) take(sk);
            if (!HALVES && pv && first) take(sv);
            auto batch = [&](int ln, int buf) {
              if (pv) named_sync(kPBar + 2 * ln + buf, 32 * n_act + 32);
              issued = true;
              tc_fence_after();
              const uint32_t sp = tmem + uint32_t(kSCol + 128 * ln + buf * SK);
              if (pv) {
                const uint64_t v = v_desc + uint64_t(sv) * (C::stage >> 4) + (first ? 0u : keys16 * (SK / 16));
                const bool acc = i >= (HALVES ? 2 : 1);   // not the lane's first step
#pragma unroll
                for (int kk = 0; kk < SK / 16; ++kk)
                  tc_mma_ts_elect(tmem + uint32_t(kOCol + 128 * ln), sp + uint32_t(kk * 8), v + uint32_t(kk) * keys16, kIdPV,
                                  (acc || kk > 0) ? 1 : 0);
                if constexpr (LOW)   // what the rounding of P left over
#pragma unroll
                  for (int kk = 0; kk < SK / 16; ++kk)
                    tc_mma_ts_elect(tmem + uint32_t(kOCol + 128 * ln), sp + uint32_t(SK / 2 + kk * 8),
                                    v + uint32_t(kk) * keys16, kIdPV, 1);
              }
              if (s) {
                const uint64_t q = q_desc + uint64_t(HALVES ? 0 : ln) * (C::stage >> 4);
                const uint64_t k = k_desc + uint64_t(sk) * (C::stage >> 4) + (first ? 0u : keys16 * (SK / 16));
#pragma unroll kUnroll
                for (int kk = 0; kk < D / 16; ++kk)
                  tc_mma_ss_elect(sp, q + uint32_t(kk >> 2) * (C::panel >> 4) + uint32_t((kk & 3) * 2),
                                  k + uint32_t(kk >> 2) * kpanel + uint32_t((kk & 3) * 2), kIdS, kk > 0);
              }
              tc_commit_elect(s ? &s_full[2 * ln + buf] : &o_full[2 * ln + buf]);   // (n is even where NB = 2)
            };
            if constexpr (HALVES) {
              if (pv || s) batch(i & 1, 0);
            } else if constexpr (LANES == 2) {
              batch(0, 0);
              if (two) batch(1, 0);
            } else {
              batch(0, i & 1);   // (step i and step i + NB have one buffer)
            }
            if (pv && last) tc_commit_elect(&empty[sv]);
            if (s && last) tc_commit_elect(&empty[sk]);
            if (uni(i + lead + 1 == n)) tc_commit_elect(q_empty);   // the query tiles are no longer read
          }
        };
        for (; uni(w.left > 0); w.next(A)) {
          const bool two = uni(w.two);
          if constexpr (LANES == 2) {
            if (two) segment(std::false_type{}, true);
            else segment(std::true_type{}, false);
          } else {
            segment(std::false_type{}, false);
          }
        }
        if (issued) {   // every MMA has completed before tensor memory is freed
          tc_commit_elect(mma_done);
          if (lane_id == 0) mbar_drain(mma_done, 0, A.err);
        }
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::mma_warp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
}

// Log-sum-exp merge of the segments of the unit that CTA blockIdx.x started and did
// not end: one thread per four output columns of M::rows rows.  The depth of the loads
// goes by batches of many units where there are two lanes, whose units are cut in two
// or three; the few units of a short chunk over a long context are cut among as many
// CTAs as single tokens' are (32 tokens over 32 K rows, 64/8/128: 8 units, 19 segments
// each; the whole call 46.4 us for 20.0 of bytes).
constexpr int kMergeThreads = 256;
template <int D, int LANES>
struct Merge {
  static constexpr int rows = LANES;                       // rows of a thread
  static constexpr int depth = LANES == 1 ? 10 : 3;        // segments whose loads are in flight
  static constexpr int step = kMergeThreads / (D / 4);     // rows at a time
  static constexpr int block = rows * step;                // rows of a block
};

template <int D, int LANES>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const __grid_constant__ PagedArgs A) {
  using M = Merge<D, LANES>;
  pdl_launch_dependents();
  pdl_wait();
  const int4 sp = __ldcg(A.split + 2 * blockIdx.x), of = __ldcg(A.split + 2 * blockIdx.x + 1);
  const int c0 = blockIdx.x, c1 = min(sp.w, int(gridDim.x) - 1);
  if (c1 <= c0) return;
  const int G = A.hq / A.hkv, c4 = threadIdx.x % (D / 4);
  const Request r{sp.x, of.x, of.y, 0};
  constexpr size_t kLane = size_t(TK) * (D + 2);
  int tok[M::rows], row[M::rows];
  bool act[M::rows];
  const float* base_o[M::rows];
  const float* base_m[M::rows];
  float top[M::rows], sum[M::rows];
  float4 acc[M::rows];
#pragma unroll
  for (int z = 0; z < M::rows; ++z) {
    const int x = blockIdx.y * M::block + z * M::step + threadIdx.x / (D / 4), ln = x / TK;
    row[z] = x % TK;
    tok[z] = (sp.z * LANES + ln) * A.nt + row[z] / G;
    act[z] = row[z] < A.qt * G && tok[z] < r.n;
    base_o[z] = A.partial + ln * kLane + size_t(row[z]) * D + 4 * c4;
    base_m[z] = A.partial + ln * kLane + size_t(TK) * D + row[z];
    top[z] = -INFINITY;
    sum[z] = 0.f;
    acc[z] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int c = c0; c <= c1; c += M::depth) {
    float m[M::rows][M::depth], l[M::rows][M::depth];
    float4 o[M::rows][M::depth];
#pragma unroll
    for (int y = 0; y < M::depth; ++y)
#pragma unroll
      for (int z = 0; z < M::rows; ++z) {
        m[z][y] = -INFINITY;
        l[z][y] = 0.f;
        o[z][y] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (act[z] && c + y <= c1) {
          const size_t off = (size_t(c + y) * 2 + (c + y == c0)) * LANES * kLane;
          m[z][y] = __ldcg(base_m[z] + off);
          l[z][y] = __ldcg(base_m[z] + off + TK);
          o[z][y] = __ldcg(reinterpret_cast<const float4*>(base_o[z] + off));
        }
      }
#pragma unroll
    for (int z = 0; z < M::rows; ++z) {
      float ref = top[z];
#pragma unroll
      for (int y = 0; y < M::depth; ++y) ref = fmaxf(ref, m[z][y]);
      const float base = ref == -INFINITY ? 0.f : ref;
      const float w0 = fast_exp2(top[z] - base);   // 2^-inf = 0
      top[z] = ref;
      sum[z] *= w0;
      acc[z] = make_float4(acc[z].x * w0, acc[z].y * w0, acc[z].z * w0, acc[z].w * w0);
#pragma unroll
      for (int y = 0; y < M::depth; ++y) {
        const float w = fast_exp2(m[z][y] - base);
        sum[z] = fmaf(l[z][y], w, sum[z]);
        acc[z].x = fmaf(o[z][y].x, w, acc[z].x);
        acc[z].y = fmaf(o[z][y].y, w, acc[z].y);
        acc[z].z = fmaf(o[z][y].z, w, acc[z].z);
        acc[z].w = fmaf(o[z][y].w, w, acc[z].w);
      }
    }
  }
#pragma unroll
  for (int z = 0; z < M::rows; ++z) {
    if (!act[z]) continue;
    const size_t orow = size_t(r.c0 + tok[z]) * A.hq + size_t(sp.y) * G + row[z] % G;
    const int position = r.kv - r.n + tok[z];
    const float inv = row_scale(sum[z], position);
    reinterpret_cast<uint2*>(A.o + orow * D)[c4] = make_uint2(pack_bf16(acc[z].x * inv, acc[z].y * inv),
                                                              pack_bf16(acc[z].z * inv, acc[z].w * inv));
    if (A.lse && c4 == 0) A.lse[orow] = row_lse(top[z], sum[z], position);
  }
}

template <int D, int LANES>
cudaError_t launch_t(const PagedArgs& a, int num_sms, cudaStream_t stream) {
  using C = Cfg<D, LANES>;
  static_assert(C::total <= 227 * 1024, "shared memory of a CTA");
  auto kern = paged_kernel<D, LANES>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t attr = once_per_device(
      done, [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::total)); });
  if (attr != cudaSuccess) return attr;
  const int grid = num_sms < kPagedGridMax ? num_sms : kPagedGridMax;
  const cudaError_t e = launch_pdl(kern, dim3(grid), dim3(C::threads), C::total, stream, a);
  if (e != cudaSuccess) return e;
  constexpr int block = Merge<D, LANES>::block;
  const int rows = LANES == 2 ? 2 * TK : a.qt * (a.hq / a.hkv);
  return launch_pdl(paged_merge_kernel<D, LANES>, dim3(grid, (rows + block - 1) / block), dim3(kMergeThreads), 0, stream, a);
}

}  // namespace

cudaError_t paged_launch(PagedArgs& a, int D, int num_sms, cudaStream_t stream) {
  if (paged_lanes(a.hq, a.hkv, a.max_new) == 1)
    return D == 128 ? launch_t<128, 1>(a, num_sms, stream) : launch_t<64, 1>(a, num_sms, stream);
  return D == 128 ? launch_t<128, 2>(a, num_sms, stream) : launch_t<64, 2>(a, num_sms, stream);
}

}  // namespace dustin
