// Equal shares of a batch's tiles when only the device knows how many tiles
// each sequence has.
#pragma once

#include "common.cuh"

namespace dustin {

// A CTA's run of flattened tiles: `count` tiles from tile `offset` of sequence
// `b` on.
struct Share {
  long long count, offset;
  int b;
};

// Called by one whole warp.  tiles(b): the tiles of sequence b (all its units
// together).  Each lane sums a run of neighbouring sequences, one scan over the
// lanes finds the one whose run holds this CTA's first tile, and that lane looks
// it up.  The batch is cut into min(CTAs, tiles) equal runs, so that every run
// holds a tile and a unit's runs lie in consecutive CTAs; later CTAs get
// count = 0.
template <typename Tiles>
__device__ __forceinline__ Share share_of(int B, Tiles tiles) {
  const int lane = threadIdx.x & 31;
  const int per = (B + 31) / 32, b0 = lane * per, b1 = min(b0 + per, B);
  long long mine = 0;
#pragma unroll 4
  for (int b = b0; b < b1; ++b) mine += tiles(b);
  long long inc = mine;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, x);
    if (lane >= x) inc += y;
  }
  const long long total = __shfl_sync(0xffffffffu, inc, 31);
  const long long ctas = total < gridDim.x ? total : gridDim.x;
  Share s{0, 0, 0};
  if (blockIdx.x >= ctas) return s;
  const long long t0 = blockIdx.x * total / ctas;
  s.count = (blockIdx.x + 1) * total / ctas - t0;
  const bool here = t0 < inc && t0 >= inc - mine;
  if (here) {
    s.b = b0;
    s.offset = t0 - (inc - mine);
    for (int n; s.offset >= (n = tiles(s.b)); ++s.b) s.offset -= n;
  }
  const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  s.b = __shfl_sync(0xffffffffu, s.b, src);
  s.offset = __shfl_sync(0xffffffffu, s.offset, src);
  return s;
}

}  // namespace dustin
