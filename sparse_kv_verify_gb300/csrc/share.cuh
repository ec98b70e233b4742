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
// together, up to 2^31 / 32).  The batch is summed 32 sequences at a time and
// cut into min(CTAs, tiles) equal runs, so that every run holds a tile and a
// unit's runs lie in consecutive CTAs; later CTAs get count = 0.
template <typename Tiles>
__device__ __forceinline__ Share share_of(int B, Tiles tiles) {
  const int lane = threadIdx.x & 31;
  long long total = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int n = b0 + lane < B ? tiles(b0 + lane) : 0;
    total += __reduce_add_sync(0xffffffffu, unsigned(n));
  }
  const long long ctas = total < gridDim.x ? total : gridDim.x;
  const long long t0 = blockIdx.x < ctas ? blockIdx.x * total / ctas : total;
  const long long t1 = blockIdx.x < ctas ? (blockIdx.x + 1) * total / ctas : total;
  Share s{t1 - t0, 0, 0};
  long long before = 0;
  for (int b0 = 0; b0 < B && s.count > 0; b0 += 32) {
    const int n = b0 + lane < B ? tiles(b0 + lane) : 0;
    int inc = n;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, x);
      if (lane >= x) inc += y;
    }
    const long long end = before + inc;
    const unsigned hit = __ballot_sync(0xffffffffu, n > 0 && t0 < end);
    if (hit) {
      const int src = __ffs(hit) - 1;
      s.b = b0 + src;
      s.offset = t0 - __shfl_sync(0xffffffffu, end - n, src);
      break;
    }
    before = __shfl_sync(0xffffffffu, end, 31);
  }
  return s;
}

}  // namespace dustin
