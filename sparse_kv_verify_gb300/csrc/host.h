// Host helpers of the C-ABI layer: argument checks, the workspace's fixed
// layout and TMA descriptor encoding, shared by the entry points' files.
#pragma once

#include <cudaTypedefs.h>

#include <cstdint>
#include <mutex>

#include "kernels.h"

namespace dustin {

constexpr size_t kHeader = 256;
constexpr size_t kCounterBytes = 65536;   // reserved
constexpr long long kVerifyUnitsMax = 16384;        // B * Hkv * layers per verification call
constexpr size_t kScratch = kHeader + kCounterBytes;

inline int num_sms() {
  static int cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (!cached[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    cached[dev] = n;
  }
  return cached[dev];
}

inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool params_ok(const dustin_params* p) {
  if (!p) return false;
  if (p->B < 1 || p->B > 65535) return false;
  if (p->Lcap < 1 || p->Lcap > DUSTIN_MAX_LCAP) return false;
  if (p->gamma < 0 || p->k < 1 || p->sinks < 0 || p->window < 0 || p->m < 0) return false;
  if (int64_t(p->sinks) + p->window > p->k) return false;
  return true;
}

inline bool kv_ok(const dustin_kv& v, int Lcap) {
  if (!v.ptr || !aligned16(v.ptr)) return false;
  if (v.d != 64 && v.d != 128) return false;
  if (v.hkv < 1) return false;
  if (v.sb <= 0 || v.sh <= 0 || v.sl <= 0) return false;
  if ((v.sb % 8) || (v.sh % 8) || (v.sl % 8)) return false;
  if (v.sl < v.d) return false;
  return true;
}

inline bool ws_ok(const void* ws, size_t ws_bytes, size_t need) {
  return ws && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0 && ws_bytes >= need;
}

inline int* err_word(void* ws) { return reinterpret_cast<int*>(ws); }

// ----------------------------------------------------------- TMA encoding

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// TMA map over a cache view with box 64 columns x 128 rows and the 128-byte
// swizzle that the score kernel's ldmatrix addressing expects.  A densely
// packed cache [B][hkv][Lcap][d] is described as 2-D rows [B*hkv*Lcap][d]
// (rows of a box that run past one head's Lcap positions are past seq_len and
// masked); any other strides use a 4-D map (d, Lcap, hkv, B).  *rank is 2 or 4.
inline bool encode_cache_map(CUtensorMap* m, const dustin_kv& v, int Lcap, int B, int* rank,
                      int box_rows = 128) {
  auto fn = encode_fn();
  if (!fn) return false;
  const bool packed = v.sl == v.d && v.sh == int64_t(Lcap) * v.d && v.sb == int64_t(v.hkv) * v.sh &&
                      int64_t(B) * v.hkv * Lcap < (int64_t(1) << 31) - 256;
  CUresult r;
  if (packed) {
    cuuint64_t dims[2] = {cuuint64_t(v.d), cuuint64_t(B) * v.hkv * Lcap};
    cuuint64_t strides[1] = {cuuint64_t(v.sl) * 2};
    cuuint32_t box[2] = {64, cuuint32_t(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, v.ptr, dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    *rank = 2;
  } else {
    cuuint64_t dims[4] = {cuuint64_t(v.d), cuuint64_t(Lcap), cuuint64_t(v.hkv), cuuint64_t(B)};
    cuuint64_t strides[3] = {cuuint64_t(v.sl) * 2, cuuint64_t(v.sh) * 2, cuuint64_t(v.sb) * 2};
    cuuint32_t box[4] = {64, cuuint32_t(box_rows), 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v.ptr, dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    *rank = 4;
  }
  return r == CUDA_SUCCESS;
}

// Verify queries [B][T][hq][d] as 3-D (d, hq, B*T) with box (64, G, T): one
// load brings the G x T query rows of one (sequence, KV head) as rows t*G + h.
inline bool encode_query_map(CUtensorMap* m, const void* q, int d, int hq, int BT, int G, int T) {
  // the encoding depends on these arguments only: repeated calls on the same
  // buffers (one per layer and step) reuse the previous result
  struct Key {
    const void* q;
    int d, hq, BT, G, T;
  };
  constexpr int kSlots = 2 * DUSTIN_MAX_LAYERS;
  static thread_local Key keys[kSlots];
  static thread_local CUtensorMap maps[kSlots];
  static thread_local int next = 0;
  for (int i = 0; i < kSlots; ++i)
    if (keys[i].q == q && keys[i].d == d && keys[i].hq == hq && keys[i].BT == BT && keys[i].G == G &&
        keys[i].T == T) {
      *m = maps[i];
      return true;
    }
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(hq), cuuint64_t(BT)};
  cuuint64_t strides[2] = {cuuint64_t(d) * 2, cuuint64_t(hq) * d * 2};
  cuuint32_t box[3] = {64, cuuint32_t(G), cuuint32_t(T)};
  cuuint32_t estr[3] = {1, 1, 1};
  if (fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  keys[next] = Key{q, d, hq, BT, G, T};
  maps[next] = *m;
  next = (next + 1) % kSlots;
  return true;
}

// TMA map over a prefix cache [hkv][cap][d] that brings a whole tile of `rows`
// rows of one KV head in one load: (64 columns, cap, d / 64, hkv) with box
// (64, rows, d / 64, 1), so that a tile's 64-column panels follow one another in
// shared memory, each with the 128-byte swizzle.
inline bool encode_prefix_map(CUtensorMap* m, const dustin_kv& v, int cap, int rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {64, cuuint64_t(cap), cuuint64_t(v.d / 64), cuuint64_t(v.hkv)};
  cuuint64_t strides[3] = {cuuint64_t(v.sl) * 2, 128, cuuint64_t(v.sh) * 2};
  cuuint32_t box[4] = {64, cuuint32_t(rows), cuuint32_t(v.d / 64), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v.ptr, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace dustin
