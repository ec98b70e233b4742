// C entry points of the cache operators (windowed and shared-prefix attention,
// accumulated attention weights, eviction): argument checks and launches.
// Nothing here allocates device memory.  Workspace: the header of api.cu, then
// the scratch of the one operator that runs.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "host.h"
#include "kernels.h"

using namespace dustin;

namespace {

float scale_log2_of(int d) { return float(1.4426950408889634 / std::sqrt(double(d))); }

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The shape rules of the attention calls.
int attend_shape(const dustin_params* p, int32_t hq, int32_t hkv, int32_t d) {
  if (!params_ok(p)) return DUSTIN_EINVAL;
  if (hkv < 1 || hq < 1 || hq % hkv || (d != 64 && d != 128)) return DUSTIN_EINVAL;
  if (p->gamma + 1 > DUSTIN_MAX_BLOCK || int64_t(p->gamma + 1) * (hq / hkv) > DUSTIN_MAX_QROWS)
    return DUSTIN_ERANGE;
  if (int64_t(p->B) * hkv > kVerifyUnitsMax) return DUSTIN_ERANGE;
  return DUSTIN_OK;
}

// Workspace of an attention call, after the fixed part: every unit's first and
// last CTA and the segment slots of the sequences' own part, then those of the
// prefix.
struct AttendPlan {
  int64_t slot_floats;
  int nt, row_tiles, pairs;
  size_t seg_off, part_off, pseg_off, ppart_off, total;
};
AttendPlan attend_plan(int B, int hq, int hkv, int d, int T, bool prefix) {
  AttendPlan pl;
  const int64_t units = int64_t(B) * hkv, NQ = int64_t(T) * (hq / hkv);
  pl.slot_floats = (NQ * d + 2 * NQ + 3) / 4 * 4;   // 16-byte aligned slots
  pl.nt = kPrefixTile / (hq / hkv);
  pl.row_tiles = int((int64_t(B) * T + pl.nt - 1) / pl.nt);
  pl.pairs = (pl.row_tiles + 1) / 2;
  pl.seg_off = kScratch;
  pl.part_off = round256(pl.seg_off + size_t(units) * 2 * 4);
  pl.pseg_off = round256(pl.part_off + size_t(units + kAttendGridMax) * size_t(pl.slot_floats) * 4);
  pl.ppart_off = round256(pl.pseg_off + (prefix ? size_t(hkv) * pl.pairs * 2 * 4 : 0));
  pl.total = pl.ppart_off;
  if (prefix)
    pl.total += round256((size_t(hkv) * pl.pairs + kPrefixGridMax) * 2 * kPrefixTile * (size_t(d) + 2) * 4);
  return pl;
}

// Workspace of an eviction, after the fixed part: rows to move per unit, then
// their lists.
struct EvictPlan {
  int list_cap;
  size_t moves_off, lists_off, total;
};
EvictPlan evict_plan(const dustin_params* p, int hkv, int n_layers) {
  EvictPlan pl;
  const size_t units = size_t(n_layers) * p->B * hkv;
  pl.list_cap = std::max(0, std::min(p->k, p->Lcap - p->k));
  pl.moves_off = kScratch;
  pl.lists_off = round256(pl.moves_off + units * 4);
  pl.total = round256(pl.lists_off + units * 2 * size_t(pl.list_cap) * 4);
  return pl;
}

// pk == nullptr: windowed attention.
int run_attend(const dustin_params* p, int32_t hq, const void* q, const dustin_kv* pk, const dustin_kv* pv,
               int32_t prefix_cap, const int32_t* prefix_len, const dustin_kv& k, const dustin_kv& v,
               const void* kb, const void* vb, const int32_t* seq_len, void* o, float* lse, void* ws,
               size_t ws_bytes, cudaStream_t stream) {
  if (!params_ok(p)) return DUSTIN_EINVAL;
  if (!q || !kb || !vb || !o || !seq_len || o == lse) return DUSTIN_EINVAL;
  // (units are written while others are still read)
  for (const void* in : {q, kb, vb, static_cast<const void*>(k.ptr), static_cast<const void*>(v.ptr),
                         static_cast<const void*>(seq_len), static_cast<const void*>(prefix_len),
                         static_cast<const void*>(pk ? pk->ptr : nullptr), static_cast<const void*>(pv ? pv->ptr : nullptr)})
    if (in && (in == o || in == lse)) return DUSTIN_EINVAL;
  if (!aligned16(q) || !aligned16(kb) || !aligned16(vb) || !aligned16(o) || !aligned4(lse)) return DUSTIN_EINVAL;
  if (!kv_ok(k, p->Lcap) || !kv_ok(v, p->Lcap) || k.hkv != v.hkv || k.d != v.d) return DUSTIN_EINVAL;
  if (pk) {
    if (!prefix_len || prefix_cap < 1) return DUSTIN_EINVAL;
    if (prefix_cap > DUSTIN_MAX_LCAP) return DUSTIN_ERANGE;
    for (const dustin_kv* t : {pk, pv})
      if (!kv_ok(*t, prefix_cap) || t->hkv != k.hkv || t->d != k.d) return DUSTIN_EINVAL;
  }
  const int st = attend_shape(p, hq, k.hkv, k.d);
  if (st != DUSTIN_OK) return st;
  const AttendPlan pl = attend_plan(p->B, hq, k.hkv, k.d, p->gamma + 1, pk != nullptr);
  if (!ws_ok(ws, ws_bytes, pl.total)) return DUSTIN_EWORKSPACE;
  AttendArgs a{};
  a.B = p->B;
  a.Lcap = p->Lcap;
  a.T = p->gamma + 1;
  a.hq = hq;
  a.hkv = k.hkv;
  a.sinks = pk ? 0 : std::min(p->sinks, kAttendFar);
  a.window = pk ? kAttendFar : std::min(p->window, kAttendFar);
  a.Pcap = pk ? prefix_cap : 0;
  a.scale_log2 = scale_log2_of(k.d);
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k.ptr);
  a.v = static_cast<const uint16_t*>(v.ptr);
  a.kb = static_cast<const uint16_t*>(kb);
  a.vb = static_cast<const uint16_t*>(vb);
  a.ksb = k.sb; a.ksh = k.sh; a.ksl = k.sl;
  a.vsb = v.sb; a.vsh = v.sh; a.vsl = v.sl;
  if (pk) {
    a.pk = static_cast<const uint16_t*>(pk->ptr);
    a.pv = static_cast<const uint16_t*>(pv->ptr);
    a.pksh = pk->sh; a.pksl = pk->sl;
    a.pvsh = pv->sh; a.pvsl = pv->sl;
    a.prefix_len = prefix_len;
  }
  a.seq_len = seq_len;
  a.err = err_word(ws);
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  const int tile = kAttendTile;
  const auto tiles = [&](int rows) { return (std::min(rows, p->Lcap) + tile - 1) / tile; };
  a.max_tiles = tiles(a.sinks) + tiles(a.window) + 1;
  a.seg_cta = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + pl.seg_off);
  a.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + pl.part_off);
  a.slot_floats = pl.slot_floats;
  if (!encode_query_map(&a.qmap, q, k.d, hq, p->B * a.T, hq / k.hkv, a.T)) return DUSTIN_ECUDA;
  // caches that a tensor map cannot describe come row by row
  a.tma = encode_cache_map(&a.kmap, k, p->Lcap, p->B, &a.krank, tile) &&
          encode_cache_map(&a.vmap, v, p->Lcap, p->B, &a.vrank, tile);
  const int sms = num_sms();
  if (sms < 1) return DUSTIN_ECUDA;
  if (pk) {
    a.pgrid = std::min(sms, kPrefixGridMax);
    a.nt = pl.nt;
    a.row_tiles = pl.row_tiles;
    a.pairs = pl.pairs;
    a.pseg_cta = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + pl.pseg_off);
    a.ppartial = reinterpret_cast<float*>(static_cast<char*>(ws) + pl.ppart_off);
    if (!encode_query_map(&a.pqmap, q, k.d, hq, p->B * a.T, hq / k.hkv, pl.nt)) return DUSTIN_ECUDA;
    a.ptma = encode_prefix_map(&a.pkmap, *pk, prefix_cap, kPrefixTile) &&
             encode_prefix_map(&a.pvmap, *pv, prefix_cap, kPrefixTile);
  }
  return attend_launch(a, k.d, sms, stream) == cudaSuccess ? DUSTIN_OK : DUSTIN_ECUDA;
}

}  // namespace

extern "C" {

size_t dustin_cache_workspace_bytes(const dustin_params* p, int32_t hq, int32_t hkv, int32_t d,
                                    int32_t n_layers, int32_t prefix_cap) {
  if (!params_ok(p) || hkv < 1 || n_layers < 0 || n_layers > DUSTIN_MAX_LAYERS || prefix_cap < 0 ||
      prefix_cap > DUSTIN_MAX_LCAP || int64_t(p->B) * hkv > kVerifyUnitsMax)
    return 0;
  size_t need = kScratch;
  if (hq != 0) {
    if (attend_shape(p, hq, hkv, d) != DUSTIN_OK) return 0;
    need = attend_plan(p->B, hq, hkv, d, p->gamma + 1, prefix_cap > 0).total;
  }
  if (n_layers != 0) {
    const size_t e = evict_plan(p, hkv, n_layers).total;
    need = e > need ? e : need;
  }
  return round256(need);
}

int dustin_window_attn(const dustin_params* p, int32_t hq, const void* q, dustin_kv k, dustin_kv v,
                       const void* kb, const void* vb, const int32_t* seq_len, void* o, float* lse,
                       void* ws, size_t ws_bytes, cudaStream_t stream) {
  return run_attend(p, hq, q, nullptr, nullptr, 0, nullptr, k, v, kb, vb, seq_len, o, lse, ws, ws_bytes, stream);
}

int dustin_prefix_attn(const dustin_params* p, int32_t hq, const void* q, dustin_kv pk, dustin_kv pv,
                       int32_t prefix_cap, const int32_t* prefix_len, dustin_kv k, dustin_kv v,
                       const void* kb, const void* vb, const int32_t* seq_len, void* o, float* lse,
                       void* ws, size_t ws_bytes, cudaStream_t stream) {
  return run_attend(p, hq, q, &pk, &pv, prefix_cap, prefix_len, k, v, kb, vb, seq_len, o, lse, ws, ws_bytes, stream);
}

int dustin_accumulate(const dustin_params* p, int32_t hq, const void* q, const float* lse, dustin_kv k,
                      const int32_t* n_new, const int32_t* seq_len, const int32_t* n_seen, float* weight,
                      int32_t* pos, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!params_ok(p)) return DUSTIN_EINVAL;
  if (!q || !lse || !n_new || !seq_len || !n_seen || !weight || !pos) return DUSTIN_EINVAL;
  if (!aligned16(q) || !aligned4(lse) || !aligned4(weight) || !aligned4(pos)) return DUSTIN_EINVAL;
  if (static_cast<const void*>(weight) == pos) return DUSTIN_EINVAL;
  for (const void* in : {q, static_cast<const void*>(lse), static_cast<const void*>(k.ptr), static_cast<const void*>(n_new),
                         static_cast<const void*>(seq_len), static_cast<const void*>(n_seen)})
    if (in == weight || in == pos) return DUSTIN_EINVAL;
  if (!kv_ok(k, p->Lcap)) return DUSTIN_EINVAL;
  const int st = attend_shape(p, hq, k.hkv, k.d);
  if (st != DUSTIN_OK) return st;
  if (!ws_ok(ws, ws_bytes, kScratch)) return DUSTIN_EWORKSPACE;
  AccumulateArgs a{};
  a.B = p->B;
  a.Lcap = p->Lcap;
  a.T = p->gamma + 1;
  a.G = hq / k.hkv;
  a.hkv = k.hkv;
  a.scale_log2 = scale_log2_of(k.d);
  a.lse = lse;
  a.n_new = n_new;
  a.seq_len = seq_len;
  a.n_seen = n_seen;
  a.weight = weight;
  a.pos = pos;
  a.err = err_word(ws);
  const int sms = num_sms();
  if (sms < 1 || !encode_query_map(&a.qmap, q, k.d, hq, p->B * a.T, a.G, a.T) ||
      !encode_cache_map(&a.kmap, k, p->Lcap, p->B, &a.krank, kAccumulateTile))
    return DUSTIN_ECUDA;
  return accumulate_launch(a, k.d, sms, stream) == cudaSuccess ? DUSTIN_OK : DUSTIN_ECUDA;
}

int dustin_evict(const dustin_params* p, int32_t n_layers, const dustin_kv* k, const dustin_kv* v,
                 float* const* weight, int32_t* const* pos, const int32_t* n_seen, int32_t* seq_len,
                 void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!params_ok(p)) return DUSTIN_EINVAL;
  if (n_layers < 1) return DUSTIN_EINVAL;
  if (n_layers > DUSTIN_MAX_LAYERS) return DUSTIN_ERANGE;
  if (!k || !v || !weight || !pos || !n_seen || !seq_len || n_seen == seq_len) return DUSTIN_EINVAL;
  EvictArgs a{};
  a.B = p->B;
  a.Lcap = p->Lcap;
  a.hkv = k[0].hkv;
  a.D = k[0].d;
  a.n_layers = n_layers;
  a.sinks = p->sinks;
  a.window = p->window;
  a.k = p->k;
  a.n_seen = n_seen;
  a.seq_len = seq_len;
  const void* seen[4 * DUSTIN_MAX_LAYERS];   // every buffer once: rows move in place
  int n_seen_bufs = 0;
  for (int l = 0; l < n_layers; ++l) {
    if (!kv_ok(k[l], p->Lcap) || !kv_ok(v[l], p->Lcap)) return DUSTIN_EINVAL;
    if (k[l].hkv != a.hkv || v[l].hkv != a.hkv || k[l].d != a.D || v[l].d != a.D) return DUSTIN_EINVAL;
    if (!weight[l] || !pos[l] || !aligned4(weight[l]) || !aligned4(pos[l])) return DUSTIN_EINVAL;
    for (const void* t : {static_cast<const void*>(k[l].ptr), static_cast<const void*>(v[l].ptr),
                          static_cast<const void*>(weight[l]), static_cast<const void*>(pos[l])}) {
      for (int x = 0; x < n_seen_bufs; ++x)
        if (seen[x] == t) return DUSTIN_EINVAL;
      seen[n_seen_bufs++] = t;
    }
    EvictLayerDev& L = a.layer[l];
    L.k = static_cast<uint16_t*>(k[l].ptr);
    L.v = static_cast<uint16_t*>(v[l].ptr);
    L.weight = weight[l];
    L.pos = pos[l];
    L.ksb = k[l].sb; L.ksh = k[l].sh; L.ksl = k[l].sl;
    L.vsb = v[l].sb; L.vsh = v[l].sh; L.vsl = v[l].sl;
  }
  if (int64_t(p->B) * a.hkv > kVerifyUnitsMax) return DUSTIN_ERANGE;
  const EvictPlan pl = evict_plan(p, a.hkv, n_layers);
  if (!ws_ok(ws, ws_bytes, pl.total)) return DUSTIN_EWORKSPACE;
  a.err = err_word(ws);
  a.moves = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + pl.moves_off);
  a.lists = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + pl.lists_off);
  a.list_cap = pl.list_cap;
  const int sms = num_sms();
  if (sms < 1) return DUSTIN_ECUDA;
  return evict_launch(a, sms, stream) == cudaSuccess ? DUSTIN_OK : DUSTIN_ECUDA;
}

}  // extern "C"
