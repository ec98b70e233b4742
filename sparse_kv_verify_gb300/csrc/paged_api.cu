// C entry points of the paged cache (block tables and slots, head norms with the
// rotation and the cache write, attention of ragged new tokens): argument checks
// and launches.  Nothing here allocates device memory.  Workspace: the header of
// api.cu, then the scratch of the attention.
#include <cmath>

#include "common.cuh"
#include "host.h"
#include "kernels.h"

using namespace dustin;

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int batch_status(const dustin_batch* bt) {
  if (!bt || bt->B < 1 || bt->N < 1 || bt->max_new < 1 || bt->max_pages < 1) return DUSTIN_EINVAL;
  return bt->B > DUSTIN_MAX_REQUESTS || bt->N > DUSTIN_MAX_TOKENS || bt->max_new > DUSTIN_MAX_TOKENS ? DUSTIN_ERANGE : DUSTIN_OK;
}

bool pool_ok(const dustin_paged_kv& v) {
  if (!v.ptr || !aligned16(v.ptr) || (v.d != 64 && v.d != 128) || v.hkv < 1 || v.n_pages < 1 || v.page < 1) return false;
  for (int64_t s : {v.sp, v.sh, v.sl})   // (a tensor map's strides are below 2^40 bytes, eight rows' among them)
    if (s <= 0 || s % 8 || s >= int64_t(1) << 35) return false;
  if (v.sl < v.d) return false;
  return int64_t(v.n_pages) * v.page < (int64_t(1) << 31);
}
bool pools_match(const dustin_paged_kv& k, const dustin_paged_kv& v) {
  return k.hkv == v.hkv && k.d == v.d && k.n_pages == v.n_pages && k.page == v.page;
}

int attn_shape(int32_t hq, int32_t hkv, int32_t d) {
  if (hkv < 1 || hq < 1 || hq % hkv || (d != 64 && d != 128)) return DUSTIN_EINVAL;
  return hq / hkv > DUSTIN_MAX_QROWS || hq > DUSTIN_MAX_HEADS ? DUSTIN_ERANGE : DUSTIN_OK;
}

// Workspace of the attention, after the fixed part: the units that CTAs start and
// do not end, and two segment slots for each CTA.
struct PagedPlan {
  size_t split_off, part_off, total;
};
PagedPlan paged_plan(int hq, int hkv, int d, int max_new) {
  PagedPlan pl;
  pl.split_off = kScratch;
  pl.part_off = round256(pl.split_off + kPagedGridMax * 2 * sizeof(int4));
  pl.total = pl.part_off + round256(size_t(kPagedGridMax) * 2 * paged_lanes(hq, hkv, max_new) * kPagedTile * (size_t(d) + 2) * 4);
  return pl;
}

}  // namespace

extern "C" {

size_t dustin_paged_workspace_bytes(const dustin_batch* bt, int32_t hq, int32_t hkv, int32_t d) {
  if (batch_status(bt) != DUSTIN_OK) return 0;
  if (hq == 0) return round256(kScratch);
  if (attn_shape(hq, hkv, d) != DUSTIN_OK) return 0;
  return paged_plan(hq, hkv, d, bt->max_new).total;
}

int dustin_page_map(const dustin_batch* bt, int32_t page, int32_t n_pages, const int32_t* seq_len,
                    const int32_t* n_new, int32_t* table, int32_t* held, int32_t* free_list,
                    int32_t* n_free, int32_t* cu, int32_t* kv_len, int32_t* slot, int32_t* pos, void* ws,
                    size_t ws_bytes, cudaStream_t stream) {
  int st = batch_status(bt);
  if (st != DUSTIN_OK) return st;
  if (page < 1 || n_pages < 1) return DUSTIN_EINVAL;
  if (int64_t(bt->max_pages) * page > DUSTIN_MAX_LCAP) return DUSTIN_ERANGE;
  if (int64_t(bt->B) * bt->max_pages >= (int64_t(1) << 31)) return DUSTIN_ERANGE;   // (sums of pages are 32 bits)
  if (int64_t(n_pages) * page >= (int64_t(1) << 31)) return DUSTIN_ERANGE;
  const void* bufs[] = {seq_len, n_new, table, held, free_list, n_free, cu, kv_len, slot, pos};
  constexpr int n = sizeof(bufs) / sizeof(bufs[0]);
  for (int i = 0; i < n; ++i) {   // every buffer once: requests are written while others are still read
    if (!bufs[i] || !aligned4(bufs[i])) return DUSTIN_EINVAL;
    for (int j = 0; j < i; ++j)
      if (bufs[i] == bufs[j]) return DUSTIN_EINVAL;
  }
  if (!ws_ok(ws, ws_bytes, kScratch)) return DUSTIN_EWORKSPACE;
  PageMapArgs a{};
  a.B = bt->B;
  a.N = bt->N;
  a.max_new = bt->max_new;
  a.max_pages = bt->max_pages;
  a.page = page;
  a.n_pages = n_pages;
  a.seq_len = seq_len;
  a.n_new = n_new;
  a.table = table;
  a.held = held;
  a.free_list = free_list;
  a.n_free = n_free;
  a.cu = cu;
  a.kv_len = kv_len;
  a.slot = slot;
  a.pos = pos;
  a.err = err_word(ws);
  return page_map_launch(a, stream) == cudaSuccess ? DUSTIN_OK : DUSTIN_ECUDA;
}

int dustin_norm_rope(const dustin_rope* r, const void* q, int64_t q_stride, const void* k,
                     int64_t k_stride, const void* v, int64_t v_stride, const void* q_w, const void* k_w,
                     const float* inv_freq, const int32_t* pos, const int32_t* slot, void* q_out,
                     int64_t q_out_stride, dustin_paged_kv kc, dustin_paged_kv vc, void* ws,
                     size_t ws_bytes, cudaStream_t stream) {
  if (!r || r->N < 1 || r->hq < 1 || !(r->eps >= 0.f) || std::isinf(r->eps)) return DUSTIN_EINVAL;
  if (r->interleaved != 0 && r->interleaved != 1) return DUSTIN_EINVAL;
  if (!q || !k || !v || !pos || !slot || !q_out) return DUSTIN_EINVAL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(q_w) || !aligned16(k_w) ||
      !aligned4(inv_freq) || !aligned4(pos) || !aligned4(slot))
    return DUSTIN_EINVAL;
  if (!pool_ok(kc) || !pool_ok(vc) || !pools_match(kc, vc) || kc.ptr == vc.ptr) return DUSTIN_EINVAL;
  if (r->rot < 0 || r->rot > kc.d || r->rot % 16 || (r->rot && !inv_freq)) return DUSTIN_EINVAL;
  if (r->N > DUSTIN_MAX_TOKENS || r->hq > DUSTIN_MAX_HEADS || kc.hkv > DUSTIN_MAX_HEADS) return DUSTIN_ERANGE;
  const int64_t wq = int64_t(r->hq) * kc.d, wk = int64_t(kc.hkv) * kc.d;
  if (q_stride < wq || q_out_stride < wq || k_stride < wk || v_stride < wk) return DUSTIN_EINVAL;
  if (q_stride % 8 || q_out_stride % 8 || k_stride % 8 || v_stride % 8) return DUSTIN_EINVAL;
  if (q_out == q && q_out_stride != q_stride) return DUSTIN_EINVAL;
  for (const void* in : {k, v, q_w, k_w, static_cast<const void*>(inv_freq), static_cast<const void*>(pos),
                         static_cast<const void*>(slot)})
    if (in && (in == q_out || in == kc.ptr || in == vc.ptr)) return DUSTIN_EINVAL;
  for (const void* c : {kc.ptr, vc.ptr})
    if (c == q || c == q_out) return DUSTIN_EINVAL;
  if (!ws_ok(ws, ws_bytes, kScratch)) return DUSTIN_EWORKSPACE;
  RopeArgs a{};
  a.N = r->N;
  a.hq = r->hq;
  a.hkv = kc.hkv;
  a.rot = r->rot;
  a.interleaved = r->interleaved;
  a.eps = r->eps;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.qst = q_stride;
  a.kst = k_stride;
  a.vst = v_stride;
  a.q_w = static_cast<const uint16_t*>(q_w);
  a.k_w = static_cast<const uint16_t*>(k_w);
  a.inv_freq = inv_freq;
  a.pos = pos;
  a.slot = slot;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.ost = q_out_stride;
  a.kc = static_cast<uint16_t*>(kc.ptr);
  a.vc = static_cast<uint16_t*>(vc.ptr);
  a.ksp = kc.sp; a.ksh = kc.sh; a.ksl = kc.sl;
  a.vsp = vc.sp; a.vsh = vc.sh; a.vsl = vc.sl;
  a.n_pages = kc.n_pages;
  a.page = kc.page;
  a.err = err_word(ws);
  const int sms = num_sms();
  if (sms < 1) return DUSTIN_ECUDA;
  return rope_launch(a, kc.d, sms, stream) == cudaSuccess ? DUSTIN_OK : DUSTIN_ECUDA;
}

int dustin_paged_attn(const dustin_batch* bt, int32_t hq, const void* q, dustin_paged_kv kc,
                      dustin_paged_kv vc, const int32_t* table, const int32_t* cu, const int32_t* kv_len,
                      void* o, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  int st = batch_status(bt);
  if (st != DUSTIN_OK) return st;
  if (!q || !table || !cu || !kv_len || !o || o == lse) return DUSTIN_EINVAL;
  if (!aligned16(q) || (reinterpret_cast<uintptr_t>(o) & 31u) || !aligned4(lse) || !aligned4(table) || !aligned4(cu) || !aligned4(kv_len))
    return DUSTIN_EINVAL;
  if (!pool_ok(kc) || !pool_ok(vc) || !pools_match(kc, vc)) return DUSTIN_EINVAL;
  if (kc.page != 16 && kc.page != 32 && kc.page != 64 && kc.page % 128) return DUSTIN_EINVAL;
  for (const void* in : {q, static_cast<const void*>(kc.ptr), static_cast<const void*>(vc.ptr),
                         static_cast<const void*>(table), static_cast<const void*>(cu), static_cast<const void*>(kv_len)})
    if (in == o || in == lse) return DUSTIN_EINVAL;
  if (int64_t(bt->max_pages) * kc.page > DUSTIN_MAX_LCAP) return DUSTIN_ERANGE;
  st = attn_shape(hq, kc.hkv, kc.d);
  if (st != DUSTIN_OK) return st;
  const PagedPlan pl = paged_plan(hq, kc.hkv, kc.d, bt->max_new);
  if (!ws_ok(ws, ws_bytes, pl.total)) return DUSTIN_EWORKSPACE;
  PagedArgs a{};
  a.B = bt->B;
  a.N = bt->N;
  a.hq = hq;
  a.hkv = kc.hkv;
  a.max_new = bt->max_new;
  a.max_pages = bt->max_pages;
  a.page = kc.page;
  a.n_pages = kc.n_pages;
  a.scale_log2 = float(1.4426950408889634 / std::sqrt(double(kc.d)));
  a.table = table;
  a.cu = cu;
  a.kv_len = kv_len;
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.err = err_word(ws);
  a.split = reinterpret_cast<int4*>(static_cast<char*>(ws) + pl.split_off);
  a.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + pl.part_off);
  a.nt = kPagedTile / (hq / kc.hkv);
  a.qt = a.nt < bt->max_new ? a.nt : bt->max_new;
  if (!encode_rows_map(&a.qmap, q, kc.d, hq, bt->N, hq / kc.hkv, a.qt)) return DUSTIN_ECUDA;
  const int rows = kc.page < kPagedTile ? kc.page : kPagedTile;
  int panels, groups;
  a.merged = pool_steps(kc, &a.map_panels, &a.map_groups) && pool_steps(vc, &panels, &groups) &&
             panels == a.map_panels && groups == a.map_groups;
  if (!encode_pool_map(&a.kmap, kc, rows, a.merged) || !encode_pool_map(&a.vmap, vc, rows, a.merged)) return DUSTIN_ECUDA;
  const int sms = num_sms();
  if (sms < 1) return DUSTIN_ECUDA;
  return paged_launch(a, kc.d, sms, stream) == cudaSuccess ? DUSTIN_OK : DUSTIN_ECUDA;
}

}  // extern "C"
