// fa_paged4_api.cu -- the C ABI of the 4-bit paged cache and of eviction (include/fa.h): argument checks and launches.
// Every check comes before any CUDA call.
#include "fa_paged_checks.cuh"
#include "fa_paged_evict.cuh"

namespace {

// Strides (page, head) in bytes of a part of the cache. (The kernels multiply a page's number and stride in 32 bits each.)
int check_bytes(const long long* s, int pages, int heads) {
  const long long extent[2] = {pages, heads};
  for (int i = 0; i < 2; ++i) {
    if (extent[i] <= 1) continue;
    if (s[i] <= 0 || s[i] > (i == 0 ? 0xffffffffLL : 1LL << 46)) return FA_ERR_INVALID;
    if (s[i] & 15) return FA_ERR_ALIGN;
  }
  return FA_OK;
}

int check_cache4(const fa_paged_cache4* c, const fa_paged_batch* b) {
  if (c == nullptr || c->num_pages < 1) return FA_ERR_INVALID;
  FA_TRY(check_ptr(c->k, 16));
  FA_TRY(check_ptr(c->v, 16));
  FA_TRY(check_ptr(c->k_scale, 16));
  FA_TRY(check_ptr(c->v_scale, 16));
  FA_TRY(check_bytes(c->k_strides, c->num_pages, b->Hkv));
  FA_TRY(check_bytes(c->v_strides, c->num_pages, b->Hkv));
  FA_TRY(check_bytes(c->k_scale_strides, c->num_pages, b->Hkv));
  return check_bytes(c->v_scale_strides, c->num_pages, b->Hkv);
}

fa::PagedCache4 device_cache4(const fa_paged_cache4* c) {
  fa::PagedCache4 x;
  x.k = static_cast<const uint8_t*>(c->k);
  x.v = static_cast<const uint8_t*>(c->v);
  x.k_scale = static_cast<const uint8_t*>(c->k_scale);
  x.v_scale = static_cast<const uint8_t*>(c->v_scale);
  x.k_page = c->k_strides[0];
  x.k_head = c->k_strides[1];
  x.v_page = c->v_strides[0];
  x.v_head = c->v_strides[1];
  x.ks_page = c->k_scale_strides[0];
  x.ks_head = c->k_scale_strides[1];
  x.vs_page = c->v_scale_strides[0];
  x.vs_head = c->v_scale_strides[1];
  return x;
}

// Where a batch has both kinds of tiles: what a unit of the small ones costs beside one of the pairs. (1000 tokens over 9000
// keys and 23 single ones over 2000 to 14000, 32 heads of 8 kv heads: 268 us with 0.23, 256 with 0.28, 265 with 0.33 at
// d = 128; 202 with 0.25, 172 with 0.32, 177 with 0.38 at d = 64. Four other batches have their least between 0.26 and 0.38.)
float row4_cost(int d) { return d == 64 ? 0.32f : 0.28f; }

// Strides (page, head) in elements of fp32 weights, the page's below 2^32; `distinct`: they are written.
int check_weights(const float* w, const long long* s, int pages, int heads, bool distinct) {
  FA_TRY(check_ptr(w, 4));
  const long long extent[2] = {pages, heads};
  for (int i = 0; i < 2; ++i)
    if (extent[i] > 1 && (s[i] < (distinct ? 1 : 0) || s[i] > (i == 0 ? 0xffffffffLL : 1LL << 46))) return FA_ERR_INVALID;
  return FA_OK;
}

// What fa_paged_weights and fa_paged_weights4 share, once the cache has been looked at.
int weights_impl(fa::PagedWeights& p, const void* q, const long long* q_strides, const float* lse, int num_pages,
                 const fa_paged_batch* batch, const float* weights, float* out, const long long* strides, float scale,
                 bool packed, fa_stream_t stream) {
  FA_TRY(check_table(batch));
  FA_TRY(check_ptr(q, 16));
  FA_TRY(check_ptr(lse, 4));
  const long long extent[2] = {batch->T, batch->Hq};
  FA_TRY(check_strides(q_strides, extent, 2, false));
  FA_TRY(check_weights(weights, strides, num_pages, batch->Hkv, false));
  FA_TRY(check_weights(out, strides + 2, num_pages, batch->Hkv, true));
  if (weights == out && ((num_pages > 1 && strides[0] != strides[2]) || (batch->Hkv > 1 && strides[1] != strides[3])))
    return FA_ERR_INVALID;
  uint32_t* status = nullptr;
  int num_sms = 0;
  FA_TRY(fa::device_state(&status, &num_sms));
  p.b = device_batch(batch, num_pages, status);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_tok = q_strides[0];
  p.q_head = q_strides[1];
  p.lse = lse;
  p.old = weights;
  p.out = out;
  p.old_page = strides[0];
  p.old_head = strides[1];
  p.out_page = strides[2];
  p.out_head = strides[3];
  p.scale_log2 = (scale > 0.f ? scale : 1.0f / std::sqrt((float)batch->d)) * 1.4426950408889634f;
  return fa::launch_paged_weights(p, batch->d, packed, num_sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_LAUNCH;
}

// Bytes that can be moved at a time.
int piece_of(const fa_paged_rows& r) {
  const unsigned long long all = reinterpret_cast<uintptr_t>(r.base) | (unsigned long long)r.strides[0] |
                                 (unsigned long long)r.strides[1] | (unsigned long long)r.strides[2] |
                                 (unsigned long long)r.bytes;
  for (int v = 16; v > 1; v = v == 16 ? 4 : v / 2)
    if (all % v == 0) return v;
  return 1;
}

size_t workspace4_bytes(const fa_paged_batch* b) {
  const int G = b->Hq / b->Hkv, row_tile = fa::row_tile_of(G, b->max_q);
  return fa::paged4_rows_workspace_bytes(b->d, row_tile, fa::row4_columns(row_tile, b->max_q, G)) +
         (with_pairs(b) ? fa::paged_tiles_workspace_bytes(b->d) : 0);
}

}  // namespace

extern "C" {

int fa_paged_append4(const void* q, void* q_out, const void* k, const void* v, void* k_out, void* v_out,
                     const long long* strides, const fa_paged_cache4* cache, const fa_paged_batch* batch,
                     const fa_rotary* rotary, const int* positions, long long pos_axis, fa_stream_t stream) {
  fa::TraceRange trace("fa_paged_append4");
  FA_TRY(check_batch(batch));
  const bool with_q = q != nullptr || q_out != nullptr;
  if (strides == nullptr || pos_axis < 0) return FA_ERR_INVALID;
  if (rotary != nullptr) {
    FA_TRY(check_rotary(rotary, batch->d));
    if (positions == nullptr && rotary->naxes != 1) return FA_ERR_INVALID;
    if (positions != nullptr) FA_TRY(check_ptr(positions, 4));
  } else if (with_q || positions != nullptr) {
    return FA_ERR_INVALID;
  }
  FA_TRY(check_cache4(cache, batch));
  if (batch->S == 0 || batch->T == 0) return FA_OK;
  FA_TRY(check_table(batch));
  const void* ptr[6] = {q, q_out, k, v, k_out, v_out};
  for (int i = with_q ? 0 : 2; i < 6; ++i) {
    if (i > 3 && ptr[i] == nullptr) continue;
    const long long extent[2] = {batch->T, i < 2 ? batch->Hq : batch->Hkv};
    FA_TRY(check_ptr(ptr[i], 16));
    FA_TRY(check_strides(strides + 2 * i, extent, 2, i == 1 || i > 3));
  }
  uint32_t* status = nullptr;
  int num_sms = 0;
  FA_TRY(fa::device_state(&status, &num_sms));
  fa::RopeLaunch p = {};
  const int in[3] = {0, 2, 3};
  for (int i = 0; i < 3; ++i) {
    p.src[i] = static_cast<const __nv_bfloat16*>(ptr[in[i]]);
    p.in[i] = {0, strides[2 * in[i] + 1], strides[2 * in[i]]};
  }
  p.dst[0] = static_cast<__nv_bfloat16*>(q_out);
  p.out[0] = {0, strides[3], strides[2]};
  if (rotary != nullptr) set_rotary(p, rotary);
  p.positions = positions;
  p.pos_axis = pos_axis;
  p.tokens = batch->T;
  p.N = batch->T;
  p.Hq = with_q ? batch->Hq : 0;
  p.Hk = p.Hv = batch->Hkv;
  p.b = device_batch(batch, cache->num_pages, status);
  fa::Append4 a = {};
  a.c = device_cache4(cache);
  for (int i = 0; i < 2; ++i) {
    a.out[i] = static_cast<__nv_bfloat16*>(const_cast<void*>(ptr[4 + i]));
    a.out_tok[i] = strides[8 + 2 * i];
    a.out_head[i] = strides[9 + 2 * i];
  }
  return fa::launch_append4(p, a, batch->d, num_sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_LAUNCH;
}

size_t fa_fwd_paged4_workspace_bytes(const fa_paged_batch* batch) {
  if (batch == nullptr || batch->Hq < 1 || batch->Hkv < 1 || batch->Hq % batch->Hkv != 0 || batch->max_q < 0 ||
      check_d(batch->d) != FA_OK)
    return 0;
  return workspace4_bytes(batch);
}

int fa_fwd_paged4(const void* q, const long long* q_strides, const fa_paged_cache4* cache, const fa_paged_batch* batch,
                  void* o, float* lse, float scale, void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  fa::TraceRange trace("fa_fwd_paged4");
  FA_TRY(check_batch(batch));
  if (q_strides == nullptr) return FA_ERR_INVALID;
  FA_TRY(check_cache4(cache, batch));
  if (workspace == nullptr || workspace_bytes < workspace4_bytes(batch)) return FA_ERR_WORKSPACE;
  FA_TRY(check_ptr(workspace, 16));
  if (batch->S == 0 || batch->T == 0) return FA_OK;
  FA_TRY(check_table(batch));
  FA_TRY(check_ptr(q, 16));
  FA_TRY(check_ptr(o, 16));
  FA_TRY(check_ptr(lse, 4));
  const long long extent[2] = {batch->T, batch->Hq};
  FA_TRY(check_strides(q_strides, extent, 2, true));
  if (overlaps(q, q_strides, o, batch)) return FA_ERR_INVALID;
  uint32_t* status = nullptr;
  int num_sms = 0;
  FA_TRY(fa::device_state(&status, &num_sms));
  fa::PagedFwd p = {};
  p.b = device_batch(batch, cache->num_pages, status);
  p.b.row_cost = row4_cost(batch->d);
  num_sms = num_sms < fa::kPagedSms ? num_sms : fa::kPagedSms;
  p.b.sms = num_sms;
  set_fwd(p, q, q_strides, o, lse, scale, workspace, batch);
  const fa::PagedCache4 c = device_cache4(cache);
  const int d = batch->d, columns = fa::row4_columns(p.b.row_tile, p.b.max_q, p.b.G), ctas = fa::row4_ctas(columns, d);
  // The bf16 cache's rule, measured over 4 bits too, without and with the joining kernel (4000 keys, d = 128): 8 tiles of 4 rows
  // 12.4 us and 10.6, of 16 rows 38.3 and 15.7, 32 of 16 rows 30.0 and 23.3; 32 of 4 rows, where it is left out, 15.6 and 16.9.
  // At d = 64 it would bring 1 to 3 us more between 16 and 32 tiles, about what its launch costs the host.
  p.row_share = few_tiles(batch, p.b, (long long)ctas * num_sms)
                    ? reinterpret_cast<fa::RowShare*>(static_cast<char*>(workspace) +
                                                      fa::paged4_rows_part_bytes(d, p.b.row_tile, columns))
                    : nullptr;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (with_pairs(batch)) {
    fa::TileMaps m;
    FA_TRY(make_query_maps(m, p, q, q_strides, o, batch));
    m.k = m.v = m.q;  // not used: warps of the kernel write the operands
    char* ws = static_cast<char*>(workspace) + fa::paged4_rows_workspace_bytes(d, p.b.row_tile, columns);
    p.tile_part = reinterpret_cast<float*>(ws);
    p.share = reinterpret_cast<fa::TileShare*>(ws + fa::plan_up((size_t)2 * fa::kPagedSms * fa::tile_part(d) * 4));
    p.tile_ctas = num_sms;
    if (fa::launch_paged4_tiles(m, p, c, d, num_sms, st) != cudaSuccess) return FA_ERR_LAUNCH;
  }
  return fa::launch_paged4_rows(p, c, d, num_sms, st) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

int fa_paged_weights(const void* q, const long long* q_strides, const float* lse, const fa_paged_cache* cache,
                     const fa_paged_batch* batch, const float* weights, float* out, const long long* weight_strides,
                     float scale, fa_stream_t stream) {
  fa::TraceRange trace("fa_paged_weights");
  FA_TRY(check_batch(batch));
  if (q_strides == nullptr || weight_strides == nullptr || cache == nullptr || cache->num_pages < 1) return FA_ERR_INVALID;
  FA_TRY(check_ptr(cache->k, 16));
  const long long extent[3] = {cache->num_pages, batch->Hkv, batch->page_size};
  FA_TRY(check_strides(cache->k_strides, extent, 3, true));
  if (batch->S == 0 || batch->T == 0) return FA_OK;
  fa::PagedWeights p = {};
  p.c.k = static_cast<const __nv_bfloat16*>(cache->k);
  p.c.k_page = cache->k_strides[0];
  p.c.k_head = cache->k_strides[1];
  p.c.k_tok = cache->k_strides[2];
  return weights_impl(p, q, q_strides, lse, cache->num_pages, batch, weights, out, weight_strides, scale, false, stream);
}

int fa_paged_weights4(const void* q, const long long* q_strides, const float* lse, const fa_paged_cache4* cache,
                      const fa_paged_batch* batch, const float* weights, float* out, const long long* weight_strides,
                      float scale, fa_stream_t stream) {
  fa::TraceRange trace("fa_paged_weights4");
  FA_TRY(check_batch(batch));
  if (q_strides == nullptr || weight_strides == nullptr || cache == nullptr || cache->num_pages < 1) return FA_ERR_INVALID;
  FA_TRY(check_ptr(cache->k, 16));
  FA_TRY(check_ptr(cache->k_scale, 16));
  FA_TRY(check_bytes(cache->k_strides, cache->num_pages, batch->Hkv));
  FA_TRY(check_bytes(cache->k_scale_strides, cache->num_pages, batch->Hkv));
  if (batch->S == 0 || batch->T == 0) return FA_OK;
  fa::PagedWeights p = {};
  p.c4.k = static_cast<const uint8_t*>(cache->k);
  p.c4.k_scale = static_cast<const uint8_t*>(cache->k_scale);
  p.c4.k_page = cache->k_strides[0];
  p.c4.k_head = cache->k_strides[1];
  p.c4.ks_page = cache->k_scale_strides[0];
  p.c4.ks_head = cache->k_scale_strides[1];
  return weights_impl(p, q, q_strides, lse, cache->num_pages, batch, weights, out, weight_strides, scale, true, stream);
}

int fa_paged_evict(const float* weights, const long long* weight_strides, const fa_paged_rows* rows, int n_rows, int num_pages,
                   const fa_paged_batch* batch, const int* keep, int max_keep, int sinks, int recent, const int* out_table,
                   long long out_stride, int out_pages, int* kept, int* kv_len_out, fa_stream_t stream) {
  fa::TraceRange trace("fa_paged_evict");
  FA_TRY(check_batch(batch));
  if (weight_strides == nullptr || n_rows < 0 || n_rows > fa::kMostRows || (n_rows > 0 && rows == nullptr) || num_pages < 1 ||
      max_keep < 0 || max_keep > kMaxTokens || sinks < 0 || recent < 0 || out_pages < 0 || out_stride < 0 ||
      (long long)out_pages * batch->page_size < max_keep)
    return FA_ERR_INVALID;
  const long long heads = (long long)batch->S * batch->Hkv;
  if (heads * 8 > 0x7fffffffLL || heads * (max_keep / 32 + 1) > 0x7fffffffLL) return FA_ERR_INVALID;
  for (int i = 0; i < n_rows; ++i) {
    FA_TRY(check_ptr(rows[i].base, 1));
    if (rows[i].bytes < 1 || rows[i].bytes > (1 << 20)) return FA_ERR_INVALID;
    const long long extent[3] = {num_pages, batch->Hkv, batch->page_size};
    for (int j = 0; j < 3; ++j)
      if (extent[j] > 1 && (rows[i].strides[j] < 1 || rows[i].strides[j] > (1LL << 46))) return FA_ERR_INVALID;
  }
  if (batch->S == 0) return FA_OK;
  FA_TRY(check_table(batch));
  FA_TRY(check_weights(weights, weight_strides, num_pages, batch->Hkv, false));
  FA_TRY(check_ptr(keep, 4));
  FA_TRY(check_ptr(kv_len_out, 4));
  if (max_keep > 0) {
    FA_TRY(check_ptr(out_table, 4));
    FA_TRY(check_ptr(kept, 4));
  }
  uint32_t* status = nullptr;
  int num_sms = 0;
  FA_TRY(fa::device_state(&status, &num_sms));
  fa::PagedEvict p = {};
  p.b = device_batch(batch, num_pages, status);
  p.weights = weights;
  p.w_page = weight_strides[0];
  p.w_head = weight_strides[1];
  for (int i = 0; i < n_rows; ++i)
    p.rows[i] = {static_cast<uint8_t*>(rows[i].base), rows[i].strides[0], rows[i].strides[1], rows[i].strides[2],
                 rows[i].bytes, piece_of(rows[i])};
  p.n_rows = n_rows;
  p.keep = keep;
  p.max_keep = max_keep;
  p.sinks = sinks;
  p.recent = recent;
  p.out_table = out_table;
  p.out_stride = out_stride;
  p.kept = kept;
  p.kv_len_out = kv_len_out;
  return fa::launch_paged_evict(p, num_sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // extern "C"
