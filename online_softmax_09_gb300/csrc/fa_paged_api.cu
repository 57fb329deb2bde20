// fa_paged_api.cu -- the C ABI of rotary positions, the paged cache and attention over it (include/fa.h):
// argument checks and launches. Every check comes before any CUDA call.
#include "fa_paged_checks.cuh"

namespace {

int rope_impl(const void* q, void* q_out, const void* k, void* k_out, const long long* strides, const int* positions,
              long long pos_axis, long long pos_batch, const fa_rotary* rotary, int B, int Hq, int Hkv, int N, int d,
              int inverse, fa_stream_t stream) {
  const bool with_k = k != nullptr || k_out != nullptr;
  if (B < 1 || N < 1 || Hq < 1 || Hkv < (with_k ? 1 : 0) || Hq > kMaxHeads || Hkv > kMaxHeads) return FA_ERR_INVALID;
  FA_TRY(check_d(d));
  FA_TRY(check_rotary(rotary, d));
  FA_TRY(check_ptr(positions, 4));
  if (strides == nullptr || pos_axis < 0 || pos_batch < 0) return FA_ERR_INVALID;
  if (((long long)B * N + fa::kPagedSms) > 0x7fffffffLL) return FA_ERR_INVALID;
  const void* ptr[4] = {q, q_out, k, k_out};
  for (int i = 0; i < (with_k ? 4 : 2); ++i) {
    const long long extent[3] = {B, i < 2 ? Hq : Hkv, N};
    FA_TRY(check_ptr(ptr[i], 16));
    FA_TRY(check_strides(strides + 3 * i, extent, 3, i & 1));
  }
  int num_sms = 0;
  FA_TRY(fa::device_state(nullptr, &num_sms));
  fa::RopeLaunch p = {};
  for (int i = 0; i < (with_k ? 2 : 1); ++i) {
    p.src[i] = static_cast<const __nv_bfloat16*>(ptr[2 * i]);
    p.dst[i] = static_cast<__nv_bfloat16*>(const_cast<void*>(ptr[2 * i + 1]));
    p.in[i] = {strides[6 * i], strides[6 * i + 1], strides[6 * i + 2]};
    p.out[i] = {strides[6 * i + 3], strides[6 * i + 4], strides[6 * i + 5]};
  }
  set_rotary(p, rotary);
  p.positions = positions;
  p.pos_axis = pos_axis;
  p.pos_batch = pos_batch;
  p.tokens = (long long)B * N;
  p.N = N;
  p.Hq = Hq;
  p.Hk = with_k ? Hkv : 0;
  p.inverse = inverse;
  return fa::launch_rope(p, d, false, num_sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK
                                                                                               : FA_ERR_LAUNCH;
}

int check_cache(const fa_paged_cache* c, const fa_paged_batch* b) {
  if (c == nullptr || c->num_pages < 1) return FA_ERR_INVALID;
  FA_TRY(check_ptr(c->k, 16));
  FA_TRY(check_ptr(c->v, 16));
  const long long extent[3] = {c->num_pages, b->Hkv, b->page_size};
  FA_TRY(check_strides(c->k_strides, extent, 3, true));
  return check_strides(c->v_strides, extent, 3, true);
}

// Workspace: the partial results of the two kernels.
size_t workspace_bytes(const fa_paged_batch* b) {
  return fa::paged_rows_workspace_bytes(b->d, fa::row_tile_of(b->Hq / b->Hkv, b->max_q)) +
         (with_pairs(b) ? fa::paged_tiles_workspace_bytes(b->d) : 0);
}

}  // namespace

extern "C" {

int fa_rope(const void* q, void* q_out, const void* k, void* k_out, const long long* strides, const int* positions,
            long long pos_axis, long long pos_batch, const fa_rotary* rotary, int B, int Hq, int Hkv, int N, int d,
            fa_stream_t stream) {
  fa::TraceRange trace("fa_rope");
  return rope_impl(q, q_out, k, k_out, strides, positions, pos_axis, pos_batch, rotary, B, Hq, Hkv, N, d, 0, stream);
}

int fa_rope_bwd(const void* dq_out, void* dq, const void* dk_out, void* dk, const long long* strides,
                const int* positions, long long pos_axis, long long pos_batch, const fa_rotary* rotary, int B, int Hq,
                int Hkv, int N, int d, fa_stream_t stream) {
  fa::TraceRange trace("fa_rope_bwd");
  return rope_impl(dq_out, dq, dk_out, dk, strides, positions, pos_axis, pos_batch, rotary, B, Hq, Hkv, N, d, 1,
                   stream);
}

size_t fa_paged_plan_bytes(int S) { return S < 0 ? 0 : fa::plan_layout(nullptr, S, nullptr); }

int fa_paged_plan(const int* cu_q, const int* kv_len, const fa_paged_batch* batch, fa_stream_t stream) {
  fa::TraceRange trace("fa_paged_plan");
  FA_TRY(check_batch(batch));
  FA_TRY(check_ptr(cu_q, 4));
  if (batch->S > 0) FA_TRY(check_ptr(kv_len, 4));
  uint32_t* status = nullptr;
  FA_TRY(fa::device_state(&status, nullptr));
  const int pair_rows = fa::pair_rows_of(batch->Hq / batch->Hkv, batch->d, batch->max_q);
  return fa::launch_paged_plan(cu_q, kv_len, device_batch(batch, 0, status), pair_rows,
                               reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_LAUNCH;
}

int fa_paged_append(const void* q, void* q_out, const void* k, const void* v, const long long* strides,
                    const fa_paged_cache* cache, const fa_paged_batch* batch, const fa_rotary* rotary,
                    const int* positions, long long pos_axis, fa_stream_t stream) {
  fa::TraceRange trace("fa_paged_append");
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
  FA_TRY(check_cache(cache, batch));
  if (batch->S == 0 || batch->T == 0) return FA_OK;
  FA_TRY(check_table(batch));
  const void* ptr[4] = {q, q_out, k, v};
  for (int i = with_q ? 0 : 2; i < 4; ++i) {
    const long long extent[2] = {batch->T, i < 2 ? batch->Hq : batch->Hkv};
    FA_TRY(check_ptr(ptr[i], 16));
    FA_TRY(check_strides(strides + 2 * i, extent, 2, i == 1));
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
  p.dst[1] = static_cast<__nv_bfloat16*>(cache->k);
  p.dst[2] = static_cast<__nv_bfloat16*>(cache->v);
  p.out[0] = {0, strides[3], strides[2]};
  p.out[1] = {cache->k_strides[0], cache->k_strides[1], cache->k_strides[2]};
  p.out[2] = {cache->v_strides[0], cache->v_strides[1], cache->v_strides[2]};
  if (rotary != nullptr) set_rotary(p, rotary);
  p.positions = positions;
  p.pos_axis = pos_axis;
  p.tokens = batch->T;
  p.N = batch->T;
  p.Hq = with_q ? batch->Hq : 0;
  p.Hk = p.Hv = batch->Hkv;
  p.b = device_batch(batch, cache->num_pages, status);
  return fa::launch_rope(p, batch->d, true, num_sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_LAUNCH;
}

size_t fa_fwd_paged_workspace_bytes(const fa_paged_batch* batch) {
  if (batch == nullptr || batch->Hq < 1 || batch->Hkv < 1 || batch->Hq % batch->Hkv != 0 || batch->max_q < 0 ||
      check_d(batch->d) != FA_OK)
    return 0;
  return workspace_bytes(batch);
}

int fa_fwd_paged(const void* q, const long long* q_strides, const fa_paged_cache* cache, const fa_paged_batch* batch,
                 void* o, float* lse, float scale, void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  fa::TraceRange trace("fa_fwd_paged");
  FA_TRY(check_batch(batch));
  if (q_strides == nullptr) return FA_ERR_INVALID;
  FA_TRY(check_cache(cache, batch));
  if (workspace == nullptr || workspace_bytes < ::workspace_bytes(batch)) return FA_ERR_WORKSPACE;
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
  num_sms = num_sms < fa::kPagedSms ? num_sms : fa::kPagedSms;
  p.b.sms = num_sms;
  p.c.k = static_cast<const __nv_bfloat16*>(cache->k);
  p.c.v = static_cast<const __nv_bfloat16*>(cache->v);
  p.c.k_page = cache->k_strides[0];
  p.c.k_head = cache->k_strides[1];
  p.c.k_tok = cache->k_strides[2];
  p.c.v_page = cache->v_strides[0];
  p.c.v_head = cache->v_strides[1];
  p.c.v_tok = cache->v_strides[2];
  set_fwd(p, q, q_strides, o, lse, scale, workspace, batch);
  const bool pairs = with_pairs(batch);
  const long long ctas = (long long)fa::row_ctas(batch->d, p.b.row_tile) * p.b.sms;
  const bool few = few_tiles(batch, p.b, ctas);
  p.row_share = few ? reinterpret_cast<fa::RowShare*>(
                          static_cast<char*>(workspace) +
                          fa::plan_up((size_t)2 * fa::row_ctas(batch->d, p.b.row_tile) * fa::kPagedSms *
                                      fa::row_part(batch->d, p.b.row_tile) * 4))
                    : nullptr;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (pairs) {
    fa::TileMaps m;
    const int d = batch->d;
    FA_TRY(make_query_maps(m, p, q, q_strides, o, batch));
    const long long cd[4] = {d, batch->page_size, batch->Hkv, cache->num_pages};
    const long long ks[3] = {p.c.k_tok, p.c.k_head, p.c.k_page}, vs[3] = {p.c.v_tok, p.c.v_head, p.c.v_page};
    const int cb[4] = {64, batch->page_size < 128 ? batch->page_size : 128, 1, 1};
    FA_TRY(make_map(&m.k, cache->k, 4, cd, ks, cb));
    FA_TRY(make_map(&m.v, cache->v, 4, cd, vs, cb));
    char* ws = static_cast<char*>(workspace) + fa::paged_rows_workspace_bytes(d, p.b.row_tile);
    p.tile_part = reinterpret_cast<float*>(ws);
    p.share = reinterpret_cast<fa::TileShare*>(ws + fa::plan_up((size_t)2 * fa::kPagedSms * fa::tile_part(d) * 4));
    p.tile_ctas = num_sms;
    if (fa::launch_paged_tiles(m, p, d, num_sms, st) != cudaSuccess) return FA_ERR_LAUNCH;
  }
  return fa::launch_paged_rows(p, batch->d, num_sms, st) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // extern "C"
