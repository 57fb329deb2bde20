// fa_paged_api.cu -- the C ABI of rotary positions, the paged cache and attention over it (include/fa.h):
// argument checks and launches. Every check comes before any CUDA call.
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdint>

#include "fa.h"
#include "fa_paged.cuh"

namespace {

#define FA_TRY(x)               \
  do {                          \
    int _r = (x);               \
    if (_r != FA_OK) return _r; \
  } while (0)

constexpr int kMaxHeads = 1 << 16;
constexpr int kMaxTokens = 0x7fffffff - (1 << 16);

int check_ptr(const void* p, uintptr_t align) {
  if (p == nullptr) return FA_ERR_INVALID;
  return (reinterpret_cast<uintptr_t>(p) & (align - 1)) ? FA_ERR_ALIGN : FA_OK;
}

// Element strides of a 16-byte-chunked tensor; `distinct`: no stride may be 0 (a tensor that is written, or
// that a tensor map describes). The stride of an extent of 1 means nothing and is not looked at.
int check_strides(const long long* s, const long long* extent, int n, bool distinct) {
  for (int i = 0; i < n; ++i) {
    if (extent[i] <= 1) continue;
    if (s[i] < 0 || s[i] > (1LL << 46) || (distinct && s[i] == 0)) return FA_ERR_INVALID;
    if (s[i] & 7) return FA_ERR_ALIGN;
  }
  return FA_OK;
}

int check_rotary(const fa_rotary* r, int d) {
  if (r == nullptr) return FA_ERR_INVALID;
  if (r->rot < 16 || r->rot > d || (r->rot & 15) || r->naxes < 1 || r->naxes > 4) return FA_ERR_INVALID;
  FA_TRY(check_ptr(r->inv_freq, 4));
  if (r->axes != nullptr)
    for (int i = 0; i < r->rot / 2; ++i)
      if (r->axes[i] >= r->naxes) return FA_ERR_INVALID;
  return FA_OK;
}

void set_rotary(fa::RopeLaunch& p, const fa_rotary* r) {
  p.inv_freq = r->inv_freq;
  p.rot = r->rot;
  p.interleaved = r->interleaved ? 1 : 0;
  for (int i = 0; i < r->rot / 2 && r->axes != nullptr; ++i) p.axes[i >> 5] |= (uint64_t)r->axes[i] << ((i & 31) * 2);
}

int check_d(int d) { return d == 64 || d == 128 ? FA_OK : FA_ERR_UNSUPPORTED; }

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

int check_batch(const fa_paged_batch* b) {
  if (b == nullptr) return FA_ERR_INVALID;
  if (b->S < 0 || b->T < 0 || b->max_q < 0 || b->max_pages < 1 || b->window < 0) return FA_ERR_INVALID;
  if (b->Hq < 1 || b->Hkv < 1 || b->Hq % b->Hkv != 0 || b->Hq > kMaxHeads) return FA_ERR_INVALID;
  if ((long long)b->max_q * (b->Hq / b->Hkv) > kMaxTokens) return FA_ERR_INVALID;
  FA_TRY(check_d(b->d));
  if (b->page_size < 16 || b->page_size > 256 || (b->page_size & (b->page_size - 1))) return FA_ERR_UNSUPPORTED;
  // Tokens and keys are ints, with room for the last block of either.
  if ((long long)b->max_pages * b->page_size > kMaxTokens || b->T > kMaxTokens) return FA_ERR_INVALID;
  if (b->plan == nullptr || b->plan_bytes < fa::plan_layout(nullptr, b->S, nullptr)) return FA_ERR_WORKSPACE;
  FA_TRY(check_ptr(b->plan, 16));
  return FA_OK;
}

int check_table(const fa_paged_batch* b) {
  FA_TRY(check_ptr(b->block_table, 4));
  return b->table_stride < 0 ? FA_ERR_INVALID : FA_OK;
}

int check_cache(const fa_paged_cache* c, const fa_paged_batch* b) {
  if (c == nullptr || c->num_pages < 1) return FA_ERR_INVALID;
  FA_TRY(check_ptr(c->k, 16));
  FA_TRY(check_ptr(c->v, 16));
  const long long extent[3] = {c->num_pages, b->Hkv, b->page_size};
  FA_TRY(check_strides(c->k_strides, extent, 3, true));
  return check_strides(c->v_strides, extent, 3, true);
}

// Queries [T][Hq][d] with strides (token, head) share memory with the dense o. (Rows along the larger stride are
// taken as solid, so that o may lie between them.)
bool overlaps(const void* q, const long long* strides, const void* o, const fa_paged_batch* b) {
  const long long n[2] = {b->T, b->Hq}, s[2] = {n[0] > 1 ? strides[0] * 2 : 0, n[1] > 1 ? strides[1] * 2 : 0};
  const int outer = s[0] >= s[1] ? 0 : 1, inner = 1 - outer;
  constexpr long long kFar = 1LL << 60;  // beyond any address
  const long long row = b->d * 2LL;
  const long long span = s[inner] > 0 && n[inner] - 1 > kFar / s[inner] ? kFar : (n[inner] - 1) * s[inner] + row;
  const long long from = static_cast<long long>(reinterpret_cast<uintptr_t>(o) - reinterpret_cast<uintptr_t>(q));
  const long long to = from + n[0] * n[1] * row;
  // The first piece that ends after `from`, and whether it begins before `to`.
  if (from < span) return to > 0;
  if (n[outer] <= 1) return false;
  const long long i = (from - span) / s[outer] + 1;
  return i < n[outer] && i * s[outer] < to;
}

fa::PagedBatch device_batch(const fa_paged_batch* b, int num_pages, uint32_t* status) {
  fa::PagedBatch x = {};
  fa::plan_layout(b->plan, b->S, &x.plan);
  x.table = b->block_table;
  x.table_stride = b->table_stride;
  x.S = b->S;
  x.T = b->T;
  x.max_q = b->max_q;
  x.Hq = b->Hq;
  x.Hkv = b->Hkv;
  x.G = b->Hq / b->Hkv;
  x.d = b->d;
  x.page_size = b->page_size;
  while ((1 << x.page_shift) < b->page_size) ++x.page_shift;
  x.max_pages = b->max_pages;
  x.num_pages = num_pages;
  x.causal = b->causal || b->window > 0;
  x.window = b->window;
  x.pair_tokens = x.G <= 128 ? 2 * (128 / x.G) : 1;
  x.row_tile = fa::row_tile_of(x.G, b->max_q);
  x.status = status;
  return x;
}

// Some sequence may have more rows than the small tiles are for: pairs of 128-row tiles are launched as well.
bool with_pairs(const fa_paged_batch* b) {
  const int G = b->Hq / b->Hkv;
  return (long long)b->max_q * G > fa::pair_rows_of(G, b->d, b->max_q);
}

// Workspace: the partial results of the two kernels.
size_t workspace_bytes(const fa_paged_batch* b) {
  return fa::paged_rows_workspace_bytes(b->d, fa::row_tile_of(b->Hq / b->Hkv, b->max_q)) +
         (with_pairs(b) ? fa::paged_tiles_workspace_bytes(b->d) : 0);
}

// Tensor map of bf16 data with 128-byte swizzled boxes of 64 elements; `strides` in elements.
int make_map(CUtensorMap* m, const void* base, int rank, const long long* dims, const long long* strides,
             const int* box) {
  const auto encode = fa::tensor_map_encoder();
  if (encode == nullptr) return FA_ERR_LAUNCH;
  cuuint64_t d[4], s[3];
  cuuint32_t x[4], e[4];
  for (int i = 0; i < rank; ++i) {
    d[i] = (cuuint64_t)dims[i];
    x[i] = (cuuint32_t)box[i];
    e[i] = 1;
    if (i > 0) s[i - 1] = (cuuint64_t)(dims[i] > 1 ? strides[i - 1] : 8) * 2;
  }
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), d, s, x, e,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? FA_OK
             : FA_ERR_INVALID;
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
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_tok = q_strides[0];
  p.q_head = q_strides[1];
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.o_wide = (reinterpret_cast<uintptr_t>(o) & 31) == 0;
  p.part = static_cast<float*>(workspace);
  const float s = scale > 0.f ? scale : 1.0f / std::sqrt((float)batch->d);
  p.scale_log2 = s * 1.4426950408889634f;
  // Few tiles among many CTAs: a tile's partial results are many, and a kernel of its own joins them, spread
  // over the GPU, in place of the tile's last CTA alone. Its launch costs 2 us of the GPU's time and as much of
  // the host's. It pays from 9 results of a tile on (16 rows at d = 128, 4000 keys: 19.7 us without, 16.7 with it
  // at 28 tiles, 22.1 and 23.0 at 36); with up to 1024 values in a result, which the last CTA joins in two
  // rounds, 16 bring as much as the host pays (4 rows: 13.1 and 12.4 us at 16 tiles), 24 and more 1.5 to 4 us
  // (8 tiles: 12.5 and 10.2 over 4000 keys, 32.0 and 27.9 over 30000). One sequence and pairs: no small tiles
  // but for what a captured batch leaves.
  const bool pairs = with_pairs(batch);
  const long long most = (long long)batch->max_q * p.b.G, rows = most < p.b.row_tile ? most : p.b.row_tile;
  const long long tiles = (long long)batch->S * batch->Hkv, need = rows * batch->d <= 1024 ? 24 : 9;
  const long long ctas = (long long)fa::row_ctas(batch->d, p.b.row_tile) * p.b.sms;
  const bool few = (batch->S > 1 || !pairs) && tiles * need < ctas &&
                   (long long)batch->max_pages * batch->page_size >= need * fa::kRowBlk;
  p.row_share = few ? reinterpret_cast<fa::RowShare*>(
                          static_cast<char*>(workspace) +
                          fa::plan_up((size_t)2 * fa::row_ctas(batch->d, p.b.row_tile) * fa::kPagedSms *
                                      fa::row_part(batch->d, p.b.row_tile) * 4))
                    : nullptr;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (pairs) {
    fa::TileMaps m;
    const int d = batch->d;
    const long long qd[3] = {d, batch->Hq, batch->T}, qs[2] = {q_strides[1], q_strides[0]};
    const int qb[3] = {64, p.b.G, p.b.pair_tokens / 2};
    FA_TRY(make_map(&m.q, q, 3, qd, qs, qb));
    const long long cd[4] = {d, batch->page_size, batch->Hkv, cache->num_pages};
    const long long ks[3] = {p.c.k_tok, p.c.k_head, p.c.k_page}, vs[3] = {p.c.v_tok, p.c.v_head, p.c.v_page};
    const int cb[4] = {64, batch->page_size < 128 ? batch->page_size : 128, 1, 1};
    FA_TRY(make_map(&m.k, cache->k, 4, cd, ks, cb));
    FA_TRY(make_map(&m.v, cache->v, 4, cd, vs, cb));
    p.warp_out = d == 128 && 32 % p.b.G == 0;
    m.o = m.q;
    if (p.warp_out) {
      const long long os[2] = {d, (long long)batch->Hq * d};
      const int ob[3] = {64, p.b.G, 32 / p.b.G};
      FA_TRY(make_map(&m.o, o, 3, qd, os, ob));
    }
    char* ws = static_cast<char*>(workspace) + fa::paged_rows_workspace_bytes(d, p.b.row_tile);
    p.tile_part = reinterpret_cast<float*>(ws);
    p.share = reinterpret_cast<fa::TileShare*>(ws + fa::plan_up((size_t)2 * fa::kPagedSms * fa::tile_part(d) * 4));
    p.tile_ctas = num_sms;
    if (fa::launch_paged_tiles(m, p, d, num_sms, st) != cudaSuccess) return FA_ERR_LAUNCH;
  }
  return fa::launch_paged_rows(p, batch->d, num_sms, st) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // extern "C"
