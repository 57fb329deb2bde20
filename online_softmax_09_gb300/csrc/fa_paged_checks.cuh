// fa_paged_checks.cuh -- what the C entry points of the rotary and paged operators share: checks of arguments, which all
// come before any CUDA call, and the batch as the kernels take it.
#pragma once

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

inline int check_ptr(const void* p, uintptr_t align) {
  if (p == nullptr) return FA_ERR_INVALID;
  return (reinterpret_cast<uintptr_t>(p) & (align - 1)) ? FA_ERR_ALIGN : FA_OK;
}

// Element strides of a 16-byte-chunked tensor; `distinct`: no stride may be 0 (a tensor that is written, or
// that a tensor map describes). The stride of an extent of 1 means nothing and is not looked at.
inline int check_strides(const long long* s, const long long* extent, int n, bool distinct) {
  for (int i = 0; i < n; ++i) {
    if (extent[i] <= 1) continue;
    if (s[i] < 0 || s[i] > (1LL << 46) || (distinct && s[i] == 0)) return FA_ERR_INVALID;
    if (s[i] & 7) return FA_ERR_ALIGN;
  }
  return FA_OK;
}

inline int check_rotary(const fa_rotary* r, int d) {
  if (r == nullptr) return FA_ERR_INVALID;
  if (r->rot < 16 || r->rot > d || (r->rot & 15) || r->naxes < 1 || r->naxes > 4) return FA_ERR_INVALID;
  FA_TRY(check_ptr(r->inv_freq, 4));
  if (r->axes != nullptr)
    for (int i = 0; i < r->rot / 2; ++i)
      if (r->axes[i] >= r->naxes) return FA_ERR_INVALID;
  return FA_OK;
}

inline void set_rotary(fa::RopeLaunch& p, const fa_rotary* r) {
  p.inv_freq = r->inv_freq;
  p.rot = r->rot;
  p.interleaved = r->interleaved ? 1 : 0;
  for (int i = 0; i < r->rot / 2 && r->axes != nullptr; ++i) p.axes[i >> 5] |= (uint64_t)r->axes[i] << ((i & 31) * 2);
}

inline int check_d(int d) { return d == 64 || d == 128 ? FA_OK : FA_ERR_UNSUPPORTED; }

inline int check_batch(const fa_paged_batch* b) {
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

inline int check_table(const fa_paged_batch* b) {
  FA_TRY(check_ptr(b->block_table, 4));
  return b->table_stride < 0 ? FA_ERR_INVALID : FA_OK;
}

// Queries [T][Hq][d] with strides (token, head) share memory with the dense o. (Rows along the larger stride are
// taken as solid, so that o may lie between them.)
inline bool overlaps(const void* q, const long long* strides, const void* o, const fa_paged_batch* b) {
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

inline fa::PagedBatch device_batch(const fa_paged_batch* b, int num_pages, uint32_t* status) {
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
  x.row_cost = fa::row_cost_of(b->d);
  x.status = status;
  return x;
}

// Some sequence may have more rows than the small tiles are for: pairs of 128-row tiles are launched as well.
inline bool with_pairs(const fa_paged_batch* b) {
  const int G = b->Hq / b->Hkv;
  return (long long)b->max_q * G > fa::pair_rows_of(G, b->d, b->max_q);
}

// Tensor map of bf16 data with 128-byte swizzled boxes of 64 elements; `strides` in elements.
inline int make_map(CUtensorMap* m, const void* base, int rank, const long long* dims, const long long* strides,
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

// Few tiles among many CTAs: a tile's partial results are many, and a kernel of its own joins them, spread
// over the GPU, in place of the tile's last CTA alone. Its launch costs 2 us of the GPU's time and as much of
// the host's. It pays from 9 results of a tile on (16 rows at d = 128, 4000 keys: 19.7 us without, 16.7 with it
// at 28 tiles, 22.1 and 23.0 at 36); with up to 1024 values in a result, which the last CTA joins in two
// rounds, 16 bring as much as the host pays (4 rows: 13.1 and 12.4 us at 16 tiles), 24 and more 1.5 to 4 us
// (8 tiles: 12.5 and 10.2 over 4000 keys, 32.0 and 27.9 over 30000). One sequence and pairs: no small tiles
// but for what a captured batch leaves.
inline bool few_tiles(const fa_paged_batch* batch, const fa::PagedBatch& b, long long ctas) {
  const long long most = (long long)batch->max_q * b.G, rows = most < b.row_tile ? most : b.row_tile;
  const long long tiles = (long long)batch->S * batch->Hkv, need = rows * batch->d <= 1024 ? 24 : 9;
  return (batch->S > 1 || !with_pairs(batch)) && tiles * need < ctas &&
         (long long)batch->max_pages * batch->page_size >= need * fa::kRowBlk;
}

// Queries, outputs, scale and partial results of an attention call.
inline void set_fwd(fa::PagedFwd& p, const void* q, const long long* q_strides, void* o, float* lse, float scale,
                    void* workspace, const fa_paged_batch* batch) {
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_tok = q_strides[0];
  p.q_head = q_strides[1];
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.o_wide = (reinterpret_cast<uintptr_t>(o) & 31) == 0;
  p.part = static_cast<float*>(workspace);
  const float s = scale > 0.f ? scale : 1.0f / std::sqrt((float)batch->d);
  p.scale_log2 = s * 1.4426950408889634f;
}

// The maps of the queries and, where a warp's rows are whole tokens, of the outputs.
inline int make_query_maps(fa::TileMaps& m, fa::PagedFwd& p, const void* q, const long long* q_strides, void* o,
                           const fa_paged_batch* batch) {
  const int d = batch->d;
  const long long qd[3] = {d, batch->Hq, batch->T}, qs[2] = {q_strides[1], q_strides[0]};
  const int qb[3] = {64, p.b.G, p.b.pair_tokens / 2};
  FA_TRY(make_map(&m.q, q, 3, qd, qs, qb));
  p.warp_out = d == 128 && 32 % p.b.G == 0;
  m.o = m.q;
  if (p.warp_out) {
    const long long os[2] = {d, (long long)batch->Hq * d};
    const int ob[3] = {64, p.b.G, 32 / p.b.G};
    FA_TRY(make_map(&m.o, o, 3, qd, os, ob));
  }
  return FA_OK;
}

}  // namespace
