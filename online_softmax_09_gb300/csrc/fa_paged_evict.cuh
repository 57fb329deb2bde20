// fa_paged_evict.cuh -- launches of the weights that cached tokens receive, and of eviction by them.
#pragma once

#include "fa_paged4.cuh"

namespace fa {

struct PagedWeights {
  PagedBatch b;
  PagedCache c;  // keys of a bf16 cache
  PagedCache4 c4;  // or of a 4-bit one
  const __nv_bfloat16* q;
  long long q_tok, q_head;
  const float* lse;  // [T][Hq]
  const float* old;  // [page][head][slot], slots dense
  float* out;        // the same; may be `old`
  long long old_page, old_head, out_page, out_head;
  float scale_log2;
  bool cleared;  // the step's own tokens' slots of `out` are 0 before the sums are added
};
cudaError_t launch_paged_weights(PagedWeights& p, int d, bool packed, int num_sms, cudaStream_t st);

constexpr int kMostRows = 8;  // tensors whose slots are moved in one call

struct SlotRows {
  uint8_t* base;
  long long page, head, slot;  // strides in bytes
  int bytes, vec;              // bytes of a slot, and those moved at a time
};

struct PagedEvict {
  PagedBatch b;
  const float* weights;
  long long w_page, w_head;
  SlotRows rows[kMostRows];
  int n_rows;
  const int* keep;  // [S]
  int max_keep, sinks, recent;
  const int* out_table;
  long long out_stride;
  int* kept;        // [S][Hkv][max_keep]
  int* kv_len_out;  // [S]
};
cudaError_t launch_paged_evict(const PagedEvict& p, int num_sms, cudaStream_t st);

}  // namespace fa
