// fa_paged_evict.cu -- which cached tokens stay, by the weight that they have received, and their move into other pages.
//
// Per sequence of n tokens and kv head, new = min(n, keep) stay: the first `sinks`, the last `recent` (each as far as there is
// room, the first before the last), and of those between, the heaviest; among equal weights those at lower places. They keep
// their order. A NaN counts as the heaviest.
//
// fa_paged_select_kernel, one CTA per sequence and head: the m-th largest weight by its digits (11, 11 and 10 bits of an
// unsigned number in the weights' order, a histogram each), then two passes in order of place, one that counts and one that
// writes the places kept, each warp over a stretch of its own. Weights that fit stay in shared memory between the passes.
// fa_paged_move_kernel: a CTA moves 32 slots of one head, all tensors. The pages written are others than those read, so
// the slots move independently, and pages that sequences share stay as they are.
#include <math.h>

#include "fa_paged_evict.cuh"

namespace fa {

constexpr int kSelectThreads = 512, kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kSelectMost = 48 * 1024;  // weights held in shared memory
constexpr int kMoveSlots = 32, kMoveThreads = 256;

// What of a sequence's n tokens stays: places [0, a), [b, n), and m of those between.
struct Split {
  int n, fresh, a, b, m;
};
__device__ __forceinline__ Split split_of(const PagedEvict& p, int seq) {
  Split s;
  s.n = p.b.plan.seq[seq].kvl;
  int keep = p.keep[seq];
  if (keep < 0 || keep > p.max_keep) {
    record_index_error(p.b.status);
    keep = 0;
  }
  s.fresh = min(s.n, keep);
  s.a = min(p.sinks, s.fresh);
  s.b = s.n - min(p.recent, s.fresh - s.a);
  s.m = s.fresh - s.a - (s.n - s.b);
  return s;
}

// An unsigned number in the order of the weights.
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t x = __float_as_uint(w + 0.f);  // -0 becomes 0
  return x & 0x80000000u ? ~x : x | 0x80000000u;
}

__global__ void __launch_bounds__(kSelectThreads) fa_paged_select_kernel(const PagedEvict p, int held) {
  extern __shared__ __align__(16) uint32_t cache[];
  __shared__ uint32_t bins[kBins];
  __shared__ uint32_t warp_sum[kSelectWarps];
  __shared__ uint32_t above_w[kSelectWarps], level_w[kSelectWarps];
  __shared__ uint32_t found[2];  // the digit, and how many of its numbers stay
  const PagedBatch& b = p.b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (!plan_matches(b, b.d)) {
    if (tid == 0) record_index_error(b.status);
    return;
  }
  const int seq = blockIdx.x / b.Hkv, head = blockIdx.x - seq * b.Hkv;
  const Split s = split_of(p, seq);
  int* kept = p.kept + (long long)blockIdx.x * p.max_keep;
  if (head == 0 && tid == 0) p.kv_len_out[seq] = s.fresh;
  for (int i = s.fresh + tid; i < p.max_keep; i += kSelectThreads) kept[i] = -1;
  if (s.m == s.b - s.a) {  // all stay
    for (int i = tid; i < s.fresh; i += kSelectThreads) kept[i] = i;
    return;
  }
  for (int i = tid; i < s.a; i += kSelectThreads) kept[i] = i;
  for (int i = tid; i < s.n - s.b; i += kSelectThreads) kept[s.a + s.m + i] = s.b + i;
  if (s.m == 0) return;
  const int* tab = b.table + (long long)seq * b.table_stride;
  const float* w = p.weights + (long long)head * p.w_head;
  const int n = s.b - s.a;
  const bool hold = n <= held;
  auto read = [&](int i) -> uint32_t {
    const int key = s.a + i, page = tab[key >> b.page_shift];
    if ((unsigned)page >= (unsigned)b.num_pages) {
      record_index_error(b.status);
      return 0;
    }
    return order_of(w[(long long)page * p.w_page + (key & (b.page_size - 1))]);
  };
  uint32_t prefix = 0, mask = 0, left = (uint32_t)s.m;  // numbers whose bits under `mask` are `prefix`
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t digit = pass == 2 ? 1023 : 2047;
    for (int i = tid; i < kBins; i += kSelectThreads) bins[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < n; i += kSelectThreads) {
      uint32_t x;
      if (hold && pass > 0) {
        x = cache[i];
      } else {
        x = read(i);
        if (hold) cache[i] = x;
      }
      if ((x & mask) == prefix) atomicAdd(&bins[(x >> shift) & digit], 1u);
    }
    __syncthreads();
    // Numbers with a larger digit, for each: thread t has digits 2047 - 4 t and the three below.
    uint32_t v[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = bins[kBins - 1 - 4 * tid - i];
      sum += v[i];
    }
    uint32_t x = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    uint32_t before = x - sum;
    for (int i = 0; i < warp; ++i) before += warp_sum[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (before < left && left <= before + v[i]) {
        found[0] = kBins - 1 - 4 * tid - i;
        found[1] = left - before;
      }
      before += v[i];
    }
    __syncthreads();
    prefix |= found[0] << shift;
    mask |= digit << shift;
    left = found[1];
    __syncthreads();
  }
  // prefix is the m-th largest number; of those equal to it the first `left` stay.
  const int each = (n + kSelectWarps - 1) / kSelectWarps, from = min(n, warp * each), to = min(n, from + each);
  uint32_t above = 0, level = 0;
  for (int i0 = from; i0 < to; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t x = i < to ? (hold ? cache[i] : read(i)) : 0;
    above += __popc(__ballot_sync(0xffffffffu, i < to && x > prefix));
    level += __popc(__ballot_sync(0xffffffffu, i < to && x == prefix));
  }
  if (lane == 0) {
    above_w[warp] = above;
    level_w[warp] = level;
  }
  __syncthreads();
  uint32_t at_above = 0, at_level = 0;  // before this lane's place
  for (int i = 0; i < warp; ++i) {
    at_above += above_w[i];
    at_level += level_w[i];
  }
  const uint32_t under = (1u << lane) - 1;
  for (int i0 = from; i0 < to; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t x = i < to ? (hold ? cache[i] : read(i)) : 0;
    const bool is_above = i < to && x > prefix, is_level = i < to && x == prefix;
    const uint32_t ma = __ballot_sync(0xffffffffu, is_above), ml = __ballot_sync(0xffffffffu, is_level);
    const uint32_t na = at_above + __popc(ma & under), nl = at_level + __popc(ml & under);
    if (is_above || (is_level && nl < left)) kept[s.a + na + min(nl, left)] = s.a + i;
    at_above += __popc(ma);
    at_level += __popc(ml);
  }
}

__global__ void __launch_bounds__(kMoveThreads) fa_paged_move_kernel(const PagedEvict p) {
  __shared__ int page_s[kMoveSlots], slot_s[kMoveSlots], to_s[kMoveSlots];  // a page below 0: nothing to move
  const PagedBatch& b = p.b;
  if (!plan_matches(b, b.d)) return;
  const unsigned chunks = (p.max_keep + kMoveSlots - 1) / kMoveSlots, row = blockIdx.x / chunks;
  const int seq = (int)(row / b.Hkv), head = (int)(row - seq * b.Hkv), tid = threadIdx.x;
  const int i0 = (int)(blockIdx.x - row * chunks) * kMoveSlots;
  const int n = min(kMoveSlots, split_of(p, seq).fresh - i0);
  if (n <= 0) return;
  if (tid < n) {
    const int i = i0 + tid, key = p.kept[((long long)seq * b.Hkv + head) * p.max_keep + i];
    int page = b.table[(long long)seq * b.table_stride + (key >> b.page_shift)];
    int to = p.out_table[(long long)seq * p.out_stride + (i >> b.page_shift)];
    if ((unsigned)page >= (unsigned)b.num_pages || (unsigned)to >= (unsigned)b.num_pages) {
      record_index_error(b.status);
      page = -1;
    }
    page_s[tid] = page;
    slot_s[tid] = key & (b.page_size - 1);
    to_s[tid] = to;
  }
  __syncthreads();
  auto move = [&](const SlotRows& r, auto zero) {
    using V = decltype(zero);
    const int per = r.bytes / (int)sizeof(V), total = n * per;
    constexpr int kAtOnce = 4;
    for (int x0 = tid; x0 < total; x0 += kAtOnce * kMoveThreads) {
      V v[kAtOnce];
      uint8_t* dst[kAtOnce];
#pragma unroll
      for (int y = 0; y < kAtOnce; ++y) {
        const int x = x0 + y * kMoveThreads;
        dst[y] = nullptr;
        if (x >= total) continue;
        const int i = x / per, piece = x - i * per;
        if (page_s[i] < 0) continue;
        const uint8_t* src = r.base + (long long)page_s[i] * r.page + (long long)head * r.head +
                             (long long)slot_s[i] * r.slot + piece * (int)sizeof(V);
        v[y] = *reinterpret_cast<const V*>(src);
        dst[y] = r.base + (long long)to_s[i] * r.page + (long long)head * r.head +
                 (long long)((i0 + i) & (b.page_size - 1)) * r.slot + piece * (int)sizeof(V);
      }
#pragma unroll
      for (int y = 0; y < kAtOnce; ++y)
        if (dst[y] != nullptr) *reinterpret_cast<V*>(dst[y]) = v[y];
    }
  };
  for (int k = 0; k < p.n_rows; ++k) {
    const SlotRows& r = p.rows[k];
    if (r.vec == 16) move(r, uint4{});
    else if (r.vec == 4) move(r, uint32_t{});
    else if (r.vec == 2) move(r, uint16_t{});
    else move(r, uint8_t{});
  }
}

cudaError_t launch_paged_evict(const PagedEvict& p, cudaStream_t st) {
  if ((long long)(p.max_keep / kMoveSlots + 1) * p.b.Hkv * p.b.S > 0x7fffffffLL) return cudaErrorInvalidValue;
  static unsigned long long known[kMaxGpus];
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(fa_paged_select_kernel), kSelectMost * 4, known);
  if (e != cudaSuccess) return e;
  const long long most = (long long)p.b.max_pages * p.b.page_size;
  const int held = (int)(most < kSelectMost ? most : kSelectMost);
  fa_paged_select_kernel<<<(unsigned)(p.b.S * p.b.Hkv), kSelectThreads, held * 4, st>>>(p, held);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.max_keep == 0 || p.n_rows == 0) return e;
  const long long grid = (long long)((p.max_keep + kMoveSlots - 1) / kMoveSlots) * p.b.Hkv * p.b.S;
  fa_paged_move_kernel<<<(unsigned)grid, kMoveThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
