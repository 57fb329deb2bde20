// fa_paged_evict.cu -- which cached tokens stay, by the weight that they have received, and their move into other pages.
//
// Per sequence of n tokens and kv head, new = min(n, keep) stay: the first `sinks`, the last `recent` (each as far as there is
// room, the first before the last), and of those between, the heaviest; among equal weights those at lower places. They keep
// their order. A NaN counts as the heaviest.
//
// fa_paged_select_kernel, one to eight CTAs per sequence and head: the m-th largest weight by its digits (11, 11 and 10 bits,
// or four times 8, of an unsigned number in the weights' order, a histogram each), then two passes in order of place, one
// that counts and one that writes the places kept, each warp over a stretch of its own. Weights that fit stay in shared memory
// between the passes.
// fa_paged_move_kernel: a CTA moves 32 slots of one head, all tensors. The pages written are others than those read, so
// the slots move independently, and pages that sequences share stay as they are.
//
// Bound by latencies: plan, table, weights, a meeting of the cluster per digit, then table, slots. 8 kv heads of 32768 tokens
// cut to 4096 (d = 128, 35 MB): 20.9 us, of which 5.2 at the copy rate; with clusters of 4, 2 and 1 CTAs 28.8, 37.5 and 42.4
// where 8 took 28. 32 sequences of 700 to 1500 tokens cut to 500 (4 heads, d = 64, 34 MB): 14.0 us. Call by call from Python, 23
// to 29 us, both are bound by the host. (With digits of 11 bits in clusters too, and keys and values moved one after the other, 33
// and 29 us there.)
#include <cooperative_groups.h>
#include <math.h>

#include "fa_paged_evict.cuh"

namespace cg = cooperative_groups;

namespace fa {

constexpr int kSelectThreads = 512, kSelectWarps = kSelectThreads / 32;
constexpr int kSelectMost = 44 * 1024;  // weights held in shared memory
// A chain of look-ups stands before each CTA's copies, so many small ones: 32 sequences cut to 500 tokens 14.2 us, 17.6 with
// 256 threads for 32 slots (14.0 with 64, but 23.5 for the long sequence), 14.8 with 64 for 16.
constexpr int kMoveSlots = 32, kMoveThreads = 128;

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

// A cluster of CTAs per sequence and head, each with a stretch of the places of its own: every CTA puts its histograms and
// counts into the shared memory of all, and adds up what it has there: nothing waits for a write. (Read from the others
// behind the barrier, the long sequence took 22.3 us; so 21.4. Equal digits of a warp counted together first: 22.3 again.)
template <bool kCluster>  // (else one CTA has all places)
__global__ void __launch_bounds__(kSelectThreads) fa_paged_select_kernel(const PagedEvict p, int held) {
  extern __shared__ __align__(16) uint32_t cache[];
  // Digits of 11 bits; of 8 in a cluster, whose CTAs all get all histograms.
  constexpr int kBits = kCluster ? 8 : 11, kBins = 1 << kBits, kPasses = (32 + kBits - 1) / kBits;
  __shared__ __align__(16) uint32_t bins[kPasses][kBins];  // of each pass: none waits for the others' reading of the one before
  constexpr int kMost = kCluster ? 8 : 1, kQuads = kBins / 4;
  // Of all CTAs, for passes in turn: who writes a pass's again two passes later has met all that read it.
  __shared__ uint4 all_bins[kCluster ? 2 : 1][kMost][kCluster ? kQuads : 1];
  __shared__ uint2 all_counts[kMost];  // of each CTA: numbers above the bound, and at it
  __shared__ uint32_t warp_sum[kSelectWarps];
  __shared__ uint32_t above_w[kSelectWarps], level_w[kSelectWarps];
  __shared__ uint32_t found[2];  // the digit, and how many of its numbers stay
  const cg::cluster_group cluster = cg::this_cluster();
  const int C = kCluster ? (int)cluster.num_blocks() : 1, rank = kCluster ? (int)cluster.block_rank() : 0;
  const PagedBatch& b = p.b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int item = (int)(blockIdx.x / C), seq = item / b.Hkv, head = item - seq * b.Hkv;
  const Split s = split_of(p, seq);  // (its loads and the check of the plan go out together)
  if (!plan_matches(b, b.d)) {
    if (tid == 0) record_index_error(b.status);
    return;
  }
  int* kept = p.kept + (long long)item * p.max_keep;
  const int all = C * kSelectThreads, at = rank * kSelectThreads + tid;
  if (head == 0 && at == 0) p.kv_len_out[seq] = s.fresh;
  for (int i = s.fresh + at; i < p.max_keep; i += all) kept[i] = -1;
  if (s.m == s.b - s.a) {  // all stay
    for (int i = at; i < s.fresh; i += all) kept[i] = i;
    return;
  }
  for (int i = at; i < s.a; i += all) kept[i] = i;
  for (int i = at; i < s.n - s.b; i += all) kept[s.a + s.m + i] = s.b + i;
  if (s.m == 0) return;
  if constexpr (kCluster) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");  // this CTA's memory is there
  const int* tab = b.table + (long long)seq * b.table_stride;
  const float* w = p.weights + (long long)head * p.w_head;
  const int each = ((s.b - s.a + C - 1) / C + 31) & ~31;  // places of a CTA: those from s.a + rank * each on
  const int a0 = s.a + min(rank * each, s.b - s.a), n = min(each, s.b - a0);
  const bool hold = n <= held;
  auto read = [&](int i) -> uint32_t {
    const int key = a0 + i, page = tab[key >> b.page_shift];
    if ((unsigned)page >= (unsigned)b.num_pages) {
      record_index_error(b.status);
      return 0;
    }
    return order_of(w[(long long)page * p.w_page + (key & (b.page_size - 1))]);
  };
  for (int i = tid; i < kPasses * kBins; i += kSelectThreads) bins[0][i] = 0;
  __syncthreads();
  uint32_t prefix = 0, mask = 0, left = (uint32_t)s.m;  // numbers whose bits under `mask` are `prefix`
#pragma unroll 1
  for (int pass = 0; pass < kPasses; ++pass) {
    const int shift = max(0, 32 - kBits * (pass + 1));
    const uint32_t digit = (1u << min(kBits, 32 - kBits * pass)) - 1;
    if (hold && pass > 0) {
#pragma unroll 4
      for (int i = tid; i < n; i += kSelectThreads) {
        const uint32_t x = cache[i];
        if ((x & mask) == prefix) atomicAdd(&bins[pass][(x >> shift) & digit], 1u);
      }
    } else {
      constexpr int kAtOnce = 8;  // loads that go out together
      for (int i0 = tid; i0 < n; i0 += kAtOnce * kSelectThreads) {
        uint32_t x[kAtOnce];
#pragma unroll
        for (int y = 0; y < kAtOnce; ++y) x[y] = i0 + y * kSelectThreads < n ? read(i0 + y * kSelectThreads) : 0;
#pragma unroll
        for (int y = 0; y < kAtOnce; ++y) {
          const int i = i0 + y * kSelectThreads;
          if (i >= n) continue;
          if (hold) cache[i] = x[y];
          if ((x[y] & mask) == prefix) atomicAdd(&bins[pass][(x[y] >> shift) & digit], 1u);
        }
      }
    }
    __syncthreads();
    if constexpr (kCluster) {
      if (pass == 0) asm volatile("barrier.cluster.wait;" ::: "memory");  // the others' too
      for (int i = tid; i < C * kQuads; i += kSelectThreads)
        *cluster.map_shared_rank(&all_bins[pass & 1][rank][i % kQuads], i / kQuads) =
            reinterpret_cast<const uint4*>(bins[pass])[i % kQuads];
      cluster.sync();
    }
    // Numbers with a larger digit, for each: thread t has digits kBins - 1 - 4 t and the three below, if there are so many.
    uint32_t v[4] = {0, 0, 0, 0}, sum = 0;
    uint4 h[kMost];
#pragma unroll
    for (int c = 0; c < kMost; ++c) {
      h[c] = make_uint4(0, 0, 0, 0);
      if (c < C && tid < kQuads)
        h[c] = kCluster ? all_bins[pass & 1][c][kQuads - 1 - tid] : reinterpret_cast<const uint4*>(bins[pass])[kQuads - 1 - tid];
    }
#pragma unroll
    for (int c = 0; c < kMost; ++c) {
      v[0] += h[c].w;
      v[1] += h[c].z;
      v[2] += h[c].y;
      v[3] += h[c].x;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += v[i];
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
      if (v[i] > 0 && before < left && left <= before + v[i]) {
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
  const int each_w = ((n + kSelectWarps - 1) / kSelectWarps + 31) & ~31, from = min(n, warp * each_w),
            to = min(n, from + each_w);
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
  if constexpr (kCluster) {
    if (tid < C) {
      uint2 x = make_uint2(0, 0);
      for (int i = 0; i < kSelectWarps; ++i) {
        x.x += above_w[i];
        x.y += level_w[i];
      }
      *cluster.map_shared_rank(&all_counts[rank], tid) = x;
    }
    __syncwarp();
    cluster.sync();  // (the last that one CTA needs of another)
    for (int c = 0; c < rank; ++c) {
      at_above += all_counts[c].x;
      at_level += all_counts[c].y;
    }
  }
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
    if (is_above || (is_level && nl < left)) kept[s.a + na + min(nl, left)] = a0 + i;
    at_above += __popc(ma);
    at_level += __popc(ml);
  }
}

__global__ void __launch_bounds__(kMoveThreads) fa_paged_move_kernel(const PagedEvict p) {
  __shared__ int page_s[kMoveSlots], slot_s[kMoveSlots], to_s[kMoveSlots];  // a page below 0: nothing to move
  const PagedBatch& b = p.b;
  const unsigned chunks = (p.max_keep + kMoveSlots - 1) / kMoveSlots, row = blockIdx.x / chunks;
  const int seq = (int)(row / b.Hkv), head = (int)(row - seq * b.Hkv), tid = threadIdx.x;
  const int i0 = (int)(blockIdx.x - row * chunks) * kMoveSlots;
  const int n = min(kMoveSlots, split_of(p, seq).fresh - i0);
  // What the selection does not write is looked up before its end (21.4 us for the long sequence otherwise, 20.9 so). All CTAs
  // wait for it, so that this kernel does not end before it.
  const bool mine = plan_matches(b, b.d);
  const int out_page = tid < n ? p.out_table[(long long)seq * p.out_stride + ((i0 + tid) >> b.page_shift)] : -1;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the places are known
  if (n <= 0 || !mine) return;
  if (tid < n) {
    const int i = i0 + tid, key = p.kept[((long long)seq * b.Hkv + head) * p.max_keep + i];
    int page = b.table[(long long)seq * b.table_stride + (key >> b.page_shift)];
    if ((unsigned)page >= (unsigned)b.num_pages || (unsigned)out_page >= (unsigned)b.num_pages) {
      record_index_error(b.status);
      page = -1;
    }
    page_s[tid] = page;
    slot_s[tid] = key & (b.page_size - 1);
    to_s[tid] = out_page;
  }
  __syncthreads();
  // Two tensors whose slots are alike (keys and values, say), or one twice over: their loads go out together.
  auto move = [&](const SlotRows& r0, const SlotRows& r1, int both, auto zero) {
    using V = decltype(zero);
    const unsigned per = r0.bytes / (unsigned)sizeof(V), total = n * per;
    constexpr int kAtOnce = 2;
    for (unsigned x0 = tid; x0 < total; x0 += kAtOnce * kMoveThreads) {
      V v[2][kAtOnce];
      uint8_t* dst[2][kAtOnce];
#pragma unroll
      for (int y = 0; y < kAtOnce; ++y) {
        const unsigned x = x0 + y * kMoveThreads, i = x / per, piece = (x - i * per) * (unsigned)sizeof(V);
        const bool on = x < total && page_s[x < total ? i : 0] >= 0;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const SlotRows& r = z == 0 ? r0 : r1;
          dst[z][y] = nullptr;
          if (!on || (z == 1 && !both)) continue;
          uint8_t* base = r.base + (long long)head * r.head + piece;
          v[z][y] = *reinterpret_cast<const V*>(base + page_s[i] * r.page + slot_s[i] * r.slot);
          dst[z][y] = base + to_s[i] * r.page + (long long)((i0 + i) & (b.page_size - 1)) * r.slot;
        }
      }
#pragma unroll
      for (int y = 0; y < kAtOnce; ++y)
#pragma unroll
        for (int z = 0; z < 2; ++z)
          if (dst[z][y] != nullptr) *reinterpret_cast<V*>(dst[z][y]) = v[z][y];
    }
  };
  for (int k = 0; k < p.n_rows;) {
    const SlotRows &r0 = p.rows[k], &r1 = p.rows[k + 1 < p.n_rows ? k + 1 : k];
    const int both = k + 1 < p.n_rows && r1.bytes == r0.bytes && r1.vec == r0.vec;
    if (r0.vec == 16) move(r0, r1, both, uint4{});
    else if (r0.vec == 4) move(r0, r1, both, uint32_t{});
    else if (r0.vec == 2) move(r0, r1, both, uint16_t{});
    else move(r0, r1, both, uint8_t{});
    k += 1 + both;
  }
}

cudaError_t launch_paged_evict(const PagedEvict& p, int num_sms, cudaStream_t st) {
  const long long items = (long long)p.b.S * p.b.Hkv, chunks = (p.max_keep + kMoveSlots - 1) / kMoveSlots;
  if (items * 8 > 0x7fffffffLL || items * chunks > 0x7fffffffLL) return cudaErrorInvalidValue;
  static unsigned long long known[2][kMaxGpus];
  const void* kernels[2] = {reinterpret_cast<const void*>(fa_paged_select_kernel<false>),
                            reinterpret_cast<const void*>(fa_paged_select_kernel<true>)};
  // CTAs per sequence and head: as many as fill the GPU, with 1024 places each at least.
  const long long most = (long long)p.b.max_pages * p.b.page_size;
  int ctas = 1;
  while (ctas < 8 && items * ctas * 2 <= 2LL * num_sms && most >= 2048LL * ctas) ctas *= 2;
  const long long each = (most + ctas - 1) / ctas + 31;
  const int held = (int)(each < kSelectMost ? each : kSelectMost);
  cudaError_t e = allow_smem(kernels[ctas > 1], kSelectMost * 4, known[ctas > 1]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * ctas));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = held * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {(unsigned)ctas, 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  e = ctas > 1 ? cudaLaunchKernelEx(&cfg, fa_paged_select_kernel<true>, p, held)
               : cudaLaunchKernelEx(&cfg, fa_paged_select_kernel<false>, p, held);
  if (e != cudaSuccess || p.max_keep == 0 || p.n_rows == 0) return e;
  cfg.gridDim = dim3((unsigned)(items * chunks));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, fa_paged_move_kernel, p);
}

}  // namespace fa
