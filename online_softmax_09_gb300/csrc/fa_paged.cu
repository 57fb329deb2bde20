// fa_paged.cu -- attention of the newest tokens of a ragged batch over a paged key/value cache.
//
// For sequence s with q_len new tokens of kv_len, token j at position p = kv_len - q_len + j, and kv
// head h, with keys and values read through the sequence's page table:
//     x_t = scale * q_j . k_t  for t < kv_len, t <= p (causal), t > p - window (window > 0)
//     o_j = sum_t exp(x_t - lse_j) v_t,  lse_j = log sum_t exp(x_t);  nothing visible: o = 0, lse = -inf.
//
// fa_paged_plan_kernel lays the batch out (fa_paged.cuh). Sequences with few rows (new tokens times heads
// per kv head) are attended by fa_paged_rows_kernel in tiles of 16 or 32, the others by fa_paged_tiles_kernel
// (fa_paged_tiles.cu) in pairs of 128, after which the rows' kernel also joins what several CTAs share. Where a
// few small tiles share all CTAs, fa_paged_join_rows_kernel joins theirs.
//
// What has to be read is each key and value that some query sees, once: 4 d bytes per key and kv head.
#include <math.h>

#include "fa_paged.cuh"

namespace fa {

// ------------------------------------------------------------------------------------------ plan
// One CTA: checks every sequence's place and lengths, counts its work in both kinds of unit and
// forms the running sums. A sequence out of range, or with tokens that an earlier one has, gets no tokens (nothing
// of it is read or written) and raises the status word; it stands where those before it end, so that the first
// tokens stay in order, as the append's search needs them. (5.3 us for 24 sequences, 9 for 2000, once per step for
// all layers; nothing is read back, so a captured step lays itself out.)
__global__ void __launch_bounds__(1024) fa_paged_plan_kernel(const int* __restrict__ cu_q,
                                                             const int* __restrict__ kv_len, PagedBatch b,
                                                             int pair_rows) {
  __shared__ long long sums[2][32];
  __shared__ long long carry[2];
  __shared__ int ends[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < 2) carry[tid] = 0;
  bool bad = false, some = false;  // some (the same in all threads): a sequence up to here is out of range
  int reached = 0;                 // once there is one: the largest end among the sequences of the rounds before
  for (int i = tid; i < kPlanCtas; i += 1024) b.plan.counters[i] = 0;
  for (int s0 = 0; s0 < b.S; s0 += 1024) {
    const int s = s0 + tid;
    PlanSeq ps = {0, 0, 0, 0};
    long long w[2] = {0, 0};
    bool ok = true;
    int e = 0;
    if (s < b.S) {
      const int a = cu_q[s], n = kv_len[s];
      e = cu_q[s + 1];
      ok = a >= 0 && e >= a && e <= b.T && e - a <= b.max_q && n >= 0 &&
           (long long)n <= (long long)b.max_pages * b.page_size;
      if (ok) ps = {a, e - a, n, 0};
    }
    const bool pairs = (long long)ps.ql * b.G > pair_rows;
    if (!pairs) {
      const int nt = tile_count<false>(ps.ql, b);
      for (int i = 0; i < nt; ++i) {
        int t0, t1, b0, nb;
        tile_tokens<false>(i, ps.ql, b, t0, t1);
        tile_blocks<false>(t0, t1, ps.ql, ps.kvl, b.causal, b.window, b0, nb);
        w[0] += tile_units<false>(t0, t1, b, nb);
      }
    }
    // Long chunks: the warp counts each one's tiles together.
    for (uint32_t todo = __ballot_sync(0xffffffffu, pairs); todo; todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      const int ql = __shfl_sync(0xffffffffu, ps.ql, src), kvl = __shfl_sync(0xffffffffu, ps.kvl, src);
      const int nt = tile_count<true>(ql, b);
      long long sum = 0;
      for (int i = lane; i < nt; i += 32) {
        int t0, t1, b0, nb;
        tile_tokens<true>(i, ql, b, t0, t1);
        tile_blocks<true>(t0, t1, ql, kvl, b.causal, b.window, b0, nb);
        sum += tile_units<true>(t0, t1, b, nb);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if (lane == src) w[1] = sum;
    }
    if (__syncthreads_or(!ok) || some) {  // (and the carry of the previous round is set)
      if (!some) reached = s0 > 0 ? cu_q[s0] : 0;  // (all before are in range, so in order)
      some = true;
      int x = ok ? e : 0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x = max(x, v);
      }
      if (lane == 31) ends[warp] = x;
      int before = __shfl_up_sync(0xffffffffu, x, 1);
      before = max(reached, lane > 0 ? before : 0);
      __syncthreads();
      for (int i = 0; i < 32; ++i) {
        if (i < warp) before = max(before, ends[i]);
        reached = max(reached, ends[i]);
      }
      if (s < b.S && (!ok || ps.q0 < before)) {
        ps = {before, 0, 0, 0};
        w[0] = w[1] = 0;
        bad = true;
      }
    }
    if (s < b.S) b.plan.seq[s] = ps;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      w[k] *= b.Hkv;
      long long x = w[k];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += v;
      }
      if (lane == 31) sums[k][warp] = x;
      w[k] = x - w[k];  // before this sequence, within the warp
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      long long before = carry[k];
      for (int i = 0; i < warp; ++i) before += sums[k][i];
      if (s < b.S) b.plan.units[k][s] = before + w[k];
    }
    __syncthreads();
    if (tid < 2)
      for (int i = 0; i < 32; ++i) carry[tid] += sums[tid][i];
  }
  __syncthreads();
  if (tid < 2) b.plan.units[tid][b.S] = carry[tid];
  if (bad) record_index_error(b.status);
  if (tid == 0) {
    PlanHeader h = {};
    h.magic = kPlanMagic;
    h.S = b.S;
    h.T = b.T;
    h.max_q = b.max_q;
    h.Hq = b.Hq;
    h.Hkv = b.Hkv;
    h.d = b.d;
    h.page_size = b.page_size;
    h.max_pages = b.max_pages;
    h.causal = b.causal;
    h.window = b.window;
    *b.plan.head = h;
  }
}

cudaError_t launch_paged_plan(const int* cu_q, const int* kv_len, const PagedBatch& b, int pair_rows, cudaStream_t st) {
  fa_paged_plan_kernel<<<1, 1024, 0, st>>>(cu_q, kv_len, b, pair_rows);
  return cudaGetLastError();
}

// -------------------------------------------------------------------------------- small tiles
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool full) {
  const int n = full ? 16 : 0;  // 0: the 16 bytes are zero-filled and nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float bf16_round(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }

constexpr int kRowWarps = 4, kRowThreads = 32 * kRowWarps;
constexpr int kGran = kRowBlk / kRowWarps;  // keys that one warp takes at a time: 16, within one page

template <int D, int MT>
struct RowSmem {
  static constexpr int kCtas = row_ctas(D, 16 * MT);
  static constexpr int kStages = D == 128 || kCtas == 3 ? 3 : 5;
  static constexpr int kJoinRows = D == 128 ? 8 : 16;  // rows that the warps join at a time
  static constexpr int kSlots = D == 128 ? 4 : 8;  // stretches queued: the one before, the present one, those ahead
  static constexpr int kTile = kGran * D * 2;        // K or V of one granule
  static constexpr int kWarp = kStages * 2 * kTile;  // ring of one warp
  static constexpr int kMerge = kRowWarps * kWarp;   // kJoinRows rows of o of each warp
  static constexpr int kStat = kMerge + kRowWarps * kJoinRows * D * 4;  // their m, l, rounded l
  static constexpr int kQueue = kStat + kRowWarps * 3 * kJoinRows * 4;
  static constexpr int kFlag = kQueue + kSlots * (int)sizeof(Seg);
  static constexpr int kBytes = (kFlag + 4 + 15) / 16 * 16;
  static_assert(kBytes <= 231424 / kCtas, "kCtas CTAs must fit an SM");
};


// The tiles of 128 rows that several CTAs of the kernel before shared: their partial results joined in the
// order of the keys, 16 rows at a time, all of this grid's CTAs together, two such pieces per CTA under way
// at once. (512 tokens over 32768 keys: about 9 us; joined by the last CTA to finish each tile, on 64 of 152
// SMs, 18 us.)
template <int D>
struct JoinPiece {
  static constexpr int kAtOnce = 4;  // partial results whose loads go out together
  TileShare s;
  int c0, t, r, tok;
  bool on;
  float4 v[kAtOnce][D / 32];
  float mi[kAtOnce], li[kAtOnce], ei[kAtOnce];
  float M, Ls, Es, acc[D / 8];
  __device__ __forceinline__ const float* part(const PagedFwd& p, int c) const {
    return p.tile_part + (size_t)(2 * c + (c == c0 ? 1 : 0)) * tile_part(D) + t * kTile * (D + 3);
  }
  __device__ __forceinline__ void load(const PagedFwd& p, int c) {
    if (!on) return;
    const int g0 = threadIdx.x >> 4;  // columns 4 * (g0 + 8 i) ..
#pragma unroll
    for (int y = 0; y < kAtOnce; ++y) {
      const float* src = part(p, min(c + y, s.c1));
      mi[y] = src[D * kTile + r];
      li[y] = src[(D + 1) * kTile + r];
      ei[y] = src[(D + 2) * kTile + r];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) v[y][i] = *reinterpret_cast<const float4*>(src + ((g0 + 8 * i) * kTile + r) * 4);
    }
  }
  __device__ __forceinline__ void add(int c) {
    if (!on) return;
#pragma unroll
    for (int y = 0; y < kAtOnce; ++y) {
      if (c + y > s.c1) continue;
      if (mi[y] == -INFINITY) {  // nothing seen there, o was not written: l = 0; or every score was NaN, as l is
        Ls += li[y];
        continue;
      }
      const float mn = fmaxf(M, mi[y]);
      const float fa = ex2(M - mn), fb = ex2(mi[y] - mn);
      M = mn;
      Ls = Ls * fa + fb * li[y];
      Es = Es * fa + fb * ei[y];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        acc[4 * i] = acc[4 * i] * fa + fb * v[y][i].x;
        acc[4 * i + 1] = acc[4 * i + 1] * fa + fb * v[y][i].y;
        acc[4 * i + 2] = acc[4 * i + 2] * fa + fb * v[y][i].z;
        acc[4 * i + 3] = acc[4 * i + 3] * fa + fb * v[y][i].w;
      }
    }
  }
};

template <int D>
__device__ __forceinline__ void join_pairs(const PagedFwd& p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the kernel before is complete
  const PagedBatch& b = p.b;
  const int tpt = b.pair_tokens >> 1, used = tpt * b.G;
  // The shared tiles, listed by every CTA for itself: all descriptors are read at once.
  extern __shared__ __align__(1024) uint8_t smem[];
  struct Entry {
    TileShare s;
    int x;  // 2 * first CTA + tile
  };
  Entry* list = reinterpret_cast<Entry*>(smem);
  int* counts = reinterpret_cast<int*>(smem + 2 * kPagedSms * sizeof(Entry));  // of each warp
  constexpr int kEach = (2 * kPagedSms + kRowThreads - 1) / kRowThreads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  TileShare mine[kEach];
  uint32_t some[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int x = i * kRowThreads + threadIdx.x;
    mine[i].c1 = -1;
    if (x < 2 * p.tile_ctas) mine[i] = p.share[x];
  }
  int n = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    some[i] = __ballot_sync(0xffffffffu, mine[i].c1 >= 0);
    n += __popc(some[i]);
  }
  __syncthreads();  // the rows' use of this memory is over
  if (lane == 0) counts[warp] = n;
  __syncthreads();
  int at = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kRowWarps; ++w) {
    at += w < warp ? counts[w] : 0;
    total += counts[w];
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (mine[i].c1 >= 0)
      list[at + __popc(some[i] & ((1u << lane) - 1))] = Entry{mine[i], i * kRowThreads + (int)threadIdx.x};
    at += __popc(some[i]);
  }
  __syncthreads();
  const int units = total * (kTile / 16);
  const int g0 = threadIdx.x >> 4;
  for (int x = blockIdx.x; x < units; x += 2 * gridDim.x) {
    JoinPiece<D> j[2];
    int longest = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int u = x + k * gridDim.x;
      j[k].on = u < units;
      if (!j[k].on) continue;
      const Entry& e = list[u >> 3];
      j[k].s = e.s;
      j[k].c0 = e.x >> 1;
      j[k].t = e.x & 1;
      j[k].r = (u & 7) * 16 + (threadIdx.x & 15);
      j[k].tok = e.s.tok0 + j[k].r / b.G;
      j[k].on = j[k].r < used && j[k].tok < e.s.ql;
      j[k].M = -INFINITY;
      j[k].Ls = j[k].Es = 0.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) j[k].acc[i] = 0.f;
      longest = max(longest, e.s.c1 - j[k].c0 + 1);
    }
    for (int c = 0; c < longest; c += JoinPiece<D>::kAtOnce) {
#pragma unroll
      for (int k = 0; k < 2; ++k) j[k].load(p, j[k].c0 + c);
#pragma unroll
      for (int k = 0; k < 2; ++k) j[k].add(j[k].c0 + c);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!j[k].on) continue;
      const float inv = (j[k].Ls > 0.f || j[k].Ls != j[k].Ls) ? 1.f / (j[k].Ls + j[k].Es) : 0.f;
      const long long out = (long long)(j[k].s.q0 + j[k].tok) * b.Hq + j[k].s.head * b.G + j[k].r % b.G;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint2 w;
        w.x = pack_bf16(j[k].acc[4 * i] * inv, j[k].acc[4 * i + 1] * inv);
        w.y = pack_bf16(j[k].acc[4 * i + 2] * inv, j[k].acc[4 * i + 3] * inv);
        *reinterpret_cast<uint2*>(p.o + out * D + (g0 + 8 * i) * 4) = w;
      }
      if (g0 == 0) p.lse[out] = (j[k].M + log2f(j[k].Ls)) * 0.6931471805599453f;
    }
  }
}

// fa_paged_rows_kernel: tiles of 16 MT rows. Four warps per CTA, two or three CTAs per SM; each warp takes every
// fourth granule of 16 keys with a ring of its own, so no barrier stands in the loop: it waits for its
// own cp.async copies, forms the 16 MT x 16 scores (m16n8k16), carries its own running max and sums, and
// adds P V. (The queries stand in registers at MT = 1; at MT = 2 there is no room for them beside o, and they
// are read from shared memory.) The ring runs on across the CTA's stretches: the copies of the next ones are
// under way while one is finished (a stretch of a short sequence is a few granules, and its chain of table,
// keys, join and store would stand in the open each time). The four warps' results are joined once per stretch, and the
// stretches of a tile that several CTAs share by the CTA that finishes last, or by a kernel that follows,
// in the order of the keys.
//
// Weights are rounded to bf16 for the product with V; o is divided by the sum of the rounded weights,
// so a row that one key dominates is not off by that rounding, and lse holds the unrounded sum.
//
// Bound by HBM: 64 sequences of 200 to 8192 keys (32 query heads, 8 kv heads, d = 128, 1.11 GB) take 172 us,
// 6.45 TB/s, 96 % of the measured copy rate, two of 131072 keys 162 us (96 %), with 96 KB of copies under way
// per CTA. mma.sync and not tcgen05, because 4 to 16 rows would leave most of a 128-row tile empty while its
// scores still pass through the softmax's threads; the tensor pipe is 19 % busy. A single token over 1000 keys
// takes 8.6 to 9 us, a chain of latencies (plan, table, keys, join, release, partial results).
template <int D, int MT>
__global__ void __launch_bounds__(kRowThreads, row_ctas(D, 16 * MT)) fa_paged_rows_kernel(const PagedFwd p) {
  using L = RowSmem<D, MT>;
  constexpr int kRows = 16 * MT;        // rows of a tile
  constexpr int kChunks = D / 8;        // 16-byte chunks of a row
  constexpr int kRowsPer = 32 / kChunks;  // rows that one copy instruction of a warp covers
  constexpr int kNT = D / 8;            // 8-column tiles of o
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = sbase + warp * L::kWarp;
  float* merge = reinterpret_cast<float*>(smem + L::kMerge);
  float* stat = reinterpret_cast<float*>(smem + L::kStat);
  Seg* queue = reinterpret_cast<Seg*>(smem + L::kQueue);
  int* flag = reinterpret_cast<int*>(smem + L::kFlag);
  const PagedBatch& b = p.b;
  // (Its loads and the check of the plan go out together.)
  SegIter<false, kRows> it(b, p.tile_ctas > 0 ? max(1, L::kCtas * (b.sms - pair_sms(b))) : gridDim.x);
  if (!plan_matches(b, D)) {
    if (threadIdx.x == 0) record_index_error(b.status);
    if (p.tile_ctas > 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (p.row_share != nullptr && threadIdx.x == 0) p.row_share[blockIdx.x].c1 = -1;
    return;
  }
  if (p.row_share != nullptr) {
    if (threadIdx.x == 0) p.row_share[blockIdx.x].c1 = -1;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  // Copies: this lane's row and chunk within a group of rows, and its swizzled place.
  const int crow = lane / kChunks, cchunk = lane % kChunks;
  // ldmatrix rows of this lane.
  const int krow = (lane & 7) + ((lane >> 4) << 3), kchk = (lane >> 3) & 1;  // K: keys 0-7 | 8-15, chunk 0 | 1
  const int vrow = lane & 15, vchk = lane >> 4;                              // V: keys 0-15, chunk 0 | 1
  const int g = lane >> 2, c2 = (lane & 3) * 2;                              // rows g, g + 8; columns c2, c2 + 1
  const unsigned G = b.G;

  // The copying side: the stretch it is at, taken from the walk and put in the queue. (All warps put the
  // same stretches in the same slots. A warp is at most kStages - 1 granules, so that many stretches, ahead
  // of its own computing, and computing warps are never a stretch apart.)
  uint32_t fetched = 0;     // stretches put in the queue
  uint32_t copied = 0;      // granules copied, of all stretches
  int ln = 0, li = 0;       // granules of the stretch, and the next one
  int lkey = 0, llo = 0, lhi = 0, lhead = 0;
  const int* ltab = nullptr;
  int pages = -1;           // lane i: the page of granule (li & ~31) + i
  auto read_pages = [&]() {
    const int key = lkey + (li + lane) * kRowBlk;
    const bool in = li + lane < ln && key < lhi && key + kGran > llo;
    pages = in ? ltab[key >> b.page_shift] : -1;
    if (in && (unsigned)pages >= (unsigned)b.num_pages) {
      record_index_error(b.status);
      pages = -1;
    }
  };
  auto fetch = [&]() {
    Seg s;
    ln = li = 0;
    if (!it.next(s)) return;
    if (lane == 0) queue[fetched % L::kSlots] = s;
    __syncwarp();
    ++fetched;
    ln = s.n;
    lhead = s.head;
    lkey = s.blk * kRowBlk + warp * kGran;  // first key of this warp's granule 0
    key_range(s.t0, s.t1, s.ql, s.kvl, b.causal, b.window, llo, lhi);
    ltab = b.table + (long long)s.seq * b.table_stride;
    read_pages();
  };
  auto issue = [&]() {  // the next granule's copies, one group (an empty one once all are issued)
    if (li < ln) {
      const int page = __shfl_sync(0xffffffffu, pages, li & 31);
      const int key = lkey + li * kRowBlk;
      const int slot = key & (b.page_size - 1);
      const uint32_t st = ring + (copied % L::kStages) * 2 * L::kTile;
      const long long pg = page < 0 ? 0 : page;
      const __nv_bfloat16* kp = p.c.k + pg * p.c.k_page + lhead * p.c.k_head + cchunk * 8;
      const __nv_bfloat16* vp = p.c.v + pg * p.c.v_page + lhead * p.c.v_head + cchunk * 8;
#pragma unroll
      for (int r = 0; r < kGran; r += kRowsPer) {
        const int row = r + crow;
        const bool in = page >= 0 && key + row >= llo && key + row < lhi;
        const uint32_t dst = st + row * (D * 2) + ((cchunk ^ (row & 7)) << 4);
        cp_async16(dst, kp + (in ? (slot + row) * p.c.k_tok : 0), in);
      }
#pragma unroll
      for (int r = 0; r < kGran; r += kRowsPer) {
        const int row = r + crow;
        const bool in = page >= 0 && key + row >= llo && key + row < lhi;
        const uint32_t dst = st + L::kTile + row * (D * 2) + ((cchunk ^ (row & 7)) << 4);
        cp_async16(dst, vp + (in ? (slot + row) * p.c.v_tok : 0), in);
      }
      ++copied;
      if (++li == ln) fetch();  // (the look-ups of the next stretch are under way before they are needed)
      else if ((li & 31) == 0) read_pages();
    }
    cp_async_commit();
  };

  // The computing side: queries as A operands, zero rows past the tile; visible keys [klo, klim] of the
  // lane's rows, and those that every row sees (a granule inside them needs no mask). 16 rows of queries
  // are held in registers; of 32 rows the warps share one copy in shared memory, in the place where the
  // results are joined (`sq`, swizzled like the keys).
  const uint32_t sq = sbase + L::kMerge;
  uint32_t qa[MT == 1 ? D / 16 : 1][4];
  constexpr int kQLoads = kRows * kChunks / kRowThreads;
  uint4 qv[MT == 1 ? 1 : kQLoads];
  int klo[MT][2], klim[MT][2], all_lo = 0, all_lim = 0;
  auto load_q = [&](const Seg& s) {
    const unsigned r0 = (unsigned)s.tile * kRows;
    const int rows = (int)min((unsigned)kRows, (unsigned)s.ql * G - r0);
    auto row_of = [&](int r, int& tok) {  // row r of the tile (row 0 for those past it)
      const unsigned rr = r0 + (r < rows ? r : 0);
      tok = (int)(rr / G);
      const int hd = (int)(rr - tok * G);
      return p.q + (long long)(s.q0 + tok) * p.q_tok + (long long)(s.head * G + hd) * p.q_head;
    };
    int top = -0x7fffffff, low = 0x7fffffff;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * t + g + 8 * h;
        int tok;
        const __nv_bfloat16* qp = row_of(r, tok);
        if constexpr (MT == 1) {
          const bool ok = r < rows;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            qa[kk][h] = ok ? *reinterpret_cast<const uint32_t*>(qp + kk * 16 + c2) : 0;
            qa[kk][2 + h] = ok ? *reinterpret_cast<const uint32_t*>(qp + kk * 16 + 8 + c2) : 0;
          }
        }
        const int pos = s.kvl - s.ql + tok;
        klim[t][h] = b.causal ? pos : s.kvl - 1;
        klo[t][h] = mask_from(pos, b.window);
        top = max(top, klo[t][h]);
        low = min(low, klim[t][h]);
      }
    all_lo = __reduce_max_sync(0xffffffffu, top);
    all_lim = __reduce_min_sync(0xffffffffu, low);
    if constexpr (MT > 1) {
#pragma unroll
      for (int i = 0; i < kQLoads; ++i) {
        const int x = i * kRowThreads + threadIdx.x, r = x / kChunks;
        int tok;
        const __nv_bfloat16* qp = row_of(r, tok);
        qv[i] = r < rows ? *reinterpret_cast<const uint4*>(qp + (x % kChunks) * 8) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  auto place_q = [&]() {  // (MT > 1) by all threads, where nothing reads the place any more
    if constexpr (MT > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kQLoads; ++i) {
        const int x = i * kRowThreads + threadIdx.x, r = x / kChunks, c = x % kChunks;
        st_shared_v4(sq + r * (D * 2) + ((c ^ (r & 7)) << 4), qv[i].x, qv[i].y, qv[i].z, qv[i].w);
      }
      __syncthreads();
    }
  };

  fetch();
#pragma unroll
  for (int i = 0; i < L::kStages - 1; ++i) issue();
  if (fetched > 0) {
    load_q(queue[0]);
    place_q();
  }
  uint32_t done = 0;  // granules computed, of all stretches
  for (uint32_t k = 0; k < fetched; ++k) {
    const Seg& s = queue[k % L::kSlots];
    const int n = s.n, key0 = s.blk * kRowBlk + warp * kGran;
    const unsigned r0 = (unsigned)s.tile * kRows;
    const int rows = (int)min((unsigned)kRows, (unsigned)s.ql * G - r0);
    float o[MT][kNT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < kNT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][j][i] = 0.f;
    float m[MT][2], l[MT][2], lr[MT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        m[t][h] = -INFINITY;
        l[t][h] = lr[t][h] = 0.f;
      }

    for (int i = 0; i < n; ++i, ++done) {
      issue();
      cp_async_wait<L::kStages - 1>();
      __syncwarp();
      const uint32_t sk = ring + (done % L::kStages) * 2 * L::kTile, sv = sk + L::kTile;
      const int key = key0 + i * kRowBlk;
      float x[MT][2][4];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[t][0][e] = x[t][1][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t kb[4];
        ldsm4(sk + krow * (D * 2) + (((2 * kk + kchk) ^ (krow & 7)) << 4), kb);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          if constexpr (MT == 1) {
            mma16816(x[t][0], qa[kk], kb[0], kb[1]);
            mma16816(x[t][1], qa[kk], kb[2], kb[3]);
          } else {
            uint32_t qt[4];  // rows 0-7 | 8-15 of the sixteen, chunk 2 kk | 2 kk + 1
            const int qr = 16 * t + vrow;
            ldsm4(sq + qr * (D * 2) + (((2 * kk + vchk) ^ (qr & 7)) << 4), qt);
            mma16816(x[t][0], qt, kb[0], kb[1]);
            mma16816(x[t][1], qt, kb[2], kb[3]);
          }
        }
      }
      const bool masked = key < all_lo || key + kGran - 1 > all_lim;
      uint32_t pa[MT][4];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if (masked) {
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int kx = key + 8 * y + c2 + (e & 1);
              if (kx > klim[t][e >> 1] || kx < klo[t][e >> 1]) x[t][y][e] = -INFINITY;
            }
        }
        float mt[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v = fmaxf(fmaxf(x[t][0][2 * h], x[t][0][2 * h + 1]), fmaxf(x[t][1][2 * h], x[t][1][2 * h + 1]));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
          mt[h] = v * p.scale_log2;
        }
        // The reference max moves only when a row has outgrown it by 2^8 (any reference gives the same
        // softmax, and weights up to 2^8 lose nothing in fp32 or bf16).
        if (__any_sync(0xffffffffu, mt[0] > m[t][0] + 8.f || mt[1] > m[t][1] + 8.f)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float mn = fmaxf(m[t][h], mt[h]);
            const float corr = mn > m[t][h] ? ex2(m[t][h] - mn) : 1.f;
            m[t][h] = mn;
            l[t][h] *= corr;
            lr[t][h] *= corr;
#pragma unroll
            for (int j = 0; j < kNT; ++j) {
              o[t][j][2 * h] *= corr;
              o[t][j][2 * h + 1] *= corr;
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mu = m[t][h] == -INFINITY ? 0.f : m[t][h];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float a = ex2(fmaf(x[t][y][2 * h], p.scale_log2, -mu));
            const float c = ex2(fmaf(x[t][y][2 * h + 1], p.scale_log2, -mu));
            const uint32_t pk = pack_bf16(a, c);
            pa[t][2 * y + h] = pk;
            l[t][h] += a + c;
            lr[t][h] += __uint_as_float(pk << 16) + __uint_as_float(pk & 0xffff0000u);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kNT; j += 2) {
        uint32_t vb[4];
        ldsm4t(sv + vrow * (D * 2) + (((j + vchk) ^ (vrow & 7)) << 4), vb);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          mma16816(o[t][j], pa[t], vb[0], vb[1]);
          mma16816(o[t][j + 1], pa[t], vb[2], vb[3]);
        }
      }
      __syncwarp();  // the stage is read: the next copies may overwrite it
    }

    // ---- join the four warps, kJoin rows at a time
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[t][h] += __shfl_xor_sync(0xffffffffu, l[t][h], 1);
        l[t][h] += __shfl_xor_sync(0xffffffffu, l[t][h], 2);
        lr[t][h] += __shfl_xor_sync(0xffffffffu, lr[t][h], 1);
        lr[t][h] += __shfl_xor_sync(0xffffffffu, lr[t][h], 2);
      }
    const bool whole = s.first && s.last;
    const int c0 = s.c0, c1 = s.c1, q0 = s.q0, head = s.head;
    float* slot = p.part + (size_t)(2 * blockIdx.x + (s.first ? 1 : 0)) * row_part(D, kRows);
    auto put = [&](int row, int col, float4 v, float sum) {  // four columns of a row of o
      const unsigned rr = r0 + row;
      const int tok = (int)(rr / G), hd = (int)(rr - tok * G);
      const long long out = (long long)(q0 + tok) * b.Hq + head * (int)G + hd;
      const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;  // a row that sees nothing: o = 0
      uint2 w;
      w.x = pack_bf16(v.x * inv, v.y * inv);
      w.y = pack_bf16(v.z * inv, v.w * inv);
      *reinterpret_cast<uint2*>(p.o + out * D + col) = w;
      return out;
    };
    constexpr int kJoin = L::kJoinRows, kPer = kRowThreads / kJoin;  // threads per row, 8 columns each
#pragma unroll
    for (int pass = 0; pass < kRows / kJoin; ++pass) {
      if (pass * kJoin >= rows) break;
      __syncthreads();  // the rows (and queries) that stood here have been read
      // Columns 8 j .. of row g at block j ^ g: the rows of a column are in different banks.
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if ((16 * t + 8 * h) / kJoin != pass) continue;
          const int at = warp * kJoin + (16 * t + 8 * h) % kJoin + g;
#pragma unroll
          for (int j = 0; j < kNT; ++j)
            *reinterpret_cast<float2*>(merge + at * D + (j ^ g) * 8 + c2) =
                make_float2(o[t][j][2 * h], o[t][j][2 * h + 1]);
          if ((lane & 3) == 0) {
            stat[at * 3] = m[t][h];
            stat[at * 3 + 1] = l[t][h];
            stat[at * 3 + 2] = lr[t][h];
          }
        }
      __syncthreads();
      const int hr = threadIdx.x / kPer, row = hr + kJoin * pass, col0 = (threadIdx.x % kPer) * 4;
      float M = -INFINITY, Ls = 0.f, Lr = 0.f;
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, stat[(w * kJoin + hr) * 3]);
      const float Mu = M == -INFINITY ? 0.f : M;
      float4 acc[2];  // columns col0 + 4 kPer i .. + 3
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) {
        const float* st = stat + (w * kJoin + hr) * 3;
        const float f = ex2(st[0] - Mu);
        Ls += f * st[1];
        Lr += f * st[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int col = col0 + 4 * kPer * i;
          const float4 v = *reinterpret_cast<const float4*>(merge + (w * kJoin + hr) * D + ((col >> 3) ^ (hr & 7)) * 8 +
                                                            (col & 7));
          acc[i].x = fmaf(f, v.x, acc[i].x);
          acc[i].y = fmaf(f, v.y, acc[i].y);
          acc[i].z = fmaf(f, v.z, acc[i].z);
          acc[i].w = fmaf(f, v.w, acc[i].w);
        }
      }
      if (row < rows) {
        if (whole) {
          long long out = 0;
#pragma unroll
          for (int i = 0; i < 2; ++i) out = put(row, col0 + 4 * kPer * i, acc[i], Lr);
          if (col0 == 0) p.lse[out] = (M + log2f(Ls)) * 0.6931471805599453f;
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) *reinterpret_cast<float4*>(slot + row * D + col0 + 4 * kPer * i) = acc[i];
          if (col0 == 0) {
            slot[kRows * D + row] = M;
            slot[kRows * (D + 1) + row] = Ls;
            slot[kRows * (D + 2) + row] = Lr;
          }
        }
      }
    }
    if (k + 1 < fetched) load_q(queue[(k + 1) % L::kSlots]);  // on its way beside what follows
    // A tile that other CTAs share: the partial result is left, for the kernel that follows if one does, or
    // for the last of them to arrive, which joins all.
    if (!whole && p.row_share != nullptr) {
      if (c0 == (int)blockIdx.x && threadIdx.x == 0)
        p.row_share[c0] = RowShare{c1, q0, (int)r0, rows, head};
    } else if (!whole) {
      __syncthreads();
      if (threadIdx.x == 0) {
        // The barrier orders the CTA's stores before this thread's release, which covers them all.
        uint32_t before;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                     : "=r"(before)
                     : "l"(&b.plan.counters[c0])
                     : "memory");
        const bool last = before == (uint32_t)(c1 - c0);
        if (last) b.plan.counters[c0] = 0;
        *flag = last;
      }
      __syncthreads();
      if (*flag != 0) {
        // Four columns of a row per thread, eight results' loads at a time.
        for (int x = threadIdx.x; x < rows * (D / 4); x += kRowThreads) {
          const int rw = x / (D / 4), col = (x - rw * (D / 4)) * 4;
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
          float m0 = -INFINITY, ls = 0.f, lsr = 0.f;
          constexpr int kAtOnce = 8;
          for (int c = c0; c <= c1; c += kAtOnce) {
            float4 v[kAtOnce];
            float mi[kAtOnce], si[kAtOnce], ri[kAtOnce], mx = m0;
#pragma unroll
            for (int y = 0; y < kAtOnce; ++y) {
              const int cc = min(c + y, c1);
              const float* src = p.part + (size_t)(2 * cc + (cc == c0 ? 1 : 0)) * row_part(D, kRows);
              v[y] = __ldcg(reinterpret_cast<const float4*>(src + rw * D + col));
              mi[y] = c + y <= c1 ? __ldcg(src + kRows * D + rw) : -INFINITY;
              si[y] = __ldcg(src + kRows * (D + 1) + rw);
              ri[y] = __ldcg(src + kRows * (D + 2) + rw);
            }
#pragma unroll
            for (int y = 0; y < kAtOnce; ++y) mx = fmaxf(mx, mi[y]);
            const float mu = mx == -INFINITY ? 0.f : mx, f0 = ex2(m0 - mu);
            m0 = mx;
            a = make_float4(a.x * f0, a.y * f0, a.z * f0, a.w * f0);
            ls *= f0;
            lsr *= f0;
#pragma unroll
            for (int y = 0; y < kAtOnce; ++y) {
              if (c + y > c1) continue;
              const float f = ex2(mi[y] - mu);
              a.x = fmaf(f, v[y].x, a.x);
              a.y = fmaf(f, v[y].y, a.y);
              a.z = fmaf(f, v[y].z, a.z);
              a.w = fmaf(f, v[y].w, a.w);
              ls = fmaf(f, si[y], ls);
              lsr = fmaf(f, ri[y], lsr);
            }
          }
          const long long out = put(rw, col, a, lsr);
          if (col == 0) p.lse[out] = (m0 + log2f(ls)) * 0.6931471805599453f;
        }
      }
    }
    if (k + 1 < fetched) place_q();
  }
  if (p.tile_ctas > 0) join_pairs<D>(p);
}

// fa_paged_join_rows_kernel: the small tiles that the rows' kernel left, spread over the GPU. A CTA takes 32
// columns of a row: eight threads along the columns, sixteen over the partial results, each of which adds
// every sixteenth, four loads at a time; the sixteen sums are then added in order (so each element's order
// of addition is set by the division among CTAs alone). It starts beside the rows' kernel and waits for its
// end. Bound by latency: launch, tile list, two or three rounds of loads, join: 2 us after the rows' kernel.
// One sequence of 60000 keys with one kv head of 8 query heads, 304 partial results of one tile: 13.3 us in
// all, against 52.7 with the last CTA joining them alone.
template <int D>
__global__ void __launch_bounds__(128) fa_paged_join_rows_kernel(const PagedFwd p) {
  constexpr int kPieces = D / 32, kMost = row_ctas(D, 16) * kPagedSms, kParts = 16;
  __shared__ RowShare share[kMost];
  __shared__ short first[kMost];  // of the tiles that are shared: their first CTA
  __shared__ int count[4];
  __shared__ float4 acc_s[kParts][8];
  __shared__ float stat_s[kParts][3];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the rows' kernel is complete
  const PagedBatch& b = p.b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rows_max = b.row_tile;
  const int ctas = row_ctas(D, rows_max) * b.sms;
  constexpr int kEach = (kMost + 127) / 128;
  RowShare mine[kEach];
  uint32_t some[kEach];
  int n = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    mine[i].c1 = -1;
    if (i * 128 + tid < ctas) mine[i] = p.row_share[i * 128 + tid];
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    some[i] = __ballot_sync(0xffffffffu, mine[i].c1 >= 0);
    n += __popc(some[i]);
  }
  if (lane == 0) count[warp] = n;
  __syncthreads();
  int at = 0, total = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    at += w < warp ? count[w] : 0;
    total += count[w];
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (mine[i].c1 >= 0) {
      const int x = at + __popc(some[i] & ((1u << lane) - 1));
      share[x] = mine[i];
      first[x] = (short)(i * 128 + tid);
    }
    at += __popc(some[i]);
  }
  __syncthreads();
  const int part = tid >> 3, col = (tid & 7) * 4;
  for (int x = blockIdx.x; x < total * rows_max * kPieces; x += gridDim.x) {
    const int tile = x / (rows_max * kPieces), rest = x % (rows_max * kPieces);
    const int row = rest / kPieces, col0 = rest % kPieces * 32 + col;
    const RowShare s = share[tile];
    const int c0 = first[tile];
    if (row >= s.rows) continue;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float m0 = -INFINITY, ls = 0.f, lr = 0.f;
    constexpr int kAtOnce = 4;
    for (int c = c0 + part; c <= s.c1; c += kAtOnce * kParts) {
      float4 v[kAtOnce];
      float mi[kAtOnce], si[kAtOnce], ri[kAtOnce], mx = m0;
#pragma unroll
      for (int y = 0; y < kAtOnce; ++y) {
        const int cc = min(c + y * kParts, s.c1);
        const float* src = p.part + (size_t)(2 * cc + (cc == c0 ? 1 : 0)) * row_part(D, rows_max);
        v[y] = *reinterpret_cast<const float4*>(src + row * D + col0);
        mi[y] = c + y * kParts <= s.c1 ? src[rows_max * D + row] : -INFINITY;
        si[y] = src[rows_max * (D + 1) + row];
        ri[y] = src[rows_max * (D + 2) + row];
      }
#pragma unroll
      for (int y = 0; y < kAtOnce; ++y) mx = fmaxf(mx, mi[y]);
      const float mu = mx == -INFINITY ? 0.f : mx, f0 = ex2(m0 - mu);
      m0 = mx;
      a = make_float4(a.x * f0, a.y * f0, a.z * f0, a.w * f0);
      ls *= f0;
      lr *= f0;
#pragma unroll
      for (int y = 0; y < kAtOnce; ++y) {
        if (c + y * kParts > s.c1) continue;
        const float f = ex2(mi[y] - mu);
        a.x = fmaf(f, v[y].x, a.x);
        a.y = fmaf(f, v[y].y, a.y);
        a.z = fmaf(f, v[y].z, a.z);
        a.w = fmaf(f, v[y].w, a.w);
        ls = fmaf(f, si[y], ls);
        lr = fmaf(f, ri[y], lr);
      }
    }
    __syncthreads();  // the last piece's sums have been read
    acc_s[part][tid & 7] = a;
    if ((tid & 7) == 0) {
      stat_s[part][0] = m0;
      stat_s[part][1] = ls;
      stat_s[part][2] = lr;
    }
    __syncthreads();
    if (part == 0) {
      float M = -INFINITY, Ls = 0.f, Lr = 0.f;
#pragma unroll
      for (int y = 0; y < kParts; ++y) M = fmaxf(M, stat_s[y][0]);
      const float mu = M == -INFINITY ? 0.f : M;
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int y = 0; y < kParts; ++y) {
        const float f = ex2(stat_s[y][0] - mu);
        const float4 v = acc_s[y][tid];
        Ls = fmaf(f, stat_s[y][1], Ls);
        Lr = fmaf(f, stat_s[y][2], Lr);
        t.x = fmaf(f, v.x, t.x);
        t.y = fmaf(f, v.y, t.y);
        t.z = fmaf(f, v.z, t.z);
        t.w = fmaf(f, v.w, t.w);
      }
      const unsigned rr = (unsigned)s.r0 + row, G = b.G;
      const int tok = (int)(rr / G), hd = (int)(rr - tok * G);
      const long long out = (long long)(s.q0 + tok) * b.Hq + s.head * (int)G + hd;
      const float inv = Lr > 0.f || Lr != Lr ? 1.f / Lr : 0.f;
      uint2 w;
      w.x = pack_bf16(t.x * inv, t.y * inv);
      w.y = pack_bf16(t.z * inv, t.w * inv);
      *reinterpret_cast<uint2*>(p.o + out * D + col0) = w;
      if (col0 == 0) p.lse[out] = (M + log2f(Ls)) * 0.6931471805599453f;
    }
  }
}

template <int D, int MT>
static cudaError_t launch_rows(const PagedFwd& p, int num_sms, cudaStream_t st) {
  constexpr int smem = RowSmem<D, MT>::kBytes;
  static unsigned long long known[kMaxGpus];
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(fa_paged_rows_kernel<D, MT>), smem, known);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(RowSmem<D, MT>::kCtas * num_sms);
  cfg.blockDim = dim3(kRowThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  // After the pairs' kernel: start on the SMs that it leaves free (what is read of it comes after a wait).
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = p.tile_ctas > 0 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, fa_paged_rows_kernel<D, MT>, p);
  if (e != cudaSuccess || p.row_share == nullptr) return e;
  cfg.gridDim = dim3(8 * num_sms);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_paged_join_rows_kernel<D>, p);
}

size_t paged_rows_workspace_bytes(int d, int row_tile) {
  const size_t ctas = (size_t)row_ctas(d, row_tile) * kPagedSms;
  return plan_up(2 * ctas * row_part(d, row_tile) * 4) + plan_up(ctas * sizeof(RowShare));
}

cudaError_t launch_paged_rows(const PagedFwd& p, int d, int num_sms, cudaStream_t st) {
  if (d == 128) return p.b.row_tile == 16 ? launch_rows<128, 1>(p, num_sms, st) : launch_rows<128, 2>(p, num_sms, st);
  return p.b.row_tile == 16 ? launch_rows<64, 1>(p, num_sms, st) : launch_rows<64, 2>(p, num_sms, st);
}

}  // namespace fa
