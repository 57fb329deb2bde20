// fa_paged_tiles.cu -- attention of chunks of new tokens over a paged cache, on the tensor cores' own
// memory: pairs of 128-row tiles against 128-key blocks with tcgen05 (the mathematics, the plan and the
// division among CTAs are in fa_paged.cu and fa_paged.cuh).
//
// A row is one query head of one new token; a tile's rows are 128 / G tokens times the G heads that
// share a kv head, so short chunks fill a tile and each key block is loaded once for all of them. One
// CTA per SM works off its stretch of the plan's units:
//   warp 8     TMA producer: the pair's queries, then per block the keys and values, one box per page
//              (lane i brings page i of the block; the table entries of the next block are read ahead).
//              Boxes of pages that no row sees are zero-filled without looking at the table.
//   warp 9     MMA issue: S_t = Q_t K^T, O_t += P_t V, the two tiles taking turns. At d = 64, where a
//              sequence has rows for one tile only, both tiles work on it, each on every other key block, so
//              that one half's products still run beside the other's softmax; the halves are joined at the end.
//   warps 0-7  softmax, one row per thread, four warps per tile: running max and sum in base 2, the
//              reference max moved only when a row outgrows it by 2^8, P as bf16 over the scores'
//              columns, and the rounding of each tile's largest weight carried along as in the dense
//              forward, so that o is not off where one key dominates.
// Slots past the sequence, and before the window of its first new token, hold anything, NaN too, and 0 * NaN is
// NaN: pages of such slots alone are not read (zeros stand for them), and where a page holds both, the rows of V
// past the last key and before the pair's first are set to zero in shared memory before the product.
// A pair that several CTAs share leaves unnormalised sums in the workspace, the rows of a warp side by
// side; the kernel that follows joins them in the order of the keys (fa_paged.cu).
//
// Bound by the loop of score product, softmax and P V, as in the dense forward: 1.52 us per block of both
// tiles at d = 128 (1.55 in a mixed batch, beside the small tiles' reads), where the products alone take 1.3 at the
// measured bf16 peak. 512 tokens over 32768 keys (32 query heads, 8 kv heads) take 191 us, 1430 TFLOP/s or 74 % of
// that peak: 4.4 us until the first scores, 165 in the loop, 3 to 4 per further stretch, 9 for the join. L2 serves
// 71 % of what the loop loads.
#include <cudaTypedefs.h>
#include <math.h>

#include "fa_paged.cuh"

namespace fa {

constexpr int kTileThreads = 320;
constexpr uint32_t kTileTmemCols = 512;
constexpr float kTileRescale = 8.f;

constexpr int kSegSlots = 4;

// A stretch as the producer hands it to the other warps: the blocks that each tile of its pair has work
// in, cnt of them from block j0 + a on, `step` apart.
struct TileSeg {
  int n_max;  // blocks that some tile has work in; -1: the end of the CTA's stretches
  int j0, a[2], cnt[2], step, exists[2];
  int head, q0, ql, kvl, t0;
  int turn;  // block j of the order is j0 + (j + turn) mod n_max
  int first, last, c0, c1;
};

template <int D>
struct TileSmem {
  static constexpr int NK = D == 128 ? 2 : 4, NV = NK;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + 2 * kTileBytes;
  static constexpr int kV = kK + NK * kTileBytes;
  static constexpr int kOStage = kV + NV * kTileBytes;  // d = 128: 4 KB per softmax warp, 32 rows x 64 columns
  static constexpr int kHalf = kOStage;  // d = 64: m, l, e of tile 1's half, one row per thread
  static constexpr int kBar = kOStage + (D == 128 ? 8 * 4096 : kTile * 16);
  static constexpr int bQ = 0;
  static constexpr int bKFull = bQ + 2;
  static constexpr int bKEmpty = bKFull + NK;
  static constexpr int bVFull = bKEmpty + NK;
  static constexpr int bVEmpty = bVFull + NV;
  static constexpr int bSFull = bVEmpty + NV;
  static constexpr int bPFull = bSFull + 2;
  static constexpr int bOFull = bPFull + 2;
  static constexpr int bQEmpty = bOFull + 2;
  static constexpr int bOFree = bQEmpty + 2;
  static constexpr int bSegFull = bOFree + 2;
  static constexpr int bSegEmpty = bSegFull + kSegSlots;
  static constexpr int bTwin = bSegEmpty + kSegSlots;  // tile 1's half is done, and has been taken over
  static constexpr int bTwinFree = bTwin + 1;
  static constexpr int bDrain = bTwinFree + 1;
  static constexpr int kNumBars = bDrain + 1;
  static constexpr int kTmemSlot = kBar + kNumBars * 8;
  static constexpr int kAbort = kTmemSlot + 4;
  static constexpr int kSeg = kAbort + 4;  // ring of stretches
  static constexpr int kBytes = kSeg + kSegSlots * sizeof(TileSeg);
  static constexpr int kAlloc = kBytes + 1024;
};

template <bool kTurn>
__device__ __forceinline__ TileSeg tile_seg(const Seg& s, const PagedBatch& p) {
  TileSeg it;
  const int tpt = p.pair_tokens >> 1;
  int lo[2], hi[2];
  bool any = false;
  it.j0 = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int t0 = s.t0 + t * tpt;
    it.exists[t] = t0 < s.ql;
    lo[t] = hi[t] = 0;
    if (!it.exists[t]) continue;
    int k0, k1;
    key_range(t0, min(t0 + tpt, s.ql) - 1, s.ql, s.kvl, p.causal, p.window, k0, k1);
    lo[t] = max(k0 / kPairBlk, s.blk);
    hi[t] = min((k1 + kPairBlk - 1) / kPairBlk, s.blk + s.n);
    if (k1 <= k0 || hi[t] < lo[t]) hi[t] = lo[t];
    if (hi[t] > lo[t]) {
      it.j0 = any ? min(it.j0, lo[t]) : lo[t];
      any = true;
    }
  }
  it.n_max = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    it.a[t] = hi[t] > lo[t] ? lo[t] - it.j0 : 0;
    it.cnt[t] = hi[t] - lo[t];
    it.n_max = max(it.n_max, it.a[t] + it.cnt[t]);
  }
  it.step = 1;
  if (halves(s.t0, s.t1, p) && it.n_max >= 2) {  // one tile of rows: both work on it, each on every other block
    it.step = 2;
    it.a[1] = 1;
    it.cnt[0] = (it.n_max + 1) / 2;
    it.cnt[1] = it.n_max / 2;
    it.exists[1] = 1;
  }
  // Where both tiles have all the blocks, their order is free. CTAs that work on other rows of the same keys
  // then start at the same keys (Seg::turn), which so come from memory about once instead of once per pair.
  const bool both = it.step == 1 && it.exists[1] && it.a[0] + it.a[1] == 0 && it.cnt[0] == it.n_max &&
                    it.cnt[1] == it.n_max;
  it.turn = kTurn && both && it.n_max == s.n ? s.turn : 0;
  it.head = s.head;
  it.q0 = s.q0;
  it.ql = s.ql;
  it.kvl = s.kvl;
  it.t0 = s.t0;
  it.first = s.first;
  it.last = s.last;
  it.c0 = s.c0;
  it.c1 = s.c1;
  return it;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

__device__ __forceinline__ float max64f(const uint32_t (&a)[32], const uint32_t (&b)[32], float init) {
  float m[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    m[k] = max3f(__uint_as_float(a[k]), __uint_as_float(a[k + 8]), __uint_as_float(a[k + 16]));
    m[k] = max3f(m[k], __uint_as_float(a[k + 24]), __uint_as_float(b[k]));
    m[k] = max3f(m[k], __uint_as_float(b[k + 8]), __uint_as_float(b[k + 16]));
    m[k] = fmaxf(m[k], __uint_as_float(b[k + 24]));
  }
  return max3f(max3f(m[0], m[1], m[2]), max3f(m[3], m[4], m[5]), max3f(m[6], m[7], init));
}

template <int D, bool kTurn>
__global__ void __launch_bounds__(kTileThreads, 1)
    fa_paged_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                          const PagedFwd p) {
  using L = TileSmem<D>;
  constexpr bool kHalves = D == 64;  // see halves() in fa_paged.cuh
  constexpr bool kBoxOut = D == 128;
  constexpr int NK = L::NK, NV = L::NV;
  const PagedBatch& b = p.b;
  SegIter<true> walk(b, max(1, pair_sms(b)));  // (its loads and the plan's check go out together)
  if (!plan_matches(b, D)) {
    if (threadIdx.x == 0) record_index_error(b.status);
    return;
  }
  if (threadIdx.x < 2) p.share[2 * blockIdx.x + threadIdx.x].c1 = -1;
  if (walk.u >= walk.u_end) return;  // no work for this CTA
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + L::kQ, sK = sbase + L::kK, sV = sbase + L::kV;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmemSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
  TileSeg* segs = reinterpret_cast<TileSeg*>(smem + L::kSeg);
  const Ctl ctl{abort_flag, b.status};
  auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8u * (uint32_t)i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tpt = b.pair_tokens >> 1;  // tokens per tile; rows tpt * G .. 127 are unused
  const int used = tpt * b.G;

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(L::bQ + t), 1);
      mbar_init(bar(L::bSFull + t), 1);
      mbar_init(bar(L::bPFull + t), 128);
      mbar_init(bar(L::bOFull + t), 1);
      mbar_init(bar(L::bQEmpty + t), 1);
      mbar_init(bar(L::bOFree + t), 128);
    }
    for (int s = 0; s < NK; ++s) {
      mbar_init(bar(L::bKFull + s), 1);
      mbar_init(bar(L::bKEmpty + s), 1);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(bar(L::bVFull + s), 1);
      mbar_init(bar(L::bVEmpty + s), 1);
    }
    for (int s = 0; s < kSegSlots; ++s) {
      mbar_init(bar(L::bSegFull + s), 1);
      mbar_init(bar(L::bSegEmpty + s), 9);  // the MMA warp and the eight softmax warps
    }
    mbar_init(bar(L::bTwin), 128);
    mbar_init(bar(L::bTwinFree), 128);
    mbar_init(bar(L::bDrain), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    if (kBoxOut && p.warp_out) tma_prefetch_desc(&tm_o);
  }
  // Rows that no load fills are zero, so that their scores are.
  for (int i = threadIdx.x; i < 2 * (D / 64) * (kTile - used) * 8; i += kTileThreads) {
    const int part = i / ((kTile - used) * 8), at = i - part * ((kTile - used) * 8);
    st_shared_v4(sQ + part * 16384 + used * 128 + at * 16, 0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), kTileTmemCols);
    tmem_relinquish();
  }
  // The producer's stretch: its place in the batch, the blocks of its tiles, and the table entry of this
  // lane's box of the next block to load. Found here for the first time, beside the setup.
  Seg s;
  TileSeg it;
  struct Look {
    const int* tab;
    int lo, hi;
  } cur = {nullptr, 0, 0};
  int entry = 0;
  bool seen = false;  // a row sees a key of the box (else its entry is not read)
  const int box = b.page_size < kPairBlk ? b.page_size : kPairBlk;  // keys of one box
  const int nbox = kPairBlk / box;
  auto read_entry = [&](int blk) {
    const int key = blk * kPairBlk + lane * box;
    seen = lane < nbox && key < cur.hi && key + box > cur.lo;
    if (seen) entry = cur.tab[key >> b.page_shift];
  };
  auto page_at = [&]() -> int {  // num_pages lies beyond the map: zeros
    if (seen && (unsigned)entry < (unsigned)b.num_pages) return entry;
    if (seen) record_index_error(b.status);
    return b.num_pages;
  };
  auto look = [&]() {
    it.n_max = -1;
    if (!walk.next(s)) return;
    it = tile_seg<kTurn>(s, b);
    key_range(s.t0, s.t1, s.ql, s.kvl, b.causal, b.window, cur.lo, cur.hi);
    cur.tab = b.table + (long long)s.seq * b.table_stride;
    if (it.n_max > 0) read_entry(it.j0 + it.turn);
  };
  if (warp == 8) look();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the next kernel may start on SMs left free

  // Stretch i of the CTA, once the producer has handed it out; and its slot given back.
  auto take = [&](uint32_t i) -> const TileSeg* {
    return mbar_wait_warp(bar(L::bSegFull + i % kSegSlots), (i / kSegSlots) & 1, ctl) ? segs + i % kSegSlots : nullptr;
  };
  auto give_back = [&](uint32_t i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(L::bSegEmpty + i % kSegSlots));
  };
  if (warp == 8) {
    // ------------------------------------------------------------------ TMA producer
    const uint32_t q_bytes = (uint32_t)used * D * 2;
    uint32_t gk = 0, gv = 0, qn[2] = {0, 0};
    uint32_t handed = 0;
    bool ok = true, next_seen = false;
    int next_entry = 0;
    Look keep, nxt = cur;
    auto hand_out = [&]() -> bool {
      if (!mbar_wait_warp(bar(L::bSegEmpty + handed % kSegSlots), ((handed / kSegSlots) & 1) ^ 1, ctl)) return false;
      if (lane == 0) {
        segs[handed % kSegSlots] = it;
        mbar_arrive(bar(L::bSegFull + handed % kSegSlots));
      }
      ++handed;
      return true;
    };
    ok = hand_out();
    while (ok && it.n_max >= 0) {
      const int head = s.head, tok = s.q0 + s.t0, j0 = it.j0, n_max = it.n_max, turn = it.turn;
      int blk = kTurn ? j0 + turn : j0;
      const bool with[2] = {it.cnt[0] > 0, it.cnt[1] > 0};
      const int tile_tok = it.step == 1 ? tpt : 0;  // from tile 0's tokens to tile 1's
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (!ok || !with[t]) continue;
        if (!(ok = mbar_wait_warp(bar(L::bQEmpty + t), (qn[t] & 1) ^ 1, ctl))) continue;
        if (lane == 0) {
          mbar_expect_tx(bar(L::bQ + t), q_bytes);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(sQ + t * L::kTileBytes + c * 16384, &tm_q, bar(L::bQ + t), c * 64, head * b.G,
                        tok + t * tile_tok);
        }
        ++qn[t];
      }
      if (n_max == 0) {  // no tile sees a key: nothing to load
        look();
        if (ok) ok = hand_out();
        continue;
      }
      for (int j = 0; ok && j < n_max; ++j) {
        const int slot = (blk * kPairBlk + lane * box) & (b.page_size - 1);
        const int pg = page_at();
        ++blk;
        if (kTurn && blk == j0 + n_max) blk = j0;
        if (j + 1 < n_max) read_entry(blk);
        const uint32_t sk = gk % NK, sv = gv % NV;
        if (!(ok = mbar_wait_warp(bar(L::bKEmpty + sk), ((gk / NK) & 1) ^ 1, ctl))) break;
        if (lane == 0) mbar_expect_tx(bar(L::bKFull + sk), L::kTileBytes);
        __syncwarp();
        if (lane < nbox) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(sK + sk * L::kTileBytes + c * 16384 + lane * box * 128, &tm_k, bar(L::bKFull + sk), c * 64, slot,
                        head, pg);
        }
        ++gk;
        if (!(ok = mbar_wait_warp(bar(L::bVEmpty + sv), ((gv / NV) & 1) ^ 1, ctl))) break;
        if (lane == 0) mbar_expect_tx(bar(L::bVFull + sv), L::kTileBytes);
        __syncwarp();
        if (lane < nbox) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(sV + sv * L::kTileBytes + c * 16384 + lane * box * 128, &tm_v, bar(L::bVFull + sv), c * 64, slot,
                        head, pg);
        }
        ++gv;
        if (j == 0) {
          // The next stretch is looked up and handed out early, so that at the end of this one its
          // queries load as soon as their buffers are free. (This one's next table entry is in hand.)
          const int e = entry;
          const bool sn = seen;
          keep = cur;
          look();
          next_entry = entry;
          next_seen = seen;
          entry = e;
          seen = sn;
          nxt = cur;
          cur = keep;
          if (!(ok = hand_out())) break;
        }
      }
      cur = nxt;
      entry = next_entry;
      seen = next_seen;
    }
    if (*abort_flag && lane == 0) {  // every copy in flight lands before shared memory is freed
      for (int t = 0; t < 2; ++t)
        if (qn[t] > 0) drain_wait(bar(L::bQ + t), (qn[t] - 1) & 1);
      for (uint32_t g = gk > NK ? gk - NK : 0; g < gk; ++g) drain_wait(bar(L::bKFull + g % NK), (g / NK) & 1);
      for (uint32_t g = gv > NV ? gv - NV : 0; g < gv; ++g) drain_wait(bar(L::bVFull + g % NV), (g / NV) & 1);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------------ MMA issue
    constexpr uint32_t idS = idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t idO = idesc_bf16_f32(128, D, false, true);
    const uint64_t dQ = sdesc_sw128(sQ, 16, 1024);
    const uint64_t dK = sdesc_sw128(sK, 16, 1024);
    const uint64_t dV = sdesc_sw128(sV, 16384, 1024);
    uint32_t gk = 0, gv = 0, qn[2] = {0, 0}, pc[2] = {0, 0};
    auto commit = [&](uint32_t x) {
      if (elect_one()) mma_commit(x);
      __syncwarp();
    };
    auto issue_s = [&](int t, uint32_t g, bool ready) -> bool {
      const uint32_t sk = g % NK;
      if (!ready && !mbar_wait_warp(bar(L::bKFull + sk), (g / NK) & 1, ctl)) return false;
      tc_fence_after();
      const uint64_t a = dQ + (uint32_t)(t * (L::kTileBytes >> 4));
      const uint64_t bk = dK + sk * (uint32_t)(L::kTileBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
          mma_ss(tmem + 128 * t, a + off, bk + off, idS, kk > 0);
        }
        mma_commit(bar(L::bSFull + t));
      }
      __syncwarp();
      return true;
    };
    auto issue_pv = [&](int t, uint32_t g, bool first, bool last, bool ready) -> bool {
      const uint32_t sv = g % NV;
      if (!mbar_wait_warp(bar(L::bPFull + t), pc[t] & 1, ctl)) return false;
      if (!ready && !mbar_wait_warp(bar(L::bVFull + sv), (g / NV) & 1, ctl)) return false;
      if (first && qn[t] > 1 && !mbar_wait_warp(bar(L::bOFree + t), (qn[t] - 2) & 1, ctl)) return false;
      tc_fence_after();
      const uint64_t bv = dV + sv * (uint32_t)(L::kTileBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          mma_ts(tmem + 256 + 128 * t, tmem + 128 * t + kk * 8, bv + (uint32_t)(kk * (2048 >> 4)), idO,
                 (!first || kk > 0));
        if (last) mma_commit(bar(L::bOFull + t));
      }
      __syncwarp();
      ++pc[t];
      return true;
    };
    bool ok = true;
    for (uint32_t i = 0; ok; ++i) {
      const TileSeg* sp = take(i);
      if (sp == nullptr) break;
      const TileSeg it = *sp;
      give_back(i);
      if (it.n_max < 0) break;
      if (it.n_max == 0) continue;
      const int step = kHalves ? it.step : 1;
      const int end[2] = {it.a[0] + (it.cnt[0] - 1) * step, it.a[1] + (it.cnt[1] - 1) * step};  // last blocks
      auto has = [&](int t, int j) {
        return it.cnt[t] > 0 && it.a[t] <= j && j <= end[t] && !((j - it.a[t]) & (step - 1));
      };
      bool k_ready = false;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (!ok || it.cnt[t] == 0) continue;
        if (!(ok = mbar_wait_warp(bar(L::bQ + t), qn[t] & 1, ctl))) continue;
        ++qn[t];
        tc_fence_after();
        if (it.a[t] < step) {
          if (!(ok = issue_s(t, gk + it.a[t], k_ready && step == 1))) continue;
          k_ready = true;
          if (it.cnt[t] == 1) commit(bar(L::bQEmpty + t));
        }
      }
      if (!ok) break;
      commit(bar(L::bKEmpty + gk % NK));
      if (step == 2) commit(bar(L::bKEmpty + (gk + 1) % NK));
      for (int j = 0; ok && j < it.n_max; ++j) {
        bool v_ready = false, k_next_ready = false;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (ok && has(t, j)) {
            if (!(ok = issue_pv(t, gv + j, j == it.a[t], j == end[t], v_ready))) continue;
            v_ready = true;
          }
          if (ok && has(t, j + step)) {
            if (!(ok = issue_s(t, gk + j + step, k_next_ready))) continue;
            k_next_ready = true;
            if (j + step == end[t]) commit(bar(L::bQEmpty + t));
          }
        }
        if (!ok) break;
        commit(bar(L::bVEmpty + (gv + j) % NV));
        if (j + step < it.n_max) commit(bar(L::bKEmpty + (gk + j + step) % NK));
      }
      gk += it.n_max;
      gv += it.n_max;
    }
    if (*abort_flag) {
      if (elect_one()) {
        mma_commit(bar(L::bDrain));
        drain_wait(bar(L::bDrain), 0);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------------ softmax
    const int t = warp >> 2;
    const int r = threadIdx.x & 127;  // row within the tile
    const int r_tok = r / b.G, r_head = r - r_tok * b.G;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + 128 * t + lane_off;
    const uint32_t tO = tmem + 256 + 128 * t + lane_off;
    const float sl2 = p.scale_log2;
    uint32_t sc = 0, on = 0, gv = 0;
    uint32_t twins = 0;  // stretches so far whose two halves were joined here
    bool owed = false;   // (tile 1) its half of the last one has not been taken over yet
    bool ok = true;
    auto row_out = [&](int q0, int tok, int ql, int head) -> long long {
      return r < used && tok < ql ? (long long)(q0 + tok) * b.Hq + head * b.G + r_head : -1;
    };
    for (uint32_t i = 0; ok; ++i) {
      const TileSeg* sp = take(i);
      if (sp == nullptr) {
        ok = false;
        break;
      }
      const TileSeg& s = *sp;
      const int n_max = s.n_max;
      if (n_max < 0) break;
      const uint32_t gv0 = gv;
      gv += n_max;
      if (!s.exists[t]) {
        give_back(i);
        continue;
      }
      const int a_t = s.a[t], n_kv = s.cnt[t], step = kHalves ? s.step : 1;
      const bool twin = kHalves && step == 2;
      const int kv_first = (s.j0 + a_t) * kPairBlk, kvl = s.kvl, turn = s.turn;
      const int tok0 = s.t0 + (twin ? 0 : t * tpt);
      const int tok = tok0 + r_tok;
      const int pos = kvl - s.ql + tok;
      const int klim = min(kvl - 1, b.causal ? pos : kvl - 1);
      const int klo = mask_from(pos, b.window);
      const int pos0 = kvl - s.ql + tok0, pos1 = pos0 + tpt - 1;
      // A warp whose rows all lie past the tile's tokens only keeps the barriers going. (At d = 128 such a
      // CTA waits for memory, and the test cost long chunks 2 %.)
      const bool idle = kHalves && (warp & 3) * 32 >= min(used, (s.ql - tok0) * b.G);
      // Rows of V that no row of the pair sees, past the last key and before the first token's window (both tiles
      // may write the same zeros): after the copy has landed, before the product that the arrival at bPFull lets
      // start. At d = 128 it is called for all masked blocks and looks for such rows itself: a bound held in a
      // register all along costs 0.3 % there. At d = 64 that is sooner (4 x 512 tokens over 8192 keys: 175.1 us, 176.2 the
      // other way; 48 x 40 over 3000 with a window of 200: 40.7 and 41.5).
      auto pair_lo = [&]() { return first_key(kvl - s.ql + s.t0, b.window); };
      const int vlo = kHalves ? pair_lo() : 0;
      auto clear_unseen = [&](int j, int kv0) -> bool {
        const int past = kvl - kv0, before = min((kHalves ? vlo : pair_lo()) - kv0, kPairBlk);
        if (past >= kPairBlk && before <= 0) return true;
        const uint32_t g = gv0 + a_t + j * step, sv = g % NV;
        if (!mbar_wait_warp(bar(L::bVFull + sv), (g / NV) & 1, ctl)) return false;
        auto clear = [&](int row) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            st_shared_v4(sV + sv * L::kTileBytes + c * 16384 + row * 128 + (r & 7) * 16, 0, 0, 0, 0);
        };
        for (int row = r >> 3; row < before; row += 16) clear(row);
        for (int row = past + (r >> 3); row < kPairBlk; row += 16) clear(row);
        fence_proxy_async_smem();
        return true;
      };
      float m_run = -INFINITY, m_hi = -INFINITY, l_run = 0.f, e_run = 0.f;
      for (int j = 0; j < n_kv; ++j) {
        if (!mbar_wait_warp(bar(L::bSFull + t), (sc + j) & 1, ctl)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // (turn > 0: step is 1, and both tiles have all the blocks)
        const int x = !kTurn ? j : (j + turn < n_kv ? j + turn : j + turn - n_kv);
        const int kv0 = kv_first + x * step * kPairBlk;
        const bool need_mask = kv0 + kPairBlk > kvl || (b.causal && kv0 + kPairBlk - 1 > pos0) ||
                               (b.window > 0 && kv0 < mask_from(pos1, b.window));
        const bool edge = kHalves ? kv0 + kPairBlk > kvl || kv0 < vlo : need_mask;
        if (idle) {
          if (edge && !(ok = clear_unseen(j, kv0))) break;
          mbar_arrive(bar(L::bPFull + t));
          continue;
        }
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, sr[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait(sr[c]);
        if (need_mask) {
          const int lim = klim - kv0, lo = klo - kv0;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c * 32 + i > lim || c * 32 + i < lo) sr[c][i] = 0xff800000u;
        }
        const float mx = max64f(sr[2], sr[3], max64f(sr[0], sr[1], -INFINITY));
        const float mt = mx * sl2;
        m_hi = fmaxf(m_hi, mt);
        const bool resc = __any_sync(0xffffffffu, m_hi > m_run + kTileRescale);
        const float m_new = resc ? m_hi : m_run;
        const float corr = (m_new > m_run) ? ex2(m_run - m_new) : 1.f;
        m_run = m_new;
        const float m_use = (m_run == -INFINITY) ? 0.f : m_run;
        {
          const float pmx = ex2(fmaf(mx, sl2, -m_use));
          e_run = e_run * corr + (__uint_as_float(pack_bf16(pmx, 0.f) << 16) - pmx);
        }
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 sl2x2 = make_float2(sl2, sl2), negm = make_float2(-m_use, -m_use);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 x = fma2(make_float2(__uint_as_float(sr[c][i]), __uint_as_float(sr[c][i + 1])), sl2x2, negm);
            const float2 pp = make_float2(ex2(x.x), ex2(x.y));
            sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], pp);
            pk[i >> 1] = pack_bf16(pp.x, pp.y);
          }
          tmem_st16(tS + c * 16, pk);
        }
        if (j > 0 && resc) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + c * 32, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 v = mul2(make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])),
                                    make_float2(corr, corr));
              o[i] = __float_as_uint(v.x);
              o[i + 1] = __float_as_uint(v.y);
            }
            tmem_st32(tO + c * 32, o);
          }
        }
        l_run = l_run * corr + ((sum[0].x + sum[1].x) + (sum[0].y + sum[1].y));
        if (edge && !(ok = clear_unseen(j, kv0))) break;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(L::bPFull + t));
      }
      if (!ok) break;
      // ---------------------------------------------------------------- epilogue
      if (n_kv > 0) {
        if (!(ok = mbar_wait_warp(bar(L::bOFull + t), on & 1, ctl))) break;
        ++on;
        sc += n_kv;
        tc_fence_after();
      }
      const TileSeg e = s;
      give_back(i);  // before the stores: an arrival after them would wait for them
      if (kHalves && owed) {  // this warp's buffer still holds its half of an earlier stretch
        if (!(ok = mbar_wait_warp(bar(L::bTwinFree), (twins - 1) & 1, ctl))) break;
        owed = false;
      }
      float4* half = reinterpret_cast<float4*>(smem + L::kHalf) + r;
      if (twin && t == 1) {  // over to tile 0: o stays in tensor memory
        *half = make_float4(m_run, l_run, e_run, 0.f);
        tc_fence_before();
        mbar_arrive(bar(L::bTwin));
        ++twins;
        owed = true;
        continue;
      }
      float f0 = 1.f, f1 = 0.f;
      if (twin) {
        if (!(ok = mbar_wait_warp(bar(L::bTwin), twins & 1, ctl))) break;
        ++twins;
        tc_fence_after();
        const float4 h = *half;
        const float mn = fmaxf(m_run, h.x), mu = mn == -INFINITY ? 0.f : mn;
        f0 = ex2(m_run - mu);
        f1 = ex2(h.x - mu);
        m_run = mn;
        l_run = l_run * f0 + h.y * f1;
        e_run = e_run * f0 + h.z * f1;
      }
      auto read_o = [&](uint32_t (&o)[D / 32][32]) {  // the row's sums
#pragma unroll
        for (int c = 0; c < D / 32; ++c) tmem_ld32(tO + c * 32, o[c]);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) tmem_ld_wait(o[c]);
        if (twin) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o1[32];
            tmem_ld32(tO + 128 + c * 32, o1);
            tmem_ld_wait(o1);
#pragma unroll
            for (int k = 0; k < 32; ++k)
              o[c][k] = __float_as_uint(__uint_as_float(o[c][k]) * f0 + __uint_as_float(o1[k]) * f1);
          }
        }
      };
      auto o_read = [&]() {  // the accumulators may be overwritten
        tc_fence_before();
        if (n_kv > 0) mbar_arrive(bar(L::bOFree + t));
        if (twin) {
          mbar_arrive(bar(L::bOFree + 1));
          mbar_arrive(bar(L::bTwinFree));
        }
      };
      if (idle) {
        o_read();
      } else if (e.first && e.last) {
        const float inv = (l_run > 0.f || l_run != l_run) ? 1.f / (l_run + e_run) : 0.f;  // nothing seen: o = 0
        uint32_t w[D / 2] = {};
        if (n_kv > 0) {
          uint32_t o[D / 32][32];
          read_o(o);
#pragma unroll
          for (int k = 0; k < D / 2; ++k) {
            const uint32_t* pair = &o[k >> 4][2 * k & 31];
            const float2 v = mul2(make_float2(__uint_as_float(pair[0]), __uint_as_float(pair[1])), make_float2(inv, inv));
            w[k] = pack_bf16(v.x, v.y);
          }
        }
        o_read();
        const long long out = row_out(e.q0, tok, e.ql, e.head);
        const bool box_out = kBoxOut && p.warp_out && __all_sync(0xffffffffu, out >= 0);
        // Out by a bulk tensor store where the warp's rows are a box of o, else each thread its row, 32 bytes (whole
        // sectors) at a time. At d = 128 the box is sooner for rows that it takes, at d = 64 no box is (16 x 2048
        // tokens, 32 heads, 8 kv heads, d = 128: 479 us, 501 without it; 16 x 1743 tokens, 16 heads, d = 64: 187,
        // 194 with it); both beat rows that go through shared memory to be stored by neighbouring threads (504, 199).
        if (box_out) {
          const uint32_t o_stage = sbase + L::kOStage + (uint32_t)warp * 4096;
          const int z = e.q0 + tok0 + (warp & 3) * 32 / b.G;  // the first row's token
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            if (lane == 0) bulk_wait_read_all();  // the last store from this buffer has read it
            __syncwarp();
#pragma unroll
            for (int g = 0; g < 8; ++g)
              st_shared_v4(o_stage + (uint32_t)lane * 128 + ((g ^ (lane & 7)) << 4), w[32 * c + 4 * g],
                           w[32 * c + 4 * g + 1], w[32 * c + 4 * g + 2], w[32 * c + 4 * g + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(&tm_o, o_stage, c * 64, e.head * b.G, z);
              bulk_commit_group();
            }
          }
          p.lse[out] = (m_run + log2f(l_run)) * 0.6931471805599453f;
        } else if (out >= 0) {
          uint8_t* dst = reinterpret_cast<uint8_t*>(p.o + out * D);
          if (p.o_wide) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) st_global_v8(dst + 32 * k, w + 8 * k);
          } else {
#pragma unroll
            for (int k = 0; k < D / 8; ++k)
              *reinterpret_cast<uint4*>(dst + 16 * k) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
          }
          p.lse[out] = (m_run + log2f(l_run)) * 0.6931471805599453f;
        }
      } else {
        float* slot = p.tile_part + (size_t)(2 * blockIdx.x + (e.first ? 1 : 0)) * tile_part(D) + t * kTile * (D + 3);
        if (n_kv > 0) {
          uint32_t o[D / 32][32];
          read_o(o);
#pragma unroll
          for (int k = 0; k < D / 4; ++k)
            *reinterpret_cast<uint4*>(slot + (k * kTile + r) * 4) =
                make_uint4(o[k >> 3][4 * k & 31], o[k >> 3][(4 * k & 31) + 1], o[k >> 3][(4 * k & 31) + 2],
                           o[k >> 3][(4 * k & 31) + 3]);
        }
        o_read();
        slot[D * kTile + r] = m_run;  // -inf: nothing seen here, and o is not there
        slot[(D + 1) * kTile + r] = l_run;
        slot[(D + 2) * kTile + r] = e_run;
        if (e.first && r == 0) p.share[2 * blockIdx.x + t] = TileShare{e.c1, e.q0, e.ql, tok0, e.head};
      }
    }
  }
  if (kBoxOut && warp < 8 && lane == 0) bulk_wait_read_all();  // before the CTA gives its shared memory up
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTileTmemCols);
  }
}

template <int D, bool kTurn>
static cudaError_t launch_tiles(const TileMaps& m, const PagedFwd& p, int num_sms, cudaStream_t st) {
  constexpr int smem = TileSmem<D>::kAlloc;
  static_assert(smem <= 232448, "shared memory exceeds the 227 KB per-CTA limit");
  static unsigned long long known[kMaxGpus];
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(fa_paged_tiles_kernel<D, kTurn>), smem, known);
  if (e != cudaSuccess) return e;
  fa_paged_tiles_kernel<D, kTurn><<<num_sms, kTileThreads, smem, st>>>(m.q, m.k, m.v, m.o, p);
  return cudaGetLastError();
}

size_t paged_tiles_workspace_bytes(int d) {
  return plan_up((size_t)2 * kPagedSms * tile_part(d) * 4) + plan_up((size_t)2 * kPagedSms * sizeof(TileShare));
}

// The turned order of blocks is for sequences whose keys and values may not stay in L2 (129 MB; counted as
// half of it, from the table's width): 512 tokens over 32768 keys of 8 kv heads take 190 us with it, 193 to
// 217 without, as the CTAs' starts happen to fall. Below that the order is free of cost, and the choice of a
// block per step is not: 16 x 1743 tokens take 232 us without it, 242 with.
cudaError_t launch_paged_tiles(const TileMaps& m, const PagedFwd& p, int d, int num_sms, cudaStream_t st) {
  const bool turn = (long long)p.b.max_pages * p.b.page_size * p.b.Hkv * d * 4 > (64LL << 20);
  if (d == 128) return turn ? launch_tiles<128, true>(m, p, num_sms, st) : launch_tiles<128, false>(m, p, num_sms, st);
  return turn ? launch_tiles<64, true>(m, p, num_sms, st) : launch_tiles<64, false>(m, p, num_sms, st);
}

}  // namespace fa
