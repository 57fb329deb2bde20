// fa_paged.cuh -- the plan of a ragged batch over a paged cache, and how a kernel's CTAs walk it.
//
// The plan is built on the device from the batch's lengths (fa_paged.cu), so no length is read back
// by the host and a captured graph follows new lengths. It holds each sequence's place, and per
// sequence the running sum of its work in units; CTA c of P takes the units [c * per, (c + 1) * per),
// per = ceil(W / P), whatever sequences and heads they belong to. So every CTA has the same number of
// key blocks however ragged the batch is, and only the first and the last item of a CTA can be part
// of a row tile that another CTA shares: at most two partial results per CTA, whatever the batch.
#pragma once

#include <stddef.h>

#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {

constexpr uint32_t kPlanMagic = 0x70a6ed01u;
constexpr int kPlanCtas = 512;  // most CTAs that a kernel over a plan may have (its merge counters)
constexpr int kPagedSms = 160;  // most SMs that are used: bounds the partial results without asking the device

// Row tiles of two kinds: 16 or 32 rows against 64-key blocks, and pairs of 128 rows against 128-key
// blocks. A row is one query head of one new token: row r of a (sequence, kv head) is token r / G,
// head r % G, so the heads that share keys share a tile.
constexpr int kRowBlk = 64;
constexpr int kPairBlk = 128;

struct PlanHeader {  // 64 words; what the plan was built for, checked by every kernel that reads it
  uint32_t magic;
  int S, T, max_q, Hq, Hkv, d, page_size, max_pages, causal, window;
  int pad[53];
};

struct PlanSeq {
  int q0, ql, kvl, pad;  // first token, new tokens, cached tokens with them
};

struct PlanView {
  PlanHeader* head;
  PlanSeq* seq;               // [S]
  long long* units[2];        // [S + 1] running sums: tiles of few rows, pairs
  uint32_t* counters;         // [kPlanCtas] arrivals at tiles of few rows that several CTAs share; zero between calls
};

__host__ __device__ inline size_t plan_up(size_t x) { return (x + 255) / 256 * 256; }

__host__ __device__ inline size_t plan_layout(void* base, int S, PlanView* v) {
  char* b = static_cast<char*>(base);
  size_t at = sizeof(PlanHeader);
  size_t off[4];
  off[0] = at;
  at += plan_up((size_t)S * sizeof(PlanSeq));
  for (int i = 0; i < 2; ++i) {
    off[1 + i] = at;
    at += plan_up(((size_t)S + 1) * 8);
  }
  off[3] = at;
  at += kPlanCtas * 4;
  if (v != nullptr) {
    v->head = reinterpret_cast<PlanHeader*>(b);
    v->seq = reinterpret_cast<PlanSeq*>(b + off[0]);
    for (int i = 0; i < 2; ++i) v->units[i] = reinterpret_cast<long long*>(b + off[1 + i]);
    v->counters = reinterpret_cast<uint32_t*>(b + off[3]);
  }
  return at;
}

// What a kernel needs of the batch (by value).
struct PagedBatch {
  PlanView plan;
  const int* table;  // [S][table_stride]
  long long table_stride;
  int S, T, max_q, Hq, Hkv, G, d, page_size, page_shift, max_pages, num_pages, causal, window;
  int pair_tokens;  // tokens of a pair of 128-row tiles: 2 * (128 / G)
  int sms;          // SMs in use: one CTA each for the pairs, two or three for the small tiles
  int row_tile;     // rows of the small tiles: 16, or 32 in batches with a sequence of more than 16
  float row_cost;   // time of a small tile's unit on an SM, counted in a pair's (pair_sms)
  uint32_t* status;
};

__device__ __forceinline__ void record_index_error(uint32_t* status) { atomicCAS(status, kStatusOk, kStatusIndex); }

// The plan was built for this batch (a stale or unset buffer would send indexes out of range). Three loads that go out
// together, and no branch between them.
__device__ __forceinline__ bool plan_matches(const PagedBatch& b, int d) {
  static_assert(offsetof(PlanHeader, Hq) == 16 && offsetof(PlanHeader, max_pages) == 32, "the header is read by fours");
  const int4* h = reinterpret_cast<const int4*>(b.plan.head);
  const int4 x = h[0], y = h[1], z = h[2];
  return (((uint32_t)x.x ^ kPlanMagic) | (uint32_t)((x.y ^ b.S) | (x.z ^ b.T) | (x.w ^ b.max_q) | (y.x ^ b.Hq) | (y.y ^ b.Hkv) |
                                                    (y.z ^ d) | (y.w ^ b.page_size) | (z.x ^ b.max_pages) |
                                                    (z.y ^ b.causal) | (z.z ^ b.window))) == 0;
}

// The first key that a query at `pos` sees. (No difference is formed for a window that reaches back to the first
// key: positions may be negative, and windows as large as an int.)
__host__ __device__ __forceinline__ int first_key(int pos, int window) {
  return window > 0 && pos >= window ? pos - window + 1 : 0;
}
// The same as a bound for masks, without the test: keys from it on are in the window. Negative where all are; it
// wraps only where pos is negative too, and such a query sees no key anyway. (first_key in its place: 191.9 us
// for 512 tokens over 32768 keys, 191.0 with this.)
__host__ __device__ __forceinline__ int mask_from(int pos, int window) {
  return window > 0 ? (int)((unsigned)pos - (unsigned)window + 1u) : 0;
}

// Keys [lo, hi) that some query of tokens [t0, t1] sees: token j stands at position kvl - ql + j and
// sees keys up to its own (causal) and after position - window (window > 0).
__host__ __device__ __forceinline__ void key_range(int t0, int t1, int ql, int kvl, int causal, int window, int& lo,
                                                   int& hi) {
  const int p0 = kvl - ql + t0, p1 = kvl - ql + t1;
  hi = causal ? (p1 + 1 < 0 ? 0 : p1 + 1) : kvl;
  lo = first_key(p0, window);
  if (lo > hi) lo = hi;
}

// Row tile `i` of a sequence: its tokens [t0, t1], and how many tiles there are. (ql * G fits an int:
// max_q * G is checked on the host.)
template <bool kPairs, int kRows = 0>  // kRows: the small tiles' rows, where the caller knows them
__host__ __device__ __forceinline__ int tile_count(int ql, const PagedBatch& b) {
  const unsigned rows = kRows ? kRows : b.row_tile;
  return kPairs ? (ql + b.pair_tokens - 1) / b.pair_tokens : (int)(((unsigned)ql * b.G + rows - 1) / rows);
}
template <bool kPairs, int kRows = 0>
__host__ __device__ __forceinline__ void tile_tokens(int i, int ql, const PagedBatch& b, int& t0, int& t1) {
  if (kPairs) {
    t0 = i * b.pair_tokens;
    t1 = (t0 + b.pair_tokens < ql ? t0 + b.pair_tokens : ql) - 1;
  } else {
    const unsigned rows = kRows ? kRows : b.row_tile, r0 = (unsigned)i * rows, R = (unsigned)ql * b.G;
    if (R <= rows) {  // one tile: no divisions
      t0 = 0;
      t1 = ql - 1;
      return;
    }
    const unsigned r1 = (r0 + rows < R ? r0 + rows : R) - 1;
    t0 = (int)(r0 / b.G);
    t1 = (int)(r1 / b.G);
  }
}
// Key blocks [b0, b0 + n) of tokens [t0, t1]; one block at least, so that rows that see nothing are
// still written.
template <bool kPairs>
__host__ __device__ __forceinline__ void tile_blocks(int t0, int t1, int ql, int kvl, int causal, int window, int& b0,
                                                     int& n) {
  constexpr int kBlk = kPairs ? kPairBlk : kRowBlk;
  int lo, hi;
  key_range(t0, t1, ql, kvl, causal, window, lo, hi);
  b0 = lo / kBlk;
  n = (int)(((long long)hi + kBlk - 1) / kBlk) - b0;
  if (n < 1) n = 1;
}

// At d = 64 a pair with tokens for one tile only is worked off as two halves of its keys
// (fa_paged_tiles.cu), in half a pair's time per block. Pairs are counted in half blocks there, and such a
// pair's count is rounded up to even, so that every pair starts at an even unit, and so does every CTA
// (SegIter::per). (At d = 128 two blocks of keys and values are all that fit beside the queries, too few
// on their way for a CTA that reads twice as fast: halves took 76 us against 63 at 20 rows over 60000 keys.)
__host__ __device__ __forceinline__ bool halves(int t0, int t1, const PagedBatch& b) {
  return b.d == 64 && t1 - t0 + 1 <= b.pair_tokens / 2;
}
// Every tile starts with some units for what it costs besides its blocks (queries in, sums out), so that
// CTAs with many short tiles get fewer blocks: three blocks' time for a pair at d = 128 (512 tokens over 32768
// keys: 191 us, 193 with two), two at d = 64 (2089 tokens of 32 heads: 44 us, 45 with three, 59 without) or three
// in halves (64 sequences of 128 tokens over 1000 keys: 56 us, 59 with two), two for a small tile (109 sequences
// of up to 421 keys: 30 us, 46 without).
template <bool kPairs>
__host__ __device__ __forceinline__ int tile_start(int t0, int t1, const PagedBatch& b) {
  if (!kPairs) return 2;
  return b.d == 64 && !halves(t0, t1, b) ? 4 : (b.d == 64 ? 6 : 3);
}
template <bool kPairs>
__host__ __device__ __forceinline__ int tile_units(int t0, int t1, const PagedBatch& b, int n) {
  const int at = tile_start<kPairs>(t0, t1, b);
  if (!kPairs || b.d != 64) return at + n;
  return at + (halves(t0, t1, b) ? (n + 1) & ~1 : 2 * n);
}

// SMs for the pairs where a batch has both kinds of tiles; the small ones have the others, at the same time: the
// pairs are bound by the tensor cores and the small tiles by HBM, of which 15 of the 152 SMs still draw 1.4 times
// their share. As many as end both soonest, with the time of a small tile's unit on an SM counted as 0.31 of a
// pair's at d = 128, and 0.37 of a half block's at d = 64. 4097 new tokens beside 23 single ones over 300 to 9000
// keys: 347 us, 366 one after the other (with 0.34: 346, 0.40: 351; too low costs more, 0.28 took 377); 4 x 30000
// keys beside 1024 new tokens over 16000: 255 us, 287 one after the other (0.34: 259, 0.40: 268).
__host__ __device__ constexpr float row_cost_of(int d) { return d == 64 ? 0.37f : 0.31f; }
__device__ __forceinline__ int pair_sms(const PagedBatch& b) {
  const long long rows = b.plan.units[0][b.S], pairs = b.plan.units[1][b.S];
  if (rows == 0 || pairs == 0) return pairs == 0 ? 0 : b.sms;
  const float r = (float)rows * b.row_cost, p = (float)pairs;
  const int n = max(1, min(b.sms - 2, (int)(b.sms * p / (p + r)))), m = b.sms - n;  // or one more: what ends sooner
  return m < 2 || fmaxf(p / n, r / m) <= fmaxf(p / (n + 1), r / (m - 1)) ? n : n + 1;
}

// One stretch of key blocks of one row tile, as a CTA works it off.
struct Seg {
  int seq, head, tile;
  int q0, ql, kvl;
  int t0, t1;      // tokens of the tile
  int blk, n;      // key blocks [blk, blk + n) of this stretch
  bool first, last;  // holds the tile's first / last block (both: no other CTA shares the tile)
  int c0, c1;        // the first and last CTA with a stretch of the tile
  int turn;          // pairs: the block to begin with, from `blk` on; the blocks before it come last
};

// Walk of one CTA's units, made by whole warps (the searches are warp-wide). The entries of 32
// sequences are held across the lanes, read together when the walk starts, so that finding the first
// stretch and moving on to the next sequence cost no chain of loads.
template <bool kPairs, int kRows = 0>
struct SegIter {
  const PagedBatch& b;
  const long long* U;
  long long u, u_end, per, tile_u0, u_begin;
  long long wU;  // lane i: U[w0 + i], past the end the largest value
  PlanSeq wS;    // lane i: sequence w0 + i
  int w0, seq, head, tile, ntiles, t0, t1;
  int b0, nblk, nb;  // the tile's first key block, its blocks and its units
  PlanSeq ps;

  __device__ __forceinline__ void load_window(int at) {
    const int i = at + (threadIdx.x & 31);
    w0 = at;
    wU = i <= b.S ? U[i] : 0x7fffffffffffffffLL;
    wS = i < b.S ? b.plan.seq[i] : PlanSeq{0, 0, 0, 0};
  }
  __device__ __forceinline__ SegIter(const PagedBatch& batch, unsigned ctas)
      : b(batch), U(batch.plan.units[kPairs ? 1 : 0]) {
    load_window(0);
    const long long W = U[b.S];
    per = W <= 0x7fffffffLL ? (long long)(((unsigned)W + ctas - 1) / ctas) : (W + ctas - 1) / ctas;
    if (kPairs && b.d == 64) per = (per + 1) & ~1LL;
    u = min(W, per * blockIdx.x);
    u_end = min(W, u + per);
    u_begin = u;
    head = b.Hkv;  // no sequence yet
  }
  __device__ __forceinline__ int owner(long long unit) const {
    return unit <= 0x7fffffffLL ? (int)((unsigned)unit / (unsigned)per) : (int)(unit / per);
  }

  __device__ __forceinline__ void measure() {  // the blocks and units of tile [t0, t1]
    tile_blocks<kPairs>(t0, t1, ps.ql, ps.kvl, b.causal, b.window, b0, nblk);
    nb = tile_units<kPairs>(t0, t1, b, nblk);
  }

  __device__ __forceinline__ void find_seq() {
    const int lane = threadIdx.x & 31;
    // The last s with U[s] <= u. The walk moves forward, so U[w0] <= u.
    int c = __popc(__ballot_sync(0xffffffffu, wU <= u));
    if (c == 32) {
      int lo = w0 + 31, hi = b.S;  // U[lo] <= u < U[hi]; a 32-way search down to one window
      while (hi - lo > 31) {
        const int step = (hi - lo + 31) / 32;
        const long long idx = (long long)lo + (long long)(lane + 1) * step;
        const int k = __popc(__ballot_sync(0xffffffffu, idx < hi && U[idx] <= u));
        lo += k * step;
        hi = (int)min((long long)hi, (long long)lo + step);
      }
      load_window(lo);
      c = __popc(__ballot_sync(0xffffffffu, wU <= u));
    }
    const int src = c - 1;  // at most 30: U[w0 + 31] > u
    seq = w0 + src;
    const long long base = __shfl_sync(0xffffffffu, wU, src), units = __shfl_sync(0xffffffffu, wU, c) - base;
    ps.q0 = __shfl_sync(0xffffffffu, wS.q0, src);
    ps.ql = __shfl_sync(0xffffffffu, wS.ql, src);
    ps.kvl = __shfl_sync(0xffffffffu, wS.kvl, src);
    ntiles = tile_count<kPairs, kRows>(ps.ql, b);
    long long per_head;
    if (units <= 0x7fffffffLL) {  // the usual case, without 64-bit divisions
      per_head = (unsigned)units / (unsigned)b.Hkv;
      head = (int)((unsigned)(u - base) / (unsigned)per_head);
    } else {
      per_head = units / b.Hkv;
      head = (int)((u - base) / per_head);
    }
    // The tile that holds unit u of this head: running sums over 32 tiles at a time.
    long long at = base + head * per_head;
    for (int i0 = 0;; i0 += 32) {
      int x0 = 0, x1 = 0, y0 = 0, yn = 0;
      if (i0 + lane < ntiles) {
        tile_tokens<kPairs, kRows>(i0 + lane, ps.ql, b, x0, x1);
        tile_blocks<kPairs>(x0, x1, ps.ql, ps.kvl, b.causal, b.window, y0, yn);
        yn = tile_units<kPairs>(x0, x1, b, yn);
      }
      long long sum = yn;
      if (ntiles > 1) {
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const long long v = __shfl_up_sync(0xffffffffu, sum, off);
          if (lane >= off) sum += v;
        }
      }
      const int k = ntiles > 1 ? __popc(__ballot_sync(0xffffffffu, at + sum <= u)) : 0;
      if (k < 32) {
        tile = i0 + k;
        t0 = __shfl_sync(0xffffffffu, x0, k);
        t1 = __shfl_sync(0xffffffffu, x1, k);
        measure();
        tile_u0 = at + __shfl_sync(0xffffffffu, sum, k) - nb;
        break;
      }
      at += __shfl_sync(0xffffffffu, sum, 31);
    }
  }

  __device__ __forceinline__ bool next(Seg& s) {
    while (u < u_end) {
      if (head == b.Hkv) find_seq();
      // The tile's blocks are its units [first_u, end_u); this CTA has those from `from` to `to`.
      const long long first_u = tile_u0 + tile_start<kPairs>(t0, t1, b), end_u = tile_u0 + nb;
      const long long from = max(u, first_u), to = min(u_end, end_u);
      const bool last = to == end_u;
      s.seq = seq;
      s.head = head;
      s.tile = tile;
      s.q0 = ps.q0;
      s.ql = ps.ql;
      s.kvl = ps.kvl;
      s.t0 = t0;
      s.t1 = t1;
      const int off = (int)(from - first_u), take = (int)(to - from);
      if (kPairs && b.d == 64 && !halves(t0, t1, b)) {
        s.blk = b0 + off / 2;
        s.n = take / 2;
      } else {
        s.blk = b0 + off;
        s.n = min(take, nblk - off);
      }
      s.first = off == 0;
      s.last = last;
      s.turn = 0;
      if (kPairs) {
        const int w = b.d == 64 ? 2 : 1;
        const unsigned round = (unsigned)(per / w), now = (unsigned)((from - u_begin) / w);
        const unsigned turn = (now + round - (unsigned)s.blk % round) % round;
        if (turn < (unsigned)s.n) s.turn = (int)turn;
      }
      // A tile that is not this CTA's alone is shared by the CTAs that own its first to its last block.
      s.c0 = s.first ? (int)blockIdx.x : owner(first_u);
      s.c1 = last ? (int)blockIdx.x : owner(end_u - 1);
      u = to;
      if (last) {  // on to the next tile, head or (at the next call) sequence
        tile_u0 += nb;
        if (ntiles > 1) {
          if (++tile == ntiles) {
            tile = 0;
            ++head;
          }
          if (head < b.Hkv) {
            tile_tokens<kPairs, kRows>(tile, ps.ql, b, t0, t1);
            measure();
          }
        } else {
          ++head;  // one tile per head: the same blocks again
        }
      }
      if (take > 0) return true;  // (else the CTA's units ended before the tile's first block)
    }
    return false;
  }
};

struct PagedCache {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long k_page, k_head, k_tok;  // strides in elements
  long long v_page, v_head, v_tok;
};

// A tile of 128 rows that CTA c (the index in PagedFwd::share) began and CTAs up to c1 went on with.
struct TileShare {
  int c1;  // -1: none
  int q0, ql, tok0, head;
};

// A small tile that CTA c (the index in PagedFwd::row_share) began, CTAs up to c1 went on with, and the
// kernel after theirs joins.
struct RowShare {
  int c1;  // -1: none
  int q0, r0, rows, head;
};

struct PagedFwd {
  PagedBatch b;
  PagedCache c;
  const __nv_bfloat16* q;
  long long q_tok, q_head;
  __nv_bfloat16* o;  // [T][Hq][d]
  float* lse;        // [T][Hq]
  float* part;       // partial results of the small tiles: 2 slots per CTA
  int row_grid;      // CTAs of the small tiles' kernel
  RowShare* row_share;  // [row_grid], or NULL: no kernel follows, every tile is joined by its last CTA
  float* tile_part;  // and of the pairs, with what each CTA shares with those after it
  TileShare* share;  // [tile_ctas][2 tiles]
  int o_wide;        // o starts at a multiple of 32 bytes
  int warp_out;      // (d = 128) 32 rows of a tile are whole tokens, and TileMaps::o has boxes of them
  int tile_ctas;     // CTAs of the pairs' kernel (0: it does not run)
  float scale_log2;
};

// CTAs per SM of the small tiles' kernel: what its registers leave room for (16 rows at d = 64: 109 single tokens
// over up to 421 keys of 16 heads 25.8 us, 29.7 with two CTAs and deeper rings; 256 over 500 keys 29.8, 33.0).
__host__ __device__ constexpr int row_ctas(int d, int row_tile) { return d == 64 && row_tile == 16 ? 3 : 2; }

// One partial result of a small tile: o [rows][D], then m, l, rounded l of the rows.
__host__ __device__ constexpr int row_part(int D, int rows) { return rows * (D + 3); }

// One partial result of a pair: per tile o [D / 4][128][4], unnormalised, and m, l, e [128].
__host__ __device__ constexpr int tile_part(int D) { return 2 * kTile * (D + 3); }

// Rotation of q and k (and a copy of v), dense or into a paged cache.
struct RopeStrides {
  long long batch, head, tok;  // in elements; of a cache: page, head, slot
};
struct RopeLaunch {
  const __nv_bfloat16* src[3];  // q, k, v
  __nv_bfloat16* dst[3];
  RopeStrides in[3], out[3];
  const int* positions;  // [axes][batch][token], or NULL: the place in the sequence (paged batch)
  long long pos_axis, pos_batch;
  const float* inv_freq;  // [rot / 2]
  uint64_t axes[2];       // two bits per pair
  long long tokens;       // B * N, or T
  int N, Hq, Hk, Hv, rot, interleaved, inverse;
  int tile;  // tokens per CTA
  PagedBatch b;
};

cudaError_t launch_paged_plan(const int* cu_q, const int* kv_len, const PagedBatch& b, int pair_rows, cudaStream_t st);
size_t paged_rows_workspace_bytes(int d, int row_tile);
cudaError_t launch_paged_rows(PagedFwd& p, int d, int num_sms, cudaStream_t st);
// The kernel that joins the small tiles left in PagedFwd::row_share, behind the kernel that leaves them.
constexpr int kMostRowGrid = 3 * kPagedSms;
cudaError_t launch_paged_join_rows(const PagedFwd& p, int d, int num_sms, cudaStream_t st);

struct TileMaps {
  CUtensorMap q;     // [T][Hq][d], box 64 dims x G heads x 128 / G tokens
  CUtensorMap k, v;  // [pages][Hkv][page_size][d], box 64 dims x min(page_size, 128) slots
  CUtensorMap o;     // [T][Hq][d], box 64 dims x G heads x 32 / G tokens, if PagedFwd::warp_out
};
size_t paged_tiles_workspace_bytes(int d);
cudaError_t launch_paged_tiles(const TileMaps& m, const PagedFwd& p, int d, int num_sms, cudaStream_t st);

// Rows of the small tiles. 32 where no sequence of the batch can have more, and some may have more than 16
// (a few drafted tokens): the keys are read once for them (8 tokens of 32 heads, 8 kv heads, 48 sequences of
// 3000 keys: 109 us against 125 in pairs at d = 128, 66 against 97 in two 16-row tiles at d = 64). Where
// longer sequences may be there too the batch's single tokens count more, which the 16-row kernel, with the
// queries in registers, has done a little sooner (the mixed batch of 24 sequences: 367 us against 373).
inline int row_tile_of(int G, int max_q) { return (long long)max_q * G > 16 && (long long)max_q * G <= 32 ? 32 : 16; }
// Sequences of more rows (new tokens times heads per kv head) than this are worked off in pairs of 128-row
// tiles, the others in the small tiles (with more than 128 heads per kv head, all of them). 17 to 32 rows
// beside longer sequences: two 16-row tiles, which read the keys twice, beat a 128-row one at d = 64 (41 us
// against 49 at 32 rows over 60000 keys of 8 kv heads), at d = 128 they do not (85 against 64). 64 rows:
// pairs (48 sequences as above: 126 us at d = 128, 77 at d = 64, against 195 and 120 in two 32-row tiles).
inline int pair_rows_of(int G, int d, int max_q) {
  return G > kTile ? 0x7fffffff : (d == 64 || row_tile_of(G, max_q) == 32 ? 32 : 16);
}

cudaError_t launch_rope(RopeLaunch& p, int d, bool paged, int num_sms, cudaStream_t st);

}  // namespace fa
