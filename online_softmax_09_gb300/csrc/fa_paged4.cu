// fa_paged4.cu -- attention of the newest tokens of a ragged batch over a 4-bit paged cache, sequences of few rows (the
// mathematics, the plan and the division among CTAs are fa_paged.cu's; fa_paged4.cuh has the cache).
//
// fa_paged4_rows_kernel: per CTA one warp that walks through its stretches and hands them out, and three or seven that
// compute, each with every third or seventh unit of 32 keys (two granules of 16, each within a page) and a ring of its own.
// The keys are the rows of the products' tiles, the queries their columns, so that up to 8 queries cost half of what 16 cost:
//     S^T = K Q^T (m16n8k16, A from codes),  O^T += V^T P^T (A from codes, P^T by a transposition of S^T's registers).
// Which dims an MMA sums in which step is free as long as both operands agree, and which dims are its rows, as long as the
// output knows: lane (g, c) of a warp (g = lane / 4, c = lane % 4) takes the quarter c of key g's dims in one piece, and of
// values 2 c, 2 c + 1, 2 c + 8 and 2 c + 9 the g-th eighth, so codes go from shared memory to operands in registers, in 16
// and 8 bytes per load, with one scale each, and a lane ends with 16 neighbouring dims of a query's output.
// At the end of a stretch the warps' sums are joined in shared memory, and parts of tiles that CTAs share in the workspace.
//
// Bound by latencies, with no unit full: one token of each of 64 sequences of 200 to 8192 keys (32 heads, 8 kv heads, d = 128,
// 314 MB) takes 89.5 us, 3.5 TB/s or 52 % of the copy rate, with 52 % of the issue slots used and the tensor pipe 19 % busy: 14 warps
// per SM, each in a chain of wait, unpacking, product, maximum over lanes, exponential, transposition and product. Instructions per
// 16 keys and warp, which fewer of have made it faster: 105 for the keys' operands and scores, 128 for the values' and sums, 29
// for the weights, 115 for copies, loop, joins. Two sequences
// of 131072 keys 80 us (292 MB); one of 1000 9.5, and 48 of 4 drafted tokens in a window of 1024 at d = 64 21.5: latencies of
// plan, table, keys, joins. (A share of the work for each warp, and no joins in CTAs: 87 us for the 64 sequences, but 16 and 30
// for those two.)
#include <math.h>

#include "fa_paged4.cuh"
#include "fa_paged_join.cuh"

namespace fa {

template <int D, int NT>
struct Row4Smem {
  static constexpr int kRows = NT <= 2 ? 16 : 32;
  static constexpr int kWarps = row4_warps(NT, D), kThreads = 32 * (kWarps + 1);  // those that compute, and one that walks
  static constexpr int kCtas = row4_ctas(NT, D);
  static constexpr int kCodes = kGran * code_bytes(D), kScales = kGran * scale_bytes(D);
  static constexpr int kPart = 2 * (kCodes + kScales);  // K codes, V codes, K scales, V scales of a granule
  static constexpr int kStage = 2 * kPart;              // two granules: what a warp takes at a time
  static constexpr int kStages = D == 128 ? 3 : 4;
  static constexpr int kSlots = kStages + 3;  // stretches handed out
  static constexpr int kWarp = kStages * kStage;
  static constexpr int kJoin = D == 128 && NT == 1 ? 4 : 8 * NT;  // rows that the warps join at a time
  static constexpr int kMerge = kWarps * kWarp;                  // these of each warp
  static constexpr int kStat = kMerge + kWarps * kJoin * D * 4;  // their m, l, rounded l
  static constexpr int kQ = kStat + kWarps * 3 * kJoin * 4;      // queries of 32 rows
  static constexpr int kQueue = kQ + (NT > 2 ? kRows * D * 2 : 0);
  static constexpr int kBar = kQueue + kSlots * (int)sizeof(Seg);
  static constexpr int bSegFull = 0, bSegEmpty = bSegFull + kSlots;
  static constexpr int kNumBars = bSegEmpty + kSlots;
  static constexpr int kFlag = kBar + kNumBars * 8;
  static constexpr int kAbort = kFlag + 8;
  static constexpr int kBytes = (kAbort + 4 + 15) / 16 * 16;
  static_assert(kBar % 8 == 0 && kQueue % 16 == 0, "layout");
  static_assert(kBytes <= 231424 / kCtas, "kCtas CTAs must fit an SM");
};

// An 8 x 8 tile of 16-bit values, two per lane (row lane / 4), transposed across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr)
                 : "memory");
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint16_t x;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(addr) : "memory");
  return x;
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void cp_async16_if(bool go, uint32_t dst, const void* src) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}\n" ::"r"(dst),
      "l"(src), "r"((uint32_t)go)
      : "memory");
}

template <int D, int NT>
__global__ void __launch_bounds__(Row4Smem<D, NT>::kThreads, Row4Smem<D, NT>::kCtas)
    fa_paged4_rows_kernel(const PagedFwd p, const PagedCache4 cache) {
  using L = Row4Smem<D, NT>;
  constexpr int kRows = L::kRows, kWarps = L::kWarps, kStages = L::kStages;
  constexpr int kSteps = D / 16;       // MMA steps over the dims of a score
  constexpr int kMT = D / 16;          // 16-dim tiles of o
  constexpr int kKW = D / 32;          // words of a key that a lane takes
  constexpr int kVW = D / 64;          // and of a value
  constexpr bool kQRegs = NT <= 2;     // queries in registers
  constexpr int kUnit = 2 * kGran;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  // (A value that all lanes have, from lane 0: the compiler then knows it, and needs no care for lanes that part.)
  auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  Seg* queue = reinterpret_cast<Seg*>(smem + L::kQueue);
  volatile int* flag = reinterpret_cast<volatile int*>(smem + L::kFlag);
  const PagedBatch& b = p.b;
  const Ctl ctl{reinterpret_cast<volatile int*>(smem + L::kAbort), b.status};
  auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8u * (uint32_t)i; };
  if (p.row_share != nullptr) {
    if (threadIdx.x == 0) p.row_share[blockIdx.x].c1 = -1;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  const unsigned G = b.G;

  if (warp == kWarps) {
    // ---------------------------------------------------------------- walk
    // One warp finds the CTA's stretches and hands them out, a few ahead of those that are worked on. (Done between the
    // stretches by a warp that computes, its state in shared memory: 110 us where this takes 91 for 64 sequences of 200 to
    // 8192 keys, 15 where it takes 10 for one of 1000.)
    SegIter<false, kRows> it(b, p.tile_ctas > 0 ? max(1, L::kCtas * (b.sms - pair_sms(b))) : gridDim.x);
    Seg s;
    bool some = plan_matches(b, D);  // (its loads go out beside the walk's)
    __syncthreads();                 // the barriers are there
    for (uint32_t i = 0; some; ++i) {
      some = it.next(s);
      const uint32_t at = i % L::kSlots;
      if (!mbar_wait_warp(bar(L::bSegEmpty + at), ((i / L::kSlots) & 1) ^ 1, ctl)) break;
      if (lane == 0) {
        queue[at] = s;
        if (!some) queue[at].n = -1;
        mbar_arrive(bar(L::bSegFull + at));
      }
    }
  }
  if (warp < kWarps) {
    if (threadIdx.x < L::kSlots) {
      mbar_init(bar(L::bSegFull + threadIdx.x), 1);
      mbar_init(bar(L::bSegEmpty + threadIdx.x), kWarps);
    }
    if (threadIdx.x == 0) *ctl.abort = 0;
    fence_mbar_init();
    __syncthreads();
  }
  if (!plan_matches(b, D)) {
    if (threadIdx.x == 0) record_index_error(b.status);
    if (p.tile_ctas > 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }

  // ------------------------------------------------------------------ products and softmax
  auto meet = [] { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); };
  const int g = lane >> 2, c = lane & 3;
  float* merge = reinterpret_cast<float*>(smem + L::kMerge);
  float* stat = reinterpret_cast<float*>(smem + L::kStat);
  const uint32_t magic = 0x43004300u, nibble = 0x000f000fu;
  // Codes 2 j and 2 j + 1 of a word as values: the masks stand in registers, so that they take one instruction.
  auto value_pair = [&](uint32_t w, int j, uint32_t s2, uint32_t cs) {
    uint32_t x;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(x) : "r"(w >> (4 * j)), "r"(nibble), "r"(magic));
    return fma_bf16x2(x, s2, cs);
  };

  const uint32_t by_G = 0xffffffffu / G + 1;  // ceil(2^32 / G): a product's high half is the quotient of up to 2^16 rows
  // Queries as B operands: column g of tile t is row 8 t + g, and lane c holds its quarter of the dims. (Zero past the
  // tile's rows.) With 32 rows they stand in shared memory, 16-byte chunk x of row r at x ^ (r & 7).
  uint32_t qb[kQRegs ? NT : 1][kQRegs ? D / 8 : 1];
  int klo[NT][2], klim[NT][2], all_lo = 0, all_lim = 0;  // of rows 8 t + 2 c and the next
  auto load_q = [&](const Seg& s) {
    const unsigned r0 = (unsigned)s.tile * kRows;
    const int rows = (int)min((unsigned)kRows, (unsigned)s.ql * G - r0);
    const bool few_rows = (unsigned)s.ql * G <= 65536 && G > 1;
    auto row_of = [&](int r, int& tok) {
      const unsigned rr = r0 + (r < rows ? r : 0);
      tok = s.ql == 1 ? 0 : (int)(few_rows ? __umulhi(rr, by_G) : rr / G);
      const int hd = (int)(rr - tok * G);
      return p.q + (long long)(s.q0 + tok) * p.q_tok + (long long)(s.head * G + hd) * p.q_head;
    };
    if constexpr (!kQRegs) {
      meet();  // the queries that stood there have been used
      for (int x = threadIdx.x; x < kRows * (D / 8); x += 32 * kWarps) {
        const int r = x / (D / 8), ch = x % (D / 8);
        int tok;
        const __nv_bfloat16* qp = row_of(r, tok);
        const uint4 v = r < rows ? *reinterpret_cast<const uint4*>(qp + ch * 8) : make_uint4(0, 0, 0, 0);
        st_shared_v4(sbase + L::kQ + r * (D * 2) + ((ch ^ (r & 7)) << 4), v.x, v.y, v.z, v.w);
      }
      meet();
    }
    int top = -0x7fffffff, low = 0x7fffffff;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      int tok;
      if constexpr (kQRegs) {
        const uint4* qp = reinterpret_cast<const uint4*>(row_of(8 * t + g, tok) + c * (D / 4));
        const bool ok = 8 * t + g < rows;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 v = ok ? qp[i] : make_uint4(0, 0, 0, 0);
          qb[t][4 * i] = v.x;
          qb[t][4 * i + 1] = v.y;
          qb[t][4 * i + 2] = v.z;
          qb[t][4 * i + 3] = v.w;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        row_of(8 * t + 2 * c + h, tok);
        const int pos = s.kvl - s.ql + tok;
        klim[t][h] = b.causal ? pos : s.kvl - 1;
        klo[t][h] = mask_from(pos, b.window);
        top = max(top, klo[t][h]);
        low = min(low, klim[t][h]);
      }
    }
    all_lo = __reduce_max_sync(0xffffffffu, top);
    all_lim = __reduce_min_sync(0xffffffffu, low);
  };

  if (warp < kWarps) {
    const uint32_t ring = sbase + warp * L::kWarp;
    const int step = kWarps * kUnit;  // from one of the warp's units to the next
    // The copying side: units of 32 keys, one of every kWarps, up to kStages ahead of the products,
    // on into the next stretches. A unit is two granules of 16 keys, each within a page. 16 bytes per lane: two rounds for a
    // granule's codes of keys and of values (one at d = 64), and one for its scales, of keys in the first lanes and of values
    // in the next. (Bulk copies of these four pieces, of 64 bytes to 1 KB, came to one per 60 cycles and SM and bound the
    // kernel: 111 us for 64 sequences of 200 to 8192 keys.) A granule that no row sees, or whose page does not exist, is
    // left out.
    constexpr int kPieces = L::kScales / 16, kRounds = L::kCodes / 512;
    uint32_t fetched = 0, in = 0, none = 0;  // stretches taken; the stage that is filled next; bits 2 i: left out in stage i
    int key_in = 0, end_in = 0, lo_in = 0, hi_in = 0;
    const int* tab = nullptr;
    const uint8_t *kp = nullptr, *vp = nullptr, *sp = nullptr;
    int pages = 0;  // lane i: the page of granule i of this warp's next 16 units
    uint32_t have = 0;  // bit i: there is one
    int batch = 0;
    bool more = true;
    auto read_pages = [&]() {
      const int key = key_in + (lane >> 1) * step + (lane & 1) * kGran;
      const bool seen = key < end_in && key < hi_in && key + kGran > lo_in;
      pages = seen ? tab[key >> b.page_shift] : 0;
      const bool bad = (unsigned)pages >= (unsigned)b.num_pages;
      if (bad) {
        record_index_error(b.status);
        pages = 0;
      }
      have = __ballot_sync(0xffffffffu, seen && !bad);
      batch = 0;
    };
    // The next stretch with units for this warp, while stretch k is worked on: no further than the slots reach without
    // k's being given back (a warp may have none in many short stretches).
    auto fetch = [&](uint32_t k) {
      while (more && key_in >= end_in && fetched - k < L::kSlots - 1) {
        const uint32_t at = fetched % L::kSlots;
        if (!mbar_wait_warp(bar(L::bSegFull + at), (fetched / L::kSlots) & 1, ctl)) more = false;
        const Seg& s = queue[at];
        if (!more || s.n < 0) {
          more = false;
          break;
        }
        ++fetched;
        int lo, hi;
        key_range(s.t0, s.t1, s.ql, s.kvl, b.causal, b.window, lo, hi);
        lo_in = uniform(lo);
        hi_in = uniform(hi);
        key_in = uniform(s.blk) * kRowBlk + warp * kUnit;
        end_in = uniform(s.blk + s.n) * kRowBlk;
        tab = b.table + (long long)s.seq * b.table_stride;
        kp = cache.k + (long long)s.head * cache.k_head + lane * 16;
        vp = cache.v + (long long)s.head * cache.v_head + lane * 16;
        sp = lane < kPieces ? cache.k_scale + (long long)s.head * cache.ks_head + lane * 16
                            : cache.v_scale + (long long)s.head * cache.vs_head + (lane - kPieces) * 16;
        read_pages();
      }
    };
    const uint32_t s_page = (uint32_t)(lane < kPieces ? cache.ks_page : cache.vs_page);
    uint32_t issued = 0, done = 0;  // units, of all stretches; a group of copies each
    auto issue = [&]() {            // the next unit's copies
      const uint32_t st = ring + in * L::kStage + lane * 16, there = have >> 2 * batch & 3;
      const uint32_t slot0 = b.page_size == kGran ? 0 : key_in & (b.page_size - 1);
      const uint32_t slot_step = b.page_size == kGran ? 0 : kGran;
      auto part = [&](int h) {
        const uint32_t page = __shfl_sync(0xffffffffu, pages, 2 * batch + h), slot = slot0 + h * slot_step;
        const uint8_t* kx = kp + (uint64_t)page * (uint32_t)cache.k_page + slot * code_bytes(D);
        const uint8_t* vx = vp + (uint64_t)page * (uint32_t)cache.v_page + slot * code_bytes(D);
        const uint8_t* sx = sp + (uint64_t)page * s_page + slot * scale_bytes(D);
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
          cp_async16(st + h * L::kPart + i * 512, kx + i * 512);
          cp_async16(st + h * L::kPart + L::kCodes + i * 512, vx + i * 512);
        }
        cp_async16_if(lane < 2 * kPieces, st + h * L::kPart + 2 * L::kCodes, sx);
      };
      if (there == 3) {
        part(0);
        part(1);
      } else if (there != 0) {
        if (there & 1) part(0);
        else part(1);
      }
      none = (none & ~(3u << 2 * in)) | (there ^ 3u) << 2 * in;
      cp_async_commit();
      ++issued;
      in = in + 1 == kStages ? 0 : in + 1;
      key_in += step;
      if (++batch == 16 && key_in < end_in) read_pages();
    };
    auto fill = [&](uint32_t k) {  // the ring, as far as units are at hand
      while (issued - done < kStages) {
        if (key_in >= end_in) fetch(k);
        if (key_in >= end_in) break;
        issue();
      }
    };
    fill(0);
    uint32_t out = 0;  // the stage that is used next
    const uint32_t k_at = g * code_bytes(D) + c * (4 * kKW);
    const uint32_t ks_at = 2 * L::kCodes + g * scale_bytes(D) + (c * (D / 4) / kGroup4) * 2;
    const uint32_t v_at = L::kCodes + 2 * c * code_bytes(D) + g * (4 * kVW);
    const uint32_t vs_at = 2 * L::kCodes + L::kScales + 2 * c * scale_bytes(D) + (g * (D / 8) / kGroup4) * 2;
    for (uint32_t k = 0;; ++k) {
      // One warp waits for the stretch, so that all of them go on or none.
      if (warp == 0) {
        const bool go = mbar_wait_warp(bar(L::bSegFull + k % L::kSlots), (k / L::kSlots) & 1, ctl);
        if (lane == 0) flag[0] = go;
      }
      meet();
      if (!uniform(flag[0])) break;
      const Seg& s = queue[k % L::kSlots];
      if (uniform(s.n) < 0) break;
      fill(k);
      load_q(s);
      const int begin = uniform(s.blk) * kRowBlk, end = begin + uniform(s.n) * kRowBlk;
      const unsigned r0 = (unsigned)s.tile * kRows;
      const int rows = uniform((int)min((unsigned)kRows, (unsigned)s.ql * G - r0));
      int lo, hi;
      key_range(s.t0, s.t1, s.ql, s.kvl, b.causal, b.window, lo, hi);
      lo = uniform(lo);
      hi = uniform(hi);
      float o[kMT][NT][4];
#pragma unroll
      for (int j = 0; j < kMT; ++j)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][t][i] = 0.f;
      float m[NT][2], l[NT][2], lr[NT][4];  // lr: a product of ones and the weights as they are rounded
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          m[t][h] = -INFINITY;
          l[t][h] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) lr[t][i] = 0.f;
      }

#pragma unroll 1
      for (int key = begin + warp * kUnit; key < end; key += step) {
        if (issued - done < kStages) {  // (usually by the one that was used last)
          if (key_in < end_in) issue();
          else fill(k);
        }
        if (issued - done == kStages) cp_async_wait<kStages - 1>();
        else cp_async_wait<0>();
        __syncwarp();
        ++done;
        const uint32_t st = ring + out * L::kStage, left_out = none >> 2 * out & 3;
        out = out + 1 == kStages ? 0 : out + 1;
        if (left_out == 3) continue;
        const bool masked = key < all_lo || key + kUnit - 1 > all_lim || left_out;
        // ---- scores
        float x[2][NT][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[u][t][e] = 0.f;
        {
          uint32_t w[2][2][kKW], s2[2][2], cs[2][2];
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              lds_words<kKW>(st + u * L::kPart + k_at + 8 * h * code_bytes(D), w[u][h]);
              s2[u][h] = lds_u16(st + u * L::kPart + ks_at + 8 * h * scale_bytes(D)) * 0x10001u;
              cs[u][h] = scale_shift(s2[u][h]);
            }
#pragma unroll
          for (int kk = 0; kk < kSteps; ++kk) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t a[4];
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  a[2 * e + h] = value_pair(w[u][h][kk >> 1], 2 * (kk & 1) + e, s2[u][h], cs[u][h]);
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                if constexpr (kQRegs) {
                  mma16816(x[u][t], a, qb[t][2 * kk], qb[t][2 * kk + 1]);
                } else {
                  const int r = 8 * t + g, byte = c * (D / 2) + 8 * kk;  // within the row
                  uint32_t q2[2];
                  lds_words<2>(sbase + L::kQ + r * (D * 2) + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15), q2);
                  mma16816(x[u][t], a, q2[0], q2[1]);
                }
              }
            }
          }
        }
        // ---- weights
        uint32_t pb[NT][2][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (masked) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int kx = key + u * kGran + g + 8 * (e >> 1);
                if (kx > klim[t][e & 1] || kx < klo[t][e & 1] || (left_out >> u & 1)) x[u][t][e] = -INFINITY;
              }
          }
          float mt[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v = max3f(fmaxf(x[0][t][h], x[0][t][2 + h]), x[1][t][h], x[1][t][2 + h]);
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            mt[h] = v * p.scale_log2;
          }
          // The reference max moves only when a row has outgrown it by 2^8 (any reference gives the same softmax).
          if (__any_sync(0xffffffffu, mt[0] > m[t][0] + 8.f || mt[1] > m[t][1] + 8.f)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float mn = fmaxf(m[t][h], mt[h]);
              const float corr = mn > m[t][h] ? ex2(m[t][h] - mn) : 1.f;
              m[t][h] = mn;
              l[t][h] *= corr;
              lr[t][h] *= corr;
#pragma unroll
              for (int j = 0; j < kMT; ++j) {
                o[j][t][h] *= corr;
                o[j][t][2 + h] *= corr;
              }
            }
          }
          const float mu[2] = {m[t][0] == -INFINITY ? 0.f : m[t][0], m[t][1] == -INFINITY ? 0.f : m[t][1]};
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int y = 0; y < 2; ++y) {  // keys g and g + 8
              const float e0 = ex2(fmaf(x[u][t][2 * y], p.scale_log2, -mu[0]));
              const float e1 = ex2(fmaf(x[u][t][2 * y + 1], p.scale_log2, -mu[1]));
              l[t][0] += e0;
              l[t][1] += e1;
              pb[t][u][y] = transpose8x8(pack_bf16(e0, e1));
            }
        }
        // ---- values
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t w[4][kVW], sc[4];  // values 2 c, 2 c + 1, 2 c + 8, 2 c + 9
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int kx = (y & 1) + 8 * (y >> 1);
            lds_words<kVW>(st + u * L::kPart + v_at + kx * code_bytes(D), w[y]);
            sc[y] = lds_u16(st + u * L::kPart + vs_at + kx * scale_bytes(D));
          }
          if (masked) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int kx = key + u * kGran + 2 * c + (y & 1) + 8 * (y >> 1);
              if (kx < lo || kx >= hi || (left_out >> u & 1)) sc[y] = 0;  // slots that no row sees may hold NaN
            }
          }
          uint32_t s2[2], cs[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            s2[y] = sc[2 * y] | sc[2 * y + 1] << 16;
            cs[y] = scale_shift(s2[y]);
          }
          // The same half words of two values side by side: pairs of keys for dims 2 j (low halves) and 2 j + 1.
          uint32_t z[2][kVW][2];
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int v = 0; v < kVW; ++v) {
              z[y][v][0] = __byte_perm(w[2 * y][v], w[2 * y + 1][v], 0x5410);
              z[y][v][1] = __byte_perm(w[2 * y][v], w[2 * y + 1][v], 0x7632);
            }
          const uint32_t ones[4] = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
#pragma unroll
          for (int t = 0; t < NT; ++t) mma16816(lr[t], ones, pb[t][u][0], pb[t][u][1]);
#pragma unroll
          for (int j = 0; j < kMT; ++j) {
            uint32_t a[4];
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                // d = 128: tile j has dims 16 g + j and 16 g + 8 + j; d = 64: 8 g + 2 j and 8 g + 2 j + 1.
                const uint32_t src = D == 128 ? z[y][h & (kVW - 1)][j & 1] : z[y][0][h];
                a[2 * y + h] = value_pair(src, D == 128 ? j >> 1 : j, s2[y], cs[y]);
              }
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816(o[j][t], a, pb[t][u][0], pb[t][u][1]);
          }
        }
        __syncwarp();  // the stage is read: the next copies may overwrite it
      }

      // ---- join the warps, kJoin rows at a time
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) l[t][h] += __shfl_xor_sync(0xffffffffu, l[t][h], off);
      const bool whole = s.first && s.last;
      const int c0 = s.c0, c1 = s.c1, q0 = s.q0, head = s.head;
      float* slot = p.part + (size_t)(2 * blockIdx.x + (s.first ? 1 : 0)) * row_part(D, kRows);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::bSegEmpty + k % L::kSlots));  // (nothing of s is read below)
      constexpr int kJoin = L::kJoin;
#pragma unroll
      for (int first_row = 0; first_row < 8 * NT; first_row += kJoin) {
        if (first_row >= rows) break;
        if (first_row > 0) meet();  // the rows that stood here have been read
        // Rows 8 t + 2 c and the next of this lane, dims from g * D / 8 on; 16-byte chunk x of row r at x ^ 2 r (two bits of r).
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = 8 * t + 2 * c + h - first_row, at = warp * kJoin + r;
            if (r < 0 || r >= kJoin) continue;
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {  // dims 4 q .. of the lane's
              float4 v;
              float* f = reinterpret_cast<float*>(&v);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int dim = 4 * q + i;
                f[i] = D == 128 ? o[(dim & 7) % kMT][t][2 * (dim >> 3) + h] : o[(dim >> 1) % kMT][t][2 * (dim & 1) + h];
              }
              *reinterpret_cast<float4*>(merge + at * D + (((g * (D / 32) + q) ^ (2 * (r & 3))) << 2)) = v;
            }
            if (g == 0) {
              stat[at * 3] = m[t][h];
              stat[at * 3 + 1] = l[t][h];
              stat[at * 3 + 2] = lr[t][h];
            }
          }
        meet();
        const int here = min(kJoin, rows - first_row);
        for (int x = threadIdx.x; x < here * (D / 4); x += 32 * kWarps) {  // four columns of a row
          const int hr = x / (D / 4), row = hr + first_row, ch = x % (D / 4);
          float M = -INFINITY, Ls = 0.f, Lr = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) M = fmaxf(M, stat[(w * kJoin + hr) * 3]);
          const float Mu = M == -INFINITY ? 0.f : M;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float* sw = stat + (w * kJoin + hr) * 3;
            const float f = ex2(sw[0] - Mu);
            Ls += f * sw[1];
            Lr += f * sw[2];
            const float4 v = *reinterpret_cast<const float4*>(merge + (w * kJoin + hr) * D + ((ch ^ (2 * (hr & 3))) << 2));
            acc.x = fmaf(f, v.x, acc.x);
            acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z);
            acc.w = fmaf(f, v.w, acc.w);
          }
          if (whole) {
            const long long place = put_row<D>(p, q0, head, r0 + row, 4 * ch, acc, Lr);
            if (ch == 0) p.lse[place] = (M + log2f(Ls)) * 0.6931471805599453f;
          } else {
            *reinterpret_cast<float4*>(slot + row * D + 4 * ch) = acc;
            if (ch == 0) {
              slot[kRows * D + row] = M;
              slot[kRows * (D + 1) + row] = Ls;
              slot[kRows * (D + 2) + row] = Lr;
            }
          }
        }
      }
      if (!whole && p.row_share != nullptr) {
        if (c0 == (int)blockIdx.x && threadIdx.x == 0) p.row_share[c0] = RowShare{c1, q0, (int)r0, rows, head};
      } else if (!whole) {
        meet();
        if (threadIdx.x == 0) {
          // The barrier orders the CTA's stores before this thread's release, which covers them all.
          uint32_t before;
          asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                       : "=r"(before)
                       : "l"(&b.plan.counters[c0])
                       : "memory");
          const bool last = before == (uint32_t)(c1 - c0);
          if (last) b.plan.counters[c0] = 0;
          flag[1] = last;
        }
        meet();
        if (flag[1]) join_row_tile<D, kRows, 32 * kWarps>(p, c0, c1, q0, head, r0, rows);
      }
    }
  }
  if constexpr (NT == 2) {  // (a batch of tiles of 8 or of 32 rows has no pairs)
    static_assert(kWarps + 1 == kRowWarps || kWarps >= kRowWarps, "join_pairs is for kRowThreads");
    // Its list stands in the first warps' rings: the others' copies, of which some may be in flight, do not reach it.
    static_assert(2 * kPagedSms * (sizeof(TileShare) + 8) + 64 <= (kWarps < kRowWarps ? kWarps : kRowWarps) * L::kWarp,
                  "room for the list");
    if (p.tile_ctas > 0 && warp < kRowWarps) {
      asm volatile("cp.async.wait_all;" ::: "memory");  // (some are in flight after a wait that gave up)
      auto meet_four = [] { asm volatile("bar.sync 2, %0;" ::"n"(kRowThreads) : "memory"); };
      meet_four();
      join_pairs<D>(p, meet_four);
    }
  }
}

template <int D, int NT>
static cudaError_t launch_rows4(PagedFwd& p, const PagedCache4& cache, int num_sms, cudaStream_t st) {
  using L = Row4Smem<D, NT>;
  static unsigned long long known[kMaxGpus];
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(fa_paged4_rows_kernel<D, NT>), L::kBytes, known);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  p.row_grid = L::kCtas * num_sms;
  cfg.gridDim = dim3(p.row_grid);
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::kBytes;
  cfg.stream = st;
  cudaLaunchAttribute early;  // beside the pairs' kernel, as in launch_paged_rows
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = p.tile_ctas > 0 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, fa_paged4_rows_kernel<D, NT>, p, cache);
  if (e != cudaSuccess || p.row_share == nullptr) return e;
  return launch_paged_join_rows(p, D, num_sms, st);
}

// Tiles of 8 columns: one where no tile of the batch can have more than 8 rows, two for 16, four for 32.
size_t paged4_rows_part_bytes(int d, int row_tile, int columns) {
  return plan_up((size_t)2 * row4_ctas(columns, d) * kPagedSms * row_part(d, row_tile) * 4);
}
size_t paged4_rows_workspace_bytes(int d, int row_tile, int columns) {
  return paged4_rows_part_bytes(d, row_tile, columns) + plan_up((size_t)row4_ctas(columns, d) * kPagedSms * sizeof(RowShare));
}

cudaError_t launch_paged4_rows(PagedFwd& p, const PagedCache4& cache, int d, int num_sms, cudaStream_t st) {
  const int nt = row4_columns(p.b.row_tile, p.b.max_q, p.b.G);
  if (d == 128)
    return nt == 4 ? launch_rows4<128, 4>(p, cache, num_sms, st)
                   : (nt == 2 ? launch_rows4<128, 2>(p, cache, num_sms, st) : launch_rows4<128, 1>(p, cache, num_sms, st));
  return nt == 4 ? launch_rows4<64, 4>(p, cache, num_sms, st)
                 : (nt == 2 ? launch_rows4<64, 2>(p, cache, num_sms, st) : launch_rows4<64, 1>(p, cache, num_sms, st));
}

}  // namespace fa
