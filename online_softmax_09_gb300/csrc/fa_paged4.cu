// fa_paged4.cu -- attention of the newest tokens of a ragged batch over a 4-bit paged cache, sequences of few rows (the
// mathematics, the plan and the division among CTAs are fa_paged.cu's; fa_paged4.cuh has the cache).
//
// fa_paged4_rows_kernel: four warps per CTA, each with every fourth granule of 16 keys and a ring of its own, filled by bulk
// copies (a granule's codes and scales are four dense pieces: 2304 bytes at d = 128). The keys are the rows of the products'
// tiles, the queries their columns, so that up to 8 queries cost half of what 16 cost:
//     S^T = K Q^T (m16n8k16, A from codes),  O^T += V^T P^T (A from codes, P^T by a transposition of S^T's registers).
// Which dims an MMA sums in which step is free as long as both operands agree, and which dims are its rows, as long as the
// output knows: lane (g, c) of a warp (g = lane / 4, c = lane % 4) takes the quarter c of key g's dims in one piece, and of
// values 2 c, 2 c + 1, 2 c + 8 and 2 c + 9 the g-th eighth, so codes go from shared memory to operands in registers, in 16
// and 8 bytes per load, with one scale each, and a lane ends with 16 neighbouring dims of a query's output.
#include <math.h>

#include "fa_paged4.cuh"
#include "fa_paged_join.cuh"

namespace fa {

template <int D, int NT>
struct Row4Smem {
  static constexpr int kRows = NT <= 2 ? 16 : 32;
  static constexpr int kCtas = row4_ctas(kRows);
  static constexpr int kCodes = kGran * code_bytes(D), kScales = kGran * scale_bytes(D);
  static constexpr int kStage = 2 * (kCodes + kScales);  // K codes, V codes, K scales, V scales of a granule
  static constexpr int kStages = D == 128 ? 6 : 8;
  static constexpr int kSlots = 16;                // stretches queued: kStages + 1 at least
  static constexpr int kWarp = kStages * kStage;
  static constexpr int kMerge = kRowWarps * kWarp;               // 8 rows of o of each warp
  static constexpr int kStat = kMerge + kRowWarps * 8 * D * 4;   // their m, l, rounded l
  static constexpr int kQ = kStat + kRowWarps * 3 * 8 * 4;       // queries of 32 rows
  static constexpr int kQueue = kQ + (NT > 2 ? kRows * D * 2 : 0);
  static constexpr int kBar = kQueue + kSlots * (int)sizeof(Seg);
  static constexpr int kSkip = kBar + kRowWarps * kStages * 8;   // granules that hold nothing to see
  static constexpr int kFlag = kSkip + kRowWarps * kStages * 4;
  static constexpr int kAbort = kFlag + 4;
  static constexpr int kBytes = (kAbort + 4 + 15) / 16 * 16;
  static_assert(kSlots > kStages && kBar % 8 == 0 && kQueue % 16 == 0, "layout");
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

template <int D, int NT>
__global__ void __launch_bounds__(kRowThreads, Row4Smem<D, NT>::kCtas)
    fa_paged4_rows_kernel(const PagedFwd p, const PagedCache4 cache) {
  using L = Row4Smem<D, NT>;
  constexpr int kRows = L::kRows;
  constexpr int kSteps = D / 16;       // MMA steps over the dims of a score
  constexpr int kMT = D / 16;          // 16-dim tiles of o
  constexpr int kKW = D / 32;          // words of a key that a lane takes
  constexpr int kVW = D / 64;          // and of a value
  constexpr bool kQRegs = NT <= 2;     // queries in registers
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t ring = sbase + warp * L::kWarp;
  float* merge = reinterpret_cast<float*>(smem + L::kMerge);
  float* stat = reinterpret_cast<float*>(smem + L::kStat);
  Seg* queue = reinterpret_cast<Seg*>(smem + L::kQueue);
  volatile int* skip = reinterpret_cast<volatile int*>(smem + L::kSkip) + warp * L::kStages;
  int* flag = reinterpret_cast<int*>(smem + L::kFlag);
  const PagedBatch& b = p.b;
  const Ctl ctl{reinterpret_cast<volatile int*>(smem + L::kAbort), b.status};
  auto bar = [&](uint32_t stage) -> uint32_t { return sbase + L::kBar + (warp * L::kStages + stage) * 8; };
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
  if (threadIdx.x == 0) *ctl.abort = 0;
  if (lane == 0) {
    for (int i = 0; i < L::kStages; ++i) mbar_init(bar(i), 1);
    fence_mbar_init();
  }
  __syncthreads();
  const unsigned G = b.G;

  // The copying side, as in fa_paged_rows_kernel: stretches from the walk into the queue, granules into the ring. A
  // granule that no row of the tile sees, or whose page does not exist, takes a stage without a copy.
  uint32_t fetched = 0, copied = 0;
  int ln = 0, li = 0, lkey = 0, llo = 0, lhi = 0, lhead = 0;
  const int* ltab = nullptr;
  int pages = -1;
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
    lkey = s.blk * kRowBlk + warp * kGran;
    key_range(s.t0, s.t1, s.ql, s.kvl, b.causal, b.window, llo, lhi);
    ltab = b.table + (long long)s.seq * b.table_stride;
    read_pages();
  };
  auto issue = [&]() {
    if (li < ln) {
      const int page = __shfl_sync(0xffffffffu, pages, li & 31);
      const uint32_t stage = copied % L::kStages;
      if (lane == 0) {
        skip[stage] = page < 0;
        if (page < 0) {
          mbar_arrive(bar(stage));
        } else {
          const int slot = (lkey + li * kRowBlk) & (b.page_size - 1);
          const uint32_t st = ring + stage * L::kStage;
          mbar_expect_tx(bar(stage), L::kStage);
          bulk_load(st, cache.k + page * cache.k_page + lhead * cache.k_head + slot * code_bytes(D), L::kCodes, bar(stage));
          bulk_load(st + 2 * L::kCodes, cache.k_scale + page * cache.ks_page + lhead * cache.ks_head + slot * scale_bytes(D),
                    L::kScales, bar(stage));
          bulk_load(st + L::kCodes, cache.v + page * cache.v_page + lhead * cache.v_head + slot * code_bytes(D), L::kCodes,
                    bar(stage));
          bulk_load(st + 2 * L::kCodes + L::kScales,
                    cache.v_scale + page * cache.vs_page + lhead * cache.vs_head + slot * scale_bytes(D), L::kScales,
                    bar(stage));
        }
      }
      __syncwarp();
      ++copied;
      if (++li == ln) fetch();
      else if ((li & 31) == 0) read_pages();
    }
  };

  // Queries as B operands: column g of tile t is row 8 t + g, and lane c holds its quarter of the dims. (Zero past the
  // tile's rows.) With 32 rows they stand in shared memory, 16-byte chunk x of row r at x ^ (r & 7).
  uint32_t qb[kQRegs ? NT : 1][kQRegs ? D / 8 : 1];
  constexpr int kQLoads = kRows * (D / 8) / kRowThreads;
  uint4 qv[kQRegs ? 1 : kQLoads];
  int klo[NT][2], klim[NT][2], all_lo = 0, all_lim = 0;  // of rows 8 t + 2 c and the next
  auto load_q = [&](const Seg& s) {
    const unsigned r0 = (unsigned)s.tile * kRows;
    const int rows = (int)min((unsigned)kRows, (unsigned)s.ql * G - r0);
    auto row_of = [&](int r, int& tok) {
      const unsigned rr = r0 + (r < rows ? r : 0);
      tok = (int)(rr / G);
      const int hd = (int)(rr - tok * G);
      return p.q + (long long)(s.q0 + tok) * p.q_tok + (long long)(s.head * G + hd) * p.q_head;
    };
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
    if constexpr (!kQRegs) {
#pragma unroll
      for (int i = 0; i < kQLoads; ++i) {
        const int x = i * kRowThreads + threadIdx.x, r = x / (D / 8);
        int tok;
        const __nv_bfloat16* qp = row_of(r, tok);
        qv[i] = r < rows ? *reinterpret_cast<const uint4*>(qp + (x % (D / 8)) * 8) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  auto place_q = [&]() {  // by all threads, where nothing reads the place any more
    if constexpr (!kQRegs) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kQLoads; ++i) {
        const int x = i * kRowThreads + threadIdx.x, r = x / (D / 8), ch = x % (D / 8);
        st_shared_v4(sbase + L::kQ + r * (D * 2) + ((ch ^ (r & 7)) << 4), qv[i].x, qv[i].y, qv[i].z, qv[i].w);
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
    int lo, hi;
    key_range(s.t0, s.t1, s.ql, s.kvl, b.causal, b.window, lo, hi);
    float o[kMT][NT][4];
#pragma unroll
    for (int j = 0; j < kMT; ++j)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][t][i] = 0.f;
    float m[NT][2], l[NT][2], lr[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        m[t][h] = -INFINITY;
        l[t][h] = lr[t][h] = 0.f;
      }

    for (int i = 0; i < n; ++i, ++done) {
      issue();
      const uint32_t stage = done % L::kStages;
      if (!mbar_wait_warp(bar(stage), (done / L::kStages) & 1, ctl)) continue;
      if (skip[stage]) continue;
      const uint32_t st = ring + stage * L::kStage;
      const int key = key0 + i * kRowBlk;
      const bool masked = key < all_lo || key + kGran - 1 > all_lim;
      // ---- scores
      float x[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[t][e] = 0.f;
      {
        uint32_t w[2][kKW], s2[2], cs[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          lds_words<kKW>(st + (g + 8 * h) * code_bytes(D) + c * (4 * kKW), w[h]);
          const uint32_t sc = lds_u16(st + 2 * L::kCodes + (g + 8 * h) * scale_bytes(D) + (c * (D / 4) / kGroup4) * 2);
          s2[h] = sc * 0x10001u;
          cs[h] = scale_shift(s2[h]);
        }
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk) {
          uint32_t a[4];
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              a[2 * e + h] = fma_bf16x2(code_pair(w[h][kk >> 1], 2 * (kk & 1) + e), s2[h], cs[h]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if constexpr (kQRegs) {
              mma16816(x[t], a, qb[t][2 * kk], qb[t][2 * kk + 1]);
            } else {
              const int r = 8 * t + g, byte = c * (D / 2) + 8 * kk;  // within the row
              uint32_t q2[2];
              lds_words<2>(sbase + L::kQ + r * (D * 2) + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15), q2);
              mma16816(x[t], a, q2[0], q2[1]);
            }
          }
        }
      }
      // ---- weights
      uint32_t pb[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (masked) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int kx = key + g + 8 * (e >> 1);
            if (kx > klim[t][e & 1] || kx < klo[t][e & 1]) x[t][e] = -INFINITY;
          }
        }
        float mt[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v = fmaxf(x[t][h], x[t][2 + h]);
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
          mt[h] = v * p.scale_log2;
        }
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
        for (int y = 0; y < 2; ++y) {  // keys g and g + 8
          const float e0 = ex2(fmaf(x[t][2 * y], p.scale_log2, -mu[0]));
          const float e1 = ex2(fmaf(x[t][2 * y + 1], p.scale_log2, -mu[1]));
          const uint32_t pk = pack_bf16(e0, e1);
          l[t][0] += e0;
          l[t][1] += e1;
          lr[t][0] += __uint_as_float(pk << 16);
          lr[t][1] += __uint_as_float(pk & 0xffff0000u);
          pb[t][y] = transpose8x8(pk);
        }
      }
      // ---- values
      {
        uint32_t w[4][kVW], sc[4];  // values 2 c, 2 c + 1, 2 c + 8, 2 c + 9
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int kx = 2 * c + (y & 1) + 8 * (y >> 1);
          lds_words<kVW>(st + L::kCodes + kx * code_bytes(D) + g * (4 * kVW), w[y]);
          sc[y] = lds_u16(st + 2 * L::kCodes + L::kScales + kx * scale_bytes(D) + (g * (D / 8) / kGroup4) * 2);
          if (masked && (key + kx < lo || key + kx >= hi)) sc[y] = 0;  // slots that no row sees may hold NaN
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
#pragma unroll
        for (int j = 0; j < kMT; ++j) {
          uint32_t a[4];
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // d = 128: tile j has dims 16 g + j and 16 g + 8 + j; d = 64: 8 g + 2 j and 8 g + 2 j + 1.
              const uint32_t src = D == 128 ? z[y][h & (kVW - 1)][j & 1] : z[y][0][h];
              a[2 * y + h] = fma_bf16x2(code_pair(src, D == 128 ? j >> 1 : j), s2[y], cs[y]);
            }
#pragma unroll
          for (int t = 0; t < NT; ++t) mma16816(o[j][t], a, pb[t][0], pb[t][1]);
        }
      }
      __syncwarp();  // the stage is read: the next copies may overwrite it
    }

    // ---- join the four warps, 8 rows at a time
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          l[t][h] += __shfl_xor_sync(0xffffffffu, l[t][h], off);
          lr[t][h] += __shfl_xor_sync(0xffffffffu, lr[t][h], off);
        }
    const bool whole = s.first && s.last;
    const int c0 = s.c0, c1 = s.c1, q0 = s.q0, head = s.head;
    float* slot = p.part + (size_t)(2 * blockIdx.x + (s.first ? 1 : 0)) * row_part(D, kRows);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (8 * t >= rows) break;
      __syncthreads();  // the rows that stood here have been read
      // Rows 2 c and 2 c + 1 of this lane, dims from g * D / 8 on; 16-byte chunk x of row r at x ^ r.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 2 * c + h, at = warp * 8 + r;
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {  // dims 4 q .. of the lane's
          float4 v;
          float* f = reinterpret_cast<float*>(&v);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int dim = 4 * q + i;
            f[i] = D == 128 ? o[(dim & 7) % kMT][t][2 * (dim >> 3) + h] : o[(dim >> 1) % kMT][t][2 * (dim & 1) + h];
          }
          *reinterpret_cast<float4*>(merge + at * D + (((g * (D / 32) + q) ^ r) << 2)) = v;
        }
        if (g == 0) {
          stat[at * 3] = m[t][h];
          stat[at * 3 + 1] = l[t][h];
          stat[at * 3 + 2] = lr[t][h];
        }
      }
      __syncthreads();
      const int hr = threadIdx.x >> 4, row = hr + 8 * t, ch = threadIdx.x & 15;  // 16 threads per row
      float M = -INFINITY, Ls = 0.f, Lr = 0.f;
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, stat[(w * 8 + hr) * 3]);
      const float Mu = M == -INFINITY ? 0.f : M;
      float4 acc[D / 64];
#pragma unroll
      for (int i = 0; i < D / 64; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) {
        const float* sw = stat + (w * 8 + hr) * 3;
        const float f = ex2(sw[0] - Mu);
        Ls += f * sw[1];
        Lr += f * sw[2];
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(merge + (w * 8 + hr) * D + (((ch + 16 * i) ^ hr) << 2));
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
          for (int i = 0; i < D / 64; ++i) out = put_row<D>(p, q0, head, r0 + row, 4 * (ch + 16 * i), acc[i], Lr);
          if (ch == 0) p.lse[out] = (M + log2f(Ls)) * 0.6931471805599453f;
        } else {
#pragma unroll
          for (int i = 0; i < D / 64; ++i) *reinterpret_cast<float4*>(slot + row * D + 4 * (ch + 16 * i)) = acc[i];
          if (ch == 0) {
            slot[kRows * D + row] = M;
            slot[kRows * (D + 1) + row] = Ls;
            slot[kRows * (D + 2) + row] = Lr;
          }
        }
      }
    }
    if (k + 1 < fetched) load_q(queue[(k + 1) % L::kSlots]);  // on its way beside what follows
    if (!whole && p.row_share != nullptr) {
      if (c0 == (int)blockIdx.x && threadIdx.x == 0) p.row_share[c0] = RowShare{c1, q0, (int)r0, rows, head};
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
      if (*flag != 0) join_row_tile<D, kRows>(p, c0, c1, q0, head, r0, rows);
    }
    if (k + 1 < fetched) place_q();
  }
  if (*ctl.abort)  // every copy in flight lands before shared memory is given up
    for (uint32_t x = copied > L::kStages ? copied - L::kStages : 0; x < copied; ++x)
      drain_wait(bar(x % L::kStages), (x / L::kStages) & 1);
  if (p.tile_ctas > 0) join_pairs<D>(p);
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
  cfg.blockDim = dim3(kRowThreads);
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

size_t paged4_rows_workspace_bytes(int d, int row_tile) {
  const size_t ctas = (size_t)row4_ctas(row_tile) * kPagedSms;
  return plan_up(2 * ctas * row_part(d, row_tile) * 4) + plan_up(ctas * sizeof(RowShare));
}

// Tiles of 8 columns: one where no tile of the batch can have more than 8 rows, two for 16, four for 32.
cudaError_t launch_paged4_rows(PagedFwd& p, const PagedCache4& cache, int d, int num_sms, cudaStream_t st) {
  const bool few = (long long)p.b.max_q * p.b.G <= 8;
  if (d == 128) {
    if (p.b.row_tile == 32) return launch_rows4<128, 4>(p, cache, num_sms, st);
    return few ? launch_rows4<128, 1>(p, cache, num_sms, st) : launch_rows4<128, 2>(p, cache, num_sms, st);
  }
  if (p.b.row_tile == 32) return launch_rows4<64, 4>(p, cache, num_sms, st);
  return few ? launch_rows4<64, 1>(p, cache, num_sms, st) : launch_rows4<64, 2>(p, cache, num_sms, st);
}

}  // namespace fa
