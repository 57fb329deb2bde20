// fa_paged_weights.cu -- the attention weight that each cached token receives from a step's new tokens.
//
// For slot t of sequence s and kv head h, over the new tokens j that see t and the query heads i that share h:
//     out[t] = old[t] + sum_ij exp(scale q_ij . k_t - lse_ij),       old[t] = 0 where t is a token of this step.
// lse is the attention's, so no maximum is carried and no key needs another: each block of 128 keys is one CTA's, and its sum
// is formed in a fixed order (the same bits at every call). In place, sums are added by atomics, since sequences may share pages.
//
// What has to be read is each key once. A warp holds 32 keys as A operands (m16n8k16), straight from global memory: which
// dims a step of the product takes is free as long as keys and queries agree, so a lane's 16-byte loads are its operands.
// CTAs take blocks by their sequences' share of the plan's units.
//
// The queries go by as columns, 8 rows at a time, from shared memory: 64 rows in the order of the lanes' operands, with
// their -lse in base 2, so that a tile costs its products, exponentials and sums and few instructions more. Up to 64 rows
// stay from block to block of a head; more are copied anew for each block, 64 beside the products of the 64 before. Tiles whose
// rows see every key of a unit go by without masks, but for 64 rows with an lse of -inf among them, whose scores may be anything.
//
// Measured, 16 heads, d = 64, the last 32 tokens of 8 prompts of 4001 to 16000 4-bit keys: 36 us; 48.7 with queries and
// their places worked out by each warp from global memory. 1000 tokens of 32 heads over 9000 bf16 keys of 8 kv heads: 169 us
// at d = 64, 356 at d = 128 (345 without the look for an lse of -inf). A decode step of 64 sequences of 200 to 8192 bf16 keys,
// d = 128, 8 kv heads (582 MB): 93 us, 6.2 TB/s. So a single token is bound by memory, and many rows by latencies at 12 to 16
// warps per SM.
#include <math.h>
#include <type_traits>

#include "fa_paged_evict.cuh"
#include "fa_paged_join.cuh"

namespace fa {

constexpr int kWeightThreads = 128;
// Granules of 16 keys that a warp holds: 64 or 32 registers of operands. (64 keys at d = 64: the 1000 tokens 239 us, the last
// 32 tokens of prompts 37.0.)
constexpr int kGrans = 2;
// CTAs per SM: what registers leave room for. (One more at d = 128: 106 us for the decode step; at d = 64 42 for the prompts.)
__host__ __device__ constexpr int weight_ctas(int D) { return D == 64 ? 4 : 3; }
constexpr int kRows = 64;  // rows of queries in shared memory at a time
// A unit of the plan's pairs (256 rows of 128 keys) in units of its small tiles. (Five batches of chunks beside single tokens,
// each over bf16 and 4-bit keys, geometric mean at d = 64: 146 us with 5, 132 with 7, 140 with 11, 156 with 16; at d = 128
// 234, 226, 214 and 215.)
__host__ __device__ constexpr long long pair_share(int D) { return D == 64 ? 7 : 11; }

// a / b of numbers that are rarely beyond 32 bits (in 64 bits the division takes over a hundred instructions).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((unsigned long long)(a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// In place and with several sequences, a step's new token may stand in a page that another sequence sees too: its slot is set
// to 0 here, before the sums, which then all add to it. (A decode step of 64 sequences in place: 92.8 us, into another tensor 90.1;
// three prompts of 3200 tokens in all: 234 and 224.)
constexpr int kClearThreads = 256, kClearHeads = 8, kClearTokens = kClearThreads / kClearHeads;
__global__ void __launch_bounds__(kClearThreads) fa_paged_weights_clear_kernel(const PagedWeights p) {
  const PagedBatch& b = p.b;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long t = (long long)blockIdx.x * kClearTokens + threadIdx.x / kClearHeads;
  if (t >= b.T || !plan_matches(b, b.d)) return;  // (the sums' kernel reports a plan or a page that is not there)
  int lo = 0, hi = b.S;  // the last sequence that starts at or before the token
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.plan.seq[mid].q0 <= t) lo = mid;
    else hi = mid;
  }
  const PlanSeq s = b.plan.seq[lo];
  const int j = (int)(t - s.q0), pos = s.kvl - s.ql + j;
  if (j < 0 || j >= s.ql || pos < 0) return;
  const int page = b.table[(long long)lo * b.table_stride + (pos >> b.page_shift)];
  if ((unsigned)page >= (unsigned)b.num_pages) return;
  float* out = p.out + (long long)page * p.out_page + (pos & (b.page_size - 1));
  for (int h = threadIdx.x % kClearHeads; h < b.Hkv; h += kClearHeads) out[h * p.out_head] = 0.f;
}

template <int D, bool kPacked>
__global__ void __launch_bounds__(kWeightThreads, weight_ctas(D)) fa_paged_weights_kernel(const PagedWeights p) {
  constexpr int kT = kGrans, kKeys = 16 * kT, kBlk = kWeightThreads / 32 * kKeys;
  __shared__ uint4 q_s[2][kRows / 8][D / 32][32];  // queries of kRows rows as B operands: a tile's i-th 16 bytes of each lane
  __shared__ float2 l_s[2][kRows / 2];             // -lse in base 2 of two rows
  const PagedBatch& b = p.b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  auto start = [&](long long s) { return b.plan.units[0][s] + pair_share(D) * b.plan.units[1][s]; };
  const long long W = start(b.S), per = quotient(W + gridDim.x - 1, gridDim.x);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // new tokens' slots are 0, if a kernel before sets them
  if (!plan_matches(b, D)) {
    if (threadIdx.x == 0) record_index_error(b.status);
    return;
  }
  // CTAs that are likely to stand on one SM (every gridDim / weight_ctas-th) have shares side by side, so that each SM's sum is
  // even where a share is a block or two: else those with two may all meet on the same SMs (399 us for the 1000 tokens at
  // d = 128).
  const unsigned sms = gridDim.x / weight_ctas(D), share = blockIdx.x % sms * weight_ctas(D) + blockIdx.x / sms;
  const long long u = per * share, u_end = min(W, u + per);
  if (u >= u_end) return;
  int seq = 0;  // the last sequence that starts at or before u
  for (int hi = b.S; hi - seq > 1;) {
    const int step = (hi - seq + 31) / 32;
    const long long at = seq + (long long)(lane + 1) * step;
    const int k = __popc(__ballot_sync(0xffffffffu, at < hi && start(at) <= u));
    seq += k * step;
    hi = min(hi, seq + step);
  }
  const unsigned G = b.G;
  const uint32_t by_G = 0xffffffffu / G + 1;  // a product's high half is the quotient of up to 2^16 rows
  int buf = 0;  // the queries' buffer in turn
  for (bool begin = true; seq < b.S; ++seq, begin = false) {
    const long long base = start(seq);
    if (base >= u_end) break;
    const long long per_head = quotient(start(seq + 1) - base, b.Hkv);
    const PlanSeq ps = b.plan.seq[seq];
    if (per_head <= 0 || ps.ql <= 0) continue;
    int lo, hi;  // keys that some new token sees
    key_range(0, ps.ql - 1, ps.ql, ps.kvl, b.causal, b.window, lo, hi);
    hi = min(hi, ps.kvl);
    if (hi <= lo) continue;
    const int blk0 = lo / kBlk, nblk = (hi - 1) / kBlk - blk0 + 1;
    const int first_new = ps.kvl - ps.ql, rows_all = ps.ql * (int)G;
    const bool few = rows_all <= kRows;  // the queries stay from block to block
    const int* tab = b.table + (long long)seq * b.table_stride;
    int head = 0;
    int k = 0;
    if (begin && u > base) {  // block k of a head begins at unit floor(k per_head / nblk) of it
      head = (int)quotient(u - base, per_head);
      const long long off = u - base - head * per_head;
      k = (int)quotient(off * nblk + per_head - 1, per_head);
      if (k == nblk) {
        ++head;
        k = 0;
      }
    }
    // Table entries of a warp's granules of 16 keys, -1 for those that no token sees.
    auto entries = [&](int key0, int (&page)[kT]) {
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        const int at = key0 + 16 * t;
        page[t] = at < hi && at + 16 > lo ? tab[at >> b.page_shift] : -1;
      }
    };
    for (; head < b.Hkv; ++head, k = 0) {
      // kRows rows from r0 on, into the other buffer than that being read. (One barrier between two calls is enough.) Behind the
      // last row its tile is filled up with copies of it at weight 0: of zeros, an infinite key would make NaN.
      float z[kRows * 4 / kWeightThreads] = {};  // lse of the rows whose copies are under way
      auto stage = [&](int r0) {
        buf ^= 1;
#pragma unroll
        for (int y = 0; y < kRows * 4 / kWeightThreads; ++y) {
          const int j = warp + y * (kWeightThreads / 32);
          if (r0 + 8 * j >= rows_all) break;
          const int r = r0 + 8 * j + g;
          const bool in = r < rows_all;
          const unsigned rr = in ? r : rows_all - 1, tok = rr < 65536 && G > 1 ? __umulhi(rr, by_G) : rr / G, hd = rr - tok * G;
          const __nv_bfloat16* src = p.q + (long long)(ps.q0 + (int)tok) * p.q_tok + (long long)(head * G + hd) * p.q_head +
                                     c * (kPacked ? D / 4 : 8);
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            cp_async16(smem_u32(&q_s[buf][j][i][lane]), src + (kPacked ? 8 * i : 32 * i));
          if (c == 0) z[y] = in ? p.lse[(long long)(ps.q0 + (int)tok) * b.Hq + head * (int)G + hd] : INFINITY;
        }
      };
      bool shut = false;  // a row that is staged has lse = -inf: among this thread's, and after a barrier among all
      // Their -lse, once it is here: later than the copies go out, so that no warp waits for it before its products.
      auto stage_lse = [&]() {
        shut = false;
#pragma unroll
        for (int y = 0; y < kRows * 4 / kWeightThreads; ++y) {
          shut = shut || z[y] == -INFINITY;
          if (c == 0)
            reinterpret_cast<float*>(l_s[buf])[8 * (warp + y * (kWeightThreads / 32)) + g] =
                z[y] == -INFINITY ? -INFINITY : z[y] * -1.4426950408889634f;
        }
      };
      // This lane's place in a key (and its scale's), and of keys g of each granule.
      const long long k_tok = kPacked ? code_bytes(D) : p.c.k_tok * 2, k_page = kPacked ? p.c4.k_page : p.c.k_page * 2;
      const uint8_t* k_head = kPacked ? p.c4.k + head * p.c4.k_head
                                      : reinterpret_cast<const uint8_t*>(p.c.k + head * p.c.k_head);
      const uint8_t* k_lane = k_head + c * (kPacked ? D / 8 : 16) + g * k_tok;
      const uint8_t* s_lane =
          kPacked ? p.c4.k_scale + head * p.c4.ks_head + g * scale_bytes(D) + c * (D / 4) / kGroup4 * 2 : nullptr;
      float* out_lane = p.out + head * p.out_head;
      const float* old_lane = p.old + head * p.old_head;
      int page[kT], page_next[kT];
      {
        const int key0 = (blk0 + k) * kBlk + warp * kKeys;
        entries(key0, page);
        entries(key0 + kBlk, page_next);
      }
      const long long left = u_end - base - head * per_head;  // units of the head that are this CTA's
      if (left <= 0) return;
      if (few) {
        stage(0);
        stage_lse();
        cp_async_wait_all();
        shut = __syncthreads_or(shut);
      }
      const int k_end = left >= per_head ? nblk : (int)quotient(left * nblk + per_head - 1, per_head);
      // (As code of its own for few rows: with one loop for both, the decode step over 4-bit keys took 159 us in place of 137.)
      auto blocks = [&](auto small) {
        constexpr bool kFew = decltype(small)::value;
        for (; k < k_end; ++k) {
          const int key0 = (blk0 + k) * kBlk + warp * kKeys;
          // Rows that see a key of the block: [r_lo, r_hi), one of this warp's unit: [r, r_end), every key of it: [full,
          // full_end).
          int r_lo = 0, r_hi = rows_all, r = 0, r_end = rows_all, full_end = rows_all;
          int full = key0 + kKeys <= ps.kvl ? 0 : rows_all;
          if (b.causal) {
            const int blk_key = key0 - warp * kKeys;
            auto rows_to = [&](int tok) { return min(max(tok, 0), ps.ql) * (int)G; };
            r_lo = rows_to(blk_key - first_new) & ~7;
            r = rows_to(key0 - first_new) & ~7;
            full = rows_to(key0 + kKeys - 1 - first_new);
            if (b.window > 0) {
              auto before = [&](int key) {  // rows whose windows begin at or before the key
                return (int)min(max((long long)key + b.window - first_new, 0LL), (long long)ps.ql) * (int)G;
              };
              r_hi = before(blk_key + kBlk - 1);
              r_end = before(key0 + kKeys - 1);
              full_end = before(key0);
            }
          }
          if (key0 >= hi || key0 + kKeys <= lo) r_end = 0;
          if (!kFew && r_lo < r_hi) {
            stage(r_lo);
            stage_lse();
          }
          bool whole = key0 >= lo && key0 + kKeys <= hi;  // every key of the unit is seen
#pragma unroll
          for (int t = 0; t < kT; ++t) {
            const int at = key0 + 16 * t;
            if (at < hi && at + 16 > lo && (unsigned)page[t] >= (unsigned)b.num_pages) {  // (-1 may stand in the table too)
              record_index_error(b.status);
              page[t] = -1;
            }
            whole = whole && page[t] >= 0;
          }
          // ---- keys g, g + 8 of each granule as A operands
          uint32_t a[kT][D / 16][4];
          auto read = [&](int t, auto all) {
            const int at = key0 + 16 * t, slot = at & (b.page_size - 1);
            const long long pg = decltype(all)::value || page[t] >= 0 ? page[t] : 0;
            const uint8_t* row = k_lane + (kPacked ? (uint64_t)(uint32_t)pg * (uint32_t)k_page : (uint64_t)(pg * k_page)) +
                                 slot * k_tok;
            [[maybe_unused]] const uint8_t* scale =
                s_lane + (kPacked ? (uint64_t)(uint32_t)pg * (uint32_t)p.c4.ks_page + slot * scale_bytes(D) : 0);
#pragma unroll
            for (int h = 0; h < 2; ++h, row += 8 * k_tok) {
              const int key = at + 8 * h + g;
              const bool in = decltype(all)::value || (page[t] >= 0 && key >= lo && key < hi);
              if constexpr (kPacked) {
                uint32_t w[D / 32];
                if constexpr (D == 128) {
                  const uint4 v = in ? *reinterpret_cast<const uint4*>(row) : make_uint4(0, 0, 0, 0);
                  w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                } else {
                  const uint2 v = in ? *reinterpret_cast<const uint2*>(row) : make_uint2(0, 0);
                  w[0] = v.x, w[1] = v.y;
                }
                const uint32_t s2 = in ? *reinterpret_cast<const uint16_t*>(scale + 8 * h * scale_bytes(D)) * 0x10001u : 0u;
                const uint32_t cs = scale_shift(s2);
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    a[t][i][2 * e + h] = fma_bf16x2(code_pair(w[i >> 1], 2 * (i & 1) + e), s2, cs);
              } else {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                  const uint4 v = in ? *reinterpret_cast<const uint4*>(row + 64 * i) : make_uint4(0, 0, 0, 0);
                  a[t][2 * i][h] = v.x;
                  a[t][2 * i][2 + h] = v.y;
                  a[t][2 * i + 1][h] = v.z;
                  a[t][2 * i + 1][2 + h] = v.w;
                }
              }
            }
          };
          if (__all_sync(0xffffffffu, whole)) {
#pragma unroll
            for (int t = 0; t < kT; ++t) read(t, std::true_type());
          } else {
#pragma unroll
            for (int t = 0; t < kT; ++t) read(t, std::false_type());
          }
          // This lane's keys for the sums: number c + 4 y of (granule, first or second eight), of those the g-th.
          float old[kT / 2];
          float* out[kT / 2];
          bool adds[kT / 2];
#pragma unroll
          for (int y = 0; y < kT / 2; ++y) {
            const int my = key0 + 32 * y + 8 * c + g, pg = c < 2 ? page[2 * y] : page[2 * y + 1];
            const unsigned slot = my & (b.page_size - 1);
            const bool mine = pg >= 0 && my >= lo && my < hi, was = my < first_new;
            out[y] = mine ? out_lane + (uint64_t)(uint32_t)pg * (uint32_t)p.out_page + slot : nullptr;
            adds[y] = (was || p.cleared) && p.old == p.out;  // (pages may be shared by sequences)
            old[y] = mine && was && !adds[y] ? old_lane[(uint64_t)(uint32_t)pg * (uint32_t)p.old_page + slot] : 0.f;
          }
#pragma unroll
          for (int t = 0; t < kT; ++t) page[t] = page_next[t];
          // The next block's keys on their way into L2: lane i brings key i.
          if (!kPacked && k + 1 < nblk) {
#pragma unroll
            for (int y = 0; y < kT / 2; ++y) {
              const int key = key0 + kBlk + 32 * y + lane, pg = lane < 16 ? page[2 * y] : page[2 * y + 1];
              if (pg >= 0 && pg < b.num_pages && key < hi) {
                const uint8_t* at = k_head + (long long)pg * k_page + (long long)(key & (b.page_size - 1)) * k_tok;
#pragma unroll
                for (int i = 0; i < D / 64; ++i) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + 128 * i));
              }
            }
          }
          entries(key0 + 2 * kBlk, page_next);
          // ---- rows [r, r_end) that may see them
          float sum[kT][2];
#pragma unroll
          for (int t = 0; t < kT; ++t) sum[t][0] = sum[t][1] = 0.f;
          auto add = [&](int buf, int r, int at, auto some) {  // rows r .. r + 7, which stand from row `at` of a buffer on
            const float2 l2 = l_s[buf][(at >> 1) + c];
            float x[kT][4];
#pragma unroll
            for (int t = 0; t < kT; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) x[t][e] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {  // (the granules' products take turns, not each its own sum's steps)
              const uint4 q = q_s[buf][at >> 3][i][lane];
#pragma unroll
              for (int t = 0; t < kT; ++t) mma16816(x[t], a[t][2 * i], q.x, q.y);
#pragma unroll
              for (int t = 0; t < kT; ++t) mma16816(x[t], a[t][2 * i + 1], q.z, q.w);
            }
            int klim[2], klo[2];
            if (decltype(some)::value) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int pos = first_new + (int)((unsigned)(r + 2 * c + e) / G);
                klim[e] = b.causal ? min(pos, ps.kvl - 1) : ps.kvl - 1;
                klo[e] = mask_from(pos, b.window);
              }
            }
#pragma unroll
            for (int t = 0; t < kT; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float l = e & 1 ? l2.y : l2.x;
                float w = ex2(fmaf(x[t][e], p.scale_log2, l));
                if (decltype(some)::value) {
                  const int key = key0 + 16 * t + 8 * (e >> 1) + g;
                  w = key <= klim[e & 1] && key >= klo[e & 1] && l != -INFINITY ? w : 0.f;
                }
                sum[t][e >> 1] += w;
              }
          };
          for (int first = kFew ? 0 : r_lo; first < r_hi; first += kRows) {
            const int here = buf;
            if (!kFew) {
              cp_async_wait_all();
              shut = __syncthreads_or(shut);  // these rows are there, and nobody reads the other buffer any more
              if (first + kRows < r_hi) stage(first + kRows);
            }
            const int to = min(first + kRows, r_end);
            int r8 = max(first, r);
            const int from = min(max(r8, (full + 7) & ~7), to);  // [from, until): tiles whose rows see all
            // (With a row of lse = -inf among them none: it gives no weight where its score is NaN or infinite either.)
            const int until = shut ? from : (full_end == rows_all ? to : max(from, min(to, full_end & ~7)));
#pragma unroll 1
            for (; r8 < from; r8 += 8) add(here, r8, r8 - first, std::true_type());
#pragma unroll 1
            for (; r8 < until; r8 += 8) add(here, r8, r8 - first, std::false_type());
#pragma unroll 1
            for (; r8 < to; r8 += 8) add(here, r8, r8 - first, std::true_type());
            if (!kFew && first + kRows < r_hi) stage_lse();
          }
          float total[kT / 2];
#pragma unroll
          for (int i = 0; i < 2 * kT; ++i) {
            float v = sum[i >> 1][i & 1];
            v += __shfl_xor_sync(0xffffffffu, v, 1);
            v += __shfl_xor_sync(0xffffffffu, v, 2);
            if ((i & 3) == c) total[i >> 2] = v;
          }
#pragma unroll
          for (int y = 0; y < kT / 2; ++y) {
            if (out[y] == nullptr) continue;
            if (adds[y]) atomicAdd(out[y], total[y]);
            else *out[y] = old[y] + total[y];
          }
        }
      };
      if (few) blocks(std::true_type());
      else blocks(std::false_type());
    }
  }
}

cudaError_t launch_paged_weights(PagedWeights& p, int d, bool packed, int num_sms, cudaStream_t st) {
  p.cleared = p.old == p.out && p.b.S > 1;
  if (p.cleared) {
    fa_paged_weights_clear_kernel<<<(unsigned)((p.b.T + (long long)kClearTokens - 1) / kClearTokens), kClearThreads, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(weight_ctas(d) * num_sms);
  cfg.blockDim = dim3(kWeightThreads);
  cfg.stream = st;
  cudaLaunchAttribute early;  // its first look-ups beside the clearing
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = p.cleared ? 1 : 0;
  if (d == 128)
    return packed ? cudaLaunchKernelEx(&cfg, fa_paged_weights_kernel<128, true>, p)
                  : cudaLaunchKernelEx(&cfg, fa_paged_weights_kernel<128, false>, p);
  return packed ? cudaLaunchKernelEx(&cfg, fa_paged_weights_kernel<64, true>, p)
                : cudaLaunchKernelEx(&cfg, fa_paged_weights_kernel<64, false>, p);
}

}  // namespace fa
