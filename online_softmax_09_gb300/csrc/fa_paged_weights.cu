// fa_paged_weights.cu -- the attention weight that each cached token receives from a step's new tokens.
//
// For slot t of sequence s and kv head h, over the new tokens j that see t and the query heads i that share h:
//     out[t] = old[t] + sum_ij exp(scale q_ij . k_t - lse_ij),       old[t] = 0 where t is a token of this step.
// lse is the attention's, so no maximum is carried and no key needs another: each block of 128 keys is one CTA's, and its sum
// is formed in a fixed order (the same bits at every call).
//
// What has to be read is each key once. A warp holds 32 keys as A operands (m16n8k16), straight from global memory: which
// dims a step of the product takes is free as long as keys and queries agree, so a lane's 16-byte loads are its operands.
// The queries go by as columns, 8 at a time. CTAs take blocks by their sequences' share of the plan's units.
#include <math.h>

#include "fa_paged_evict.cuh"
#include "fa_paged_join.cuh"

namespace fa {

constexpr int kWeightThreads = 128;
constexpr int kWeightKeys = 32;   // of a warp
constexpr int kWeightBlk = kWeightThreads / 32 * kWeightKeys;
constexpr int kWeightCtas = 4;    // per SM
constexpr long long kPairShare = 16;  // a unit of the plan's pairs (256 rows of 128 keys), in units of its small tiles

template <int D, bool kPacked>
__global__ void __launch_bounds__(kWeightThreads, kWeightCtas) fa_paged_weights_kernel(const PagedWeights p) {
  const PagedBatch& b = p.b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  auto start = [&](long long s) { return b.plan.units[0][s] + kPairShare * b.plan.units[1][s]; };
  const long long W = start(b.S), per = (W + gridDim.x - 1) / gridDim.x;
  if (!plan_matches(b, D)) {
    if (threadIdx.x == 0) record_index_error(b.status);
    return;
  }
  const long long u = per * blockIdx.x, u_end = min(W, u + per);
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
  const int q8 = (int)(8 / G), r8 = (int)(8 % G);  // 8 rows on: tokens and heads
  for (bool begin = true; seq < b.S; ++seq, begin = false) {
    const long long base = start(seq);
    if (base >= u_end) break;
    const long long per_head = (start(seq + 1) - base) / b.Hkv;
    const PlanSeq ps = b.plan.seq[seq];
    if (per_head <= 0 || ps.ql <= 0) continue;
    int lo, hi;  // keys that some new token sees
    key_range(0, ps.ql - 1, ps.ql, ps.kvl, b.causal, b.window, lo, hi);
    if (b.causal) hi = min(hi, ps.kvl);
    if (hi <= lo) continue;
    const int blk0 = lo / kWeightBlk, nblk = (hi - 1) / kWeightBlk - blk0 + 1;
    const int first_new = ps.kvl - ps.ql, rows_all = ps.ql * (int)G;
    const int* tab = b.table + (long long)seq * b.table_stride;
    int head = 0;
    long long k = 0;
    if (begin && u > base) {  // block k of a head begins at unit floor(k per_head / nblk) of it
      head = (int)((u - base) / per_head);
      const long long off = u - base - head * per_head;
      k = (off * nblk + per_head - 1) / per_head;
      if (k == nblk) {
        ++head;
        k = 0;
      }
    }
    for (; head < b.Hkv; ++head, k = 0) {
      for (; k < nblk; ++k) {
        if (base + head * per_head + k * per_head / nblk >= u_end) return;
        const int key0 = (blk0 + (int)k) * kWeightBlk + warp * kWeightKeys;
        if (key0 >= hi || key0 + kWeightKeys <= lo) continue;
        // ---- keys g, g + 8 of both halves as A operands
        int page[2];
        uint32_t a[2][D / 16][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int at = key0 + 16 * t;
          page[t] = -1;
          if (at < hi && at + 16 > lo) {
            page[t] = tab[at >> b.page_shift];
            if ((unsigned)page[t] >= (unsigned)b.num_pages) {
              record_index_error(b.status);
              page[t] = -1;
            }
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = key0 + 16 * t + 8 * h + g;
            const int slot = key & (b.page_size - 1);
            const bool in = page[t] >= 0 && key >= lo && key < hi;
            if constexpr (kPacked) {
              const uint8_t* kp = p.c4.k + (long long)page[t] * p.c4.k_page + head * p.c4.k_head + slot * code_bytes(D) + c * (D / 8);
              const uint8_t* sp = p.c4.k_scale + (long long)page[t] * p.c4.ks_page + head * p.c4.ks_head +
                                  slot * scale_bytes(D) + c * (D / 4) / kGroup4 * 2;
              uint32_t w[D / 32];
              if constexpr (D == 128) {
                const uint4 v = in ? *reinterpret_cast<const uint4*>(kp) : make_uint4(0, 0, 0, 0);
                w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
              } else {
                const uint2 v = in ? *reinterpret_cast<const uint2*>(kp) : make_uint2(0, 0);
                w[0] = v.x, w[1] = v.y;
              }
              const uint32_t s2 = in ? *reinterpret_cast<const uint16_t*>(sp) * 0x10001u : 0u, cs = scale_shift(s2);
#pragma unroll
              for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  a[t][i][2 * e + h] = fma_bf16x2(code_pair(w[i >> 1], 2 * (i & 1) + e), s2, cs);
            } else {
              const uint4* kp = reinterpret_cast<const uint4*>(p.c.k + (long long)page[t] * p.c.k_page +
                                                               head * p.c.k_head + (in ? slot : 0) * p.c.k_tok) + c;
#pragma unroll
              for (int i = 0; i < D / 32; ++i) {
                const uint4 v = in ? kp[4 * i] : make_uint4(0, 0, 0, 0);
                a[t][2 * i][h] = v.x;
                a[t][2 * i][2 + h] = v.y;
                a[t][2 * i + 1][h] = v.z;
                a[t][2 * i + 1][2 + h] = v.w;
              }
            }
          }
        // This lane's key for the sum: (half c / 2, + 8 for odd c, g).
        const int my = key0 + 8 * c + g, my_page = c < 2 ? page[0] : page[1];
        const bool mine = my_page >= 0 && my >= lo && my < hi;
        const long long my_slot = my & (b.page_size - 1);
        float old = 0.f;
        if (mine && my < first_new && p.old != p.out)
          old = p.old[(long long)my_page * p.old_page + head * p.old_head + my_slot];
        // ---- rows [r, r_end) that may see them
        long long r = 0, r_end = rows_all;
        if (b.causal) {
          r = max(0, key0 - first_new) * (long long)G & ~7LL;
          if (b.window > 0) {
            const long long past = (long long)key0 + kWeightKeys - 1 + b.window - first_new;  // tokens from here on do not
            r_end = min(r_end, max(past, 0LL) * G);
          }
        }
        float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
        int tok[3], hd[3];  // of row r + g (as a column of queries), and of rows r + 2 c, r + 2 c + 1
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const unsigned rr = (unsigned)r + (i == 0 ? g : 2 * c + i - 1);
          tok[i] = (int)(rr / G);
          hd[i] = (int)(rr - tok[i] * G);
        }
        for (; r < r_end; r += 8) {
          const __nv_bfloat16* qp = p.q + (long long)(ps.q0 + tok[0]) * p.q_tok + ((long long)head * G + hd[0]) * p.q_head;
          const bool q_in = tok[0] < ps.ql;
          uint4 qv[D / 32];
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            qv[i] = q_in ? *reinterpret_cast<const uint4*>(qp + (kPacked ? c * (D / 4) + 8 * i : 8 * (c + 4 * i)))
                         : make_uint4(0, 0, 0, 0);
          float l2[2];
          int klim[2], klo[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool in = tok[1 + e] < ps.ql;
            const float z = in ? p.lse[(long long)(ps.q0 + tok[1 + e]) * b.Hq + head * G + hd[1 + e]] : 0.f;
            l2[e] = z == -INFINITY ? INFINITY : z * 1.4426950408889634f;  // a row that sees nothing gives nothing
            const int pos = first_new + tok[1 + e];
            klim[e] = !in ? -1 : (b.causal ? min(pos, ps.kvl - 1) : ps.kvl - 1);
            klo[e] = mask_from(pos, b.window);
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              mma16816(x, a[t][2 * i], qv[i].x, qv[i].y);
              mma16816(x, a[t][2 * i + 1], qv[i].z, qv[i].w);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + 16 * t + 8 * (e >> 1) + g;
              const float w = ex2(fmaf(x[e], p.scale_log2, -l2[e & 1]));
              sum[t][e >> 1] += key <= klim[e & 1] && key >= klo[e & 1] ? w : 0.f;
            }
          }
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            tok[i] += q8;
            hd[i] += r8;
            if (hd[i] >= (int)G) {
              hd[i] -= (int)G;
              ++tok[i];
            }
          }
        }
        float total = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v = sum[i >> 1][i & 1];
          v += __shfl_xor_sync(0xffffffffu, v, 1);
          v += __shfl_xor_sync(0xffffffffu, v, 2);
          if (i == c) total = v;
        }
        if (mine) {
          float* out = p.out + (long long)my_page * p.out_page + head * p.out_head + my_slot;
          if (p.old == p.out && my < first_new) atomicAdd(out, total);  // (pages may be shared by sequences)
          else *out = old + total;
        }
      }
    }
  }
}

cudaError_t launch_paged_weights(const PagedWeights& p, int d, bool packed, int num_sms, cudaStream_t st) {
  const int grid = kWeightCtas * num_sms;
  if (d == 128) {
    if (packed) fa_paged_weights_kernel<128, true><<<grid, kWeightThreads, 0, st>>>(p);
    else fa_paged_weights_kernel<128, false><<<grid, kWeightThreads, 0, st>>>(p);
  } else {
    if (packed) fa_paged_weights_kernel<64, true><<<grid, kWeightThreads, 0, st>>>(p);
    else fa_paged_weights_kernel<64, false><<<grid, kWeightThreads, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace fa
