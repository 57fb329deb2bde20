// fa_paged_join.cuh -- what the kernels of small tiles share (fa_paged.cu, fa_paged4.cu): their shape, outputs, and the
// joining of results that several CTAs hold parts of.
#pragma once

#include <math.h>

#include "fa_paged.cuh"

namespace fa {

constexpr int kRowWarps = 4, kRowThreads = 32 * kRowWarps;
constexpr int kGran = kRowBlk / kRowWarps;  // keys that one warp takes at a time: 16, within one page

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four columns of row rr of a small tile's (sequence, kv head), normalised by `sum`, out; returns the row's place in lse.
template <int D>
__device__ __forceinline__ long long put_row(const PagedFwd& p, int q0, int head, unsigned rr, int col, float4 v,
                                             float sum) {
  const unsigned G = p.b.G;
  const int tok = (int)(rr / G), hd = (int)(rr - tok * G);
  const long long out = (long long)(q0 + tok) * p.b.Hq + head * (int)G + hd;
  const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;  // a row that sees nothing: o = 0
  uint2 w;
  w.x = pack_bf16(v.x * inv, v.y * inv);
  w.y = pack_bf16(v.z * inv, v.w * inv);
  *reinterpret_cast<uint2*>(p.o + out * D + col) = w;
  return out;
}

// The partial results that CTAs c0 to c1 left of a small tile, joined in the order of the keys by one CTA (the last of
// them to arrive).
template <int D, int kRows, int kThreads = kRowThreads>
__device__ __forceinline__ void join_row_tile(const PagedFwd& p, int c0, int c1, int q0, int head, unsigned r0,
                                              int rows) {
  // Four columns of a row per thread, eight results' loads at a time.
  for (int x = threadIdx.x; x < rows * (D / 4); x += kThreads) {
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
    const long long out = put_row<D>(p, q0, head, r0 + rw, col, a, lsr);
    if (col == 0) p.lse[out] = (m0 + log2f(ls)) * 0.6931471805599453f;
  }
}

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

// By kRowThreads threads (the first of the CTA) that meet in `sync`.
template <int D, class Sync>
__device__ __forceinline__ void join_pairs(const PagedFwd& p, Sync sync) {
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
  sync();  // the rows' use of this memory is over
  if (lane == 0) counts[warp] = n;
  sync();
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
  sync();
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

}  // namespace fa
