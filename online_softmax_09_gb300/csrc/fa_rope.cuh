// fa_rope.cuh -- the rotation of a head's pairs and the place of a token, for the kernels that rotate (fa_rope.cu has the
// mathematics).
#pragma once

#include "fa_paged.cuh"

namespace fa {

template <int D>
__device__ __forceinline__ void turn8(uint4& va, uint4& vb, const float4* t, bool interleaved) {
  constexpr int kStep = D / 16;  // t[kStep * i]: cos, sin of this thread's pairs 2i, 2i + 1
  uint32_t* a = reinterpret_cast<uint32_t*>(&va);
  uint32_t* c = reinterpret_cast<uint32_t*>(&vb);
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xffff0000u); };
  if (!interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = t[kStep * i];
      const float x0 = lo(a[i]), x1 = hi(a[i]), y0 = lo(c[i]), y1 = hi(c[i]);
      a[i] = pack_bf16(x0 * f.x - y0 * f.y, x1 * f.z - y1 * f.w);
      c[i] = pack_bf16(y0 * f.x + x0 * f.y, y1 * f.z + x1 * f.w);
    }
  } else {  // words a[0..3], c[0..3] hold pairs 8j .. 8j + 7
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = t[kStep * i];
      uint32_t& w0 = i < 2 ? a[2 * i] : c[2 * i - 4];
      uint32_t& w1 = i < 2 ? a[2 * i + 1] : c[2 * i - 3];
      const float x0 = lo(w0), y0 = hi(w0), x1 = lo(w1), y1 = hi(w1);
      w0 = pack_bf16(x0 * f.x - y0 * f.y, y0 * f.x + x0 * f.y);
      w1 = pack_bf16(x1 * f.z - y1 * f.w, y1 * f.z + x1 * f.w);
    }
  }
}

struct RopeToken {
  long long in[3];   // element offset of the token in q, k, v
  long long out[3];  // and in their outputs; v and k of a paged batch: in the cache
  int pos;           // paged batch without given positions
  int state;         // bit 0: a token of the batch, bit 1: its cache slot exists
  int page, slot;    // of a paged batch, where the cache slot exists
};

// Token t of the grid's dense batch, or of the plan's ragged one.
template <bool kPaged>
__device__ __forceinline__ RopeToken rope_token(const RopeLaunch& p, long long t) {
  RopeToken k = {};
  if (t >= p.tokens) return k;
  if constexpr (!kPaged) {
    const long long bi = t / p.N, n = t - bi * p.N;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      k.in[i] = bi * p.in[i].batch + n * p.in[i].tok;
      k.out[i] = bi * p.out[i].batch + n * p.out[i].tok;
    }
    k.state = 3;
  } else {
    const PagedBatch& b = p.b;
    // The last sequence that starts at or before the token; sequences without tokens share a start.
    int lo = 0, hi = b.S;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (b.plan.seq[mid].q0 <= t) lo = mid;
      else hi = mid;
    }
    const PlanSeq s = b.plan.seq[lo];
    const long long j = t - s.q0;
    if (j < 0 || j >= s.ql) return k;
    k.state = 1;
    k.pos = s.kvl - s.ql + (int)j;
    k.in[0] = t * p.in[0].tok;
    k.out[0] = t * p.out[0].tok;
    k.in[1] = t * p.in[1].tok;
    k.in[2] = t * p.in[2].tok;
    if (k.pos >= 0) {
      const int page = b.table[(long long)lo * b.table_stride + (k.pos >> b.page_shift)];
      if ((unsigned)page < (unsigned)b.num_pages) {
        const int slot = k.pos & (b.page_size - 1);
        k.out[1] = page * p.out[1].batch + slot * p.out[1].tok;
        k.out[2] = page * p.out[2].batch + slot * p.out[2].tok;
        k.page = page;
        k.slot = slot;
        k.state = 3;
      } else {
        record_index_error(b.status);
      }
    } else {
      record_index_error(b.status);  // more new tokens than the sequence has
    }
  }
  return k;
}

// cos and sin (of the angle to turn by) of pair i at the token with position `pos`.
__device__ __forceinline__ uint64_t turn_fraction(const RopeLaunch& p, int i) {
  const double turns = (double)p.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
  return __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
}
__device__ __forceinline__ float2 turn_angle(const RopeLaunch& p, uint64_t w, long long pos) {
  const int phase = (int)(uint32_t)(((uint64_t)pos * w) >> 32);  // 2^-32 turns, signed
  float s, c;
  sincospif((float)phase * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
  return make_float2(c, p.inverse ? -s : s);
}

}  // namespace fa
