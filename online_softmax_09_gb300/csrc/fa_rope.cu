// fa_rope.cu -- rotary positions: q and k of a dense batch (forward and gradient), and the newest
// tokens of a ragged batch on their way into a paged cache.
//
// Pair i of a head's first `rot` dims, (x_i, x_{i + rot/2}) or (x_{2i}, x_{2i+1}), is turned by
//     phi = pos[axis(i)] * inv_freq[i]:   (a, b) -> (a cos phi - b sin phi, b cos phi + a sin phi);
// the gradient is the same with -phi. The other dims pass through.
//
// Angles. inv_freq / 2 pi is kept as a fraction of a turn in 64-bit fixed point, w = inv_freq / 2 pi * 2^64,
// so pos * w in 64-bit integers drops whole turns exactly, for any 32-bit position. What is lost: the double that
// w comes from is off by 2^-52.3 of itself (the product and the constant; below 0, by 2^-54 of a turn more), times
// pos; the top half keeps 2^-32 of a turn; and as a float the remainder, at most half a turn, keeps 2^-26 of one.
// In all 2^-26 of a turn up to positions of about 2^27, 2^-24 at 2^31. cos and sin follow from cospi and sinpi.
//
// Memory-bound: 2 bytes in and 2 out per element. A thread takes 8 pairs of one head (two 16-byte
// chunks in, two out); the cos and sin of a CTA's tokens are made once, in shared memory, for all heads.
// q and k of 4 x 4096 tokens (40 heads, d = 128) and their gradients back, 671 MB, take 109 us: 6.16 TB/s,
// 92 % of the measured copy rate; 8500 prompt tokens into the cache 34.5 us, 5.9 TB/s; one token 3.8 us.
#include "fa_rope.cuh"

namespace fa {

constexpr int kRopeThreads = 256;  // most threads per CTA
constexpr int kRopeTokens = 2;     // most tokens per CTA

template <int D, bool kPaged>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_kernel(const RopeLaunch p) {
  constexpr int kGroups = D / 16;  // threads per head
  const int slots = blockDim.x / kGroups;
  // cos, sin of pair 8 g + 2 i + e of each token at [i][g][e]: the eight (or four) threads of a head read
  // neighbouring 16 bytes (in the pairs' own order they met in two banks, and this bound the kernel).
  __shared__ __align__(16) float2 cs[kRopeTokens][4][kGroups][2];
  __shared__ RopeToken tok[kRopeTokens];
  const int tid = threadIdx.x;
  if (kPaged && !plan_matches(p.b, D)) {
    if (tid == 0) record_index_error(p.b.status);
    return;
  }
  const long long t0 = (long long)blockIdx.x * p.tile;
  if (tid < p.tile) tok[tid] = rope_token<kPaged>(p, t0 + tid);
  __syncthreads();

  const int np = p.rot >> 1;
  const int g = tid % kGroups, slot = tid / kGroups;
  const bool turned = g < p.rot / 16;
  const int ea = turned && !p.interleaved ? 8 * g : 16 * g;
  const int eb = turned && !p.interleaved ? np + 8 * g : ea + 8;
  const int heads = p.Hq + p.Hk + p.Hv;
  const int total = p.tile * heads;
  int t = slot / heads, h = slot - t * heads;
  uint4 va, vb;
  __nv_bfloat16* dst;
  const float4* angles;
  auto load = [&]() {  // this thread's chunks of head h of token t, then on to its next head
    dst = nullptr;
    angles = nullptr;
    const int part = h < p.Hq ? 0 : (h < p.Hq + p.Hk ? 1 : 2);
    const int hh = h - (part == 0 ? 0 : (part == 1 ? p.Hq : p.Hq + p.Hk));
    const RopeToken& k = tok[t];
    if (k.state == 3 || (k.state == 1 && part == 0)) {
      const __nv_bfloat16* src = p.src[part] + k.in[part] + hh * p.in[part].head;
      dst = p.dst[part] + k.out[part] + hh * p.out[part].head;
      if (turned && part < 2) angles = reinterpret_cast<const float4*>(cs[t][0][g]);
      va = *reinterpret_cast<const uint4*>(src + ea);
      vb = *reinterpret_cast<const uint4*>(src + eb);
    }
    h += slots;
    while (h >= heads) {
      h -= heads;
      ++t;
    }
  };
  if (slot < total) load();  // on its way while the angles are formed
  if (np > 0) {
    const int per = blockDim.x / np;  // tokens at a time
    const int i = tid % np, first = tid / np;
    if (first < per && first < p.tile) {
      const uint64_t w = turn_fraction(p, i);
      const int axis = (int)(p.axes[i >> 5] >> ((i & 31) * 2)) & 3;
      for (int k = first; k < p.tile; k += per) {
        long long pos = 0;
        if (t0 + k < p.tokens) {
          if (p.positions == nullptr) {
            pos = tok[k].pos;
          } else {
            const long long bi = kPaged ? 0 : (t0 + k) / p.N;
            pos = p.positions[axis * p.pos_axis + bi * p.pos_batch + (t0 + k - bi * p.N)];
          }
        }
        cs[k][(i >> 1) & 3][i >> 3][i & 1] = turn_angle(p, w, pos);
      }
    }
  }
  __syncthreads();
  for (int x = slot; x < total; x += slots) {
    if (x != slot) load();
    if (dst == nullptr) continue;
    if (angles != nullptr) turn8<D>(va, vb, angles, p.interleaved);
    *reinterpret_cast<uint4*>(dst + ea) = va;
    *reinterpret_cast<uint4*>(dst + eb) = vb;
  }
}

// Threads and tokens per CTA. While the tokens fit one wave of CTAs (six per SM), one token each with all
// 256 threads: latency counts (17 tokens: 3.2 us a call against 4.1 with two tokens and 128 threads).
// Beyond that 128 threads, and two tokens in a dense batch: sharing the setup pays (4 x 4096 tokens of 40
// heads: 109.6 us for both directions, one token 113.8, 256 threads with four 112.8). A paged batch keeps one:
// its CTA starts with a chain of look-ups, and more CTAs hide more of it (8500 tokens: 34.7 us, two 36.7).
cudaError_t launch_rope(RopeLaunch& p, int d, bool paged, int num_sms, cudaStream_t st) {
  const bool one_wave = p.tokens <= 6LL * num_sms;
  const int threads = one_wave ? kRopeThreads : 128;
  p.tile = one_wave || paged ? 1 : kRopeTokens;
  const long long grid = (p.tokens + p.tile - 1) / p.tile;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (d == 128) {
    if (paged) fa_rope_kernel<128, true><<<(unsigned)grid, threads, 0, st>>>(p);
    else fa_rope_kernel<128, false><<<(unsigned)grid, threads, 0, st>>>(p);
  } else {
    if (paged) fa_rope_kernel<64, true><<<(unsigned)grid, threads, 0, st>>>(p);
    else fa_rope_kernel<64, false><<<(unsigned)grid, threads, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace fa
