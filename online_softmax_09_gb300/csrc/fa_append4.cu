// fa_append4.cu -- new tokens' keys and values into a 4-bit paged cache (fa_paged4.cuh has its layout), keys and queries
// rotated on the way (fa_rope.cu has the rotation).
//
// A group of 32 dims x is stored with s = max|x| / 7 rounded to four significant bits and u = 8 + x / s rounded, ties to even
// both times: |x / s| <= 7 * 17 / 16, so u stays in 1..15 and a value is off by at most s / 2. Keys are rounded to bf16 after
// the rotation, as a bf16 cache would have them, and quantised from that. From bf16 numbers both quotients are nearer to
// a tie than fp32 resolves only where they are at it: the codes are those of exact arithmetic.
//
// One CTA per token. A thread takes eight dims, its four neighbours' lanes a group. Memory-bound for prompts: 2 bytes in per
// element, 0.56 out, and 2 more where the caller wants the values. A few tokens are bound by the chain of plan, table and
// stores.
#include "fa_paged4.cuh"
#include "fa_rope.cuh"

namespace fa {

constexpr int kAppendHeads = 32;  // key heads that are rotated at a time

// Eight values' codes as a word, given their group's scale; and the values that they stand for.
__device__ __forceinline__ uint32_t quantise8(const uint4& x, uint32_t& scale, uint4& stored) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&x);
  uint32_t top = 0;  // the bits of a magnitude order like it, NaN above all
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  uint32_t code = 0x88888888u;
  stored = make_uint4(0, 0, 0, 0);
  uint32_t* out = reinterpret_cast<uint32_t*>(&stored);
  if (top >= kScaleBig) {
    scale = 0x7fc0;
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = 0x7fc07fc0u;
    return code;
  }
  scale = 0;
  if (top < kScaleTiny) return code;
  uint32_t q = __float_as_uint(__fdiv_rn(__uint_as_float(top << 16), 7.f));
  q = (q + 0x7ffffu + ((q >> 20) & 1)) & 0xfff00000u;
  scale = q >> 16;
  const float s = __uint_as_float(q);
  code = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a = rintf(__fdiv_rn(__uint_as_float(w[j] << 16), s));
    const float b = rintf(__fdiv_rn(__uint_as_float(w[j] & 0xffff0000u), s));
    code |= (uint32_t)((int)a + 8) << (4 * j) | (uint32_t)((int)b + 8) << (4 * j + 16);
    out[j] = pack_bf16((a + 0.f) * s, (b + 0.f) * s);
  }
  return code;
}

template <int D>
__global__ void __launch_bounds__(256) fa_paged_append4_kernel(const RopeLaunch p, const Append4 a) {
  constexpr int kGroups = D / 16, kChunks = D / 8;
  __shared__ __align__(16) float2 cs[4][kGroups][2];
  __shared__ __align__(16) __nv_bfloat16 rows[kAppendHeads][D];
  __shared__ RopeToken tok_s;
  const int tid = threadIdx.x;
  if (!plan_matches(p.b, D)) {
    if (tid == 0) record_index_error(p.b.status);
    return;
  }
  const long long t = blockIdx.x;
  if (tid == 0) tok_s = rope_token<true>(p, t);
  const bool rotary = p.rot > 0;
  const int units = p.Hk * kChunks;  // of the keys, and of the values
  uint4 x = make_uint4(0, 0, 0, 0);
  auto load = [&](int u) {  // eight dims of a value or of a key that is not turned
    const int part = u < units ? 0 : 1, r = u - part * units, h = r / kChunks;
    x = *reinterpret_cast<const uint4*>(p.src[1 + part] + t * p.in[1 + part].tok + h * p.in[1 + part].head +
                                        (r % kChunks) * 8);
  };
  const int first = rotary ? units : 0;
  if (first + tid < 2 * units) load(first + tid);  // on its way beside the look-ups
  __syncthreads();
  const RopeToken k = tok_s;
  if (k.state == 0) return;
  auto store = [&](int u, const uint4& y, bool on) {  // by whole groups of four lanes
    uint32_t scale;
    uint4 stored;
    const uint32_t code = quantise8(y, scale, stored);
    if (!on || k.state != 3) return;
    const int part = u < units ? 0 : 1, r = u - part * units, h = r / kChunks, c = r % kChunks;
    uint8_t* codes = const_cast<uint8_t*>(part == 0 ? a.c.k : a.c.v) + (long long)k.page * (part == 0 ? a.c.k_page : a.c.v_page) +
                     h * (part == 0 ? a.c.k_head : a.c.v_head);
    uint8_t* scales = const_cast<uint8_t*>(part == 0 ? a.c.k_scale : a.c.v_scale) +
                      (long long)k.page * (part == 0 ? a.c.ks_page : a.c.vs_page) +
                      h * (part == 0 ? a.c.ks_head : a.c.vs_head);
    *reinterpret_cast<uint32_t*>(codes + k.slot * code_bytes(D) + c * 4) = code;
    if ((c & 3) == 0) *reinterpret_cast<uint16_t*>(scales + k.slot * scale_bytes(D) + (c >> 2) * 2) = (uint16_t)scale;
    if (a.out[part] != nullptr)
      *reinterpret_cast<uint4*>(a.out[part] + t * a.out_tok[part] + h * a.out_head[part] + c * 8) = stored;
  };
  const int lanes = blockDim.x;
  if (rotary) {
    const int np = p.rot >> 1;
    if (tid < np) {
      const int axis = (int)(p.axes[tid >> 5] >> ((tid & 31) * 2)) & 3;
      const long long pos = p.positions == nullptr ? k.pos : p.positions[axis * p.pos_axis + t];
      cs[(tid >> 1) & 3][tid >> 3][tid & 1] = turn_angle(p, turn_fraction(p, tid), pos);
    }
    __syncthreads();
    const int g = tid % kGroups;
    const bool turned = g < p.rot / 16;
    const int ea = turned && !p.interleaved ? 8 * g : 16 * g;
    const int eb = turned && !p.interleaved ? np + 8 * g : ea + 8;
    const float4* angles = reinterpret_cast<const float4*>(cs[0][g]);
    auto turn = [&](const __nv_bfloat16* src, __nv_bfloat16* dst) {
      uint4 va = *reinterpret_cast<const uint4*>(src + ea), vb = *reinterpret_cast<const uint4*>(src + eb);
      if (turned) turn8<D>(va, vb, angles, p.interleaved);
      *reinterpret_cast<uint4*>(dst + ea) = va;
      *reinterpret_cast<uint4*>(dst + eb) = vb;
    };
    for (int h = tid / kGroups; h < p.Hq; h += lanes / kGroups)
      turn(p.src[0] + k.in[0] + h * p.in[0].head, p.dst[0] + k.out[0] + h * p.out[0].head);
    if (k.state == 3) {
      for (int h0 = 0; h0 < p.Hk; h0 += kAppendHeads) {
        const int n = min(kAppendHeads, p.Hk - h0);
        if (h0 > 0) __syncthreads();
        for (int h = tid / kGroups; h < n; h += lanes / kGroups)
          turn(p.src[1] + k.in[1] + (h0 + h) * p.in[1].head, rows[h]);
        __syncthreads();
        for (int w = tid & ~31; w < n * kChunks; w += lanes) {
          const int u = w + (tid & 31);
          const bool on = u < n * kChunks;
          store(h0 * kChunks + u, on ? *reinterpret_cast<const uint4*>(&rows[u / kChunks][(u % kChunks) * 8]) : make_uint4(0, 0, 0, 0),
                on);
        }
      }
    }
  }
  for (int w = tid & ~31; w < 2 * units - first; w += lanes) {
    const int u = first + w + (tid & 31);
    const bool on = u < 2 * units;
    if (w >= lanes && on) load(u);
    store(u, x, on);
  }
}

cudaError_t launch_append4(const RopeLaunch& p, const Append4& a, int d, int num_sms, cudaStream_t st) {
  const int threads = p.tokens <= 6LL * num_sms ? 256 : 128;
  if (d == 128) fa_paged_append4_kernel<128><<<(unsigned)p.tokens, threads, 0, st>>>(p, a);
  else fa_paged_append4_kernel<64><<<(unsigned)p.tokens, threads, 0, st>>>(p, a);
  return cudaGetLastError();
}

}  // namespace fa
