// fa_append4.cu -- new tokens' keys and values into a 4-bit paged cache (fa_paged4.cuh has its layout), keys and queries
// rotated on the way (fa_rope.cu has the rotation).
//
// A group of 32 dims x is stored with s = max|x| / 7 rounded to four significant bits and u = 8 + x / s rounded, ties to even
// both times: |x / s| <= 7 * 17 / 16, so u stays in 1..15 and a value is off by at most s / 2. Keys are rounded to bf16 after
// the rotation, as a bf16 cache would have them, and quantised from that. From bf16 numbers both quotients are nearer to
// a tie than fp32 resolves only where they are at it: the codes are those of exact arithmetic.
//
// One CTA per token or four. A thread takes eight dims, four neighbouring lanes a group. Read are 2 bytes per element, written
// 0.56, and 2 more where the caller wants the values. 8500 tokens of 8 kv heads, d = 128, values wanted (77 MB): 17.7 us,
// 4.4 TB/s, 65 % of the copy rate, at which they would take 11.6; the chain of look-ups before a CTA's stores is the rest. (28 with
// divisions and one token per CTA, 25.5 with reciprocals and four loads per thread.) 1 token 2.5 us, 64 tokens 3.3: that chain
// alone.
#include "fa_paged4.cuh"
#include "fa_rope.cuh"

namespace fa {

constexpr int kAppendHeads = 32;  // key heads that are rotated at a time

// Eight values' codes as a word, given with their group's scale and the values that they stand for. By whole groups of lanes.
//
// Both quotients are products with reciprocals, off by a few units of 2^-23, and their ties are made out by what numbers they
// can be. max|x| / 7 is T 2^f / 7 with T of 8 bits: a tie of four significant bits is a number of five, and any other value is
// off every tie by 2^-12 of itself or more, so the quotient's last four bits may be rounded away first. x / s, where it is 1/4
// or more, is 2^p X / m with integers X < 256, 8 <= m < 16, p >= -6: off every odd multiple of 1/2 by 2^-7 / 15 or more, or
// at it. So 1 / s a little too small and a little too large give the same integer, or the two about a tie, of which the
// even one is taken.
__device__ __forceinline__ uint32_t quantise8(const uint4& x, uint32_t& scale, uint4& stored) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&x);
  uint32_t top = 0;  // the bits of a magnitude order like it, NaN above all
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const bool none = top < kScaleTiny, bad = top >= kScaleBig;
  uint32_t q = (__float_as_uint(__uint_as_float(top << 16) * (1.f / 7.f)) + 8) & ~15u;
  q = (q + 0x7ffffu + ((q >> 20) & 1)) & 0xfff00000u;
  if (none || bad) q = 0x3f800000u;  // (any number: the codes are replaced)
  scale = bad ? 0x7fc0u : (none ? 0u : q >> 16);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__uint_as_float(q)));
  const float low = r * (1.f - 0x1p-21f), high = r * (1.f + 0x1p-21f);
  constexpr uint32_t kBits = 0x4b400000u;  // of 1.5 * 2^23: from there on a float's last bits are an integer
  uint32_t code = 0u - kBits * 0x11111111u;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float y = __uint_as_float(e == 0 ? w[j] << 16 : w[j] & 0xffff0000u);
      const uint32_t a = __float_as_uint(fmaf(y, low, 12582920.f)), b = __float_as_uint(fmaf(y, high, 12582920.f));
      code += ((a & 1) ? b : a) << (4 * j + 16 * e);
    }
  if (none || bad) code = 0x88888888u;
  const uint32_t s2 = scale * 0x10001u, cs = scale_shift(s2);
  stored = make_uint4(fma_bf16x2(code_pair(code, 0), s2, cs), fma_bf16x2(code_pair(code, 1), s2, cs),
                      fma_bf16x2(code_pair(code, 2), s2, cs), fma_bf16x2(code_pair(code, 3), s2, cs));
  return code;
}

// Where chunk c of head h of the keys (part 0) or values goes, but for page, slot and token.
struct Dest4 {
  uint8_t *codes, *scales;  // scales: of the group's first lane, else NULL
  uint32_t code_page, scale_page;
  __nv_bfloat16* out;
  long long out_tok;
};
template <int D>
__device__ __forceinline__ Dest4 dest4(const Append4& a, int part, int h, int c) {
  Dest4 d;
  d.codes = const_cast<uint8_t*>(part == 0 ? a.c.k : a.c.v) + h * (part == 0 ? a.c.k_head : a.c.v_head) + c * 4;
  d.scales = (c & 3) == 0 ? const_cast<uint8_t*>(part == 0 ? a.c.k_scale : a.c.v_scale) +
                                h * (part == 0 ? a.c.ks_head : a.c.vs_head) + (c >> 2) * 2
                          : nullptr;
  d.code_page = (uint32_t)(part == 0 ? a.c.k_page : a.c.v_page);
  d.scale_page = (uint32_t)(part == 0 ? a.c.ks_page : a.c.vs_page);
  d.out = a.out[part] == nullptr ? nullptr : a.out[part] + h * a.out_head[part] + c * 8;
  d.out_tok = a.out_tok[part];
  return d;
}
template <int D>
__device__ __forceinline__ void store4(const Dest4& d, const RopeToken& k, long long t, uint32_t code, uint32_t scale,
                                       const uint4& stored) {
  *reinterpret_cast<uint32_t*>(d.codes + (uint64_t)(uint32_t)k.page * d.code_page + k.slot * code_bytes(D)) = code;
  if (d.scales != nullptr)
    *reinterpret_cast<uint16_t*>(d.scales + (uint64_t)(uint32_t)k.page * d.scale_page + k.slot * scale_bytes(D)) =
        (uint16_t)scale;
  if (d.out != nullptr) *reinterpret_cast<uint4*>(d.out + t * d.out_tok) = stored;
}

// Without a rotation: kTokens per CTA, a thread with the same eight dims of each, which are on their way while the tokens'
// places are looked up.
template <int D, int kTokens>
__global__ void __launch_bounds__(256) fa_paged_append4_kernel(const RopeLaunch p, const Append4 a) {
  constexpr int kChunks = D / 8;
  __shared__ RopeToken tok[kTokens];
  const int tid = threadIdx.x, lanes = blockDim.x, lane = tid & 31;
  const long long t0 = (long long)blockIdx.x * kTokens;
  const int units = p.Hk * kChunks, total = 2 * units;  // eight dims each, of keys, then of values
  uint4 x[kTokens];
  auto load = [&](int u) {
    const int part = u < units ? 0 : 1, r = u - part * units;
    const long long step = p.in[1 + part].tok;
    const __nv_bfloat16* src = p.src[1 + part] + t0 * step + (long long)(r / kChunks) * p.in[1 + part].head + (r % kChunks) * 8;
#pragma unroll
    for (int t = 0; t < kTokens; ++t)
      x[t] = u < total && t0 + t < p.tokens ? *reinterpret_cast<const uint4*>(src + t * step) : make_uint4(0, 0, 0, 0);
  };
  load(tid);
  if (!plan_matches(p.b, D)) {
    if (tid == 0) record_index_error(p.b.status);
    return;
  }
  if (tid < kTokens) tok[tid] = rope_token<true>(p, t0 + tid);
  __syncthreads();
  for (int w = tid & ~31; w < total; w += lanes) {
    const int u = w + lane;
    if (w >= lanes) load(u);
    const int part = u < units ? 0 : 1, r = u - part * units, h = r / kChunks, c = r % kChunks;
    const Dest4 to = dest4<D>(a, part, h, c);
#pragma unroll
    for (int t = 0; t < kTokens; ++t) {
      uint32_t scale;
      uint4 stored;
      const uint32_t code = quantise8(x[t], scale, stored);
      if (u < total && tok[t].state == 3) store4<D>(to, tok[t], t0 + t, code, scale, stored);
    }
  }
}

// With a rotation: one token per CTA; keys are turned into shared memory, and quantised from there.
template <int D>
__global__ void __launch_bounds__(256) fa_paged_append4_rope_kernel(const RopeLaunch p, const Append4 a) {
  constexpr int kGroups = D / 16, kChunks = D / 8;
  __shared__ __align__(16) float2 cs[4][kGroups][2];
  __shared__ __align__(16) __nv_bfloat16 rows[kAppendHeads][D];
  __shared__ RopeToken tok_s;
  const int tid = threadIdx.x, lanes = blockDim.x;
  const long long t = blockIdx.x;
  const int units = p.Hk * kChunks;
  uint4 x = make_uint4(0, 0, 0, 0);
  auto load = [&](int u) {
    x = *reinterpret_cast<const uint4*>(p.src[2] + t * p.in[2].tok + (long long)(u / kChunks) * p.in[2].head + (u % kChunks) * 8);
  };
  if (tid < units) load(tid);  // on its way beside the look-ups
  if (!plan_matches(p.b, D)) {
    if (tid == 0) record_index_error(p.b.status);
    return;
  }
  if (tid == 0) tok_s = rope_token<true>(p, t);
  __syncthreads();
  const RopeToken k = tok_s;
  if (k.state == 0) return;
  auto store = [&](int part, int u, const uint4& y, bool on) {
    uint32_t scale;
    uint4 stored;
    const uint32_t code = quantise8(y, scale, stored);
    if (on && k.state == 3) store4<D>(dest4<D>(a, part, u / kChunks, u % kChunks), k, t, code, scale, stored);
  };
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
    turn(p.src[0] + k.in[0] + (long long)h * p.in[0].head, p.dst[0] + k.out[0] + (long long)h * p.out[0].head);
  if (k.state != 3) return;
  for (int h0 = 0; h0 < p.Hk; h0 += kAppendHeads) {
    const int n = min(kAppendHeads, p.Hk - h0);
    if (h0 > 0) __syncthreads();
    for (int h = tid / kGroups; h < n; h += lanes / kGroups)
      turn(p.src[1] + k.in[1] + (long long)(h0 + h) * p.in[1].head, rows[h]);
    __syncthreads();
    for (int w = tid & ~31; w < n * kChunks; w += lanes) {
      const int u = w + (tid & 31);
      const bool on = u < n * kChunks;
      store(0, h0 * kChunks + u,
            on ? *reinterpret_cast<const uint4*>(&rows[u / kChunks][(u % kChunks) * 8]) : make_uint4(0, 0, 0, 0), on);
    }
  }
  for (int w = tid & ~31; w < units; w += lanes) {
    const int u = w + (tid & 31);
    const bool on = u < units;
    if (w >= lanes && on) load(u);
    store(1, u, x, on);
  }
}

// Threads and tokens per CTA as in launch_rope: one token each, with all threads, while they fit one wave. Beyond that
// several, so that a thread has four loads on their way while the places are looked up (8500 tokens: 18 us, 28 with divisions and one token
// of 128 threads).
cudaError_t launch_append4(const RopeLaunch& p, const Append4& a, int d, int num_sms, cudaStream_t st) {
  const bool one_wave = p.tokens <= 6LL * num_sms;
  const unsigned T = (unsigned)p.tokens;
  if (p.rot > 0) {
    if (d == 128) fa_paged_append4_rope_kernel<128><<<T, one_wave ? 256 : 128, 0, st>>>(p, a);
    else fa_paged_append4_rope_kernel<64><<<T, one_wave ? 256 : 128, 0, st>>>(p, a);
  } else if (one_wave) {
    if (d == 128) fa_paged_append4_kernel<128, 1><<<T, 256, 0, st>>>(p, a);
    else fa_paged_append4_kernel<64, 1><<<T, 256, 0, st>>>(p, a);
  } else {
    if (d == 128) fa_paged_append4_kernel<128, 4><<<(T + 3) / 4, 256, 0, st>>>(p, a);
    else fa_paged_append4_kernel<64, 4><<<(T + 3) / 4, 256, 0, st>>>(p, a);
  }
  return cudaGetLastError();
}

}  // namespace fa
