// fa_paged4.cuh -- a paged cache in 4 bits: its layout, and how codes become bf16 operands.
//
// A group of 32 dims of a key or value has a scale s and a code u in 1..15 per dim, and stands for (u - 8) s. s is a bf16
// number of four significant bits, so (u - 8) s has at most seven, and bf16 holds it exactly: operands made from codes lose
// nothing, and attention over them is attention over the cache's values. Two values come from one packed multiply-add,
//     (128 + u) s + (-136 s):
// 128 + u is the code beside the bits of 128, 136 s = 17 * 8 s has at most eight significant bits, so both are bf16 numbers,
// and the sum is rounded once, to a number that bf16 has. (A scale of eight bits would halve the scales' bytes, 6 % of a
// row, at two more instructions per scale in kernels whose time follows theirs; one of bf16's own eight significant
// bits would round each value.)
//
// The 32-bit word i of a group holds dims 8 i .. 8 i + 7, dim 8 i + 2 j + e in the bits from 4 j + 16 e on, so that one shift
// and one mask bring out a pair of neighbouring dims as a packed pair.
#pragma once

#include "fa_paged.cuh"

namespace fa {

constexpr int kGroup4 = 32;                            // dims that share a scale
constexpr uint32_t kScaleBig = 0x7b80, kScaleTiny = 0x0d80;  // bf16 bits of 2^120 and 2^-100: groups from the one on hold
                                                       // NaN (136 s must be finite), below the other zeros

__host__ __device__ constexpr int code_bytes(int D) { return D / 2; }               // of a slot
__host__ __device__ constexpr int scale_bytes(int D) { return D / kGroup4 * 2; }

struct PagedCache4 {
  const uint8_t *k, *v, *k_scale, *v_scale;  // slots of a page and head are dense
  long long k_page, k_head, v_page, v_head;  // strides in bytes
  long long ks_page, ks_head, vs_page, vs_head;
};

// Codes 2 j and 2 j + 1 of a word as 128 + u, packed.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int j) { return ((w >> (4 * j)) & 0x000f000fu) | 0x43004300u; }
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t scale_shift(uint32_t s2) {  // -136 s of a pair of scales
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(s2), "r"(0xc308c308u));
  return d;
}

struct Append4 {
  PagedCache4 c;
  __nv_bfloat16* out[2];  // the values that k and v are stored as, or NULL
  long long out_tok[2], out_head[2];
};

cudaError_t launch_append4(const RopeLaunch& p, const Append4& a, int d, int num_sms, cudaStream_t st);

// The small tiles' kernel over a 4-bit cache: tiles of 8 columns (queries), by the most rows that a tile of the batch can have;
// warps that compute (one more makes them a multiple of four, as they are allotted), and CTAs per SM: what registers leave
// room for.
__host__ __device__ constexpr int row4_columns(int row_tile, int max_q, int G) {
  return row_tile == 32 ? 4 : ((long long)max_q * G <= 8 ? 1 : 2);
}
__host__ __device__ constexpr int row4_warps(int columns, int d) { return columns * d <= 128 ? 7 : 3; }
__host__ __device__ constexpr int row4_ctas(int columns, int d) { return columns == 2 && d == 128 ? 3 : 2; }
// Their workspace: two partial results per CTA, then RowShares.
size_t paged4_rows_part_bytes(int d, int row_tile, int columns);
size_t paged4_rows_workspace_bytes(int d, int row_tile, int columns);
cudaError_t launch_paged4_rows(PagedFwd& p, const PagedCache4& c, int d, int num_sms, cudaStream_t st);
cudaError_t launch_paged4_tiles(const TileMaps& m, const PagedFwd& p, const PagedCache4& c, int d, int num_sms,
                                cudaStream_t st);

}  // namespace fa
