// Shared by the attention kernels: arguments, which positions a row sees, and
// E2M1 pairs as bf16.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kq_cache.cuh"
#include "kq_internal.h"

namespace kq {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNaN = __builtin_nanf("");

struct AttnArgs {
  CacheView view;
  const uint8_t *kc, *ks, *vc, *vs;
  const uint16_t* q;
  uint16_t* out;
  float* lse;                      // [batch][heads][M], or null
  const int32_t* lens;
  int64_t qb, qm, qh, ob, om, oh;  // strides in elements
  int32_t M, D, max_len;
  int32_t rows;                    // query rows of one K/V head: group * M
  int32_t causal;
  FastDiv group;                   // query heads per K/V head
  float scale_log2;                // scale * log2(e)
  int32_t chunk, n_chunks;         // positions per CTA, CTAs along the positions
  // Decoded tiles of 128 positions (the tensor-core kernel): which positions of
  // [batch][tile] there are, and [batch][K/V head][tile] images of K and V.
  const uint4* tile_mask;
  const uint8_t* images;
  int32_t tiles, d16;              // tiles of max_len; D rounded up to 16
  float* part_o;                   // [batch][K/V head][chunk][row][Dp]
  float2* part_ml;                 // (maximum, sum) of the same
  int* err;
};

// Row r of a K/V head is query m = r / group of head group * hk + r % group.
__device__ __forceinline__ int seq_len(const AttnArgs& a, int64_t b) {
  return max(0, min(a.lens[b], a.max_len));
}
// Positions row r sees: [0, row_limit).
__device__ __forceinline__ int row_limit(const AttnArgs& a, int len, int r) {
  if (r >= a.rows) return 0;
  return a.causal ? max(0, len - a.M + static_cast<int>(a.group.div(r)) + 1) : len;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Four pairs of codes out of a word: pair i is nibble i of the low half and
// nibble i of the high half, as bf16 bits.  A code's sign goes to bit 15 and
// its exponent and mantissa (two bits and one) to bits 8..6, the low end of
// bf16's fields, where they mean the code's value times 2^-126: the exponent
// 0 of E2M1 is bf16's own subnormal.  mx_mul puts the factor right together
// with the block's scale.  One product copies a nibble to both places (2^6 and
// 2^12 above the lowest nibble; nothing carries into the other half), on the
// multipliers, which are free; as shifts, all of it was work for the
// logic pipe that bounds the single-token kernel (15 instead of 9 a word).
__device__ __forceinline__ void e2m1_pairs(uint32_t w, uint32_t (&p)[4]) {
  constexpr uint32_t kOut = 0x81C081C0u;
  const uint32_t u = w >> 8;
  p[0] = ((w & 0x000F000Fu) * 0x1040u) & kOut;
  p[1] = ((w & 0x00F000F0u) * 0x0104u) & kOut;
  p[2] = ((u & 0x000F000Fu) * 0x1040u) & kOut;
  p[3] = ((u & 0x00F000F0u) * 0x0104u) & kOut;
}

// bf16 bits of 2^(s - 63) for scale byte s <= 190: a raw code times it is the
// value times 2^-62 (2^-126 of the raw bits, 2^(s - 127) of the scale), exactly from
// s = 57 on, where the smallest code becomes bf16's smallest number, 2^-133; below, the
// value is off by up to 2^-72, which is half that step times 2^62, and from s = 52 on
// down nothing is left of it.  The 2^62 keeps the multiplier in bf16's range for
// every scale byte up to 190 (values below 2^66).  It is undone in the scores' scale, and in the
// softmax weights, which are held as 2^62 exp2(.): their products with V then
// have V's own range, so small weights are not lost to underflow.
__device__ __forceinline__ uint32_t mx_mul(uint32_t s) { return (s + 64) << 7; }
constexpr int kShift = 62;
constexpr float kUnscale = 4611686018427387904.0f;      // 2^kShift

// Out of a row's maximum and sum of weights: the factor that makes its accumulator
// the output, and its log-sum-exp.  A sum of 0 is a row that sees nothing, a NaN one
// that is not a number; the maximum, which drops NaN, is -inf in both.
__device__ __forceinline__ float unscale(float sum) { return sum == 0.0f ? 0.0f : kUnscale / sum; }
__device__ __forceinline__ float row_lse(float top, float sum) {
  return sum == 0.0f ? -INFINITY : (top + (log2f(sum) - kShift)) * kLn2;
}

// How a call is cut: from its sizes alone, so that the workspace query and the
// call agree.
struct AttnPlan {
  bool tensor_core;
  int row_groups, nt;              // few rows: groups of 8 nt rows
  int64_t chunk, n_chunks, tiles;
  size_t ml_bytes, part_bytes, mask_bytes, image_bytes, bytes;
};

// Many query rows: decodes the cache into the workspace, then multiplies on
// the tensor cores (kq_attention_tc.cu).
int launch_attention_tc(const AttnArgs& a, const AttnPlan& p, int64_t batch, int dev, cudaStream_t st);

}  // namespace kq
