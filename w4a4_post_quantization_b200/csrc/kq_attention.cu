// Attention of bf16 queries over the MXFP4 K/V cache:
//
//   S = scale q K^T over the positions p < len[b] (causal: and
//       p <= len[b] - M + m for query m of M),   O = softmax(S) V.
//
// The positions are walked once with the running maximum and sum of the
// softmax, all of them float32; a row that sees no position has O = 0 and a
// log-sum-exp of -inf.
//
// A query with a NaN or an infinity has no finite score (the cache holds finite
// values), and maxima drop NaN: its maximum can be -inf, as that of a row that sees
// nothing.  The sum tells them apart: it is NaN where a score is NaN or +inf, and 0
// where nothing is seen; one whose scores are all -inf is made NaN (row_sees).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "kq_attention.cuh"

namespace kq {
namespace {

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kN>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kN) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------------------
// Few query rows: one warp walks 32 positions at a time with mma.sync, its
// operands decoded in registers.  The products are taken transposed,
//   S^T = K q^T  [positions][rows]   and   O^T = V^T P^T  [channels][rows],
// so that the cache fills the MMA's 16 and the few query rows its 8: the usual
// single-token group of up to 8 heads costs half the MMAs, exponentials and
// accumulators of the other way round.  What is left is the decoding of the
// codes, 13 instructions for 8 of them, and that bounds the kernel.
//
// Lane (g, c) = (lane / 4, lane mod 4).  The products contract over the head's
// channels (S) and the positions (O) in any order, as long as both operands
// use the same one, so each lane takes what is contiguous for it:
//   K  for positions tau(g) and tau(g) + 8 of 16, lane c's quarter of the row, one
//      4-byte word being the channels of two MMA k-steps,
//   V  for positions c, c + 4, c + 8, c + 12, the g-th eighth of the row,
// with tau(2 c) = c, tau(2 c + 1) = c + 4, which keeps both free of bank conflicts.
// P comes out of the first product with positions along g and goes into the second
// with positions along c: an 8 x 8 transpose, movmatrix.
constexpr int kWarps = 4;
constexpr int kTile = 32;                     // positions a warp holds at a time
constexpr int kStages = 3;

template <int kW>                             // 32-channel blocks of a row
struct SplitGeom {
  static constexpr int kDp = 32 * kW;
  static constexpr int kCodes = kTile * kDp / 2;
  static constexpr int kScales = kTile * kW;
  static constexpr int kStage = 2 * kCodes + 2 * kScales;
  static constexpr int kRing = kWarps * kStages * kStage;
};
// The ring; in the end the warps' parts.
template <int kW, int kNT>
constexpr int split_smem() {
  const int merge = kWarps * 8 * kNT * (32 * kW + 2) * 4;
  return merge > SplitGeom<kW>::kRing ? merge : SplitGeom<kW>::kRing;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Whether there is a page for any position of [begin, end).  Asked only of a row
// whose sum is 0.
__device__ __forceinline__ bool row_sees(const AttnArgs& a, int64_t b, int begin, int end) {
  for (int64_t pos = begin; pos < end; pos += int64_t(1) << a.view.page_shift)
    if (cache_row(a.view, b, pos, 0) >= 0) return true;
  return end > begin && cache_row(a.view, b, end - 1, 0) >= 0;
}

// kNT: groups of 8 query rows.  Four with heads of 128 take all 255 registers and spill 268
// bytes a thread.
template <int kW, int kNT>
__global__ void __launch_bounds__(32 * kWarps, kNT == 1 ? 4 : kNT == 2 ? 3 : 2)
    attn_split_kernel(const AttnArgs a) {
  using G = SplitGeom<kW>;
  constexpr int kRows = 8 * kNT;
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int tau = (g >> 1) + 4 * (g & 1);
  const int chunk = blockIdx.x % a.n_chunks, r0 = blockIdx.x / a.n_chunks * kRows;
  const int hk = blockIdx.y;
  const int64_t b = blockIdx.z;
  pdl_wait_then_trigger();

  const int begin = chunk * a.chunk;
  // This warp's tile i: positions begin + 32 (warp + 4 i).
  auto tile_pos = [&](int i) { return begin + kTile * (warp + kWarps * i); };
  // The table's entry for half (lane mod 2) of tile i + lane / 2.
  auto table_entry = [&](int i) {
    const int at = (tile_pos(i + (lane >> 1)) + 16 * (lane & 1)) >> a.view.page_shift;
    return at < a.view.table_pages ? __ldg(a.view.table + b * a.view.table_pages + at) : -1;
  };
  // The first 16 tiles' beside the length, not after it.
  int entry = table_entry(0);
  const int len = seq_len(a, b);
  const int first_limit = row_limit(a, len, r0);                       // the fewest a row sees
  const int last_limit = row_limit(a, len, min(r0 + kRows, a.rows) - 1);
  const int end = min(begin + a.chunk, last_limit);
  int limit[kNT][2];
#pragma unroll
  for (int t = 0; t < kNT; ++t) {
    limit[t][0] = row_limit(a, len, r0 + 8 * t + 2 * c);
    limit[t][1] = row_limit(a, len, r0 + 8 * t + 2 * c + 1);
  }

  const int n_tiles = end > begin + kTile * warp
                          ? (end - begin - kTile * warp + kTile * kWarps - 1) / (kTile * kWarps) : 0;
  uint8_t* ring = smem + warp * (kStages * G::kStage);
  // Pages of 16 tiles at a time, lane 2 i + half holding half `half` of tile
  // i: the table is read once, ahead of the loads that need it.  -1: nothing
  // to load there.
  int page = -1;
  auto load_pages = [&](int i) {
    const int pos = tile_pos(i + (lane >> 1)) + 16 * (lane & 1);
    if (i > 0) entry = table_entry(i);
    page = -1;
    if (i + (lane >> 1) < n_tiles && pos < end) {
      if (entry >= 0 && entry < a.view.pages) page = entry;
      else atomicOr(a.err, kErrCacheIndex);
    }
  };
  uint32_t absent = 0;                        // bit 2 (i mod kStages) + half: that half has no page
  auto load_tile = [&](int i) {
    if (i < n_tiles) {
      if ((i & 15) == 0) load_pages(i);
      uint8_t* st = ring + (i % kStages) * G::kStage;
      const int pos = tile_pos(i);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int p = __shfl_sync(0xFFFFFFFFu, page, 2 * (i & 15) + half);
        const uint32_t bit = 1u << (2 * (i % kStages) + half);
        absent = p < 0 ? absent | bit : absent & ~bit;
        if (p >= 0) {
          const int64_t row = ((static_cast<int64_t>(p) * a.view.heads + hk) << a.view.page_shift) +
                              ((pos + 16 * half) & ((1 << a.view.page_shift) - 1));
          const uint8_t* kc = a.kc + row * (G::kDp / 2);
          const uint8_t* vc = a.vc + row * (G::kDp / 2);
          uint8_t* dk = st + half * (G::kCodes / 2);
#pragma unroll
          for (int j = 0; j < (G::kCodes / 2 + 511) / 512; ++j) {
            const int off = 16 * lane + 512 * j;
            if (off < G::kCodes / 2) {
              cp_async16(dk + off, kc + off);
              cp_async16(dk + G::kCodes + off, vc + off);
            }
          }
          if (lane < 2 * kW) {
            const bool v = lane >= kW;
            const int off = 16 * (v ? lane - kW : lane);
            cp_async16(st + 2 * G::kCodes + v * G::kScales + half * (G::kScales / 2) + off,
                       (v ? a.vs : a.ks) + row * kW + off);
          }
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) load_tile(i);

  // Query row 8 t + g as B fragments, in the channel order of the K words.
  uint32_t q[kNT][2 * kW][2];
#pragma unroll
  for (int t = 0; t < kNT; ++t) {
    const int r = r0 + 8 * t + g;
    const int m = a.group.div(r), h = hk * a.group.d + r - m * a.group.d;
#pragma unroll
    for (int j = 0; j < kW; ++j) {
      const int d0 = (c * kW + j) * 8;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (r < a.rows && d0 < a.D)
        x = __ldg(reinterpret_cast<const uint4*>(a.q + b * a.qb + m * a.qm + h * a.qh + d0));
      q[t][2 * j][0] = __byte_perm(x.x, x.z, 0x5410);
      q[t][2 * j][1] = __byte_perm(x.x, x.z, 0x7632);
      q[t][2 * j + 1][0] = __byte_perm(x.y, x.w, 0x5410);
      q[t][2 * j + 1][1] = __byte_perm(x.y, x.w, 0x7632);
    }
  }

  // O^T: MMA tile n holds channels 4 kW g + 2 n (rows g) and the next (rows g + 8).
  float o[kNT][2 * kW][4], mx[kNT][2], l[kNT][2];
#pragma unroll
  for (int t = 0; t < kNT; ++t) {
#pragma unroll
    for (int n = 0; n < 2 * kW; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[t][n][k] = 0.0f;
    mx[t][0] = mx[t][1] = -INFINITY;
    l[t][0] = l[t][1] = 0.0f;
  }

  for (int i = 0; i < n_tiles; ++i) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    const uint32_t gone = (absent >> (2 * (i % kStages))) & 3u;
    load_tile(i + kStages - 1);               // into the stage read in the last step
    const uint8_t* st = ring + (i % kStages) * G::kStage;
    const uint8_t* ksc = st + 2 * G::kCodes;
    const uint8_t* vsc = ksc + G::kScales;
    const int pos = tile_pos(i);

    // S^T of 2 x 16 positions.
    float s[2][kNT][4];
    {
      uint32_t w[4][kW], m2[4][kW];           // positions tau + 8 u
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int tok = 8 * u + tau;
        const uint32_t* kw = reinterpret_cast<const uint32_t*>(st + tok * (G::kDp / 2)) + c * kW;
        if constexpr (kW == 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(kw);
          w[u][0] = x.x, w[u][1] = x.y, w[u][2] = x.z, w[u][3] = x.w;
        } else if constexpr (kW == 2) {
          const uint2 x = *reinterpret_cast<const uint2*>(kw);
          w[u][0] = x.x, w[u][1] = x.y;
        } else {
#pragma unroll
          for (int j = 0; j < kW; ++j) w[u][j] = kw[j];
        }
#pragma unroll
        for (int j = 0; j < kW; ++j) m2[u][j] = mx_mul(ksc[tok * kW + ((c * kW + j) >> 2)]) * 0x10001u;
      }
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int t = 0; t < kNT; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[half][t][k] = 0.0f;
#pragma unroll
      for (int j = 0; j < kW; ++j)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t p[2][4];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            e2m1_pairs(w[2 * half + u][j], p[u]);
#pragma unroll
            for (int k = 0; k < 4; ++k) p[u][k] = mul_bf16x2(p[u][k], m2[2 * half + u][j]);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t x[4] = {p[0][2 * e], p[1][2 * e], p[0][2 * e + 1], p[1][2 * e + 1]};
#pragma unroll
            for (int t = 0; t < kNT; ++t) mma_bf16(s[half][t], x, q[t][2 * j + e][0], q[t][2 * j + e][1]);
          }
        }
    }

    // Running maximum and sum of rows 8 t + 2 c and the next; element k is position
    // tau + 8 (k / 2) of its 16, row 2 c + k mod 2.
    const bool ragged = pos + kTile > first_limit || gone;
    uint32_t pb[2][kNT][2];
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
      const float sc = a.scale_log2 * kUnscale;
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float v = s[half][t][k] * sc;
          if (ragged) {
            const int p = pos + 16 * half + tau + 8 * (k >> 1);
            if (p >= limit[t][k & 1] || (gone >> half & 1)) v = -INFINITY;
          }
          s[half][t][k] = v;
          top[k & 1] = fmaxf(top[k & 1], v);
        }
      bool grew = false;
      float base[2], alpha[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], x));
        const float m_new = fmaxf(mx[t][e], top[e]);
        // A row that has seen nothing yet: exp2(-inf - 0) = 0.
        base[e] = m_new == -INFINITY ? 0.0f : m_new;
        alpha[e] = ex2(mx[t][e] - base[e]);
        base[e] -= kShift;
        grew |= m_new > mx[t][e];
        mx[t][e] = m_new;
      }
      if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
        for (int n = 0; n < 2 * kW; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[t][n][k] *= alpha[k & 1];
        l[t][0] *= alpha[0];
        l[t][1] *= alpha[1];
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          s[half][t][k] = ex2(s[half][t][k] - base[k & 1]);
          l[t][k & 1] += s[half][t][k];
        }
        // The weights are rounded to bf16, the type of the product (each by at
        // most 2^-8 of itself); their sum is taken before.
        pb[half][t][0] = transpose8x8(bf16x2(s[half][t][0], s[half][t][1]));
        pb[half][t][1] = transpose8x8(bf16x2(s[half][t][2], s[half][t][3]));
      }
    }

    // O^T += V^T P^T.
    const bool tail = pos + kTile > len || gone;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t hw[4][(kW + 1) / 2];           // two 4-channel units a word
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint8_t* vp = st + G::kCodes + (16 * half + c + 4 * k) * (G::kDp / 2) + g * 2 * kW;
        if constexpr (kW == 4) {
          const uint2 x = *reinterpret_cast<const uint2*>(vp);
          hw[k][0] = x.x, hw[k][1] = x.y;
        } else if constexpr (kW == 2) {
          hw[k][0] = *reinterpret_cast<const uint32_t*>(vp);
        } else {
          const uint16_t* vh = reinterpret_cast<const uint16_t*>(vp);
          hw[k][0] = vh[0];
          if constexpr (kW == 3) {
            hw[k][0] |= static_cast<uint32_t>(vh[1]) << 16;
            hw[k][1] = vh[2];
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kW; ++u) {
        uint32_t m[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = mx_mul(vsc[(16 * half + c + 4 * k) * kW + ((g * kW + u) >> 3)]);
        // What lies behind the sequence is unknown: its codes times zero.
        if (tail)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (pos + 16 * half + c + 4 * k >= len || (gone >> half & 1)) m[k] = 0;
        const uint32_t m01 = m[0] | m[1] << 16, m23 = m[2] | m[3] << 16;
        const uint32_t sel = u & 1 ? 0x7632 : 0x5410;
        uint32_t x[4], y[4];
        e2m1_pairs(__byte_perm(hw[0][u >> 1], hw[1][u >> 1], sel), x);
        e2m1_pairs(__byte_perm(hw[2][u >> 1], hw[3][u >> 1], sel), y);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[k] = mul_bf16x2(x[k], m01);
          y[k] = mul_bf16x2(y[k], m23);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t va[4] = {x[2 * k], x[2 * k + 1], y[2 * k], y[2 * k + 1]};
#pragma unroll
          for (int t = 0; t < kNT; ++t) mma_bf16(o[t][2 * u + k], va, pb[half][t][0], pb[half][t][1]);
        }
      }
    }
    __syncwarp();
  }
  cp_async_wait<0>();

  // The four warps' parts, joined in a fixed order.
#pragma unroll
  for (int t = 0; t < kNT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[t][e] += __shfl_xor_sync(0xFFFFFFFFu, l[t][e], x);
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem);                    // [warp][row][Dp]
  float2* sml = reinterpret_cast<float2*>(so + kWarps * kRows * G::kDp);
#pragma unroll
  for (int t = 0; t < kNT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * t + 2 * c + e;
      float* dst = so + (warp * kRows + r) * G::kDp + g * 4 * kW;
#pragma unroll
      for (int n = 0; n < 2 * kW; n += 2)
        *reinterpret_cast<float4*>(dst + 2 * n) =
            make_float4(o[t][n][e], o[t][n][2 + e], o[t][n + 1][e], o[t][n + 1][2 + e]);
      if (g == 0) sml[warp * kRows + r] = make_float2(mx[t][e], l[t][e]);
    }
  __syncthreads();
  for (int i = tid; i < kRows * (G::kDp / 4); i += 32 * kWarps) {
    const int r = i / (G::kDp / 4), d = 4 * (i - r * (G::kDp / 4));
    if (r0 + r >= a.rows) break;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sml[w * kRows + r].x);
    const float base = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = sml[w * kRows + r];
      const float k = ex2(ml.x - base);
      const float4 x = *reinterpret_cast<const float4*>(so + (w * kRows + r) * G::kDp + d);
      sum += k * ml.y;
      acc.x += k * x.x, acc.y += k * x.y, acc.z += k * x.z, acc.w += k * x.w;
    }
    if (sum == 0.0f && row_sees(a, b, begin, min(end, row_limit(a, len, r0 + r)))) sum = kNaN;
    if (a.n_chunks > 1) {
      const int64_t at = ((b * a.view.heads + hk) * a.n_chunks + chunk) * a.rows + r0 + r;
      if (sum != 0.0f) *reinterpret_cast<float4*>(a.part_o + at * G::kDp + d) = acc;
      if (d == 0) a.part_ml[at] = make_float2(top, sum);
      continue;
    }
    const int m = a.group.div(r0 + r), h = hk * a.group.d + r0 + r - m * a.group.d;
    const float inv = unscale(sum);
    if (d < a.D)
      *reinterpret_cast<uint2*>(a.out + b * a.ob + m * a.om + h * a.oh + d) =
          make_uint2(bf16x2(acc.x * inv, acc.y * inv), bf16x2(acc.z * inv, acc.w * inv));
    if (a.lse && d == 0) a.lse[(b * a.view.heads * a.group.d + h) * a.M + m] = row_lse(top, sum);
  }
}

// Joins the chunks of each row, in their order: a warp per row and 32 channels.
template <int kW>
__global__ void __launch_bounds__(128) attn_join_kernel(const AttnArgs a, int64_t n_rows) {
  pdl_wait_then_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t at = item / kW;
  const int j = static_cast<int>(item - at * kW);
  if (at >= n_rows) return;
  const int64_t bh = at / a.rows;
  const int r = static_cast<int>(at - bh * a.rows);
  const int64_t b = bh / a.view.heads;
  const int hk = static_cast<int>(bh - b * a.view.heads);
  const int n = (row_limit(a, seq_len(a, b), r) + a.chunk - 1) / a.chunk;
  const float2* ml = a.part_ml + bh * a.n_chunks * a.rows + r;
  const float* po = a.part_o + (bh * a.n_chunks * a.rows + r) * (32 * kW) + 32 * j + lane;
  const int64_t step = static_cast<int64_t>(a.rows) * (32 * kW);
  // The first chunks' O is on its way while the weights are worked out; O of a
  // chunk in which the row sees nothing has not been written, and is not used (its
  // sum is 0; a NaN sum makes the whole row NaN).
  constexpr int kAhead = 8;
  float x[kAhead];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) x[i] = i0 + i < n ? po[(i0 + i) * step] : 0.0f;
  };
  fetch(0);
  float top = -INFINITY;
  for (int i = lane; i < n; i += 32) top = fmaxf(top, ml[static_cast<int64_t>(i) * a.rows].x);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, k));
  const float base = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f, acc = 0.0f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    // This lane's chunk of the 32: its weight.
    float2 y = make_float2(-INFINITY, 0.0f);
    if (i0 + lane < n) y = ml[static_cast<int64_t>(i0 + lane) * a.rows];
    const float k = ex2(y.x - base);
    float part = k * y.y;
#pragma unroll
    for (int e = 16; e > 0; e >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, e);
    sum += part;
    for (int i1 = i0; i1 < min(i0 + 32, n); i1 += kAhead) {
      float z[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) z[i] = x[i];
      fetch(i1 + kAhead);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float w = __shfl_sync(0xFFFFFFFFu, k, i1 - i0 + i);
        if (w > 0.0f) acc += w * z[i];
      }
    }
  }
  const int m = a.group.div(r), h = hk * a.group.d + r - m * a.group.d;
  const float inv = unscale(sum);
  if (32 * j + lane < a.D)
    a.out[b * a.ob + m * a.om + h * a.oh + 32 * j + lane] = __bfloat16_as_ushort(__float2bfloat16_rn(acc * inv));
  if (a.lse && j == 0 && lane == 0)
    a.lse[(b * a.view.heads * a.group.d + h) * a.M + m] = row_lse(top, sum);
}

AttnPlan make_plan(int64_t batch, int64_t kv_heads, int64_t rows, int64_t max_len, int64_t head_dim) {
  AttnPlan p{};
  constexpr int64_t kSms = 148;
  const int64_t nb = (head_dim + 31) / 32, d16 = (head_dim + 15) / 16 * 16;
  p.tiles = (max_len + 127) / 128;
  const int64_t images = batch * kv_heads * p.tiles * 512 * d16;
  // Up to 64 rows the split kernel's passes over the codes (one for 32 rows) cost
  // less than decoding the cache to memory: 8 x 8 heads of 128 over 16384
  // positions, 64 rows 242 against 291 us, 96 rows 345 against 297.  Past 4 GiB of
  // decoded tiles it serves any number of rows, 33 x 2048 queries of 32 / 8 heads over
  // 512 positions of a table for 32768 in 4.4 ms (0.73 with max_len = 512).
  p.tensor_core = rows > 64 && images <= (int64_t(1) << 32) && kv_heads < 32768;
  if (p.tensor_core) {
    // Cut along the positions where there are too few tiles of rows, into parts of at
    // least four tiles.
    const int64_t units = batch * kv_heads * ((rows + 127) / 128);
    const int64_t want = std::max<int64_t>(1, std::min(2 * kSms / units, (p.tiles + 3) / 4));
    p.chunk = (p.tiles + want - 1) / want * 128;
    p.mask_bytes = static_cast<size_t>((batch * p.tiles * 16 + 255) / 256 * 256);
    p.image_bytes = static_cast<size_t>(images);
  } else {
    p.nt = rows > 16 ? 4 : rows > 8 ? 2 : 1;
    p.row_groups = static_cast<int>((rows + 8 * p.nt - 1) / (8 * p.nt));
    constexpr int64_t kStep = kTile * kWarps;
    // About twelve CTAs for each SM, of at least 512 positions (8 x 8 heads, 18 to
    // 33 thousand positions: six 96 us, eight 87, twelve 85, twenty-four 90; with the
    // tests for rows that are no numbers twelve takes 87).
    const int64_t units = batch * kv_heads * p.row_groups;
    const int64_t want = std::max<int64_t>(1, 12 * kSms / units);
    const int64_t chunk = std::max<int64_t>(512, (max_len + want - 1) / want);
    p.chunk = (chunk + kStep - 1) / kStep * kStep;
  }
  p.n_chunks = std::max<int64_t>(1, (max_len + p.chunk - 1) / p.chunk);
  if (p.n_chunks > 1) {
    const int64_t parts = batch * kv_heads * p.n_chunks * rows;
    p.ml_bytes = static_cast<size_t>((parts * 8 + 255) / 256 * 256);
    p.part_bytes = static_cast<size_t>(parts) * nb * 32 * 4;
    p.part_bytes = (p.part_bytes + 255) / 256 * 256;
  }
  p.bytes = p.ml_bytes + p.part_bytes + p.mask_bytes + p.image_bytes;
  return p;
}

template <int kW, int kNT>
int launch_split(const AttnArgs& a, const AttnPlan& p, int64_t batch, int dev, cudaStream_t st) {
  if (p.n_chunks * p.row_groups >= (int64_t(1) << 31)) return KQ_ERR_INVALID;
  constexpr int smem = split_smem<kW, kNT>();
  const int rc = allow_smem<attn_split_kernel<kW, kNT>>(smem, dev);
  if (rc != KQ_OK) return rc;
  const dim3 grid(static_cast<unsigned>(p.n_chunks * p.row_groups),
                  static_cast<unsigned>(a.view.heads), static_cast<unsigned>(batch));
  cudaError_t e = launch_pdl(attn_split_kernel<kW, kNT>, grid, dim3(32 * kWarps), smem, st, a);
  if (e != cudaSuccess) return record_cuda_error(e);
  return KQ_OK;
}

template <int kW>
int launch(const AttnArgs& a, const AttnPlan& p, int64_t batch, int dev, cudaStream_t st) {
  const int rc = p.tensor_core ? launch_attention_tc(a, p, batch, dev, st)
                 : p.nt == 1   ? launch_split<kW, 1>(a, p, batch, dev, st)
                 : p.nt == 2   ? launch_split<kW, 2>(a, p, batch, dev, st)
                               : launch_split<kW, 4>(a, p, batch, dev, st);
  if (rc != KQ_OK || p.n_chunks == 1) return rc;
  const int64_t n_rows = batch * a.view.heads * a.rows;
  const cudaError_t e = launch_pdl(attn_join_kernel<kW>, dim3(static_cast<unsigned>((n_rows * kW + 3) / 4)),
                                   dim3(128), 0, st, a, n_rows);
  return e == cudaSuccess ? KQ_OK : record_cuda_error(e);
}

// Sizes a call can have: 0 where they are not valid, else the rows of a K/V
// head.
int64_t attention_rows(int64_t batch, int64_t M, int64_t heads, int64_t kv_heads, int64_t head_dim,
                       int64_t max_len) {
  if (batch < 1 || batch > 65535 || M < 1 || heads < 1 || kv_heads < 1 || kv_heads > 65535 ||
      heads % kv_heads != 0 || head_dim < 8 || head_dim > 128 || head_dim % 8 != 0 || max_len < 1 ||
      max_len > (int64_t(1) << 30))
    return 0;
  if (M > (int64_t(1) << 30) || heads > (int64_t(1) << 30)) return 0;
  const int64_t rows = M * (heads / kv_heads);
  return rows <= (int64_t(1) << 30) && batch * kv_heads <= (int64_t(1) << 30) / rows ? rows : 0;
}

}  // namespace
}  // namespace kq

using namespace kq;

extern "C" size_t kq_attention_workspace_bytes(int64_t batch, int64_t M, int64_t heads,
                                               int64_t kv_heads, int64_t head_dim, int64_t max_len) {
  const int64_t rows = attention_rows(batch, M, heads, kv_heads, head_dim, max_len);
  if (rows == 0) return 0;
  return make_plan(batch, kv_heads, rows, max_len, head_dim).bytes;
}

extern "C" int kq_attention_mxfp4(const uint16_t* q, int64_t q_sb, int64_t q_sm, int64_t q_sh,
                                  int64_t batch, int64_t M, int64_t heads, const kq_cache* cache,
                                  const int32_t* block_table, int64_t table_pages,
                                  const int32_t* lens, int64_t max_len, float scale, int causal,
                                  uint16_t* out, int64_t o_sb, int64_t o_sm, int64_t o_sh,
                                  float* lse, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  if (batch < 0 || M < 0) return KQ_ERR_INVALID;
  if (batch == 0 || M == 0) return KQ_OK;
  AttnArgs a{};
  if (!cache_view(cache, block_table, batch, table_pages, &a.view)) return KQ_ERR_INVALID;
  const int64_t rows = attention_rows(batch, M, heads, cache->heads, cache->head_dim, max_len);
  if (rows == 0 || max_len > table_pages * cache->page_size) return KQ_ERR_INVALID;
  auto al = [](const void* p, uintptr_t n) { return p && reinterpret_cast<uintptr_t>(p) % n == 0; };
  auto strides = [](int64_t x, int64_t y, int64_t z) {
    return x >= 0 && y >= 0 && z >= 0 && x % 8 == 0 && y % 8 == 0 && z % 8 == 0;
  };
  if (!al(q, 16) || !al(out, 16) || !al(lens, 4) || !strides(q_sb, q_sm, q_sh) ||
      !strides(o_sb, o_sm, o_sh) || (lse && !al(lse, 4)))
    return KQ_ERR_INVALID;
  // The kernels multiply the scores by 2^62 times this.
  const float scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  if (!std::isfinite(scale_log2 * kUnscale)) return KQ_ERR_INVALID;
  const AttnPlan p = make_plan(batch, cache->heads, rows, max_len, cache->head_dim);
  if (p.bytes > 0 && (!al(workspace, 256) || workspace_bytes < p.bytes)) return KQ_ERR_INVALID;
  const DeviceInfo* di = nullptr;
  int dev = 0;
  int rc = device_info(&di, &dev);
  if (rc != KQ_OK) return rc;
  rc = device_error_word(dev, &a.err);
  if (rc != KQ_OK) return rc;
  a.kc = cache->k_codes, a.ks = cache->k_scales, a.vc = cache->v_codes, a.vs = cache->v_scales;
  a.q = q, a.qb = q_sb, a.qm = q_sm, a.qh = q_sh;
  a.out = out, a.ob = o_sb, a.om = o_sm, a.oh = o_sh;
  a.lse = lse;
  a.lens = lens;
  a.M = static_cast<int32_t>(M);
  a.D = static_cast<int32_t>(cache->head_dim);
  a.max_len = static_cast<int32_t>(max_len);
  a.rows = static_cast<int32_t>(rows);
  a.causal = causal != 0;
  a.group = FastDiv(static_cast<uint32_t>(heads / cache->heads));
  a.scale_log2 = scale_log2;
  a.chunk = static_cast<int32_t>(p.chunk);
  a.n_chunks = static_cast<int32_t>(p.n_chunks);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(ws);
  a.part_o = reinterpret_cast<float*>(ws + p.ml_bytes);
  a.tile_mask = reinterpret_cast<const uint4*>(ws + p.ml_bytes + p.part_bytes);
  a.images = ws + p.ml_bytes + p.part_bytes + p.mask_bytes;
  a.tiles = static_cast<int32_t>(p.tiles);
  a.d16 = static_cast<int32_t>((cache->head_dim + 15) / 16 * 16);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (a.view.nb) {
    case 1: return launch<1>(a, p, batch, dev, st);
    case 2: return launch<2>(a, p, batch, dev, st);
    case 3: return launch<3>(a, p, batch, dev, st);
    default: return launch<4>(a, p, batch, dev, st);
  }
}
