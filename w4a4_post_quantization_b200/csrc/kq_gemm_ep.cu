// The W4A4 product with its epilogue:
//
//   C[m][n] = residual[m][n] + gate[m / tokens][n] * act((A B^T)[m][n] + bias[n])
//
// A transformer layer's product is followed by these four; as passes of their
// own over C they would move its bytes several times.  Here they are applied to
// the float32 accumulator on its way out of tensor memory, with one rounding
// at the end.
//
// CTA pairs (kq_gemm.cuh) walk 256 x kN tiles.  Warp 0 loads, warp 1 of the even
// CTA issues the MMAs, warps 2..9 are the epilogue: two warps for each quarter
// of the 128 accumulator rows, each taking half of the columns.  A thread holds
// one row's kN / 2 columns in registers, so the accumulator is handed back as
// soon as it has been read and the next tile's MMAs run under the activation.
// The output, and the residual before it, pass through 4 KB boxes of 32 rows x
// 128 bytes in shared memory, private to a warp: the residual's loads are under
// way while the tile is still being multiplied, and nothing waits for a store
// within a tile of bf16.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kq.h"
#include "kq_device.cuh"
#include "kq_gemm.cuh"
#include "kq_internal.h"
#include "kq_tc.cuh"

namespace kq {
namespace {

constexpr int kEpWarps = 8;
constexpr int kEpThreads = 32 * (2 + kEpWarps);
constexpr int kBoxRows = 32;
constexpr int kBoxBytes = kBoxRows * 128;
constexpr int kSlots = 2;                     // boxes per warp
constexpr int kEpStaging = kEpWarps * kSlots * kBoxBytes;

template <int kN>
struct EpGeom {
  static constexpr int kStages = kN == 256 ? 4 : 6;
  using P = PairGeom<kN, kStages>;
  static constexpr int kCols = kN / 2;        // columns per thread
  static constexpr int kSmem = 1024 + kStages * P::kStage + kEpStaging +
                               (2 * kStages + 2 * P::kAcc + kEpWarps) * 8 + 16;
  static_assert(kSmem <= 232448, "shared memory");
};

struct EpArgs {
  PairTiles tiles;
  int32_t M, N;
  int32_t tokens;                             // rows of one gate vector
  int32_t boxes;                              // the output and residual rows take TMA boxes
  const uint16_t* bias;
  const uint16_t* gate;
  const void* residual;
  void* out;
  int* err;
};

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x0 / (1 + 2^t0), x1 / (1 + 2^t1) with one reciprocal: 1 / a = b (1 / ab).
// t is capped at 60, so the product stays finite; past it the quotients are
// 2^-60 of x and less (the special-function pipe, not the FMAs, bounds the
// activations, and this takes a quarter of its work away).
__device__ __forceinline__ void over_one_plus_exp2(float& x0, float& x1, float t0, float t1) {
  const float a = 1.0f + ex2_approx(fminf(t0, 60.0f));
  const float b = 1.0f + ex2_approx(fminf(t1, 60.0f));
  const float r = rcp_approx(a * b);
  x0 *= r * b;
  x1 *= r * a;
}

// Two values through the activation.
template <int kAct>
__device__ __forceinline__ void activate(float& x0, float& x1) {
  if constexpr (kAct == KQ_ACT_GELU_TANH) {
    // 0.5 x (1 + tanh u) = x / (1 + exp(-2 u)), u = sqrt(2 / pi) (x + 0.044715 x^3):
    // no difference of near-equal numbers for negative x.
    constexpr float k1 = -2.302208198f;       // -2 sqrt(2 / pi) log2(e)
    constexpr float k3 = -0.1029432408f;      // 0.044715 k1
    over_one_plus_exp2(x0, x1, x0 * fmaf(k3, x0 * x0, k1), x1 * fmaf(k3, x1 * x1, k1));
  } else if constexpr (kAct == KQ_ACT_SILU) {
    constexpr float k = -1.4426950409f;       // -log2(e)
    over_one_plus_exp2(x0, x1, k * x0, k * x1);
  } else if constexpr (kAct == KQ_ACT_GELU) {
    // x Phi(x) with Abramowitz and Stegun 7.1.26:
    //   erfc(z) = t (a1 + t (a2 + ... + a5 t^3)) exp(-z^2) + e, t = 1 / (1 + p z),
    //   |e| <= 1.5e-7 for z >= 0.
    float* x[2] = {&x0, &x1};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float v = *x[i], z = fabsf(v) * 0.7071067812f;
      const float t = rcp_approx(fmaf(0.3275911f, z, 1.0f));
      float s = fmaf(1.061405429f, t, -1.453152027f);
      s = fmaf(s, t, 1.421413741f);
      s = fmaf(s, t, -0.284496736f);
      s = fmaf(s, t, 0.254829592f);
      const float q = 0.5f * s * t * ex2_approx(z * z * -1.4426950409f);   // Phi(-|v|)
      *x[i] = v * (v < 0.0f ? q : 1.0f - q);
    }
  }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float bf16_at(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
}

// 32 columns of a row, from column `col`: bias, activation, gate.  kVec: N is
// a multiple of 8, so a group of 8 columns is inside or outside as one and
// starts on 16 bytes.
template <int kAct, bool kVec>
__device__ __forceinline__ void finish(uint32_t (&x)[32], const EpArgs& a, int col,
                                       const uint16_t* gate) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float v[8], k[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(x[8 * c + i]);
    const int c0 = col + 8 * c;
    auto row = [&](const uint16_t* p) {
      if constexpr (kVec) {
        const uint4 w = c0 < a.N ? __ldg(reinterpret_cast<const uint4*>(p + c0)) : make_uint4(0, 0, 0, 0);
        k[0] = bf16_lo(w.x), k[1] = bf16_hi(w.x), k[2] = bf16_lo(w.y), k[3] = bf16_hi(w.y);
        k[4] = bf16_lo(w.z), k[5] = bf16_hi(w.z), k[6] = bf16_lo(w.w), k[7] = bf16_hi(w.w);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) k[i] = c0 + i < a.N ? bf16_at(p + c0 + i) : 0.0f;
      }
    };
    if (a.bias) {
      row(a.bias);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += k[i];
    }
#pragma unroll
    for (int i = 0; i < 8; i += 2) activate<kAct>(v[i], v[i + 1]);
    if (gate) {
      row(gate);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= k[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[8 * c + i] = __float_as_uint(v[i]);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

template <int kN, bool kBf16, int kAct>
__global__ void __launch_bounds__(kEpThreads, 1)
    gemm_mxf4_ep(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                 const __grid_constant__ CUtensorMap sfamap, const __grid_constant__ CUtensorMap sfbmap,
                 const __grid_constant__ CUtensorMap cmap, const __grid_constant__ CUtensorMap rmap,
                 const EpArgs a) {
  using E = EpGeom<kN>;
  using P = typename E::P;
  constexpr int kStages = E::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint8_t* staging = base + kStages * P::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kEpStaging);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + P::kAcc;
  uint64_t* res_full = acc_empty + P::kAcc;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(res_full + kEpWarps);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  const int n_tiles_total = a.tiles.m_tiles * a.tiles.n_tiles;

  if (tid == 0) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(&full[st], 1);                       // rank 0's producer, plus the pair's bytes
      mbar_init(&empty[st], 1);                      // rank 0's commit, multicast
    }
    for (int b = 0; b < P::kAcc; ++b) {
      mbar_init(&acc_full[b], 1);                    // rank 0's commit, multicast
      mbar_init(&acc_empty[b], 2 * kEpWarps);        // the epilogue warps of each CTA
    }
    for (int w = 0; w < kEpWarps; ++w) mbar_init(&res_full[w], 1);
    fence_mbar_init_cluster();
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, kTmemCols);
  tmem_fence_before();
  cluster_sync();                                    // barriers of both CTAs initialised
  tmem_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait_then_trigger();

  if (warp == 0) {
    if (elect_one() && !pair_produce<kN, kStages>(base, full, empty, &amap, &bmap, &sfamap, &sfbmap,
                                                a.tiles, rank, pair, n_pairs))
      atomicOr(a.err, kErrProducerWait);
  } else if (warp == 1) {
    const uint32_t tm = __reduce_max_sync(0xFFFFFFFFu, tmem_base);       // uniform
    if (rank == 0 && elect_one() &&
        !pair_mma<kN, kStages>(base, full, empty, acc_full, acc_empty, tm, a.tiles, pair, n_pairs))
      atomicOr(a.err, kErrConsumerWait);
  } else {
    constexpr int kGroups = E::kCols / 32;           // 32-column groups of a thread
    constexpr int kBoxCols = kBf16 ? 64 : 32;
    constexpr int kBoxes = E::kCols / kBoxCols;      // boxes of a warp and tile
    constexpr int kRound = kBoxes < kSlots ? kBoxes : kSlots;
    const int quarter = warp & 3, side = (warp - 2) >> 2;
    const uint32_t taddr = tmem_base + (uint32_t(quarter * 32) << 16) + side * E::kCols;
    uint8_t* slots = staging + (warp - 2) * (kSlots * kBoxBytes);
    uint64_t* rbar = &res_full[warp - 2];
    uint32_t rphase = 0;
    int i = 0;
    for (int t = pair; t < n_tiles_total; t += n_pairs, ++i) {
      int m0, n0;
      pair_tile_origin<kN>(a.tiles, t, m0, n0);
      const int row0 = m0 + (int)rank * kBM + quarter * 32, col0 = n0 + side * E::kCols;
      const bool live = row0 < a.M && col0 < a.N;    // some of this warp's box is inside
      // Boxes of round r: their slots are free once the stores out of them
      // have been read; the residual goes in first.
      auto begin_round = [&](int r) {
        if (lane == 0) {
          bulk_wait_read_0();
          if (a.residual) {
            int n = 0;
#pragma unroll
            for (int k = 0; k < kRound; ++k) n += col0 + (r * kRound + k) * kBoxCols < a.N;
            mbar_arrive_expect_tx(rbar, n * kBoxBytes);
            for (int k = 0; k < n; ++k)
              tma_load_2d(slots + k * kBoxBytes, &rmap, col0 + (r * kRound + k) * kBoxCols, row0, rbar);
          }
        }
        __syncwarp();
      };
      if (live && a.boxes) begin_round(0);
      const int b = i % P::kAcc;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&acc_full[b], (i / P::kAcc) & 1))) {
        if (lane == 0) {
          atomicOr(a.err, kErrConsumerWait);
          // The residual's copies are in flight: let them land.
          if (live && a.boxes && a.residual) mbar_wait(rbar, rphase);
        }
        break;
      }
      tmem_fence_after();
      uint32_t x[kGroups][32];
#pragma unroll
      for (int v = 0; v < kGroups; ++v) tmem_ld32(taddr + b * kN + 32 * v, x[v]);
      tmem_wait_ld();
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(&acc_empty[b], 0));
      if (!live) continue;
      const uint16_t* gate =
          a.gate ? a.gate + static_cast<int64_t>(min(row0 + lane, a.M - 1) / a.tokens) * a.N : nullptr;

      if (a.boxes) {
#pragma unroll
        for (int r = 0; r < kBoxes / kRound; ++r) {
          if (r > 0) begin_round(r);
#pragma unroll
          for (int v = r * kRound * kBoxCols / 32; v < (r + 1) * kRound * kBoxCols / 32; ++v)
            finish<kAct, true>(x[v], a, col0 + 32 * v, gate);
          if (a.residual) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(rbar, rphase))) {
              if (lane == 0) atomicOr(a.err, kErrConsumerWait);
            }
            rphase ^= 1;
          }
#pragma unroll
          for (int k = 0; k < kRound; ++k) {
            // Row r's 16-byte chunk c of a box is at c ^ (r mod 8).
            uint8_t* srow = slots + k * kBoxBytes + lane * 128;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              uint4* at = reinterpret_cast<uint4*>(srow + 16 * (c ^ (lane & 7)));
              uint4 w = make_uint4(0, 0, 0, 0);
              if (a.residual) w = *at;
              if constexpr (kBf16) {
                const int v = (r * kRound + k) * 2 + (c >> 2), e = 8 * (c & 3);
                const uint32_t rw[4] = {w.x, w.y, w.z, w.w};
                uint32_t ow[4];
#pragma unroll
                for (int h = 0; h < 4; ++h)
                  ow[h] = pack_bf16(__uint_as_float(x[v][e + 2 * h]) + bf16_lo(rw[h]),
                                    __uint_as_float(x[v][e + 2 * h + 1]) + bf16_hi(rw[h]));
                *at = make_uint4(ow[0], ow[1], ow[2], ow[3]);
              } else {
                const int v = r * kRound + k, e = 4 * c;
                *reinterpret_cast<float4*>(at) =
                    make_float4(__uint_as_float(x[v][e]) + __uint_as_float(w.x),
                                __uint_as_float(x[v][e + 1]) + __uint_as_float(w.y),
                                __uint_as_float(x[v][e + 2]) + __uint_as_float(w.z),
                                __uint_as_float(x[v][e + 3]) + __uint_as_float(w.w));
              }
            }
          }
          fence_proxy_async_smem();                  // generic stores -> TMA store reads
          __syncwarp();
          if (lane == 0) {
#pragma unroll
            for (int k = 0; k < kRound; ++k)
              if (col0 + (r * kRound + k) * kBoxCols < a.N)
                tma_store_2d(&cmap, slots + k * kBoxBytes, col0 + (r * kRound + k) * kBoxCols, row0);
            bulk_commit();
          }
        }
      } else {
        // Rows whose pitch or width TMA cannot take: 32 columns at a time
        // through a box of 32 x 32 floats, so that a warp's global accesses run
        // along a row.
        float* box = reinterpret_cast<float*>(slots);
#pragma unroll
        for (int v = 0; v < kGroups; ++v) {
          const int col = col0 + 32 * v;
          finish<kAct, false>(x[v], a, col, gate);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<uint4*>(box + lane * 32 + 4 * (c ^ (lane & 7))) =
                make_uint4(x[v][4 * c], x[v][4 * c + 1], x[v][4 * c + 2], x[v][4 * c + 3]);
          __syncwarp();
          if (col + lane < a.N) {
            const int n_rows = min(32, a.M - row0);
            const int64_t at0 = static_cast<int64_t>(row0) * a.N + col + lane;
#pragma unroll 8
            for (int r = 0; r < n_rows; ++r) {
              float y = box[r * 32 + 4 * ((lane >> 2) ^ (r & 7)) + (lane & 3)];
              const int64_t at = at0 + static_cast<int64_t>(r) * a.N;
              if constexpr (kBf16) {
                if (a.residual) y += bf16_at(static_cast<const uint16_t*>(a.residual) + at);
                static_cast<uint16_t*>(a.out)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
              } else {
                if (a.residual) y += static_cast<const float*>(a.residual)[at];
                static_cast<float*>(a.out)[at] = y;
              }
            }
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    tmem_fence_before();
  }
  // Neither CTA leaves, nor frees its TMEM, before the other has made all its
  // arrivals on its barriers and the MMAs on its memory have completed: every
  // wait above is bounded, so both CTAs get here.
  __syncwarp();
  cluster_sync();
  if (warp == 1) {
    tmem_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// Row-major output or residual as boxes of 32 rows x 128 bytes, 128-byte swizzle.
bool encode_rows_map(CUtensorMap* map, const void* p, int64_t M, int64_t N, bool bf16) {
  const int esize = bf16 ? 2 : 4;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(N) * esize};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / esize), kBoxRows};
  const cuuint32_t estr[2] = {1, 1};
  return tensor_map_encoder()(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                              2, const_cast<void*>(p), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_NONE,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct EpCall {
  const uint8_t *qa, *sa, *qb, *sb;
  int64_t M, N, K;
  bool bf16;
  const DeviceInfo* di;
  int dev;
  cudaStream_t st;
};

template <int kN, bool kBf16, int kAct>
int launch_ep(const EpCall& c, EpArgs a) {
  using E = EpGeom<kN>;
  using P = typename E::P;
  a.tiles.K = static_cast<int32_t>(c.K);
  a.tiles.k_tiles = static_cast<int32_t>((c.K + kBK - 1) / kBK);
  a.tiles.m_tiles = static_cast<int32_t>((c.M + kPairM - 1) / kPairM);
  a.tiles.n_tiles = static_cast<int32_t>((c.N + kN - 1) / kN);
  const int64_t sf_cols = (c.K / 32 + 3) / 4;
  CUtensorMap amap, bmap, sfamap, sfbmap, cmap, rmap;
  if (!encode_codes_map(&amap, c.qa, c.M, c.K, kBM) || !encode_codes_map(&bmap, c.qb, c.N, c.K, P::kBRows) ||
      !encode_scales_map(&sfamap, c.sa, (c.M + 127) / 128, sf_cols, 1) ||
      !encode_scales_map(&sfbmap, c.sb, (c.N + 127) / 128, sf_cols, P::kGroups))
    return record_cuda_error(cudaErrorInvalidValue);
  cmap = rmap = amap;
  if (a.boxes && (!encode_rows_map(&cmap, a.out, c.M, c.N, kBf16) ||
                  (a.residual && !encode_rows_map(&rmap, a.residual, c.M, c.N, kBf16))))
    return record_cuda_error(cudaErrorInvalidValue);
  const int rc = allow_smem<gemm_mxf4_ep<kN, kBf16, kAct>>(E::kSmem, c.dev);
  if (rc != KQ_OK) return rc;
  return launch_pairs<gemm_mxf4_ep<kN, kBf16, kAct>>(
      kEpThreads, E::kSmem, (int64_t)a.tiles.m_tiles * a.tiles.n_tiles, c.di, c.dev, true, c.st, amap,
      bmap, sfamap, sfbmap, cmap, rmap, a);
}

template <int kN, bool kBf16>
int launch_ep_act(const EpCall& c, const EpArgs& a, int act) {
  switch (act) {
    case KQ_ACT_NONE: return launch_ep<kN, kBf16, KQ_ACT_NONE>(c, a);
    case KQ_ACT_GELU_TANH: return launch_ep<kN, kBf16, KQ_ACT_GELU_TANH>(c, a);
    case KQ_ACT_GELU: return launch_ep<kN, kBf16, KQ_ACT_GELU>(c, a);
    default: return launch_ep<kN, kBf16, KQ_ACT_SILU>(c, a);
  }
}

// Tile width: what fills the pairs in fewer column-steps.  Tiles of 128 columns
// quantize the work more finely and hide the accumulator's drain behind a
// second accumulator, but bring 1.5 times the operand bytes per product.
bool wide_tiles(int64_t M, int64_t N, int pairs) {
  const int64_t mt = (M + kPairM - 1) / kPairM;
  const int64_t wide = (mt * ((N + 255) / 256) + pairs - 1) / pairs * 2;
  const int64_t narrow = (mt * ((N + 127) / 128) + pairs - 1) / pairs;
  return 5 * narrow >= 4 * wide;
}

}  // namespace
}  // namespace kq

using namespace kq;

extern "C" int kq_gemm_mxfp4_epilogue(const uint8_t* qa, const uint8_t* sa_tiled, const uint8_t* qb,
                                      const uint8_t* sb_tiled, int64_t M, int64_t N, int64_t K,
                                      const uint16_t* bias, int activation, const uint16_t* gate,
                                      int64_t tokens_per_sample, const void* residual, void* c,
                                      int c_dtype, void* stream) {
  if (M < 0 || N < 0 || K < 32 || K % 32 != 0) return KQ_ERR_INVALID;
  if (c_dtype != KQ_OUT_F32 && c_dtype != KQ_OUT_BF16) return KQ_ERR_INVALID;
  if (activation < KQ_ACT_NONE || activation > KQ_ACT_SILU) return KQ_ERR_INVALID;
  if (gate && tokens_per_sample < 1) return KQ_ERR_INVALID;
  if (M == 0 || N == 0) return KQ_OK;
  constexpr int64_t kMost = (int64_t(1) << 31) - 2 * kBK;
  if (M > kMost || N > kMost || K > kMost) return KQ_ERR_INVALID;
  if (((M + kPairM - 1) / kPairM) * ((N + 127) / 128) > (int64_t(1) << 31) - 65536) return KQ_ERR_INVALID;
  auto al = [](const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  if (!qa || !sa_tiled || !qb || !sb_tiled || !c) return KQ_ERR_INVALID;
  if (!al(qa, 16) || !al(qb, 16) || !al(sa_tiled, 16) || !al(sb_tiled, 16) || !al(c, 16) ||
      !al(bias, 16) || !al(gate, 16) || !al(residual, 16))
    return KQ_ERR_INVALID;
  EpCall call{qa, sa_tiled, qb, sb_tiled, M, N, K, c_dtype == KQ_OUT_BF16, nullptr, 0,
              static_cast<cudaStream_t>(stream)};
  int rc = device_info(&call.di, &call.dev);
  if (rc != KQ_OK) return rc;
  EpArgs a{};
  rc = device_error_word(call.dev, &a.err);
  if (rc != KQ_OK) return rc;
  a.M = static_cast<int32_t>(M);
  a.N = static_cast<int32_t>(N);
  a.tokens = static_cast<int32_t>(std::min<int64_t>(gate ? tokens_per_sample : 1, M));
  a.boxes = N % 8 == 0;
  a.bias = bias;
  a.gate = gate;
  a.residual = residual;
  a.out = c;
  const bool wide = wide_tiles(M, N, call.di->sms / 2);
  if (call.bf16)
    return wide ? launch_ep_act<256, true>(call, a, activation) : launch_ep_act<128, true>(call, a, activation);
  return wide ? launch_ep_act<256, false>(call, a, activation) : launch_ep_act<128, false>(call, a, activation);
}
