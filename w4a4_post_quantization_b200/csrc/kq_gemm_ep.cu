// The W4A4 product with its epilogue:
//
//   C[m][n] = residual[m][n] + gate[m / tokens][n] * act((A B^T)[m][n] + bias[n])
//
// A transformer layer's product is followed by these four; as passes of their
// own over C they would move its bytes several times.  Here they are applied to
// the float32 accumulator on its way out of tensor memory, with one rounding
// at the end.
//
// CTA pairs (kq_gemm.cuh) walk 256 x kN tiles.  kN / 16 warps are the epilogue:
// kN / 64 for each quarter of the 128 accumulator rows, a thread holding 64
// columns of one row in registers, so the accumulator is handed back as soon as it
// has been read and the next tile's MMAs run under the activation.  (With 128
// columns a thread, and half the warps, the activation's chain of dependent
// instructions was what the kernel waited for: GELU took 8000 cycles a tile.)  One
// further warp loads, and one of the even CTA issues the MMAs.  The output, and
// the residual before it, pass through 4 KB boxes of 32 rows x 128 bytes in shared
// memory, private to a warp: the residual's loads are under way while the tile
// is still being multiplied.
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

constexpr int kCols = 64;                     // columns per epilogue thread
constexpr int kBoxRows = 32;
constexpr int kBoxBytes = kBoxRows * 128;
constexpr int kEpStaging = 65536;             // the epilogue warps' boxes

// Registers a thread: wide tiles have 20 warps, launched with 96, of which the
// epilogue's take 104 and the others keep 64.  Some spill: 4 and 16 bytes with GELU and
// tanh-GELU, and the narrow bf16 tiles, with 168, 8 to 124 bytes.
constexpr int kEpRegs = 104, kRestRegs = 64;

template <int kN>
struct EpGeom {
  static constexpr int kStages = kN == 256 ? 4 : 6;
  using P = PairGeom<kN, kStages>;
  static constexpr int kWarps = kN / 16;      // epilogue warps
  static constexpr int kThreads = 32 * (kWarps + 4);
  static constexpr int kSlots = kEpStaging / kBoxBytes / kWarps;   // boxes per warp
  static constexpr bool kSplit = kN == 256;   // registers shared out as above
  static constexpr int kVectors = kWarps * 2 * kCols * 4;   // bias and gate of each warp's columns
  static constexpr int kSmem = 1024 + kStages * P::kStage + kEpStaging + kVectors +
                               (2 * kStages + 2 * P::kAcc + kWarps) * 8 + 16;
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

// The larger of x and lo; NaN stays NaN.  Where an activation has come down to 2^-57 its
// argument is held: x / (1 + 2^t) with t capped would be 2^-63 of x, however large that
// is.  (0.7 of 34 us at 8192 x 4608 x 1152 with tanh-GELU; a reciprocal of its own for
// either half, which needs no cap, 1.7.)
__device__ __forceinline__ float max_nan(float x, float lo) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(lo));
  return y;
}
__device__ __forceinline__ f2 not_below(f2 x, float lo) {
  float a, b;
  unpack2(x, a, b);
  return pack2(max_nan(a, lo), max_nan(b, lo));
}

// x / (1 + 2^t) for both halves, t up to 63, with one reciprocal: 1 / a = b (1 / ab), the
// product finite (the special-function unit bounds the activations, and this takes a
// quarter of its work away; the polynomial exponential of the attention, for every
// second pair, cost more issue slots than it freed: 38 against 34 us for 8192 x
// 4608 x 1152 with GELU).
__device__ __forceinline__ f2 over_one_plus_exp2(f2 x, f2 t) {
  float t0, t1, a, b;
  unpack2(t, t0, t1);
  // A NaN does not reach the other half.
  a = ex2(fminf(t0, 63.0f));
  b = ex2(fminf(t1, 63.0f));
  unpack2(add2(pack2(a, b), pack2(1.0f, 1.0f)), a, b);
  const float r = rcp_approx(a * b);
  return mul2(x, mul2(pack2(r, r), pack2(b, a)));
}

// Two values through the activation.
template <int kAct>
__device__ __forceinline__ f2 activate(f2 x) {
  if constexpr (kAct == KQ_ACT_GELU_TANH) {
    // 0.5 x (1 + tanh u) = x / (1 + exp(-2 u)), u = sqrt(2 / pi) (x + 0.044715 x^3):
    // no difference of near-equal numbers for negative x.
    constexpr float k1 = -2.302208198f;       // -2 sqrt(2 / pi) log2(e)
    constexpr float k3 = -0.1029432408f;      // 0.044715 k1
    x = not_below(x, -7.6f);
    return over_one_plus_exp2(x, mul2(x, fma2(pack2(k3, k3), mul2(x, x), pack2(k1, k1))));
  } else if constexpr (kAct == KQ_ACT_SILU) {
    constexpr float k = -1.4426950409f;       // -log2(e)
    x = not_below(x, -43.5f);
    return over_one_plus_exp2(x, mul2(x, pack2(k, k)));
  } else if constexpr (kAct == KQ_ACT_GELU) {
    // x Phi(x) with Abramowitz and Stegun 7.1.26:
    //   erfc(z) = t (a1 + t (a2 + ... + a5 t^3)) exp(-z^2) + e, t = 1 / (1 + p z),
    //   |e| <= 1.5e-7 for z >= 0; the two reciprocals as above.
    auto both = [](float k) { return pack2(k, k); };
    float v0, v1, a, b, z0, z1;
    unpack2(x, v0, v1);
    const f2 z = mul2(pack2(fabsf(v0), fabsf(v1)), both(0.7071067812f));
    unpack2(fma2(z, both(0.3275911f), both(1.0f)), a, b);
    // 1 + p z is capped so that the product of the two stays finite; Phi is 0 there.
    a = fminf(a, 1e18f);
    b = fminf(b, 1e18f);
    const float r = rcp_approx(a * b);
    const f2 t = mul2(both(r), pack2(b, a));
    f2 s = fma2(t, both(1.061405429f), both(-1.453152027f));
    s = fma2(s, t, both(1.421413741f));
    s = fma2(s, t, both(-0.284496736f));
    s = fma2(s, t, both(0.254829592f));
    unpack2(mul2(mul2(z, z), both(-1.4426950409f)), z0, z1);
    // Phi(-|v|)
    const f2 q = mul2(mul2(s, t), mul2(both(0.5f), pack2(ex2(z0), ex2(z1))));
    float q0, q1;
    unpack2(q, q0, q1);
    return mul2(x, pack2(v0 < 0.0f ? q0 : 1.0f - q0, v1 < 0.0f ? q1 : 1.0f - q1));
  }
  return x;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float bf16_at(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
}

// 32 columns of a row: bias, activation, gate.  The two vectors come as float32
// from shared memory (`bias`, `gate`: these columns of the warp's copy), the same
// address in every lane; a row whose sample differs within the warp has its gate
// in `own_gate` (column `col` of it; columns from N on are not read).
template <int kAct>
__device__ __forceinline__ void finish(uint32_t (&x)[32], const float* bias, const float* gate,
                                       const uint16_t* own_gate, int col, int N) {
  // One branch a part, not one a column: they cost as much as the arithmetic.
  auto each = [&](const float* k, auto op) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float4 w = reinterpret_cast<const float4*>(k)[c];
      float y[4];
      unpack2(op(pack2(__uint_as_float(x[4 * c]), __uint_as_float(x[4 * c + 1])), pack2(w.x, w.y)), y[0], y[1]);
      unpack2(op(pack2(__uint_as_float(x[4 * c + 2]), __uint_as_float(x[4 * c + 3])), pack2(w.z, w.w)), y[2], y[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * c + i] = __float_as_uint(y[i]);
    }
  };
  if (bias) each(bias, [](f2 a, f2 b) { return add2(a, b); });
  if constexpr (kAct != KQ_ACT_NONE) {
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      float a, b;
      unpack2(activate<kAct>(pack2(__uint_as_float(x[c]), __uint_as_float(x[c + 1]))), a, b);
      x[c] = __float_as_uint(a);
      x[c + 1] = __float_as_uint(b);
    }
  }
  if (gate) each(gate, [](f2 a, f2 b) { return mul2(a, b); });
  if (own_gate) {
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (col + c < N) x[c] = __float_as_uint(__uint_as_float(x[c]) * bf16_at(own_gate + col + c));
  }
}

template <int kN, bool kBf16, int kAct>
__global__ void __launch_bounds__(EpGeom<kN>::kThreads, 1)
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
  float* vectors = reinterpret_cast<float*>(staging + kEpStaging);
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kEpStaging + E::kVectors);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + P::kAcc;
  uint64_t* res_full = acc_empty + P::kAcc;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(res_full + E::kWarps);
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
      mbar_init(&acc_empty[b], 2 * E::kWarps);       // the epilogue warps of each CTA
    }
    for (int w = 0; w < E::kWarps; ++w) mbar_init(&res_full[w], 1);
    fence_mbar_init_cluster();
  }
  if (warp == E::kWarps + 1) tmem_alloc_pair(tmem_slot, kTmemCols);
  tmem_fence_before();
  cluster_sync();                                    // barriers of both CTAs initialised
  tmem_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait_then_trigger();

  if (warp >= E::kWarps) {
    if constexpr (E::kSplit) regs_down<kRestRegs>();
    const uint32_t tm = __reduce_max_sync(0xFFFFFFFFu, tmem_base);       // uniform
    if (warp == E::kWarps) {
      if (elect_one() && !pair_produce<kN, kStages>(base, full, empty, &amap, &bmap, &sfamap, &sfbmap,
                                                    a.tiles, rank, pair, n_pairs))
        atomicOr(a.err, kErrProducerWait);
    } else if (warp == E::kWarps + 1) {
      if (rank == 0 && elect_one() &&
          !pair_mma<kN, kStages>(base, full, empty, acc_full, acc_empty, tm, a.tiles, pair, n_pairs))
        atomicOr(a.err, kErrConsumerWait);
    }
  } else {
    if constexpr (E::kSplit) regs_up<kEpRegs>();
    constexpr int kGroups = kCols / 32;           // 32-column groups of a thread
    constexpr int kBoxCols = kBf16 ? 64 : 32;
    constexpr int kBoxes = kCols / kBoxCols;      // boxes of a warp and tile
    constexpr int kRound = kBoxes < E::kSlots ? kBoxes : E::kSlots;
    const int quarter = warp & 3, side = warp >> 2;
    const uint32_t taddr = tmem_base + (uint32_t(quarter * 32) << 16) + side * kCols;
    uint8_t* slots = staging + warp * (E::kSlots * kBoxBytes);
    uint64_t* rbar = &res_full[warp];
    float* vec = vectors + warp * (2 * kCols);
    uint32_t rphase = 0;
    // Bias and gate of a tile's columns, a column in each lane, as float bits.  The
    // rows of a warp mostly belong to one sample.
    constexpr int kPer = kCols / 32;
    uint32_t nb[kPer], ng[kPer];
    bool n_one = true;
    auto load_vectors = [&](int tile) {
      if (tile >= n_tiles_total) return;
      int m0, n0;
      pair_tile_origin<kN>(a.tiles, tile, m0, n0);
      const int row0 = min(m0 + (int)rank * kBM + quarter * 32, a.M - 1), col = n0 + side * kCols + lane;
      const int sample = a.gate ? row0 / a.tokens : 0;
      n_one = !a.gate || min(row0 + 31, a.M - 1) / a.tokens == sample;
      const uint16_t* gate = a.gate ? a.gate + static_cast<int64_t>(sample) * a.N : nullptr;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const bool in = col + 32 * k < a.N;
        nb[k] = a.bias && in ? static_cast<uint32_t>(__ldg(a.bias + col + 32 * k)) << 16 : 0u;
        ng[k] = gate && in ? static_cast<uint32_t>(__ldg(gate + col + 32 * k)) << 16 : 0u;
      }
    };
    load_vectors(pair);
    int i = 0;
    for (int t = pair; t < n_tiles_total; t += n_pairs, ++i) {
      int m0, n0;
      pair_tile_origin<kN>(a.tiles, t, m0, n0);
      const int row0 = m0 + (int)rank * kBM + quarter * 32, col0 = n0 + side * kCols;
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
      if (live) {
        // This tile's bias and gate, loaded under the last one's arithmetic.
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          vec[lane + 32 * k] = __uint_as_float(nb[k]);
          vec[kCols + lane + 32 * k] = __uint_as_float(ng[k]);
        }
        __syncwarp();
      }
      const bool one_sample = n_one;
      const int b = i % P::kAcc;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&acc_full[b], (i / P::kAcc) & 1, a.tiles.polls))) {
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
      if (lane == 0) mbar_arrive_cluster_relaxed(cluster_addr(&acc_empty[b], 0));
      load_vectors(t + n_pairs);
      if (!live) continue;
      const float* bias = a.bias ? vec : nullptr;
      const float* gate = a.gate && one_sample ? vec + kCols : nullptr;
      const uint16_t* own_gate =
          a.gate && !one_sample ? a.gate + static_cast<int64_t>(min(row0 + lane, a.M - 1) / a.tokens) * a.N : nullptr;
      auto act = [&](uint32_t (&y)[32], int v) {
        finish<kAct>(y, bias ? bias + 32 * v : nullptr, gate ? gate + 32 * v : nullptr, own_gate,
                     col0 + 32 * v, a.N);
      };

      if (a.boxes) {
#pragma unroll
        for (int r = 0; r < kBoxes / kRound; ++r) {
          if (r > 0) begin_round(r);
#pragma unroll
          for (int v = r * kRound * kBoxCols / 32; v < (r + 1) * kRound * kBoxCols / 32; ++v)
            act(x[v], v);
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
                  ow[h] = bf16x2(__uint_as_float(x[v][e + 2 * h]) + bf16_lo(rw[h]),
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
      } else if constexpr (kN == 128) {
        // Rows whose pitch or width TMA cannot take (narrow tiles only): 32 columns
        // at a time through a box of 32 x 32 floats, so that a warp's global
        // accesses run along a row, the residual's all in flight at once and under
        // the arithmetic.
        float* box = reinterpret_cast<float*>(slots);
        const int n_rows = min(32, a.M - row0);
#pragma unroll
        for (int v = 0; v < kGroups; ++v) {
          const int col = col0 + 32 * v + lane;
          const int64_t at0 = static_cast<int64_t>(row0) * a.N + col;
          const bool in = col < a.N;
          float res[32];
          if (a.residual) {
#pragma unroll
            for (int r = 0; r < 32; ++r) {
              const int64_t at = at0 + static_cast<int64_t>(r) * a.N;
              res[r] = 0.0f;
              if (in && r < n_rows) {
                if constexpr (kBf16) res[r] = bf16_at(static_cast<const uint16_t*>(a.residual) + at);
                else res[r] = __ldcs(static_cast<const float*>(a.residual) + at);
              }
            }
          }
          act(x[v], v);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<uint4*>(box + lane * 32 + 4 * (c ^ (lane & 7))) =
                make_uint4(x[v][4 * c], x[v][4 * c + 1], x[v][4 * c + 2], x[v][4 * c + 3]);
          __syncwarp();
#pragma unroll
          for (int r = 0; r < 32; ++r) {
            float y = box[r * 32 + 4 * ((lane >> 2) ^ (r & 7)) + (lane & 3)];
            if (a.residual) y += res[r];
            const int64_t at = at0 + static_cast<int64_t>(r) * a.N;
            if (in && r < n_rows) {
              if constexpr (kBf16) static_cast<uint16_t*>(a.out)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
              else static_cast<float*>(a.out)[at] = y;
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
  if (warp == E::kWarps + 1) {
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
  a.tiles.polls = product_polls(a.tiles.k_tiles);
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
  if constexpr (E::kSplit) {
    // setmaxnreg draws on what the block was launched with: were that less than
    // the warps' shares, the kernel would wait for good.
    static const int regs = launched_regs(gemm_mxf4_ep<kN, kBf16, kAct>);
    if (regs * (E::kWarps + 4) < kEpRegs * E::kWarps + kRestRegs * 4)
      return record_cuda_error(cudaErrorLaunchOutOfResources);
  }
  return launch_pairs<gemm_mxf4_ep<kN, kBf16, kAct>>(
      E::kThreads, E::kSmem, (int64_t)a.tiles.m_tiles * a.tiles.n_tiles, c.di, c.dev, true, c.st, amap,
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
// second accumulator, but bring 1.5 times the operand bytes per product.  Only
// bf16 rows that take TMA boxes have wide tiles: a thread's half of a wide float32
// row, or the residual of one that is read along its rows, does not fit beside the
// 128 accumulator registers.
bool wide_tiles(const EpArgs& a, bool bf16, int pairs) {
  if (!bf16 || !a.boxes) return false;
  const int64_t mt = (a.M + kPairM - 1) / kPairM;
  const int64_t wide = (mt * ((a.N + 255) / 256) + pairs - 1) / pairs * 2;
  const int64_t narrow = (mt * ((a.N + 127) / 128) + pairs - 1) / pairs;
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
  // The epilogue's wait for a whole product along K lasts with its stages; 2^21 is the
  // longest that has been run with every pair at work.
  if (M > kMost || N > kMost || K > (int64_t(1) << 21)) return KQ_ERR_INVALID;
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
  if (wide_tiles(a, call.bf16, call.di->sms / 2)) return launch_ep_act<256, true>(call, a, activation);
  return call.bf16 ? launch_ep_act<128, true>(call, a, activation)
                   : launch_ep_act<128, false>(call, a, activation);
}
