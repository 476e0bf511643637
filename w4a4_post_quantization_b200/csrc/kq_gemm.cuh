// Shared by the W4A4 product's kernels: tile and scale geometry, the operand
// tensor maps, and the load and MMA roles of a CTA pair.
#pragma once

#include <cuda.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "kq_device.cuh"
#include "kq_internal.h"
#include "kq_tc.cuh"

namespace kq {

constexpr int kBM = 128;                       // UMMA M: rows of A per tile
constexpr int kBN = 256;                       // UMMA N: rows of B per tile
constexpr int kBK = 256;                       // K elements per stage
constexpr int kBKBytes = kBK / 2;              // 128 bytes of codes per row
constexpr int kMmaK = 64;                      // K elements per MMA
constexpr int kATile = kBM * kBKBytes;         // 16 KiB
constexpr int kBTile = kBN * kBKBytes;         // 32 KiB
constexpr int kSfChunk = 512;                  // 128 rows x 4 scale bytes
constexpr int kChunksPerStage = kBK / 128;     // 2 chunks of 4 scales per row
constexpr int kSfaBytes = kChunksPerStage * kSfChunk;
constexpr int kSfbBytes = kChunksPerStage * (kBN / 128) * kSfChunk;
constexpr int kBandN = 16;                     // column tiles per raster band

// TMEM: the accumulator in columns [0, 256), then per stage 4 columns per
// scale chunk of A and 8 per chunk of B (two 128-row groups).
constexpr int kSfColsA = 4 * kChunksPerStage;
constexpr int kSfColsB = 8 * kChunksPerStage;
constexpr int kSfCol0 = kBN;
constexpr int kTmemCols = 512;

// Polls of the wait for a whole product along K, in k_tiles stages.  A stage takes 1.2 us
// at most (the 50 KB of every SM at once out of HBM); two polls, 2.5 us each or more, are
// waited for it, beside the bound of every other wait.
inline int product_polls(int64_t k_tiles) { return static_cast<int>(kWaitPolls + 2 * k_tiles); }

// The same MMA over a CTA pair (M = 256): issued by the even CTA, A rows and
// accumulator rows 0..127 in it and 128..255 in the odd one, B's N rows split
// 128 / 128 between their shared memories, each CTA's scales in its TMEM.
__device__ __forceinline__ void mma_mxf4_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                              uint32_t idesc, uint32_t tsfa, uint32_t tsfb,
                                              uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;"
      "\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(tsfa), "r"(tsfb)
      : "memory");
}

// Row-major packed codes [rows][K/2] as a 2-D byte tensor; a box is
// `box_rows` rows of 128 bytes (256 codes), 128-byte swizzle.
inline bool encode_codes_map(CUtensorMap* map, const uint8_t* q, int64_t rows, int64_t K, int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K / 2), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K / 2)};
  const cuuint32_t box[2] = {kBKBytes, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(q), dims,
                              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tiled scales [row tiles][4-scale columns][512 bytes] as a 4-D byte tensor
// {256, 2, columns, row tiles}; a box {256, 2, 2, box_tiles} is the two
// columns of one k-tile for box_tiles row tiles (zeros past either end).
inline bool encode_scales_map(CUtensorMap* map, const uint8_t* sf, int64_t row_tiles, int64_t cols,
                       int box_tiles) {
  const cuuint64_t dims[4] = {256, 2, static_cast<cuuint64_t>(cols),
                              static_cast<cuuint64_t>(row_tiles)};
  const cuuint64_t strides[3] = {256, 512, static_cast<cuuint64_t>(cols) * 512};
  const cuuint32_t box[4] = {256, 2, 2, static_cast<cuuint32_t>(box_tiles)};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(sf),
                              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---------------------------------------------------------------- CTA pairs
// A cluster of two CTAs computes tiles of 256 rows and kN columns of C
// (tcgen05.mma.cta_group::2, M = 256).  Each CTA loads its 128 rows of A and
// its kN / 2 rows of B, so B costs each SM half the bytes per flop of a
// one-CTA tile, plus the scales of its A rows and of all kN B rows (the MMA
// reads B's scales from each CTA's own TMEM).  With kN = 128 there are two
// accumulators, so that the next tile's MMAs run while one is drained.
constexpr int kPairM = 2 * kBM;

template <int kN, int kStagesP>
struct PairGeom {
  static constexpr int kBRows = kN / 2;                       // B rows per CTA
  static constexpr int kBBytes = kBRows * kBKBytes;
  static constexpr int kGroups = kN / 128;                    // 128-row groups of B's scales
  static constexpr int kSfb = kChunksPerStage * kGroups * kSfChunk;
  static constexpr int kStage = kATile + kBBytes + kSfaBytes + kSfb;
  static constexpr int kAcc = kN == 128 ? 2 : 1;              // accumulators
  static constexpr int kColsB = 4 * kGroups * kChunksPerStage;
  static constexpr int kSf0 = kAcc * kN;                      // first TMEM column of the scales
  static constexpr uint32_t kIdesc = (1u << 7) | (1u << 10) | (uint32_t(kN >> 3) << 17) | (1u << 23) |
                                     (uint32_t(kPairM >> 4) << 24);
  // Bytes one k-tile brings into the pair.
  static constexpr uint32_t kTx = 2u * kStage;
  static_assert(kStage % 1024 == 0, "stages keep the 1024-byte swizzle alignment");
  static_assert(kSf0 + kStagesP * (kSfColsA + kColsB) <= kTmemCols, "TMEM columns");
};

struct PairTiles {
  int32_t K, k_tiles, m_tiles, n_tiles;     // tiles of 256 x kN
  int32_t polls;                            // bound of the epilogue's wait (product_polls)
};

// Tile t of the banded order (bands of kBandN column tiles, the row tile
// changing fastest).
template <int kN>
__device__ __forceinline__ void pair_tile_origin(const PairTiles& a, int t, int& m0, int& n0) {
  const int band = t / (kBandN * a.m_tiles);
  const int r = t - band * kBandN * a.m_tiles;
  const int width = min(kBandN, a.n_tiles - band * kBandN);
  m0 = (r / width) * kPairM;
  n0 = (band * kBandN + r % width) * kN;
}

// One thread of each CTA: the stages' loads.  Every load of the pair counts
// its bytes on rank 0's stage barrier; none uses cluster multicast.  False if
// a bounded wait gave up; the copies still counted then were issued before that wait,
// of 10 ms and more, and have landed.
template <int kN, int kStagesP>
__device__ __forceinline__ bool pair_produce(uint8_t* base, uint64_t* full, uint64_t* empty,
                                             const CUtensorMap* amap, const CUtensorMap* bmap,
                                             const CUtensorMap* sfamap, const CUtensorMap* sfbmap,
                                             const PairTiles& a, uint32_t rank, int pair,
                                             int n_pairs) {
  using P = PairGeom<kN, kStagesP>;
  tma_prefetch_map(amap);
  tma_prefetch_map(bmap);
  tma_prefetch_map(sfamap);
  tma_prefetch_map(sfbmap);
  const int n_tiles_total = a.m_tiles * a.n_tiles;
  int s = 0, g = 0;
  uint32_t phase = 0;
  for (int t = pair; t < n_tiles_total; t += n_pairs) {
    int m0, n0;
    pair_tile_origin<kN>(a, t, m0, n0);
    const int am0 = m0 + (int)rank * kBM, bn0 = n0 + (int)rank * P::kBRows;
    for (int kt = 0; kt < a.k_tiles; ++kt, ++g) {
      if (g >= kStagesP && !mbar_wait(&empty[s], phase)) return false;
      uint8_t* stg = base + s * P::kStage;
      const uint32_t fb = cluster_addr(&full[s], 0);
      if (rank == 0) mbar_arrive_expect_tx(&full[s], P::kTx);
      uint8_t* sfa = stg + kATile + P::kBBytes;
      // Scales: chunks 2 kt, 2 kt + 1 of this CTA's A row tile and of the
      // tile's B row tiles (zero past the ends).
      tma_load_4d_pair(sfa, sfamap, 0, 0, 2 * kt, am0 / 128, fb);
      tma_load_4d_pair(sfa + kSfaBytes, sfbmap, 0, 0, 2 * kt, n0 / 128, fb);
      tma_load_2d_pair(stg, amap, kt * kBKBytes, am0, fb);
      tma_load_2d_pair(stg + kATile, bmap, kt * kBKBytes, bn0, fb);
      if (++s == kStagesP) {
        s = 0;
        if (g >= kStagesP) phase ^= 1;
      }
    }
  }
  return true;
}

// One thread of the even CTA: scale copies and MMAs.  The commits arrive on
// the barriers of both CTAs.  acc_empty completes once both CTAs' epilogues
// have read an accumulator.  False if a bounded wait gave up (the tile's commit
// is sent all the same, so that the epilogues go on).
template <int kN, int kStagesP>
__device__ __forceinline__ bool pair_mma(uint8_t* base, uint64_t* full, uint64_t* empty,
                                         uint64_t* acc_full, uint64_t* acc_empty, uint32_t tmem_base,
                                         const PairTiles& a, int pair, int n_pairs) {
  using P = PairGeom<kN, kStagesP>;
  const int n_tiles_total = a.m_tiles * a.n_tiles;
  int s = 0, i = 0;
  uint32_t phase = 0;
  uint32_t tacc = tmem_base;
  bool ok = true;
  auto ktile = [&](int kt, auto full_tile) -> bool {
    if (!mbar_wait(&full[s], phase)) return false;
    tmem_fence_after();
    const uint8_t* stg = base + s * P::kStage;
    const uint8_t* sfa = stg + kATile + P::kBBytes;
    const uint8_t* sfb = sfa + kSfaBytes;
    const uint32_t tsfa = tmem_base + P::kSf0 + s * (kSfColsA + P::kColsB);
    const uint32_t tsfb = tsfa + kSfColsA;
#pragma unroll
    for (int c = 0; c < kChunksPerStage; ++c) {
      tmem_cp_pair_32x128b_x4(tsfa + 4 * c, smem_desc_rows16(smem_addr(sfa + c * kSfChunk)));
#pragma unroll
      for (int gb = 0; gb < P::kGroups; ++gb)
        tmem_cp_pair_32x128b_x4(tsfb + 4 * P::kGroups * c + 4 * gb,
                                smem_desc_rows16(smem_addr(sfb + (2 * gb + c) * kSfChunk)));
    }
    const uint64_t adesc = smem_desc_sw128(smem_addr(stg));
    const uint64_t bdesc = smem_desc_sw128(smem_addr(stg + kATile));
    const int n_mma = decltype(full_tile)::value
                          ? kBK / kMmaK
                          : min(kBK / kMmaK, (a.K - kt * kBK + kMmaK - 1) / kMmaK);
#pragma unroll
    for (int kk = 0; kk < kBK / kMmaK; ++kk) {
      if (!decltype(full_tile)::value && kk >= n_mma) break;
      const uint32_t sf_id = 2u * (kk & 1);
      const uint32_t idesc = P::kIdesc | (sf_id << 29) | (sf_id << 4);
      mma_mxf4_pair(tacc, adesc + 2 * kk, bdesc + 2 * kk, idesc, tsfa + 4 * (kk >> 1),
                    tsfb + 4 * P::kGroups * (kk >> 1), (kt | kk) != 0);
    }
    mma_commit_pair(&empty[s]);
    if (++s == kStagesP) {
      s = 0;
      phase ^= 1;
    }
    return true;
  };
  for (int t = pair; t < n_tiles_total && ok; t += n_pairs, ++i) {
    const int b = i % P::kAcc;
    if (i >= P::kAcc && !mbar_wait_cluster(&acc_empty[b], ((i / P::kAcc) - 1) & 1)) {
      ok = false;
      break;
    }
    tacc = tmem_base + b * kN;
    tmem_fence_after();
    const int nk_full = a.K % kBK == 0 ? a.k_tiles : a.k_tiles - 1;
    int kt = 0;
    for (; ok && kt < nk_full; ++kt) ok = ktile(kt, std::true_type{});
    if (ok && kt < a.k_tiles) ok = ktile(kt, std::false_type{});
    mma_commit_pair(&acc_full[b]);
  }
  return ok;
}

// Launches a pair kernel: clusters of two, as many as can be resident (asked of
// the driver once per device), with programmatic dependent launch where `pdl`
// is set (the kernel then waits for the previous one before its first global
// access).
template <auto kKernel, typename... Args>
int launch_pairs(int threads, int smem, int64_t tiles, const DeviceInfo* di, int dev, bool pdl,
                 cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static std::mutex mu;
  static int resident[kMaxDevices] = {0};
  int clusters;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (resident[dev] == 0) {
      cfg.gridDim = dim3(static_cast<unsigned>(2 * (di->sms / 2)));
      int n = 0;
      const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kKernel, &cfg);
      if (e != cudaSuccess || n < 1)
        return record_cuda_error(e != cudaSuccess ? e : cudaErrorInvalidConfiguration);
      resident[dev] = n;
    }
    clusters = resident[dev];
  }
  cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(tiles, clusters)));
  cfg.numAttrs = pdl ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kKernel, args...);
  return e == cudaSuccess ? KQ_OK : record_cuda_error(e);
}

}  // namespace kq
