// MXFP4 K/V cache: rows quantized as they are written into their pages, and
// decoded as they are read back.
//
// Both directions are one pass over the data, bound by HBM.  A thread keeps one
// position and 8 channels of its rows and walks the heads: the page is looked up
// once, and from head to head only two pointers move by constant strides.  8
// channels are a 16-byte load (or store) of bf16 and 4 bytes of codes, and four
// neighbouring lanes share the block's scale byte.  That keeps the bf16 side,
// four times the bytes of the codes, fully coalesced; a thread per 32-element
// block would read its 64 bytes at a stride of 64 (half of every sector fetched
// twice).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kq_cache.cuh"
#include "kq_internal.h"

namespace kq {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;              // heads in flight per thread

struct CacheArgs {
  CacheView view;
  uint8_t* codes[2];                   // K, V
  uint8_t* scales[2];
  uint16_t* x[2];                      // bf16 rows (float32 for a float32 read)
  int64_t sb[2], st[2], sh[2];         // strides of x in elements
  const int32_t* start;
  const int32_t* lens;
  int32_t tokens, head_dim;
  int32_t rows;                        // positions of a block
  int32_t heads;                       // heads of a block
  FastDiv chunk;                       // 8-channel pieces of a row
  int* err;
};

// What a thread works on: piece c of the rows of one position.
struct Place {
  int t, c, h0, n;                     // position in x, piece, first head, heads (0: nothing)
  int64_t row;                         // cache row of head h0, -1: no page
};

__device__ __forceinline__ Place place_of(const CacheArgs& a, int64_t b, int split, bool lookup_all) {
  Place p;
  const uint32_t r = a.chunk.div(threadIdx.x);
  p.c = static_cast<int>(threadIdx.x - r * a.chunk.d);
  p.t = static_cast<int>(blockIdx.x) * a.rows + static_cast<int>(r);
  p.h0 = split * a.heads;
  p.n = static_cast<int>(r) < a.rows && p.t < a.tokens ? min(a.heads, a.view.heads - p.h0) : 0;
  const int lens = a.lens ? min(a.lens[b], a.tokens) : a.tokens;
  p.row = -1;
  if (p.n > 0 && p.t < lens) {
    p.row = cache_row(a.view, b, (a.start ? a.start[b] : 0) + static_cast<int64_t>(p.t), p.h0);
    if (p.row < 0 && p.c == 0) atomicOr(a.err, kErrCacheIndex);
  }
  if (!lookup_all && p.row < 0) p.n = 0;
  return p;
}

__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheArgs a) {
  pdl_wait_then_trigger();
  const int64_t b = blockIdx.y;
  const int kv = blockIdx.z & 1;
  const Place p = place_of(a, b, blockIdx.z >> 1, false);
  const bool real = p.c * 8 < a.head_dim;
  const uint16_t* src = a.x[kv] + b * a.sb[kv] + p.t * a.st[kv] + p.h0 * a.sh[kv] + p.c * 8;
  uint32_t* codes = reinterpret_cast<uint32_t*>(a.codes[kv]) + p.row * (4 * a.view.nb) + p.c;
  uint8_t* scales = a.scales[kv] + p.row * a.view.nb + (p.c >> 2);
  const int64_t step = int64_t(1) << a.view.page_shift;        // rows from head to head
  // The heads of every lane's block alike, so that the block's four lanes meet.
  const int heads = min(a.heads, a.view.heads - p.h0);
  for (int h = 0; h < heads; h += kHeads) {
    uint4 raw[kHeads];
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      raw[k] = make_uint4(0, 0, 0, 0);
      if (real && h + k < p.n) raw[k] = __ldcs(reinterpret_cast<const uint4*>(src + (h + k) * a.sh[kv]));
    }
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      f2 u[4] = {bf16x2_to_f2(raw[k].x), bf16x2_to_f2(raw[k].y), bf16x2_to_f2(raw[k].z),
                 bf16x2_to_f2(raw[k].w)};
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) unpack2(u[j], v[2 * j], v[2 * j + 1]);
      float amax = fmaxf(max3(fabsf(v[0]), fabsf(v[1]), fabsf(v[2])),
                         max3(fabsf(v[3]), fabsf(v[4]), max3(fabsf(v[5]), fabsf(v[6]), fabsf(v[7]))));
      // The block's four lanes.
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      f2 inv;
      const uint32_t s = e8m0_from_amax(amax, inv);
#pragma unroll
      for (int j = 0; j < 4; ++j) unpack2(mul2(u[j], inv), v[2 * j], v[2 * j + 1]);
      const uint32_t w = e2m1x8(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
      if (h + k < p.n) {
        codes[(h + k) * step * (4 * a.view.nb)] = w;
        if ((p.c & 3) == 0) scales[(h + k) * step * a.view.nb] = static_cast<uint8_t>(s);
      }
    }
  }
}

template <bool kF32>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheArgs a) {
  pdl_wait_then_trigger();
  const int64_t b = blockIdx.y;
  const int kv = blockIdx.z & 1;
  const Place p = place_of(a, b, blockIdx.z >> 1, true);
  if (p.c * 8 >= a.head_dim) return;
  const int64_t at = b * a.sb[kv] + p.t * a.st[kv] + p.h0 * a.sh[kv] + p.c * 8;
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(a.codes[kv]) + p.row * (4 * a.view.nb) + p.c;
  const uint8_t* scales = a.scales[kv] + p.row * a.view.nb + (p.c >> 2);
  const int64_t step = int64_t(1) << a.view.page_shift;
  for (int h = 0; h < p.n; h += kHeads) {
    uint32_t w[kHeads], s[kHeads];
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      w[k] = 0;
      s[k] = 127;
      if (p.row >= 0 && h + k < p.n) {
        w[k] = __ldg(codes + (h + k) * step * (4 * a.view.nb));
        s[k] = __ldg(scales + (h + k) * step * a.view.nb);
      }
    }
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      if (h + k >= p.n) break;
      float v[8];
      e2m1x8_to_float(w[k], v);
      // Exact: a product with a power of two, and at most two significant bits.
      const float x = e8m0_to_float(s[k]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= x;
      const int64_t to = at + (h + k) * a.sh[kv];
      if constexpr (kF32) {
        float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.x[kv]) + to);
        __stcs(dst, make_float4(v[0], v[1], v[2], v[3]));
        __stcs(dst + 1, make_float4(v[4], v[5], v[6], v[7]));
      } else {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 p2 = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
          o[j] = *reinterpret_cast<const uint32_t*>(&p2);
        }
        __stcs(reinterpret_cast<uint4*>(a.x[kv] + to), make_uint4(o[0], o[1], o[2], o[3]));
      }
    }
  }
}

bool fill(CacheArgs* a, const kq_cache* c, const int32_t* table, int64_t batch, int64_t table_pages,
          int64_t tokens) {
  if (!cache_view(c, table, batch, table_pages, &a->view)) return false;
  if (tokens >= (int64_t(1) << 31) - kThreads) return false;
  const int64_t chunk = 4 * a->view.nb;
  a->rows = static_cast<int32_t>(std::min<int64_t>(kThreads / chunk, tokens));
  a->chunk = FastDiv(static_cast<uint32_t>(chunk));
  // All heads in one block where the positions fill the GPU, else a few each.
  const int64_t blocks = (tokens + a->rows - 1) / a->rows * batch;
  const int64_t splits = std::min<int64_t>((c->heads + kHeads - 1) / kHeads, std::max<int64_t>(1, 148 * 8 / blocks));
  a->heads = static_cast<int32_t>((c->heads + splits - 1) / splits);
  if ((c->heads + a->heads - 1) / a->heads > 32767) return false;
  a->tokens = static_cast<int32_t>(tokens);
  a->head_dim = static_cast<int32_t>(c->head_dim);
  a->codes[0] = c->k_codes;
  a->codes[1] = c->v_codes;
  a->scales[0] = c->k_scales;
  a->scales[1] = c->v_scales;
  return true;
}

// x: 16-byte aligned, rows on 16-byte boundaries.
bool rows_ok(const void* x, int64_t sb, int64_t st, int64_t sh, int esize) {
  const int64_t unit = 16 / esize;
  return x && reinterpret_cast<uintptr_t>(x) % 16 == 0 && sb >= 0 && st >= 0 && sh >= 0 &&
         sb % unit == 0 && st % unit == 0 && sh % unit == 0;
}

// Whole warps for the rows of a block.
dim3 cache_block(const CacheArgs& a) { return dim3((a.rows * a.chunk.d + 31) / 32 * 32); }

dim3 cache_grid(const CacheArgs& a, int64_t batch) {
  return dim3((a.tokens + a.rows - 1) / a.rows, static_cast<unsigned>(batch),
              2 * ((a.view.heads + a.heads - 1) / a.heads));
}

}  // namespace
}  // namespace kq

using namespace kq;

extern "C" int kq_cache_write(const kq_cache* cache, const int32_t* block_table, int64_t batch,
                              int64_t table_pages, const uint16_t* k, int64_t k_sb, int64_t k_st,
                              int64_t k_sh, const uint16_t* v, int64_t v_sb, int64_t v_st,
                              int64_t v_sh, int64_t tokens, const int32_t* start,
                              const int32_t* lens, void* stream) {
  if (batch < 0 || tokens < 0) return KQ_ERR_INVALID;
  if (batch == 0 || tokens == 0) return KQ_OK;
  CacheArgs a{};
  if (!fill(&a, cache, block_table, batch, table_pages, tokens)) return KQ_ERR_INVALID;
  if (!rows_ok(k, k_sb, k_st, k_sh, 2) || !rows_ok(v, v_sb, v_st, v_sh, 2)) return KQ_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(start) % 4 || reinterpret_cast<uintptr_t>(lens) % 4)
    return KQ_ERR_INVALID;
  a.x[0] = const_cast<uint16_t*>(k);
  a.x[1] = const_cast<uint16_t*>(v);
  a.sb[0] = k_sb, a.st[0] = k_st, a.sh[0] = k_sh;
  a.sb[1] = v_sb, a.st[1] = v_st, a.sh[1] = v_sh;
  a.start = start;
  a.lens = lens;
  const DeviceInfo* di = nullptr;
  int dev = 0;
  int rc = device_info(&di, &dev);
  if (rc != KQ_OK) return rc;
  rc = device_error_word(dev, &a.err);
  if (rc != KQ_OK) return rc;
  cudaError_t e = launch_pdl(cache_write_kernel, cache_grid(a, batch), cache_block(a), 0,
                             static_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? KQ_OK : record_cuda_error(e);
}

extern "C" int kq_cache_read(const kq_cache* cache, const int32_t* block_table, int64_t batch,
                             int64_t table_pages, int64_t tokens, const int32_t* start,
                             const int32_t* lens, void* k, int64_t k_sb, int64_t k_st,
                             int64_t k_sh, void* v, int64_t v_sb, int64_t v_st, int64_t v_sh,
                             int dtype, void* stream) {
  if (batch < 0 || tokens < 0 || (dtype != KQ_OUT_F32 && dtype != KQ_OUT_BF16)) return KQ_ERR_INVALID;
  if (batch == 0 || tokens == 0) return KQ_OK;
  CacheArgs a{};
  if (!fill(&a, cache, block_table, batch, table_pages, tokens)) return KQ_ERR_INVALID;
  const int esize = dtype == KQ_OUT_F32 ? 4 : 2;
  if (!rows_ok(k, k_sb, k_st, k_sh, esize) || !rows_ok(v, v_sb, v_st, v_sh, esize))
    return KQ_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(start) % 4 || reinterpret_cast<uintptr_t>(lens) % 4)
    return KQ_ERR_INVALID;
  a.x[0] = static_cast<uint16_t*>(k);
  a.x[1] = static_cast<uint16_t*>(v);
  a.sb[0] = k_sb, a.st[0] = k_st, a.sh[0] = k_sh;
  a.sb[1] = v_sb, a.st[1] = v_st, a.sh[1] = v_sh;
  a.start = start;
  a.lens = lens;
  const DeviceInfo* di = nullptr;
  int dev = 0;
  int rc = device_info(&di, &dev);
  if (rc != KQ_OK) return rc;
  rc = device_error_word(dev, &a.err);
  if (rc != KQ_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = dtype == KQ_OUT_F32
                      ? launch_pdl(cache_read_kernel<true>, cache_grid(a, batch), cache_block(a), 0, st, a)
                      : launch_pdl(cache_read_kernel<false>, cache_grid(a, batch), cache_block(a), 0, st, a);
  return e == cudaSuccess ? KQ_OK : record_cuda_error(e);
}
