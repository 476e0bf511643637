// MXFP4 K/V cache: rows quantized as they are written into their pages, and
// decoded as they are read back.
//
// Both directions are one pass over the data, bound by HBM.  A work item is 8
// channels of one head's row: a 16-byte load (or store) of bf16, 4 bytes of
// codes, and four neighbouring lanes share the block's scale byte.  That keeps
// the bf16 side, four times the bytes of the codes, fully coalesced; a thread
// per 32-element block would read its 64 bytes at a stride of 64 (half of
// every sector fetched twice).  Items run over the positions of one head before
// the next head, the order of the bytes in a page.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kq_cache.cuh"
#include "kq_internal.h"

namespace kq {
namespace {

constexpr int kThreads = 256;
constexpr int kItems = 4;              // work items per thread

struct CacheArgs {
  CacheView view;
  uint8_t* codes[2];                   // K, V
  uint8_t* scales[2];
  uint16_t* x[2];                      // bf16 rows (float32 for a float32 read)
  int64_t sb[2], st[2], sh[2];         // strides of x in elements
  const int32_t* start;
  const int32_t* lens;
  int32_t tokens, head_dim;
  int32_t t_shift;                     // positions in a tile: 2^t_shift
  uint32_t items;                      // per sequence
  FastDiv tile, head;                  // items of a tile, of one head in it
  FastDiv chunk;                       // 8-channel items of a row
  int* err;
};

struct Item {
  int t, h, c;
  bool in;                             // a row of x
};

__device__ __forceinline__ Item item_at(const CacheArgs& a, uint32_t i) {
  const uint32_t tile = a.tile.div(i), r = i - tile * a.tile.d;
  const uint32_t h = a.head.div(r), q = r - h * a.head.d;
  const uint32_t row = a.chunk.div(q);
  Item it;
  it.t = static_cast<int>((tile << a.t_shift) + row);
  it.h = static_cast<int>(h);
  it.c = static_cast<int>(q - row * a.chunk.d);
  it.in = i < a.items && it.t < a.tokens;
  return it;
}

__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheArgs a) {
  pdl_wait_then_trigger();
  const int64_t b = blockIdx.y;
  const int kv = blockIdx.z;
  const int64_t start = a.start ? a.start[b] : 0;
  const int rows = a.lens ? min(a.lens[b], a.tokens) : a.tokens;
  const uint32_t i0 = blockIdx.x * (kThreads * kItems) + threadIdx.x;
  Item it[kItems];
  uint4 raw[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    it[k] = item_at(a, i0 + k * kThreads);
    it[k].in = it[k].in && it[k].t < rows;
    raw[k] = make_uint4(0, 0, 0, 0);
    if (it[k].in && it[k].c * 8 < a.head_dim)
      raw[k] = __ldg(reinterpret_cast<const uint4*>(a.x[kv] + b * a.sb[kv] + it[k].t * a.st[kv] +
                                                     it[k].h * a.sh[kv] + it[k].c * 8));
  }
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
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
    if (!it[k].in) continue;
    const int64_t row = cache_row(a.view, b, start + it[k].t, it[k].h);
    if (row < 0) {
      if (it[k].c == 0) atomicOr(a.err, kErrCacheIndex);
      continue;
    }
    reinterpret_cast<uint32_t*>(a.codes[kv])[row * (4 * a.view.nb) + it[k].c] = w;
    if ((it[k].c & 3) == 0) a.scales[kv][row * a.view.nb + (it[k].c >> 2)] = static_cast<uint8_t>(s);
  }
}

template <bool kF32>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheArgs a) {
  pdl_wait_then_trigger();
  const int64_t b = blockIdx.y;
  const int kv = blockIdx.z;
  const int64_t start = a.start ? a.start[b] : 0;
  const int rows = a.lens ? min(a.lens[b], a.tokens) : a.tokens;
  const uint32_t i0 = blockIdx.x * (kThreads * kItems) + threadIdx.x;
  Item it[kItems];
  uint32_t w[kItems];
  uint32_t s[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    it[k] = item_at(a, i0 + k * kThreads);
    it[k].in = it[k].in && it[k].c * 8 < a.head_dim;
    w[k] = 0;
    s[k] = 127;
    if (it[k].in && it[k].t < rows) {
      const int64_t row = cache_row(a.view, b, start + it[k].t, it[k].h);
      if (row < 0) {
        if (it[k].c == 0) atomicOr(a.err, kErrCacheIndex);
      } else {
        w[k] = __ldg(reinterpret_cast<const uint32_t*>(a.codes[kv]) + row * (4 * a.view.nb) + it[k].c);
        s[k] = __ldg(a.scales[kv] + row * a.view.nb + (it[k].c >> 2));
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    if (!it[k].in) continue;
    float v[8];
    e2m1x8_to_float(w[k], v);
    // Exact: a product with a power of two, and at most two significant bits.
    const float p = e8m0_to_float(s[k]);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= p;
    const int64_t at = b * a.sb[kv] + it[k].t * a.st[kv] + it[k].h * a.sh[kv] + it[k].c * 8;
    if constexpr (kF32) {
      float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.x[kv]) + at);
      dst[0] = make_float4(v[0], v[1], v[2], v[3]);
      dst[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 p2 = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        o[j] = *reinterpret_cast<const uint32_t*>(&p2);
      }
      *reinterpret_cast<uint4*>(a.x[kv] + at) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

bool fill(CacheArgs* a, const kq_cache* c, const int32_t* table, int64_t batch, int64_t table_pages,
          int64_t tokens) {
  if (!cache_view(c, table, batch, table_pages, &a->view)) return false;
  const int64_t chunk = 4 * a->view.nb;
  // Tiles of up to 16 positions, fewer where there are fewer (a power of two).
  a->t_shift = 0;
  while (a->t_shift < 4 && (int64_t(1) << a->t_shift) < tokens) ++a->t_shift;
  const int64_t head = chunk << a->t_shift, tile = head * c->heads;
  const int64_t tiles = (tokens + (int64_t(1) << a->t_shift) - 1) >> a->t_shift;
  if (tile > (int64_t(1) << 30) || tiles > ((int64_t(1) << 31) - kThreads * kItems - 1) / tile) return false;
  a->items = static_cast<uint32_t>(tiles * tile);
  a->tile = FastDiv(static_cast<uint32_t>(tile));
  a->head = FastDiv(static_cast<uint32_t>(head));
  a->chunk = FastDiv(static_cast<uint32_t>(chunk));
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

dim3 cache_grid(const CacheArgs& a, int64_t batch) {
  return dim3((a.items + kThreads * kItems - 1) / (kThreads * kItems), static_cast<unsigned>(batch), 2);
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
  cudaError_t e = launch_pdl(cache_write_kernel, cache_grid(a, batch), dim3(kThreads), 0,
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
                      ? launch_pdl(cache_read_kernel<true>, cache_grid(a, batch), dim3(kThreads), 0, st, a)
                      : launch_pdl(cache_read_kernel<false>, cache_grid(a, batch), dim3(kThreads), 0, st, a);
  return e == cudaSuccess ? KQ_OK : record_cuda_error(e);
}
