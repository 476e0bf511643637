// Shared by the kernels of the MXFP4 K/V cache: how a head's row is laid out
// in a page, E2M1 decoding, and division by a launch constant.
//
// A page holds page_size positions of every K/V head, head by head:
//   codes  [page][head][slot][Dp / 2]   Dp = head_dim rounded up to 32
//   scales [page][head][slot][Dp / 32]
// so that neighbouring positions of one head are neighbouring bytes, which is
// the order the attention walks them in.
#pragma once

#include <cstdint>

#include "kq_device.cuh"
#include "kq.h"

namespace kq {

// Bit of the device error word: a block table named a page outside the pool,
// or a position lay outside its table (that row was left out).
constexpr int kErrCacheIndex = 8;

// n / d for n < 2^31 by a multiplication and a shift (Granlund and
// Montgomery, division by invariant integers).
struct FastDiv {
  uint32_t d = 1, mul = 0, shift = 0;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div) {
    while ((uint64_t(1) << shift) < d) ++shift;
    mul = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << shift) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return (__umulhi(mul, n) + n) >> shift;
  }
};

// Eight E2M1 codes, two a byte, as eight floats (each code is a float16 value
// exactly).
__device__ __forceinline__ void e2m1x8_to_float(uint32_t w, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\t"
        "cvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
        : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
        : "r"(h[i]));
}

// 2^(s - 127) in float32: a subnormal for s = 0, NaN for s = 255 (E8M0's NaN).
__device__ __forceinline__ float e8m0_to_float(uint32_t s) {
  return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7FC00000u : s << 23);
}

// A sequence's positions in the cache.
struct CacheView {
  const int32_t* table;       // [batch][table_pages]
  int32_t table_pages;
  int32_t pages, heads;
  int32_t page_shift;         // page_size = 2^page_shift
  int32_t nb;                 // 32-element blocks of a head's row
};

// Row index of (position, head) in units of one head's row, or -1 where the
// position has no page in the pool.
__device__ __forceinline__ int64_t cache_row(const CacheView& c, int64_t b, int64_t pos, int head) {
  if (pos < 0) return -1;
  const int64_t at = pos >> c.page_shift;
  if (at >= c.table_pages) return -1;
  const int32_t page = __ldg(c.table + b * c.table_pages + at);
  if (page < 0 || page >= c.pages) return -1;
  return ((static_cast<int64_t>(page) * c.heads + head) << c.page_shift) +
         (pos & ((int64_t(1) << c.page_shift) - 1));
}

// Host: checks a cache and a table, and fills in the view.
inline bool cache_view(const kq_cache* c, const int32_t* table, int64_t batch, int64_t table_pages,
                       CacheView* v) {
  if (!c || !c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales || !table) return false;
  if (c->pages < 1 || c->pages >= (int64_t(1) << 31) || c->heads < 1 || c->heads > 65535) return false;
  if (c->page_size < 16 || c->page_size > 65536 || (c->page_size & (c->page_size - 1))) return false;
  if (c->head_dim < 8 || c->head_dim > 128 || c->head_dim % 8) return false;
  if (batch < 1 || batch > 65535 || table_pages < 1 || table_pages >= (int64_t(1) << 31)) return false;
  if (table_pages > ((int64_t(1) << 31) - 1) / c->page_size) return false;
  auto al = [](const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  if (!al(c->k_codes, 16) || !al(c->v_codes, 16) || !al(c->k_scales, 16) || !al(c->v_scales, 16) ||
      !al(table, 4))
    return false;
  v->table = table;
  v->table_pages = static_cast<int32_t>(table_pages);
  v->pages = static_cast<int32_t>(c->pages);
  v->heads = static_cast<int32_t>(c->heads);
  v->page_shift = __builtin_ctzll(static_cast<unsigned long long>(c->page_size));
  v->nb = static_cast<int32_t>((c->head_dim + 31) / 32);
  return true;
}

}  // namespace kq
