// Attention with many query rows: on the tensor cores (tcgen05, kind::f16).
//
// Every 128-row tile of queries multiplies the same keys and values, so they
// are decoded once per call, by a first kernel, into tiles of 128 positions laid
// out as the MMA reads them, in bf16:
//   K image  [channel panel][position][channels of the panel]   (B of S = Q K^T)
//   V image  [position / 64][channel][64 positions]             (B of O = P V)
// both K-major.  V's rows are 128 bytes with the 128-byte swizzle.  K's channels
// (a multiple of 16) are cut into panels of 64, then one of 32 and one of 16
// for the rest, each with the swizzle of its row, so that a head of 72 or 112
// channels takes no padding beyond 16 and a tile arrives as one plain bulk copy of
// 256 D bytes.  (Panels of 16 throughout, with the 32-byte swizzle, made the
// operand reads the bound: 2048 x 8192 causal, 32 heads of 128, took 295 us.)
//
// The second kernel works on items: a tile of 128 rows (query, head of the group) of
// one K/V head, over all positions or a part of them.  Two blocks are resident on an
// SM, so that the products of one run under the softmax of the other, and each takes
// items in turn.  Warps 0 .. 3 hold one row a thread: scores out of tensor memory, the
// running maximum and sum, weights back into it as bf16 in the scores' place, where
// the second product reads them.  One thread loads keys and values, one issues the
// MMAs, and two warps fetch the next item's queries.  The accumulator O stays in
// tensor memory.  It is rescaled only when a row's maximum has grown by more than 2^8:
// until then the weights are relative to the older maximum, which float32 and bf16
// hold as well.  (A block with two query tiles that take turns at the exponentials,
// alone on its SM, reads keys and values half as often, but nothing covers its start
// and end: 2048 x 8192 causal, 32 heads of 128, 229 against 232 us, without the mask
// 240 against 250; 4096 x 4096, 24 heads of 96, 198 against 194; 4096 x 300,
// 2 x 16 heads, 45 against 38 us for heads of 72, 53 against 45 for 96 and 54
// against 46 for 128.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kq_attention.cuh"
#include "kq_tc.cuh"

namespace kq {
namespace {

constexpr int kKv = 128;                       // positions of a tile
constexpr int kQr = 128;                       // rows of a query tile

// K-major operand in 32-byte rows, 32-byte swizzle: 8-row atoms of 256 bytes.
__device__ __forceinline__ uint64_t smem_desc_sw32(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) |
         (uint64_t(256 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(6) << 61);
}

// Channel panels of 128 rows (Q and K): byte offset of 16-byte chunk c (8
// channels) of row r.  A swizzle moves chunk c of a row of n chunks to
// c ^ (bits 3.. of the row's 128-byte line).
__device__ __forceinline__ int panel_chunk(int d16, int r, int c) {
  const int wide = d16 >> 6;
  if (c < 8 * wide) return (c >> 3) * 16384 + r * 128 + 16 * ((c & 7) ^ (r & 7));
  c -= 8 * wide;
  if (d16 & 32) {
    if (c < 4) return wide * 16384 + r * 64 + 16 * (c ^ ((r >> 1) & 3));
    c -= 4;
  }
  return wide * 16384 + (d16 & 32) * 256 + r * 32 + 16 * (c ^ ((r >> 2) & 1));
}
// Descriptor of K step k (16 channels) of such a tile at a 1024-byte-aligned
// address.  The head's width is a template argument where MMAs are issued: the
// one issuing thread bounds the kernel if it has to work the descriptors out.
template <int kD16>
__device__ __forceinline__ uint64_t panel_desc(uint32_t saddr, int k) {
  constexpr int kWide = kD16 >> 6;
  if (k < 4 * kWide) return smem_desc_sw128(saddr) + ((k >> 2) * 16384 + (k & 3) * 32) / 16;
  if ((kD16 & 32) && k < 4 * kWide + 2)
    return smem_desc_sw64(saddr) + (kWide * 16384 + (k - 4 * kWide) * 32) / 16;
  return smem_desc_sw32(saddr) + (kWide * 16384 + (kD16 & 32) * 256) / 16;
}

// ------------------------------------------------------------------ decode
constexpr int kDecodeThreads = 256;

// One tile of one K/V head of one sequence: K for even blockIdx.y, V for odd.
// The tile's codes and scales are staged in shared memory by 16-byte loads, all
// in flight together, so that the decoding reads them in whatever order makes
// the stores whole 128-byte lines.
__global__ void __launch_bounds__(kDecodeThreads) attn_decode_kernel(const AttnArgs a, uint4* masks,
                                                                     uint8_t* images) {
  pdl_wait_then_trigger();
  const int tile = blockIdx.x, hk = blockIdx.y >> 1, tid = threadIdx.x;
  const bool is_v = blockIdx.y & 1;
  const int64_t b = blockIdx.z;
  const int pos0 = tile * kKv, nb = a.view.nb;
  // The table's entries beside the length, not after it.
  const int64_t row = tid < kKv / 16 ? cache_row(a.view, b, pos0 + 16 * tid, hk) : -1;
  const int len = seq_len(a, b);
  if (pos0 >= len) return;
  __shared__ int64_t rows[kKv / 16];           // cache row of each 16 positions, -1: none
  __shared__ uint32_t there[kKv / 32];         // which positions there are
  __shared__ __align__(16) uint8_t codes[kKv * 64];
  __shared__ __align__(16) uint8_t scales[kKv * 4];
  if (tid < kKv / 16) {
    const bool in = pos0 + 16 * tid < len;
    rows[tid] = in ? row : -1;
    if (in && row < 0) atomicOr(a.err, kErrCacheIndex);
  }
  __syncthreads();
  if (tid < kKv / 32) {
    uint32_t bits = (rows[2 * tid] >= 0 ? 0xFFFFu : 0u) | (rows[2 * tid + 1] >= 0 ? 0xFFFF0000u : 0u);
    const int left = len - pos0 - 32 * tid;
    if (left < 32) bits &= left <= 0 ? 0u : (1u << left) - 1u;
    there[tid] = bits;
    if (hk == 0 && !is_v) reinterpret_cast<uint32_t*>(masks + b * a.tiles + tile)[tid] = bits;
  }
  // 16 positions are 16 nb 16-byte pieces of codes and nb of scales in a row.
  const uint8_t* gc = is_v ? a.vc : a.kc;
  const uint8_t* gs = is_v ? a.vs : a.ks;
  for (int i = tid; i < kKv * nb; i += kDecodeThreads) {
    const int64_t r = rows[i / (16 * nb)];
    uint4 x = make_uint4(0, 0, 0, 0);
    if (r >= 0) x = __ldg(reinterpret_cast<const uint4*>(gc + r * (16 * nb)) + i % (16 * nb));
    reinterpret_cast<uint4*>(codes)[i] = x;
  }
  if (tid < kKv / 16 * nb) {
    const int64_t r = rows[tid / nb];
    uint4 x = make_uint4(0, 0, 0, 0);
    if (r >= 0) x = __ldg(reinterpret_cast<const uint4*>(gs + r * nb) + tid % nb);
    reinterpret_cast<uint4*>(scales)[tid] = x;
  }
  __syncthreads();
  uint8_t* img = images + (((b * a.view.heads + hk) * a.tiles + tile) * 2 + is_v) * (256 * a.d16);
  if (!is_v) {
    // Item: 16 channels of a position; a row's panels to neighbouring lanes.
    const int np = a.d16 / 16;
    for (int i = tid; i < np * kKv; i += kDecodeThreads) {
      const int t = i / np, p = i - t * np;
      const uint2 w = *reinterpret_cast<const uint2*>(codes + t * (16 * nb) + 8 * p);
      const bool in = there[t >> 5] >> (t & 31) & 1;
      const uint32_t m = in ? mx_mul(scales[t * nb + (p >> 1)]) * 0x10001u : 0u;
      uint32_t o[8];
      // A word's channels come out as the pairs (k, k + 4): put back in order.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t x[4];
        e2m1_pairs(h ? w.y : w.x, x);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = mul_bf16x2(x[k], m);
        o[4 * h] = __byte_perm(x[0], x[1], 0x5410);
        o[4 * h + 1] = __byte_perm(x[2], x[3], 0x5410);
        o[4 * h + 2] = __byte_perm(x[0], x[1], 0x7632);
        o[4 * h + 3] = __byte_perm(x[2], x[3], 0x7632);
      }
      *reinterpret_cast<uint4*>(img + panel_chunk(a.d16, t, 2 * p)) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(img + panel_chunk(a.d16, t, 2 * p + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
  } else {
    // Item: 8 channels of 8 positions, transposed pair by pair; the positions of
    // a channel to neighbouring lanes.
    for (int i = tid; i < a.d16 / 8 * (kKv / 8); i += kDecodeThreads) {
      const int p = i & 15, wd = i >> 4;
      const uint32_t in = there[p >> 2] >> (8 * (p & 3));
      uint32_t o[8][4];                        // [channel][pair of positions]
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = 8 * p + 2 * k;
        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(codes + t * (16 * nb) + 4 * wd);
        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(codes + (t + 1) * (16 * nb) + 4 * wd);
        const uint32_t m = (in >> (2 * k) & 1 ? mx_mul(scales[t * nb + (wd >> 2)]) : 0u) |
                           (in >> (2 * k + 1) & 1 ? mx_mul(scales[(t + 1) * nb + (wd >> 2)]) << 16 : 0u);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t x[4];
          e2m1_pairs(__byte_perm(w0, w1, h ? 0x7632 : 0x5410), x);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[4 * h + e][k] = mul_bf16x2(x[e], m);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = 8 * wd + e;
        *reinterpret_cast<uint4*>(img + (p >> 3) * (a.d16 * 128) + d * 128 + 16 * ((p & 7) ^ (d & 7))) =
            make_uint4(o[e][0], o[e][1], o[e][2], o[e][3]);
      }
    }
  }
}

// --------------------------------------------------------------- attention
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
// A operand from tensor memory: 8 columns of bf16 pairs per K step of 16.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t ta, uint64_t bdesc, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(ta), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void bulk_load_1d(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}

// D float32, A and B bf16, both K-major, M = 128.
__host__ __device__ constexpr uint32_t idesc_bf16(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (uint32_t(kQr >> 4) << 24);
}

template <int kD16>
struct TcGeom {
  // Two blocks share an SM: 113 KB each.
  static constexpr int kStages = kD16 <= 80 ? 2 : 1;
  // A softmax warpgroup, and one that loads and issues the MMAs (its registers go to
  // the other: the sum of the shares is within what the two are launched with).
  static constexpr int kThreads = 256;
  static constexpr int kSoftRegs = 184;
  static constexpr int kRestRegs = 72;
  static constexpr int kTmem = 256;            // S (128 columns), then O (up to 128)
  // Q, K and V stages, barriers.
  static constexpr int kSmem = 1024 + (1 + 2 * kStages) * 256 * kD16 + 256;
  static_assert(kSmem <= 115712, "shared memory");
};

// mbar_wait as one tight loop, for the waits on every tile's critical path; each
// poll suspends the warp for a time that the hardware bounds.
__device__ __forceinline__ bool mbar_spin(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, 0;\n"
      "POLL:\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "add.u32 n, n, 1;\n\tsetp.lt.u32 q, n, 1000;\n\t@q bra POLL;\n"
      "DONE:\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done ? true : mbar_wait(bar, parity);
}

// Every so many pairs of weights of a whole tile take ex2_poly, the others the
// special-function unit, which alone would need 8 cycles for each of a warp's 128
// columns.  2048 x 8192 causal, 32 heads of 128, and 4096 x 300, 2 x 16 heads of 72:
// every 2nd 265 and 42.0 us, 3rd 248 and 39.2, 4th 234 and 37.8, 5th 237 and 39.0,
// 6th 231 and 41.0, none 240 and 39.6.
constexpr int kPolyEvery = 4;

// -inf for the positions a row does not see.
__device__ __forceinline__ void hide(uint32_t (&x)[32], uint32_t see) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (!(see >> e & 1)) x[e] = 0xFF800000u;
}

// This warp's stores of weights so far are in tensor memory.  The second product
// starts on the first half of a tile's weights.
__device__ __forceinline__ void weights_ready(uint64_t* bar, int lane) {
  tmem_wait_st();
  tmem_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// A row's 128 scores to weights.  kWhole: the row sees every position; else
// `see` says which, `words` of 32 of them are looked at, and the others' weights
// are not used.
template <bool kWhole, int kD16>
__device__ __forceinline__ void softmax_tile(uint32_t ts, uint32_t to, float sc, float& mx, float& l,
                                             bool first, const uint32_t (&see)[4], int words,
                                             uint64_t* p_half, int lane) {
  // The maximum of words 2 and 3 is taken first and they are read again later,
  // so that 64 scores at a time are in registers.
  uint32_t x[2][32];
  float peak = -INFINITY;
#pragma unroll
  for (int h = 1; h >= 0; --h) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (kWhole || 2 * h + u < words) tmem_ld32(ts + 32 * (2 * h + u), x[u]);
    tmem_wait_ld();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int v = 2 * h + u;
      if (!kWhole && v >= words) continue;
      if (!kWhole) hide(x[u], see[v]);
      float top[2] = {__uint_as_float(x[u][0]), __uint_as_float(x[u][1])};
#pragma unroll
      for (int e = 2; e < 30; e += 4) {
        top[0] = max3(top[0], __uint_as_float(x[u][e]), __uint_as_float(x[u][e + 1]));
        top[1] = max3(top[1], __uint_as_float(x[u][e + 2]), __uint_as_float(x[u][e + 3]));
      }
      peak = max3(peak, top[0], max3(top[1], __uint_as_float(x[u][30]), __uint_as_float(x[u][31])));
    }
  }
  const float peak2 = peak * sc;
  if (__any_sync(0xFFFFFFFFu, peak2 > mx + 8.0f)) {
    const float m_new = fmaxf(mx, peak2);
    const float alpha = m_new == -INFINITY ? 1.0f : ex2(mx - m_new);
    mx = m_new;
    l *= alpha;
    if (mx == INFINITY) l = kNaN;
    // These scores were issued after the last weights' product, so O is
    // complete.
    if (!first) {
#pragma unroll 1
      for (int c = 0; c < kD16 / 16; ++c) {
        uint32_t o[16];
        tmem_ld16(to + 16 * c, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
        tmem_st16(to + 16 * c, o);
      }
    }
  }
  // A row that sees positions and has no score above -inf so far is not a number.
  // (Its sum would not always show it: the polynomial has a least value.)
  if (mx == -INFINITY && (kWhole || (see[0] | see[1] | see[2] | see[3]) != 0)) l = kNaN;
  const float shift = kShift - (mx == -INFINITY ? 0.0f : mx);
  const f2 sc2 = pack2(sc, sc), shift2 = pack2(shift, shift);
  f2 sum[2] = {pack2(0.0f, 0.0f), pack2(0.0f, 0.0f)};
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int u = v & 1;
    if (kWhole || v < words) {
      if (v >= 2) {
        if (v == 2) tmem_wait_ld();
        if (!kWhole) hide(x[u], see[v]);
      }
      uint32_t p[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const f2 y = fma2(pack2(__uint_as_float(x[u][2 * e]), __uint_as_float(x[u][2 * e + 1])), sc2,
                          shift2);
        float p0, p1;
        unpack2(y, p0, p1);
        if (kWhole && e % kPolyEvery == kPolyEvery - 1) {
          ex2_poly(pack2(fmaxf(p0, -126.0f), fmaxf(p1, -126.0f)), p0, p1);
        } else {
          p0 = ex2(p0);
          p1 = ex2(p1);
        }
        sum[e & 1] = add2(sum[e & 1], pack2(p0, p1));
        // Rounded to bf16, the type of the product; the sum is taken before.
        p[e] = bf16x2(p0, p1);
      }
      // The weights of word v lie in the first half of the scores' columns,
      // which have all been read.
      if (v == 2) weights_ready(p_half, lane);              // words 0 and 1, stored a while ago
      tmem_st16(ts + 16 * v, p);
    } else if (v == 2) {
      weights_ready(p_half, lane);
    }
    if (v < 2 && (kWhole || v + 2 < words)) tmem_ld32(ts + 32 * (v + 2), x[u]);
  }
  weights_ready(p_half + 1, lane);
  float s0, s1;
  unpack2(add2(sum[0], sum[1]), s0, s1);
  l += s0 + s1;
}

// An item of work: a query tile of one K/V head of one sequence over one part of the
// positions.
struct Item {
  int64_t b;
  int hk, chunk, r0;
  int len, begin, end, n;                      // n: tiles of positions
};

// Item w: the latest rows first (in a causal call they see most).
__device__ __forceinline__ Item place_item(const AttnArgs& a, uint32_t w) {
  Item it;
  const uint32_t row_tiles = (a.rows + kQr - 1) / kQr;
  uint32_t q = w / a.n_chunks;
  it.chunk = static_cast<int>(w - q * a.n_chunks);
  w = q / row_tiles;
  it.r0 = static_cast<int>(row_tiles - 1 - (q - w * row_tiles)) * kQr;
  q = w / a.view.heads;
  it.hk = static_cast<int>(w - q * a.view.heads);
  it.b = q;
  it.len = it.begin = it.end = it.n = 0;
  return it;
}
__device__ __forceinline__ Item item_span(const AttnArgs& a, Item it) {
  it.len = seq_len(a, it.b);
  it.begin = it.chunk * a.chunk;
  it.end = min(it.begin + a.chunk, row_limit(a, it.len, min(it.r0 + kQr, a.rows) - 1));
  it.n = it.end > it.begin ? (it.end - it.begin + kKv - 1) / kKv : 0;
  return it;
}

// 16 bytes from global to shared memory, or zeros.
__device__ __forceinline__ void cp_async16_or_zero(void* dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(real ? 16 : 0)
               : "memory");
}

// 32 kQuarters rows of queries (from quarter `q` on of the item's tile) into the
// swizzled tile at `tile`, by one warp: a row's 16-byte chunks to neighbouring
// lanes, all copies in flight together (through registers in three groups, the
// two warps that fetch the next item's queries took 10000 cycles, longer than the
// item).  A negative scale goes into the queries' signs.
template <int kD16, int kQuarters>
__device__ __forceinline__ void load_queries(const AttnArgs& a, const Item& it, uint8_t* tile, int q, int lane) {
  constexpr int kNc = kD16 / 8, kDr = 32 / kNc, kDc = 32 - kDr * kNc;   // a step of 32 chunks
  const int qr0 = lane / kNc, qc0 = lane - qr0 * kNc;
  int qr = qr0, qc = qc0;
  auto step = [&] {
    qr += kDr;
    qc += kDc;
    if (qc >= kNc) qc -= kNc, ++qr;
  };
#pragma unroll 1
  for (int k = 0; k < kQuarters * kNc; ++k, step()) {
    const int rr = q * 32 + qr, rg = it.r0 + rr;
    const bool real = rg < a.rows && 8 * qc < a.D;
    const int mm = real ? a.group.div(rg) : 0, hh = it.hk * a.group.d + (real ? rg - mm * a.group.d : 0);
    cp_async16_or_zero(tile + panel_chunk(kD16, rr, qc),
                       a.q + it.b * a.qb + mm * a.qm + hh * a.qh + (real ? 8 * qc : 0), real);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (a.scale_log2 < 0.0f) {
    qr = qr0, qc = qc0;
#pragma unroll 1
    for (int k = 0; k < kQuarters * kNc; ++k, step()) {
      uint4* x = reinterpret_cast<uint4*>(tile + panel_chunk(kD16, q * 32 + qr, qc));
      const uint4 y = *x;
      *x = make_uint4(y.x ^ 0x80008000u, y.y ^ 0x80008000u, y.z ^ 0x80008000u, y.w ^ 0x80008000u);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
}

template <int kD16>
__global__ void __launch_bounds__(TcGeom<kD16>::kThreads, 2)
    attn_tc_kernel(const AttnArgs a, uint32_t items) {
  using G = TcGeom<kD16>;
  constexpr int kStages = G::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  constexpr int d16 = kD16, img = 256 * d16;
  uint8_t* sq = base;
  uint8_t* sk = sq + img;
  uint8_t* sv = sk + kStages * img;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(sv + kStages * img);
  uint64_t* k_empty = k_full + kStages;
  uint64_t* v_full = k_empty + kStages;
  uint64_t* v_empty = v_full + kStages;
  uint64_t* q_full = v_empty + kStages;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;
  uint64_t* p_half = s_full + 1;               // for each half of a tile's weights
  uint64_t* o_full = p_half + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_full + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kSoft = 4;               // softmax warps
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(q_full, 4);
    mbar_init(q_empty, 1);
    mbar_init(s_full, 1);
    mbar_init(&p_half[0], 4);
    mbar_init(&p_half[1], 4);
    mbar_init(o_full, 1);
    fence_mbar_init();
  }
  if (warp == kSoft + 1) tmem_alloc(tmem_slot, G::kTmem);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The first item's queries.  Before the wait for the decoded tiles: whatever wrote
  // them was complete before the decoding kernel let this one start.
  if (warp < kSoft) {
    load_queries<kD16, 1>(a, place_item(a, blockIdx.x), sq, warp, lane);
    if (lane == 0) mbar_arrive(q_full);
  }
  pdl_wait_then_trigger();

  if (warp >= kSoft) {
    regs_down<G::kRestRegs>();
    if (warp == kSoft && lane == 0) {
      // ---------------------------------------------------------- loads
      bool ok = true;
      uint32_t g = 0;                          // tiles loaded, over all items
      for (uint32_t w = blockIdx.x; w < items && ok; w += gridDim.x) {
        const Item it = item_span(a, place_item(a, w));
        const uint8_t* src =
            a.images + ((it.b * a.view.heads + it.hk) * a.tiles + it.begin / kKv) * (2ll * img);
        for (int j = 0; j < it.n; ++j, ++g) {
          const int s = g % kStages;
          const uint32_t ph = ((g / kStages) - 1) & 1;
          if (g >= kStages && !(ok = mbar_wait(&k_empty[s], ph))) break;
          mbar_arrive_expect_tx(&k_full[s], img);
          bulk_load_1d(sk + s * img, src + 2ll * img * j, img, &k_full[s]);
          if (g >= kStages && !(ok = mbar_wait(&v_empty[s], ph))) {
            mbar_wait(&k_full[s], (g / kStages) & 1);
            break;
          }
          mbar_arrive_expect_tx(&v_full[s], img);
          bulk_load_1d(sv + s * img, src + 2ll * img * j + img, img, &v_full[s]);
        }
      }
      if (!ok) {
        // The copies in flight land before the block ends.
        atomicOr(a.err, kErrProducerWait);
        for (uint32_t i = g > kStages ? g - kStages : 0; i < g; ++i) {
          mbar_wait(&k_full[i % kStages], (i / kStages) & 1);
          mbar_wait(&v_full[i % kStages], (i / kStages) & 1);
        }
      }
    }
    if (warp >= kSoft + 2) {
      // ----------------------- the next items' queries, half a tile a warp
      // (each warp stands for two of the softmax warps' four arrivals).
      uint32_t i = 1;
      for (uint32_t w = blockIdx.x + gridDim.x; w < items; w += gridDim.x, ++i) {
        // The one wait that lasts an item, of up to half a million tiles: its bound
        // grows with them (a wait gives up after some 20 ms, 512 tiles take under one).
        bool ok = false;
        for (int left = item_span(a, place_item(a, w - gridDim.x)).n; !ok && left >= 0; left -= 512)
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(q_empty, (i - 1) & 1));
        if (!ok) {
          if (lane == 0) atomicOr(a.err, kErrProducerWait);
          break;
        }
        const Item it = place_item(a, w);
        load_queries<kD16, 2>(a, it, sq, 2 * (warp - kSoft - 2), lane);
        if (lane == 0) {
          mbar_arrive(q_full);
          mbar_arrive(q_full);
        }
      }
    }
    if (warp == kSoft + 1) {
      // ---------------------------------------------------------------- MMAs
      // Warp reductions and votes hand their results over in uniform registers.
      constexpr uint32_t kAll = 0xFFFFFFFFu;
      const uint32_t tm = __reduce_max_sync(kAll, tmem);
      constexpr uint32_t id_o = idesc_bf16(d16);
      const uint32_t aq = smem_addr(sq), ak = smem_addr(sk), av = smem_addr(sv);
      const uint32_t ts = tm, to = tm + kKv;
      bool ok = true;
      uint32_t g0 = 0, i = 0, done = 0;        // tiles, items, items with tiles so far
      for (uint32_t w = blockIdx.x; w < items && ok; w += gridDim.x, ++i) {
        const Item it = item_span(a, place_item(a, w));
        const int n = __reduce_max_sync(kAll, it.n), span = __reduce_max_sync(kAll, it.end - it.begin);
        auto words = [&](int j) { return min(4, (span - j * kKv + 31) >> 5); };
        if (elect_one()) {
          // S of tile j; with it its K stage has been read, and with the last one
          // the queries.
          auto scores = [&](int j) {
            const int s = (g0 + j) % kStages;
            const uint32_t kk = ak + s * img;
            const uint32_t id = idesc_bf16(0) | static_cast<uint32_t>(words(j)) << 19;    // N = 32 words
#pragma unroll
            for (int k = 0; k < d16 / 16; ++k)
              mma_ss(ts, panel_desc<kD16>(aq, k), panel_desc<kD16>(kk, k), id, k != 0);
            mma_commit(s_full);
            mma_commit(&k_empty[s]);
            if (j + 1 == n) mma_commit(q_empty);
          };
          // K steps (16 positions) first .. first + 3 of the second product.
          auto output = [&](int s, int first, int n_k, bool fresh) {
            const uint64_t v = smem_desc_sw128(av + s * img) + first * (d16 * 32) / 16;
            if (n_k >= 4) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ts(to, ts + 8 * (first + k), v + 2 * k, id_o, k != 0 || !fresh);
            } else if (n_k > 0) {
              for (int k = 0; k < n_k; ++k)
                mma_ts(to, ts + 8 * (first + k), v + 2 * k, id_o, k != 0 || !fresh);
            }
          };
          // The last item's weights have been multiplied in their order before
          // these scores take their place; its O is read by the warps that then
          // make this one's first weights.
          ok = mbar_spin(q_full, i & 1);
          if (n == 0) {
            mbar_arrive(q_empty);
          } else {
            ok = ok && mbar_spin(&k_full[g0 % kStages], (g0 / kStages) & 1);
            tmem_fence_after();
            if (ok) scores(0);
          }
          for (int j = 0; j < n && ok; ++j) {
            const uint32_t g = g0 + j, s = g % kStages;
            const int steps = 2 * words(j);
            // The loads first: they are there long before the weights.  With one
            // stage the next K follows the end of these scores' products.
            ok = mbar_spin(&v_full[s], (g / kStages) & 1);
            if (j + 1 < n) ok = ok && mbar_spin(&k_full[(g + 1) % kStages], ((g + 1) / kStages) & 1);
            ok = ok && mbar_spin(&p_half[0], g & 1);
            if (!ok) break;
            tmem_fence_after();
            output(s, 0, min(steps, 4), j == 0);
            if (!(ok = mbar_spin(&p_half[1], g & 1))) break;
            tmem_fence_after();
            output(s, 4, steps - 4, false);
            mma_commit(&v_empty[s]);
            // The next scores take the place of these weights: MMAs of one thread
            // run in the order of their issue.
            if (j + 1 < n) scores(j + 1);
          }
          if (!ok) atomicOr(a.err, kErrConsumerWait);
          // Every MMA of the item has completed before its epilogue.  (An item without
          // tiles has no MMA to wait for, and its softmax warps do not: with a phase
          // of its own, this thread could be two ahead of them.)
          if (n > 0) mma_commit(o_full);
        }
        ok = __all_sync(kAll, ok);
        g0 += n;
        done += n > 0;
      }
      // And before the columns are released.
      if (done > 0) mbar_wait(o_full, (done - 1) & 1);
    }
    __syncwarp();
  } else {
    // ----------------------------------------------------------- softmax
    regs_up<G::kSoftRegs>();
    const int row = warp * 32 + lane;
    // Not zero: a masked score, -inf, stays -inf through it.
    const float sc = fmaxf(fabsf(a.scale_log2) * kUnscale, 1e-38f);
    const uint32_t ts = tmem + (uint32_t(warp * 32) << 16);
    const uint32_t to = ts + kKv;
    bool ok = true;
    uint32_t g = 0, done = 0;                  // tiles, and items with tiles, so far
    for (uint32_t w = blockIdx.x; w < items; w += gridDim.x) {
      const Item it = item_span(a, place_item(a, w));
      const int r = it.r0 + row;
      const bool mine = r < a.rows;
      const int m = mine ? a.group.div(r) : 0, h = it.hk * a.group.d + (mine ? r - m * a.group.d : 0);
      const int limit = row_limit(a, it.len, r);
      const int tile_limit = row_limit(a, it.len, it.r0);      // the fewest of the tile
      float mx = -INFINITY, l = 0.0f;
      const uint4* mask = a.tile_mask + it.b * a.tiles + it.begin / kKv;
      const int n = it.n;
      for (int j = 0; j < n; ++j, ++g) {
        const uint4 there = __ldg(mask + j);
        ok = __all_sync(0xFFFFFFFFu, mbar_spin(s_full, g & 1));
        if (!ok) break;
        tmem_fence_after();
        const int pos0 = it.begin + j * kKv;
        const int words = min(4, (it.end - pos0 + 31) >> 5);   // that any row of the block sees
        uint32_t see[4] = {there.x, there.y, there.z, there.w};
        if (pos0 + kKv > tile_limit || (there.x & there.y & there.z & there.w) != 0xFFFFFFFFu) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int left = limit - pos0 - 32 * v;          // positions of this word the row sees
            see[v] = left >= 32 ? see[v] : left <= 0 ? 0u : see[v] & ((1u << left) - 1u);
          }
          softmax_tile<false, kD16>(ts, to, sc, mx, l, j == 0, see, words, p_half, lane);
        } else {
          softmax_tile<true, kD16>(ts, to, sc, mx, l, j == 0, see, 4, p_half, lane);
        }
      }
      if (!ok) break;
      if (n > 0) ok = __all_sync(0xFFFFFFFFu, mbar_wait(o_full, done & 1));
      done += n > 0;
      if (!ok) break;
      tmem_fence_after();
      const bool part = a.n_chunks > 1;
      const int64_t at = ((it.b * a.view.heads + it.hk) * a.n_chunks + it.chunk) * a.rows + r;
      const float inv = unscale(l);
      float* po = a.part_o + at * (32 * a.view.nb);
      uint16_t* out = a.out + it.b * a.ob + m * a.om + h * a.oh;
      // 32 channels at a time.  (Through shared memory, four lanes to a row's 64 bytes:
      // 38.8 against 37.5 us for 4096 x 300, 2 x 16 heads of 72.)
#pragma unroll 1
      for (int c = 0; c < d16; c += 32) {
        uint32_t o[2][16];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[u][e] = 0;
        if (n > 0) {
          tmem_ld16(to + c, o[0]);
          if (c + 16 < d16) tmem_ld16(to + c + 16, o[1]);
          tmem_wait_ld();
        }
        if (mine && part && l != 0.0f) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (c + 16 * u < d16)
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<uint4*>(po + c + 16 * u + e) =
                    make_uint4(o[u][e], o[u][e + 1], o[u][e + 2], o[u][e + 3]);
        }
        if (mine && !part) {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (c + 8 * x < a.D) {
              uint32_t w4[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w4[k] = bf16x2(__uint_as_float(o[x >> 1][8 * (x & 1) + 2 * k]) * inv,
                               __uint_as_float(o[x >> 1][8 * (x & 1) + 2 * k + 1]) * inv);
              *reinterpret_cast<uint4*>(out + c + 8 * x) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
            }
        }
        __syncwarp();
      }
      if (mine && part) a.part_ml[at] = make_float2(mx, l);
      if (mine && !part && a.lse)
        a.lse[(it.b * a.view.heads * a.group.d + h) * a.M + m] = row_lse(mx, l);
      // O has been read: the next item's first weights come after.
      tmem_fence_before();
    }
    if (!ok && lane == 0) atomicOr(a.err, kErrConsumerWait);
    tmem_fence_before();
  }
  __syncthreads();
  if (warp == kSoft + 1) {
    tmem_fence_after();
    tmem_dealloc(tmem, G::kTmem);
  }
}

// setmaxnreg draws on what the block was launched with: were that less than the
// warpgroups' shares, the kernel would wait for good.
template <int kD16>
bool registers_suffice() {
  using G = TcGeom<kD16>;
  static const int regs = launched_regs(attn_tc_kernel<kD16>);
  return regs * 2 >= G::kSoftRegs + G::kRestRegs;
}

template <int kD16>
int launch_tc(const AttnArgs& a, const AttnPlan& p, int64_t batch, int dev, cudaStream_t st) {
  using G = TcGeom<kD16>;
  const int rc = allow_smem<attn_tc_kernel<kD16>>(G::kSmem, dev);
  if (rc != KQ_OK) return rc;
  if (!registers_suffice<kD16>()) return record_cuda_error(cudaErrorLaunchOutOfResources);
  const int64_t items = (a.rows + kQr - 1) / kQr * p.n_chunks * a.view.heads * batch;
  if (items > (int64_t(1) << 31) - 65536) return KQ_ERR_INVALID;
  // The blocks that are resident at once take the items in turn, the next one's
  // queries and keys on their way under the last one's output.
  const int64_t grid = std::min<int64_t>(items, 2 * 148);
  const cudaError_t e = launch_pdl(attn_tc_kernel<kD16>, dim3(static_cast<unsigned>(grid)),
                                   dim3(G::kThreads), G::kSmem, st, a,
                                   static_cast<uint32_t>(items));
  return e == cudaSuccess ? KQ_OK : record_cuda_error(e);
}

}  // namespace

int launch_attention_tc(const AttnArgs& a, const AttnPlan& p, int64_t batch, int dev, cudaStream_t st) {
  const cudaError_t e = launch_pdl(
      attn_decode_kernel,
      dim3(static_cast<unsigned>(p.tiles), static_cast<unsigned>(2 * a.view.heads), static_cast<unsigned>(batch)),
      dim3(kDecodeThreads), 0, st, a, const_cast<uint4*>(a.tile_mask), const_cast<uint8_t*>(a.images));
  if (e != cudaSuccess) return record_cuda_error(e);
  switch (a.d16) {
    case 16: return launch_tc<16>(a, p, batch, dev, st);
    case 32: return launch_tc<32>(a, p, batch, dev, st);
    case 48: return launch_tc<48>(a, p, batch, dev, st);
    case 64: return launch_tc<64>(a, p, batch, dev, st);
    case 80: return launch_tc<80>(a, p, batch, dev, st);
    case 96: return launch_tc<96>(a, p, batch, dev, st);
    case 112: return launch_tc<112>(a, p, batch, dev, st);
    default: return launch_tc<128>(a, p, batch, dev, st);
  }
}

}  // namespace kq
