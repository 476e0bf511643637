// Attention with many query rows: on the tensor cores (tcgen05, kind::f16).
//
// Every 128-row tile of queries multiplies the same keys and values, so they
// are decoded once per call, by a first kernel, into tiles of 128 positions laid
// out as the MMA reads them:
//   K image  [channel / 16][position][16 channels]   (K-major B operand of S = Q K^T)
//   V image  [position / 16][channel][16 positions]  (K-major B operand of O = P V)
// in bf16, both in 32-byte rows with the 32-byte swizzle, so a head of any
// multiple of 16 channels takes no padding beyond that, and a tile arrives as one
// plain bulk copy of 256 D bytes.
//
// The second kernel gives a CTA kQT tiles of 128 rows (query, head of the group)
// of one K/V head.  Warps 0 .. 4 kQT - 1 hold one row a thread: scores out of
// tensor memory, the running maximum and sum, weights back into it as bf16 in
// the scores' place, where the second product reads them.  One thread loads and
// one issues the MMAs; with two query tiles the products of one run under the
// softmax of the other.  The accumulator O stays in tensor memory.  It is
// rescaled only when a row's maximum has grown by more than 2^8: until then the
// weights are relative to the older maximum, which float32 and bf16 hold as
// well.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kq_attention.cuh"
#include "kq_tc.cuh"

namespace kq {
namespace {

constexpr int kKv = 128;                       // positions of a tile
constexpr int kQr = 128;                       // rows of a query tile

// K-major operand in 32-byte rows, 32-byte swizzle: 8-row atoms of 256 bytes;
// 16-byte chunk c of row r lies at c ^ (r / 4 mod 2).
__device__ __forceinline__ uint64_t smem_desc_sw32(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) |
         (uint64_t(256 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(6) << 61);
}

// ------------------------------------------------------------------ decode
constexpr int kDecodeThreads = 256;

// One tile of one K/V head of one sequence: K by blockIdx.z even, V odd.
__global__ void __launch_bounds__(kDecodeThreads) attn_decode_kernel(const AttnArgs a, uint4* masks,
                                                                     uint8_t* images) {
  pdl_wait_then_trigger();
  const int tile = blockIdx.x, hk = blockIdx.y >> 1, tid = threadIdx.x;
  const bool is_v = blockIdx.y & 1;
  const int64_t b = blockIdx.z;
  const int len = seq_len(a, b);
  const int pos0 = tile * kKv;
  if (pos0 >= len) return;
  __shared__ int64_t rows[kKv];                // cache row of each position, -1: none
  if (tid < kKv) {
    const int64_t r = pos0 + tid < len ? cache_row(a.view, b, pos0 + tid, hk) : -1;
    rows[tid] = r;
    const bool there = r >= 0;
    const uint32_t bits = __ballot_sync(0xFFFFFFFFu, there);
    if (!there && pos0 + tid < len) atomicOr(a.err, kErrCacheIndex);
    if (hk == 0 && !is_v && (tid & 31) == 0)
      reinterpret_cast<uint32_t*>(masks + b * a.tiles + tile)[tid >> 5] = bits;
  }
  __syncthreads();
  uint8_t* img = images + (((b * a.view.heads + hk) * a.tiles + tile) * 2 + is_v) * (256 * a.d16);
  const int nb = a.view.nb;
  if (!is_v) {
    // Item: 16 channels of a position.
    for (int i = tid; i < (a.d16 / 16) * kKv; i += kDecodeThreads) {
      const int p = i >> 7, t = i & 127;
      const int64_t r = rows[t];
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = 0;
      if (r >= 0) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(a.kc + r * (16 * nb)) + p);
        const uint32_t m = mx_mul(__ldg(a.ks + r * nb + (p >> 1))) * 0x10001u;
        // Channels 0..3 and 4..7 of a word come out as the pairs (k, k + 4):
        // put back in order.
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
      }
      uint8_t* dst = img + p * (kKv * 32) + t * 32;
      const int sw = (t >> 2) & 1;
      *reinterpret_cast<uint4*>(dst + 16 * sw) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(dst + 16 * (1 - sw)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
  } else {
    // Item: 8 channels of 16 positions, transposed pair by pair.
    const int words = a.d16 / 8;
    for (int i = tid; i < words * (kKv / 16); i += kDecodeThreads) {
      const int p = i / words, wd = i - p * words;
      uint32_t o[8][8];                        // [channel][pair of positions]
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t r0 = rows[16 * p + 2 * k], r1 = rows[16 * p + 2 * k + 1];
        uint32_t w0 = 0, w1 = 0, m = 0;
        if (r0 >= 0) {
          w0 = __ldg(reinterpret_cast<const uint32_t*>(a.vc + r0 * (16 * nb)) + wd);
          m = mx_mul(__ldg(a.vs + r0 * nb + (wd >> 2)));
        }
        if (r1 >= 0) {
          w1 = __ldg(reinterpret_cast<const uint32_t*>(a.vc + r1 * (16 * nb)) + wd);
          m |= mx_mul(__ldg(a.vs + r1 * nb + (wd >> 2))) << 16;
        }
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
        const int d = 8 * wd + e, sw = (d >> 2) & 1;
        uint8_t* dst = img + p * (a.d16 * 32) + d * 32;
        *reinterpret_cast<uint4*>(dst + 16 * sw) = make_uint4(o[e][0], o[e][1], o[e][2], o[e][3]);
        *reinterpret_cast<uint4*>(dst + 16 * (1 - sw)) = make_uint4(o[e][4], o[e][5], o[e][6], o[e][7]);
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
__device__ __forceinline__ uint32_t idesc_bf16(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (uint32_t(kQr >> 4) << 24);
}

template <int kQT>
struct TcGeom {
  static constexpr int kStages = kQT == 2 ? 2 : 1;
  static constexpr int kThreads = 128 * kQT + 64;
  static constexpr int kTmem = 256 * kQT;      // S (128 columns), then O (up to 128), per query tile
  // Q tiles, K and V stages, barriers.
  static constexpr int smem(int d16) { return 1024 + (kQT + 2 * kStages) * 256 * d16 + 256; }
};

template <int kQT>
__global__ void __launch_bounds__(TcGeom<kQT>::kThreads, kQT == 2 ? 1 : 2)
    attn_tc_kernel(const AttnArgs a) {
  using G = TcGeom<kQT>;
  constexpr int kStages = G::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const int d16 = a.d16, img = 256 * d16;
  uint8_t* sq = base;
  uint8_t* sk = sq + kQT * img;
  uint8_t* sv = sk + kStages * img;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(sv + kStages * img);
  uint64_t* k_empty = k_full + kStages;
  uint64_t* v_full = k_empty + kStages;
  uint64_t* v_empty = v_full + kStages;
  uint64_t* q_full = v_empty + kStages;
  uint64_t* s_full = q_full + 1;
  uint64_t* p_full = s_full + kQT;
  uint64_t* o_full = p_full + kQT;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_full + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kSoft = 4 * kQT;               // softmax warps
  const int hk = blockIdx.y;
  const int64_t b = blockIdx.z;
  // The latest rows first: in a causal call they see most.
  const int row_tiles = gridDim.x / a.n_chunks;
  const int chunk = blockIdx.x % a.n_chunks;
  const int r0 = (row_tiles - 1 - static_cast<int>(blockIdx.x) / a.n_chunks) * (kQT * kQr);

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(q_full, kSoft);
    for (int t = 0; t < kQT; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);
    }
    mbar_init(o_full, 1);
    fence_mbar_init();
  }
  if (warp == kSoft + 1) tmem_alloc(tmem_slot, G::kTmem);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait_then_trigger();

  const int len = seq_len(a, b);
  const int last_limit = row_limit(a, len, min(r0 + kQT * kQr, a.rows) - 1);
  const int begin = chunk * a.chunk;
  const int end = min(begin + a.chunk, last_limit);
  const int n = end > begin ? (end - begin + kKv - 1) / kKv : 0;
  const int tile0 = begin / kKv;

  if (warp == kSoft) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      const uint8_t* src = a.images + ((b * a.view.heads + hk) * a.tiles + tile0) * (2ll * img);
      bool ok = true;
      int j = 0;
      for (; j < n; ++j) {
        const int s = j % kStages;
        const uint32_t ph = ((j / kStages) - 1) & 1;
        if (j >= kStages && !(ok = mbar_wait(&k_empty[s], ph))) break;
        mbar_arrive_expect_tx(&k_full[s], img);
        bulk_load_1d(sk + s * img, src + 2ll * img * j, img, &k_full[s]);
        if (j >= kStages && !(ok = mbar_wait(&v_empty[s], ph))) {
          mbar_wait(&k_full[s], (j / kStages) & 1);
          break;
        }
        mbar_arrive_expect_tx(&v_full[s], img);
        bulk_load_1d(sv + s * img, src + 2ll * img * j + img, img, &v_full[s]);
      }
      if (!ok) {
        // The copies in flight land before the block ends.
        atomicOr(a.err, kErrProducerWait);
        for (int i = j > kStages ? j - kStages : 0; i < j; ++i) {
          mbar_wait(&k_full[i % kStages], (i / kStages) & 1);
          mbar_wait(&v_full[i % kStages], (i / kStages) & 1);
        }
      }
    }
    __syncwarp();
  } else if (warp == kSoft + 1) {
    // -------------------------------------------------------------- MMAs
    if (lane == 0 && n > 0) {
      const uint32_t id_s = idesc_bf16(kKv), id_o = idesc_bf16(d16);
      auto scores = [&](int t, int s) {
        for (int k = 0; k < d16 / 16; ++k)
          mma_ss(tmem + t * kKv, smem_desc_sw32(smem_addr(sq + t * img + k * (kQr * 32))),
                 smem_desc_sw32(smem_addr(sk + s * img + k * (kKv * 32))), id_s, k != 0);
        mma_commit(&s_full[t]);
      };
      bool ok = mbar_wait(q_full, 0) && mbar_wait(&k_full[0], 0);
      tmem_fence_after();
      if (ok) {
        for (int t = 0; t < kQT; ++t) scores(t, 0);
        mma_commit(&k_empty[0]);
      }
      for (int j = 0; j < n && ok; ++j) {
        const int s = j % kStages, sn = (j + 1) % kStages;
        for (int t = 0; t < kQT && ok; ++t) {
          ok = mbar_wait(&p_full[t], j & 1);
          if (ok && t == 0) ok = mbar_wait(&v_full[s], (j / kStages) & 1);
          if (!ok) break;
          tmem_fence_after();
          for (int k = 0; k < kKv / 16; ++k)
            mma_ts(tmem + kQT * kKv + t * 128, tmem + t * kKv + 8 * k,
                   smem_desc_sw32(smem_addr(sv + s * img + k * (d16 * 32))), id_o, (j | k) != 0);
          if (t == kQT - 1) mma_commit(&v_empty[s]);
          if (j + 1 < n) {
            // The next scores take the place of these weights: MMAs of one
            // thread run in the order of their issue.
            if (t == 0) ok = mbar_wait(&k_full[sn], ((j + 1) / kStages) & 1);
            if (!ok) break;
            tmem_fence_after();
            scores(t, sn);
            if (t == kQT - 1) mma_commit(&k_empty[sn]);
          }
        }
      }
      if (!ok) atomicOr(a.err, kErrConsumerWait);
      // Every MMA has completed before the epilogue, and before the columns
      // are released.
      mma_commit(o_full);
      mbar_wait(o_full, 0);
    }
    __syncwarp();
  } else {
    // ----------------------------------------------------------- softmax
    const int t = warp >> 2, row = (warp & 3) * 32 + lane;
    const int r = r0 + t * kQr + row;
    const bool mine = r < a.rows;
    const int m = mine ? a.group.div(r) : 0, h = hk * a.group.d + (mine ? r - m * a.group.d : 0);
    // Not zero: a masked score, -inf, stays -inf through it.
    const float sc = fmaxf(fabsf(a.scale_log2) * kUnscale, 1e-38f);
    {
      // The row into the swizzled Q tile; a negative scale goes into its signs.
      const uint16_t* src = a.q + b * a.qb + m * a.qm + h * a.qh;
      const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
      const int sw = (row >> 2) & 1;
      uint8_t* dst = sq + t * img + row * 32;
      for (int c = 0; c < d16 / 8; ++c) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (mine && 8 * c < a.D) x = __ldg(reinterpret_cast<const uint4*>(src) + c);
        x.x ^= flip, x.y ^= flip, x.z ^= flip, x.w ^= flip;
        *reinterpret_cast<uint4*>(dst + (c >> 1) * (kQr * 32) + 16 * ((c & 1) ^ sw)) = x;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const int limit = row_limit(a, len, r);
    const int tile_limit = row_limit(a, len, min(r0 + t * kQr, a.rows - 1));   // the fewest of the tile
    const uint32_t ts = tmem + (uint32_t((warp & 3) * 32) << 16) + t * kKv;
    const uint32_t to = tmem + (uint32_t((warp & 3) * 32) << 16) + kQT * kKv + t * 128;
    float mx = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const uint4 there = __ldg(a.tile_mask + b * a.tiles + tile0 + j);
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&s_full[t], j & 1))) {
        ok = false;
        break;
      }
      tmem_fence_after();
      uint32_t x[4][32];
#pragma unroll
      for (int v = 0; v < 4; ++v) tmem_ld32(ts + 32 * v, x[v]);
      tmem_wait_ld();
      const int pos0 = begin + j * kKv;
      if (pos0 + kKv > tile_limit || (there.x & there.y & there.z & there.w) != 0xFFFFFFFFu) {
        const uint32_t w[4] = {there.x, there.y, there.z, there.w};
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int left = limit - pos0 - 32 * v;          // positions of this word the row sees
          const uint32_t see = left >= 32 ? w[v] : left <= 0 ? 0u : w[v] & ((1u << left) - 1u);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!(see >> e & 1)) x[v][e] = 0xFF800000u;    // -inf
        }
      }
      float top[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        top[v] = fmaxf(__uint_as_float(x[v][0]), __uint_as_float(x[v][1]));
#pragma unroll
        for (int e = 2; e < 32; e += 2)
          top[v] = max3(top[v], __uint_as_float(x[v][e]), __uint_as_float(x[v][e + 1]));
      }
      const float peak = max3(top[0], top[1], fmaxf(top[2], top[3]));
      const float peak2 = peak * sc;
      if (__any_sync(0xFFFFFFFFu, peak2 > mx + 8.0f)) {
        const float m_new = fmaxf(mx, peak2);
        const float alpha = m_new == -INFINITY ? 1.0f : ex2(mx - m_new);
        mx = m_new;
        l *= alpha;
        // These scores were issued after the last weights' product, so O is
        // complete.
        if (j > 0) {
          for (int c = 0; c < d16 / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(to + 16 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st16(to + 16 * c, o);
          }
        }
      }
      const float shift = kShift - (mx == -INFINITY ? 0.0f : mx);
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float p0 = ex2(fmaf(__uint_as_float(x[v][2 * e]), sc, shift));
          const float p1 = ex2(fmaf(__uint_as_float(x[v][2 * e + 1]), sc, shift));
          sum[v] += p0 + p1;
          // Rounded to bf16, the type of the product; the sum is taken before.
          p[e] = bf16x2(p0, p1);
        }
        tmem_st16(ts + 16 * v, p);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tmem_wait_st();
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[t]);
    }
    if (ok && n > 0) ok = __all_sync(0xFFFFFFFFu, mbar_wait(o_full, 0));
    if (!ok) {
      if (lane == 0) atomicOr(a.err, kErrConsumerWait);
    } else {
      tmem_fence_after();
      const bool part = a.n_chunks > 1;
      const int64_t at = ((b * a.view.heads + hk) * a.n_chunks + chunk) * a.rows + r;
      const float inv = l > 0.0f ? kUnscale / l : 0.0f;
      uint16_t* out = a.out + b * a.ob + m * a.om + h * a.oh;
      float* po = a.part_o + at * (32 * a.view.nb);
      for (int c = 0; c < d16 / 16; ++c) {
        uint32_t o[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = 0;
        if (n > 0) {
          tmem_ld16(to + 16 * c, o);
          tmem_wait_ld();
        }
        if (!mine) continue;
        if (part) {
          if (mx != -INFINITY)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<uint4*>(po + 16 * c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          continue;
        }
#pragma unroll
        for (int e = 0; e < 16; e += 8) {
          if (16 * c + e >= a.D) continue;
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = bf16x2(__uint_as_float(o[e + 2 * k]) * inv, __uint_as_float(o[e + 2 * k + 1]) * inv);
          *reinterpret_cast<uint4*>(out + 16 * c + e) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (mine && part) a.part_ml[at] = make_float2(mx, l);
      if (mine && !part && a.lse)
        a.lse[(b * a.view.heads * a.group.d + h) * a.M + m] =
            mx == -INFINITY ? -INFINITY : (mx + (log2f(l) - kShift)) * kLn2;
    }
    tmem_fence_before();
  }
  __syncthreads();
  if (warp == kSoft + 1) {
    tmem_fence_after();
    tmem_dealloc(tmem, G::kTmem);
  }
}

template <int kQT>
int launch_tc(const AttnArgs& a, const AttnPlan& p, int64_t batch, int dev, cudaStream_t st) {
  using G = TcGeom<kQT>;
  const int rc = allow_smem<attn_tc_kernel<kQT>>(G::smem(128), dev);
  if (rc != KQ_OK) return rc;
  const int64_t row_tiles = (a.rows + kQT * kQr - 1) / (kQT * kQr);
  if (row_tiles * p.n_chunks >= (int64_t(1) << 31)) return KQ_ERR_INVALID;
  const dim3 grid(static_cast<unsigned>(row_tiles * p.n_chunks), static_cast<unsigned>(a.view.heads),
                  static_cast<unsigned>(batch));
  const cudaError_t e = launch_pdl(attn_tc_kernel<kQT>, grid, dim3(G::kThreads), G::smem(a.d16), st, a);
  return e == cudaSuccess ? KQ_OK : record_cuda_error(e);
}

}  // namespace

int launch_attention_tc(const AttnArgs& a, const AttnPlan& p, int64_t batch, int dev, cudaStream_t st) {
  if (2 * a.view.heads > 65535) return KQ_ERR_INVALID;
  const cudaError_t e = launch_pdl(
      attn_decode_kernel,
      dim3(static_cast<unsigned>(p.tiles), static_cast<unsigned>(2 * a.view.heads), static_cast<unsigned>(batch)),
      dim3(kDecodeThreads), 0, st, a, const_cast<uint4*>(a.tile_mask), const_cast<uint8_t*>(a.images));
  if (e != cudaSuccess) return record_cuda_error(e);
  return p.q_tiles == 2 ? launch_tc<2>(a, p, batch, dev, st) : launch_tc<1>(a, p, batch, dev, st);
}

}  // namespace kq
