// Attention over the 8-bit cache for many query rows (prefill chunks, packed prompts) on tcgen05.
//
// A pair of CTAs takes up to 512 rows (a row is a query token and a head of the kv head's group) as two row tiles of 256,
// 128 of each tile's rows per CTA, and a range of keys in tiles of 128 (eight 16-key cells).  Per key tile and row tile
//   S = Q K^T (M = 256 rows, N = 128 keys, K = d),   P = 2^(z - m),   O += P V (N = d, K = 128 keys)
// as pair MMAs (cta_group::2) with S, P (fp16) and O in tensor memory.  Each CTA makes half of the shared operands: 64 keys
// of K, half of V's dimensions.  With one CTA per tile the shared memory that feeds S (M = N = 128, both operands from
// there) is the limit: 117 clocks per 128 x 128 x 16 MMA measured against 64 for the pair's 256 x 128 x 16, and every
// code is converted twice.  Roles in each CTA:
//   warps 0-3, 4-7  softmax of row tile 0 and 1: a thread owns a row (a tensor-memory lane)
//   warps 8-11      load codes into registers, a key tile ahead, and turn them into fp16 operands in shared memory; K and V,
//                   which lie alike (rows of keys), are a K-major and an MN-major operand
//   warp 12         issues the MMAs (first CTA);  warp 13 looks up block ids and scales, four key tiles at a time
//   warps 14, 15    of the second CTA pass on that its K or V is in place: a release at cluster scope takes about 1000
//                   clocks, too long for the converters
// P is written over the columns of S that it came from.  The softmax goes through a tile's scores twice in tensor memory, 32
// at a time by loops, and masks and caps are a loop too: with unrolled code the warps' different programs evict each other
// from the instruction caches (the same source took 1.17 to 1.36 ms from build to build, 1.24 ms as it is).  While one
// row tile is in its softmax the tensor cores work for the other; the chain S, softmax, P V of a row tile, about 5000 clocks
// a key tile, is what a key tile takes (the MMAs need 2048 of them, exp2 as many).  Measured on 2048 queries at 32768
// keys beside this: two warps a row 1.24 ms; 64-key tiles with two S buffers, so that S never waits, 1.32 ms with two
// warps a row and 1.36 to 1.42 ms with one (more hand-overs for each key); the row tiles taking turns at exp2 1.43 ms.
//
// Codes are exact in fp16; scales stay out of the operands as in kv8_stream.cuh: the K scale multiplies the fp32 score,
// the V scale is part of the exponent z = score + log2(v scale), and the sum of weights takes it out again.  The running
// maximum is raised (and O rescaled in tensor memory) only when a row passes it by more than 2^8.
#pragma once

#include <algorithm>
#include <cstddef>

#include "kv8_append.cuh"
#include "kv8_stream.cuh"

namespace dkv {

constexpr int kTileThreads = 512, kTileRows = 512, kTileKeys = 128, kTileCells = kTileKeys / kKv8CellKeys;
constexpr int kTileStages = 3;       // of K and of V
constexpr float kTileSlack = 8.0f;   // log2 of the most a weight may exceed 1 before the maximum is raised (fp16: 2^16)
// Key tiles looked up at a time (a lane per cell), and how many such batches are kept.
constexpr int kMetaBatch = 32 / kTileCells, kMetaBatches = 4, kMetaSlots = kMetaBatch * kMetaBatches;

struct __align__(16) TileMeta {  // of one key tile
  int64_t at[kTileCells];  // byte offset of a cell's K codes
  int key0[kTileCells];    // its first key
  float ks[kTileCells], lv[kTileCells], iv[kTileCells];  // K scale, log2 and inverse of the V scale
  int there, last, pad[2];  // cells that are mapped; the last key, INT_MAX where the cells are not mapped keys in a row
};

// Bytes of a CTA's shared memory: 256 rows of Q, its halves of K and V as fp16.  At least more than half of an SM's: a CTA takes
// all of its SM's tensor memory, and two pairs that share two SMs and each get one of them would wait for one another.
template <int D>
struct TileSmem {
  static constexpr uint32_t kQ = 128 * D * 2, kHalf = kTileKeys * D;
  static constexpr uint32_t q = 0, k = q + 2 * kQ, v = k + kTileStages * kHalf, total = v + kTileStages * kHalf;
  static constexpr size_t bytes = std::max<size_t>(1024 + total, 116 * 1024);
};

struct TileBars {
  uint64_t meta_full[kMetaBatches], meta_empty[kMetaBatches];
  uint64_t p_full[2];                                // of the pair, in the first CTA: both CTAs' warps arrive
  uint64_t k_full[kTileStages], v_full[kTileStages];    // of each CTA's converters; in the first, the second's word too
  uint64_t k_empty[kTileStages], v_empty[kTileStages], s_full[2], o_full[2], drain;  // in both: the MMAs' commits arrive
};
constexpr int kTileBars = sizeof(TileBars) / 8;

// Matrix descriptors as two words, so that stepping through an operand is one addition to the low word (address / 16; the
// leading byte offset, unused by these layouts, is 1): 8-row groups `stride` bytes apart; swizzle 2 = 128 bytes, 4 = 64.
__device__ __forceinline__ uint32_t desc_lo(uint32_t smem_addr) { return ((smem_addr >> 4) & 0x3FFFu) | 1u << 16; }
__host__ __device__ constexpr uint32_t desc_hi(uint32_t stride, uint32_t swizzle) {
  return stride >> 4 | 1u << 14 | swizzle << 29;
}
// kind::f16, D fp32, A and B fp16; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// One lane of a converged warp, always the same.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// Pair MMAs, operand descriptors by their words: D[tmem] (+)= A[smem] * B[smem], and with A in tensor memory; and the commit
// to a barrier of both CTAs.  The whole warp executes them and `on` holds for one lane: operands then are uniform registers
// from the start, where a lone thread's have to be moved there (70 to 90 clocks an MMA measured).
template <uint32_t A_HI, uint32_t B_HI, uint32_t IDESC>
__device__ __forceinline__ void umma_f16_ss_pair(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t accumulate,
                                                 uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %4};\n\tmov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %3, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %6, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(accumulate), "n"(A_HI), "n"(B_HI), "r"(IDESC), "r"(on)
      : "memory");
}
template <uint32_t B_HI, uint32_t IDESC>
__device__ __forceinline__ void umma_f16_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t accumulate,
                                                 uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %4};\n\t"
      "setp.ne.b32 p, %3, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], db, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(accumulate), "n"(B_HI), "r"(IDESC), "r"(on)
      : "memory");
}
__device__ __forceinline__ void umma_commit_both(uint32_t bar, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
      "h"(static_cast<uint16_t>(3)), "r"(on)
      : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Bits lo .. hi-1 (clamped to 0 .. 32).
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  lo = min(max(lo, 0), 32), hi = min(max(hi, 0), 32);
  const uint32_t below_hi = hi >= 32 ? ~0u : (1u << hi) - 1u, below_lo = lo >= 32 ? ~0u : (1u << lo) - 1u;
  return below_hi & ~below_lo;
}
// Keys key0 .. key0+15 that a row sees.
__device__ __forceinline__ uint32_t cell_bits(const Kv8Row& r, int prefix, int key0) {
  const uint32_t b = bit_range(r.lo - key0, r.hi + 1 - key0) | bit_range(r.first - key0, prefix - key0);
  return b & 0xffffu;
}

// 16 codes as 32 bytes of fp16, stored as the 16-byte chunks ch and ch + 1 of a row whose chunks are permuted by `swz`;
// swap: in the other order (so that eight lanes of a store cover all banks).
template <bool E4M3>
__device__ __forceinline__ void store_codes(uint8_t* row, int ch, int swz, int swap, const uint4& v) {
  const uint32_t x[4] = {flip_sign<E4M3>(v.x), flip_sign<E4M3>(v.y), flip_sign<E4M3>(v.z), flip_sign<E4M3>(v.w)};
  uint32_t y[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) y[2 * k] = codes_f16<E4M3, false>(x[k]), y[2 * k + 1] = codes_f16<E4M3, true>(x[k]);
  const uint4 lo = make_uint4(y[0], y[1], y[2], y[3]), hi = make_uint4(y[4], y[5], y[6], y[7]);
  *reinterpret_cast<uint4*>(row + (((ch + swap) ^ swz) << 4)) = swap ? hi : lo;
  *reinterpret_cast<uint4*>(row + (((ch + 1 - swap) ^ swz) << 4)) = swap ? lo : hi;
}
__device__ __forceinline__ uint4 load_codes16(const uint8_t* p) {
  uint4 w;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
               : "l"(p));
  return w;
}

// A converter warp's share of a CTA's half of a key tile, in registers: K rows 64 rank + 16 warp .. + 15, all dimensions; V
// rows 32 warp .. + 31, dimensions (d / 2) rank .. + d / 2.
template <int D>
struct TileCodes {
  static constexpr int kKLanes = D / 16, kKRows = 32 / kKLanes, kVLanes = D / 32, kVRows = 32 / kVLanes;
  uint4 k[16 / kKRows], v[32 / kVRows];

  __device__ __forceinline__ void load_k(const uint8_t* codes, const TileMeta& M, int rank, int warp, int lane) {
    const int cell = 4 * rank + warp;  // 16 rows of one cell
#pragma unroll
    for (int i = 0; i < 16 / kKRows; ++i) {
      k[i] = make_uint4(0u, 0u, 0u, 0u);
      if ((M.there >> cell) & 1)
        k[i] = load_codes16(codes + M.at[cell] + (i * kKRows + lane / kKLanes) * D + (lane % kKLanes) * 16);
    }
  }
  __device__ __forceinline__ void load_v(const uint8_t* codes, const TileMeta& M, int rank, int warp, int lane) {
#pragma unroll
    for (int i = 0; i < 32 / kVRows; ++i) {
      const int r = 32 * warp + i * kVRows + lane / kVLanes, cell = r / kKv8CellKeys;
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if ((M.there >> cell) & 1)
        v[i] = load_codes16(codes + M.at[cell] + (r % kKv8CellKeys) * D + rank * (D / 2) + (lane % kVLanes) * 16);
    }
  }
  template <bool E4M3>
  __device__ __forceinline__ void store_k(uint8_t* dst, int warp, int lane) const {  // panels of 64 rows of 128 bytes
    const int c = lane % kKLanes;
#pragma unroll
    for (int i = 0; i < 16 / kKRows; ++i) {
      const int r = 16 * warp + i * kKRows + lane / kKLanes;
      store_codes<E4M3>(dst + (c / 4) * (64 * 128) + r * 128, (c % 4) * 2, r & 7, c / 4, k[i]);
    }
  }
  // Rows of no key, from T on, are stored as 0: weight 0 times them must stay 0, and e4m3 bytes may be NaN.
  template <bool E4M3>
  __device__ __forceinline__ void store_v(uint8_t* dst, const TileMeta& M, int T, int warp, int lane) const {
    const int c = lane % kVLanes;  // rows of d / 2 fp16: 128 or 64 bytes
#pragma unroll
    for (int i = 0; i < 32 / kVRows; ++i) {
      const int r = 32 * warp + i * kVRows + lane / kVLanes;
      uint4 x = v[i];
      if (M.key0[r / kKv8CellKeys] + r % kKv8CellKeys >= T) x = make_uint4(0u, 0u, 0u, 0u);
      store_codes<E4M3>(dst + r * D, 2 * c, D == 128 ? r & 7 : (r >> 1) & 3, 0, x);
    }
  }
};

// Softmax of a CTA's 128 rows of one row tile by four warps.  BIAS: scores may be capped or biased.
template <int D, bool BIAS>
struct TileSoftmax {
  const Kv8Attn& a;
  const Kv8Seq& seq;
  const TileMeta* metas;
  TileBars* bars;
  volatile int* abort_flag;
  uint32_t s_tmem, o_tmem;  // of this warp's lanes
  uint32_t p_full;          // cluster address of the pair's barrier
  int tile;
  Kv8Row row;
  float scl, slope;  // row scale times the softmax scale (natural units); slope in log2 units
  float m, l;

  // The scores of cell `cell` (16 columns) as z, in place.  into, out_of: z = tanh(s into) out_of, or s into without a cap.
  __device__ __forceinline__ void scores(const TileMeta& M, int cell, uint32_t (&r)[16], float into, float out_of) {
    const float kk = M.ks[cell] * scl * into, lv = M.lv[cell], gap = static_cast<float>(row.pos - M.key0[cell]);
    const bool cap = BIAS && a.softcap > 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x = __uint_as_float(r[i]);
      x = cap ? fmaf(kv8_tanh(x * kk), out_of, lv) : fmaf(x, kk, lv);
      if (BIAS) x = fmaf(-slope, fabsf(gap - static_cast<float>(i)), x);
      r[i] = __float_as_uint(x);
    }
  }

  // The same without masks, for keys that stand at or before the row's position (or no distance bias), two columns to an
  // instruction.  Capped scores: by kv8_tanh_near alone, where exp2 and a reciprocal would keep the special-function unit for
  // three times as long as the softmax's own exp2 does; `most` is raised to the largest y^2, which must stay within kCapNear.
  __device__ __forceinline__ void scores_quick(const TileMeta& M, int cell, uint32_t (&r)[16], float into, float out_of,
                                               float& most) {
    const float lv = fmaf(-slope, static_cast<float>(row.pos - M.key0[cell]), M.lv[cell]);
    const bool cap = a.softcap > 0.f;
    const float kk = M.ks[cell] * scl * into;
    const uint64_t kk2 = pack2(kk, kk), out2 = pack2(out_of, out_of), lv2 = pack2(lv, lv), sl2 = pack2(slope, slope);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      uint64_t y = mul2(pack2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), kk2);
      float x0, x1;
      if (cap) {
        const uint64_t u = mul2(y, y);
        unpack2(u, x0, x1);
        most = fmaxf(fmaxf(most, x0), x1);
        uint64_t p = fma2(u, pack2(kCapP4, kCapP4), pack2(kCapP3, kCapP3));
        p = fma2(u, p, pack2(kCapP2, kCapP2));
        p = fma2(u, p, pack2(kCapP1, kCapP1));
        p = fma2(u, p, pack2(kCapP0, kCapP0));
        y = mul2(mul2(y, p), out2);
      }
      y = add2(y, fma2(sl2, pack2(static_cast<float>(i), static_cast<float>(i + 1)), lv2));
      unpack2(y, x0, x1);
      r[i] = __float_as_uint(x0), r[i + 1] = __float_as_uint(x1);
    }
  }

  // The row's scores in tensor memory as z, masked unless `whole`; returns their maximum.
  __device__ __forceinline__ float transform(const TileMeta& M, bool whole, bool behind, float into, float out_of) {
    float top = -INFINITY;
#pragma unroll 1
    for (int cell = 0; cell < kTileCells; ++cell) {
      uint32_t r[16];
      tmem_ld_32x32b_x16(s_tmem + 16 * cell, r);
      tmem_ld_wait();
      bool quick = BIAS && behind;
      if (quick) {
        float most = 0.f;
        scores_quick(M, cell, r, into, out_of, most);
        quick = __all_sync(~0u, most <= kCapNear);
        if (!quick) {
          tmem_ld_32x32b_x16(s_tmem + 16 * cell, r);
          tmem_ld_wait();
        }
      }
      if (!quick) scores(M, cell, r, into, out_of);
      if (!whole) {
        const uint32_t bits = (M.there >> cell) & 1 ? cell_bits(row, seq.prefix, M.key0[cell]) : 0u;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (!((bits >> i) & 1u)) r[i] = 0xff800000u;
      }
#pragma unroll
      for (int i = 0; i < 16; i += 2) top = fmaxf(fmaxf(top, __uint_as_float(r[i])), __uint_as_float(r[i + 1]));
      tmem_st_32x32b_x16(s_tmem + 16 * cell, r);
    }
    tmem_st_wait();
    return top;
  }

  __device__ __forceinline__ bool run(int n) {
    const float scl2 = scl * kLog2e;
    const float into = BIAS && a.softcap > 0.f ? 1.0f / a.softcap : kLog2e, out_of = a.softcap * kLog2e;
    const bool behind = BIAS && __all_sync(~0u, slope == 0.f || seq.prefix <= row.pos + 1);
    for (int j = 0; j < n; ++j) {
      bool ok = true;
      if (j % kMetaBatch == 0)
        ok = mbar_wait(smem_u32(&bars->meta_full[j / kMetaBatch % kMetaBatches]), (j / kMetaSlots) & 1, abort_flag);
      if (!__all_sync(~0u, ok && mbar_wait(smem_u32(&bars->s_full[tile]), j & 1, abort_flag))) return false;
      tc_fence_after();
      const TileMeta& M = metas[j % kMetaSlots];
      // whole: every key of the tile is seen by all of the warp's rows
      const bool whole = __all_sync(~0u, row.lo <= M.key0[0] && M.last <= row.hi);
      // raw: without a bias z is one fused multiply-add of the raw score, done again in the second pass.  m then is not
      // the exact maximum of those sums, but within a rounding of it, so scores whose rounding is not small against 1 take
      // the other path: z made cell by cell in tensor memory.
      bool raw = !BIAS && whole;
      float top = -INFINITY;
      if (raw) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(s_tmem + 32 * c, r);
          const float2 ks = reinterpret_cast<const float2*>(M.ks)[c], lv = reinterpret_cast<const float2*>(M.lv)[c];
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t* x = &r[16 * e + 4 * i];
              y[i] = fmaxf(fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1])), fmaxf(__uint_as_float(x[2]), __uint_as_float(x[3])));
            }
            top = fmaxf(top, fmaf(fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])), (e ? ks.y : ks.x) * scl2, e ? lv.y : lv.x));
          }
        }
        raw = __all_sync(~0u, fabsf(top) < 65536.0f);
      }
      if (!raw) top = transform(M, whole, behind, into, out_of);
      const bool rise = top > m + kTileSlack;
      if (__any_sync(~0u, rise)) {
        const float now = rise ? top : m, fix = fast_exp2(m - now);
        m = now;
        l *= fix;
        if (j > 0) {
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t x[16];
            tmem_ld_32x32b_x16(o_tmem + 16 * c, x);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * fix);
            tmem_st_32x32b_x16(o_tmem + 16 * c, x);
          }
        }
      }
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t r[32], p[16];
        tmem_ld_32x32b_x32(s_tmem + 32 * c, r);
        const float2 ks = reinterpret_cast<const float2*>(M.ks)[c], lv = reinterpret_cast<const float2*>(M.lv)[c];
        const float2 iv = reinterpret_cast<const float2*>(M.iv)[c];
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float kk = raw ? (e ? ks.y : ks.x) * scl2 : 1.0f, add = raw ? (e ? lv.y : lv.x) - m : -m;
          const uint64_t kk2 = pack2(kk, kk), add_2 = pack2(add, add);
          uint64_t sum2 = 0;
          float x, y;
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const uint32_t* q = &r[16 * e + i];
            unpack2(fma2(pack2(__uint_as_float(q[0]), __uint_as_float(q[1])), kk2, add_2), x, y);
            x = fast_exp2(x), y = fast_exp2(y);
            sum2 = add2(sum2, pack2(x, y));
            p[8 * e + i / 2] = pack_f16(x, y);
          }
          unpack2(sum2, x, y);
          x += y;
          if (x != 0.f) l = fmaf(x, e ? iv.y : iv.x, l);  // a cell out of sight adds nothing, even where its scale is NaN
        }
        tmem_st_32x32b_x16(s_tmem + 16 * c, p);  // over scores that this thread has read
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane_id() == 0) {
        mbar_arrive_remote(p_full);
        if (j % kMetaBatch == kMetaBatch - 1)
          mbar_arrive(smem_u32(&bars->meta_empty[j / kMetaBatch % kMetaBatches]));
      }
    }
    return true;
  }
};

template <int D, bool E4M3, bool BIAS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTileThreads, 1)
    kv8_tile_kernel(const __grid_constant__ Kv8Attn a, int row_tiles) {
  using L = TileSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) TileBars bars;
  __shared__ TileMeta metas[kMetaSlots];
  __shared__ float qscale[256];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  uint8_t* smem = align_shared<1024>(smem_raw);

  int64_t id = blockIdx.x / 2;
  const int rank = static_cast<int>(cluster_ctarank());
  const int split = static_cast<int>(id % a.nsplit);
  id /= a.nsplit;
  const int s = static_cast<int>(id % a.num_seqs);
  id /= a.num_seqs;
  const int h = static_cast<int>(id % a.heads);
  const int rt = row_tiles - 1 - static_cast<int>(id / a.heads);  // later rows see more keys: longest first
  griddep_launch_dependents();
  const Kv8Seq seq = kv8_seq(a, s);
  const int nrows = seq.nq * a.group, r0 = rt * kTileRows;
  if (!seq.ok || r0 >= nrows) return;  // the same for both CTAs
  const int r1 = min(r0 + kTileRows, nrows), hq = a.heads * a.group;
  const int tiles = r1 - r0 > 256 ? 2 : 1;
  const int i0 = r0 / a.group, i1 = (r1 - 1) / a.group;
  const int warp = warp_id(), lane = lane_id();
  // global row of this CTA's row r (0 .. 255): row tile r / 128, this CTA's half of it
  auto global_row = [&](int r) { return r0 + (r / 128) * 256 + rank * 128 + r % 128; };

  if (threadIdx.x == 0) {
    abort_flag = 0;
    const uint32_t b = smem_u32(&bars);
    constexpr int kP = 2 * kMetaBatches, kFull = kP + 2, kRest = kFull + 2 * kTileStages;
    for (int i = 0; i < kTileBars; ++i)  // meta_empty: the CTA's warps that read the scales
      mbar_init(b + 8 * i, i < kMetaBatches ? 1 : i < kP ? 4 * tiles + 4 : i < kFull ? 8 : i < kRest ? (rank == 0 ? 5 : 4) : 1);
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc_pair(smem_u32(&tmem_base), 512);
    tmem_relinquish_pair();
  }
  int first = 0;
  if (a.first_key) {
    first = INT_MAX;
    for (int i = i0 + lane; i <= i1; i += 32) first = min(first, max(a.first_key[seq.q0 + i], 0));
    first = __reduce_min_sync(~0u, first);
  }
  const Kv8Span span = kv8_span(seq, a.window, seq.T - seq.nq + i0, seq.T - seq.nq + i1, first, kKv8CellKeys);
  int v0, v1;
  kv8_split(span.count(), a.nsplit, split, v0, v1, kTileCells);
  const int n = (v1 - v0 + kTileCells - 1) / kTileCells;  // key tiles

  // Q as fp16, rows scaled by powers of two; four threads a row
#pragma unroll 2
  for (int r = threadIdx.x / 4; r < tiles * 128; r += kTileThreads / 4) {
    const int part = threadIdx.x % 4, rr = global_row(r);
    constexpr int kVecs = D / 32;  // 16-byte vectors of a thread
    uint4 w[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (rr < r1) {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + (seq.q0 + rr / a.group) * a.q_stride +
                                 (h * a.group + rr % a.group) * D + part * (D / 4);
#pragma unroll
      for (int i = 0; i < kVecs; ++i) w[i] = reinterpret_cast<const uint4*>(src)[i];
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, max((x[j] << 16) & 0x7fffffffu, x[j] & 0x7fff0000u));
    }
    const uint32_t quad = 0xfu << (lane & ~3);
    top = max(top, __shfl_xor_sync(quad, top, 1));
    top = max(top, __shfl_xor_sync(quad, top, 2));
    const int ex = min(max(static_cast<int>(top >> 23), 1), 253);
    const float down = __uint_as_float(static_cast<uint32_t>(254 - ex) << 23);
    if (part == 0)
      qscale[r] = top >= 0x7f800000u ? NAN : __uint_as_float(static_cast<uint32_t>(ex) << 23) * a.scale;
    uint8_t* dst = smem + L::q + (r / 128) * L::kQ + (r % 128) * 128;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      uint32_t y[4];
      q_pairs(w[i], down, y);
      const int c = part * kVecs + i;  // 16-byte chunk of the fp16 row
      *reinterpret_cast<uint4*>(dst + (c / 8) * (128 * 128) + (((c % 8) ^ (r & 7)) << 4)) =
          make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
  fence_proxy_async_shared();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // barriers of both CTAs initialised, both halves of Q in place, tensor memory allocated
  tc_fence_after();
  const uint32_t tmem = tmem_base;

  auto issue_mmas = [&]() {  // one warp of the first CTA; what it does between two MMAs delays all
    constexpr uint32_t kIdS = idesc_f16_f32(256, kTileKeys, false), kIdO = idesc_f16_f32(256, D, true);
    constexpr uint32_t kHiK = desc_hi(1024, 2), kHiV = desc_hi(8 * D, D == 128 ? 2 : 4);
    const uint32_t on = elect_one();
    auto same = [](uint32_t x) { return __shfl_sync(~0u, x, 0); };  // known to the compiler to be uniform
    const uint32_t sb = same(smem_u32(smem)), bar = same(smem_u32(&bars)), tm = same(tmem);
    const int num = static_cast<int>(same(n)), num_t = static_cast<int>(same(tiles));
    const uint32_t q_lo = desc_lo(sb + L::q), k_lo = desc_lo(sb + L::k), v_lo = desc_lo(sb + L::v);
    constexpr uint32_t kKFull = offsetof(TileBars, k_full), kVFull = offsetof(TileBars, v_full),
                       kKEmpty = offsetof(TileBars, k_empty), kVEmpty = offsetof(TileBars, v_empty),
                       kPFull = offsetof(TileBars, p_full), kSFull = offsetof(TileBars, s_full),
                       kOFull = offsetof(TileBars, o_full), kDrain = offsetof(TileBars, drain);
    auto wait_pair = [&](uint32_t b, uint32_t par) { return __all_sync(~0u, mbar_wait_cluster(b, par, &abort_flag)) != 0; };
    auto wait = [&](uint32_t b, uint32_t par) { return __all_sync(~0u, mbar_wait(b, par, &abort_flag)) != 0; };
    auto scores = [&](int t, int st) {
      const uint32_t qa = q_lo + t * (L::kQ / 16), ka = k_lo + st * (L::kHalf / 16);
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        umma_f16_ss_pair<kHiK, kHiK, kIdS>(tm + 128 * t, qa + ((i / 4) * (128 * 128) + (i % 4) * 32) / 16,
                                           ka + ((i / 4) * (64 * 128) + (i % 4) * 32) / 16, i > 0, on);
      umma_commit_both(bar + kSFull + 8 * t, on);
    };
    bool ok = wait_pair(bar + kKFull, 0);
    if (ok) {
      tc_fence_after();
      scores(0, 0);
      if (num_t > 1) scores(1, 0);
      umma_commit_both(bar + kKEmpty, on);
    }
    int st = 0, nx = 1 % kTileStages;     // stage of key tile j and of j + 1
    uint32_t st_par = 0, nx_par = 0, par = 0;
    for (int j = 0; ok && j < num; ++j) {
      const bool more = j + 1 < num;
      ok = wait_pair(bar + kVFull + 8 * st, st_par) && (!more || wait_pair(bar + kKFull + 8 * nx, nx_par));
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (!ok || t >= num_t) break;
        // what p_full hands over lies in tensor memory, ordered by the tcgen05 fences around the barrier
        if (!(ok = wait(bar + kPFull + 8 * t, par))) break;
        tc_fence_after();
        const uint32_t va = v_lo + st * (L::kHalf / 16);
#pragma unroll
        for (int i = 0; i < kTileKeys / 16; ++i)
          umma_f16_ts_pair<kHiV, kIdO>(tm + 256 + D * t, tm + 128 * t + 8 * i, va + i * D, i > 0 ? 1 : j, on);
        if (more) scores(t, nx);
        else umma_commit_both(bar + kOFull + 8 * t, on);
      }
      if (ok) {
        umma_commit_both(bar + kVEmpty + 8 * st, on);
        if (more) umma_commit_both(bar + kKEmpty + 8 * nx, on);
      }
      par ^= 1;
      st = nx, st_par = nx_par;
      if (++nx == kTileStages) nx = 0, nx_par ^= 1;
    }
    // whatever was issued has finished before shared and tensor memory are given up
    umma_commit_both(bar + kDrain, on);
    mbar_drain(bar + kDrain, 0);
  };
  auto look_up = [&]() {
    for (int b = 0; b * kMetaBatch < n; ++b) {
      // lane: cell lane % 8 of key tile 4 b + lane / 8; tiles go from the nearest keys to the farthest
      const int j = b * kMetaBatch + lane / kTileCells, v = v0 + (n - 1 - j) * kTileCells + lane % kTileCells;
      int key0 = INT_MAX / 2;
      int64_t at = -1;
      float2 sc = make_float2(0.f, 1.f);
      if (j < n && v < v1) {
        key0 = span.cell(v) * kKv8CellKeys;
        const int blk = kv8_block(a.block_tables, a.max_blocks, a.num_blocks, s, key0 / a.block);
        if (blk >= 0) {
          const int64_t cell = (static_cast<int64_t>(blk) * a.heads + h) * 2;
          sc = *reinterpret_cast<const float2*>(a.scales + cell);
          at = (cell * a.block + key0 % a.block) * D;
        }
      }
      const uint32_t there = __ballot_sync(~0u, at >= 0);
      if (!__all_sync(~0u, mbar_wait(smem_u32(&bars.meta_empty[b % kMetaBatches]), ((b / kMetaBatches) & 1) ^ 1,
                                     &abort_flag)))
        break;
      TileMeta& M = metas[j % kMetaSlots];
      const int c = lane % kTileCells;
      const float vs = sc.y < kLeastScale ? kLeastScale : sc.y;  // NaN stays
      M.at[c] = at, M.key0[c] = key0, M.ks[c] = sc.x, M.lv[c] = __log2f(vs), M.iv[c] = __frcp_rn(vs);
      const int next = __shfl_down_sync(~0u, key0, kTileCells - 1);  // of a tile's first lane: its last cell's first key
      if (c == 0) {
        const int mapped = (there >> (lane & ~(kTileCells - 1))) & ((1 << kTileCells) - 1);
        M.there = mapped;
        M.last = mapped == (1 << kTileCells) - 1 && next - key0 == kTileKeys - kKv8CellKeys ? key0 + kTileKeys - 1 : INT_MAX;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.meta_full[b % kMetaBatches]));
    }
  };
  auto convert = [&]() {
    TileCodes<D> x;
    const int w = warp - 8;
    const uint8_t* vcodes = a.codes + static_cast<int64_t>(a.block) * D;
    for (int j = 0; j <= n; ++j) {  // stores key tile j - 1, loads j
      if (j < n && j % kMetaBatch == 0 &&
          !__all_sync(~0u, mbar_wait(smem_u32(&bars.meta_full[j / kMetaBatch % kMetaBatches]),
                                     (j / kMetaSlots) & 1, &abort_flag)))
        break;
      const TileMeta &last = metas[(j + kMetaSlots - 1) % kMetaSlots], &next = metas[j % kMetaSlots];
      const int st = (j + kTileStages - 1) % kTileStages;
      const uint32_t free_par = (((j - 1) / kTileStages) & 1) ^ 1;
      if (j > 0) {
        if (!__all_sync(~0u, mbar_wait(smem_u32(&bars.k_empty[st]), free_par, &abort_flag))) break;
        x.template store_k<E4M3>(smem + L::k + st * L::kHalf, w, lane);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.k_full[st]));
      }
      if (j < n) x.load_k(a.codes, next, rank, w, lane);
      if (j > 0) {
        if (!__all_sync(~0u, mbar_wait(smem_u32(&bars.v_empty[st]), free_par, &abort_flag))) break;
        x.template store_v<E4M3>(smem + L::v + st * L::kHalf, last, seq.T, w, lane);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&bars.v_full[st]));
          if ((j - 1) % kMetaBatch == kMetaBatch - 1)
            mbar_arrive(smem_u32(&bars.meta_empty[(j - 1) / kMetaBatch % kMetaBatches]));
        }
      }
      if (j < n) x.load_v(vcodes, next, rank, w, lane);
    }
  };

  auto pass_on = [&](uint64_t* full) {  // one thread of the second CTA
    for (int j = 0; j < n; ++j) {
      const uint32_t bar = smem_u32(full + j % kTileStages);
      if (!mbar_wait(bar, (j / kTileStages) & 1, &abort_flag)) break;
      mbar_arrive_cluster(mapa_shared(bar, 0));
    }
  };

  if (warp < 8) {
    const int tile = warp / 4;
    if (tile < tiles) {
      const uint32_t lanes = static_cast<uint32_t>(warp % 4) << 21;  // (32 * quarter) << 16
      const int r = tile * 128 + (warp % 4) * 32 + lane, rr = min(global_row(r), r1 - 1);
      const bool mine = global_row(r) < r1;
      TileSoftmax<D, BIAS> sm{a, seq, metas, &bars, &abort_flag, (tmem + 128 * tile) | lanes,
                              (tmem + 256 + D * tile) | lanes, mapa_shared(smem_u32(&bars.p_full[tile]), 0), tile,
                              kv8_row(a, seq, rr / a.group), mine ? qscale[r] : 0.f,
                              a.slopes ? a.slopes[h * a.group + rr % a.group] * kLog2e : 0.f, kNoMax, 0.f};
      bool ok = sm.run(n);
      if (ok && n > 0) ok = __all_sync(~0u, mbar_wait(smem_u32(&bars.o_full[tile]), 0, &abort_flag));
      tc_fence_after();
      const float sum = ok ? sm.l : NAN;
      const float inv = a.nsplit > 1 ? 1.0f : (sum == 0.f ? 0.f : 1.0f / sum);
      const int64_t at = static_cast<int64_t>(seq.q0 + rr / a.group) * hq + h * a.group + rr % a.group;
      const int64_t prow = split * (a.total_q * hq) + at;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[32];
        if (n > 0) {
          tmem_ld_32x32b_x32(sm.o_tmem + 32 * c, x);
          tmem_ld_wait();
        }
        if (n == 0 || sum == 0.f)
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = 0u;
        if (mine) {
          if (a.nsplit > 1) {
            float4* dst = reinterpret_cast<float4*>(a.o + prow * D + 32 * c);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[i] = make_float4(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1]),
                                   __uint_as_float(x[4 * i + 2]), __uint_as_float(x[4 * i + 3]));
          } else {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at * D + 32 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t y[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(x[8 * i + 2 * k]) * inv,
                                                               __uint_as_float(x[8 * i + 2 * k + 1]) * inv);
                y[k] = *reinterpret_cast<const uint32_t*>(&b);
              }
              dst[i] = make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
        }
      }
      if (mine) {
        if (a.nsplit > 1) a.ml[prow] = make_float2(sm.m, sum);
        else if (a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (sm.m + log2f(sum)) * kLn2;
      }
      tc_fence_before();
    }
  } else if (warp < 12) {
    convert();
  } else {
    if (warp == 12 && rank == 0 && n > 0) issue_mmas();
    if (warp >= 14 && lane == 0 && rank == 1) pass_on(warp == 14 ? bars.k_full : bars.v_full);
    __syncwarp();
    if (warp == 13) look_up();
  }
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves while the other's MMAs, commits or arrivals may reach it
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace dkv
