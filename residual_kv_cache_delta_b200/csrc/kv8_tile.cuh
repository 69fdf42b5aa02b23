// Attention over the 8-bit cache for many query rows (prefill chunks, packed prompts) on tcgen05.
//
// A CTA takes up to 256 rows (a row is a query token and a head of the kv head's group) as two tiles of 128, and a range
// of keys in tiles of 128 (eight 16-key cells).  Per key tile and row tile
//   S = Q K^T (M = 128 rows, N = 128 keys, K = d),   P = 2^(z - m),   O += P V (N = d, K = 128 keys),
// S and O in tensor memory, P written over S as fp16 and read by the second MMA from there.  Roles:
//   warps 0-3, 4-7  softmax of row tile 0 and 1: a thread owns a row (a tensor-memory lane)
//   warps 8-11      turn codes into fp16 operands in shared memory; K and V, which lie alike (keys by 64-dimension
//                   panels of 128 bytes, 128-byte swizzle), are a K-major and an MN-major operand
//   warp 12         issues the MMAs;  warp 13 loads codes (tensor-map boxes of 16 rows), scales and block ids
// While one row tile is in its softmax the tensor cores work for the other.
//
// Codes are exact in fp16; scales stay out of the operands as in kv8_stream.cuh: the K scale multiplies the fp32 score,
// the V scale is part of the exponent z = score + log2(v scale), and the sum of weights takes it out again.  The running
// maximum is raised (and O rescaled in tensor memory) only when a row passes it by more than 2^4.
#pragma once

#include "kv8_stream.cuh"

namespace dkv {

constexpr int kTileThreads = 448, kTileRows = 256, kTileKeys = 128, kTileCells = kTileKeys / kKv8CellKeys;
constexpr int kMetaSlots = 4;

struct TileMeta {  // of one key tile: per cell the first key, K scale, log2 and inverse of the V scale; mapped cells
  int key0[kTileCells];
  float ks[kTileCells], lv[kTileCells], iv[kTileCells];
  int there, pad[3];
};

// Bytes of shared memory: Q, two stages of fp16 K and V, one stage of codes.
template <int D>
struct TileSmem {
  static constexpr uint32_t kOperand = kTileKeys * D * 2;  // an fp16 operand of 128 rows
  static constexpr uint32_t kRaw = kTileKeys * D;          // 128 rows of codes
  static constexpr uint32_t q = 0, k = q + 2 * kOperand, v = k + 2 * kOperand, rk = v + 2 * kOperand, rv = rk + kRaw;
  static constexpr uint32_t total = rv + kRaw;
  static constexpr size_t bytes = 1024 + total;
};

struct TileBars {
  uint64_t rk_full, rk_empty, rv_full, rv_empty;
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2], drain;
};

// Matrix descriptor of an MN-major operand in 64-element panels of 128-byte rows with the 128-byte swizzle: 8-row groups
// 1024 bytes apart (stride), panels `panel` bytes apart (leading).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr, uint32_t panel) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(panel >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
// kind::f16, D fp32, A and B fp16; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// D[tmem] (+)= A[tmem] * B[smem].
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
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
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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

template <int D, bool E4M3>
__device__ __forceinline__ void convert_tile(const uint8_t* raw, uint8_t* dst, const TileMeta* zero_from, int T) {
  const int tid = threadIdx.x - 256;  // 128 threads: a thread per row
  constexpr int kChunks = D / 16;
  const int r = tid;
  bool clear = false;
  if (zero_from) {  // V rows of no key: weight 0 times them must stay 0, and e4m3 bytes may be NaN
    const int c = r / kKv8CellKeys;
    clear = !((zero_from->there >> c) & 1) || zero_from->key0[c] + r % kKv8CellKeys >= T;
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    uint4 w = *reinterpret_cast<const uint4*>(raw + stream_chunk<D>(r, c));
    if (clear) w = make_uint4(0u, 0u, 0u, 0u);
    const uint32_t x[4] = {flip_sign<E4M3>(w.x), flip_sign<E4M3>(w.y), flip_sign<E4M3>(w.z), flip_sign<E4M3>(w.w)};
    uint32_t y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[2 * i] = codes_f16<E4M3, false>(x[i]), y[2 * i + 1] = codes_f16<E4M3, true>(x[i]);
    uint8_t* p = dst + (c / 4) * (kTileKeys * 128) + r * 128;
    const int ch = (c % 4) * 2;
    *reinterpret_cast<uint4*>(p + ((ch ^ (r & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
    *reinterpret_cast<uint4*>(p + (((ch + 1) ^ (r & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
  }
}

// Softmax of one row tile by its four warps.  BIAS: scores may be capped or biased.
template <int D, bool BIAS>
struct TileSoftmax {
  const Kv8Attn& a;
  const Kv8Seq& seq;
  const TileMeta* metas;
  TileBars* bars;
  volatile int* abort_flag;
  uint32_t s_tmem, o_tmem;  // of this warp's lanes
  int tile;
  Kv8Row row;
  float scl, slope;  // row scale times the softmax scale (natural units); slope in log2 units
  float m, l, two_over_cap;

  // The scores of 32 columns (cells 2c, 2c + 1) as z; returns their maximum.
  __device__ __forceinline__ float scores(const TileMeta& M, int c, uint32_t (&r)[32]) {
    float top = -INFINITY;
#pragma unroll
    for (int gq = 0; gq < 2; ++gq) {
      const int cell = 2 * c + gq, key0 = M.key0[cell];
      const float kk = M.ks[cell] * scl, lv = M.lv[cell];
      uint32_t bits = cell_bits(row, seq.prefix, key0);
      if (!((M.there >> cell) & 1)) bits = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float x = __uint_as_float(r[gq * 16 + i]) * kk;
        if (BIAS && a.softcap > 0.f) x = kv8_cap(x, a.softcap, two_over_cap);
        x = fmaf(x, kLog2e, lv);
        if (BIAS) x -= slope * static_cast<float>(abs(row.pos - key0 - i));
        if (!((bits >> i) & 1u)) x = -INFINITY;
        r[gq * 16 + i] = __float_as_uint(x);
        top = fmaxf(top, x);
      }
    }
    return top;
  }

  __device__ __forceinline__ bool run(int n) {
    for (int j = 0; j < n; ++j) {
      if (!__all_sync(~0u, mbar_wait(smem_u32(&bars->s_full[tile]), j & 1, abort_flag))) return false;
      tc_fence_after();
      const TileMeta& M = metas[j % kMetaSlots];
      const int k0 = M.key0[0], k1 = M.key0[kTileCells - 1] + kKv8CellKeys - 1;
      // quick: every key of the tile is seen by all of the warp's rows and z is one fused multiply-add of the raw score,
      // done again in the second pass.  m then is not the exact maximum of those sums, but within a rounding of
      // it, so scores whose rounding is not small against 1 take the other path.
      bool quick = !BIAS && __all_sync(~0u, M.there == (1 << kTileCells) - 1 && k1 - k0 == kTileKeys - 1 &&
                                                      row.lo <= k0 && k1 <= row.hi);
      float top = -INFINITY;
      uint32_t r[32];
      if (quick) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_ld_32x32b_x32(s_tmem + 32 * c, r);
          tmem_ld_wait();
#pragma unroll
          for (int gq = 0; gq < 2; ++gq) {
            float x = __uint_as_float(r[16 * gq]);
#pragma unroll
            for (int i = 1; i < 16; ++i) x = fmaxf(x, __uint_as_float(r[16 * gq + i]));
            top = fmaxf(top, fmaf(x, M.ks[2 * c + gq] * scl * kLog2e, M.lv[2 * c + gq]));
          }
        }
        quick = __all_sync(~0u, fabsf(top) < 65536.0f);
      }
      if (!quick) {
        top = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_ld_32x32b_x32(s_tmem + 32 * c, r);
          tmem_ld_wait();
          top = fmaxf(top, scores(M, c, r));
          tmem_st_32x32b_x32(s_tmem + 32 * c, r);  // z in place of the raw score
        }
        tmem_st_wait();
      }
      const bool rise = top > m + kMaxSlack;
      if (__any_sync(~0u, rise)) {
        const float now = rise ? top : m, fix = fast_exp2(m - now);
        m = now;
        l *= fix;
        if (j > 0) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            tmem_ld_32x32b_x32(o_tmem + 32 * c, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * fix);
            tmem_st_32x32b_x32(o_tmem + 32 * c, r);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t p[16];
        tmem_ld_32x32b_x32(s_tmem + 32 * c, r);
        tmem_ld_wait();
#pragma unroll
        for (int gq = 0; gq < 2; ++gq) {
          const int cell = 2 * c + gq;
          const float kk = quick ? M.ks[cell] * scl * kLog2e : 1.0f, add = quick ? M.lv[cell] - m : -m;
          const float iv = M.iv[cell];
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float x = fast_exp2(fmaf(__uint_as_float(r[gq * 16 + i]), kk, add));
            const float y = fast_exp2(fmaf(__uint_as_float(r[gq * 16 + i + 1]), kk, add));
            sum += x + y;
            p[gq * 8 + i / 2] = pack_f16(x, y);
          }
          if (sum != 0.f) l = fmaf(sum, iv, l);  // a cell out of sight adds nothing, even where its scale is NaN
        }
        tmem_st_32x32b_x16(s_tmem + 16 * c, p);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane_id() == 0) mbar_arrive(smem_u32(&bars->p_full[tile]));
    }
    return true;
  }
};

template <int D, bool E4M3, bool BIAS>
__global__ void __launch_bounds__(kTileThreads, 1)
    kv8_tile_kernel(const __grid_constant__ CUtensorMap map, const Kv8Attn a, int row_tiles) {
  using L = TileSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) TileBars bars;
  __shared__ TileMeta metas[kMetaSlots];
  __shared__ float qscale[kTileRows];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  uint8_t* smem = align_shared<1024>(smem_raw);

  int64_t id = blockIdx.x;
  const int split = static_cast<int>(id % a.nsplit);
  id /= a.nsplit;
  const int s = static_cast<int>(id % a.num_seqs);
  id /= a.num_seqs;
  const int h = static_cast<int>(id % a.heads);
  const int rt = row_tiles - 1 - static_cast<int>(id / a.heads);  // later rows see more keys: longest first
  griddep_launch_dependents();
  const Kv8Seq seq = kv8_seq(a, s);
  const int nrows = seq.nq * a.group, r0 = rt * kTileRows;
  if (!seq.ok || r0 >= nrows) return;
  const int r1 = min(r0 + kTileRows, nrows), hq = a.heads * a.group;
  const int tiles = r1 - r0 > 128 ? 2 : 1;
  const int i0 = r0 / a.group, i1 = (r1 - 1) / a.group;
  const int warp = warp_id(), lane = lane_id();

  if (threadIdx.x == 0) {
    abort_flag = 0;
    const uint32_t b = smem_u32(&bars);
    constexpr int kCounts[] = {1, 4, 1, 4, 4, 4, 1, 1, 4, 4, 1, 1, 1, 1, 4, 4, 1, 1, 1};
    static_assert(sizeof(TileBars) == sizeof(kCounts) / 4 * 8, "one count per barrier");
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(TileBars) / 8); ++i) mbar_init(b + 8 * i, kCounts[i]);
    fence_barrier_init();
    prefetch_tensormap(&map);
  }
  if (warp == 12) {
    tmem_alloc(smem_u32(&tmem_base), 512);
    tmem_relinquish();
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
  for (int r = threadIdx.x / 4; r < tiles * 128; r += kTileThreads / 4) {
    const int part = threadIdx.x % 4;
    constexpr int kVecs = D / 32;  // 16-byte vectors of a thread
    uint4 w[kVecs] = {};
    if (r0 + r < r1) {
      const int rr = r0 + r;
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
    uint8_t* dst = smem + L::q + (r / 128) * L::kOperand + (r % 128) * 128;
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
  tc_fence_after();
  const uint32_t tmem = tmem_base;

  if (warp < 8) {
    const int tile = warp / 4;
    if (tile < tiles) {
      const uint32_t lanes = static_cast<uint32_t>(warp % 4) << 21;  // (32 * quarter) << 16
      const int r = tile * 128 + (warp % 4) * 32 + lane, rr = min(r0 + r, r1 - 1);
      TileSoftmax<D, BIAS> sm{a, seq, metas, &bars, &abort_flag, (tmem + 128 * tile) | lanes,
                              (tmem + 256 + D * tile) | lanes, tile, kv8_row(a, seq, rr / a.group),
                              qscale[min(r, r1 - 1 - r0)],
                              a.slopes ? a.slopes[h * a.group + rr % a.group] * kLog2e : 0.f, kNoMax, 0.f,
                              BIAS && a.softcap > 0.f ? 2.0f * kLog2e / a.softcap : 0.f};
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
        if (r0 + r < r1) {
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
      if (r0 + r < r1) {
        if (a.nsplit > 1) a.ml[prow] = make_float2(sm.m, sum);
        else if (a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (sm.m + log2f(sum)) * kLn2;
      }
      tc_fence_before();
    }
  } else if (warp < 12) {
    for (int j = 0; j < n; ++j) {
      const int st = j & 1;
      const uint32_t free_par = ((j >> 1) & 1) ^ 1;
      bool ok = mbar_wait(smem_u32(&bars.rk_full), j & 1, &abort_flag) &&
                mbar_wait(smem_u32(&bars.k_empty[st]), free_par, &abort_flag);
      if (!__all_sync(~0u, ok)) break;
      convert_tile<D, E4M3>(smem + L::rk, smem + L::k + st * L::kOperand, nullptr, 0);
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&bars.rk_empty));
        mbar_arrive(smem_u32(&bars.k_full[st]));
      }
      ok = mbar_wait(smem_u32(&bars.rv_full), j & 1, &abort_flag) &&
           mbar_wait(smem_u32(&bars.v_empty[st]), free_par, &abort_flag);
      if (!__all_sync(~0u, ok)) break;
      convert_tile<D, E4M3>(smem + L::rv, smem + L::v + st * L::kOperand, &metas[j % kMetaSlots], seq.T);
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&bars.rv_empty));
        mbar_arrive(smem_u32(&bars.v_full[st]));
      }
    }
  } else if (warp == 12) {
    if (lane == 0 && n > 0) {
      constexpr uint32_t kIdS = idesc_f16_f32(128, kTileKeys, false), kIdO = idesc_f16_f32(128, D, true);
      const uint32_t sb = smem_u32(smem);
      auto scores = [&](int tile, int j) {
        const uint32_t qa = sb + L::q + tile * L::kOperand, ka = sb + L::k + (j & 1) * L::kOperand;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t off = (i / 4) * (128 * 128) + (i % 4) * 32;
          umma_bf16(tmem + 128 * tile, sw128_kmajor_desc(qa + off), sw128_kmajor_desc(ka + off), kIdS, i > 0);
        }
        umma_commit(smem_u32(&bars.s_full[tile]));
      };
      bool ok = mbar_wait(smem_u32(&bars.k_full[0]), 0, &abort_flag);
      if (ok) {
        tc_fence_after();
        for (int t = 0; t < tiles; ++t) scores(t, 0);
        umma_commit(smem_u32(&bars.k_empty[0]));
      }
      for (int j = 0; ok && j < n; ++j) {
        const int st = j & 1;
        for (int t = 0; ok && t < tiles; ++t) {
          ok = mbar_wait(smem_u32(&bars.p_full[t]), j & 1, &abort_flag) &&
               mbar_wait(smem_u32(&bars.v_full[st]), (j >> 1) & 1, &abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t va = sb + L::v + st * L::kOperand;
#pragma unroll
          for (int i = 0; i < kTileKeys / 16; ++i)
            umma_f16_ts(tmem + 256 + D * t, tmem + 128 * t + 8 * i, sw128_mnmajor_desc(va + i * 2048, 128 * 128), kIdO,
                        j > 0 || i > 0);
          if (j + 1 < n) {
            ok = mbar_wait(smem_u32(&bars.k_full[st ^ 1]), ((j + 1) >> 1) & 1, &abort_flag);
            if (!ok) break;
            tc_fence_after();
            scores(t, j + 1);
          } else {
            umma_commit(smem_u32(&bars.o_full[t]));
          }
        }
        if (ok) {
          umma_commit(smem_u32(&bars.v_empty[st]));
          if (j + 1 < n) umma_commit(smem_u32(&bars.k_empty[st ^ 1]));
        }
      }
      // whatever was issued has finished before shared and tensor memory are given up
      umma_commit(smem_u32(&bars.drain));
      mbar_drain(smem_u32(&bars.drain), 0);
    }
    __syncwarp();
  } else {
    int sent_k = 0, sent_v = 0;
    for (int j = 0; j < n; ++j) {
      // lanes 0-7: the tile's cells
      const int v = v0 + (n - 1 - j) * kTileCells + lane;  // from the nearest keys to the farthest
      int key0 = INT_MAX / 2, row = -1;
      float2 sc = make_float2(0.f, 1.f);
      if (lane < kTileCells && v < v1) {
        key0 = span.cell(v) * kKv8CellKeys;
        const int blk = kv8_block(a.block_tables, a.max_blocks, a.num_blocks, s, key0 / a.block);
        if (blk >= 0) {
          const int cell = (blk * a.heads + h) * 2;
          sc = *reinterpret_cast<const float2*>(a.scales + cell);
          row = cell * a.block + key0 % a.block;
        }
      }
      const uint32_t there = __ballot_sync(~0u, row >= 0);
      if (!__all_sync(~0u, mbar_wait(smem_u32(&bars.rk_empty), (j & 1) ^ 1, &abort_flag))) break;
      TileMeta& M = metas[j % kMetaSlots];
      if (lane < kTileCells) {
        const float vs = sc.y < kLeastScale ? kLeastScale : sc.y;  // NaN stays
        M.key0[lane] = key0, M.ks[lane] = sc.x, M.lv[lane] = __log2f(vs), M.iv[lane] = __frcp_rn(vs);
        if (lane == 0) M.there = static_cast<int>(there);
      }
      __syncwarp();
      const uint32_t bytes = __popc(there) * kKv8CellKeys * D;
      if (lane == 0) mbar_arrive_expect_tx(smem_u32(&bars.rk_full), bytes);
      __syncwarp();
      if (row >= 0)
        tma_load_2d(smem_u32(smem) + L::rk + lane * (kKv8CellKeys * D), &map, 0, row, smem_u32(&bars.rk_full));
      ++sent_k;
      if (!__all_sync(~0u, mbar_wait(smem_u32(&bars.rv_empty), (j & 1) ^ 1, &abort_flag))) break;
      if (lane == 0) mbar_arrive_expect_tx(smem_u32(&bars.rv_full), bytes);
      __syncwarp();
      if (row >= 0)
        tma_load_2d(smem_u32(smem) + L::rv + lane * (kKv8CellKeys * D), &map, 0, row + a.block, smem_u32(&bars.rv_full));
      ++sent_v;
    }
    // every copy has landed before the CTA leaves (at once, unless another role gave up)
    if (lane == 0) {
      if (sent_k) mbar_drain(smem_u32(&bars.rk_full), (sent_k - 1) & 1);
      if (sent_v) mbar_drain(smem_u32(&bars.rv_full), (sent_v - 1) & 1);
    }
  }
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace dkv
