// Attention over the 8-bit cache for few query rows (one or a few tokens per sequence): the cache streams through
// registers once and both products run on mma.sync m16n8k16 (fp16 operands, fp32 accumulation).
//
// A row is a query token and a head of the kv head's group; a CTA takes 8 NT rows and a range of keys, its warps take
// the range's 16-key cells in turn.  Bound by memory at 8 rows: 8 x 32768 tokens, 8 kv heads, d = 128 take 96 us (5.6 TB/s,
// 86% of the measured copy rate; issue slots 58% busy).  More than 16 rows are several CTAs, each of which reads, converts and
// multiplies the whole cache again: 17 to 80 rows take time in proportion (32 and 64 rows there: 282 and 510 us), and what
// bounds them is the latency of the 8 warps that an SM holds (32 rows: issue slots 41% busy, tensor pipe 22%, DRAM 24%).
// Each warp has its own ring of cells in shared memory (two tensor-map boxes of 16 rows, K and V) and waits for nobody else,
// so there is no CTA barrier until the warps' results are joined.
//
//   scores   S[16 keys][8 rows] = K q^T: the keys are the MMA's 16 rows, the query rows its 8 columns, so that no
//            part of the MMA is padding for 8 rows.  A lane reads 16 or 32 bytes of two keys; the dimensions are
//            contracted in the order in which they lie in a lane's words, and q's fragments follow that order.
//   output   O^T[d][8 rows] += V^T P: V bytes of two neighbouring MMA keys are interleaved into operand pairs in
//            registers (a lane reads 16 or 8 dimensions of four keys), P's accumulators become its operand by
//            movmatrix.
// int8 and e4m3 codes are exact in fp16.  q (bf16) is scaled per row by a power of two into [1, 4), which is exact down
// to 2^-24 of the row's largest value.  The cell's K scale multiplies the fp32 score.  Its V scale goes into the
// exponent: with z = score + log2(v scale), the weights 2^(z - max z) are what multiplies V's codes, at most 2^4 and so
// in fp16's range with 11 bits whatever the scales are, and the softmax sum adds 2^(z - max z) / (v scale) in fp32.
// The running maximum is raised only when a score passes it by more than 2^4 (a warp vote per cell).  exp2 and log2 are the
// hardware's (2^-21 of the weight).
//
// Key order inside a cell: MMA row g stands for key kPerm[g] (and 8 + kPerm[g]), chosen so that with the tensor map's
// swizzle neither the K reads (16 bytes, lanes of two keys) nor the V reads (lanes of four keys) conflict on banks.
#pragma once

// deltakv.cu includes this after compress.cuh (get_encode_fn) and decode.cuh (fast_exp2).
#include "kv8_common.cuh"
#include "launch.h"

namespace dkv {

constexpr int kStreamWarps = 8;
constexpr float kLeastScale = 8.271806125530277e-25f;  // 2^-80, below any scale that an append writes
constexpr float kMaxSlack = 4.0f;  // log2 of the most a weight may exceed 1 before the maximum is raised

// CTAs of an SM: two, unless 16 rows of 128 dimensions take the registers of both.  (64 dimensions, 16 rows: one CTA with
// twice the stages left the warps' latencies in sight, 24.8 us for 8 sequences of 5 tokens.)
template <int D>
__host__ __device__ constexpr int stream_ctas(int nt) { return D == 128 && nt > 1 ? 1 : 2; }
template <int D>
__host__ __device__ constexpr int stream_stages(int nt) { return (D == 128 ? 6 : 12) / stream_ctas<D>(nt); }
template <int D>
constexpr size_t stream_smem(int nt) {
  return 1024 + static_cast<size_t>(kStreamWarps) * stream_stages<D>(nt) * 32 * D;
}

// Key of MMA row g: [0 4 2 6 5 1 7 3] under the 128-byte swizzle (rows of 128 bytes), [0 1 3 2 4 5 7 6] under the
// 64-byte one.
template <int D>
__device__ __forceinline__ int stream_perm(int g) {
  return static_cast<int>((D == 128 ? 0x37156240u : 0x67542310u) >> (4 * g)) & 15;
}
// Shared-memory offset of 16-byte chunk c of row r of a box.
template <int D>
__device__ __forceinline__ uint32_t stream_chunk(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two codes (bytes 0 and 1 of the lower or upper half of w) as a pair of fp16.  int8 codes come with their sign bit
// flipped: 0x64xx is 1024 + xx, and 1024 + 128 is taken off.
template <bool E4M3, bool HI>
__device__ __forceinline__ uint32_t codes_f16(uint32_t w) {
  uint32_t r;
  if constexpr (E4M3) {
    const uint16_t h = static_cast<uint16_t>(HI ? w >> 16 : w);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
  } else {
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(w), "r"(0x64646464u), "n"(HI ? 0x4342 : 0x4140));
    asm("sub.f16x2 %0, %0, %1;" : "+r"(r) : "r"(0x64806480u));
  }
  return r;
}
template <bool E4M3>
__device__ __forceinline__ uint32_t flip_sign(uint32_t w) { return E4M3 ? w : w ^ 0x80808080u; }

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  return __byte_perm(a, b, sel);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// fp16 fragment pairs of a query row from 4 consecutive bf16 values times f.
__device__ __forceinline__ void q_pairs(const uint4& w, float f, uint32_t* out) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    out[i] = pack_f16(__uint_as_float(x[i] << 16) * f, __uint_as_float(x[i] & 0xffff0000u) * f);
}

// BIAS: scores may be capped or biased by distance.
template <int D, bool E4M3, int NT, bool BIAS>
__global__ void __launch_bounds__(kStreamWarps * 32, stream_ctas<D>(NT))
    kv8_stream_kernel(const __grid_constant__ CUtensorMap map, const Kv8Attn a, int row_tiles) {
  constexpr int kSteps = D / 16, kStg = stream_stages<D>(NT), kRows = 8 * NT;
  constexpr uint32_t kCellBytes = 32 * D;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kStreamWarps * kStg];
  __shared__ int abort_flag;
  __shared__ float sml[kStreamWarps][kRows][2];
  uint8_t* smem = align_shared<1024>(smem_raw);

  int64_t id = blockIdx.x;
  const int split = static_cast<int>(id % a.nsplit);
  id /= a.nsplit;
  const int tile = static_cast<int>(id % row_tiles);
  id /= row_tiles;
  const int h = static_cast<int>(id % a.heads), s = static_cast<int>(id / a.heads);
  const int warp = warp_id(), lane = lane_id(), g = lane >> 2, t = lane & 3;
  griddep_launch_dependents();
  const Kv8Seq seq = kv8_seq(a, s);
  const int nrows = seq.nq * a.group, r0 = tile * kRows;
  if (!seq.ok || r0 >= nrows) return;
  const int r1 = min(r0 + kRows, nrows), hq = a.heads * a.group;
  const int i0 = r0 / a.group, i1 = (r1 - 1) / a.group;
  int first = a.first_key ? INT_MAX : 0;
  if (a.first_key)
    for (int i = i0; i <= i1; ++i) first = min(first, max(a.first_key[seq.q0 + i], 0));
  const Kv8Span span = kv8_span(seq, a.window, seq.T - seq.nq + i0, seq.T - seq.nq + i1, first, kKv8CellKeys);
  int v0, v1;
  kv8_split(span.count(), a.nsplit, split, v0, v1);

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < kStreamWarps * kStg; ++i) mbar_init(smem_u32(&bars[i]), 1);
    fence_barrier_init();
    prefetch_tensormap(&map);
  }
  __syncthreads();

  // q rows of the columns, on their way while the first block ids are
  uint4 qw[NT][D / 32];
#pragma unroll
  for (int c = 0; c < NT; ++c) {
    const int r = r0 + c * 8 + g;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) qw[c][i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < r1) {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) +
                                 (seq.q0 + r / a.group) * a.q_stride + (h * a.group + r % a.group) * D;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        qw[c][2 * i] = *reinterpret_cast<const uint4*>(src + 64 * i + 16 * t);
        qw[c][2 * i + 1] = *reinterpret_cast<const uint4*>(src + 64 * i + 16 * t + 8);
      }
    }
  }

  // This warp's j-th cell is v1 - 1 - warp - W j: from the nearest keys to the farthest, so that a distance bias does not
  // raise the running maximum at every cell
  const int n = v1 - v0 > warp ? (v1 - v0 - warp + kStreamWarps - 1) / kStreamWarps : 0;
  const uint32_t ring = smem_u32(smem) + warp * kStg * kCellBytes;
  const uint32_t bar0 = smem_u32(&bars[warp * kStg]);
  // lane i holds cell (batch * 32 + i): first row of its K codes in the tensor map (-1: no such block), its K scale, and
  // log2 and inverse of its V scale
  int krow[2] = {-1, -1};
  float ksc[2] = {0.f, 0.f}, vlog[2] = {0.f, 0.f}, vinv[2] = {1.f, 1.f};
  auto first_key = [&](int j) { return span.cell(v1 - 1 - warp - j * kStreamWarps) * kKv8CellKeys; };
  auto load_row = [&](int j) {
    if (j >= n) return -1;
    const int key = first_key(j), blk = kv8_block(a.block_tables, a.max_blocks, a.num_blocks, s, key / a.block);
    return blk < 0 ? -1 : (blk * a.heads + h) * 2 * a.block + key % a.block;
  };
  auto load_scales = [&](int row, float& ks, float& lv, float& iv) {
    float2 sc = make_float2(0.f, 1.f);
    if (row >= 0) sc = *reinterpret_cast<const float2*>(a.scales + row / (2 * a.block) * 2);
    const float vs = sc.y < kLeastScale ? kLeastScale : sc.y;  // a zero scale has no logarithm; NaN stays
    ks = BIAS ? sc.x : sc.x * kLog2e, lv = __log2f(vs), iv = __frcp_rn(vs);
  };
  auto issue = [&](int j, int row) {  // lane 0
    const uint32_t bar = bar0 + (j % kStg) * 8, dst = ring + (j % kStg) * kCellBytes;
    if (row < 0) {
      mbar_arrive(bar);
      return;
    }
    mbar_arrive_expect_tx(bar, kCellBytes);
    tma_load_2d(dst, &map, 0, row, bar);
    tma_load_2d(dst + kCellBytes / 2, &map, 0, row + a.block, bar);
  };
  krow[0] = load_row(lane);
#pragma unroll
  for (int j = 0; j < kStg; ++j) {
    const int row = __shfl_sync(~0u, krow[0], j);
    if (lane == 0 && j < n) issue(j, row);
  }
  load_scales(krow[0], ksc[0], vlog[0], vinv[0]);

  // q fragments and the columns' parameters
  uint32_t qf[NT][2 * kSteps];
  float scl[NT][2], slope[NT][2];
  Kv8Row row[NT][2];
#pragma unroll
  for (int c = 0; c < NT; ++c) {
    const uint4(&w)[D / 32] = qw[c];
    uint32_t top = 0;  // largest magnitude of the row, as bits
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, max((x[j] << 16) & 0x7fffffffu, x[j] & 0x7fff0000u));
    }
    top = max(top, __shfl_xor_sync(~0u, top, 1));
    top = max(top, __shfl_xor_sync(~0u, top, 2));
    const int ex = min(max(static_cast<int>(top >> 23), 1), 253);
    const float down = __uint_as_float(static_cast<uint32_t>(254 - ex) << 23);
    float up = __uint_as_float(static_cast<uint32_t>(ex) << 23) * a.scale;
    if (top >= 0x7f800000u) up = NAN;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) q_pairs(w[i], down, &qf[c][4 * i]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      scl[c][j] = __shfl_sync(~0u, up, (2 * t + j) * 4);
      const int rr = min(r0 + c * 8 + 2 * t + j, r1 - 1);
      row[c][j] = kv8_row(a, seq, rr / a.group);
      slope[c][j] = a.slopes ? a.slopes[h * a.group + rr % a.group] * kLog2e : 0.f;
    }
  }

  int all_lo = 0, all_hi = INT_MAX;  // keys that every row sees
#pragma unroll
  for (int c = 0; c < NT; ++c)
#pragma unroll
    for (int j = 0; j < 2; ++j) all_lo = max(all_lo, row[c][j].lo), all_hi = min(all_hi, row[c][j].hi);
  all_lo = __reduce_max_sync(~0u, all_lo);
  all_hi = __reduce_min_sync(~0u, all_hi);

  float m[NT][2], l[NT][2], o[NT][kSteps][4];
#pragma unroll
  for (int c = 0; c < NT; ++c) {
#pragma unroll
    for (int j = 0; j < 2; ++j) m[c][j] = kNoMax, l[c][j] = 0.f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[c][i][j] = 0.f;
  }
  // z = tanh(s into) out_of, or s into without a cap, s the score in natural units
  const bool cap = BIAS && a.softcap > 0.f;
  const float into = cap ? 1.0f / a.softcap : kLog2e, out_of = a.softcap * kLog2e;
  const int kg = stream_perm<D>(g);
  int kt[4];  // keys whose V a lane reads
#pragma unroll
  for (int j = 0; j < 4; ++j) kt[j] = stream_perm<D>(2 * t + (j & 1)) + 8 * (j >> 1);

  int stage = 0;
  uint32_t phase = 0;
  bool alive = true;
  for (int j = 0; j < n; ++j) {
    if ((j & 31) == 0) {
      if (j > 0) krow[0] = krow[1], ksc[0] = ksc[1], vlog[0] = vlog[1], vinv[0] = vinv[1];
      krow[1] = load_row(j + 32 + lane);
      load_scales(krow[1], ksc[1], vlog[1], vinv[1]);
    }
    const int ahead = (j & 31) + kStg;  // cell j + kStg lies in this batch or the next
    const int next_row = __shfl_sync(~0u, ahead < 32 ? krow[0] : krow[1], ahead & 31);
    const bool there = __shfl_sync(~0u, krow[0], j & 31) >= 0;
    const float ks = __shfl_sync(~0u, ksc[0], j & 31);
    const float lv = __shfl_sync(~0u, vlog[0], j & 31), iv = __shfl_sync(~0u, vinv[0], j & 31);
    alive = __all_sync(~0u, mbar_wait(bar0 + stage * 8, phase, &abort_flag));
    if (!alive) break;
    if (there) {
      const uint8_t* kbuf = smem + (warp * kStg + stage) * kCellBytes;
      const uint8_t* vbuf = kbuf + kCellBytes / 2;
      const int key0 = first_key(j);
      const bool whole = key0 >= all_lo && key0 + kKv8CellKeys <= all_hi + 1;  // every row sees every key
      // scores
      uint32_t kw[2][D / 16];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const uint4 x = *reinterpret_cast<const uint4*>(kbuf + stream_chunk<D>(kg + 8 * r, t + 4 * i));
          kw[r][4 * i] = flip_sign<E4M3>(x.x), kw[r][4 * i + 1] = flip_sign<E4M3>(x.y);
          kw[r][4 * i + 2] = flip_sign<E4M3>(x.z), kw[r][4 * i + 3] = flip_sign<E4M3>(x.w);
        }
      float sc[NT][2][4];
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) sc[c][i / 4][i % 4] = 0.f;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const uint32_t f[4] = {codes_f16<E4M3, false>(kw[0][i]), codes_f16<E4M3, false>(kw[1][i]),
                               codes_f16<E4M3, true>(kw[0][i]), codes_f16<E4M3, true>(kw[1][i])};
#pragma unroll
        for (int c = 0; c < NT; ++c) mma_f16_16816(sc[c][i & 1], f, qf[c][2 * i], qf[c][2 * i + 1]);
      }
      // weights; element i: key kg + 8 (i / 2), column 2t + i % 2
      uint32_t pf[NT][2];
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        float z[4];
        bool over = false;
        float kk[2] = {ks * scl[c][0], ks * scl[c][1]};
        if (BIAS) kk[0] *= into, kk[1] *= into;
        float add[4] = {lv, lv, lv, lv};
        if (BIAS) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float gap = static_cast<float>(row[c][e].pos - key0 - kg);
            add[e] = fmaf(-slope[c][e], fabsf(gap), lv), add[2 + e] = fmaf(-slope[c][e], fabsf(gap - 8.f), lv);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = sc[c][0][i] + sc[c][1][i];
        if (cap) {
          float most = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] *= kk[i & 1], most = fmaxf(most, z[i] * z[i]);
          if (__all_sync(~0u, most <= kCapNear)) {  // the usual case, without special functions
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = fmaf(kv8_tanh_near(z[i]), out_of, add[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = fmaf(kv8_tanh(z[i]), out_of, add[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = fmaf(z[i], kk[i & 1], add[i]);
        }
        if (!whole) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!kv8_sees(row[c][i & 1], seq.prefix, key0 + kg + 8 * (i >> 1))) z[i] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) over |= z[i] > m[c][i & 1] + kMaxSlack;
        if (__any_sync(~0u, over)) {  // some column's maximum rises: all lanes of a column take the same new one
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(m[c][e], fmaxf(z[e], z[2 + e]));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
            const float fix = fast_exp2(m[c][e] - top);
            m[c][e] = top;
            l[c][e] *= fix;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) o[c][i][e] *= fix, o[c][i][2 + e] *= fix;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = fast_exp2(z[i] - m[c][i & 1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // a key out of sight adds nothing, even where its block's scale is NaN
          const float sum = z[e] + z[2 + e];
          if (whole || sum != 0.f) l[c][e] = fmaf(sum, iv, l[c][e]);
        }
        pf[c][0] = movmatrix_t(pack_f16(z[0], z[1]));
        pf[c][1] = movmatrix_t(pack_f16(z[2], z[3]));
      }
      // output; operand rows g and g + 8 of product i are dimensions (D/8) g + 2i and + 1
      uint32_t vw[4][D / 32];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(vbuf + stream_chunk<D>(kt[r], g));
          vw[r][0] = x.x, vw[r][1] = x.y, vw[r][2] = x.z, vw[r][3] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(vbuf + stream_chunk<D>(kt[r], g >> 1) + (g & 1) * 8);
          vw[r][0] = x.x, vw[r][1] = x.y;
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) vw[r][i] = flip_sign<E4M3>(vw[r][i]);
      }
      if (!whole && key0 + kKv8CellKeys > seq.T) {
        // rows behind the context's end hold anything, e4m3 NaN codes too: weight 0 times them must stay 0
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (key0 + kt[r] >= seq.T)
#pragma unroll
            for (int i = 0; i < D / 32; ++i) vw[r][i] = 0;
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const uint32_t sel = i & 1 ? 0x7362 : 0x5140;
        const uint32_t x = prmt(vw[0][i / 2], vw[1][i / 2], sel), y = prmt(vw[2][i / 2], vw[3][i / 2], sel);
        const uint32_t f[4] = {codes_f16<E4M3, false>(x), codes_f16<E4M3, true>(x), codes_f16<E4M3, false>(y),
                               codes_f16<E4M3, true>(y)};
#pragma unroll
        for (int c = 0; c < NT; ++c) mma_f16_16816(o[c][i], f, pf[c][0], pf[c][1]);
      }
    }
    __syncwarp();  // every lane has read the stage
    if (lane == 0 && j + kStg < n) issue(j + kStg, next_row);
    if (++stage == kStg) stage = 0, phase ^= 1;
  }
  if (!alive) {  // a wait ran out (recorded): let the copies in flight land before the CTA leaves
    for (int i = 0; i < kStg; ++i) mbar_drain(bar0 + ((stage + i) % kStg) * 8, phase ^ (stage + i >= kStg ? 1 : 0));
#pragma unroll
    for (int c = 0; c < NT; ++c) l[c][0] = l[c][1] = NAN;
  }

  // join the warps
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem) + warp * kRows * D;
#pragma unroll
  for (int c = 0; c < NT; ++c) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = l[c][e];
      x += __shfl_xor_sync(~0u, x, 4);
      x += __shfl_xor_sync(~0u, x, 8);
      x += __shfl_xor_sync(~0u, x, 16);
      const int col = c * 8 + 2 * t + e;
      if (g == 0) sml[warp][col][0] = m[c][e], sml[warp][col][1] = x;
      float* dst = so + col * D + g * (D / 8);
#pragma unroll
      for (int i = 0; i < kSteps; i += 2)
        *reinterpret_cast<float4*>(dst + 2 * i) =
            make_float4(o[c][i][e], o[c][i][2 + e], o[c][i + 1][e], o[c][i + 1][2 + e]);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < (r1 - r0) * (D / 4); e += kStreamWarps * 32) {
    const int col = e / (D / 4), d = (e % (D / 4)) * 4;
    float M = kNoMax, L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kStreamWarps; ++w) M = fmaxf(M, sml[w][col][0]);
#pragma unroll
    for (int w = 0; w < kStreamWarps; ++w) {
      const float f = fast_exp2(sml[w][col][0] - M);
      const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<float*>(smem) + (w * kRows + col) * D + d);
      L = fmaf(f, sml[w][col][1], L);
      acc[0] = fmaf(f, x.x, acc[0]), acc[1] = fmaf(f, x.y, acc[1]);
      acc[2] = fmaf(f, x.z, acc[2]), acc[3] = fmaf(f, x.w, acc[3]);
    }
    const int r = r0 + col;
    const int64_t at = static_cast<int64_t>(seq.q0 + r / a.group) * hq + h * a.group + r % a.group;
    if (a.nsplit > 1) {
      const int64_t prow = split * (a.total_q * hq) + at;
      if (d == 0) a.ml[prow] = make_float2(M, L);
      *reinterpret_cast<float4*>(a.o + prow * D + d) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    } else {
      const float inv = L == 0.f ? 0.f : 1.0f / L;
      const __nv_bfloat162 x = __floats2bfloat162_rn(acc[0] * inv, acc[1] * inv);
      const __nv_bfloat162 y = __floats2bfloat162_rn(acc[2] * inv, acc[3] * inv);
      uint2 u;
      u.x = *reinterpret_cast<const uint32_t*>(&x), u.y = *reinterpret_cast<const uint32_t*>(&y);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at * D + d) = u;
      if (d == 0 && a.lse) a.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
    }
  }
}

// The cache as rows of one token, head and half: [num_blocks H_kv 2 B][d] bytes, boxes of 16 rows.
static bool make_map_codes(CUtensorMap* map, const void* base, uint64_t rows, int d) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), rows};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(d)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(d), kKv8CellKeys};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace dkv
