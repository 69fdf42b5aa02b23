// Attention over the 8-bit cache on CUDA cores, fp32 arithmetic throughout: the path of fp32 tensors.  8 x 32768 tokens of
// d = 128, 8 kv heads, 4 heads each: 818 us, 0.66 TB/s, where memory alone would take 82; 512 tokens at 8192 keys: 5.8 ms.
// Bound by its scalar products and three CTA barriers per 32 keys.
//
// One CTA takes kRows query rows (a row is a query token and a head of the kv head's group) and a range of keys.
// Tiles of 32 keys are dequantised into shared memory; a warp scores two rows against the tile (one key per lane),
// updates their running maximum and sum, and the CTA's threads, one per output dimension, add p * V.  V lies there as codes and
// its scale is part of the row's weight, which is 0 for a key out of the row's sight: a block whose scale is NaN then
// reaches only the rows that see it.
#pragma once

#include "kv8_common.cuh"

namespace dkv {

constexpr int kSimpleRows = 8, kSimpleKeys = 32;

template <int D, bool E4M3>
__global__ void __launch_bounds__(128) kv8_attn_simple_kernel(const Kv8Attn a, int row_tiles) {
  constexpr int kPad = D + 4;
  __shared__ __align__(16) float sk[kSimpleKeys * kPad];
  __shared__ __align__(16) float sv[kSimpleKeys * D];
  __shared__ __align__(16) float sq[kSimpleRows * D];
  __shared__ float sp[kSimpleRows][kSimpleKeys];
  __shared__ float sfix[kSimpleRows];
  __shared__ float svs[kSimpleKeys];   // V scale of the tile's key
  __shared__ int sthere[kSimpleKeys];  // whether the tile's key lies in the context, in a mapped block
  __shared__ float sm[kSimpleRows], sl[kSimpleRows];
  griddep_launch_dependents();
  int64_t id = blockIdx.x;
  const int split = static_cast<int>(id % a.nsplit);
  id /= a.nsplit;
  const int tile = static_cast<int>(id % row_tiles);
  id /= row_tiles;
  const int h = static_cast<int>(id % a.heads), s = static_cast<int>(id / a.heads);
  const Kv8Seq sq_ = kv8_seq(a, s);
  const int nrows = sq_.nq * a.group, r0 = tile * kSimpleRows;
  if (!sq_.ok || r0 >= nrows) return;
  const int r1 = min(r0 + kSimpleRows, nrows), hq = a.heads * a.group;
  const int i0 = r0 / a.group, i1 = (r1 - 1) / a.group;
  int first = INT_MAX;
  for (int i = i0; i <= i1; ++i) first = min(first, kv8_row(a, sq_, i).first);
  const Kv8Span span =
      kv8_span(sq_, a.window, sq_.T - sq_.nq + i0, sq_.T - sq_.nq + i1, first, kKv8CellKeys);
  int v0, v1;
  kv8_split(span.count(), a.nsplit, split, v0, v1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int e = tid; e < kSimpleRows * D; e += 128) {
    const int r = r0 + e / D;
    float x = 0.f;
    if (r < r1)
      x = static_cast<const float*>(a.q)[(sq_.q0 + r / a.group) * a.q_stride + (h * a.group + r % a.group) * D + e % D];
    sq[e] = x * a.scale;
  }
  float m[2] = {kNoMax, kNoMax}, l[2] = {0.f, 0.f}, acc[kSimpleRows] = {};
  Kv8Row row[2];
  float slope[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = min(r0 + warp * 2 + j, r1 - 1);
    row[j] = kv8_row(a, sq_, r / a.group);
    if (a.slopes) slope[j] = a.slopes[h * a.group + r % a.group] * kLog2e;
  }
  for (int v = v0; v < v1; v += 2) {  // two cells of 16 keys
    __syncthreads();
    for (int e = tid; e < kSimpleKeys * D / 16; e += 128) {  // 16 codes of K and of V
      const int k = e / (D / 16), c = (e % (D / 16)) * 16;
      const int cell = v + k / kKv8CellKeys;
      float kf[16] = {}, vf[16] = {}, vs = 0.f;
      int there = 0;
      if (cell < v1) {
        const int key = span.cell(cell) * kKv8CellKeys + k % kKv8CellKeys;
        const int blk =
            key < sq_.T ? kv8_block(a.block_tables, a.max_blocks, a.num_blocks, s, key / a.block) : -1;
        if (blk >= 0) {
          const int64_t cellbase = (static_cast<int64_t>(blk) * a.heads + h) * 2;
          const uint8_t* src = a.codes + (cellbase * a.block + key % a.block) * D + c;
          const uint4 kw = *reinterpret_cast<const uint4*>(src);
          const uint4 vw = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(a.block) * D);
          there = 1;
          const float ks = a.scales[cellbase];
          vs = a.scales[cellbase + 1];
          const uint32_t kk[4] = {kw.x, kw.y, kw.z, kw.w}, vv[4] = {vw.x, vw.y, vw.z, vw.w};
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            kf[j] = kv8_decode<E4M3>(static_cast<uint8_t>(kk[j / 4] >> (8 * (j % 4)))) * ks;
            vf[j] = kv8_decode<E4M3>(static_cast<uint8_t>(vv[j / 4] >> (8 * (j % 4))));
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) sk[k * kPad + c + j] = kf[j], sv[k * D + c + j] = vf[j];
      if (c == 0) sthere[k] = there, svs[k] = vs;
    }
    __syncthreads();
    const bool there = sthere[lane] != 0;
    float d[2] = {0.f, 0.f};
#pragma unroll 8
    for (int c = 0; c < D; c += 4) {
      const float4 kk = *reinterpret_cast<const float4*>(sk + lane * kPad + c);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 qq = *reinterpret_cast<const float4*>(sq + (warp * 2 + j) * D + c);
        d[j] += qq.x * kk.x + qq.y * kk.y + qq.z * kk.z + qq.w * kk.w;
      }
    }
    const int cell = min(v + lane / kKv8CellKeys, v1 - 1);
    const int key = span.cell(cell) * kKv8CellKeys + lane % kKv8CellKeys;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float z = a.softcap > 0.f ? a.softcap * tanhf(d[j] / a.softcap) : d[j];
      z = z * kLog2e - slope[j] * abs(row[j].pos - key);
      const bool seen = there && kv8_sees(row[j], sq_.prefix, key);
      if (!seen) z = -INFINITY;
      float top = z;
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
      top = fmaxf(top, m[j]);
      const float p = exp2f(z - top), fix = exp2f(m[j] - top);
      m[j] = top;
      l[j] = l[j] * fix + p;
      sp[warp * 2 + j][lane] = seen ? p * svs[lane] : 0.f;
      if (lane == 0) sfix[warp * 2 + j] = fix;
    }
    __syncthreads();
    if (tid < D) {
#pragma unroll
      for (int r = 0; r < kSimpleRows; ++r) acc[r] *= sfix[r];
#pragma unroll 4
      for (int k = 0; k < kSimpleKeys; ++k) {
        const float x = sv[k * D + tid];
#pragma unroll
        for (int r = 0; r < kSimpleRows; ++r) acc[r] += sp[r][k] * x;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
#pragma unroll
    for (int o = 16; o; o >>= 1) l[j] += __shfl_xor_sync(~0u, l[j], o);
    if (lane == 0) sm[warp * 2 + j] = m[j], sl[warp * 2 + j] = l[j];
  }
  __syncthreads();
  for (int r = r0; r < r1; ++r) {
    const int64_t at = static_cast<int64_t>(sq_.q0 + r / a.group) * hq + h * a.group + r % a.group;
    const float mm = sm[r - r0], ll = sl[r - r0];
    float o = 0.f;
#pragma unroll
    for (int j = 0; j < kSimpleRows; ++j)
      if (j == r - r0) o = acc[j];
    if (a.nsplit > 1) {
      const int64_t prow = split * (a.total_q * hq) + at;
      if (tid == 0) a.ml[prow] = make_float2(mm, ll);
      if (tid < D && ll != 0.f) a.o[prow * D + tid] = o;
    } else {
      if (tid < D) static_cast<float*>(a.out)[at * D + tid] = ll == 0.f ? 0.f : o / ll;
      if (tid == 0 && a.lse) a.lse[at] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
    }
  }
}

}  // namespace dkv
