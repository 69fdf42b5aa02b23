// Device-side helpers of the 8-bit paged cache: the cell layout, visibility of keys and the split of a query
// row's keys into cells.
//
// A physical block holds, per kv head, `block` rows of head_dim 8-bit K codes and then as many V codes, and two
// fp32 scales (K, V): a value is code * scale.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "kv8.h"

namespace dkv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The running maximum of a row that has seen no key: finite, so that exp2(-inf - m) is 0 and not NaN.
constexpr float kNoMax = -3.0e38f;

struct Kv8Attn {
  const uint8_t* codes;
  const float* scales;
  int num_blocks, heads, group, block;
  const void* q;
  int64_t q_stride;
  const int* cu_q;
  const int* context_lens;
  const int* block_tables;
  int max_blocks, num_seqs;
  int64_t total_q;
  int max_q, max_ctx;
  float scale;    // softmax scale
  float softcap;  // 0: none
  const float* slopes;
  int window;  // 0: none
  const int* prefix_lens;
  const int* first_key;
  void* out;
  float* lse;
  int nsplit;
  float2* ml;  // [nsplit][total_q][H_q] (maximum, sum), log2 domain
  float* o;    // [nsplit][total_q][H_q][d]
};

// One sequence of an attention call.  ok = false: no queries, or a device length breaks its host bound (recorded);
// its rows are left as they were.
struct Kv8Seq {
  int q0, nq, T, prefix;
  bool ok;
};

__device__ __forceinline__ Kv8Seq kv8_seq(const Kv8Attn& a, int s) {
  Kv8Seq v;
  v.q0 = a.cu_q ? a.cu_q[s] : s;
  v.nq = a.cu_q ? a.cu_q[s + 1] - v.q0 : 1;
  v.T = a.context_lens[s];
  v.prefix = a.prefix_lens ? min(max(a.prefix_lens[s], 0), v.T) : 0;
  const bool fits = v.q0 >= 0 && v.nq >= 0 && v.nq <= a.max_q && static_cast<int64_t>(v.q0) + v.nq <= a.total_q &&
                    v.T >= 0 && v.T <= a.max_ctx;
  if (!fits) record_error(DKV_DEVERR_BOUNDS);
  v.ok = fits && v.nq > 0;
  return v;
}

// Keys that query token i of a sequence sees: [lo, hi] and [first, prefix).
struct Kv8Row {
  int pos, lo, hi, first;
};

__device__ __forceinline__ Kv8Row kv8_row(const Kv8Attn& a, const Kv8Seq& s, int i) {
  Kv8Row r;
  r.pos = s.T - s.nq + i;
  r.first = a.first_key ? max(a.first_key[s.q0 + i], 0) : 0;
  r.lo = a.window > 0 ? max(r.first, r.pos - a.window + 1) : r.first;
  r.hi = r.pos;
  return r;
}

__device__ __forceinline__ bool kv8_sees(const Kv8Row& r, int prefix, int key) {
  return (key >= r.lo && key <= r.hi) || (key >= r.first && key < prefix);
}

// The cells (of `keys` keys each) that hold every key seen by query tokens i0 .. i1-1: [a0, a1) and [b0, b1).
struct Kv8Span {
  int a0, a1, b0, b1;
  __device__ __forceinline__ int count() const { return (a1 - a0) + (b1 - b0); }
  __device__ __forceinline__ int cell(int v) const { return v < a1 - a0 ? a0 + v : b0 + v - (a1 - a0); }
};

__device__ __forceinline__ Kv8Span kv8_span(const Kv8Seq& s, int window, int p0, int p1, int first, int keys) {
  Kv8Span v;
  int lo = window > 0 ? max(0, p0 - window + 1) : 0;
  lo = max(lo, first);
  const int hi = min(p1 + 1, s.T);
  v.a0 = v.a1 = 0;
  if (first < s.prefix) {
    v.a0 = first / keys;
    v.a1 = (s.prefix + keys - 1) / keys;
  }
  v.b0 = lo / keys;
  v.b1 = hi > lo ? (hi + keys - 1) / keys : v.b0;
  if (v.a1 > v.a0) v.b0 = max(v.b0, v.a1);
  v.b1 = max(v.b1, v.b0);
  return v;
}

// Cells [v0, v1) of split `split`: an even share of the span, at least kKv8MinSplitCells, in multiples of `unit`.
__device__ __forceinline__ void kv8_split(int cells, int nsplit, int split, int& v0, int& v1, int unit = 1) {
  int per = max((cells + nsplit - 1) / nsplit, nsplit > 1 ? kKv8MinSplitCells : 1);
  per = (per + unit - 1) / unit * unit;
  v0 = static_cast<int>(min(static_cast<int64_t>(cells), static_cast<int64_t>(split) * per));
  v1 = min(cells, v0 + per);
}

// Physical block of logical block b of sequence s, or -1 (recorded) when the table's entry is out of range.
__device__ __forceinline__ int kv8_block(const int* tables, int max_blocks, int num_blocks, int s, int b) {
  int id = -1;
  if (b >= 0 && b < max_blocks) id = tables[static_cast<int64_t>(s) * max_blocks + b];
  if (id < 0 || id >= num_blocks) {
    record_error(DKV_DEVERR_BLOCK_ID);
    return -1;
  }
  return id;
}

template <bool E4M3>
__device__ __forceinline__ float kv8_decode(uint8_t c) {
  if (E4M3) {
    __nv_fp8_e4m3 x;
    x.__x = c;
    return static_cast<float>(x);
  }
  return static_cast<float>(static_cast<int8_t>(c));
}

// tanh(y) of a capped score cap tanh(x / cap), y = x / cap, in two forms:
//   y^2 <= kCapNear  y P(y^2), P a polynomial (Chebyshev interpolation of degree 4 in y^2 on [0, 0.36], relative error
//                    7.2e-8).  The other form takes the difference of two numbers near 1 here: an error of 2^-21, which is
//                    all of a score that is small against its cap.
//   beyond           1 - 2 / (1 + exp(2 y)) with the hardware's exp2 and reciprocal: off by 4e-7, where tanh is 0.54 at least.
// Either is within 2^-20 of the value.  Both are computed and one is selected: for 1024 tokens at 16384 keys, 32 heads of
// d = 128, scores of the cap's size, that takes 0.99 ms, a branch that parts the warp at every score 1.65 ms.
constexpr float kCapNear = 0.36f;
constexpr float kCapP0 = 0.9999999403953552f, kCapP1 = -0.33332324028015137f, kCapP2 = 0.13310357928276062f,
                kCapP3 = -0.052109625190496445f, kCapP4 = 0.01548669021576643f;
__device__ __forceinline__ float kv8_tanh_near(float y) {
  const float u = y * y;
  return fmaf(u, fmaf(u, fmaf(u, fmaf(u, kCapP4, kCapP3), kCapP2), kCapP1), kCapP0) * y;
}
__device__ __forceinline__ float kv8_tanh(float y) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y * (2.0f * kLog2e)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  asm("{\n\t.reg .pred p;\n\tsetp.le.f32 p, %1, %2;\n\tselp.f32 %0, %3, %4, p;\n\t}"
      : "=f"(r)
      : "f"(y * y), "f"(kCapNear), "f"(kv8_tanh_near(y)), "f"(fmaf(-2.0f, r, 1.0f)));
  return r;
}

// Merges the splits of a query row and head: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.  WPR warps work on a row: a
// lane weighs split `lane` (and + 32, ...), then the warps go through the splits' rows, several loads in flight.
// T: out type.
template <typename T, int D, int WPR>
__global__ void __launch_bounds__(128) kv8_combine_kernel(const __grid_constant__ Kv8Attn a) {
  constexpr int kRows = 4 / WPR, kVec = D / 32;  // rows of a CTA; values of a lane
  __shared__ float part[4][D];
  const int hq = a.heads * a.group, warp = warp_id(), lane = lane_id(), sub = warp % WPR;
  const int64_t rows = a.total_q * hq, row = static_cast<int64_t>(blockIdx.x) * kRows + warp / WPR;
  bool on = row < rows;
  if (on) {
    int s = static_cast<int>(row / hq);
    if (a.cu_q) {  // rows outside every sequence stay as they were
      const int tok = s;
      int lo = 0, hi = a.num_seqs;  // the last sequence that begins at or before tok
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_q[mid] <= tok) lo = mid; else hi = mid;
      }
      s = lo;
      on = tok >= a.cu_q[lo] && tok < a.cu_q[lo + 1];
    }
    if (on) on = kv8_seq(a, s).ok;
  }
  griddep_wait();
  float M = kNoMax, l = 0.f, acc[kVec] = {};
  if (on) {
    float2 p[kKv8MaxSplits / 32];
#pragma unroll
    for (int b = 0; b < kKv8MaxSplits / 32; ++b) {
      const int i = 32 * b + lane;
      p[b] = i < a.nsplit ? a.ml[i * rows + row] : make_float2(kNoMax, 0.f);
      M = fmaxf(M, p[b].x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
#pragma unroll
    for (int b = 0; b < kKv8MaxSplits / 32; ++b) {
      if (32 * b >= a.nsplit) break;
      const float w = p[b].y == 0.f ? 0.f : exp2f(p[b].x - M);  // 0: nothing seen there (a NaN sum goes on)
      l += w * p[b].y;
      const int top = min(32, a.nsplit - 32 * b);
#pragma unroll 8
      for (int i = sub; i < top; i += WPR) {
        const float wi = __shfl_sync(~0u, w, i);
        if (wi == 0.f) continue;
        const float* o = a.o + ((32 * b + i) * rows + row) * D + lane * kVec;
        if constexpr (kVec == 4) {
          const float4 x = *reinterpret_cast<const float4*>(o);
          acc[0] += wi * x.x, acc[1] += wi * x.y, acc[2] += wi * x.z, acc[3] += wi * x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(o);
          acc[0] += wi * x.x, acc[1] += wi * x.y;
        }
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) part[warp][lane * kVec + j] = acc[j];
    __syncthreads();
    if (sub != 0) return;
#pragma unroll
    for (int w = 1; w < WPR; ++w)
#pragma unroll
      for (int j = 0; j < kVec; ++j) acc[j] += part[warp + w][lane * kVec + j];
  }
  if (!on) return;
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  T* out = static_cast<T*>(a.out) + row * D + lane * kVec;
#pragma unroll
  for (int j = 0; j < kVec; ++j) out[j] = Elem<T>::from_f(acc[j] * inv);
  if (lane == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
}

}  // namespace dkv
