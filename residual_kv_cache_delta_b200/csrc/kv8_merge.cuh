// Merge of partial attentions over disjoint key sets: with w_i = exp(lse_i - max_j lse_j),
//   out = sum_i w_i out_i / sum_i w_i,   lse = max + log sum_i w_i.
// One pass, bound by memory: a thread owns 16 bytes of a row (3 parts of 16381 x 32 rows of 128: 80 us, 6.8 TB/s).
#pragma once

#include "kv8_append.cuh"

namespace dkv {

constexpr int kMergeMax = 8;

struct MergeArgs {
  const void* outs[kMergeMax];
  const float* lses[kMergeMax];
  void* out;
  float* lse;
  int64_t rows;
};

// VPR: 16-byte vectors of a row (a power of two that divides the warp, so a row never leaves its warp).
template <typename T, int VPR, int N>
__global__ void __launch_bounds__(256) merge_kernel(const MergeArgs a) {
  constexpr int kElems = 16 / sizeof(T);
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row = id / VPR;
  const bool in = row < a.rows;
  float l[N], m = -INFINITY;
  bool nan = false;
  uint4 x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    l[i] = in ? a.lses[i][row] : 0.f;
    if (in) x[i] = static_cast<const uint4*>(a.outs[i])[id];
  }
  __syncwarp();  // lse may be one of lses: every thread of the row has read before one of them writes
  if (!in) return;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, l[i]), nan |= l[i] != l[i];
  float sum = 0.f, acc[kElems] = {};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (l[i] == -INFINITY) continue;  // a part that saw no key: its out is not read into the sum
    const float w = l[i] == m ? 1.0f : exp2f((l[i] - m) * kLog2e);
    sum += w;
    const T* e = reinterpret_cast<const T*>(&x[i]);
#pragma unroll
    for (int j = 0; j < kElems; ++j) acc[j] += w * Elem<T>::to_f(e[j]);
  }
  const float inv = nan ? NAN : (sum > 0.f ? 1.0f / sum : 0.f);
  uint4 y;
  T* e = reinterpret_cast<T*>(&y);
#pragma unroll
  for (int j = 0; j < kElems; ++j) e[j] = Elem<T>::from_f(acc[j] * inv);
  static_cast<uint4*>(a.out)[id] = y;
  if (id % VPR == 0 && a.lse) a.lse[row] = nan ? NAN : (sum > 0.f ? m + logf(sum) : -INFINITY);
}

template <typename T, int VPR>
static dkv_status merge_n(const MergeArgs& p, int n, cudaStream_t st) {
  const int64_t ctas = ceil_div64(p.rows * VPR, 256);
  if (ctas > INT32_MAX) return DKV_ERR_UNSUPPORTED;
  const dim3 g(static_cast<unsigned>(ctas));
  switch (n) {
    case 1: merge_kernel<T, VPR, 1><<<g, 256, 0, st>>>(p); break;
    case 2: merge_kernel<T, VPR, 2><<<g, 256, 0, st>>>(p); break;
    case 3: merge_kernel<T, VPR, 3><<<g, 256, 0, st>>>(p); break;
    case 4: merge_kernel<T, VPR, 4><<<g, 256, 0, st>>>(p); break;
    case 5: merge_kernel<T, VPR, 5><<<g, 256, 0, st>>>(p); break;
    case 6: merge_kernel<T, VPR, 6><<<g, 256, 0, st>>>(p); break;
    case 7: merge_kernel<T, VPR, 7><<<g, 256, 0, st>>>(p); break;
    default: merge_kernel<T, VPR, 8><<<g, 256, 0, st>>>(p); break;
  }
  return cudaGetLastError() == cudaSuccess ? DKV_OK : DKV_ERR_CUDA;
}

dkv_status launch_merge(int dtype, int64_t rows, int head_dim, int n, const void* const* outs,
                        const float* const* lses, void* out, float* lse, cudaStream_t st) {
  MergeArgs p = {};
  for (int i = 0; i < n; ++i) p.outs[i] = outs[i], p.lses[i] = lses[i];
  p.out = out, p.lse = lse, p.rows = rows;
  if (dtype == DKV_F32)
    return head_dim == 64 ? merge_n<float, 16>(p, n, st) : merge_n<float, 32>(p, n, st);
  return head_dim == 64 ? merge_n<__nv_bfloat16, 8>(p, n, st) : merge_n<__nv_bfloat16, 16>(p, n, st);
}

}  // namespace dkv
