// Append to the 8-bit paged cache: position rotation of K (and q), quantisation, paged write.
//
// A CTA owns one block of one sequence and walks kv heads; a thread owns 16 dimensions of one row ("unit") of K and
// of V, so that a block's largest magnitude is one reduction over registers and each input value is read once.
// Unit u of a rotated row holds the dimensions whose partners it also holds: 8u .. 8u+7 of the first half and of
// the second (halves), or 16u .. 16u+15 (pairs); both use entries 8u .. 8u+7 of the cosines and sines.
#pragma once

#include "kv8_common.cuh"

namespace dkv {

constexpr float kKv8Floor = 5.421010862427522e-20f;  // 2^-64: a block's largest magnitude counts as at least this

struct Kv8Append {
  uint8_t* codes;
  float* scales;
  int num_blocks, heads, q_heads, block;
  const void* k;
  const void* v;
  const void* q;
  void* q_out;
  int64_t k_stride, v_stride, q_stride;
  const int* cu_new;
  const int* start_pos;
  const int* block_tables;
  int max_blocks, num_seqs;
  int64_t total_new;
  int max_new;
  const float* rope;
  int rot, max_pos;
  const int* positions;
  int blocks_per_seq;  // blocks that max_new tokens can touch
  int head_steps;      // kv heads a CTA walks
  int64_t kv_ctas;
  int q_head_steps;    // q heads a thread walks
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    unpack16(*reinterpret_cast<const uint4*>(p), f, static_cast<__nv_bfloat16*>(nullptr));
  } else {
    const float4 x = reinterpret_cast<const float4*>(p)[0], y = reinterpret_cast<const float4*>(p)[1];
    f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w, f[4] = y.x, f[5] = y.y, f[6] = y.z, f[7] = y.w;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    __nv_bfloat162 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(w);
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// First dimensions of the two 8-wide halves of unit u.
template <bool PAIRS>
__device__ __forceinline__ void unit_dims(int u, int rot, int& a, int& b) {
  if (PAIRS || u * 16 >= rot) {
    a = 16 * u;
    b = 16 * u + 8;
  } else {
    a = 8 * u;
    b = 8 * u + rot / 2;
  }
}

// Rotates a unit; products and sums are rounded one by one, so that the result does not depend on contraction.
template <bool PAIRS>
__device__ __forceinline__ void rotate_unit(float (&x)[8], float (&y)[8], const float (&c)[8], const float (&s)[8]) {
  if (PAIRS) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float& a = j < 4 ? x[2 * j] : y[2 * j - 8];
      float& b = j < 4 ? x[2 * j + 1] : y[2 * j - 7];
      const float ra = __fsub_rn(__fmul_rn(a, c[j]), __fmul_rn(b, s[j]));
      const float rb = __fadd_rn(__fmul_rn(b, c[j]), __fmul_rn(a, s[j]));
      a = ra, b = rb;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float ra = __fsub_rn(__fmul_rn(x[j], c[j]), __fmul_rn(y[j], s[j]));
      const float rb = __fadd_rn(__fmul_rn(y[j], c[j]), __fmul_rn(x[j], s[j]));
      x[j] = ra, y[j] = rb;
    }
  }
}

// Cosines and sines 8u .. 8u+7 of a token; false when the unit is not rotated.  A position outside the table is
// recorded and leaves the row unrotated.
__device__ __forceinline__ bool load_angles(const Kv8Append& a, int pos, int u, float (&c)[8], float (&s)[8]) {
  if (u * 16 >= a.rot) return false;
  if (pos < 0 || pos >= a.max_pos) {
    record_error(DKV_DEVERR_BOUNDS);
    return false;
  }
  const float* t = a.rope + static_cast<int64_t>(pos) * a.rot + 8 * u;
  load8(t, c);
  load8(t + a.rot / 2, s);
  return true;
}

__device__ __forceinline__ uint32_t max_bits(uint32_t m, const float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
  return m;
}

// 8 codes of f * inv, round to nearest even, saturating.
template <bool E4M3>
__device__ __forceinline__ uint2 quantise8(const float (&f)[8], float inv) {
  uint32_t w[2] = {0, 0};
  if constexpr (E4M3) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t p = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * j] * inv, f[2 * j + 1] * inv), __NV_SATFINITE,
                                                  __NV_E4M3);
      w[j / 2] |= p << (16 * (j % 2));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = __float2int_rn(fminf(fmaxf(f[j] * inv, -127.f), 127.f));
      w[j / 4] |= (static_cast<uint32_t>(c) & 0xffu) << (8 * (j % 4));
    }
  }
  return make_uint2(w[0], w[1]);
}

template <typename T, int D, bool E4M3, bool PAIRS>
__device__ __forceinline__ void append_q(const Kv8Append& a, int64_t cta) {
  constexpr int kUnits = D / 16;
  const int per = blockDim.x / kUnits;  // tokens of a CTA
  const int chunks = (a.q_heads + a.q_head_steps - 1) / a.q_head_steps;
  const int h0 = static_cast<int>(cta % chunks) * a.q_head_steps;
  const int64_t tok = cta / chunks * per + threadIdx.x / kUnits;
  if (tok >= a.total_new) return;
  const int u = threadIdx.x % kUnits;
  int lo = 0, hi = a.num_seqs;  // the last sequence that begins at or before the token
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_new[mid] <= tok) lo = mid; else hi = mid;
  }
  if (tok < a.cu_new[lo] || tok >= a.cu_new[lo + 1]) return;  // a row of no sequence
  const int pos = a.positions ? a.positions[tok] : a.start_pos[lo] + static_cast<int>(tok - a.cu_new[lo]);
  float c[8], s[8], x[8], y[8];
  const bool turn = load_angles(a, pos, u, c, s);
  int da, db;
  unit_dims<PAIRS>(u, a.rot, da, db);
  const T* src = static_cast<const T*>(a.q) + tok * a.q_stride;
  T* dst = static_cast<T*>(a.q_out) + tok * a.q_heads * D;
  for (int h = h0; h < min(h0 + a.q_head_steps, a.q_heads); ++h) {
    load8(src + h * D + da, x);
    load8(src + h * D + db, y);
    if (turn) rotate_unit<PAIRS>(x, y, c, s);
    store8(dst + h * D + da, x);
    store8(dst + h * D + db, y);
  }
}

template <typename T, int D, bool E4M3, bool PAIRS>
__global__ void __launch_bounds__(512) kv8_append_kernel(const Kv8Append a) {
  constexpr int kUnits = D / 16;
  constexpr float kTop = E4M3 ? 448.0f : 127.0f;
  __shared__ uint2 top[2][16];
  if (blockIdx.x >= a.kv_ctas) {
    append_q<T, D, E4M3, PAIRS>(a, blockIdx.x - a.kv_ctas);
    return;
  }
  const int steps = (a.heads + a.head_steps - 1) / a.head_steps;
  int64_t id = blockIdx.x;
  const int h0 = static_cast<int>(id % steps) * a.head_steps;
  id /= steps;
  const int nth = static_cast<int>(id % a.blocks_per_seq), s = static_cast<int>(id / a.blocks_per_seq);
  const int row0 = a.cu_new[s], n = a.cu_new[s + 1] - row0, start = a.start_pos[s];
  if (n <= 0) return;
  if (row0 < 0 || n > a.max_new || static_cast<int64_t>(row0) + n > a.total_new || start < 0 ||
      start > INT32_MAX - n) {
    if (threadIdx.x == 0) record_error(DKV_DEVERR_BOUNDS);
    return;
  }
  const int b = start / a.block + nth;
  if (static_cast<int64_t>(b) * a.block >= static_cast<int64_t>(start) + n) return;
  const int blk = kv8_block(a.block_tables, a.max_blocks, a.num_blocks, s, b);
  if (blk < 0) return;
  const int u = threadIdx.x % kUnits, r = threadIdx.x / kUnits;
  const int at = b * a.block + r - start;  // row of this call, or before (< 0) or after (>= n) its rows
  const bool fresh = at >= 0 && at < n;
  const bool held = b * a.block < start;   // the block holds earlier rows
  const int64_t tok = row0 + (fresh ? at : 0);
  float c[8], sn[8];
  bool turn = false;
  int da, db;
  unit_dims<PAIRS>(u, a.rot, da, db);
  if (fresh && a.rot > 0) turn = load_angles(a, a.positions ? a.positions[tok] : start + at, u, c, sn);
  const T* kp = static_cast<const T*>(a.k) + tok * a.k_stride;
  const T* vp = static_cast<const T*>(a.v) + tok * a.v_stride;
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32;
  for (int h = h0; h < min(h0 + a.head_steps, a.heads); ++h) {
    float kx[8] = {}, ky[8] = {}, vx[8] = {}, vy[8] = {};
    if (fresh) {
      load8(kp + h * D + da, kx);
      load8(kp + h * D + db, ky);
      load8(vp + h * D + 16 * u, vx);
      load8(vp + h * D + 16 * u + 8, vy);
      if (turn) rotate_unit<PAIRS>(kx, ky, c, sn);
    }
    // bit patterns of magnitudes order like the magnitudes, with infinities and then NaN on top
    const uint32_t km = __reduce_max_sync(~0u, max_bits(max_bits(0u, kx), ky));
    const uint32_t vm = __reduce_max_sync(~0u, max_bits(max_bits(0u, vx), vy));
    uint2* t = top[(h - h0) & 1];
    if (threadIdx.x % 32 == 0) t[warp] = make_uint2(km, vm);
    __syncthreads();
    uint32_t m[2] = {0u, 0u};
    for (int w = 0; w < warps; ++w) {
      const uint2 x = t[w];
      m[0] = max(m[0], x.x), m[1] = max(m[1], x.y);
    }
    const int64_t cell = (static_cast<int64_t>(blk) * a.heads + h) * 2;
    float inv[2], ratio[2], now[2];
    bool bad[2], grew[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      now[j] = fmaxf(__uint_as_float(m[j]), kKv8Floor) * (1.0f / kTop);
      bad[j] = m[j] >= 0x7f800000u;  // a value is not finite: the block reads as NaN from here on
      float old = 0.f;
      if (held) {
        old = a.scales[cell + j];
        bad[j] |= !(fabsf(old) <= 3.402823466e38f);
        now[j] = fmaxf(now[j], old);
      }
      grew[j] = held && now[j] > old;
      inv[j] = __frcp_rn(now[j]);
      ratio[j] = __fmul_rn(old, inv[j]);
      if (bad[j]) now[j] = __uint_as_float(0x7fc00000u), inv[j] = 0.f;
    }
    uint8_t* kc = a.codes + (cell * a.block + r) * D;
    uint8_t* vc = kc + static_cast<int64_t>(a.block) * D;
    if (fresh) {
      *reinterpret_cast<uint2*>(kc + da) = bad[0] ? make_uint2(0u, 0u) : quantise8<E4M3>(kx, inv[0]);
      *reinterpret_cast<uint2*>(kc + db) = bad[0] ? make_uint2(0u, 0u) : quantise8<E4M3>(ky, inv[0]);
      const uint2 x = bad[1] ? make_uint2(0u, 0u) : quantise8<E4M3>(vx, inv[1]);
      const uint2 y = bad[1] ? make_uint2(0u, 0u) : quantise8<E4M3>(vy, inv[1]);
      *reinterpret_cast<uint4*>(vc + 16 * u) = make_uint4(x.x, x.y, y.x, y.y);
    } else if (at < 0) {  // an earlier row: its codes follow a scale that grew
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (bad[j] || !grew[j]) continue;
        uint8_t* p = (j ? vc : kc) + 16 * u;
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
        float f[8], g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[i] = kv8_decode<E4M3>(static_cast<uint8_t>(ww[i / 4] >> (8 * (i % 4))));
          g[i] = kv8_decode<E4M3>(static_cast<uint8_t>(ww[2 + i / 4] >> (8 * (i % 4))));
        }
        const uint2 x = quantise8<E4M3>(f, ratio[j]), y = quantise8<E4M3>(g, ratio[j]);
        *reinterpret_cast<uint4*>(p) = make_uint4(x.x, x.y, y.x, y.y);
      }
    }
    __syncthreads();  // every thread has read the old scales
    if (threadIdx.x < 2) a.scales[cell + threadIdx.x] = threadIdx.x ? now[1] : now[0];
  }
}

template <typename T, int D, bool E4M3>
static dkv_status append_pairs(const Kv8Append& p, bool pairs, dim3 grid, int threads, cudaStream_t st) {
  if (pairs)
    kv8_append_kernel<T, D, E4M3, true><<<grid, threads, 0, st>>>(p);
  else
    kv8_append_kernel<T, D, E4M3, false><<<grid, threads, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? DKV_OK : DKV_ERR_CUDA;
}

dkv_status launch_kv8_append(const Kv8AppendArgs& a, cudaStream_t st) {
  const dkv_kv8_shape& sh = *a.shape;
  Kv8Append p = {};
  p.codes = static_cast<uint8_t*>(a.cache->codes);
  p.scales = a.cache->scales;
  p.num_blocks = a.cache->num_blocks;
  p.heads = sh.num_kv_heads, p.q_heads = sh.num_q_heads, p.block = sh.block_tokens;
  p.k = a.k_new, p.v = a.v_new, p.q = a.q, p.q_out = a.q_out;
  p.k_stride = a.k_stride, p.v_stride = a.v_stride, p.q_stride = a.q_stride;
  p.cu_new = a.cu_new, p.start_pos = a.start_pos, p.block_tables = a.block_tables;
  p.max_blocks = a.max_blocks, p.num_seqs = a.num_seqs, p.total_new = a.total_new, p.max_new = a.max_new;
  if (a.rope) {
    p.rope = a.rope->table, p.rot = a.rope->rot_dim, p.max_pos = a.rope->max_pos;
    p.positions = a.rope->positions;
  }
  p.blocks_per_seq = static_cast<int>((static_cast<int64_t>(a.max_new) + sh.block_tokens - 2) / sh.block_tokens + 1);
  const int threads = sh.block_tokens * sh.head_dim / 16;
  p.head_steps = 1;
  p.kv_ctas = static_cast<int64_t>(a.num_seqs) * p.blocks_per_seq * p.heads;
  int64_t q_ctas = 0;
  if (a.q) {
    p.q_head_steps = 4;
    const int per = threads / (sh.head_dim / 16);
    q_ctas = ceil_div64(a.total_new, per) * ceil_div64(p.q_heads, p.q_head_steps);
  }
  if (p.kv_ctas + q_ctas > INT32_MAX) return DKV_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(p.kv_ctas + q_ctas));
  const bool pairs = a.rope && a.rope->pairs, e4 = sh.code == DKV_KV8_E4M3, d64 = sh.head_dim == 64;
  if (sh.dtype == DKV_F32) {
    if (d64) return e4 ? append_pairs<float, 64, true>(p, pairs, grid, threads, st)
                       : append_pairs<float, 64, false>(p, pairs, grid, threads, st);
    return e4 ? append_pairs<float, 128, true>(p, pairs, grid, threads, st)
              : append_pairs<float, 128, false>(p, pairs, grid, threads, st);
  }
  if (d64) return e4 ? append_pairs<__nv_bfloat16, 64, true>(p, pairs, grid, threads, st)
                     : append_pairs<__nv_bfloat16, 64, false>(p, pairs, grid, threads, st);
  return e4 ? append_pairs<__nv_bfloat16, 128, true>(p, pairs, grid, threads, st)
            : append_pairs<__nv_bfloat16, 128, false>(p, pairs, grid, threads, st);
}

}  // namespace dkv
