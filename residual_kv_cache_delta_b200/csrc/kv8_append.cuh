// Append to the 8-bit paged cache: position rotation of K (and q), quantisation, paged write.
//
// Bound by memory: every input value is read once and every code written once (two prompts of 32768 tokens, 32 + 2 x 8 heads
// of 128: 211 us, 5.8 TB/s with 80 registers; an earlier build took 216 us with 72, 235 with 64 and 233 with 98).
// A CTA owns K or V of one block of one sequence for a few kv heads; a thread owns 16 dimensions of one row ("unit"), so that a
// block's largest magnitude is a reduction over registers, and loads several heads at once, before anything that it does not
// need for their addresses.
// Unit u of a rotated row holds dimensions whose partners it also holds: 8u .. 8u+7 of the first half and of the second
// (halves), or 16u .. 16u+15 (pairs); both use entries 8u .. 8u+7 of the cosines and sines, which stay in registers.
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
  int64_t kv_ctas;
  int q_head_steps;    // q heads a thread walks
  float neg_zero;      // -0, not known to the compiler
};

// Rows of one sequence of an append; ok = false when they break a bound (nothing of the sequence is written then).
struct AppendSeq {
  int row0, n, start;
  bool ok;
};
__device__ __forceinline__ AppendSeq append_seq(const Kv8Append& a, int s) {
  AppendSeq v;
  v.row0 = a.cu_new[s], v.n = a.cu_new[s + 1] - v.row0, v.start = a.start_pos[s];
  v.ok = v.row0 >= 0 && v.n <= a.max_new && static_cast<int64_t>(v.row0) + v.n <= a.total_new && v.start >= 0 &&
         static_cast<int64_t>(v.start) + v.n <= INT32_MAX - 64;  // positions of a block's rows fit an int
  return v;
}

// Eight values of type T as they lie in memory.
template <typename T>
struct Oct;
template <>
struct Oct<float> {
  float4 v, w;
  __device__ __forceinline__ void get(float* f) const {
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w, f[4] = w.x, f[5] = w.y, f[6] = w.z, f[7] = w.w;
  }
  static __device__ __forceinline__ Oct make(const float* f) {
    return {make_float4(f[0], f[1], f[2], f[3]), make_float4(f[4], f[5], f[6], f[7])};
  }
  __device__ __forceinline__ void forget() {
    asm volatile("" : "+f"(v.x), "+f"(v.y), "+f"(v.z), "+f"(v.w), "+f"(w.x), "+f"(w.y), "+f"(w.z), "+f"(w.w));
  }
};
template <>
struct Oct<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) f[2 * j] = __uint_as_float(w[j] << 16), f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
  static __device__ __forceinline__ Oct make(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&x);
    }
    return {make_uint4(w[0], w[1], w[2], w[3])};
  }
  // Makes the compiler take the value for a new one, so that what was computed from it before is not kept in registers.
  __device__ __forceinline__ void forget() { asm volatile("" : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)); }
};
template <typename T>
struct Unit {
  Oct<T> a, b;
};
template <typename T>
__device__ __forceinline__ Unit<T> load_unit(const T* p, int da, int db) {
  return {*reinterpret_cast<const Oct<T>*>(p + da), *reinterpret_cast<const Oct<T>*>(p + db)};
}

// First dimensions of the two octets of unit u.
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

// Two fp32 operations to an instruction.  A product is a fused multiply-add of -0 that the compiler does not know (nz, from
// the kernel's arguments): it is rounded by itself, where a packed product is contracted with the sum behind it.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Rotates a unit; products and sums are rounded one by one.
template <bool PAIRS>
__device__ __forceinline__ void rotate_unit(float (&x)[16], const float (&cs)[16], uint64_t nz) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    float &a0 = PAIRS ? x[2 * j] : x[j], &a1 = PAIRS ? x[2 * j + 2] : x[j + 1];
    float &b0 = PAIRS ? x[2 * j + 1] : x[8 + j], &b1 = PAIRS ? x[2 * j + 3] : x[9 + j];
    const uint64_t a = pack2(a0, a1), b = pack2(b0, b1), c = pack2(cs[j], cs[j + 1]), s = pack2(cs[8 + j], cs[9 + j]);
    unpack2(fma2(fma2(b, s, nz), pack2(-1.f, -1.f), fma2(a, c, nz)), a0, a1);
    unpack2(add2(fma2(b, c, nz), fma2(a, s, nz)), b0, b1);
  }
}

// Cosines and sines 8u .. 8u+7 of a token; false when the unit is not rotated.  A position outside the table is
// recorded and leaves the row unrotated.
__device__ __forceinline__ bool load_angles(const Kv8Append& a, int pos, int u, float (&cs)[16]) {
  if (u * 16 >= a.rot) return false;
  if (pos < 0 || pos >= a.max_pos) {
    record_error(DKV_DEVERR_BOUNDS);
    return false;
  }
  const float* t = a.rope + static_cast<int64_t>(pos) * a.rot + 8 * u;
  reinterpret_cast<const Oct<float>*>(t)->get(cs);
  reinterpret_cast<const Oct<float>*>(t + a.rot / 2)->get(cs + 8);
  return true;
}

// 8 codes of f * inv, round to nearest even.  |f * inv| exceeds the largest code by a few roundings at most, so that the
// nearest int8 code is in range without a clamp.
template <bool E4M3>
__device__ __forceinline__ uint2 quantise8(const float* f, float inv, uint64_t nz) {
  const uint64_t i2 = pack2(inv, inv);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint64_t y0 = fma2(pack2(f[4 * h], f[4 * h + 1]), i2, nz), y1 = fma2(pack2(f[4 * h + 2], f[4 * h + 3]), i2, nz);
    float v[4];
    if constexpr (E4M3) {
      uint16_t lo, hi;
      unpack2(y0, v[0], v[1]), unpack2(y1, v[2], v[3]);
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[1]), "f"(v[0]));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[3]), "f"(v[2]));
      w[h] = static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
    } else {  // adding 1.5 2^23 leaves the rounded integer in the low mantissa bits
      const uint64_t magic = pack2(12582912.f, 12582912.f);
      unpack2(add2(y0, magic), v[0], v[1]), unpack2(add2(y1, magic), v[2], v[3]);
      w[h] = __byte_perm(__byte_perm(__float_as_uint(v[0]), __float_as_uint(v[1]), 0x0040),
                         __byte_perm(__float_as_uint(v[2]), __float_as_uint(v[3]), 0x0040), 0x5410);
    }
  }
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Heads of a thread's loads in flight (32 registers)
template <typename T>
constexpr int kAppendHeads = sizeof(T) == 2 ? 4 : 2;

// Loads the unit of the next heads from h on (those below h1).
template <typename T, int D>
__device__ __forceinline__ void load_heads(const T* src, int h, int h1, int da, int db, bool on,
                                           Unit<T> (&x)[kAppendHeads<T>]) {
#pragma unroll
  for (int i = 0; i < kAppendHeads<T>; ++i) {
    x[i] = Unit<T>{};
    if (on && h + i < h1) x[i] = load_unit(src + (h + i) * D, da, db);
  }
}

template <typename T, int D, bool PAIRS>
__device__ __forceinline__ void append_q(const Kv8Append& a, int64_t cta) {
  constexpr int kUnits = D / 16, kN = kAppendHeads<T>;
  const int per = blockDim.x / kUnits;  // tokens of a CTA
  const int chunks = (a.q_heads + a.q_head_steps - 1) / a.q_head_steps;
  const int h0 = static_cast<int>(cta % chunks) * a.q_head_steps, h1 = min(h0 + a.q_head_steps, a.q_heads);
  const int64_t tok = cta / chunks * per + threadIdx.x / kUnits;
  if (tok >= a.total_new) return;
  const int u = threadIdx.x % kUnits;
  int da, db;
  unit_dims<PAIRS>(u, a.rot, da, db);
  const T* src = static_cast<const T*>(a.q) + tok * a.q_stride;
  T* dst = static_cast<T*>(a.q_out) + tok * a.q_heads * D;
  Unit<T> raw[kN];
  load_heads<T, D>(src, h0, h1, da, db, true, raw);
  int lo = 0, hi = a.num_seqs;  // the last sequence that begins at or before the token
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_new[mid] <= tok) lo = mid; else hi = mid;
  }
  const AppendSeq q = append_seq(a, lo);
  // a row of no sequence, or of one that the K and V part records and refuses
  if (tok < q.row0 || tok >= static_cast<int64_t>(q.row0) + q.n || !q.ok) return;
  const int pos = a.positions ? a.positions[tok] : q.start + static_cast<int>(tok - q.row0);
  float cs[16], x[16];
  const uint64_t nz = pack2(a.neg_zero, a.neg_zero);
  const bool turn = load_angles(a, pos, u, cs);
#pragma unroll 1
  for (int h = h0; h < h1; h += kN) {
    if (h > h0) load_heads<T, D>(src, h, h1, da, db, true, raw);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      if (h + i >= h1) continue;
      raw[i].a.get(x), raw[i].b.get(x + 8);
      if (turn) rotate_unit<PAIRS>(x, cs, nz);
      *reinterpret_cast<Oct<T>*>(dst + (h + i) * D + da) = Oct<T>::make(x);
      *reinterpret_cast<Oct<T>*>(dst + (h + i) * D + db) = Oct<T>::make(x + 8);
    }
  }
}

template <typename T, int D, bool E4M3, bool PAIRS>
__global__ void __maxnreg__(80) kv8_append_kernel(const __grid_constant__ Kv8Append a) {
  constexpr int kUnits = D / 16, kN = kAppendHeads<T>;
  constexpr float kTop = E4M3 ? 448.0f : 127.0f;
  __shared__ uint32_t tops[kN][16];
  if (blockIdx.x >= a.kv_ctas) {
    append_q<T, D, PAIRS>(a, blockIdx.x - a.kv_ctas);
    return;
  }
  const int steps = (a.heads + kN - 1) / kN;
  int64_t id = blockIdx.x;
  const int half = static_cast<int>(id & 1);  // 0: K, 1: V
  id >>= 1;
  const int h0 = static_cast<int>(id % steps) * kN, h1 = min(h0 + kN, a.heads);
  id /= steps;
  const int nth = static_cast<int>(id % a.blocks_per_seq), s = static_cast<int>(id / a.blocks_per_seq);
  const AppendSeq seq = append_seq(a, s);
  const int row0 = seq.row0, n = seq.n, start = seq.start;
  if (n <= 0) return;
  if (!seq.ok) {
    if (threadIdx.x == 0) record_error(DKV_DEVERR_BOUNDS);
    return;
  }
  const int b = start / a.block + nth;
  if (static_cast<int64_t>(b) * a.block >= static_cast<int64_t>(start) + n) return;
  const int u = threadIdx.x % kUnits, r = threadIdx.x / kUnits;
  const int at = b * a.block + r - start;  // row of this call, or before (< 0) or after (>= n) its rows
  const bool fresh = at >= 0 && at < n;
  const bool held = b * a.block < start;   // the block holds earlier rows
  const int64_t tok = row0 + (fresh ? at : 0);
  int da = 16 * u, db = 16 * u + 8;
  if (half == 0) unit_dims<PAIRS>(u, a.rot, da, db);
  const T* src = half ? static_cast<const T*>(a.v) + tok * a.v_stride : static_cast<const T*>(a.k) + tok * a.k_stride;
  Unit<T> raw[kN];
  load_heads<T, D>(src, h0, h1, da, db, fresh, raw);
  const int blk = kv8_block(a.block_tables, a.max_blocks, a.num_blocks, s, b);
  if (blk < 0) return;
  float cs[16];
  const uint64_t nz = pack2(a.neg_zero, a.neg_zero);
  bool turn = false;
  if (half == 0 && fresh && a.rot > 0) turn = load_angles(a, a.positions ? a.positions[tok] : start + at, u, cs);
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float x[16], old[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    old[i] = 0.f;
    if (held && h0 + i < h1) old[i] = a.scales[(static_cast<int64_t>(blk) * a.heads + h0 + i) * 2 + half];
    raw[i].a.get(x), raw[i].b.get(x + 8);
    if (turn) rotate_unit<PAIRS>(x, cs, nz);
    float top = fabsf(x[0]);
#pragma unroll
    for (int j = 1; j < 16; ++j) top = max_nan(top, fabsf(x[j]));
    // bit patterns of magnitudes order like the magnitudes, with infinities and then NaN on top
    const uint32_t m = __reduce_max_sync(~0u, __float_as_uint(top) & 0x7fffffffu);
    if (lane == 0) tops[i][warp] = m;
  }
  __syncthreads();  // also: every thread has read the old scales
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    if (h0 + i >= h1) continue;
    const uint32_t m = __reduce_max_sync(~0u, lane < warps ? tops[i][lane] : 0u);
    const int64_t cell = (static_cast<int64_t>(blk) * a.heads + h0 + i) * 2 + half;
    const float now = fmaxf(fmaxf(__uint_as_float(m), kKv8Floor) * (1.0f / kTop), old[i]);
    // a value is not finite: the block reads as NaN from here on
    const bool bad = m >= 0x7f800000u || !(fabsf(old[i]) <= 3.402823466e38f);
    const float inv = __frcp_rn(now);
    uint8_t* codes = a.codes + (cell * a.block + r) * D;
    if (fresh) {  // rotated once more: cheaper than to keep the fp32 values of four heads
      raw[i].a.forget(), raw[i].b.forget();
      raw[i].a.get(x), raw[i].b.get(x + 8);
      if (turn) rotate_unit<PAIRS>(x, cs, nz);
      *reinterpret_cast<uint2*>(codes + da) = bad ? make_uint2(0u, 0u) : quantise8<E4M3>(x, inv, nz);
      *reinterpret_cast<uint2*>(codes + db) = bad ? make_uint2(0u, 0u) : quantise8<E4M3>(x + 8, inv, nz);
    } else if (at < 0 && !bad && now > old[i]) {  // an earlier row: its codes follow the scale
      const float ratio = __fmul_rn(old[i], inv);
      const uint4 w = *reinterpret_cast<const uint4*>(codes + 16 * u);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = kv8_decode<E4M3>(static_cast<uint8_t>(ww[j / 4] >> (8 * (j % 4))));
      const uint2 y = quantise8<E4M3>(x, ratio, nz), z = quantise8<E4M3>(x + 8, ratio, nz);
      *reinterpret_cast<uint4*>(codes + 16 * u) = make_uint4(y.x, y.y, z.x, z.y);
    }
    if (threadIdx.x == 0) a.scales[cell] = bad ? __uint_as_float(0x7fc00000u) : now;
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
  p.neg_zero = -0.0f;
  p.blocks_per_seq = static_cast<int>((static_cast<int64_t>(a.max_new) + sh.block_tokens - 2) / sh.block_tokens + 1);
  const int threads = sh.block_tokens * sh.head_dim / 16;
  const int batch = sh.dtype == DKV_F32 ? kAppendHeads<float> : kAppendHeads<__nv_bfloat16>;
  const int64_t blocks = static_cast<int64_t>(a.num_seqs) * p.blocks_per_seq;
  p.kv_ctas = blocks * ceil_div64(p.heads, batch) * 2;
  int64_t q_ctas = 0;
  if (a.q) {
    const int per = threads / (sh.head_dim / 16);
    // two batches where there are tokens enough: a thread's search for its sequence and its angles serve more heads
    p.q_head_steps = a.total_new * p.q_heads * sh.head_dim / 16 >= int64_t{16} * 1024 * num_sms() ? 2 * batch : batch;
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
